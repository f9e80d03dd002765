// Internal declarations shared by the host side of the C ABI (hwkv_host.cpp) and the
// sm_103a kernels (hwkv_copy.cu, hwkv_decode.cu).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

struct hwkv_pool;

namespace hwkv {

constexpr int kMaxKvHeads = 32;
constexpr int kMergeBlock = 8;   // CTAs whose partials one first-level merge folds
constexpr int kMaxGroup = 16;  // query heads per KV head (GQA group)
constexpr int kGroupPads = 3;   // tensor-core decode instances: 4, 8 or 16 query-head columns

// Geometry of one layer, passed by value to every kernel of that layer.
//   table entry of (seq s, kv head h, logical block j) = tbl[tbl_base + s*tbl_seq_stride
//                                                          + nblk_prefix[h] + j]
struct LayerGeom {
  int64_t tbl_base;
  int32_t tbl_seq_stride;                 // sum_h nblk[h]
  int32_t nblk_prefix[kMaxKvHeads + 1];   // prefix sums of nblk over heads
  int32_t window[kMaxKvHeads];            // static window w per head
};

struct PoolView {
  void* pool;              // physical blocks [total_blocks][2][bs][D]
  const int32_t* tbl;      // flat block table
  int32_t* err;            // device error word
  int64_t total_blocks;
  int32_t block_size;
  int32_t head_dim;
  int32_t kv_heads;
  int32_t num_seqs;
  int32_t elem_bytes;      // 4 (f32), 2 (bf16) or 1 (e4m3)
  float* scales;           // e4m3: [total_blocks][bs / 16][2] scales of K and V, after the blocks; else null
};

struct CopyArgs {
  PoolView pv;
  LayerGeom g;
  const void* k;           // materialise: full prefill; append: new token rows
  const void* v;
  int64_t seq_stride;      // elements (materialise only)
  int64_t head_stride;     // elements (materialise only)
  int64_t max_len;         // rows per (s, h) in the source (materialise only)
  const int32_t* lens;     // materialise: prefill lengths; append: positions
  int32_t rows_per_cta;    // materialise only
};

// tanh(u) = u * (kTanh0 + kTanh1 u^2 + ... + kTanh5 u^10) for |u| <= 1: the polynomial of degree 5 in
// u^2 whose largest relative error on [0, 1] is smallest (found by linear programming on 4001
// Chebyshev points: 2^-20.7; 2^-20.4 with fp32 steps).
constexpr float kTanh0 = 0.9999994039535522f, kTanh1 = -0.3332904279232025f, kTanh2 = 0.13281433284282684f;
constexpr float kTanh3 = -0.05160565674304962f, kTanh4 = 0.016743095591664314f, kTanh5 = -0.0030670526903122663f;

// The same for |u| <= 1/2 with degree 3 in u^2 (2^-20.8; 2^-20.6 with fp32 steps).
constexpr float kTanhHalf0 = 0.999999463558197f, kTanhHalf1 = -0.33326318860054016f;
constexpr float kTanhHalf2 = 0.13190296292304993f, kTanhHalf3 = -0.04440220072865486f;

// What happens to a score s = scale <q, k> before the softmax: cap * tanh(s / cap) when capped,
// then less slope * (distance of the key from the query).
struct ScoreArgs {
  int32_t on;              // the scored kernel instances run
  int32_t capped;
  float cap_in;            // scale / cap
  float cap_out;           // cap * log2(e)
  // below the cap, the score in log2 units of a raw dot product x is x * (poly[0] + poly[1] x^2 + ..):
  // tanh's polynomials with the scale and 1 / cap worked in, half[] below half of the cap; poly_on:
  // their coefficients are normal fp32
  int32_t poly_on;
  float poly[6];
  float half[4];
  const float* slopes;     // [Hq] slopes, or null
};

struct DecodeArgs {
  PoolView pv;
  LayerGeom g;
  const void* q;           // [B][Hq][D]
  void* out;               // [B][Hq][D]
  const int32_t* lens;     // [B]; length after the append = lens[s] + len_add
  int32_t len_add;         // 0: lens are lengths after the append; 1: positions (fused append)
  int32_t early;           // schedule and first tile loads may run before the dependent-launch wait
  const void* k_new;       // fused append: new K / V rows [B][H][D], else null
  const void* v_new;
  float* part_acc;         // [slots][G][D]   unnormalised split accumulators
  float* part_ml;          // [slots][G][2]   (running max in log2 units, sum of weights)
  uint32_t* counters;      // [B*H] arrival counters of this layer (tensor-core kernel), all 0
  uint32_t* counters1;     // [B*H][merge_blocks] first-level arrival counters, all 0
  float* part2_acc;        // [B*H*merge_blocks][G][D] second-level partials
  float* part2_ml;         // [B*H*merge_blocks][G][2]
  int32_t merge_blocks;    // first-level merge blocks per head: ceil(CTAs / kMergeBlock) + 1
  float scale_log2;        // scale * log2(e)
  int32_t group;           // G = Hq / H
  int32_t split_tokens;    // CUDA-core kernel: tokens per split-K chunk (power of two)
  int32_t chunk_prefix[kMaxKvHeads + 1];  // CUDA-core kernel: prefix over heads of ceil(C_h / split)
  // last: among the others they cost the plain kernels 0.4% at batch 1
  int32_t bs_log2;         // 8-bit pools: log2(block_size), or -1 when it is not a power of two
  ScoreArgs score;         // capped or distance-biased scores (scored instances only)
  // open instances: every (seq, kv head) leaves its (m, l) and accumulators here instead of an output
  float* open_acc;         // [B*H][G][D]
  float* open_ml;          // [B*H][G][2]
};

// log2 of the factor that the 8-bit decode takes out of sums and accumulators alike (hwkv_decode_tile_q8.cuh)
constexpr float kQ8Shift = 5.f;

// Decode behind shared prefixes: the attention to the prefixes' keys, one partial per row and key range,
// joined with the sequences' own parts (open instances of the decode kernels).
struct SharedArgs {
  PoolView pv;             // the prefixes' pool
  LayerGeom g;
  const void* q;           // [B][Hq][D]
  void* out;               // [B][Hq][D]
  const int32_t* lens;     // [B] own lengths; length after the append = lens[s] + len_add
  int32_t len_add;
  const int32_t* prefix_of;    // [B] prefix of each sequence, below 0: none
  const int32_t* prefix_lens;  // [num_prefixes]
  int32_t num_seqs;        // B
  int32_t num_prefixes;
  int32_t group;           // G = Hq / H
  float scale_log2;
  ScoreArgs score;
  const float* own_acc;    // the open decode's results
  const float* own_ml;
  float own_shift;         // log2 of the factor that own sums and accumulators are short of
  float* part_o;           // prefix partials: unnormalised sums ...
  float* part_ml;          // ... and (reference maximum in log2 units, sum of weights) of each
  // CUDA-core kernel: key ranges of split_tokens ring slots; partial [seq][chunk of the head][G]
  int32_t split_tokens;
  int32_t seqs_per_cta;
  int32_t chunk_prefix[kMaxKvHeads + 1];
  // tensor cores: partials of (item, CTA) slots x two chains x rows, found by a record per (seq, KV head):
  // (first chain of a slot, step, number, first row)
  int32_t tc;              // 1: that kernel's partials
  int32_t bs_log2;         // log2(block_size), or -1 when it is not a power of two
  int32_t stage_tb;        // rows of one block in a 64-key pool copy (16, 32, 64), 0: per-tile copies only
  int32_t chain_rows;      // rows of a chain's partial
  int32_t slots;           // slots of partials
  int32_t stage_ns;        // time of a stage
  int32_t own_ctas;        // CTAs of the own parts' kernel (0: it does not run beside), those an SM holds, a CTA's time and that per tile
  int32_t own_per_sm;
  int32_t own_base_ns;
  int32_t own_tile_ns;
  int32_t own_window[kMaxKvHeads];
  int4* rec;
};

struct PrefillArgs {
  PoolView pv;
  LayerGeom g;
  const void* q;           // [B][n_max][Hq][D]
  const void* k_new;       // [B][n_max][H][D] chunk keys / values
  const void* v_new;
  void* out;               // [B][n_max][Hq][D]
  const int32_t* pos0;     // [B] lengths before the chunk
  const int32_t* nlen;     // [B] chunk lengths (<= n_max)
  int32_t n_max;
  int32_t group;           // G = Hq / H
  int32_t q_tiles;         // query-tile pairs per (seq, head): ceil(n_max / chunk tokens per pair)
  float scale_log2;
  ScoreArgs score;         // capped or distance-biased scores (the scored instance only)
  int32_t bs_log2;         // log2(block_size), or -1 when it is not a power of two
  int32_t stage_tb;        // rows of one block in a 64-key pool copy (16, 32, 64), 0: per-tile copies only
  int32_t head_order[kMaxKvHeads];  // heads in work order (longest CTAs first)
  // split of long key streams: head order position i has splits[i] CTAs per (seq, tile pair),
  // each streaming split_stages[i] stages; its CTAs are [head_ctas[i], head_ctas[i + 1])
  int32_t splits[kMaxKvHeads];
  int32_t split_stages[kMaxKvHeads];
  int32_t head_ctas[kMaxKvHeads + 1];
  float* part_o;           // [CTA][256 rows][D] unnormalised partial outputs of split streams
  float* part_ml;          // [CTA][256 rows][2] (reference maximum in log2 units, sum)
};

struct RopeTensor {
  void* data;              // element (s, i, head, d) at s * seq_stride + i * row_stride + head * D + d
  int64_t seq_stride;      // elements
  int64_t row_stride;
};

struct RopeArgs {
  RopeTensor q, k, q_out, k_out;
  const int32_t* pos;      // [B] position of row 0
  const int32_t* n;        // [B] rows, null: n_max
  int32_t* err;            // device error word
  int32_t num_seqs, n_max;
  int32_t q_heads, k_heads;  // 0: that tensor is not given
  int32_t head_dim, rot;   // the first rot dims of a row turn
  int32_t copy;            // 1: the other dims are written too (not in place)
  int32_t rows;            // rows of one CTA (set by launch_rope)
  float magnitude;
  uint64_t turns[64];      // turns per position of each pair, times 2^64
};

// Rotary positions on the way into the pool: the heads of a row are the q_heads turned to q_out, the
// k_heads turned and stored, and as many value heads stored as they are.
struct RopeAppendArgs : RopeArgs {
  PoolView pv;
  LayerGeom g;
  RopeTensor v;
  const int32_t* turn_pos;  // [B] position whose angle row 0 turns by, null: pos
  int32_t keys_out;         // 1: k_out receives the turned keys too
  int32_t q_parts;          // 8-bit pools: CTAs that share the query rows of a tile (set by launch_rope_append_q8)
};

// Counts every kernel launch the library makes (read by hwkv_kernel_launches).
void count_launches(uint64_t n);

// Records a message for hwkv_last_error() on this thread and returns `code`.
int set_error(int code, const char* fmt, ...);

// HWKV_OK when the pool's device is the current one, else an error (message recorded).
int check_pool_device(const struct ::hwkv_pool* p);

// Launchers.  dtype: 0 = f32, 1 = bf16 (e4m3 pools have launchers of their own).
cudaError_t launch_append(const CopyArgs& a, int dtype, cudaStream_t st);
// out[i] = in[i] + delta for i < n (in == out allowed)
cudaError_t launch_advance_positions(const int32_t* in, int32_t* out, int n, int32_t delta, cudaStream_t st);
// the bounded wait of every kernel, on a phase that completes and one that never does
cudaError_t launch_wait_selftest(int32_t* out, uint32_t limit_us, cudaStream_t st);
// max_rows: the most positions any (seq, head) of the layer copies, min(max window, max_len)
cudaError_t launch_materialize(const CopyArgs& a, int dtype, int max_rows, cudaStream_t st);
// append and materialise of e4m3 pools (hwkv_copy_q8.cu): groups of 16 slots stored at a scale each
cudaError_t launch_append_q8(const CopyArgs& a, cudaStream_t st);
cudaError_t launch_materialize_q8(const CopyArgs& a, cudaStream_t st);
// once per device before the first launch; returns resident CTAs per SM of the instances
// for 4, 8 and 16 query-head columns (fp32 pools: 4 only, the others 0)
cudaError_t configure_decode_tc(int head_dim, int dtype, int ctas_per_sm[kGroupPads]);
// stream-K kernel (tensor cores for bf16, CUDA cores for fp32 with group <= 4): `ctas`
// persistent CTAs split the resident tiles of the layer evenly
cudaError_t launch_decode_tc(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st);
// the same for e4m3 pools (hwkv_decode_q8.cu)
cudaError_t configure_decode_q8(int head_dim, int ctas_per_sm[kGroupPads]);
cudaError_t launch_decode_q8(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st);
// the same for capped or distance-biased scores, bf16 and fp32 pools (hwkv_decode_score.cu)
cudaError_t launch_decode_score(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st);
int decode_tc_group_pad(int group);  // query-head columns the kernel instance holds (4, 8 or 16)
int decode_tc_pad_index(int group);  // 0, 1, 2 for 4, 8, 16 columns
cudaError_t launch_decode_simt(const DecodeArgs& a, int dtype, int items, cudaStream_t st);
cudaError_t launch_combine(const DecodeArgs& a, int dtype, cudaStream_t st);
// open instances for a decode behind shared prefixes (hwkv_decode_open.cu; e4m3 pools hwkv_decode_open_q8.cu): results
// to a.open_acc / open_ml; they may start before the grid ahead of them ends and end after it
cudaError_t launch_decode_open(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st);
cudaError_t launch_decode_open_q8(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st);
// shared prefixes (hwkv_shared.cu): partials of the prefixes' keys, CUDA cores; and the join
int shared_simt_seqs(int group);  // sequences of one CTA
cudaError_t launch_shared_simt(const SharedArgs& a, int dtype, int chunks, cudaStream_t st);
// the same on the tensor cores (hwkv_shared_tc.cu, 8-bit pools hwkv_shared_tc_q8.cu)
constexpr int kMaxPrefixes = 768;  // what shared memory leaves room for beside 8-bit stages
int shared_tc_seqs(int group);  // sequences of a query tile
cudaError_t launch_shared_tc(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas, cudaStream_t st);
cudaError_t launch_shared_tc_q8(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas,
                                cudaStream_t st);
cudaError_t launch_shared_join(const SharedArgs& a, bool f32, cudaStream_t st);
// rotary positions (hwkv_rope.cu)
cudaError_t launch_rope(RopeArgs a, int layout, bool f32, cudaStream_t st);  // sets a.rows
// the same with keys and values stored (bf16 and fp32 pools here, e4m3 pools in hwkv_rope_q8.cu)
cudaError_t launch_rope_append(RopeAppendArgs a, int layout, bool f32, cudaStream_t st);
cudaError_t launch_rope_append_q8(RopeAppendArgs a, int layout, cudaStream_t st);
// chunked prefill (hwkv_prefill.cu): attention, then the chunk appended to the rings
int prefill_tokens_per_cta(int group);  // chunk tokens one CTA answers (two query tiles)
int prefill_tile_tokens(int group);     // chunk tokens of one 128-row query tile
// pool_map: 16-row tiles of the pool; stage_map: 64 keys of consecutive blocks (see
// hwkv_pool::stage_map); knew/vnew maps: 16-row and 64-row boxes of the chunk
cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map,
                           const CUtensorMap* knew_map, const CUtensorMap* vnew_map, const CUtensorMap* knew64_map,
                           const CUtensorMap* vnew64_map, const CUtensorMap* q_map, cudaStream_t st);
// after launch_prefill: merge of the partials of split key streams, if any, and the append of the
// chunk, at most max_rows of its rows per (seq, head)
cudaError_t launch_prefill_finish(const PrefillArgs& a, bool combine, int max_rows, cudaStream_t st);
// upper bound on the 64-key stages of one prefill CTA's key stream for a head
int prefill_max_stages(int window, int ring_capacity, int group, int n_max);
// the 64-key stages the tile pair starting at chunk row qa streams when the context before the
// chunk is longer than the ring and the chunk holds n_max rows (work estimate for planning)
int prefill_stages_estimate(int window, int ring_capacity, int group, int n_max, int qa);

}  // namespace hwkv
