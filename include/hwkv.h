/*
 * hwkv -- per-head budgeted KV residency on one GB300 (sm_103a).
 *
 * C ABI of the grouped-cache runtime described in "HeadWiseKV: Budgeted Per-Head Cache
 * Residency for Hybrid Long-Context Language Models" (blog summary):
 *
 *   - abstract: every physical KV head of a residual global-attention layer gets a static
 *     history window w; the runtime MATERIALISES that residency (it keeps only the window)
 *     instead of masking a full cache, so the cache footprint is exact before serving;
 *   - section "Grouped-Cache Runtime": a paged block table gives each head
 *     ceil(w / block_size) KV blocks, pre-allocated before serving.
 *
 * Terms used below
 *   L  layers (global-attention layers only), H kv heads, Hq query heads (Hq = G * H),
 *   D  head_dim, bs block_size, B num_seqs, eb element bytes (4 for F32, 2 for BF16).
 *   nblk[l][h] = ceil(w[l][h] / bs);  ring capacity C[l][h] = nblk[l][h] * bs tokens.
 *   Token position p of (seq, layer, head) lives in ring slot p mod C; slot t is row
 *   t mod bs of logical block t / bs, which the block table maps to a physical block.
 *   A physical block is [2][bs][D] elements: bs K rows, then bs V rows (2*bs*D*eb bytes).
 *   Query head q reads kv head q / G (consecutive groups).
 *   Decode attention at length len covers positions [max(0, len - w), len): the last
 *   min(w, len) tokens, including the one appended in the same step.
 *
 * 8-bit pools (HWKV_E4M3)
 *   Blocks hold e4m3 codes (eb = 1), and bs % 16 == 0.  The pool buffer continues after the
 *   blocks with fp32 scales [total_blocks][bs / 16][2]: one for the K rows and one for the V rows
 *   of each group of 16 consecutive slots; a stored value is code * scale.  The scale is 2^e with
 *   the smallest e >= -120 such that the group's largest finite magnitude is at most 448 * 2^e;
 *   codes are rounded to nearest even (a magnitude of 248 * 2^120, 3.3e38, or more is stored as
 *   2^128, which a bf16 result shows as infinity); what is not finite is stored as NaN.
 *   Storing a token stores its whole group anew: the slots of the group whose positions are in
 *   the window of the new length keep their values at the new scale (rounded again where a code
 *   becomes subnormal), every other slot becomes zero.  Materialise does so with every group
 *   that holds a resident position.  Slots outside the window never reach a result, whatever
 *   they hold.
 *
 * Conventions
 *   - Every function returns an int status (HWKV_OK or a negative HWKV_ERR_*); on error
 *     hwkv_last_error() (thread-local) describes it.  Argument errors are reported before
 *     anything is launched.
 *   - Pointers named *_dev and every tensor argument are DEVICE pointers on the current
 *     CUDA device; the caller owns them (e.g. torch tensors).  `stream` is a cudaStream_t
 *     (NULL = legacy default stream).  Calls that take a stream are asynchronous on it.
 *   - Lengths and positions live on the device so that a captured CUDA graph stays valid
 *     across decode steps; kernels check them and record problems in a device error word
 *     that hwkv_check_device_errors() reads.  Kernels never trap or spin without bound.
 *   - Inputs must be finite: a masked pool row that holds Inf/NaN bits can still poison
 *     a result (0 * Inf), as in any attention kernel (not so in 8-bit pools).  Weighted sums are
 *     held in fp32 relative to the largest weight: the sum of |value| over keys of like weight
 *     must stay below 2^128.
 */
#ifndef HWKV_H
#define HWKV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HWKV_ABI_VERSION 3

/* status codes */
#define HWKV_OK 0
#define HWKV_ERR_INVALID_ARG (-1)
#define HWKV_ERR_ALIGNMENT (-2)
#define HWKV_ERR_POOL_TOO_SMALL (-3)
#define HWKV_ERR_CUDA (-4)
#define HWKV_ERR_DEVICE_CHECK (-5)
#define HWKV_ERR_UNSUPPORTED (-6)
#define HWKV_ERR_WORKSPACE_TOO_SMALL (-7)
#define HWKV_ERR_BUDGET (-8)

/* element types of the pool and of every tensor passed with it; HWKV_E4M3 pools hold 8-bit codes
 * and take and return BF16 tensors */
#define HWKV_F32 0
#define HWKV_BF16 1
#define HWKV_E4M3 2

/* decode kernel selection for hwkv_set_decode_config */
#define HWKV_KERNEL_AUTO 0   /* stream-K kernel where supported, else the split kernel       */
#define HWKV_KERNEL_TENSOR 1 /* stream-K kernel: tensor cores for bf16 and 8 bit, CUDA cores for fp32
                                (fp32: up to 4 query heads per KV head); bs % 16 == 0 only  */
#define HWKV_KERNEL_SIMT 2   /* split-K CUDA-core kernel, any supported shape but 8-bit pools  */

/* bits of the device error word */
#define HWKV_DEVERR_NEG_LENGTH 1     /* a length / position below 0                    */
#define HWKV_DEVERR_BAD_BLOCK 2      /* a block-table entry outside the pool            */
#define HWKV_DEVERR_SRC_RANGE 4      /* materialise length above max_len               */
#define HWKV_DEVERR_WAIT_TIMEOUT 8   /* a pipeline wait gave up (work was skipped)      */
#define HWKV_DEVERR_BAD_PREFIX 16    /* a sequence's prefix that the prefix pool does not hold */

typedef struct hwkv_pool* hwkv_pool_t;

/* ABI / layout version (kernel-ABI compatibility check of the cache layout).  Returns
 * HWKV_ABI_VERSION of the loaded library. */
int hwkv_abi_version(void);

/* Thread-local description of the last error on this thread ("" if none). */
const char* hwkv_last_error(void);

/* Short constant name of a status code. */
const char* hwkv_status_string(int status);

/* Pre-serving footprint prediction ("Grouped-Cache Runtime": ceil(w / bs) blocks per head;
 * abstract: demand known exactly before serving).  Pure host, needs no GPU.
 *   windows: host int32 [layers][kv_heads], each >= 1.
 *   out_bytes = num_seqs * sum_{l,h} ceil(w[l][h]/bs) * bs * head_dim * 2 * eb,
 *   for HWKV_E4M3 plus the scales: 8 bytes per 16 slots, their sum rounded up to 16 bytes.
 * Supported: 1 <= kv_heads <= 32, head_dim in {64, 128}, block_size >= 1 (E4M3: a multiple of
 * 16), dtype F32/BF16/E4M3, every ring capacity below 2^31 tokens and at most 2^31 - 1 blocks in
 * total.
 * Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_UNSUPPORTED. */
int hwkv_pool_bytes(int layers, int kv_heads, int head_dim, int block_size, const int32_t* windows,
                    int num_seqs, int dtype, uint64_t* out_bytes);

/* Binds a caller-owned device buffer as the per-head paged pool ("Grouped-Cache Runtime").
 *   dev_pool: device pointer, 256-byte aligned, dev_pool_bytes >= hwkv_pool_bytes().
 *   The pool is zero-filled on `stream`.  The block table starts as the identity map with
 *   physical ids handed out in (layer, seq, kv head, logical block) order.
 *   The library allocates its own small device metadata (block table, error word) and
 *   frees it in hwkv_pool_destroy; the pool buffer itself is never freed by the library.
 *   Synchronises `stream` before returning.
 * Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_UNSUPPORTED, HWKV_ERR_ALIGNMENT (pool pointer),
 *         HWKV_ERR_POOL_TOO_SMALL (checked before anything is written), HWKV_ERR_CUDA. */
int hwkv_pool_create(int layers, int kv_heads, int head_dim, int block_size, const int32_t* windows,
                     int num_seqs, int dtype, void* dev_pool, uint64_t dev_pool_bytes, void* stream,
                     hwkv_pool_t* out);

/* Frees the library-owned metadata.  The caller must make sure no work using the pool is
 * still in flight.  NULL is accepted. */
int hwkv_pool_destroy(hwkv_pool_t pool);

/* Geometry of a created pool: bytes, physical block count, bytes per block (an 8-bit pool's
 * scales, total_blocks * block_bytes into the pool, are not part of a block). */
int hwkv_pool_geometry(hwkv_pool_t pool, uint64_t* pool_bytes, int64_t* total_blocks, int64_t* block_bytes);

/* Copies the physical block ids of (seq, layer, kv_head) -- nblk of them, logical block
 * order -- into host_out[0 .. cap).  *n receives nblk.  Host copy of the library's table. */
int hwkv_block_table(hwkv_pool_t pool, int seq, int layer, int kv_head, int32_t* host_out, int cap, int* n);

/* Replaces the whole block table (the cache manager above the runtime chooses physical
 * blocks).  host_table: int32 [total_blocks] in (layer, seq, kv head, logical block) order;
 * it must be a permutation of 0 .. total_blocks-1 (checked; HWKV_ERR_INVALID_ARG otherwise).
 * The pool bytes are NOT moved.  Copies on `stream` and synchronises it. */
int hwkv_set_block_table(hwkv_pool_t pool, const int32_t* host_table, int64_t n, void* stream);

/* Materialise ("Grouped-Cache Runtime", abstract): compacts one layer of a contiguous full
 * prefill KV into the pool.  For every seq s and kv head h, the last min(w, L_s) positions
 * p of the prefill are copied to ring slot p mod C (K and V rows); nothing else is written.
 *   k_full, v_full: device, element (s, h, p, d) at s*seq_stride + h*head_stride + p*D + d
 *                   (strides in elements; rows contiguous), 16-byte aligned, strides*eb
 *                   multiples of 16.
 *   max_len: rows available per (s, h) in the source; lens_dev[s] must be in [0, max_len]
 *            (checked on the device: HWKV_DEVERR_NEG_LENGTH / HWKV_DEVERR_SRC_RANGE, the
 *            sequence is skipped).
 *   lens_dev: device int32 [num_seqs] prefill lengths L_s.
 * max_len == 0 is an empty prefill: nothing is read or written and the pointers may be NULL.
 * 8-bit pools take a bf16 source and store whole groups (see above). */
int hwkv_materialize(hwkv_pool_t pool, int layer, const void* k_full, const void* v_full,
                     int64_t seq_stride, int64_t head_stride, int64_t max_len, const int32_t* lens_dev,
                     void* stream);

/* Append: writes the new token of every (seq, kv head) of one layer into its ring slot
 * pos mod C (the slot of the oldest token, which has just left the window when C == w).
 *   k_new, v_new: device [num_seqs][kv_heads][D], 16-byte aligned.
 *   pos_dev: device int32 [num_seqs], the length BEFORE the append (position of the new
 *            token); negative values are flagged (HWKV_DEVERR_NEG_LENGTH) and skipped. */
int hwkv_append(hwkv_pool_t pool, int layer, const void* k_new, const void* v_new, const int32_t* pos_dev,
                void* stream);

/* Position bookkeeping of a serving loop, on the device: out_dev[s] = pos_dev[s] + delta for the
 * pool's num_seqs sequences (int32, wrapping; out_dev may be pos_dev).  It lets a decode step
 * captured in a CUDA graph advance its positions after the step (delta 1), or form the lengths
 * after the append from the positions before it, without a kernel from outside this library.
 * The pages have no counterpart: this is a service of this library, not a step of the method.
 *   pos_dev, out_dev: device int32 [num_seqs], 4-byte aligned.  One kernel on `stream`. */
int hwkv_advance_positions(hwkv_pool_t pool, const int32_t* pos_dev, int32_t* out_dev, int32_t delta, void* stream);

/* Check of the bounded waits (a service of this library; the pages have no counterpart).
 * Every wait of every kernel here gives up after a time limit (~2 s) and records
 * HWKV_DEVERR_WAIT_TIMEOUT in the error word instead of spinning forever.  This runs that same
 * wait loop on its own, in one warp, so a host can see the path work without faulting or
 * hanging a GPU: first on an mbarrier phase that has completed, then on one that nothing will
 * complete, given up after limit_us microseconds.
 *   out_dev: device int32 [3], 4-byte aligned, written by the kernel: [0] the error bits it
 *            recorded (HWKV_DEVERR_WAIT_TIMEOUT when the second wait gave up), [1] 1 when the
 *            first wait returned true, [2] the microseconds the second wait took.
 *   limit_us: 1 .. 2 000 000 (HWKV_ERR_INVALID_ARG otherwise).
 * One kernel on `stream`, on the current device; HWKV_ERR_CUDA if it cannot be launched. */
int hwkv_wait_selftest(uint32_t limit_us, int32_t* out_dev, void* stream);

/* Bytes of scratch hwkv_decode_attn / hwkv_append_decode_attn need for the current decode
 * configuration (fp32 split-K partials; maximum over layers). */
int hwkv_decode_workspace_bytes(hwkv_pool_t pool, int q_heads, uint64_t* out);

/* Split-K decode attention over the resident window of one layer (abstract: attention reads
 * the materialised window, never a masked full cache).  For query head q of seq s, with
 * h = q / G and w = w[layer][h]:
 *     out[s][q] = sum_{p in [max(0,len_s-w), len_s)} softmax_p(scale * <q, k_p>) v_p
 * computed with fp32 accumulation and an online softmax; out has the pool's dtype.
 *   q, out: device [num_seqs][q_heads][D], 16-byte aligned; q_heads = G * kv_heads, G <= 16
 *           (the stream-K kernel pads the group to 4, 8 or 16 query-head columns on the
 *           tensor cores for bf16 pools, to 4 on the CUDA cores for fp32 pools).
 *   lens_dev: device int32 [num_seqs], lengths AFTER this step's append.  len 0 gives 0s.
 *   workspace: device scratch of >= hwkv_decode_workspace_bytes(), 16-byte aligned; its
 *              contents need no initialisation and are clobbered.  Launches that may run
 *              at the same time need distinct workspaces.
 * The stream-K kernel splits the layer's resident tiles evenly over a persistent grid and
 * merges partial results through per-(seq, head) arrival counters that the library keeps in
 * its own device memory (one set per layer); concurrent launches of the SAME layer race.
 * Other shapes (block_size not a multiple of 16, fp32 groups above 4) take the split-K
 * CUDA-core kernel and a merge kernel.  8-bit pools always take the stream-K kernel, on the
 * tensor cores; q, k_new, v_new and out are bf16.
 *   8-bit pools: a softmax weight times its group's V scale is rounded to 11 bits down to 2^-25 of
 *   the largest such product of its query head, and is off by at most 2^-36 of that product below.
 * Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_ALIGNMENT, HWKV_ERR_WORKSPACE_TOO_SMALL,
 *         HWKV_ERR_UNSUPPORTED, HWKV_ERR_CUDA (launch failure). */
int hwkv_decode_attn(hwkv_pool_t pool, int layer, const void* q, int q_heads, float scale,
                     const int32_t* lens_dev, void* out, void* workspace, uint64_t workspace_bytes,
                     void* stream);

/* One decode step of one layer: hwkv_append followed by hwkv_decode_attn, with the same
 * results.  pos_dev holds the lengths BEFORE the append; attention runs at pos + 1.  On the
 * tensor-core path this is a single kernel: the CTA that streams the tile holding the new
 * token's slot takes the new rows from k_new / v_new and also writes them into the pool. */
int hwkv_append_decode_attn(hwkv_pool_t pool, int layer, const void* q, int q_heads, float scale,
                            const void* k_new, const void* v_new, const int32_t* pos_dev, void* out,
                            void* workspace, uint64_t workspace_bytes, void* stream);

/* Flags of hwkv_decode_attn_ex. */
#define HWKV_DECODE_EARLY_READS 1

/* hwkv_decode_attn (k_new = v_new = NULL; lens_dev = lengths after the append) or
 * hwkv_append_decode_attn (k_new, v_new given; lens_dev = positions before the append), with
 * flags:
 *   HWKV_DECODE_EARLY_READS  the caller guarantees that lens_dev, the block table and this
 *     layer's pool were last written by work that completed before the kernel that immediately
 *     precedes this call in `stream` started (e.g. lengths set once per step before layer 0,
 *     and a previous layer's attention just before).  The tensor-core kernel then computes its
 *     schedule and issues its first K/V loads while that kernel is still finishing (it is
 *     launched as a programmatic dependent), and waits for it only before it reads q, k_new,
 *     v_new or writes anything.  Same results as without the flag.  Do not set it on the call
 *     that follows the kernel which updates the lengths.  Ignored by the CUDA-core kernel.
 * Errors as hwkv_decode_attn; HWKV_ERR_INVALID_ARG for unknown flags. */
int hwkv_decode_attn_ex(hwkv_pool_t pool, int layer, const void* q, int q_heads, float scale, const void* k_new,
                        const void* v_new, const int32_t* lens_dev, void* out, void* workspace,
                        uint64_t workspace_bytes, int flags, void* stream);

/* A score that is more than scale * <q, k>: capped, then lowered with the distance of the key,
 *     s = scale * <q, k>;  if softcap > 0: s = softcap * tanh(s / softcap);
 *     s = s - slope[query head] * (position of the query - position of the key).
 * In a decode step the query's position is len - 1, so the newest token's distance is 0.
 *   softcap: finite, 0 (none) or positive, with scale / softcap and softcap * log2(e) finite in
 *            fp32;  slopes_dev: device float [q_heads] or NULL (none), finite, as must be
 *            slope * log2(e) * distance in fp32 for every distance within a window or chunk. */
typedef struct hwkv_score {
  float scale;
  float softcap;
  const float* slopes_dev;
} hwkv_score_t;

/* hwkv_decode_attn_ex with such a score, for every pool type and shape; the same workspace, flags
 * and errors.  The cap is off by at most 2^-20 of the capped score, the difference with the bias by
 * a few fp32 roundings of the larger term (fp32 pools: the cap likewise).  8-bit decode and chunked
 * prefill take longer where scores pass the cap, or where scale * (scale / softcap)^10 is below fp32's normal
 * range (caps from about 250 at scale 128^-1/2).  A score with neither cap nor slopes runs the plain kernels. */
int hwkv_decode_attn_score(hwkv_pool_t pool, int layer, const void* q, int q_heads, const hwkv_score_t* score,
                           const void* k_new, const void* v_new, const int32_t* lens_dev, void* out, void* workspace,
                           uint64_t workspace_bytes, int flags, void* stream);

/* Decode behind shared prefixes: sequences whose contexts begin with the same tokens keep those once, in a
 * pool of prefixes (its sequences), and only what follows in their own pool, at positions counted from 0
 * behind the prefix.  For query head q of sequence s with own length L (after the append), behind prefix f of N tokens,
 * with w' the own pool's and w the prefix pool's window of the head:
 *     out[s][q] = softmax over the own positions [max(0, L - w'), L) and the prefix's [max(0, N + L - w), N),
 * so that own windows w' >= min(w, the longest own part) give the last w tokens of the whole context.  Each
 * prefix's keys are read once for all the sequences behind it.
 *   prefix: a pool of the same layers, kv_heads and head_dim, whose tensors have the same type (an 8-bit pool goes with a
 *   bf16 or an 8-bit one); blocks and windows may differ.  Its sequences hold the prefixes, stored by any call.
 *   prefix_of_dev: device int32 [num_seqs], the prefix of each sequence, negative for none; one past the
 *   prefix pool's sequences flags HWKV_DEVERR_BAD_PREFIX and counts as none.  prefix_lens_dev: device int32
 *   [prefix num_seqs], tokens of each prefix (negative: HWKV_DEVERR_NEG_LENGTH, counts as 0).  What is flagged is
 *   recorded in `pool`.
 *   k_new, v_new (both or neither): appended to the own pool first, lens_dev then holding the own lengths before the
 *   append, as in hwkv_decode_attn_ex.  score: as hwkv_decode_attn_score (a prefix key's distance counts the
 *   tokens of both pools; its bias is off by a few fp32 roundings of slope * (distance + 64), and slope * log2(e) *
 *   distance must be finite up to 64 tokens past the prefix pool's window; scale * <q, k> must stay below 2^26 in
 *   magnitude for prefixes in bf16 and 8-bit pools);
 *   nothing to attend to gives zeros.  Weights of a prefix's keys are rounded to bf16 (2^-8 of each) before they multiply
 *   its values, in bf16 and 8-bit prefix pools alike (an 8-bit decode rounds its own to fp16, 2^-11); those of fp32 pools, and of
 *   bf16 pools with block_size % 16 != 0, are not.  Stored keys and values must be finite, as for every call (and below
 *   2^128 in 8-bit pools): the prefix's are operands of products over all sequences behind it.
 *   workspace: hwkv_decode_shared_workspace_bytes() bytes, otherwise as for hwkv_decode_attn.
 * Three kernels on `stream` or more: the prefixes' keys, the own parts, their join.  Concurrent launches of the same
 * layer of `pool` race, decode calls included; `prefix` may be shared by any number of launches that only read it.
 * At most 65535 sequences and 768 prefixes; a group of up to 16 query heads per KV head, as in every decode.
 * Errors: as hwkv_decode_attn; HWKV_ERR_INVALID_ARG also for pools that do not go together. */
int hwkv_decode_attn_shared(hwkv_pool_t pool, hwkv_pool_t prefix, int layer, const void* q, int q_heads,
                            const hwkv_score_t* score, const void* k_new, const void* v_new, const int32_t* lens_dev,
                            const int32_t* prefix_of_dev, const int32_t* prefix_lens_dev, void* out, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Bytes of workspace hwkv_decode_attn_shared needs, the most over the layers (host only). */
int hwkv_decode_shared_workspace_bytes(hwkv_pool_t pool, hwkv_pool_t prefix, int q_heads, uint64_t* out);

/* Bytes of the static scratch array behind hwkv_decode_attn_noalloc. */
#define HWKV_NOALLOC_SCRATCH_BYTES (4u << 20)

/* hwkv_decode_attn without a workspace argument, for callers that cannot allocate device
 * memory where they run attention (during CUDA graph capture, under an allocator that owns
 * all device memory, inside hosts that forbid allocation after start-up).  The pages have
 * no counterpart: this is a service of this library, not a step of the method.
 *   Results are those of hwkv_decode_attn with the same arguments, bit for bit.  The split-K
 *   scratch is a fixed array of HWKV_NOALLOC_SCRATCH_BYTES (4 MiB) inside the library; the
 *   call allocates nothing (no cudaMalloc / cudaFree, no allocating library routine).
 *   A configuration whose scratch (hwkv_decode_workspace_bytes) exceeds the array is
 *   rejected with HWKV_ERR_WORKSPACE_TOO_SMALL before anything is launched.
 *   The pool's device must be current (HWKV_ERR_INVALID_ARG otherwise).  The first call on a
 *   device looks up the array's device address there; under CUDA's default lazy module
 *   loading that lookup also loads the module holding the array and commits its 4 MiB on
 *   that device, which then stay committed until the process exits.  Make that first call
 *   before any stream capture.
 *   All calls share the one array and it keeps the last call's contents; nothing in it has
 *   to start at zero.  Calls whose kernels overlap on the GPU (other streams, other threads)
 *   race on the array: serialise them. */
int hwkv_decode_attn_noalloc(hwkv_pool_t pool, int layer, const void* q, int q_heads, float scale,
                             const int32_t* lens_dev, void* out, void* stream);

/* Chunked prefill of one layer ("Grouped-Cache Runtime": every head keeps only its window):
 * for each sequence s, a chunk of n_s new tokens at positions pos_s .. pos_s + n_s - 1 attends
 * causally, per KV head h, to the positions [max(0, p + 1 - w_h), p] of each token p -- the
 * ones before the chunk read from the head's ring in the pool, the others from the chunk --
 * and the chunk is then appended to the rings (slot p mod C; the last min(C, n_s) tokens are
 * written).  The result equals appending the tokens one by one and decoding each.
 *   q, out: device bf16 [num_seqs][n_max][q_heads][D]; k_new, v_new: [num_seqs][n_max][kv_heads][D];
 *   all 16-byte aligned.  pos_dev / n_dev: device int32 [num_seqs], lengths before the chunk
 *   and chunk lengths (0 <= n_s <= n_max, checked on the device; a bad sequence is skipped and
 *   flagged HWKV_DEVERR_NEG_LENGTH).  Rows of out at or past n_s are left untouched.
 *   workspace: device scratch of hwkv_prefill_workspace_bytes() bytes (16-byte aligned) that lets
 *   the library split long key streams over several CTAs and merge their fp32 partials; NULL or
 *   a smaller size runs one CTA per stream (same results up to rounding, slower for long windows
 *   at small batch).  Contents need no initialisation and are clobbered.
 * Needs a bf16 pool with block_size % 16 == 0 and q_heads = G * kv_heads with G <= 16
 * (HWKV_ERR_UNSUPPORTED otherwise).  Two kernels on `stream`: the attention, then the merge of
 * split streams together with the append. */
int hwkv_prefill_attn(hwkv_pool_t pool, int layer, const void* q, int q_heads, float scale, const void* k_new,
                      const void* v_new, int n_max, const int32_t* pos_dev, const int32_t* n_dev, void* out,
                      void* workspace, uint64_t workspace_bytes, void* stream);

/* hwkv_prefill_attn with a capped or distance-biased score (see hwkv_score_t; a query's position
 * is that of its token).  The bias adds a few fp32 roundings of 64 slopes to a score's error, and a slope
 * beyond +-2^17 / log2(e) (9.08e4) counts as that, which no result shows while the scores of neighbouring
 * keys differ by less. */
int hwkv_prefill_attn_score(hwkv_pool_t pool, int layer, const void* q, int q_heads, const hwkv_score_t* score,
                            const void* k_new, const void* v_new, int n_max, const int32_t* pos_dev,
                            const int32_t* n_dev, void* out, void* workspace, uint64_t workspace_bytes, void* stream);

/* Bytes of workspace hwkv_prefill_attn uses to split the key streams of `layer` for chunks of up
 * to n_max tokens and q_heads query heads (0 when nothing would be split).  Host only; depends on
 * the geometry, the GPU's SM count and hwkv_set_prefill_config. */
int hwkv_prefill_workspace_bytes(hwkv_pool_t pool, int layer, int q_heads, int n_max, uint64_t* out);

/* The launch plan hwkv_prefill_attn uses for `layer` (host only: no pool, no device).  The
 * geometry arguments are those of hwkv_pool_create (bf16); num_sms is the GPU's SM count and
 * max_stages the cap of hwkv_set_prefill_config (0 = automatic).  For launch position
 * i < kv_heads: head_order[i] is the KV head, splits[i] its CTAs per (sequence, query-tile pair)
 * and split_stages[i] the 64-key stages each of them streams (CTA k of a split stream takes
 * stages [k * split_stages[i], (k + 1) * split_stages[i]) of it, so splits[i] * split_stages[i]
 * covers the longest stream of the head).  *workspace_bytes is what hwkv_prefill_workspace_bytes
 * returns for a pool of this geometry on such a GPU (0 when nothing is split).  The arrays hold
 * kv_heads entries each and are caller-owned.  Errors as hwkv_pool_bytes and
 * hwkv_prefill_attn's argument checks. */
int hwkv_prefill_plan(int layers, int kv_heads, int head_dim, int block_size, const int32_t* windows, int num_seqs,
                      int layer, int q_heads, int n_max, int num_sms, int max_stages, int32_t* head_order,
                      int32_t* splits, int32_t* split_stages, uint64_t* workspace_bytes);

/* Prefill configuration: max_stages caps the 64-key stages one CTA streams before its stream is
 * split, the same cap for every head (0 = automatic: a cap of about three waves of one CTA per
 * SM, then, for launches of at most 2048 unsplit CTAs, split counts refined per head against a
 * time model of the launch, planned once per (layer, q_heads, n_max) and kept).  Results differ
 * only by rounding. */
int hwkv_set_prefill_config(hwkv_pool_t pool, int max_stages);

/* Decode configuration.  kernel = HWKV_KERNEL_*.  split_tokens: tokens of one split-K chunk of
 * the CUDA-core kernel (0 = automatic; else a power of two in [16, 65536]).  workers: CTAs of
 * the tensor-core kernel's persistent grid (0 = automatic: every SM, as many CTAs as fit; 95% of
 * that when a layer's ring capacity is under 128 16-token tiles per CTA, so the next launch's
 * first CTAs find free slots).
 * Changes the workspace size.  Results differ between configurations only by rounding.  Graphs captured
 * before keep their configuration, their workspace and the library's counters. */
int hwkv_set_decode_config(hwkv_pool_t pool, int split_tokens, int workers, int kernel);

/* Rotary positions: before a key is appended and a query attends, the pairs of their rows turn
 * with the position.  (The pages store keys after this step and leave it to the caller.)  Pair i
 * of a row at position p, (a, b), becomes
 *     magnitude * (a cos t - b sin t, b cos t + a sin t),   t = p * freq[i],
 * in fp32, with the angle exact to 2^-23 rad at every position (|freq| < 2^40), rounded once. */
#define HWKV_ROPE_HALF 0         /* pairs (i, i + rot_dim / 2)                                   */
#define HWKV_ROPE_INTERLEAVED 1  /* pairs (2 i, 2 i + 1)                                         */
typedef struct hwkv_rope {
  int32_t rot_dim;   /* the first rot_dim dims of a head turn (even, 2 .. head_dim), others pass  */
  int32_t layout;    /* HWKV_ROPE_*                                                              */
  double magnitude;  /* factor on the turned dims                                                */
  double freq[64];   /* radians per position of pair i < rot_dim / 2                             */
} hwkv_rope_t;

/* Fills a table: freq[i] = base^(-2 i / rot_dim), magnitude 1, then for longer contexts
 *   HWKV_ROPE_SCALE_NONE
 *   HWKV_ROPE_SCALE_LINEAR    every freq divided by factor;
 *   HWKV_ROPE_SCALE_NTK       base * factor^(rot_dim / (rot_dim - 2)) in place of base (no change
 *                             for rot_dim 2, whose one freq is 1);
 *   HWKV_ROPE_SCALE_BY_PARTS  a pair that makes r turns over original_len positions keeps the
 *                             share c = clamp((r - beta_slow) / (beta_fast - beta_slow), 0, 1):
 *                             freq = c freq + (1 - c) freq / factor; magnitude 0.1 ln(factor) + 1.
 *                             (Over turns.  A ramp over the pair's index between two rounded bounds, as many
 *                             configurations compute it, has other frequencies: up to 1.7 times these at
 *                             rot_dim 128, base 1e6, 32768 and factor 4, 3.0 times at base 1e4, 4096 and
 *                             16; and a ramp over turns may go with magnitude 1.  Such a caller sets
 *                             freq and magnitude.)
 * factor >= 1 and finite; original_len > 0 and beta_fast > beta_slow for BY_PARTS (ignored
 * otherwise); base > 0 and finite.  Host only.  Errors: HWKV_ERR_INVALID_ARG.  A caller may also
 * fill the struct itself. */
#define HWKV_ROPE_SCALE_NONE 0
#define HWKV_ROPE_SCALE_LINEAR 1
#define HWKV_ROPE_SCALE_NTK 2
#define HWKV_ROPE_SCALE_BY_PARTS 3
int hwkv_rope_table(int rot_dim, int layout, double base, int scaling, double factor, double original_len,
                    double beta_fast, double beta_slow, hwkv_rope_t* out);

/* Rows of a chunk: element (seq s, row i, head, d) at s * seq_stride + i * row_stride + head * D + d
 * (strides in elements, 0 allowed where that index takes one value), so the query and key heads of
 * a fused projection's output need no copy.  16-byte aligned, strides multiples of 16 bytes. */
typedef struct hwkv_rows {
  void* data;
  int64_t seq_stride;
  int64_t row_stride;
} hwkv_rows_t;

/* Turns the queries and keys of a chunk: row i of sequence s, at position pos_dev[s] + i, for
 * 0 <= i < n_dev[s] (n_dev NULL: all n_max rows).  Rows at or past n_s are not touched.  Tensors
 * are of the pool's type (bf16 for 8-bit pools), with q_heads query and the pool's kv_heads key
 * heads; q with q_out, or k with k_out, may be NULL.  An output may be its input (same pointer and
 * strides); outputs must not overlap anything else.
 *   pos_dev, n_dev: device int32 [num_seqs]; a negative position or n_s outside [0, n_max] flags
 *   HWKV_DEVERR_NEG_LENGTH and skips the sequence.
 * One kernel on `stream`.  A decode call with HWKV_DECODE_EARLY_READS may follow it: it writes
 * neither lengths nor pool.
 * Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_ALIGNMENT, HWKV_ERR_UNSUPPORTED, HWKV_ERR_CUDA. */
int hwkv_rope(hwkv_pool_t pool, const hwkv_rope_t* rope, const hwkv_rows_t* q, int q_heads, const hwkv_rows_t* k,
              int n_max, const int32_t* pos_dev, const int32_t* n_dev, const hwkv_rows_t* q_out,
              const hwkv_rows_t* k_out, void* stream);

/* Rotary positions on the way into the pool: one call turns the queries and keys of a chunk (or of one token, n_max 1)
 * and stores the turned keys and the values in one layer.  Row i of sequence s, 0 <= i < n_s, is token pos_s + i of the
 * sequence: its slot is (pos_s + i) mod C, and its query and key turn by position turn_pos_s + i (turn_pos_dev
 * NULL: pos_s + i; a prefix kept in a pool of its own puts the two apart).  The last min(C, n_s) rows are written, as
 * hwkv_prefill_attn does; it is the append of any pool type for a chunk that is attended elsewhere.
 *   rope: as hwkv_rope, or NULL: nothing turns.  q with q_out, or neither; k_out (the turned keys, rows below
 *   n_s, beside those stored) or NULL.  q_out may be q; k_out may be k, but not for 8-bit pools; outputs
 *   must not overlap anything else.  q_heads is a multiple of kv_heads.  Strides as in hwkv_rows_t.
 *   pos_dev, turn_pos_dev, n_dev: device int32 [num_seqs]; a negative position, one that reaches 2^31, or n_s outside
 *   [0, n_max] flags HWKV_DEVERR_NEG_LENGTH and skips the sequence.  n_dev NULL: all n_max rows.
 * Cosines and sines are fp32 of angles as exact as hwkv_rope's (queries, bf16 and fp32 keys 2^-23; keys of 8-bit pools and
 * the queries beside them 2^-26).
 * bf16 and fp32 pools hold what hwkv_rope and then hwkv_append of each row in turn leave, bit for bit.  8-bit pools store every
 * group of 16 slots that a row goes to once, anew: the slots whose positions are in the window of the new length take their row,
 * rounded once from the turned fp32 value, or keep their value at the new scale; every other slot becomes zero.
 * One kernel on `stream`.  It writes the pool: the call right behind it may not have HWKV_DECODE_EARLY_READS.
 * Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_ALIGNMENT, HWKV_ERR_UNSUPPORTED, HWKV_ERR_CUDA. */
int hwkv_rope_append(hwkv_pool_t pool, int layer, const hwkv_rope_t* rope, const hwkv_rows_t* q, int q_heads,
                     const hwkv_rows_t* k, const hwkv_rows_t* v, int n_max, const int32_t* pos_dev,
                     const int32_t* turn_pos_dev, const int32_t* n_dev, const hwkv_rows_t* q_out,
                     const hwkv_rows_t* k_out, void* stream);

/* Number of kernels this library has launched in this process (all pools, all devices).
 * Lets a caller count the launches inside a timed region. */
int hwkv_kernel_launches(uint64_t* out);

/* Distortion of a candidate window vector, supplied by the caller (e.g. measured with a
 * model).  windows: [kv_heads] candidate of `layer`; chosen: [layer][kv_heads] window vectors
 * already chosen for layers 0 .. layer-1 (execution order), so the distortion may depend on
 * them.  Return the distortion; smaller is better. */
typedef double (*hwkv_distortion_fn)(void* user, int layer, const int32_t* windows, const int32_t* chosen);

/* Host-side policy search of "HeadWiseKV: Budgeted Per-Head Cache Residency for Hybrid
 * Long-Context Language Models", section "SeqCalib": layers are visited in execution order;
 * for each layer the candidate window vector of smallest distortion whose cost fits the
 * remaining budget is chosen (ties: the first such candidate), and its cost is taken off the
 * budget.  The cost of a vector is its exact pool footprint, the bytes hwkv_pool_bytes predicts:
 * num_seqs * sum_h ceil(w_h / block_size) * block_size * head_dim * 2 * eb, and an 8-bit pool's
 * scales (rounded up to 16 bytes once, for all layers together).
 *   candidates: host int32 [layers][num_candidates][kv_heads], every window >= 1.
 *   out_windows: host int32 [layers][kv_heads] (may be the windows argument of pool_create);
 *   out_choice: host int32 [layers] chosen candidate index; out_bytes: total pool bytes.
 * Pure host, needs no GPU.  Errors: HWKV_ERR_INVALID_ARG, HWKV_ERR_UNSUPPORTED, HWKV_ERR_BUDGET
 * (no candidate of some layer fits what is left of the budget; the message names the layer). */
int hwkv_seqcalib(int layers, int kv_heads, int head_dim, int block_size, int num_seqs, int dtype,
                  int num_candidates, const int32_t* candidates, hwkv_distortion_fn distortion, void* user,
                  uint64_t budget_bytes, int32_t* out_windows, int32_t* out_choice, uint64_t* out_bytes);

/* Synchronises `stream`, reads and clears the device error word.  *out_bits receives the
 * HWKV_DEVERR_* bits seen since the last call.  Returns HWKV_ERR_DEVICE_CHECK if any bit
 * was set, HWKV_OK otherwise. */
int hwkv_check_device_errors(hwkv_pool_t pool, void* stream, int32_t* out_bits);

#ifdef __cplusplus
}
#endif

#endif /* HWKV_H */
