// The prefixes' keys of a decode behind shared prefixes (hwkv_shared.cu) on the sm_100-family tensor cores
// (tcgen05, accumulators in tensor memory), for bf16 pools whose blocks are whole 16-row tiles and for 8-bit pools.
//
// The queries of all sequences behind a prefix are rows of one product with its keys: with r rows a key's
// 4 D bytes serve 4 r D operations, so up to ~290 rows the keys' bytes bound the call and beyond that the
// products do.  A query tile holds floor(128 / G) sequences x G heads.
//
//   item  = (prefix, KV head, up to two query tiles): a stream of 64-key stages, the ring tiles of the
//           positions that the sequence with the shortest own part still sees;
//   line  = all items in a row, each kGap positions without work and then its stages.  The persistent grid (a CTA per SM) splits it evenly; a CTA walks its range item by
//           item (segments) and leaves a partial (reference maximum, sum, unnormalised sums) per row and segment.
//
// The own parts' kernel needs nothing of this one and starts on the SMs that it leaves: how many CTAs are used is chosen from the
// lengths, so that the two run side by side and end together (pick_ctas).
//
// Two query tiles of an item share every stage (each key is staged once for 256 rows).  An item of one tile gives its stages in
// turn to two chains of the same rows, so the S -> softmax -> P.V latency of one hides behind the other's; at a
// segment's end their states are joined out of tensor memory.
//
// Warp roles: 0 plans (segments, their sequences, and the records the join reads) and brings the keys by TMA; 1 and 3
// issue S = Q K^T of chain 0 and 1, 2 issues O += P V of both; 4-7 softmax of tile (or chain) 0, 8-11 of 1, a thread per row.  Warps without a live row only keep
// the barriers in step.  Segments are handed out through two descriptors in shared memory, so the
// producer runs into the next one while the last is finished.
//
// 8-bit pools: warps 12-15 turn the codes that the producer brings into a stage of bf16 rows, code x scale, which bf16 holds
// exactly (3 mantissa bits, a power of two); a warp takes the K and V rows of one 16-slot tile.  The same products follow.
// V rows of slots outside the prefix's window become zeros, whatever they hold.
//
// Weights are rounded to bf16 for P V (2^-8 of each, half a step), as in the decode of bf16 pools; their sum is of the unrounded ones.
// That goes for 8-bit prefixes too, where the decode has fp16 weights (2^-11): a product's operands have one type, and only bf16
// holds code x scale.  Keys and values of theirs are off by up to 2^-4 already.  (The weight as two bf16 numbers, the second
// of what the first leaves, gives 2^-15 but takes 17-26% of the call: one 64K prefix, 64 rows 76 -> 91 us, 1024 rows 293 -> 370.)
//
// Measured (head_dim 128, 8 KV heads, all SMs; a stage of 64 keys on an SM, from calls with prefixes of 16K and 128K): 0.78 us at 64
// rows, 0.95 of the measured copy rate; 0.88 at 256; 0.98 at 1024, where 1300 TFLOP/s are 0.68 of the measured peak, bound by the
// exponentials between the products.  Scored stages of 256 rows (32K and 96K): capped 1.26, biased 1.34, both 1.94 us.  8-bit: 0.89 us at
// 64 rows, bound by the conversion (1180 of 1700 cycles), 1.1 from 256 on.  The keys' bytes cross from DRAM once (88.2 of 88.1 MB for 64
// rows; 1024 rows share them through L2).
//
// Waits are bounded (~2 s) and record HWKV_DEVERR_WAIT_TIMEOUT; then all roles stop.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "hwkv_fp8.cuh"
#include "hwkv_shared.cuh"
#include "hwkv_tcgen05.cuh"

namespace hwkv {
namespace {

constexpr int kM = 128;                 // query rows per tile (MMA M)
constexpr int kKeys = 64;               // keys per stage
constexpr int kSub = kKeys / kTile;     // ring tiles per stage
constexpr int kMinStages = 4;           // fewest line positions of a CTA
// Line positions charged for an item's start: what another segment costs a CTA (its queries, the first stage's
// latency, the last's and the partial), in stages.
constexpr int kGap = 5;
constexpr int kRoleWarps = 11;          // warps that read a segment's descriptor

template <int D, bool Q8>
struct Cfg {
  static constexpr int kThreads = (Q8 ? 16 : 12) * 32;
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = kM * D * 2;
  static constexpr int kKBytes = kKeys * D * 2;
  static constexpr int kStageBytes = 2 * kKBytes;
  static constexpr int kStages = (D == 128 ? 4 : 8) - (Q8 ? (D == 128 ? 1 : 2) : 0);
  // An issuer of S that takes every other stage does not see each phase of a slot.  The parity it waits for tells phases
  // k - 1 and k + 1 apart only if it knows that the stage kStages before has arrived: that was its own where kStages is
  // even; codes are converted in order, so there it came before the issuer's last one.  (Copies land in any order.)
  static_assert(Q8 ? kStages >= 3 : kStages % 2 == 0, "an issuer may take a slot for full before its copy has landed");
  static constexpr int kStageOff = 2 * kQBytes;
  // 8-bit: stages of codes, four tiles of 16 K and 16 V rows each
  static constexpr int kTileBytes = 2 * kTile * D;
  static constexpr int kCodeBytes = kSub * kTileBytes;
  static constexpr int kCodeStages = Q8 ? (D == 128 ? 3 : 4) : 1;
  static constexpr int kCodeOff = kStageOff + kStages * kStageBytes;
  static constexpr int kHistOff = kCodeOff + (Q8 ? kCodeStages * kCodeBytes : 0);  // sequences, shortest own part and length of each prefix
  static constexpr uint32_t kCols = 512;
  static constexpr uint32_t kColO = 4 * kKeys;
  static int smem(int prefixes) { return kHistOff + 12 * prefixes + 1024; }
};

// A CTA's part of one item.
struct Segment {
  int f, h;
  int N;           // tokens of the prefix
  int w, C;        // window and ring capacity
  int first_tile;  // ring tile of the item's first stage
  int tiles;       // ring tiles of the item
  int j0, stages;  // this CTA's stages of it, 0: no more segments
  int seqs;        // sequences
  int one;         // a single query tile: its stages alternate between two chains
  int slot;        // where the partials go
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Waits for a phase; gives up when another role has (`abort`) or after ~2 s, which it records and announces.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > 2000000000ull) {
        *abort = 1;
        atomicOr(err, HWKV_DEVERR_WAIT_TIMEOUT);
        return false;
      }
    }
  }
}

// One lane of the warp.  (A branch on it, unlike one on lane == 0, is known to run a single thread, which leaves
// descriptors in uniform registers.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// bits lo .. hi (inclusive, clamped to 0 .. 15) of a 16-key tile
__device__ __forceinline__ uint32_t bits16(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 15);
  return lo > hi ? 0u : ((0xFFFFu >> (15 - hi)) & (0xFFFFu << lo));
}

// 64 values folded by a tree of three-input operations, not a dependent chain
template <typename Op>
__device__ __forceinline__ float fold64(const float (&v)[kKeys], Op op) {
  float t1[22], t2[8];
#pragma unroll
  for (int i = 0; i < 21; ++i) t1[i] = op(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  t1[21] = v[63];
#pragma unroll
  for (int i = 0; i < 7; ++i) t2[i] = op(t1[3 * i], t1[3 * i + 1], t1[3 * i + 2]);
  t2[7] = t1[21];
  return op(op(t2[0], t2[1], t2[2]), op(t2[3], t2[4], t2[5]), op(t2[6], t2[7], t2[7]));
}

// First stage of CTA c's share of a line of T stages over n CTAs, and the CTA whose share holds stage t: 32-bit
// divisions where the products fit.
__device__ __forceinline__ long long line_start(long long T, int c, int n) {
  return T < (1 << 22) ? (long long)((uint32_t)T * (uint32_t)c / (uint32_t)n) : T * c / n;
}
__device__ __forceinline__ int line_cta(long long t, long long T, int n) {
  return T < (1 << 22) ? (int)((((uint32_t)t + 1u) * (uint32_t)n - 1u) / (uint32_t)T) : (int)(((t + 1) * n - 1) / T);
}

// CTAs for T line positions beside the own parts' kernel of `tiles` tiles in `groups` groups: the number that lets the later of the two
// end first, by a model of both in ns.  Here 8 us and a stage per position; there a CTA takes its tiles, 4.8 us a group and 12 to 18 us
// (fitted to that kernel alone on 16 to 288 CTAs: within 10% from 20 to 500 us), and its CTAs go through the SMs left to them in waves
// (lane w tries w + 1 of them, with two SMs to spare: a straggler is another wave; the last lane tries all SMs here and the own
// parts after).  In integers: every CTA must choose alike.
__device__ __forceinline__ int pick_ctas(const SharedArgs& a, long long T, uint32_t tiles, uint32_t groups, int sms, int lane) {
  const long long each = a.own_base_ns + ((long long)tiles * a.own_tile_ns + (long long)groups * 4800) / a.own_ctas;
  const int waves = lane + 1;
  const int slots = (a.own_ctas + waves - 1) / waves, theirs = (slots + a.own_per_sm - 1) / a.own_per_sm + 2;
  const int mine = lane == 31 ? sms : sms - theirs;
  long long time = (long long)1 << 60;
  if (mine >= 1) {
    const long long here = 8000 + T * a.stage_ns / mine;
    time = lane == 31 ? here + each + 3000 : max(here, waves * each);
  }
  long long best = time;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  return __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, time == best)) - 1);
}

// The ring tiles of the newest `need` of N tokens: first tile and their number.
__device__ __forceinline__ void need_tiles(int N, int need, int C, int& first_tile, int& tiles) {
  first_tile = tiles = 0;
  if (need <= 0) return;
  const int first = (N - need) % C;
  first_tile = first >> 4;
  tiles = min(C >> 4, (int)(((uint32_t)first + (uint32_t)need - 1u) >> 4) - first_tile + 1);
}

// age of a ring tile's first slot: its slots' ages fall by one from it, past 0 they go on at C - 1
__device__ __forceinline__ int tile_age(const Segment& sg, int last, int i) {
  int t = sg.first_tile + i;
  if (t >= sg.C >> 4) t -= sg.C >> 4;
  const int d = last - (t << 4);
  return d < 0 ? d + sg.C : d;
}

__device__ __forceinline__ void store_part(float* p, const float (&o)[32]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<float4*>(p + 4 * k) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
}

// What is done to the scores between the two products, an instance each.
enum { kPlain = 0, kCap = 1, kBias = 2 };

// A biased stage's keys share an offset, the bias of its first, kept beside the scores; their own terms of up to 64 slopes cancel what is
// over.  Both leave a few fp32 roundings of the bias.  Where it may pass this (log2 units) within the window, or 64 slopes pass half of it, that
// would be more than a log2 unit in a weight (past 2^31 the weight overflows), and a slope over a small scale is infinite: warps with
// such a slope keep no offset, and each tile's scores take what its distance takes.
constexpr float kFarBias = 0x1p24f;

template <int D, int SC, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::kThreads, 1) shared_tc_kernel(const __grid_constant__ CUtensorMap pool_map,
                                                               const __grid_constant__ CUtensorMap stage_map,
                                                               const __grid_constant__ SharedArgs a) {
  using K = Cfg<D, Q8>;
  constexpr int NS = K::kStages, kThreads = K::kThreads;
  constexpr int NC = K::kCodeStages;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  int* s_count = reinterpret_cast<int*>(smem + K::kHistOff);
  int* s_short = s_count + a.num_prefixes;
  int* s_len = s_short + a.num_prefixes;
  __shared__ __align__(8) uint64_t kv_full[NS], kv_empty[NS];
  __shared__ __align__(8) uint64_t code_full[NC], code_empty[NC];
  constexpr int kScaleRing = Q8 ? 64 : 1;  // scales (K, V) of the stages' tiles, planned up to 32 stages ahead
  __shared__ float2 s_scale[kScaleRing][kSub];
  // per chain x and parity b of its stages (a phase is one stage of that parity, so no waiter falls two behind)
  __shared__ __align__(8) uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2], drain[3];
  __shared__ __align__(8) uint64_t seg_full[2], seg_empty[2];
  __shared__ __align__(8) uint64_t ml_full, o_read;  // two chains of the same rows: states published, O of both read
  __shared__ float2 s_ml[2][kM];
  __shared__ Segment s_seg[2];
  __shared__ int s_seq[2][2 * kM];
  __shared__ int4 s_copy[32];  // copy plan of the producer's next 32 stages: pool rows of the four tiles
  __shared__ int4 s_rows[Q8 ? 32 : 1];  // 8-bit: blocks in s_copy, rows in them here
  __shared__ int2 s_box[32];   // ... or the one box that holds them: first block (-1: none) and row in it
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_own, s_groups;  // tiles of the own parts, (sequence, head) groups that have some

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.pv.kv_heads, G = a.group, bs = a.pv.block_size;
  const int QT = kM / G;  // sequences per query tile
  const int cta = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();  // the own parts may start where SMs are free: all before this grid has completed

  // ---- sequences, shortest own part and length of each prefix ---------------------------------
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], Q8 ? 4 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < NC; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], 4);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[x][b], 1);
        mbar_init(&p_full[x][b], 4);
        mbar_init(&o_done[x][b], 1);
      }
      mbar_init(&q_full[x], 4);
      mbar_init(&seg_full[x], 1);
      mbar_init(&seg_empty[x], kRoleWarps + (Q8 ? 4 : 0));
    }
    for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
    mbar_init(&ml_full, 8);
    mbar_init(&o_read, 8);
    s_abort = 0;
    s_own = s_groups = 0u;
    fence_mbar_init();
    prefetch_tensormap(&pool_map);
    prefetch_tensormap(&stage_map);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, K::kCols);
    tmem_relinquish();
  }
  for (int f = threadIdx.x; f < a.num_prefixes; f += kThreads) {
    s_count[f] = 0;
    s_short[f] = INT32_MAX;
  }
  // the first sequence's and prefix's loads are on their way while the counts are cleared
  const int s_own_seq = (int)threadIdx.x < a.num_seqs ? (int)threadIdx.x : -1;
  const int f_own = s_own_seq >= 0 ? a.prefix_of[s_own_seq] : -1;
  const int n_own = s_own_seq >= 0 ? shared_len(a, s_own_seq) : 0;
  for (int f = threadIdx.x; f < a.num_prefixes; f += kThreads) {
    const int N = a.prefix_lens[f];
    if (N < 0 && cta == 0) atomicOr(a.pv.err, HWKV_DEVERR_NEG_LENGTH);
    s_len[f] = max(N, 0);
  }
  __syncthreads();
  auto count = [&](int f, int n) {
    if (f >= a.num_prefixes && cta == 0) atomicOr(a.pv.err, HWKV_DEVERR_BAD_PREFIX);
    if (f < 0 || f >= a.num_prefixes) return;
    atomicAdd(&s_count[f], 1);
    atomicMin(&s_short[f], n);
  };
  uint32_t own_tiles = 0u, own_groups = 0u;
  auto own_work = [&](int n) {
    if (n <= 0 || a.own_ctas == 0) return;
    for (int h = 0; h < H; ++h) own_tiles += (uint32_t)((min(n, a.own_window[h]) + 15) >> 4);
    own_groups += (uint32_t)H;
  };
  if (s_own_seq >= 0) {
    count(f_own, n_own);
    own_work(n_own);
  }
  for (int s = threadIdx.x + kThreads; s < a.num_seqs; s += kThreads) {
    const int n = shared_len(a, s);
    count(a.prefix_of[s], n);
    own_work(n);
  }
  if (own_tiles > 0u) {
    atomicAdd(&s_own, own_tiles);
    atomicAdd(&s_groups, own_groups);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t sbase = smem_addr(smem);
  volatile int* abort = &s_abort;

  // Segment i as the roles see it; false: no more, or a wait was given up.
  auto next_segment = [&](int i, Segment& sg) {
    if (!__all_sync(0xffffffffu, wait(&seg_full[i & 1], (uint32_t)(i >> 1) & 1u, abort, a.pv.err))) return false;
    sg = s_seg[i & 1];
    return sg.stages > 0;
  };
  // A role's warp is through with segment i's descriptor and sequences.
  auto done_segment = [&](int i) {
    __syncwarp();
    if (lane == 0) arrive(&seg_empty[i & 1]);
  };

  if (warp == 0) {
    // ---- plan and TMA producer (whole warp) ----------------------------------------------------
    // The line: entries (prefix, head) of items x stages, some consecutive ones per lane.
    struct Entry {
      int f, h, C, first_tile, tiles, stages, items;
    };
    auto entry_of = [&](int e) {
      Entry n;
      n.f = e / H;
      n.h = e - n.f * H;
      n.C = (a.g.nblk_prefix[n.h + 1] - a.g.nblk_prefix[n.h]) * bs;
      n.items = (s_count[n.f] + 2 * QT - 1) / (2 * QT);
      const int w = a.g.window[n.h];
      need_tiles(s_len[n.f], n.items > 0 ? min(s_len[n.f], w - min(w, s_short[n.f])) : 0, n.C, n.first_tile, n.tiles);
      n.stages = (n.tiles + kSub - 1) / kSub;
      return n;
    };
    auto span_of = [](const Entry& n) { return n.stages > 0 ? (long long)n.stages + kGap : 0ll; };  // line positions of an item
    const int entries = a.num_prefixes * H;
    const int per = (entries + 31) / 32;
    const int e_lo = min(entries, lane * per), e_hi = min(entries, e_lo + per);
    long long mine = 0, sum = 0;
    int mine_items = 0, sum_items = 0;
    for (int e = e_lo; e < e_hi; ++e) {
      const Entry n = entry_of(e);
      mine += n.items * span_of(n);
      mine_items += n.items;
    }
    sum = mine;
    sum_items = mine_items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      const int z = __shfl_up_sync(0xffffffffu, sum_items, o);
      if (lane >= o) {
        sum += y;
        sum_items += z;
      }
    }
    const long long T = __shfl_sync(0xffffffffu, sum, 31);
    const int share = T > 0 && s_own > 0u ? pick_ctas(a, T, s_own, s_groups, (int)gridDim.x, lane) : (int)gridDim.x;
    const int ctas = T < (long long)kMinStages * share ? max(1, (int)T / kMinStages) : share;
    long long at = 0, t_hi = 0, pre = 0;
    int e = 0, items = 0;
    Entry n{};
    if (cta < ctas && T > 0) {
      at = line_start(T, cta, ctas);
      t_hi = line_start(T, cta + 1, ctas);
      // the lane whose entries hold the range's first stage
      const int who = __ffs(__ballot_sync(0xffffffffu, sum - mine <= at && at < sum)) - 1;
      pre = __shfl_sync(0xffffffffu, sum - mine, who);
      items = __shfl_sync(0xffffffffu, sum_items - mine_items, who);
      e = who * per;
      n = entry_of(e);
    }
    int issued = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (i >= 2 && !__all_sync(0xffffffffu, wait(&seg_empty[i & 1], (uint32_t)((i >> 1) - 1) & 1u, abort, a.pv.err))) break;
      // the next item with stages in the range: over its gap, or past it
      int off = 0;
      long long begin = 0, end = 0;  // the item's stages on the line
      while (at < t_hi) {
        while (at >= pre + n.items * span_of(n)) {
          pre += n.items * span_of(n);
          items += n.items;
          n = entry_of(++e);
        }
        const int span = n.stages + kGap;
        off = at - pre <= INT32_MAX ? (int)(at - pre) / span : (int)((at - pre) / span);
        begin = pre + (long long)off * span + kGap;
        end = begin + n.stages;
        at = max(at, begin);
        if (at < min(end, t_hi)) break;
        at = end;
      }
      if (at >= t_hi) {
        if (lane == 0) {
          s_seg[i & 1].stages = 0;
          arrive(&seg_full[i & 1]);
        }
        break;
      }
      Segment sg;
      sg.f = n.f, sg.h = n.h, sg.N = s_len[n.f], sg.w = a.g.window[n.h], sg.C = n.C, sg.first_tile = n.first_tile, sg.tiles = n.tiles;
      sg.j0 = (int)(at - begin);
      sg.stages = (int)(min(end, t_hi) - at);
      sg.seqs = shared_members(a, n.f, off * 2 * QT, 2 * QT, s_seq[i & 1], lane);
      sg.one = sg.seqs <= QT;
      sg.slot = (int)(items + off) + cta;  // unique along the line: each step of it moves on the item or the CTA
      if (lane == 0) {
        s_seg[i & 1] = sg;
        __threadfence_block();
        arrive(&seg_full[i & 1]);
      }
      if (sg.j0 == 0) {  // the item's records: its partials lie one slot per CTA
        const int parts = line_cta(end - 1, T, ctas) - cta + 1;
        for (int k = lane; k < sg.seqs; k += 32) {
          const int x = sg.one ? 0 : k / QT;
          a.rec[(int64_t)s_seq[i & 1][k] * H + n.h] =
              make_int4(2 * sg.slot + x, 2, parts, (k - x * QT) * G);
        }
      }
      at += sg.stages;
      const int32_t* tbl = a.pv.tbl + a.g.tbl_base + (int64_t)sg.f * a.g.tbl_seq_stride + a.g.nblk_prefix[sg.h];
      const int C16 = sg.C >> 4;
      // 32 stages planned at a time, one per lane (table look-ups in parallel); lane 0 issues the copies
      for (int c0 = 0; ok && c0 < sg.stages; c0 += 32) {
        if (c0 + lane < sg.stages) {
          int row[kSub], blk[kSub], r0[kSub];
          bool box = a.stage_tb > 0;  // one box of the stage map: stage_tb rows of each of consecutive blocks
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int k = (sg.j0 + c0 + lane) * kSub + u;
            blk[u] = 0;  // past the item: row 0 of the pool, masked
            r0[u] = 0;
            if (k < sg.tiles) {
              int t = sg.first_tile + k;
              if (t >= C16) t -= C16;
              const int t0 = t << 4;
              const int jb = a.bs_log2 >= 0 ? t0 >> a.bs_log2 : t0 / bs;
              blk[u] = __ldg(tbl + jb);
              r0[u] = t0 - jb * bs;
            } else {
              box = false;
            }
          }
          const int step_log2 = a.stage_tb == 64 ? 6 : a.stage_tb == 32 ? 5 : 4;
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            if (blk[u] < 0 || (int64_t)blk[u] >= a.pv.total_blocks) {
              atomicOr(a.pv.err, HWKV_DEVERR_BAD_BLOCK);
              blk[u] = r0[u] = 0;
              box = false;
            }
            row[u] = blk[u] * 2 * bs + r0[u];
            box = box && blk[u] == blk[0] + ((kTile * u) >> step_log2) && r0[u] == r0[0] + ((kTile * u) & (a.stage_tb - 1));
          }
          box = box && r0[0] + a.stage_tb <= bs;
          if constexpr (Q8) {
            const int groups = bs / kScaleGroup;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
              s_scale[(issued + lane) % kScaleRing][u] =
                  __ldcg(reinterpret_cast<const float2*>(a.pv.scales) + (int64_t)blk[u] * groups + (r0[u] >> 4));
          }
          s_copy[lane] = Q8 ? make_int4(blk[0], blk[1], blk[2], blk[3]) : make_int4(row[0], row[1], row[2], row[3]);
          s_box[lane] = make_int2(box ? blk[0] : -1, r0[0]);
          if constexpr (Q8) s_rows[lane] = make_int4(r0[0], r0[1], r0[2], r0[3]);
        }
        __syncwarp();
        if (lane == 0) {
          for (int l = 0; l < 32 && c0 + l < sg.stages; ++l, ++issued) {
            if constexpr (Q8) {
              const int cs = issued % NC;
              if (issued >= NC && !wait(&code_empty[cs], (uint32_t)(issued / NC - 1) & 1u, abort, a.pv.err)) {
                ok = false;
                break;
              }
              const int4 cb = s_copy[l], cr = s_rows[l];
              const int cblk[kSub] = {cb.x, cb.y, cb.z, cb.w}, crow[kSub] = {cr.x, cr.y, cr.z, cr.w};
              mbar_arrive_expect_tx(&code_full[cs], K::kCodeBytes);
#pragma unroll
              for (int u = 0; u < kSub; ++u)
                tma_3d(sbase + K::kCodeOff + cs * K::kCodeBytes + u * K::kTileBytes, &pool_map, 0, crow[u], 2 * cblk[u], &code_full[cs]);
              continue;
            }
            const int st = issued % NS;
            if (issued >= NS && !wait(&kv_empty[st], (uint32_t)(issued / NS - 1) & 1u, abort, a.pv.err)) {
              ok = false;
              break;
            }
            const int4 c = s_copy[l];
            const int row[kSub] = {c.x, c.y, c.z, c.w};
            const uint32_t kdst = sbase + K::kStageOff + st * K::kStageBytes, vdst = kdst + K::kKBytes;
            mbar_arrive_expect_tx(&kv_full[st], K::kStageBytes);
            const int2 box = s_box[l];
            if (box.x >= 0) {
#pragma unroll
              for (int hf = 0; hf < K::kHalves; ++hf) {
                tma_3d(kdst + hf * (kKeys * 128), &stage_map, hf * 64, box.y, box.x, &kv_full[st]);
                tma_3d(vdst + hf * (kKeys * 128), &stage_map, hf * 64, bs + box.y, box.x, &kv_full[st]);
              }
            } else {
#pragma unroll
              for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int hf = 0; hf < K::kHalves; ++hf) {
                  const uint32_t at = hf * (kKeys * 128) + u * (kTile * 128);
                  tma_2d(kdst + at, &pool_map, hf * 64, row[u], &kv_full[st]);
                  tma_2d(vdst + at, &pool_map, hf * 64, row[u] + bs, &kv_full[st]);
                }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        issued = __shfl_sync(0xffffffffu, issued, 0);
      }
    }
    if (lane == 0 && *abort) {  // let the copies in flight land before the shared memory is released
      constexpr int n = Q8 ? NC : NS;
      uint64_t* full = Q8 ? code_full : kv_full;
      for (int j = max(0, issued - n); j < issued; ++j)
        if (!mbar_wait_bounded(&full[j % n], (uint32_t)(j / n) & 1u)) break;
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---- MMA issuers: warps 1 and 3 the S of chain 0 and 1, warp 2 the P . V of both ------------------
    constexpr uint32_t idS = umma_idesc_bf16(kM, kKeys, false, false);
    constexpr uint32_t idO = umma_idesc_bf16(kM, D, false, true);
    const uint64_t dq = umma_desc_sw128(sbase, 16, 1024);
    const uint64_t dk = umma_desc_sw128(sbase + K::kStageOff, 16, 1024);
    const uint64_t dv = umma_desc_sw128(sbase + K::kStageOff + K::kKBytes, kKeys * 128, 1024);
    int stage = 0;              // stages of this CTA so far
    int done[2] = {0, 0};       // stages of each chain (an S issuer: of its own)
    int queries = 0;            // segments of an S issuer's chain
    bool ok = true;
    Segment sg;
    for (int i = 0; ok && next_segment(i, sg); ++i) {
      if (elect_one()) {
        if (warp != 2) {
          // S of each of the chain's stages into its buffers in turn, once the P . V of the stage two before, which read
          // the P there, has completed
          const int x = warp >> 1;
          int n = done[0];
          for (int jj = sg.one ? x : 0; ok && jj < sg.stages; jj += sg.one ? 2 : 1, ++n) {
            const int g = stage + jj, st = g % NS, b = n & 1;
            if (jj < 1 + sg.one) {  // the segment's first
              ok = wait(&q_full[x], (uint32_t)queries & 1u, abort, a.pv.err);
              if (!ok) break;
              ++queries;
            }
            if (n >= 2) {
              ok = wait(&o_done[x][b], (uint32_t)((n - 2) >> 1) & 1u, abort, a.pv.err);
              if (!ok) break;
            }
            ok = wait(&kv_full[st], (uint32_t)(g / NS) & 1u, abort, a.pv.err);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t dqx = dq + (uint64_t)((x * K::kQBytes) >> 4);
            const uint64_t dks = dk + (uint64_t)((st * K::kStageBytes) >> 4);
            const uint32_t to = tmem + (2 * x + b) * kKeys;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              umma_bf16(to, dqx + (uint64_t)(((k >> 2) * (kM * 128) + (k & 3) * 32) >> 4),
                        dks + (uint64_t)(((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4), idS, k > 0 ? 1u : 0u);
            umma_commit(&s_full[x][b]);
          }
          done[0] = n;
        } else {
          // O += P . V once the softmax has written P into tensor memory
          for (int jj = 0; ok && jj < sg.stages; ++jj) {
            const int st = (stage + jj) % NS;
            const uint64_t dvs = dv + (uint64_t)((st * K::kStageBytes) >> 4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (sg.one && (jj & 1) != x) continue;
              const int b = done[x] & 1;
              ok = wait(&p_full[x][b], (uint32_t)(done[x] >> 1) & 1u, abort, a.pv.err);
              if (!ok) break;
              tc_fence_after_sync();
              const uint32_t pcol = tmem + (2 * x + b) * kKeys;
              const uint32_t add = jj < 1 + sg.one ? 0u : 1u;  // 0: the segment's first
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                umma_bf16_tmem_a(tmem + K::kColO + x * D, pcol + k * 8, dvs + (uint64_t)((k * 16 * 128) >> 4), idO, k > 0 ? 1u : add);
              umma_commit(&o_done[x][b]);
              ++done[x];
            }
            if (!ok) break;
            umma_commit(&kv_empty[st]);  // (its S was complete before P was written)
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      stage += sg.stages;
      done_segment(i);
    }
    if (elect_one()) {
      umma_commit(&drain[warp - 1]);  // all that this lane issued completes before tensor memory is freed
      mbar_wait_bounded(&drain[warp - 1], 0);
    }
    __syncwarp();
  } else if (Q8 && warp >= 12) {
    // ---- 8-bit: codes to bf16 rows, a warp per tile of the stage -------------------------------
    const int u = warp - 12;
    constexpr int kC = D / 16;        // 16-code chunks of a row
    constexpr int kR = 32 / kC;       // rows a warp covers at a time
    const int c = lane % kC, r_lane = lane / kC;
    int stage = 0;
    bool ok = true;
    Segment sg;
    for (int i = 0; ok && next_segment(i, sg); ++i) {
      const int last = sg.N > 0 ? (sg.N - 1) % sg.C : 0;
      const int window = min(sg.N, sg.w);
      for (int jj = 0; jj < sg.stages; ++jj, ++stage) {
        const int st = stage % NS, cs = stage % NC;
        ok = __all_sync(0xffffffffu, wait(&code_full[cs], (uint32_t)(stage / NC) & 1u, abort, a.pv.err));
        if (ok && stage >= NS) ok = __all_sync(0xffffffffu, wait(&kv_empty[st], (uint32_t)(stage / NS - 1) & 1u, abort, a.pv.err));
        if (!ok) break;
        const float2 scale = s_scale[stage % kScaleRing][u];
        const int k = (sg.j0 + jj) * kSub + u;  // tile of the item
        const int age0 = k < sg.tiles ? tile_age(sg, last, k) : 0;
        const uint32_t code = sbase + K::kCodeOff + cs * K::kCodeBytes + u * K::kTileBytes;
        const uint32_t rows = sbase + K::kStageOff + st * K::kStageBytes + u * (kTile * 128);
        // all loads ahead of the arithmetic: rows of D bytes, their 16-byte chunks swizzled with the row (head_dim 128: by row % 8,
        // 64: by row / 2 % 4)
        constexpr int kG = kTile / kR;
        uint4 w[2][kG];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const int r = g * kR + r_lane;
            const uint32_t from = code + kv * (kTile * D) + r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[kv][g].x), "=r"(w[kv][g].y), "=r"(w[kv][g].z), "=r"(w[kv][g].w)
                         : "r"(from));
          }
        if (!(k < sg.tiles && age0 >= kTile - 1 && age0 < window)) {  // a tile with slots outside the window
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            int age = age0 - (g * kR + r_lane);
            if (age < 0) age += sg.C;
            if (k >= sg.tiles || age >= window) w[1][g] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const float f = kv ? scale.y : scale.x;
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const int r = g * kR + r_lane;
            const uint32_t in[4] = {w[kv][g].x, w[kv][g].y, w[kv][g].z, w[kv][g].w};
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t lo, hi;
              e4m3x4_to_f16(in[e], lo, hi);
              const float2 x = fmul2(half2_to_float2(lo), make_float2(f, f)), y = fmul2(half2_to_float2(hi), make_float2(f, f));
              out[2 * e] = pack_bf16(x.x, x.y);
              out[2 * e + 1] = pack_bf16(y.x, y.y);
            }
            // 16 values are chunks 2 c and 2 c + 1 of the bf16 row: column block c / 4, swizzled by the row
            const uint32_t to = rows + kv * K::kKBytes + (c >> 2) * (kKeys * 128) + r * 128;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t at = to + (((2 * (c & 3) + e) ^ (r & 7)) << 4);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(out[4 * e]), "r"(out[4 * e + 1]), "r"(out[4 * e + 2]),
                           "r"(out[4 * e + 3])
                           : "memory");
            }
          }
        }
        fence_proxy_async_smem();  // before the products read the rows
        __syncwarp();
        if (lane == 0) {
          arrive(&kv_full[st]);
          arrive(&code_empty[cs]);
        }
      }
      done_segment(i);
    }
  } else {
    // ---- softmax of chain x: a thread per row ---------------------------------------------
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int seq_r = r / G, head_r = r - seq_r * G;  // the row's sequence of the tile, and query head
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t colO = K::kColO + x * D;
    // with a positive scale the maximum is of scores that are still to be multiplied by it; masked ones become -inf before (else +inf)
    const bool pos_scale = SC || a.scale_log2 > 0.f;
    const float masked = pos_scale ? kNegInf : -kNegInf;
    int done = 0;
    uint32_t joins = 0;   // segments of two chains so far
    bool joined = false;  // after one: O may still be read by the other chain's warps
    bool ok = true;
    Segment sg;
    for (int i = 0; ok && next_segment(i, sg); ++i) {
      const int first_seq = sg.one ? 0 : x * QT;
      const int seqs = min(QT, sg.seqs - first_seq);
      const int mine = sg.one ? (sg.stages + 1 - x) >> 1 : sg.stages;  // stages of this chain
      const bool live = r < seqs * G;
      const int s = live ? s_seq[i & 1][first_seq + seq_r] : 0;
      {
        // this warp's rows of Q into shared memory, as a 128-byte-swizzled K-major tile
        constexpr int kC = D / 8, kR = 32 / kC;  // 16-byte chunks of a row, rows per step
        const int c = lane % kC;
        const int row = live ? (s * H + sg.h) * G + head_r : -1;  // the lane's row among the queries
        uint4 v[kC];
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          const int from = __shfl_sync(0xffffffffu, row, k * kR + lane / kC);
          v[k] = make_uint4(0u, 0u, 0u, 0u);
          if (from >= 0) v[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (int64_t)from * D + 8 * c);
        }
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          const int rr = quarter * 32 + k * kR + lane / kC;
          const uint32_t at = sbase + x * K::kQBytes + (c >> 3) * (kM * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[k].x), "r"(v[k].y), "r"(v[k].z), "r"(v[k].w)
                       : "memory");
        }
        fence_proxy_async_smem();
      }
      done_segment(i);
      if (mine > 0 && lane == 0) arrive(&q_full[x]);
      const int own = live ? shared_len(a, s) : 0;
      // a key is seen when its age, counted from the prefix's last token, is below this
      const int reach = live ? min(sg.N, sg.w - min(sg.w, own)) : 0;
      const int last = sg.N > 0 ? (sg.N - 1) % sg.C : 0;
      const bool any_live = __any_sync(0xffffffffu, live);
      int reach_all = live ? reach : INT32_MAX;  // the least over the warp's rows
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) reach_all = min(reach_all, __shfl_xor_sync(0xffffffffu, reach_all, o));
      const float slope2 = (SC & kBias) && live ? slope_log2(a.score, sg.h * G + head_r) : 0.f;
      const bool steep = (SC & kBias) && __any_sync(0xffffffffu, fabsf(slope2) * (float)max(reach + own, 128) > kFarBias);
      // capped scores are in log2 units when they meet the softmax; biased ones alone stay raw, the slope divided by the scale, unless
      // that is too small or negative, or a slope too steep
      const bool raw_bias = SC == kBias && a.scale_log2 > 0x1p-40f && !steep;
      const float sl2 = SC && !raw_bias ? 1.f : a.scale_log2;
      const float slope = slope2 / sl2;
      float m_ref = kNegInf, l = 0.f;
      uint32_t clean_word = 0u;
      for (int jj = 0; jj < mine; ++jj, ++done) {
        const int b = done & 1;
        const int j = sg.j0 + (sg.one ? 2 * jj + x : jj);  // stage of the item
        if ((jj & 31) == 0) {  // stages whose keys all the warp's rows see, 32 at a time
          const int jl = sg.j0 + (sg.one ? 2 * (jj + lane) + x : jj + lane);
          bool clean = jl * kSub + kSub <= sg.tiles;
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int age = tile_age(sg, last, min(jl * kSub + u, sg.tiles - 1));
            clean = clean && (age >= kTile - 1 ? age : sg.C - 1) < reach_all;
          }
          clean_word = __ballot_sync(0xffffffffu, clean);
        }
        ok = __all_sync(0xffffffffu, wait(&s_full[x][b], (uint32_t)(done >> 1) & 1u, abort, a.pv.err));
        if (ok && joined) {  // the other chain's warps may still read O: no P . V into it before
          ok = __all_sync(0xffffffffu, wait(&o_read, (joins - 1u) & 1u, abort, a.pv.err));
          joined = false;
        }
        if (!ok) break;
        if (!any_live) {  // rows that nothing reads
          if (lane == 0) arrive(&p_full[x][b]);
          continue;
        }
        tc_fence_after_sync();
        float sv[kKeys];
        tmem_ld64(lane_base + (2 * x + b) * kKeys, sv);
        const bool clean = (clean_word >> (jj & 31)) & 1u;
        uint32_t vis[kSub];
        int age[kSub];
        if (!clean || (SC & kBias) != 0) {
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            age[u] = tile_age(sg, last, min(j * kSub + u, sg.tiles - 1));
            // slots up to the newest, then (a tile that holds it) the oldest ones
            vis[u] = bits16(age[u] - reach + 1, age[u]) | bits16(max(age[u] + 1, age[u] + sg.C - reach + 1), kTile - 1);
            if (j * kSub + u >= sg.tiles) vis[u] = 0u;
          }
        }
        float row_off = 0.f;      // what is still to be added to every score of the row, in log2 units
        float row_max = 0.f;      // the row's maximum, when have_max
        bool have_max = false;
        if constexpr ((SC & kCap) != 0) {
          if (!clean) {  // what is masked does not decide how the others are capped
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
              for (int k = 0; k < kTile; ++k) sv[u * kTile + k] = (vis[u] >> k) & 1u ? sv[u * kTile + k] : 0.f;
          }
          const float hi = fold64(sv, [](float p, float q, float z) { return fmax3(p, q, z); });
          const float lo = fold64(sv, [](float p, float q, float z) { return fmin3(p, q, z); });
          const float u_max = fmaxf(hi, -lo) * fabsf(a.score.cap_in);
          // no score of the warp reaches the cap (or half of it): a polynomial in x^2 alone, on packed pairs
          auto polynomial = [&](auto degree, const float* coef) {
            constexpr int n = decltype(degree)::value;
            auto capped = [&](float2 v) {
              const float2 z = fmul2(v, v);
              float2 p = make_float2(coef[n], coef[n]);
#pragma unroll
              for (int k = n - 1; k >= 0; --k) p = ffma2(z, p, make_float2(coef[k], coef[k]));
              return fmul2(v, p);
            };
#pragma unroll
            for (int c = 0; c < kKeys; c += 2) {
              const float2 y = capped(make_float2(sv[c], sv[c + 1]));
              sv[c] = y.x;
              sv[c + 1] = y.y;
            }
            if (clean && SC == kCap) {  // the cap keeps the order
              const float top = a.scale_log2 > 0.f ? hi : lo;
              row_max = capped(make_float2(top, top)).x;
              have_max = true;
            }
          };
          if (a.score.poly_on && __all_sync(0xffffffffu, u_max <= 0.5f || !live)) {
            polynomial(std::integral_constant<int, 3>(), a.score.half);
          } else if (a.score.poly_on && __all_sync(0xffffffffu, u_max <= 1.f || !live)) {
            polynomial(std::integral_constant<int, 5>(), a.score.poly);
          } else {  // both forms of tanh_f32, and a choice per score
#pragma unroll
            for (int c = 0; c < kKeys; c += 2) {
              const float2 v = make_float2(sv[c], sv[c + 1]);
              const float2 u = fmul2(v, make_float2(a.score.cap_in, a.score.cap_in));
              const float2 y = fmul2(fmul2(v, make_float2(a.scale_log2, a.scale_log2)), tanh_poly2(fmul2(u, u)));
              sv[c] = fabsf(u.x) <= 1.f ? y.x : a.score.cap_out * tanh_exp(u.x);
              sv[c + 1] = fabsf(u.y) <= 1.f ? y.y : a.score.cap_out * tanh_exp(u.y);
            }
          }
        } else if (SC && !raw_bias) {
#pragma unroll
          for (int c = 0; c < kKeys; c += 2) {
            const float2 y = fmul2(make_float2(sv[c], sv[c + 1]), make_float2(a.scale_log2, a.scale_log2));
            sv[c] = y.x;
            sv[c + 1] = y.y;
          }
        }
        if constexpr ((SC & kBias) != 0) {
          // less slope * distance: key c of the stage gets slope * c, an immediate operand, and the row its first key's distance
          row_off = steep ? 0.f : -slope * sl2 * (float)((uint32_t)age[0] + (uint32_t)own);
#pragma unroll
          for (int c = 0; c < kKeys; ++c) sv[c] = fmaf(slope, (float)c, sv[c]);
          bool run = age[kSub - 1] >= kTile - 1 && !steep;  // 64 consecutive positions
#pragma unroll
          for (int u = 1; u < kSub; ++u) run = run && age[u] == age[0] - u * kTile;
          if (!run) {
            // tile by tile, what its keys are off a run from the first (or from the query); past the newest slot come the oldest, a ring
            // away
            const int from = steep ? own : -age[0];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              const float near = -slope * (float)(int)((uint32_t)age[u] + (uint32_t)from + u * kTile), wrapped = near - slope * (float)sg.C;
#pragma unroll
              for (int k = 0; k < kTile; ++k) sv[u * kTile + k] += k <= age[u] ? near : wrapped;
            }
          }
        }
        if (!clean) {
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int k = 0; k < kTile; ++k) sv[u * kTile + k] = (vis[u] >> k) & 1u ? sv[u * kTile + k] : masked;
        }
        // row maximum in log2 units
        float mx;
        if (pos_scale) {
          const float top = SC && have_max ? row_max : fold64(sv, [](float p, float q, float z) { return fmax3(p, q, z); });
          mx = top == kNegInf ? kNegInf : SC ? fmaf(top, sl2, row_off) : top * sl2;
        } else {
          mx = kNegInf;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) {
            sv[c] = sv[c] == -kNegInf ? kNegInf : sv[c] * sl2;
            mx = fmaxf(mx, sv[c]);
          }
        }
        // The reference lies 2^8 above a maximum and moves only when one passes it, so O is rarely touched (a row that has seen no
        // key yet has nothing in O: rows of other reaches would otherwise touch it stage after stage).  Weights are at most 1:
        // no value overflows by itself.
        const bool grow = mx > m_ref;
        const float m_new = mx + 8.f;
        if (jj > 0 && __any_sync(0xffffffffu, grow && m_ref != kNegInf)) {
          const int before = done - 1;  // O may be rescaled once the last P . V into it has completed
          ok = __all_sync(0xffffffffu, wait(&o_done[x][before & 1], (uint32_t)(before >> 1) & 1u, abort, a.pv.err));
          if (!ok) break;
          tc_fence_after_sync();
          const float f = grow && m_ref != kNegInf ? ex2(m_ref - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(lane_base + colO + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f;
            tmem_st32(lane_base + colO + c, o);
          }
        }
        if (grow) {
          l *= ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const float bm = m_ref == kNegInf ? 0.f : m_ref;
        // P (bf16 pairs) over the S columns it came from
        const float2 sl2v = make_float2(pos_scale ? sl2 : 1.f, pos_scale ? sl2 : 1.f);
        const float2 nb = make_float2(row_off - bm, row_off - bm);
        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float pk[kKeys / 2];
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) {
          const float2 t = ffma2(make_float2(sv[2 * c], sv[2 * c + 1]), sl2v, nb);
          const float2 p = make_float2(ex2(t.x), ex2(t.y));
          ls[c & 3] = fadd2(ls[c & 3], p);
          pk[c] = __uint_as_float(pack_bf16(p.x, p.y));
        }
        l += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
        tmem_st32(lane_base + (2 * x + b) * kKeys, pk);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&p_full[x][b]);
      }
      // the segment's partial, once the last P . V is in O
      if (!ok) break;
      if (mine > 0) {
        const int before = done - 1;
        ok = __all_sync(0xffffffffu, wait(&o_done[x][before & 1], (uint32_t)(before >> 1) & 1u, abort, a.pv.err));
        if (!ok) break;
        tc_fence_after_sync();
      }
      int64_t row = ((int64_t)2 * sg.slot + x) * a.chain_rows + r;
      if (!sg.one) {
        if (any_live) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(lane_base + colO + c, o);
            if (live) store_part(a.part_o + row * D + c, o);
          }
        }
        if (live) reinterpret_cast<float2*>(a.part_ml)[row] = make_float2(m_ref, l);
      } else {
        // Two chains of the same rows: each warp learns the other chain's state and writes half of the columns,
        // sum_x O_x 2^(m_x - M).  (The o_done that each waited for, with the fences around the barrier, orders the
        // other chain's products before these loads.)
        if (joined) {  // (a chain without a stage since the last one)
          ok = __all_sync(0xffffffffu, wait(&o_read, (joins - 1u) & 1u, abort, a.pv.err));
          if (!ok) break;
        }
        s_ml[x][r] = make_float2(m_ref, l);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&ml_full);
        ok = __all_sync(0xffffffffu, wait(&ml_full, joins & 1u, abort, a.pv.err));
        if (!ok) break;
        tc_fence_after_sync();
        if (any_live) {
          const float2 e0 = s_ml[0][r], e1 = s_ml[1][r];
          const float M = fmaxf(e0.x, e1.x);
          const float f0 = e0.x == kNegInf ? 0.f : ex2(e0.x - M), f1 = e1.x == kNegInf ? 0.f : ex2(e1.x - M);
          const bool two = sg.stages > 1;  // else chain 1 has no product, and its O is of an earlier segment
          row = (int64_t)2 * sg.slot * a.chain_rows + r;
#pragma unroll 1
          for (int c = x * (D / 2); c < (x + 1) * (D / 2); c += 32) {
            float o[32];
            tmem_ld32(lane_base + K::kColO + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f0;
            if (two) {
              float p[32];
              tmem_ld32(lane_base + K::kColO + D + c, p);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = fmaf(p[k], f1, o[k]);
            }
            if (live) store_part(a.part_o + row * D + c, o);
          }
          if (live && x == 0) reinterpret_cast<float2*>(a.part_ml)[row] = make_float2(M, e0.y * f0 + e1.y * f1);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&o_read);
        ++joins;
        joined = true;
      }
    }
  }

  // teardown: every tensor-memory access has completed (loads waited, the issuers drained)
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, K::kCols);
  }
}

template <int D, int SC, bool Q8>
cudaError_t launch(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas, cudaStream_t st) {
  auto* kernel = shared_tc_kernel<D, SC, Q8>;
  const int smem = Cfg<D, Q8>::smem(a.num_prefixes);
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, Q8>::smem(kMaxPrefixes));
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(Cfg<D, Q8>::kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, *pool_map, *stage_map, a);
}

template <int D, bool Q8>
cudaError_t launch(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas, cudaStream_t st) {
  switch ((a.score.capped ? kCap : kPlain) | (a.score.slopes != nullptr ? kBias : kPlain)) {
    case kPlain: return launch<D, kPlain, Q8>(a, pool_map, stage_map, ctas, st);
    case kCap: return launch<D, kCap, Q8>(a, pool_map, stage_map, ctas, st);
    case kBias: return launch<D, kBias, Q8>(a, pool_map, stage_map, ctas, st);
    default: return launch<D, kCap | kBias, Q8>(a, pool_map, stage_map, ctas, st);
  }
}

}  // namespace
}  // namespace hwkv
