// Stream-K decode attention for 8-bit pools (HWKV_E4M3), optionally fused with the append of the
// step's new token.
//
// "HeadWiseKV: Budgeted Per-Head Cache Residency for Hybrid Long-Context Language Models",
// abstract and section "Grouped-Cache Runtime": attention reads only the materialised window
// of each KV head (the last min(w, len) tokens), through the head's block table.
//
// The line of tiles, its split over the CTAs and the merges are those of hwkv_decode_sk.cuh; the
// tile's mathematics is in hwkv_decode_tile_q8.cuh.  What differs is how tiles reach the warps: an
// 8-bit tile holds half the bytes, so what it costs to find and issue one weighs twice as much, and
// goes to a producer warp (a policy layer of four sequences at 112K: 83 -> 62 us):
//   warp W      producer: 32 tiles of a segment per round, one per lane -- ring slot, table entry
//               (read two rounds ahead), scales (one round ahead) -- then, stage by stage once it is
//               free, the scales stored by their lanes and the TMA copies issued by one;
//   warps 0-2   consumers: a stage holds M consecutive tiles of a segment (32 tokens at head_dim
//               128, 64 at 64: 8 KB), stage n of the CTA goes to warp n % W.
// Stages are handed over by mbarriers: full[] (bytes landed), empty[] (its consumer has read it).
//
// Bound: HBM, with ~8 us per launch that no byte covers (a policy layer of four sequences at 112K: 311 MB
// in 54.5 us, 0.84 of the measured copy rate); at batch 1 the latency of schedule and merges (45 MB in
// 20.9 us).  Waits are bounded (~2 s); a timeout records HWKV_DEVERR_WAIT_TIMEOUT, all roles stop and
// the copies in flight land before the shared memory is released.
#pragma once

#include <atomic>

#include "hwkv_decode_merge.cuh"
#include "hwkv_decode_tile_q8.cuh"

namespace hwkv {
namespace {

// Line positions charged for a group's boundary (see kGapTiles): more than bf16's, as a position
// stands for half the bytes.  Policy layer / 64 ragged sequences at head_dim 64 / batch 1 at 161K:
// 24 55.6 / 54.7 / 21.0 us, 32 54.3 / 53.5 / 22.5, 40 54.1 / 54.4 / 20.8, 48 55.4 / 54.7 / 21.2, 64 55.8 /
// 56.8 / 20.7.
constexpr int kGap = 40;

// Fewest line positions of a CTA: a short line is split over fewer CTAs, as each one more costs the
// groups a partial to publish, count and merge; but a CTA takes ~0.35 us per position.  One sequence
// with windows of 4096 and 1024: 1 16.2 us, 16 13.0, 20 14.0, 32 14.5, 64 17.5; five short sequences:
// 16 15.5 us, 24 17.3, 32 18.1, 64 25.
constexpr int kMinPositions = 16;

template <int D>
struct Q8Cfg {
  // 3 consumers and the producer: with two CTAs per SM a warp may then hold 255 registers, and only 16
  // columns of 128 spill, 12 bytes (4 or 5 consumers: 168, with spills, and slower: policy layer 58.6 -> 62.1 and
  // 59.7 us)
  static constexpr int W = 3;
  static constexpr int kThreads = (W + 1) * 32;
  static constexpr int M = D == 128 ? 2 : 4;          // tiles of a stage
  static constexpr int kTileBytes = 2 * kTile * D;    // K and V codes
  static constexpr int kStageBytes = M * kTileBytes;  // 8 KB
  static constexpr int NS = 9;                        // stages of a CTA (12: batch 1 0.5 us slower)
  static constexpr int kCtas = 2;                     // CTAs per SM
  using Sync = PartSync<W * 32>;
  // A buffer's stages must all go to one warp: it has then seen a buffer's use k before it waits for
  // use k + 1.  Another warp could wait while use k is still landing, and a wait for a phase parity
  // cannot tell use k - 1 from use k + 1.
  static_assert(NS % W == 0, "a stage buffer belongs to one consumer warp");
};

// query heads whose warp states meet in shared memory per merge pass: a whole 8-column n-tile
// (three warps leave the room that four take at head_dim 128)
template <int GP>
__host__ __device__ constexpr int q8_merge_heads() {
  return GP < 8 ? GP : 8;
}

template <int D, int GP>
constexpr int q8_smem_bytes() {
  using Cfg = Q8Cfg<D>;
  return Cfg::NS * Cfg::kStageBytes + Cfg::W * q8_merge_heads<GP>() * D * 4 + 1024;
}

__device__ __forceinline__ void mbar_arrive_one(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Waits for a phase; gives up when another role has (`abort`) or after ~2 s, which it records and
// announces.
__device__ __forceinline__ bool q8_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
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

// The end of a CTA's segment [seg_begin, seg_end) of group sg (whose boundary sits at spre on the
// line of T positions): the consuming warps' states are merged in shared memory (sc_m, sc_l,
// sc_acc) into the group's output, or into this CTA's partial, which the group's last arriver merges with
// the others.  A thread folds four columns at a time: fewer threads than a whole CTA, so a head's weights
// serve four.  `more`: the CTA has another segment; `failed`: this thread's warp gave up a wait.  smem: the
// stage buffers, free after the last segment.
template <int D, int GP, bool kOpen, typename Sync, typename State>
__device__ __forceinline__ void end_segment(const DecodeArgs& a, State& ws, const Group& sgr, int sg, long long spre,
                                            long long seg_begin, long long seg_end, long long T, int nctas, int cta,
                                            bool more, bool failed, uint8_t* smem, float* sc_m, float* sc_l,
                                            float* sc_acc, int* s_last, MergeStage& ms) {
  constexpr int W = Sync::kThreads / 32;
  constexpr int SG = q8_merge_heads<GP>();      // query heads merged per pass
  constexpr int NT = State::NT;                 // 8-column groups of query heads
  constexpr int kPasses = GP < 8 ? 1 : 8 / SG;  // passes per 8-column group
  // the partial merge's (m, l) scratch reuses the warps' merge area: 2 * slots * G floats
  constexpr int kMlCap = W * SG * D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group;
  ws.finish();
  const bool whole = seg_begin == spre + kGap && seg_end == spre + group_span<kGap>(sgr);
  const long long slot = (long long)sg + cta;  // unique per (group, CTA) along the line
  using Out = __nv_bfloat16;
  Out* const out_grp = kOpen ? nullptr : static_cast<Out*>(a.out) + ((int64_t)sgr.s * a.pv.kv_heads + sgr.h) * G * D;
  float* const open_acc = kOpen ? a.open_acc : nullptr;
  float* const open_ml = kOpen ? a.open_ml : nullptr;
  const long long open_slot = kOpen ? sg : 0;
  // pass (nt, hh): the warps' states of query heads [8*nt + hh*SG, 8*nt + (hh+1)*SG) meet in
  // shared memory and are folded into the output or this CTA's partial
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
  for (int hh = 0; hh < kPasses; ++hh) {
    if (nt > 0 || hh > 0) Sync::sync();  // the previous pass has read the scratch
    ws.template publish<SG>(nt, hh, warp, lane, sc_m, sc_l, sc_acc);
    Sync::sync();
    const int g0 = 8 * nt + hh * SG;
    const int ng = min(SG, G - g0);  // real query heads of this pass
    for (int e = threadIdx.x * 4; e < ng * D; e += Sync::kThreads * 4) {
      const int gl = e / D, d = e - (e / D) * D;
      const int g = g0 + gl;
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, sc_m[w * SG + gl]);
      float Ls = 0.f;
      float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
      if (M != kNegInf) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float f = ex2(sc_m[w * SG + gl] - M);
          Ls += sc_l[w * SG + gl] * f;
          const float4 v = *reinterpret_cast<const float4*>(sc_acc + (w * SG + gl) * D + d);
          A.x += v.x * f;
          A.y += v.y * f;
          A.z += v.z * f;
          A.w += v.w * f;
        }
      }
      if (kOpen && whole) store_merged<Out, D>(M, Ls, A, g, d / 4, G, (Out*)nullptr, open_acc, open_ml, open_slot);
      else store_merged<Out, D>(M, Ls, A, g, d / 4, G, whole ? out_grp : nullptr, a.part_acc, a.part_ml, slot);
    }
  }
  if (whole) return;
  // The partial is published; count arrivals.  Up to kFlatMerge contributors: the last
  // CTA of the group merges them all.  More (long windows at small batch): blocks of
  // kMergeBlock consecutive contributors are merged by their last arriver into a second-
  // level partial, and the last of those merges the blocks (one level of ~100 partials,
  // streamed through the stage buffers in chunks by one CTA, was slower at batch 1: 877
  // against 955 tokens/s; it moves ~200 KB through one SM where the tree spreads it).
  // After the last segment no copy is in flight (unless a wait timed out): merges may
  // stage partial blocks in the stage buffers.
  if (!more) ms.buf = Sync::sync_or(failed) ? nullptr : reinterpret_cast<float*>(smem);
  const int c_lo = cta_of(spre + kGap, T, nctas), c_hi = cta_of(spre + group_span<kGap>(sgr) - 1, T, nctas);
  const bool all_live = T >= nctas;  // then no CTA range is empty
  const int k = c_hi - c_lo + 1;
  if (!all_live || k <= kFlatMerge) {
    int expected = k;
    if (!all_live) {
      expected = 0;
      for (int c = c_lo; c <= c_hi; ++c) expected += range_start(T, c + 1, nctas) > range_start(T, c, nctas);
    }
    if (arrive_last<Sync>(&a.counters[sg], expected, s_last)) {
      auto live = [&](int i) {
        return all_live || range_start(T, c_lo + i + 1, nctas) > range_start(T, c_lo + i, nctas);
      };
      merge_slots<Out, D, GP, Sync>(a.part_acc, a.part_ml, (long long)sg + c_lo, k, G, live, all_live, out_grp, open_acc,
                                    open_ml, open_slot, sc_acc, kMlCap, ms, a.pv.err);
    }
  } else {
    auto live = [](int) { return true; };
    const int nb = (k + kMergeBlock - 1) / kMergeBlock;
    const int b = (cta - c_lo) / kMergeBlock;
    const int b_lo = c_lo + b * kMergeBlock;
    const int b_n = min(kMergeBlock, c_hi - b_lo + 1);
    const long long slot2 = (long long)sg * a.merge_blocks + b;
    if (arrive_last<Sync>(&a.counters1[slot2], b_n, s_last)) {
      merge_slots<Out, D, GP, Sync>(a.part_acc, a.part_ml, (long long)sg + b_lo, b_n, G, live, true, (Out*)nullptr,
                                    a.part2_acc, a.part2_ml, slot2, sc_acc, kMlCap, ms, a.pv.err);
      if (arrive_last<Sync>(&a.counters[sg], nb, s_last))
        merge_slots<Out, D, GP, Sync>(a.part2_acc, a.part2_ml, (long long)sg * a.merge_blocks, nb, G, live, true, out_grp,
                                      open_acc, open_ml, open_slot, sc_acc, kMlCap, ms, a.pv.err);
    }
  }
}

// kOpen: as in hwkv_decode_sk.cuh
template <int D, int GP, bool SC, bool kOpen>
__global__ void __launch_bounds__(Q8Cfg<D>::kThreads, Q8Cfg<D>::kCtas)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ DecodeArgs a) {
  using Cfg = Q8Cfg<D>;
  using Sync = typename Cfg::Sync;
  using State = WarpState<E4m3, D, GP, SC>;
  constexpr int W = Cfg::W, M = Cfg::M, NS = Cfg::NS;
  constexpr int SG = q8_merge_heads<GP>();
  constexpr int kThreads = Cfg::kThreads;

  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  float* sc_acc = reinterpret_cast<float*>(smem + NS * Cfg::kStageBytes);  // [W][SG][D]
  __shared__ __align__(8) uint64_t full[NS], empty[NS];
  __shared__ __align__(8) uint64_t merge_bar[2];  // bulk copies of partial blocks
  // scales (K, V) of each stage's tiles.  A round of 32 tiles stores its scales before its stages are
  // free: at most 32 / M stages ahead of one whose buffer, NS stages back, has been read.
  constexpr int kRing = 32;
  static_assert(kRing >= 32 / M + NS, "scales of stages still being read stay");
  __shared__ float2 s_scale[kRing][M];
  __shared__ float sc_m[W * SG], sc_l[W * SG];
  __shared__ long long s_scan[W + 1];
  __shared__ long long s_start[2];
  __shared__ int s_last, s_abort;
  __shared__ int s_lens_buf[kLensCache];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.pv.kv_heads;
  const int B = a.pv.num_seqs;
  const int ngroups = B * H;
  const int cta = blockIdx.x;
  const int G = a.group;

  // the next grid in the stream may start at once (see hwkv_decode_sk.cuh); with a.early the
  // schedule and the loads run before the dependent-launch wait, all else after it
  griddep_launch_dependents();
  if (threadIdx.x == 0) prefetch_tensormap(&tmap);
  if (!kOpen && !a.early) griddep_wait();

  if (cta == 0) {
    for (int s = threadIdx.x; s < B; s += kThreads)
      if (__ldcg(a.lens + s) < 0) atomicOr(a.pv.err, HWKV_DEVERR_NEG_LENGTH);
  }
  const int* s_lens = B <= kLensCache ? s_lens_buf : nullptr;
  if (s_lens != nullptr) {
    for (int s = threadIdx.x; s < B; s += kThreads) s_lens_buf[s] = seq_len(a, s);
    __syncthreads();
  }

  // ---- schedule: needed tiles per group, their prefix sums, this CTA's range ----------
  if (threadIdx.x == 0) {
    s_start[0] = -1;
    s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&merge_bar[0], 1);
    mbar_init(&merge_bar[1], 1);
    fence_mbar_init();
  }
  const int per = (ngroups + kThreads - 1) / kThreads;
  const int g_lo = min(ngroups, (int)threadIdx.x * per), g_hi = min(ngroups, g_lo + per);
  long long mine = 0;
  for (int g = g_lo; g < g_hi; ++g) mine += group_span<kGap>(load_group(a, s_lens, g));
  long long T;
  const long long excl = block_exclusive_scan<W + 1>(mine, s_scan, T);
  const int nctas = (int)min((long long)gridDim.x, max(1LL, T / kMinPositions));  // CTAs with a range
  const long long t_lo = cta < nctas ? range_start(T, cta, nctas) : T;
  const long long t_hi = cta < nctas ? range_start(T, cta + 1, nctas) : T;
  if (t_lo < t_hi && excl <= t_lo && t_lo < excl + mine) {
    long long pre = excl;
    for (int g = g_lo; g < g_hi; ++g) {
      const int c = group_span<kGap>(load_group(a, s_lens, g));
      if (t_lo < pre + c) {
        s_start[0] = g;
        s_start[1] = pre;
        break;
      }
      pre += c;
    }
  }
  __syncthreads();
  // the range holds a tile unless it lies within one group's gap
  const bool has_range =
      t_lo < t_hi && s_start[0] >= 0 && t_hi > (t_lo > s_start[1] + kGap ? t_lo : s_start[1] + kGap);
  volatile int* abort = &s_abort;
  // segment cursor: group, its boundary on the line
  int sg = has_range ? (int)s_start[0] : 0;
  long long spre = has_range ? s_start[1] : 0;
  Group sgr = load_group(a, s_lens, sg);
  // the segment's tiles of the group, [first, first + count); true when another segment follows
  auto segment = [&](int& first, int& count) {
    const long long lo = t_lo > spre + kGap ? t_lo : spre + kGap;
    const long long hi = t_hi < spre + group_span<kGap>(sgr) ? t_hi : spre + group_span<kGap>(sgr);
    first = (int)(lo - spre) - kGap;
    count = (int)(hi - lo);
    return spre + group_span<kGap>(sgr) + kGap < t_hi;
  };
  auto next_segment = [&]() {
    do {
      spre += group_span<kGap>(sgr);
      sgr = load_group(a, s_lens, ++sg);
    } while (sgr.tiles == 0);
  };

  if (warp == W) {
    // ---- producer ----------------------------------------------------------------------
    if (!has_range) return;  // (kOpen: the consumers wait for the grid ahead)
    const uint64_t policy = evict_first_policy();
    const uint32_t sbase = smem_addr(smem);
    int stage = 0;  // stages issued
    bool ok = true;
    struct Look {  // one lane's tile of a round
      int blk, r0;
    };
    for (;;) {
      int first, count;
      const bool more = segment(first, count);
      auto look = [&](int i) {
        Look l{0, 0};
        if (i < count) {
          const int t0 = tile_slot(sgr, first + i);
          const int jb = a.bs_log2 >= 0 ? t0 >> a.bs_log2 : t0 / a.pv.block_size;
          l.blk = __ldcg(sgr.tbl + jb);
          l.r0 = t0 - jb * a.pv.block_size;
        }
        return l;
      };
      auto checked = [&](Look l) {  // a bad entry is flagged and block 0 read, so the barriers stay in step
        if (l.blk < 0 || (int64_t)l.blk >= a.pv.total_blocks) {
          atomicOr(a.pv.err, HWKV_DEVERR_BAD_BLOCK);
          l.blk = 0;
        }
        return l;
      };
      auto scales = [&](Look l) {
        const int64_t group = (int64_t)l.blk * (a.pv.block_size / kScaleGroup) + (l.r0 >> 4);
        return __ldcg(reinterpret_cast<const float2*>(a.pv.scales) + group);
      };
      // One round: the tiles [i0, i0 + 32) in `now`, their scales in `sc`, whose loads were issued a
      // round ago; `next` (two rounds ago) gives the next round's scales, and `after` is looked up.
      // Rounds rotate three register sets by name: a copy between sets would wait for the loads.
      auto round = [&](int i0, const Look& now, const float2& sc, Look& next, float2& sc_next, Look& after) {
        after = look(i0 + 64 + lane);
        next = checked(next);
        sc_next = scales(next);
        const int n = min(32, count - i0);
        if (lane < n) s_scale[(stage + lane / M) % kRing][lane % M] = sc;
        __syncwarp();
        for (int i = 0; i < n; i += M, ++stage) {
          const int st = stage % NS;
          if (stage >= NS) {
            ok = __all_sync(0xffffffffu, q8_wait(&empty[st], (uint32_t)(stage / NS - 1) & 1u, abort, a.pv.err));
            if (!ok) return;
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)min(M, n - i) * Cfg::kTileBytes);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const int blk = __shfl_sync(0xffffffffu, now.blk, i + m), r0 = __shfl_sync(0xffffffffu, now.r0, i + m);
            if (lane == 0 && i + m < n)
              issue_tile_q8<D>(&tmap, blk, r0, sbase + st * Cfg::kStageBytes + m * Cfg::kTileBytes, &full[st], policy);
          }
        }
      };
      Look la = checked(look(lane)), lb = look(32 + lane), lc{0, 0};
      float2 sa = scales(la), sb, sc;
      for (int i0 = 0; ok && i0 < count; i0 += 96) {
        round(i0, la, sa, lb, sb, lc);
        if (!ok || i0 + 32 >= count) break;
        round(i0 + 32, lb, sb, lc, sc, la);
        if (!ok || i0 + 64 >= count) break;
        round(i0 + 64, lc, sc, la, sa, lb);
      }
      if (!ok || !more) break;
      next_segment();
    }
    if (!ok) {  // let the copies in flight land before the shared memory is released
      for (int j = max(0, stage - NS); j < stage; ++j)
        if (!mbar_wait_bounded(&full[j % NS], (uint32_t)(j / NS) & 1u)) break;
    }
    return;
  }

  // ---- consumers -------------------------------------------------------------------------
  if (!kOpen && a.early) griddep_wait();
  // groups with nothing resident (length 0) get a zero output, each from one CTA
  for (int g = cta; g < ngroups; g += (int)gridDim.x) {
    const Group gr = load_group(a, s_lens, g);
    if (gr.tiles == 0) {
      if constexpr (kOpen) {
        for (int e = threadIdx.x; e < G; e += W * 32)
          reinterpret_cast<float2*>(a.open_ml)[(int64_t)g * G + e] = make_float2(kNegInf, 0.f);
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)gr.s * H + gr.h) * G * D;
        for (int e = threadIdx.x; e < G * D; e += W * 32) store_out<__nv_bfloat16>(o + e, 0.f);
      }
    }
  }
  if (!has_range) {
    if constexpr (kOpen) open_end();
    return;
  }

  int stage0 = 0;  // the segment's first stage
  bool ok = true;
  MergeStage ms{nullptr, (uint32_t)(NS * Cfg::kStageBytes), &merge_bar[0], &merge_bar[1], 0u, 0u, -1, -1};
  for (;;) {
    int first, count;
    const bool more = segment(first, count);
    State ws;
    ws.begin(a, sgr, G, lane);
    const int new_slot = a.k_new != nullptr ? (sgr.len - 1) % sgr.rs.C : -1;
    const int nstages = (count + M - 1) / M;
    int k = warp - stage0 % W;
    if (k < 0) k += W;
    for (; ok && k < nstages; k += W) {
      const int n = stage0 + k, st = n % NS;
      ok = __all_sync(0xffffffffu, q8_wait(&full[st], (uint32_t)(n / NS) & 1u, abort, a.pv.err));
      if (!ok) break;
      const int have = min(M, count - k * M);
      int t[M];
      uint32_t sk[M];
      const float2* sl[M];
      bool dirty = false;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        t[m] = tile_slot(sgr, first + k * M + m);
        sk[m] = smem_addr(smem) + st * Cfg::kStageBytes + m * Cfg::kTileBytes;
        sl[m] = &s_scale[n % kRing][m];
        if (m < have && new_slot >= t[m] && new_slot < t[m] + kTile) {
          patch_new_row_q8<D>(a, sgr.tbl, sgr.s, sgr.h, sgr.len - 1, sgr.rs.C, t[m], new_slot, sk[m], &s_scale[n % kRing][m],
                              lane);
          dirty = true;
        }
      }
      if (have == M) {
        if (ws.template consume<M>(a, sgr, t, sk, sl, lane)) dirty = true;
      } else {
        for (int m = 0; m < have; ++m) {
          const int t1[1] = {tile_slot(sgr, first + k * M + m)};
          const uint32_t sk1[1] = {smem_addr(smem) + st * Cfg::kStageBytes + m * Cfg::kTileBytes};
          const float2* sl1[1] = {&s_scale[n % kRing][m]};
          if (ws.template consume<1>(a, sgr, t1, sk1, sl1, lane)) dirty = true;
        }
      }
      if (dirty) fence_proxy_async_smem();  // this lane's shared-memory writes before the next TMA
      __syncwarp();
      if (lane == 0) mbar_arrive_one(&empty[st]);
    }
    const long long seg_begin = spre + kGap + first;
    end_segment<D, GP, kOpen, Sync>(a, ws, sgr, sg, spre, seg_begin, seg_begin + count, T, nctas, cta, more, !ok, smem, sc_m,
                             sc_l, sc_acc, &s_last, ms);
    Sync::sync();  // the merge scratch is rewritten by the next segment
    if (!more) break;
    stage0 += nstages;
    next_segment();
  }
  if (ms.stuck0 >= 0) mbar_wait_bounded(&merge_bar[0], (uint32_t)ms.stuck0);
  if (ms.stuck1 >= 0) mbar_wait_bounded(&merge_bar[1], (uint32_t)ms.stuck1);
  if constexpr (kOpen) open_end();
}

template <int D, int GP, bool SC, bool kOpen = false>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(decode_q8_kernel<D, GP, SC, kOpen>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              q8_smem_bytes<D, GP>());
}

template <int D, int GP>
cudaError_t configure_one(int* ctas_per_sm) {
  const cudaError_t e = prepare_one<D, GP, false>();
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, decode_q8_kernel<D, GP, false, false>, Q8Cfg<D>::kThreads,
                                                       q8_smem_bytes<D, GP>());
}

// Scored and open instances (SC, kOpen) are prepared at their first launch on a device, not with every pool, and
// run on the grid of the plain ones.
template <int D, int GP, bool SC, bool kOpen = false>
cudaError_t launch_one(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if constexpr (SC || kOpen) {
    static std::atomic<uint64_t> prepared{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(prepared.load(std::memory_order_relaxed) & bit)) {
      if ((e = prepare_one<D, GP, SC, kOpen>()) != cudaSuccess) return e;
      prepared.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(Q8Cfg<D>::kThreads);
  cfg.dynamicSmemBytes = q8_smem_bytes<D, GP>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_q8_kernel<D, GP, SC, kOpen>, *tmap, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace hwkv
