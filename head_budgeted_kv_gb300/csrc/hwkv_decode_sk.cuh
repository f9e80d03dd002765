// Stream-K split-K decode attention over per-head paged rings (block_size % 16 == 0, head_dim
// 64 or 128), optionally fused with the append of the step's new token: tile work on the
// tensor cores for bf16 pools (up to 16 query heads per KV head), on the CUDA cores for fp32
// pools (up to 4).  (8-bit pools: hwkv_decode_q8.cuh, the same line of tiles and merges.)
//
// "HeadWiseKV: Budgeted Per-Head Cache Residency for Hybrid Long-Context Language Models",
// abstract and section "Grouped-Cache Runtime": attention reads only the materialised window
// of each KV head (the last min(w, len) tokens), through the head's block table.
//
// Work decomposition ("stream-K"): every (seq, kv head) group contributes the 16-token ring
// tiles that hold resident tokens -- a cyclic run of tiles starting at the tile of the oldest
// resident slot.  Numbering those tiles group after group gives one line of T equal-cost
// tiles; the persistent grid of N CTAs splits it into N equal contiguous ranges, so every
// CTA streams the same number of bytes whatever the windows and lengths are.  A CTA walks its
// range group by group ("segments"); its 4 warps take the segment's tiles round-robin, each
// through its own TMA + mbarrier pipeline that runs on across segment boundaries.  At the end
// of a segment the warps' online-softmax states are merged in shared memory; a group held by
// one CTA is written out directly, otherwise the CTA stores a partial (m, l, acc) and bumps
// the group's arrival counter, and the CTA that arrives last merges all partials of the group
// and writes the output (no CTA ever waits for another).  After a CTA's last tile its stage
// buffers are free, and a merge there fetches the whole partial block with one bulk copy.
// The sequence lengths are staged in shared memory once, so crossing into the next group
// costs no global round trip.
//
// Per tile (16 tokens), per warp, bf16 (hwkv_decode_tile.cuh, consume_tile), with the GQA
// group (G <= 16 query heads, zero-padded to one or two 8-column n-tiles) on the N side of
// mma.sync.m16n8k16 bf16 -> fp32:
//   S[16 tok][8 q] = K_tile . Q^T over head_dim per n-tile (K tile loaded once with ldmatrix
//   from the 128-byte-swizzled TMA tile and shared by the n-tiles), masked to resident slots,
//   online softmax in fp32 in the log2 domain; P is moved from the accumulator layout to the
//   operand layout with movmatrix.trans; O^T[D][8 q] = alpha * O^T + V_tile^T . P (V tile
//   loaded once with ldmatrix.trans).
// fp32 (consume_tile_f32): lanes own consecutive dims; the tile's 16 x 4 dot products are summed
// over the warp by a butterfly transpose-reduction, P goes through shared memory for the FMAs.
//
// Waits are bounded (~2 s); a timeout records HWKV_DEVERR_WAIT_TIMEOUT and the warp stops.
#pragma once

#include <atomic>

#include "hwkv_decode_merge.cuh"

namespace hwkv {
namespace {

// Tiles per warp pulled into L2 while the CTA waits for the preceding grid (early reads only),
// when its range holds at least kL2PrefetchMin positions.  Short ranges (small batches) skip it:
// there the preceding grid's last streams and merges, which the prefetch would slow, are most of
// what the wait is for.  Depth swept on the full geometry with the dependent-launch trigger at
// kernel entry: head_dim 128, 0 -> 957, 2 -> 969, 4 -> 982, 6 -> 989, 8 -> 988 tokens/s; head_dim
// 64 (three CTAs per SM, half the bytes per tile), GQA 4: 0 -> 0.828, 2 -> 0.836, 4 -> 0.819,
// 6 -> 0.807 of the copy peak.
template <int D>
__host__ __device__ constexpr int l2_prefetch() {
  return D == 128 ? 6 : 2;
}
constexpr int kL2PrefetchMin = 64;

// CTAs per SM: bf16 two at head_dim 128, three at 64 (4 stages of half-size tiles fit three in
// shared memory, and the per-tile instruction chain, twice as long per byte there, needs the
// warps); fp32 tiles are twice the bytes: one at 128, two at 64.
template <typename T, int D>
__host__ __device__ constexpr int sk_min_ctas() {
  return sizeof(T) == 2 ? (D == 64 ? 3 : 2) : (D == 64 ? 2 : 1);
}

// kOpen: the results stay open, each group's (m, l) and accumulators to be joined with those of other keys.
// Such a grid needs nothing of the grid ahead of it, which starts it only once all before has completed: its last
// CTA alone waits for that grid, at its end, so that what follows this grid follows both (and the others leave
// their SMs to those still to come).
template <typename Elem, int D, int GP, int NS, bool SC, bool kOpen>
__global__ void __launch_bounds__(kWarps * 32, sk_min_ctas<Elem, D>())
    decode_sk_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ DecodeArgs a) {
  using State = WarpState<Elem, D, GP, SC>;
  constexpr int W = kWarps;
  constexpr int kEB = (int)sizeof(Elem);
  constexpr int kTileBytes = kTile * D * kEB;  // 16 rows
  constexpr int kStageBytes = 2 * kTileBytes;  // K tile + V tile
  constexpr int NT = State::NT;                 // 8-column groups of query heads
  constexpr int SG = merge_heads<D, GP>();      // query heads merged per pass in shared memory
  constexpr int kPasses = GP < 8 ? 1 : 8 / SG;  // passes per 8-column group
  // the partial merge's (m, l) scratch reuses the warps' merge area: 2 * slots * G floats
  constexpr int kMlCap = W * SG * D;

  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  float* sc_acc = reinterpret_cast<float*>(smem + W * NS * kStageBytes);  // [W][SG][D]
  __shared__ __align__(8) uint64_t bars[W * NS];
  __shared__ float sc_m[W * SG], sc_l[W * SG];
  __shared__ __align__(8) uint64_t merge_bar[2];  // bulk copies of partial blocks
  __shared__ long long s_scan[W];
  __shared__ long long s_start[2];
  __shared__ int s_last;
  __shared__ int s_lens_buf[kLensCache];
  __shared__ __align__(16) float s_p[kEB == 4 ? W * 64 : 4];  // fp32 tiles: each warp's P

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.pv.kv_heads;
  const int B = a.pv.num_seqs;
  const int ngroups = B * H;
  const int nctas = gridDim.x, cta = blockIdx.x;
  const int G = a.group;
  const int Hq = H * G;
  const int bs = a.pv.block_size;
  Elem* const out = static_cast<Elem*>(a.out);

  // The next grid in the stream may start at once: its CTAs take the slots this grid's CTAs
  // free, run their own early reads, and wait for this grid before anything else (with the
  // trigger at the end of each CTA's stream instead, they started only after the slowest
  // stream: full workload 961 -> 971 tokens/s, batch 1 unchanged).
  griddep_launch_dependents();
  // the descriptor is a kernel parameter, so it may be fetched before the wait below
  if (threadIdx.x == 0) prefetch_tensormap(&tmap);
  // Launched as a programmatic dependent.  By default everything waits for the grids this one
  // depends on.  With a.early the caller guarantees that the lengths, the block table and this
  // layer's pool were written before the preceding grid in the stream started, so the schedule
  // and the first tile loads run before the wait; q, k_new / v_new and every write of this
  // grid come after it.
  if (!kOpen && !a.early) griddep_wait();

  if (cta == 0) {
    for (int s = threadIdx.x; s < B; s += W * 32)
      if (__ldcg(a.lens + s) < 0) atomicOr(a.pv.err, HWKV_DEVERR_NEG_LENGTH);
  }
  // the lengths are staged once, so crossing into the next group never waits on global memory
  const int* s_lens = B <= kLensCache ? s_lens_buf : nullptr;
  if (s_lens != nullptr) {
    for (int s = threadIdx.x; s < B; s += W * 32) s_lens_buf[s] = seq_len(a, s);
    __syncthreads();
  }

  // ---- schedule: needed tiles per group, their prefix sums, this CTA's range ----------
  if (threadIdx.x == 0) s_start[0] = -1;
  const int per = (ngroups + W * 32 - 1) / (W * 32);
  const int g_lo = min(ngroups, (int)threadIdx.x * per), g_hi = min(ngroups, g_lo + per);
  long long mine = 0;
  for (int g = g_lo; g < g_hi; ++g) mine += group_span(load_group(a, s_lens, g));
  long long T;
  const long long excl = block_exclusive_scan<W>(mine, s_scan, T);
  const long long t_lo = range_start(T, cta, nctas), t_hi = range_start(T, cta + 1, nctas);
  if (t_lo < t_hi && excl <= t_lo && t_lo < excl + mine) {
    long long pre = excl;
    for (int g = g_lo; g < g_hi; ++g) {
      const int c = group_span(load_group(a, s_lens, g));
      if (t_lo < pre + c) {
        s_start[0] = g;
        s_start[1] = pre;
        break;
      }
      pre += c;
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < W * NS; ++i) mbar_init(&bars[i], 1);
    mbar_init(&merge_bar[0], 1);
    mbar_init(&merge_bar[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  // the range holds a tile unless it lies within one group's gap
  const bool has_range =
      t_lo < t_hi && s_start[0] >= 0 && t_hi > (t_lo > s_start[1] + kGapTiles ? t_lo : s_start[1] + kGapTiles);
  const int g_start = has_range ? (int)s_start[0] : 0;
  const long long pre_start = has_range ? s_start[1] : 0;

  // ---- per-warp TMA pipeline ---------------------------------------------------------
  uint64_t* wbar = bars + warp * NS;
  const uint32_t wstage = smem_addr(smem + warp * NS * kStageBytes);
  const uint64_t policy = evict_first_policy();

  int ig = g_start;            // issue cursor: group, its first tile on the line, the group
  long long ipre = pre_start;
  Group igr = load_group(a, s_lens, ig);
  long long j_issue = t_lo + warp;
  int issued = 0;
  auto issue_next = [&](int issuer) {
    // this warp's next position that holds a tile: past a group's end go to the next group,
    // within its gap step on; nothing is issued once the range is done
    for (;;) {
      if (j_issue >= t_hi) return;
      if (j_issue >= ipre + group_span(igr)) {
        ipre += group_span(igr);
        igr = load_group(a, s_lens, ++ig);
      } else if (j_issue < ipre + kGapTiles) {
        j_issue += W;
      } else {
        break;
      }
    }
    if (lane == issuer) {
      const int st = issued % NS;
      // the first stages may be issued before the dependent-launch wait: read through L2
      issue_tile<kEB, D>(&tmap, a, igr, tile_slot(igr, j_issue - ipre - kGapTiles), wstage + st * kStageBytes,
                         &wbar[st], policy, issued < NS);
    }
    j_issue += W;
    ++issued;
  };
  // the first stages are issued by different lanes so their table lookups overlap
  if (has_range)
    for (int i = 0; i < NS && j_issue < t_hi; ++i) issue_next(i);
  if (!kOpen && a.early && has_range && lane < l2_prefetch<D>() && t_hi - t_lo >= kL2PrefetchMin) {
    // Until the wait below ends, the preceding grid only merges and completes and the memory
    // system is nearly idle: pull the tiles this warp takes after its staged ones into L2
    // (lane i: the position i steps on; a position inside a gap is skipped).
    const long long p = j_issue + (long long)lane * W;
    if (p < t_hi) {
      int g = ig;
      long long pre = ipre;
      Group gr = igr;
      while (p >= pre + group_span(gr)) {
        pre += group_span(gr);
        gr = load_group(a, s_lens, ++g);
      }
      if (p >= pre + kGapTiles) {
        const int t0 = tile_slot(gr, p - pre - kGapTiles);
        const int jb = t0 / bs;
        const int32_t blk = __ldcg(gr.tbl + jb);
        if (blk >= 0 && (int64_t)blk < a.pv.total_blocks) {
          const char* rows = static_cast<const char*>(a.pv.pool) + ((int64_t)blk * 2 * bs + (t0 - jb * bs)) * D * kEB;
          prefetch_l2_bulk(rows, kTileBytes);                         // K rows of the tile
          prefetch_l2_bulk(rows + (int64_t)bs * D * kEB, kTileBytes);  // V rows
        }
      }
    }
  }
  if (!kOpen && a.early) griddep_wait();
  // groups with nothing resident (length 0) get a zero output, each from one CTA
  for (int g = cta; g < ngroups; g += nctas) {
    const Group gr = load_group(a, s_lens, g);
    if (gr.tiles == 0) {
      if constexpr (kOpen) {
        for (int e = threadIdx.x; e < G; e += W * 32)
          reinterpret_cast<float2*>(a.open_ml)[(int64_t)g * G + e] = make_float2(kNegInf, 0.f);
      } else {
        for (int e = threadIdx.x; e < G * D; e += W * 32)
          store_out<Elem>(out + ((int64_t)gr.s * Hq + gr.h * G + e / D) * D + e % D, 0.f);
      }
    }
  }
  if (!has_range) {
    if constexpr (kOpen) open_end();
    return;
  }

  int sg = g_start;            // segment cursor (uniform in the CTA)
  long long spre = pre_start;
  Group sgr = load_group(a, s_lens, sg);
  long long j_cons = t_lo + warp;
  int consumed = 0;
  int drain_from = -1;         // set when a wait timed out
  bool patched_stage = false;  // a generic-proxy write went into the stage just released
  MergeStage ms{nullptr, (uint32_t)(W * NS * kStageBytes), &merge_bar[0], &merge_bar[1], 0u, 0u, -1, -1};

  for (;;) {
    // the segment: the group's tiles within the range
    const long long seg_begin = t_lo > spre + kGapTiles ? t_lo : spre + kGapTiles;
    const long long seg_end = t_hi < spre + group_span(sgr) ? t_hi : spre + group_span(sgr);
    // another segment follows when the next group's first tile is within the range
    const bool more = spre + group_span(sgr) + kGapTiles < t_hi;
    while (j_cons < seg_begin) j_cons += W;  // over the group's gap

    State ws;
    ws.begin(a, sgr, G, lane);
    const int new_slot = (a.k_new != nullptr) ? (sgr.len - 1) % sgr.rs.C : -1;

    while (j_cons < seg_end) {
      const int st = consumed % NS;
      if (drain_from < 0 && !mbar_wait_bounded(&wbar[st], (uint32_t)(consumed / NS) & 1u)) {
        drain_from = consumed;
        if (lane == 0) atomicOr(a.pv.err, HWKV_DEVERR_WAIT_TIMEOUT);
      }
      if (drain_from < 0) {
        const uint32_t sK = wstage + st * kStageBytes;
        const int t0 = tile_slot(sgr, j_cons - spre - kGapTiles);
        if (ws.consume(a, sgr, t0, new_slot, sK, sK + kTileBytes, s_p + warp * 64, lane)) patched_stage = true;
      }
      __syncwarp();
      ++consumed;
      if (drain_from < 0 && j_issue < t_hi) {
        if (patched_stage) {  // every lane orders its shared-memory writes before the next TMA
          fence_proxy_async_smem();
          __syncwarp();
        }
        issue_next(0);
      }
      patched_stage = false;
      j_cons += W;
    }

    // ---- end of segment: merge the warps, then store output or partial -----------------
    // (in place: as functions shared with the 8-bit kernel the fold cost batch 1 0.5% and what follows
    // it fp32 pools 1%)
    ws.finish();
    const bool whole = seg_begin == spre + kGapTiles && seg_end == spre + group_span(sgr);
    const long long slot = (long long)sg + cta;  // unique per (group, CTA) along the line
    // pass (nt, hh): the warps' states of query heads [8*nt + hh*SG, 8*nt + (hh+1)*SG) meet in
    // shared memory and are folded into the output or this CTA's partial
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int hh = 0; hh < kPasses; ++hh) {
      if (nt > 0 || hh > 0) __syncthreads();  // the previous pass has read the scratch
      ws.template publish<SG>(nt, hh, warp, lane, sc_m, sc_l, sc_acc);
      __syncthreads();
      const int g0 = 8 * nt + hh * SG;
      const int ng = min(SG, G - g0);  // real query heads of this pass
      for (int e = threadIdx.x; e < ng * D; e += W * 32) {
        const int gl = e / D, d = e - (e / D) * D;
        const int g = g0 + gl;
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sc_m[w * SG + gl]);
        float Ls = 0.f, A = 0.f;
        if (M != kNegInf) {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float f = ex2(sc_m[w * SG + gl] - M);
            Ls += sc_l[w * SG + gl] * f;
            A += sc_acc[(w * SG + gl) * D + d] * f;
          }
        }
        if (kOpen && whole) {
          a.open_acc[((int64_t)sg * G + g) * D + d] = A;
          if (d == 0) reinterpret_cast<float2*>(a.open_ml)[(int64_t)sg * G + g] = make_float2(M, Ls);
        } else if (whole) {
          store_out<Elem>(out + ((int64_t)sgr.s * Hq + sgr.h * G + g) * D + d, Ls > 0.f ? A / Ls : 0.f);
        } else {
          a.part_acc[(slot * G + g) * D + d] = A;
          if (d == 0) {
            a.part_ml[(slot * G + g) * 2 + 0] = M;
            a.part_ml[(slot * G + g) * 2 + 1] = Ls;
          }
        }
      }
    }
    if (!whole) {
      // The partial is published; count arrivals.  Up to kFlatMerge contributors: the last
      // CTA of the group merges them all.  More (long windows at small batch): blocks of
      // kMergeBlock consecutive contributors are merged by their last arriver into a second-
      // level partial, and the last of those merges the blocks (one level of ~100 partials,
      // streamed through the stage buffers in chunks by one CTA, was slower at batch 1: 877
      // against 955 tokens/s; it moves ~200 KB through one SM where the tree spreads it).
      // After the last segment no copy is in flight (unless a wait timed out): merges may
      // stage partial blocks in the stage buffers.
      if (!more) ms.buf = __syncthreads_or(drain_from >= 0) ? nullptr : reinterpret_cast<float*>(smem);
      const int c_lo = cta_of(spre + kGapTiles, T, nctas), c_hi = cta_of(spre + group_span(sgr) - 1, T, nctas);
      const bool all_live = T >= nctas;  // then no CTA range is empty
      const int k = c_hi - c_lo + 1;
      Elem* const out_grp = kOpen ? nullptr : out + ((int64_t)sgr.s * Hq + sgr.h * G) * D;
      float* const open_acc = kOpen ? a.open_acc : nullptr;
      float* const open_ml = kOpen ? a.open_ml : nullptr;
      const long long open_slot = kOpen ? sg : 0;
      if (!all_live || k <= kFlatMerge) {
        int expected = k;
        if (!all_live) {
          expected = 0;
          for (int c = c_lo; c <= c_hi; ++c) expected += range_start(T, c + 1, nctas) > range_start(T, c, nctas);
        }
        if (arrive_last<CtaSync>(&a.counters[sg], expected, &s_last)) {
          auto live = [&](int i) {
            return all_live || range_start(T, c_lo + i + 1, nctas) > range_start(T, c_lo + i, nctas);
          };
          merge_slots<Elem, D, GP, CtaSync>(a.part_acc, a.part_ml, (long long)sg + c_lo, k, G, live, all_live, out_grp, open_acc,
                         open_ml, open_slot, sc_acc, kMlCap, ms, a.pv.err);
        }
      } else {
        auto live = [](int) { return true; };
        const int nb = (k + kMergeBlock - 1) / kMergeBlock;
        const int b = (cta - c_lo) / kMergeBlock;
        const int b_lo = c_lo + b * kMergeBlock;
        const int b_n = min(kMergeBlock, c_hi - b_lo + 1);
        const long long slot2 = (long long)sg * a.merge_blocks + b;
        if (arrive_last<CtaSync>(&a.counters1[slot2], b_n, &s_last)) {
          merge_slots<Elem, D, GP, CtaSync>(a.part_acc, a.part_ml, (long long)sg + b_lo, b_n, G, live, true, (Elem*)nullptr, a.part2_acc,
                         a.part2_ml, slot2, sc_acc, kMlCap, ms, a.pv.err);
          if (arrive_last<CtaSync>(&a.counters[sg], nb, &s_last))
            merge_slots<Elem, D, GP, CtaSync>(a.part2_acc, a.part2_ml, (long long)sg * a.merge_blocks, nb, G, live, true, out_grp,
                           open_acc, open_ml, open_slot, sc_acc, kMlCap, ms, a.pv.err);
        }
      }
    }
    __syncthreads();  // the merge scratch is rewritten by the next segment
    if (!more) break;
    do {
      spre += group_span(sgr);
      sgr = load_group(a, s_lens, ++sg);
    } while (sgr.tiles == 0);
  }

  if (drain_from >= 0) {
    // let copies still in flight land before the shared memory is released
    for (int c = drain_from; c < issued; ++c)
      if (!mbar_wait_bounded(&wbar[c % NS], (uint32_t)(c / NS) & 1u)) break;
  }
  if (ms.stuck0 >= 0) mbar_wait_bounded(&merge_bar[0], (uint32_t)ms.stuck0);
  if (ms.stuck1 >= 0) mbar_wait_bounded(&merge_bar[1], (uint32_t)ms.stuck1);
  if constexpr (kOpen) open_end();
}

template <typename T, int D, int GP, int NS>
constexpr int sk_smem_bytes() {
  // stages + merge scratch (merge_heads query heads per pass) + align slack
  return kWarps * NS * (2 * kTile * D * (int)sizeof(T)) + kWarps * merge_heads<D, GP>() * D * 4 + 1024;
}

// pipeline depth: bf16 3 (head_dim 128) or 4 (head_dim 64) stages of 16 tokens per warp; at 64
// the same bytes stay in flight per SM with three CTAs (4 stages: D64 decode 0.75 -> 0.81 of
// the copy peak against 6 stages and two CTAs).  fp32: 3 stages (192 KB at 128, one CTA per
// SM; 96 KB at 64, two).
template <typename T, int D>
constexpr int stages() {
  return sizeof(T) == 2 && D == 64 ? 4 : 3;
}

template <typename T, int D, int GP>
cudaError_t configure_one(int* ctas_per_sm) {
  constexpr int NS = stages<T, D>();
  cudaError_t e = cudaFuncSetAttribute(decode_sk_kernel<T, D, GP, NS, false, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, sk_smem_bytes<T, D, GP, NS>());
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, decode_sk_kernel<T, D, GP, NS, false, false>, kWarps * 32,
                                                       sk_smem_bytes<T, D, GP, NS>());
}

// Scored and open instances (SC, kOpen) are prepared at their first launch on a device, not with every pool, and
// run on the grid of the plain ones.
template <typename T, int D, int GP, bool SC = false, bool kOpen = false>
cudaError_t launch_one(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  constexpr int NS = stages<T, D>();
  if constexpr (SC || kOpen) {
    static std::atomic<uint64_t> prepared{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(prepared.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(decode_sk_kernel<T, D, GP, NS, SC, kOpen>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sk_smem_bytes<T, D, GP, NS>());
      if (e != cudaSuccess) return e;
      prepared.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  // programmatic dependent launch: the CTAs may become resident while the previous kernel in
  // the stream finishes; they wait for it (griddepcontrol.wait) before reading anything
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = sk_smem_bytes<T, D, GP, NS>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_sk_kernel<T, D, GP, NS, SC, kOpen>, *tmap, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace hwkv
