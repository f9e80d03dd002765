// The line of tiles the stream-K decode kernels split over their CTAs, and the merges of the
// partial results (hwkv_decode_sk.cuh for bf16 and fp32 pools, hwkv_decode_q8.cuh for 8-bit ones).
#pragma once

#include "hwkv_decode_tile.cuh"

namespace hwkv {
namespace {

constexpr int kFlatMerge = 24;  // most contributors one CTA merges directly

// Line positions charged for each group's boundary.  A group with tiles spans kGapTiles
// positions that hold no tile, then its tiles; a CTA whose range takes in a group's start thus
// streams kGapTiles fewer tiles, which pays for what a boundary costs it (the warps' merge,
// publishing a partial, the next group's q), so CTAs with boundaries do not end last.
constexpr int kGapTiles = 24;

// The end of a CTA of an open instance (hwkv_decode_sk.cuh)
__device__ __forceinline__ void open_end() {
  if (blockIdx.x == gridDim.x - 1) griddep_wait();
}

// The threads that merge: the whole CTA, or its first N threads (those that consumed the tiles)
// while a producer warp runs on.  Thread indices count from 0 in both.  A whole CTA's number is read at
// run time: given the constant the compiler unrolls the merges' loops, and the longer kernel costs batch 1 1%.
struct CtaSync {
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMergeCols = kThreads;  // most 4-float columns a head pass of a merge sums
  static __device__ __forceinline__ unsigned threads() { return blockDim.x; }
  static __device__ __forceinline__ void sync() { __syncthreads(); }
  static __device__ __forceinline__ bool sync_and(bool p) { return __syncthreads_and(p) != 0; }
  static __device__ __forceinline__ bool sync_or(bool p) { return __syncthreads_or(p) != 0; }
};

template <int N>
struct PartSync {
  static constexpr int kThreads = N;
  // a pass may hold more columns than threads: half the heads a pass would double the passes' round
  // trips (96 threads, 16 query heads of 128: 85 -> 80 us for a policy layer of 8-bit pools)
  static constexpr int kMergeCols = (N + 127) / 128 * 128;
  static __device__ __forceinline__ unsigned threads() { return N; }
  static __device__ __forceinline__ void sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory"); }
  static __device__ __forceinline__ bool sync_and(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p), "n"(N)
        : "memory");
    return r != 0;
  }
  static __device__ __forceinline__ bool sync_or(bool p) { return !sync_and(!p); }
};

// line positions of a group whose boundary is charged Gap of them
template <int Gap = kGapTiles>
__device__ __forceinline__ int group_span(const Group& gr) {
  return gr.tiles > 0 ? gr.tiles + Gap : 0;
}

// Writes a merged (M, L, acc) of query head q, columns 4*d4 .. 4*d4 + 3: normalised to the
// output `out_grp` (bf16 or fp32) when it is non-null, else unnormalised to partial slot `dst_slot`.
template <typename T, int D>
__device__ __forceinline__ void store_merged(float M, float L, float4 acc, int q, int d4, int G, T* out_grp,
                                             float* dst_acc, float* dst_ml, long long dst_slot) {
  if (out_grp != nullptr) {
    const float inv = L > 0.f ? 1.f / L : 0.f;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(out_grp + (int64_t)q * D + d4 * 4) =
          make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      uint2 packed;
      packed.x = *reinterpret_cast<uint32_t*>(&lo);
      packed.y = *reinterpret_cast<uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(out_grp + (int64_t)q * D + d4 * 4) = packed;
    }
  } else {
    const long long slot = dst_slot * G + q;
    reinterpret_cast<float4*>(dst_acc + slot * D)[d4] = acc;
    if (d4 == 0) reinterpret_cast<float2*>(dst_ml)[slot] = make_float2(M, L);
  }
}
// Folds `count` consecutive partial slots [first, first + count) of a partial buffer out of
// registers, with exactly the arithmetic of the shared-memory merge below: first the maximum
// M = max_i m_i, then, slot after slot, w_i = 2^(m_i - M), L = fma(l_i, w_i, L) and
// acc = fma(acc_i, w_i, acc).  Whichever path a group's last arriver takes, the output is the
// same bit for bit.  Each thread owns 4 consecutive output columns of one query head and keeps
// 8 slots' loads in flight.  Output as store_merged.  `live(i)` tells whether slot first + i
// holds a partial.
template <typename T, int D, typename Sync, typename Live>
__device__ __forceinline__ void merge_slots_regs(const float* src_acc, const float* src_ml, long long first,
                                                 int count, int G, Live live, T* out_grp,
                                                 float* dst_acc, float* dst_ml, long long dst_slot) {
  constexpr int kV = D / 4;  // float4 columns per query head
  constexpr int kBatch = 8;
  for (int e = threadIdx.x; e < G * kV; e += Sync::threads()) {
    const int q = e / kV, d4 = e - (e / kV) * kV;
    float M = kNegInf;
    for (int i0 = 0; i0 < count; i0 += kBatch) {
      float m[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j;
        m[j] = i < count && live(i) ? __ldcg(src_ml + ((first + i) * G + q) * 2) : kNegInf;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) M = fmaxf(M, m[j]);
    }
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < count; i0 += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j;
        if (i < count && live(i)) {
          const long long slot = (first + i) * G + q;
          ml[j] = __ldcg(reinterpret_cast<const float2*>(src_ml) + slot);
          v[j] = __ldcg(reinterpret_cast<const float4*>(src_acc + slot * D) + d4);
        } else {
          ml[j] = make_float2(kNegInf, 0.f);
          v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (i0 + j < count && live(i0 + j)) {
          const float w = M == kNegInf ? 0.f : ex2(ml[j].x - M);
          L = fmaf(ml[j].y, w, L);
          acc.x = fmaf(v[j].x, w, acc.x);
          acc.y = fmaf(v[j].y, w, acc.y);
          acc.z = fmaf(v[j].z, w, acc.z);
          acc.w = fmaf(v[j].w, w, acc.w);
        }
      }
    }
    store_merged<T, D>(M, L, acc, q, d4, G, out_grp, dst_acc, dst_ml, dst_slot);
  }
}
constexpr uint32_t kBulkChunk = 16384;  // bytes per bulk copy of a partial block

// Shared-memory resources a merge may use: the stage buffers (free once the CTA has consumed
// its last tile), two mbarriers for bulk copies into them and the phases they are at.
struct MergeStage {
  float* buf;               // null: not available
  uint32_t bytes;
  uint64_t* bar0;           // copies into the whole buffer or its first half ...
  uint64_t* bar1;           // ... and into its second half
  uint32_t phase0, phase1;  // completed uses of bar0 / bar1 (uniform in the CTA)
  int stuck0, stuck1;       // parity of a use that may still be in flight after a timeout, else -1
};

// Folds `count` consecutive partial slots [first, first + count) into the output or partial
// slot of store_merged.  When every slot holds a partial (`dense`), the stage buffers are free
// and the accumulators fit them and the (m, l) of every (slot, head) fit `s_ml` (2 * count * G
// <= ml_cap floats), the accumulators are fetched in one bulk copy while those (m, l) are read
// into `s_ml`; each thread then forms its head's maximum M = max_i m_i and, slot after slot,
// w_i = 2^(m_i - M), L = fma(l_i, w_i, L) and the sum of w_i * acc_i over its 4 columns out of
// shared memory (the threads of a warp share a head, so the reads are broadcasts).  The whole
// merge waits for about one round trip to L2.  Otherwise the register merge above runs, with
// the same arithmetic, so an output does not depend on which path its last arriver took.
// `live(i)` tells whether slot first + i holds a partial.
template <typename T, int D, typename Sync, typename Live>
__device__ __forceinline__ void merge_slots_one(const float* src_acc, const float* src_ml, long long first, int count,
                                            int G, Live live, bool dense, T* out_grp, float* dst_acc,
                                            float* dst_ml, long long dst_slot, float* s_ml, int ml_cap,
                                            MergeStage& ms, int32_t* err) {
  const uint32_t bytes = (uint32_t)count * (uint32_t)G * D * 4u;
  if (!dense || ms.buf == nullptr || 2 * count * G > ml_cap || bytes > ms.bytes) {
    merge_slots_regs<T, D, Sync>(src_acc, src_ml, first, count, G, live, out_grp, dst_acc, dst_ml, dst_slot);
    return;
  }
  if (threadIdx.x == 0) {
    // the partials were written and acquired, and the buffer last read, through the generic proxy
    fence_proxy_async_all();
    mbar_arrive_expect_tx(ms.bar0, bytes);
    const char* src = reinterpret_cast<const char*>(src_acc + first * G * D);
    for (uint32_t off = 0; off < bytes; off += kBulkChunk)
      bulk_load(smem_addr(ms.buf) + off, src + off, bytes - off < kBulkChunk ? bytes - off : kBulkChunk, ms.bar0);
  }
  for (int p = threadIdx.x; p < count * G; p += Sync::threads()) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(src_ml) + first * G + p);
    s_ml[p] = ml.x;
    s_ml[count * G + p] = ml.y;
  }
  Sync::sync();
  const bool landed = mbar_wait_bounded(ms.bar0, ms.phase0 & 1u);
  ++ms.phase0;
  if (!landed && threadIdx.x == 0) atomicOr(err, HWKV_DEVERR_WAIT_TIMEOUT);
  constexpr int kV = D / 4;  // float4 columns per query head
  const float4* sacc = reinterpret_cast<const float4*>(ms.buf);
  for (int e = threadIdx.x; e < G * kV; e += Sync::threads()) {
    const int q = e / kV, d4 = e - (e / kV) * kV;
    float M = kNegInf;
    for (int i = 0; i < count; ++i) M = fmaxf(M, s_ml[i * G + q]);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < count; ++i) {
      const float w = M == kNegInf ? 0.f : ex2(s_ml[i * G + q] - M);
      L = fmaf(s_ml[count * G + i * G + q], w, L);
      if (landed) {
        const float4 v = sacc[(i * G + q) * kV + d4];
        acc.x = fmaf(v.x, w, acc.x);
        acc.y = fmaf(v.y, w, acc.y);
        acc.z = fmaf(v.z, w, acc.z);
        acc.w = fmaf(v.w, w, acc.w);
      }
    }
    store_merged<T, D>(M, L, acc, q, d4, G, out_grp, dst_acc, dst_ml, dst_slot);
  }
  if (!landed) {  // a copy may still be in flight: no later merge reuses the buffer
    ms.stuck0 = (int)((ms.phase0 - 1u) & 1u);
    ms.buf = nullptr;
  }
}

// Folds `count` consecutive partial slots [first, first + count) into the output or partial
// slot of store_merged.  When every slot holds a partial (`dense`), the stage buffers are free
// and the accumulators fit them and the (m, l) of every (slot, head) fit `s_ml` (2 * count * G
// <= ml_cap floats), the accumulators are fetched in one bulk copy while those (m, l) are read
// into `s_ml`; each thread then forms its head's maximum M = max_i m_i and, slot after slot,
// w_i = 2^(m_i - M), L = fma(l_i, w_i, L) and the sum of w_i * acc_i over its 4 columns out of
// shared memory (the threads of a warp share a head, so the reads are broadcasts).  The whole
// merge waits for about one round trip to L2.  Accumulators larger than the buffers (large GQA
// groups: 8 KB per partial at 16 query heads) are merged in passes over subsets of the query
// heads, one bulk copy per slot and pass, the next pass landing in one half of the buffers
// while the previous one is summed out of the other.  Otherwise the register merge above runs.
// Every path has the same arithmetic, so an output does not depend on which one its last
// arriver took.  `live(i)` tells whether slot first + i holds a partial.
template <typename T, int D, typename Sync, typename Live>
__device__ __forceinline__ void merge_slots_passes(const float* src_acc, const float* src_ml, long long first, int count,
                                            int G, Live live, bool dense, T* out_grp, float* dst_acc,
                                            float* dst_ml, long long dst_slot, float* s_ml, int ml_cap,
                                            MergeStage& ms, int32_t* err) {
  constexpr int kV = D / 4;  // float4 columns per query head
  const uint32_t bytes = (uint32_t)count * (uint32_t)G * D * 4u;
  const bool one = bytes <= ms.bytes;
  // heads per pass when the accumulators exceed the buffers: the largest power of two dividing
  // G whose pass fits half the buffers and whose columns Sync allows
  int hp = one ? G : 0;
  if (!one)
    for (int h = G; h >= 1; h >>= 1)
      if (G % h == 0 && (uint32_t)count * (uint32_t)h * D * 4u <= ms.bytes / 2u && h * kV <= Sync::kMergeCols) {
        hp = h;
        break;
      }
  if (!dense || ms.buf == nullptr || 2 * count * G > ml_cap || hp == 0) {
    merge_slots_regs<T, D, Sync>(src_acc, src_ml, first, count, G, live, out_grp, dst_acc, dst_ml, dst_slot);
    return;
  }
  const int passes = G / hp;
  const uint32_t pass_bytes = (uint32_t)count * (uint32_t)hp * D * 4u;
  // pass p: heads [p hp, (p + 1) hp) of every slot, into half p % 2 (the whole buffer with one pass)
  auto issue = [&](int p) {
    uint64_t* bar = (p & 1) ? ms.bar1 : ms.bar0;
    // the partials were written and acquired, and the buffer last read, through the generic proxy
    fence_proxy_async_all();
    mbar_arrive_expect_tx(bar, pass_bytes);
    const uint32_t dst = smem_addr(ms.buf) + (uint32_t)(p & 1) * (ms.bytes / 2u);
    if (one) {
      const char* src = reinterpret_cast<const char*>(src_acc + first * G * D);
      for (uint32_t off = 0; off < pass_bytes; off += kBulkChunk)
        bulk_load(dst + off, src + off, pass_bytes - off < kBulkChunk ? pass_bytes - off : kBulkChunk, bar);
    } else {
      const uint32_t row = (uint32_t)hp * D * 4u;
      for (int i = 0; i < count; ++i)
        bulk_load(dst + (uint32_t)i * row, src_acc + ((first + i) * G + (long long)p * hp) * D, row, bar);
    }
  };
  const uint32_t base0 = ms.phase0, base1 = ms.phase1;
  if (threadIdx.x == 0) {
    issue(0);
    if (passes > 1) issue(1);
  }
  for (int p = threadIdx.x; p < count * G; p += Sync::threads()) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(src_ml) + first * G + p);
    s_ml[p] = ml.x;
    s_ml[count * G + p] = ml.y;
  }
  Sync::sync();
  ms.phase0 = base0 + (uint32_t)((passes + 1) / 2);
  ms.phase1 = base1 + (uint32_t)(passes / 2);
  // the weighted sum of heads [p hp, (p + 1) hp) out of the buffer half holding pass p
  auto sum_pass = [&](int p, bool landed) {
    const float4* sacc = reinterpret_cast<const float4*>(ms.buf) + (size_t)(p & 1) * (ms.bytes / 32u);
    for (int e = threadIdx.x; e < hp * kV; e += Sync::threads()) {
      const int ql = e / kV, d4 = e - (e / kV) * kV;
      const int q = p * hp + ql;
      float M = kNegInf;
      for (int i = 0; i < count; ++i) M = fmaxf(M, s_ml[i * G + q]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < count; ++i) {
        const float w = M == kNegInf ? 0.f : ex2(s_ml[i * G + q] - M);
        L = fmaf(s_ml[count * G + i * G + q], w, L);
        if (landed) {
          const float4 v = sacc[(i * hp + ql) * kV + d4];
          acc.x = fmaf(v.x, w, acc.x);
          acc.y = fmaf(v.y, w, acc.y);
          acc.z = fmaf(v.z, w, acc.z);
          acc.w = fmaf(v.w, w, acc.w);
        }
      }
      store_merged<T, D>(M, L, acc, q, d4, G, out_grp, dst_acc, dst_ml, dst_slot);
    }
  };
  if (one) {  // every thread waits for the one copy itself: no CTA barrier on the merge chain
    const bool landed = mbar_wait_bounded(ms.bar0, base0 & 1u);
    if (!landed && threadIdx.x == 0) atomicOr(err, HWKV_DEVERR_WAIT_TIMEOUT);
    sum_pass(0, landed);
    if (!landed) {  // a copy may still be in flight: no later merge reuses the buffer
      ms.stuck0 = (int)(base0 & 1u);
      ms.buf = nullptr;
    }
    return;
  }
  bool ok = true;
  for (int p = 0; p < passes; ++p) {
    const int h = p & 1;
    const uint32_t parity = ((h ? base1 : base0) + (uint32_t)(p >> 1)) & 1u;
    ok = Sync::sync_and(ok && mbar_wait_bounded(h ? ms.bar1 : ms.bar0, parity));
    sum_pass(p, ok);
    if (!ok) {  // copies of this and the next pass may still be in flight: no later merge reuses the buffer
      if (threadIdx.x == 0) atomicOr(err, HWKV_DEVERR_WAIT_TIMEOUT);
      const int next = p + 1 < passes ? (int)(((h ? base0 : base1) + (uint32_t)((p + 1) >> 1)) & 1u) : -1;
      if (h) {
        ms.stuck1 = (int)parity;
        ms.stuck0 = next;
      } else {
        ms.stuck0 = (int)parity;
        ms.stuck1 = next;
      }
      ms.buf = nullptr;
      break;
    }
    Sync::sync();  // half h is read: the copy of pass p + 2 may land there
    if (threadIdx.x == 0 && p + 2 < passes) issue(p + 2);
  }
}

// The merge of a group's partials: instances holding 16 query-head columns may meet partials
// larger than the stage buffers and take the head-pass merge; the others the one-copy merge.
template <typename T, int D, int GP, typename Sync, typename Live>
__device__ __forceinline__ void merge_slots(const float* src_acc, const float* src_ml, long long first, int count,
                                            int G, Live live, bool dense, T* out_grp, float* dst_acc,
                                            float* dst_ml, long long dst_slot, float* s_ml, int ml_cap,
                                            MergeStage& ms, int32_t* err) {
  if constexpr (GP == 16)
    merge_slots_passes<T, D, Sync>(src_acc, src_ml, first, count, G, live, dense, out_grp, dst_acc, dst_ml, dst_slot, s_ml,
                             ml_cap, ms, err);
  else
    merge_slots_one<T, D, Sync>(src_acc, src_ml, first, count, G, live, dense, out_grp, dst_acc, dst_ml, dst_slot, s_ml,
                          ml_cap, ms, err);
}

// Bumps an arrival counter and tells the whole CTA whether it arrived last; the last arriver
// resets the counter to 0 for the next launch.  Call after the CTA's partial is written (by any
// of its threads): the barrier orders those writes before thread 0's atomic, whose release
// half makes them visible device-wide before the count moves, and whose acquire half (with
// the second barrier) lets the last arriver's threads read every other contributor's partial.
template <typename Sync>
__device__ __forceinline__ bool arrive_last(uint32_t* counter, int expected, int* s_flag) {
  Sync::sync();
  if (threadIdx.x == 0) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    *s_flag = old + 1u == (unsigned)expected;
    if (*s_flag) *counter = 0u;
  }
  Sync::sync();
  return *s_flag != 0;
}

// Query heads whose warp states meet in shared memory per merge pass: a whole 8-column n-tile,
// except at head_dim 128 with 8 or 16 columns, where passes of 4 keep the scratch at 8 KB so two
// CTAs fit an SM.
template <int D, int GP>
__host__ __device__ constexpr int merge_heads() {
  return GP < 8 ? GP : (D == 128 ? 4 : 8);
}

}  // namespace
}  // namespace hwkv
