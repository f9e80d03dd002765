// Append and materialise for 8-bit pools (HWKV_E4M3): the rows are stored as e4m3 codes, 16
// consecutive ring slots of a head sharing a scale for K and one for V (hwkv_fp8.cuh).
//
// "HeadWiseKV: Budgeted Per-Head Cache Residency for Hybrid Long-Context Language Models",
// abstract and section "Grouped-Cache Runtime": each KV head keeps its newest w tokens in a ring
// of ceil(w / bs) blocks; position p lives in slot p mod C.
//
// Both kernels write whole groups: slots of a group that hold no position of the window become
// zero.  Bad lengths and table entries are recorded in the device error word and skipped.
#include "hwkv_fp8.cuh"

namespace hwkv {
namespace {

// Block of ring slot t of (seq s, kv head h), or -1 (recorded) when the table entry is bad.
__device__ __forceinline__ int32_t slot_block(const PoolView& pv, const LayerGeom& g, int s, int h, int t, int lane) {
  const int32_t blk = pv.tbl[g.tbl_base + (int64_t)s * g.tbl_seq_stride + g.nblk_prefix[h] + t / pv.block_size];
  if (blk >= 0 && (int64_t)blk < pv.total_blocks) return blk;
  if (lane == 0) atomicOr(pv.err, HWKV_DEVERR_BAD_BLOCK);
  return -1;
}

// One warp per (seq, kv head, K or V): the new token's group is stored anew (GroupRecode).
template <int D>
__global__ void __launch_bounds__(128) append_q8_kernel(const __grid_constant__ CopyArgs a) {
  const int warp = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  const int H = a.pv.kv_heads;
  if (warp >= 2 * a.pv.num_seqs * H) return;
  const int kv = warp & 1, sh = warp >> 1;
  const int s = sh / H, h = sh - s * H;
  const int32_t p = a.lens[s];
  if (p < 0) {
    if (lane == 0) atomicOr(a.pv.err, HWKV_DEVERR_NEG_LENGTH);
    return;
  }
  const int bs = a.pv.block_size;
  const int C = (a.g.nblk_prefix[h + 1] - a.g.nblk_prefix[h]) * bs;
  const int slot = p % C, t0 = slot & ~(kScaleGroup - 1);
  const int32_t blk = slot_block(a.pv, a.g, s, h, t0, lane);
  if (blk < 0) return;
  const int r0 = t0 % bs;
  uint8_t* rows = static_cast<uint8_t*>(a.pv.pool) + (((int64_t)blk * 2 + kv) * bs + r0) * D;
  float* scale = a.pv.scales + ((int64_t)blk * (bs / kScaleGroup) + r0 / kScaleGroup) * 2 + kv;
  const float old = *scale;
  GroupRecode<D> g;
  g.load(static_cast<const __nv_bfloat16*>(kv ? a.v : a.k) + (int64_t)sh * D, t0, slot, p, a.g.window[h], C,
         [&](int r, int c) { return *reinterpret_cast<const uint4*>(rows + r * D + 16 * c); }, lane);
  const float now = g.store(warp_max(g.amax(old)), old,
                            [&](int r, int c, uint4 v) { *reinterpret_cast<uint4*>(rows + r * D + 16 * c) = v; }, lane);
  if (lane == 0) *scale = now;
}

constexpr int kMatWarps = 8;

// grid.x: per sequence, the CTA's share of its groups of 16 ring slots (all heads in a row, so no
// CTA is empty whatever the windows).  A warp takes K or V of one group (head_dim 128) or both (64):
// 4 KB of source either way, a lane 8 dims of a row, all loads issued before any is used.  The
// largest magnitude is taken on packed bf16 pairs; a group that holds anything not finite (the
// NaN-propagating maximum shows it) goes the careful way.
//
// Bound: HBM, 2 bytes read and 1 written per value (+ 8 bytes per group and K/V pair): four prompts of
// 30-32K, head_dim 128, 512 MB in 80.3 us, 0.94 of the measured copy rate.
template <int D>
__global__ void __launch_bounds__(kMatWarps * 32) materialize_q8_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int kLanes = D / 8;               // lanes per row
  constexpr int kRows = 32 / kLanes;          // rows per load
  constexpr int kPer = kScaleGroup / kRows;   // loads per lane of one group's K or V
  constexpr int kBoth = D == 64 ? 2 : 1;      // K and V by the same warp
  constexpr int kGroups = kMatWarps * kBoth / 2;  // groups of a CTA
  const int H = a.pv.kv_heads;
  const int per_group = a.pv.block_size / kScaleGroup;  // groups per block
  const int ngroups = a.g.nblk_prefix[H] * per_group;
  const int nchunks = (ngroups + kGroups - 1) / kGroups;
  const int s = (int)blockIdx.x / nchunks;
  const int32_t L = a.lens[s];
  if (L < 0 || (int64_t)L > a.max_len) {
    if (threadIdx.x == 0 && (int)blockIdx.x == s * nchunks)
      atomicOr(a.pv.err, L < 0 ? HWKV_DEVERR_NEG_LENGTH : HWKV_DEVERR_SRC_RANGE);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bs = a.pv.block_size;
  const int gi = ((int)blockIdx.x - s * nchunks) * kGroups + (kBoth == 2 ? warp : warp >> 1);
  if (gi >= ngroups) return;
  int h = 0;
  while (a.g.nblk_prefix[h + 1] * per_group <= gi) ++h;
  const int C = (a.g.nblk_prefix[h + 1] - a.g.nblk_prefix[h]) * bs;
  const int t0 = (gi - a.g.nblk_prefix[h] * per_group) * kScaleGroup;
  const Resident rs = resident(L, a.g.window[h], C);
  const int c = lane % kLanes, r_lane = lane / kLanes;
  const int64_t off = a.seq_stride * s + a.head_stride * h + 8 * c;
  uint4 x[kBoth][kPer];
  bool any = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    int d = t0 + i * kRows + r_lane - rs.first_slot;  // positions above the oldest resident one
    if (d < 0) d += C;
    const bool live = d < rs.n;
    any = any || live;
#pragma unroll
    for (int b = 0; b < kBoth; ++b) {
      const void* src = (kBoth == 2 ? b : warp & 1) ? a.v : a.k;
      x[b][i] = make_uint4(0u, 0u, 0u, 0u);
      if (live)
        x[b][i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + off + (int64_t)(L - rs.n + d) * D));
    }
  }
  if (!__any_sync(0xffffffffu, any)) return;
  const int32_t blk = slot_block(a.pv, a.g, s, h, t0, lane);
  if (blk < 0) return;
  const int r0 = t0 % bs;
#pragma unroll
  for (int b = 0; b < kBoth; ++b) {
    const int kv = kBoth == 2 ? b : warp & 1;
    __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t w[4] = {x[b][i].x, x[b][i].y, x[b][i].z, x[b][i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
    }
    const float hi = __high2float(top), lo = __low2float(top);
    const bool fine = __all_sync(0xffffffffu, hi < __builtin_huge_valf() && lo < __builtin_huge_valf());
    float amax = fmaxf(lo, hi);
    if (!fine) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint4 v = x[b][i];
        for (uint32_t w : {v.x, v.y, v.z, v.w})
          amax = fmaxf(amax, fmaxf(finite_abs(__uint_as_float(w << 16)), finite_abs(__uint_as_float(w & 0xFFFF0000u))));
      }
    }
    const float scale = pow2i(scale_exponent(warp_max(amax))), inv = pow2_inverse(scale);
    uint8_t* rows = static_cast<uint8_t*>(a.pv.pool) + (((int64_t)blk * 2 + kv) * bs + r0) * D;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      *reinterpret_cast<uint2*>(rows + (i * kRows + r_lane) * D + 8 * c) = fine ? encode8_finite(x[b][i], inv) : encode8(x[b][i], inv);
    if (lane == 0) a.pv.scales[((int64_t)blk * per_group + r0 / kScaleGroup) * 2 + kv] = scale;
  }
}

}  // namespace

cudaError_t launch_append_q8(const CopyArgs& a, cudaStream_t st) {
  const int warps = 2 * a.pv.num_seqs * a.pv.kv_heads;
  const int blocks = (warps + 3) / 4;
  if (a.pv.head_dim == 128) append_q8_kernel<128><<<blocks, 128, 0, st>>>(a);
  else if (a.pv.head_dim == 64) append_q8_kernel<64><<<blocks, 128, 0, st>>>(a);
  else return cudaErrorInvalidValue;
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_materialize_q8(const CopyArgs& a, cudaStream_t st) {
  const int per_cta = a.pv.head_dim == 64 ? kMatWarps : kMatWarps / 2;
  const int64_t groups = (int64_t)a.g.nblk_prefix[a.pv.kv_heads] * (a.pv.block_size / kScaleGroup);
  // at most the pool's rows / 64, which is below 2^31
  const unsigned grid = (unsigned)((groups + per_cta - 1) / per_cta * a.pv.num_seqs);
  if (a.pv.head_dim == 128) materialize_q8_kernel<128><<<grid, kMatWarps * 32, 0, st>>>(a);
  else if (a.pv.head_dim == 64) materialize_q8_kernel<64><<<grid, kMatWarps * 32, 0, st>>>(a);
  else return cudaErrorInvalidValue;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace hwkv
