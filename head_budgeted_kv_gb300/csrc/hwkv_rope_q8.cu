// Rotary positions on the way into an 8-bit pool (HWKV_E4M3): a chunk's (or a token's) queries turned,
// its keys turned and stored, its values stored.  bf16 and fp32 pools: hwkv_rope.cu, kAppend.
//
// 16 consecutive ring slots share a scale, so what is stored is a group at a time.  C is a multiple of
// 16: position p lies in slot p mod 16 of its group in every ring, and the chunk's rows
// fall into tiles of 16 positions that are groups of every head.  Slot r of a head's group m holds the newest
// position p of m * 16 + r and m * 16 + r - C, ... below the end of the chunk.  A group a row goes to is
// stored once: the chunk's rows, turned in fp32, and the stored values of older positions, if they are in
// the window of the new length, else zeros; its scale is the smallest power of two that holds their
// largest magnitude.  Where the ring is shorter than the chunk, only the last tile of a group stores it.
//
// Roundings: a key is rounded once, from its turned fp32 value to the code (through bf16, as hwkv_rope and
// hwkv_append in turn, twice); a kept code moves by a power of two, which rounds only those that become
// subnormal.
//
// A CTA takes, of a tile of one sequence, two KV heads -- a warp K or V of one head's group, 16 rows of which a lane holds pairs of
// 16-byte vectors, all loaded before the angles are computed and any is used -- or some rows of all query heads, kAhead
// pairs of vectors of a thread on their way at once.  The cosines and sines of its rows go through shared
// memory.
//
// Bound: HBM for chunks, the launch for tokens.  4 sequences of 2048 rows, 32 + 8 + 8 heads of 128 with turned keys out:
// 151 MB in 37 us, 0.61 of the measured copy rate (an angle's sine and cosine, two conversions per element and the scale's
// reduction share the issue slots with the copies: half of them taken).  It was 67 before CTAs took two heads or some
// query rows with four loads ahead (48), and 48 before the angles' vectors in shared memory avoided each other's banks.
// 64 tokens: 11 us alone with cold caches.
#include <algorithm>

#include "hwkv_fp8.cuh"
#include "hwkv_rope.cuh"

namespace hwkv {
namespace {

constexpr int kQ8Threads = 128;
constexpr int kAhead = 4;

enum { kHalf = 0, kInterleaved = 1, kHalfAny = 2 };

// A lane's pair of 16-byte vectors j of a row: dims [a, a + 8) and [b, b + 8).  kHalf (rot / 2 a multiple of 8): the two
// halves' vectors that turn together, then neighbours past rot; else neighbours.
struct Place {
  int a, b;
  bool turned;  // (kHalf) whether they turn
};

template <int kLayout>
__device__ __forceinline__ Place place_of(int j, int rot) {
  if constexpr (kLayout == kHalf) {
    const int n = rot / 16;
    if (j < n) return {8 * j, rot / 2 + 8 * j, true};
    return {16 * j, 16 * j + 8, false};
  }
  return {16 * j, 16 * j + 8, true};
}

using Vec8 = RopeVec<__nv_bfloat16>;

// Where the cosine and sine of pair i of a row lie, in float2: two pairs to a 16-byte vector, vector v at (v % 4) * (D / 16) + v / 4, so
// that the lanes of a row, which want pairs 8 j and up, read neighbouring vectors.
template <int D>
__device__ __forceinline__ int cs_slot(int i) {
  const int v = i >> 1;
  return 2 * ((v & 3) * (D / 16) + (v >> 2)) + (i & 1);
}

// Turns the pair of vectors in place, place j of a row; cs(i): cosine and sine of pair i (kHalfAny); cs2(k): of pairs 8 j + 2 k
// and the next; mate(d): element d of the row (kHalfAny).
template <int kLayout, typename Cs, typename Cs2, typename Mate>
__device__ __forceinline__ void turn_pair(Vec8& x, Vec8& y, const Place& at, int rot, Cs cs, Cs2 cs2, Mate mate) {
  if constexpr (kLayout == kHalf) {
    if (!at.turned) return;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 c = cs2(e / 2);
      turn(x.v[e], y.v[e], c.x, c.y);
      turn(x.v[e + 1], y.v[e + 1], c.z, c.w);
    }
  } else if constexpr (kLayout == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float* v = (e < 8 ? x.v : y.v) + (e & 7);
      const float4 c = cs2(e / 4);
      if (at.a + e < rot) turn(v[0], v[1], c.x, c.y);
      if (at.a + e + 2 < rot) turn(v[2], v[3], c.z, c.w);
    }
  } else {
    const int half = rot / 2;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = at.a + e;
      if (d >= rot) continue;
      float& v = e < 8 ? x.v[e & 7] : y.v[e & 7];
      const float2 c = cs(d < half ? d : d - half);
      const float m = mate(d < half ? d + half : d - half);
      v = d < half ? fmaf(v, c.x, -(m * c.y)) : fmaf(v, c.x, m * c.y);
    }
  }
}

template <int D, int kLayout>
__global__ void __launch_bounds__(kQ8Threads, 4) rope_append_q8_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int kPairs = D / 16;         // pairs of vectors of a row
  constexpr int kRows = 32 / kPairs;     // rows the lanes of a warp cover
  constexpr int kPer = kScaleGroup / kRows;
  static_assert(kQ8Threads % kPairs == 0, "a thread keeps its place in the rows");
  __shared__ __align__(16) float2 s_cs[kScaleGroup][D / 2];
  griddep_wait();
  griddep_launch_dependents();

  const int H = a.pv.kv_heads, bs = a.pv.block_size;
  const int kv_parts = (H + 1) / 2;
  const int per = kv_parts + a.q_parts;         // CTAs of a tile
  const int tiles = (a.n_max + 2 * kScaleGroup - 2) / kScaleGroup;  // the most that a chunk touches
  const int s = (int)blockIdx.x / (tiles * per);
  const int rem = (int)blockIdx.x - s * tiles * per;
  const int ti = rem / per, part = rem - ti * per;
  const int pos = a.pos[s];
  const int n = a.n != nullptr ? a.n[s] : a.n_max;
  const int turn_pos = a.turn_pos != nullptr ? a.turn_pos[s] : pos;
  if (pos < 0 || n < 0 || n > a.n_max || turn_pos < 0 || pos > INT32_MAX - n || turn_pos > INT32_MAX - n) {
    if (threadIdx.x == 0 && rem == 0) atomicOr(a.err, HWKV_DEVERR_NEG_LENGTH);
    return;
  }
  const int end = pos + n;
  const int m = pos / kScaleGroup + ti;         // tile: positions [16 m, 16 m + 16)
  if (n == 0 || m > (end - 1) / kScaleGroup) return;
  const int p0 = m * kScaleGroup;
  int r_lo = max(0, pos - p0), r_hi = min(kScaleGroup, end - p0);  // the CTA's rows of the chunk, at first the tile's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rot = a.rot, half = rot / 2;
  const Place at = place_of<kLayout>((int)threadIdx.x % kPairs, rot);

  const int j = (int)threadIdx.x % kPairs;
  auto cs2 = [&](int r, int k) { return *reinterpret_cast<const float4*>(&s_cs[r][2 * (k * kPairs + j)]); };  // pairs 8 j + 2 k and the next
  auto angles = [&]() {
    for (int e = threadIdx.x; e < (r_hi - r_lo) * half; e += kQ8Threads) {
      const int r = r_lo + e / half, i = e - (r - r_lo) * half;
      float cn, sn;
      turn_angle_fine(a.turns[i], (uint32_t)turn_pos + (uint32_t)(p0 + r - pos), a.magnitude, cn, sn);
      s_cs[r][cs_slot<D>(i)] = make_float2(cn, sn);
    }
  };

  if (part >= kv_parts) {
    // ---- queries: rows x heads x pairs of vectors, a row's head within one warp -----------------
    const int rows = kScaleGroup / a.q_parts, first = (part - kv_parts) * rows;
    r_lo = max(r_lo, first);
    r_hi = min(r_hi, first + rows);
    if (r_lo >= r_hi) return;
    const int Hq = a.q_heads;
    const int units = (r_hi - r_lo) * Hq * kPairs;
    constexpr int kStep = kQ8Threads / kPairs;  // heads from one of a thread's units to the next
    int r = r_lo, h = (int)threadIdx.x / kPairs;
    auto settle = [&]() {
      while (h >= Hq) {
        h -= Hq;
        ++r;
      }
    };
    settle();
    for (int u0 = 0; u0 < units; u0 += kQ8Threads * kAhead) {
      uint4 u[kAhead], v[kAhead];
      int rk[kAhead], hk[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        rk[k] = r;
        hk[k] = h;
        h += kStep;
        settle();
        if (rk[k] < r_hi) {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.data) + s * a.q.seq_stride +
                                     (int64_t)(p0 + rk[k] - pos) * a.q.row_stride + (int64_t)hk[k] * D;
          u[k] = *reinterpret_cast<const uint4*>(src + at.a);
          v[k] = *reinterpret_cast<const uint4*>(src + at.b);
        }
      }
      if (u0 == 0 && rot > 0) {
        angles();
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool in = rk[k] < r_hi;
        const int64_t i = p0 + rk[k] - pos;
        if (in && rot > 0) {
          const __nv_bfloat16* src =
              static_cast<const __nv_bfloat16*>(a.q.data) + s * a.q.seq_stride + i * a.q.row_stride + (int64_t)hk[k] * D;
          Vec8 x, y;
          x.load(u[k]);
          y.load(v[k]);
          turn_pair<kLayout>(x, y, at, rot, [&](int c) { return s_cs[rk[k]][cs_slot<D>(c)]; }, [&](int c) { return cs2(rk[k], c); },
                             [&](int d) { return __bfloat162float(src[d]); });
          u[k] = x.store();
          v[k] = y.store();
        }
        if constexpr (kLayout == kHalfAny) __syncwarp();  // a row may be turned in place: its lanes have read their mates
        if (in) {
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(a.q_out.data) + s * a.q_out.seq_stride + i * a.q_out.row_stride + (int64_t)hk[k] * D;
          *reinterpret_cast<uint4*>(dst + at.a) = u[k];
          *reinterpret_cast<uint4*>(dst + at.b) = v[k];
        }
      }
    }
    return;
  }

  // ---- keys and values: one group of a head and K or V per warp ------------------------
  const int h = part * 2 + (warp >> 1);
  const bool val = warp & 1;
  const int r_lane = lane / kPairs;
  const RopeTensor& src = val ? a.v : a.k;
  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(src.data) + s * src.seq_stride + (int64_t)h * D;
  const bool there = h < H;
  const int C = there ? (a.g.nblk_prefix[h + 1] - a.g.nblk_prefix[h]) * bs : kScaleGroup;
  const int w = there ? a.g.window[h] : 0;
  const bool stores = there && (end - 1) / kScaleGroup - m < C / kScaleGroup;  // no later tile is the same group
  const bool out = there && !val && a.keys_out;
  int32_t blk = -1;
  int row0 = 0;
  if (stores) {
    const int slot = p0 % C, jb = slot / bs;
    row0 = slot - jb * bs;
    blk = a.pv.tbl[a.g.tbl_base + (int64_t)s * a.g.tbl_seq_stride + a.g.nblk_prefix[h] + jb];
    if (blk < 0 || (int64_t)blk >= a.pv.total_blocks) {
      if (lane == 0) atomicOr(a.err, HWKV_DEVERR_BAD_BLOCK);
      blk = -1;
    }
  }
  uint8_t* codes = static_cast<uint8_t*>(a.pv.pool) + (((int64_t)max(blk, 0) * 2 + (val ? 1 : 0)) * bs + row0) * D;
  float* scale_at = a.pv.scales + ((int64_t)max(blk, 0) * (bs / kScaleGroup) + row0 / kScaleGroup) * 2 + (val ? 1 : 0);
  const float old = blk >= 0 ? *scale_at : 1.f;

  uint4 u[kPer], v[kPer];
  uint32_t kinds = 0u;  // two bits a row: 0 zero, 1 a kept row (its codes), 2 a row of the chunk, 3 one that is not stored
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r_lane + i * kRows;
    int p = p0 + r;
    const bool here = p >= pos && p < end;  // of this tile (not of the ring's lap before)
    if (p >= end) p -= C;  // the newest position of the slot (p0 is a multiple of 16: p0 + r < 2^31)
    const bool fresh = p >= pos;
    const bool live = p >= 0 && p >= end - w;
    const int kind = fresh && live && (stores || out) ? 2 : fresh && here && out ? 3 : !fresh && live && blk >= 0 ? 1 : 0;
    kinds |= (uint32_t)kind << (2 * i);
    u[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (kind >= 2) {
      const __nv_bfloat16* row = in + (int64_t)(p - pos) * src.row_stride;
      u[i] = *reinterpret_cast<const uint4*>(row + at.a);
      v[i] = *reinterpret_cast<const uint4*>(row + at.b);
    } else if (kind == 1) {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + r * D + at.a), d = *reinterpret_cast<const uint2*>(codes + r * D + at.b);
      u[i] = make_uint4(c.x, c.y, d.x, d.y);
    }
  }
  if (rot > 0) {
    angles();
    __syncthreads();
  }
  if (!stores && !out) return;

  // the rows in fp32: turned keys, values, codes' values
  Vec8 x[kPer], y[kPer];
  float top = 0.f, kept = 0.f;  // largest finite magnitudes: rows of the chunk, kept codes
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r_lane + i * kRows;
    const int kind = (kinds >> (2 * i)) & 3;
    if (kind == 1) {
      const uint32_t cw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t lo, hi;
        e4m3x4_to_f16(cw[k], lo, hi);
        const float2 f = half2_to_float2(lo), g = half2_to_float2(hi);
        float* t = (k < 2 ? x[i].v : y[i].v) + 4 * (k & 1);
        t[0] = f.x;
        t[1] = f.y;
        t[2] = g.x;
        t[3] = g.y;
      }
    } else {
      x[i].load(u[i]);
      y[i].load(v[i]);
    }
    if (!val && kind >= 2 && rot > 0) {
      const bool here = p0 + r < end;
      const int i_row = here ? p0 + r - pos : p0 + r - C - pos;  // chunk row
      const __nv_bfloat16* row = in + (int64_t)i_row * src.row_stride;
      auto mate = [&](int d) { return __bfloat162float(row[d]); };
      if (here) {
        turn_pair<kLayout>(x[i], y[i], at, rot, [&](int k) { return s_cs[r][cs_slot<D>(k)]; }, [&](int k) { return cs2(r, k); }, mate);
      } else {  // a row of the lap before: its angles are not the tile's
        auto far = [&](int k) {
          float2 c = make_float2(1.f, 0.f);
          if (k < half) turn_angle_fine(a.turns[k], (uint32_t)turn_pos + (uint32_t)i_row, a.magnitude, c.x, c.y);
          return c;
        };
        turn_pair<kLayout>(x[i], y[i], at, rot, far, [&](int k) {
          const float2 c = far(8 * j + 2 * k), d = far(8 * j + 2 * k + 1);
          return make_float4(c.x, c.y, d.x, d.y);
        }, mate);
      }
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaxf(finite_abs(x[i].v[e]), finite_abs(y[i].v[e])));
    if (kind == 1) kept = fmaxf(kept, mx);
    if (kind == 2) top = fmaxf(top, mx);
  }
  const float scale = pow2i(scale_exponent(warp_max(fmaxf(top, kept * old)))), inv = pow2_inverse(scale);
  const float factor = fminf(old * inv, 0x1p100f);  // see GroupRecode
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r_lane + i * kRows;
    const int kind = (kinds >> (2 * i)) & 3;
    if (out && p0 + r >= pos && p0 + r < end) {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(a.k_out.data) + s * a.k_out.seq_stride +
                           (int64_t)(p0 + r - pos) * a.k_out.row_stride + (int64_t)h * D;
      *reinterpret_cast<uint4*>(row + at.a) = x[i].store();
      *reinterpret_cast<uint4*>(row + at.b) = y[i].store();
    }
    if (blk < 0) continue;
    const float f = kind == 2 ? inv : factor;
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* t = (k < 2 ? x[i].v : y[i].v) + 4 * (k & 1);
      c[k] = kind == 0 || kind == 3 ? 0u : e4m3x2(t[0] * f, t[1] * f) | (e4m3x2(t[2] * f, t[3] * f) << 16);
    }
    *reinterpret_cast<uint2*>(codes + r * D + at.a) = make_uint2(c[0], c[1]);
    *reinterpret_cast<uint2*>(codes + r * D + at.b) = make_uint2(c[2], c[3]);
  }
  if (lane == 0 && blk >= 0) *scale_at = scale;
}

template <int D, int kLayout>
cudaError_t launch_q8(const RopeAppendArgs& a, unsigned grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kQ8Threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_q8_kernel<D, kLayout>, a);
}

template <int D>
cudaError_t launch_dim(const RopeAppendArgs& a, int layout, unsigned grid, cudaStream_t st) {
  if (layout == HWKV_ROPE_INTERLEAVED && a.rot > 0) return launch_q8<D, kInterleaved>(a, grid, st);
  if (a.rot % 16 == 0) return launch_q8<D, kHalf>(a, grid, st);
  return launch_q8<D, kHalfAny>(a, grid, st);
}

}  // namespace

cudaError_t launch_rope_append_q8(RopeAppendArgs a, int layout, cudaStream_t st) {
  // queries: a CTA's rows of a tile, four of its 16 where chunks fill tiles
  a.q_parts = a.q_heads == 0 ? 0 : a.n_max >= kScaleGroup ? 4 : 1;
  const int64_t tiles = (int64_t)a.num_seqs * ((a.n_max + 2 * kScaleGroup - 2) / kScaleGroup);
  const int64_t grid = tiles * ((a.pv.kv_heads + 1) / 2 + a.q_parts);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const cudaError_t e = a.head_dim == 128  ? launch_dim<128>(a, layout, (unsigned)grid, st)
                        : a.head_dim == 64 ? launch_dim<64>(a, layout, (unsigned)grid, st)
                                           : cudaErrorInvalidValue;
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace hwkv
