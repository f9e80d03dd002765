// Rotary positions: the pairs of a query or key row turn by an angle proportional to the row's
// position, before the key is appended and the query attends.
//
//   pair i of a row at position p:  (a, b) -> m * (a cos t - b sin t, b cos t + a sin t),  t = p f_i
//
// with f_i radians per position and a common magnitude m; pairs are (i, i + rot / 2) or
// (2i, 2i + 1) of the first rot dims, the others pass through.
//
// Angles of far positions: p f_i reaches thousands of turns, of which fp32 would keep none of the
// fraction's last bits (p = 161K: an error of 0.01 rad).  The host turns f_i into turns as a
// 64-bit fraction F_i = f_i / (2 pi) * 2^64, from a product kept in two parts (one rounded fp64 product would be off
// by up to 2^-21 rad near p = 2^31), so that p * F_i modulo 2^64 -- one integer multiplication -- is the
// fraction of a turn of p f_i to 2^-29; its top 32 bits go to fp32 as half turns in [-1, 1) and sincospif()
// does the rest: 2^-23 rad at every int32 position, for |f_i| < 2^40.  fp64 on the device would give the same at this
// GPU's far lower fp64 rate.
//
// A CTA takes a few rows (tokens) of one sequence: their cosines and sines are computed once into
// shared memory, then each thread turns units of 16-byte vectors across all query and key heads,
// kAhead units' loads in flight.
//
// Bound: reading and writing each row once, HBM for long chunks (4 sequences of 2048 rows, 32 + 8
// heads of 128 in bf16: 126 MB in 19.4-23.3 us by box and run, 0.80-0.95 of the measured copy rate; pairs side by
// side 26) and the launch for short ones (one row: 3.1 us).
#include <algorithm>
#include <type_traits>

#include "hwkv_rope.cuh"

namespace hwkv {
namespace {

constexpr int kRopeRows = 4;  // most rows of a CTA

// How the rows are shared out.  A call that leaves SMs idle wants short work per thread (kWide: 256
// threads, 2 units ahead); one that fills them wants many small CTAs whose angles and loads overlap
// (128 threads, 3 ahead).  One row 3.1 us wide, 3.5 narrow; 512 rows of 40 heads 3.9 and 4.0; 1024
// 6.0 and 4.8; 2048 9.6 and 7.8.
constexpr int64_t kWideTokens = 512;
template <bool kWide>
struct RopeShape {
  static constexpr int kThreads = kWide ? 256 : 128;
  static constexpr int kAhead = kWide ? 2 : 3;
};

// Cosines and sines of a row, two pairs to a 16-byte vector: (cos 2v, cos 2v + 1, sin 2v, sin 2v + 1).
// A unit takes K consecutive vectors; vector v is stored at (v % K) * (32 / K) + v / K, so that the
// units of neighbouring threads read neighbouring vectors (unit after unit they would share banks).
template <int K>
__device__ __forceinline__ int cs_slot(int v) {
  return v % K * (32 / K) + v / K;
}

// Layouts of the pairs across 16-byte vectors
enum { kRopeHalf = 0, kRopeInterleaved = 1, kRopeHalfAny = 2 };

// kRopeHalf: rot / 2 is a multiple of the vector, a unit holds vector j of both halves (or one
// vector past rot); kRopeInterleaved: a unit is one vector; kRopeHalfAny: a unit is one vector
// whose partners are read one by one, all loads of a pass before its stores (a barrier between,
// since a row may be turned in place).
//
// kAppend: keys and values go to their ring slots instead of an output; a row's heads are the queries,
// the keys and the values, and a value's vectors pass as they are.  The slots of the CTA's rows are
// looked up once per head, beside the angles.  4 sequences of 2048 rows, 32 + 8 + 8 heads of 128 in bf16: 151 MB in
// 26.5-27.6 us, 0.82-0.85 of the measured copy rate (a turn and the appends in separate launches move 42 MB more);
// one token 3.8 us.
template <typename T, int kLayout, bool kWide, bool kAppend>
__global__ void __launch_bounds__(RopeShape<kWide>::kThreads)
    rope_kernel(const __grid_constant__ std::conditional_t<kAppend, RopeAppendArgs, RopeArgs> a) {
  constexpr int kRopeThreads = RopeShape<kWide>::kThreads, kRopeAhead = RopeShape<kWide>::kAhead;
  // kRopeHalfAny: a pass holds whole heads (of 8, 16 or 32 vectors), so no later one reads what it turned
  static_assert(kRopeThreads * kRopeAhead % 32 == 0, "a pass holds whole heads");
  using Vec = RopeVec<T>;
  constexpr int V = Vec::V;
  constexpr int K = kLayout == kRopeHalf ? V / 2 : kLayout == kRopeInterleaved ? (V >= 4 ? V / 4 : 1) : 1;
  __shared__ float4 s_cs[kRopeRows][32];
  __shared__ int32_t s_row[kAppend ? kRopeRows * kMaxKvHeads : 1];  // pool row of (row, KV head), -1: not stored
  // Launched as a programmatic dependent.  A decode that follows with early reads may start its
  // schedule and loads once the kernels before this one have completed: its caller vouches for what
  // they wrote, not for less.
  griddep_wait();
  griddep_launch_dependents();

  const int tiles = (a.n_max + a.rows - 1) / a.rows;
  const int s = (int)blockIdx.x / tiles;
  const int i0 = ((int)blockIdx.x - s * tiles) * a.rows;
  const int pos = a.pos[s];
  const int n = a.n != nullptr ? a.n[s] : a.n_max;
  if (pos < 0 || n < 0 || n > a.n_max) {
    if (threadIdx.x == 0 && i0 == 0) atomicOr(a.err, HWKV_DEVERR_NEG_LENGTH);
    return;
  }
  int turn_pos = pos;
  if constexpr (kAppend) {
    if (a.turn_pos != nullptr) turn_pos = a.turn_pos[s];
    if (turn_pos < 0 || pos > INT32_MAX - n || turn_pos > INT32_MAX - n) {
      if (threadIdx.x == 0 && i0 == 0) atomicOr(a.err, HWKV_DEVERR_NEG_LENGTH);
      return;
    }
  }
  const int rows = min(a.rows, n - i0);
  if (rows <= 0) return;

  bool keys_out = false;
  if constexpr (kAppend) keys_out = a.keys_out != 0;
  const int D = a.head_dim, half = a.rot / 2;
  const int nh = a.q_heads + (kAppend ? 2 : 1) * a.k_heads;
  const int turned = kLayout == kRopeHalf ? half / V : D / V;         // units of a head that turn
  const int per_head = kLayout == kRopeHalf ? turned + (kAppend ? 1 : a.copy) * (D - a.rot) / V : turned;
  const int units = rows * nh * per_head;

  // cosines and sines; pairs past rot / 2 do not turn
  auto angles = [&]() {
    const int pairs = D / 2;
    for (int e = threadIdx.x; e < rows * pairs; e += kRopeThreads) {
      const int r = e / pairs, i = e - r * pairs;
      float sn = 0.f, cn = 1.f;
      if (i < half) {
        turn_angle(a.turns[i], (uint32_t)turn_pos + (uint32_t)(i0 + r), a.magnitude, cn, sn);
      }
      float* at = reinterpret_cast<float*>(&s_cs[r][cs_slot<K>(i >> 1)]) + (i & 1);
      at[0] = cn;
      at[2] = sn;
    }
  };

  // kAppend: where the rows go, -1 for those whose slot a later row of the chunk takes
  auto slots = [&]() {
    if constexpr (kAppend) {
      for (int e = threadIdx.x; e < rows * a.k_heads; e += kRopeThreads) {
        const int r = e / a.k_heads, h = e - r * a.k_heads;
        const int bs = a.pv.block_size;
        const int C = (a.g.nblk_prefix[h + 1] - a.g.nblk_prefix[h]) * bs;
        int32_t at = -1;
        if (n - (i0 + r) <= C) {
          const int slot = (pos + i0 + r) % C, jb = slot / bs;
          const int32_t blk = a.pv.tbl[a.g.tbl_base + (int64_t)s * a.g.tbl_seq_stride + a.g.nblk_prefix[h] + jb];
          if (blk >= 0 && (int64_t)blk < a.pv.total_blocks) at = blk * 2 * bs + (slot - jb * bs);
          else atomicOr(a.err, HWKV_DEVERR_BAD_BLOCK);
        }
        s_row[e] = at;
      }
    }
  };

  // the thread's units are kRopeThreads apart: (row, head, place in the head) steps on without divisions
  struct Unit {
    int r, h, j;
  };
  const int dj = kRopeThreads % per_head, dh = kRopeThreads / per_head;
  Unit at;
  at.h = (int)threadIdx.x / per_head;
  at.j = (int)threadIdx.x - at.h * per_head;
  at.r = at.h / nh;
  at.h -= at.r * nh;
  auto step = [&]() {
    at.j += dj;
    at.h += dh;
    if (at.j >= per_head) {
      at.j -= per_head;
      ++at.h;
    }
    while (at.h >= nh) {
      at.h -= nh;
      ++at.r;
    }
  };
  auto row_of = [&](const Unit& x, const RopeTensor& q, const RopeTensor& k) {
    const bool key = x.h >= a.q_heads;
    int h = key ? x.h - a.q_heads : x.h;
    const RopeTensor* t = key ? &k : &q;
    if constexpr (kAppend) {
      if (h >= a.k_heads && key) {
        t = &a.v;
        h -= a.k_heads;
      }
    }
    return static_cast<T*>(t->data) + s * t->seq_stride + (i0 + x.r) * t->row_stride + (int64_t)h * D;
  };
  // Stores a vector of a turned row: to its output and, kAppend, a key's or value's to its slot
  auto put = [&](const Unit& x, T* dst, int d, uint4 v) {
    if constexpr (!kAppend) {
      *reinterpret_cast<uint4*>(dst + d) = v;
    } else {
      const int kh = x.h - a.q_heads;
      if (kh < 0 || (kh < a.k_heads && a.keys_out)) *reinterpret_cast<uint4*>(dst + d) = v;
      if (kh < 0) return;
      const bool val = kh >= a.k_heads;
      const int32_t at = s_row[x.r * a.k_heads + (val ? kh - a.k_heads : kh)];
      if (at < 0) return;
      *reinterpret_cast<uint4*>(static_cast<T*>(a.pv.pool) + ((int64_t)at + (val ? a.pv.block_size : 0)) * D + d) = v;
    }
  };
  // whether a unit's row turns (a value's does not)
  auto turns_at = [&](const Unit& x) { return !kAppend || x.h < a.q_heads + a.k_heads; };

  for (int u0 = 0; u0 < units; u0 += kRopeThreads * kRopeAhead) {
    uint4 lo[kRopeAhead], hi[kRopeAhead];
    Unit un[kRopeAhead];
    T mate[kLayout == kRopeHalfAny ? kRopeAhead : 1][V];
#pragma unroll
    for (int k = 0; k < kRopeAhead; ++k) {
      const int u = u0 + k * kRopeThreads + (int)threadIdx.x;
      un[k] = at;
      step();
      if (u >= units) continue;
      const int j = un[k].j;
      const T* src = row_of(un[k], a.q, a.k);
      if constexpr (kLayout == kRopeHalf) {
        const int at = j < turned ? j * V : a.rot + (j - turned) * V;
        lo[k] = *reinterpret_cast<const uint4*>(src + at);
        if (j < turned) hi[k] = *reinterpret_cast<const uint4*>(src + half + at);
      } else {
        lo[k] = *reinterpret_cast<const uint4*>(src + j * V);
        if constexpr (kLayout == kRopeHalfAny) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int d = j * V + e;
            if (d < a.rot && turns_at(un[k])) mate[k][e] = src[d < half ? d + half : d - half];
          }
        }
      }
    }
    if (u0 == 0) {
      angles();
      slots();
      __syncthreads();
    } else if (kLayout == kRopeHalfAny) {
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRopeAhead; ++k) {
      const int u = u0 + k * kRopeThreads + (int)threadIdx.x;
      if (u >= units) continue;
      const int j = un[k].j;
      const float4* cs = s_cs[un[k].r];
      T* dst = kAppend && un[k].h >= a.q_heads && !(keys_out && un[k].h < nh - a.k_heads) ? nullptr : row_of(un[k], a.q_out, a.k_out);
      if constexpr (kLayout == kRopeHalf) {
        if (j < turned && !turns_at(un[k])) {
          put(un[k], dst, j * V, lo[k]);
          put(un[k], dst, half + j * V, hi[k]);
        } else if (j < turned) {
          Vec x, y;
          x.load(lo[k]);
          y.load(hi[k]);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float4 t = cs[e / 2 * (32 / K) + j];  // cs_slot<K>((j * V + e) / 2)
            const float2 c = make_float2(t.x, t.y), sn = make_float2(t.z, t.w);
            const float2 xe = make_float2(x.v[e], x.v[e + 1]), ye = make_float2(y.v[e], y.v[e + 1]);
            const float2 p = ffma2(xe, c, fmul2(ye, make_float2(-sn.x, -sn.y))), q = ffma2(ye, c, fmul2(xe, sn));
            x.v[e] = p.x;
            x.v[e + 1] = p.y;
            y.v[e] = q.x;
            y.v[e + 1] = q.y;
          }
          put(un[k], dst, j * V, x.store());
          put(un[k], dst, half + j * V, y.store());
        } else {
          put(un[k], dst, a.rot + (j - turned) * V, lo[k]);
        }
      } else if constexpr (kLayout == kRopeInterleaved) {
        if (j * V >= a.rot || !turns_at(un[k])) {  // past the pairs: unchanged, whatever its bits
          if (kAppend || a.copy) put(un[k], dst, j * V, lo[k]);
          continue;
        }
        Vec x;
        x.load(lo[k]);
#pragma unroll
        for (int e = 0; e < V; e += 4) {  // two pairs; those past rot do not turn
          const float4 t = cs[e / 4 * (32 / K) + j];  // cs_slot<K>((j * V + e) / 4)
          if (j * V + e < a.rot) turn(x.v[e], x.v[e + 1], t.x, t.z);
          if (j * V + e + 2 < a.rot) turn(x.v[e + 2], x.v[e + 3], t.y, t.w);
        }
        put(un[k], dst, j * V, x.store());
      } else {
        if (j * V >= a.rot || !turns_at(un[k])) {
          if (kAppend || a.copy) put(un[k], dst, j * V, lo[k]);
          continue;
        }
        Vec x;
        x.load(lo[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int d = j * V + e;
          if (d >= a.rot) continue;
          const float m = load_in<T>(&mate[k][e]);
          const int i = d < half ? d : d - half;
          const float* t = reinterpret_cast<const float*>(&cs[i >> 1]) + (i & 1);
          x.v[e] = d < half ? fmaf(x.v[e], t[0], -(m * t[2])) : fmaf(x.v[e], t[0], m * t[2]);
        }
        put(un[k], dst, j * V, x.store());
      }
    }
  }
}

template <typename T, int kLayout, bool kWide, bool kAppend, typename Args>
cudaError_t launch_shape(const Args& a, unsigned grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(RopeShape<kWide>::kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<T, kLayout, kWide, kAppend>, a);
}

template <typename T, int kLayout, bool kAppend, typename Args>
cudaError_t launch_one(const Args& a, unsigned grid, cudaStream_t st) {
  return (int64_t)a.num_seqs * a.n_max <= kWideTokens ? launch_shape<T, kLayout, true, kAppend>(a, grid, st)
                                                      : launch_shape<T, kLayout, false, kAppend>(a, grid, st);
}

template <typename T, bool kAppend, typename Args>
cudaError_t launch_layout(const Args& a, int layout, unsigned grid, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  if (layout == HWKV_ROPE_INTERLEAVED && a.rot > 0) return launch_one<T, kRopeInterleaved, kAppend>(a, grid, st);
  if (a.rot % (2 * V) == 0) return launch_one<T, kRopeHalf, kAppend>(a, grid, st);
  return launch_one<T, kRopeHalfAny, kAppend>(a, grid, st);
}

// Rows of a CTA: enough vectors for its threads (5 heads of 64 in bf16, 20 units to a row, 4096 rows:
// 1 row 7.4 us, 4 rows 4.6), and two where CTAs are many (40 heads of 128: 4096 rows 13.6 us with 1,
// 13.9 with 2; 8192 rows 22.2 and 21.2).
template <bool kAppend, typename Args>
cudaError_t launch_rows(Args a, int heads, int layout, bool f32, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.num_seqs * a.n_max;
  const int vectors = heads * a.head_dim * (f32 ? 4 : 2) / 16;
  const int units = layout == HWKV_ROPE_INTERLEAVED ? vectors : vectors / 2;
  a.rows = std::min(kRopeRows, std::max(tokens >= 8192 ? 2 : 1, 512 / units));
  const int64_t grid = (int64_t)a.num_seqs * ((a.n_max + a.rows - 1) / a.rows);
  const cudaError_t e = f32 ? launch_layout<float, kAppend>(a, layout, (unsigned)grid, st)
                            : launch_layout<__nv_bfloat16, kAppend>(a, layout, (unsigned)grid, st);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int layout, bool f32, cudaStream_t st) {
  return launch_rows<false>(a, a.q_heads + a.k_heads, layout, f32, st);
}

cudaError_t launch_rope_append(RopeAppendArgs a, int layout, bool f32, cudaStream_t st) {
  return launch_rows<true>(a, a.q_heads + 2 * a.k_heads, layout, f32, st);
}

}  // namespace hwkv
