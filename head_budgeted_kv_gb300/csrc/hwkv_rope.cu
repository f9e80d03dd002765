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
// 64-bit fraction F_i = f_i / (2 pi) * 2^64, so that p * F_i modulo 2^64 -- one integer
// multiplication -- is the exact fraction of a turn of p f_i, whatever p; its top 32 bits go to
// fp32 as half turns in [-1, 1) and sincospif() does the rest: 2^-23 rad at any position.  fp64
// would give the same at this GPU's far lower fp64 rate.
//
// A CTA takes up to T rows (tokens) of one sequence: their cosines and sines are computed once
// into shared memory, then each thread turns units of 16-byte vectors across all query and key
// heads, kAhead units' loads in flight.  The work is reading and writing each row once.
#include "hwkv_device.cuh"

namespace hwkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 2;
constexpr int kRopeRows = 4;  // most rows of a CTA

template <typename T>
struct RopeVec {  // a 16-byte vector as fp32
  static constexpr int V = 16 / (int)sizeof(T);
  float v[V];
  __device__ __forceinline__ void load(uint4 w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(u[i]);
      else v[i] = __uint_as_float((i & 1) ? (u[i >> 1] & 0xFFFF0000u) : (u[i >> 1] << 16));
    }
  }
  __device__ __forceinline__ uint4 store() const {
    if constexpr (sizeof(T) == 4)
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};

__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = fmaf(x, cs.x, -(y * cs.y));
  b = fmaf(y, cs.x, x * cs.y);
}

// Layouts of the pairs across 16-byte vectors
enum { kRopeHalf = 0, kRopeInterleaved = 1, kRopeHalfAny = 2 };

// kRopeHalf: rot / 2 is a multiple of the vector, a unit holds vector j of both halves (or one
// vector past rot); kRopeInterleaved: a unit is one vector; kRopeHalfAny: a unit is one vector
// whose partners are read one by one, all loads of a pass before its stores (a barrier between,
// since a row may be turned in place).
template <typename T, int kLayout>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  using Vec = RopeVec<T>;
  constexpr int V = Vec::V;
  __shared__ __align__(16) float2 s_cs[kRopeRows][64];
  griddep_launch_dependents();  // a decode launched with early reads may start its schedule and loads

  const int tiles = (a.n_max + a.rows - 1) / a.rows;
  const int s = (int)blockIdx.x / tiles;
  const int i0 = ((int)blockIdx.x - s * tiles) * a.rows;
  const int pos = a.pos[s];
  const int n = a.n != nullptr ? a.n[s] : a.n_max;
  if (pos < 0 || n < 0 || n > a.n_max) {
    if (threadIdx.x == 0 && i0 == 0) atomicOr(a.err, HWKV_DEVERR_NEG_LENGTH);
    return;
  }
  const int rows = min(a.rows, n - i0);
  if (rows <= 0) return;

  const int D = a.head_dim, half = a.rot / 2;
  const int nh = a.q_heads + a.k_heads;
  const int turned = kLayout == kRopeHalf ? half / V : D / V;         // units of a head that turn
  const int per_head = kLayout == kRopeHalf ? turned + a.copy * (D - a.rot) / V : turned;
  const int units = rows * nh * per_head;

  // cosines and sines; pairs past rot / 2 do not turn
  auto angles = [&]() {
    const int pairs = D / 2;
    for (int e = threadIdx.x; e < rows * pairs; e += kRopeThreads) {
      const int r = e / pairs, i = e - r * pairs;
      float2 cs = make_float2(1.f, 0.f);
      if (i < half) {
        const uint64_t t = a.turns[i] * (uint64_t)((uint32_t)pos + (uint32_t)(i0 + r));
        const float x = (float)(int32_t)(t >> 32) * 0x1p-31f;  // half turns
        sincospif(x, &cs.y, &cs.x);
        cs.x *= a.magnitude;
        cs.y *= a.magnitude;
      }
      s_cs[r][i] = cs;
    }
  };

  struct Unit {
    const T* src;
    T* dst;
    int r, j;
  };
  auto unit_at = [&](int u) {
    Unit x;
    const int rh = u / per_head;
    x.j = u - rh * per_head;
    x.r = rh / nh;
    const int h = rh - x.r * nh;
    const bool key = h >= a.q_heads;
    const RopeTensor& in = key ? a.k : a.q;
    const RopeTensor& out = key ? a.k_out : a.q_out;
    const int64_t col = (int64_t)(key ? h - a.q_heads : h) * D;
    x.src = static_cast<const T*>(in.data) + s * in.seq_stride + (i0 + x.r) * in.row_stride + col;
    x.dst = static_cast<T*>(out.data) + s * out.seq_stride + (i0 + x.r) * out.row_stride + col;
    return x;
  };

  for (int u0 = 0; u0 < units; u0 += kRopeThreads * kRopeAhead) {
    uint4 lo[kRopeAhead], hi[kRopeAhead];
    Unit un[kRopeAhead];
    T mate[kLayout == kRopeHalfAny ? kRopeAhead : 1][V];
#pragma unroll
    for (int k = 0; k < kRopeAhead; ++k) {
      const int u = u0 + k * kRopeThreads + (int)threadIdx.x;
      if (u >= units) continue;
      un[k] = unit_at(u);
      const int j = un[k].j;
      if constexpr (kLayout == kRopeHalf) {
        const int at = j < turned ? j * V : a.rot + (j - turned) * V;
        lo[k] = *reinterpret_cast<const uint4*>(un[k].src + at);
        if (j < turned) hi[k] = *reinterpret_cast<const uint4*>(un[k].src + half + at);
      } else {
        lo[k] = *reinterpret_cast<const uint4*>(un[k].src + j * V);
        if constexpr (kLayout == kRopeHalfAny) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int d = j * V + e;
            if (d < a.rot) mate[k][e] = un[k].src[d < half ? d + half : d - half];
          }
        }
      }
    }
    if (u0 == 0) {
      angles();
      __syncthreads();
    } else if (kLayout == kRopeHalfAny) {
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRopeAhead; ++k) {
      const int u = u0 + k * kRopeThreads + (int)threadIdx.x;
      if (u >= units) continue;
      const int j = un[k].j;
      const float2* cs = s_cs[un[k].r];
      if constexpr (kLayout == kRopeHalf) {
        if (j < turned) {
          Vec x, y;
          x.load(lo[k]);
          y.load(hi[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) turn(x.v[e], y.v[e], cs[j * V + e]);
          *reinterpret_cast<uint4*>(un[k].dst + j * V) = x.store();
          *reinterpret_cast<uint4*>(un[k].dst + half + j * V) = y.store();
        } else {
          *reinterpret_cast<uint4*>(un[k].dst + a.rot + (j - turned) * V) = lo[k];
        }
      } else if constexpr (kLayout == kRopeInterleaved) {
        if (j * V >= a.rot) {  // past the pairs: unchanged, whatever its bits
          if (a.copy) *reinterpret_cast<uint4*>(un[k].dst + j * V) = lo[k];
          continue;
        }
        Vec x;
        x.load(lo[k]);
#pragma unroll
        for (int e = 0; e < V; e += 2)
          if (j * V + e < a.rot) turn(x.v[e], x.v[e + 1], cs[(j * V + e) / 2]);
        *reinterpret_cast<uint4*>(un[k].dst + j * V) = x.store();
      } else {
        if (j * V >= a.rot) {
          if (a.copy) *reinterpret_cast<uint4*>(un[k].dst + j * V) = lo[k];
          continue;
        }
        Vec x;
        x.load(lo[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int d = j * V + e;
          if (d >= a.rot) continue;
          const float m = load_in<T>(&mate[k][e]);
          const float2 c = cs[d < half ? d : d - half];
          x.v[e] = d < half ? fmaf(x.v[e], c.x, -(m * c.y)) : fmaf(x.v[e], c.x, m * c.y);
        }
        *reinterpret_cast<uint4*>(un[k].dst + j * V) = x.store();
      }
    }
  }
}

template <typename T>
void launch_layout(const RopeArgs& a, int layout, unsigned grid, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  if (layout == HWKV_ROPE_INTERLEAVED) rope_kernel<T, kRopeInterleaved><<<grid, kRopeThreads, 0, st>>>(a);
  else if (a.rot % (2 * V) == 0) rope_kernel<T, kRopeHalf><<<grid, kRopeThreads, 0, st>>>(a);
  else rope_kernel<T, kRopeHalfAny><<<grid, kRopeThreads, 0, st>>>(a);
}

}  // namespace

// rows of a CTA: one while that fills the SMs at most a few times over, else kRopeRows
int rope_rows(int64_t tokens) { return tokens >= 1024 ? kRopeRows : 1; }

cudaError_t launch_rope(const RopeArgs& a, int layout, bool f32, cudaStream_t st) {
  const int64_t grid = (int64_t)a.num_seqs * ((a.n_max + a.rows - 1) / a.rows);
  if (f32) launch_layout<float>(a, layout, (unsigned)grid, st);
  else launch_layout<__nv_bfloat16>(a, layout, (unsigned)grid, st);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace hwkv
