// Decode behind shared prefixes: sequences whose contexts begin alike keep the common part once, in a pool of
// prefixes, and their own tokens in their own pool.  The query of sequence s (own length n, prefix f of N tokens) attends
// to its own window and to the prefix's positions in [max(0, N + n - w), N):
//
//   out = (sum_own p v + sum_prefix p v) / (sum_own p + sum_prefix p),   p = 2^(score - m)
//
// Three launches.  The prefixes' keys are read once for all sequences behind them, as a product of
// (sequences x group) rows with the keys (on tcgen05: hwkv_shared_tc.cuh; here: CUDA cores, for fp32 pools and
// block sizes that no 16-row tile divides); the own parts come from the decode kernels, left open
// (hwkv_decode_sk.cuh, kOpen); and the join below weighs the partials of both by their reference maxima.
#include <algorithm>
#include <atomic>

#include "hwkv_shared.cuh"

namespace hwkv {
namespace {

constexpr int kRows = 32;     // query rows of a CTA
constexpr int kKeys = 32;     // keys of a pass
constexpr int kThreads = 128;  // four per row

// CTA = (prefix, head, chunk of ring slots; sequences).  A pass brings 32 keys and values into shared memory; the four
// threads of a row take eight scores each, the row's maximum and sum over them by shuffles, then a quarter
// of head_dim each of the weighted sum.  fp32 throughout.  Bound: latency of the passes for few keys, fp32 work and shared memory
// reads for many.  6 sequences behind two prefixes of up to 3K tokens in fp32, with own parts and join: 28 us
// (142 with larger chunks and 4-byte loads; 45 with the own parts behind this kernel, not beside it).
template <typename T, int D, bool SC>
__global__ void __launch_bounds__(kThreads) shared_simt_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int kLd = D + 4;  // floats per row in shared memory: rows 16 bytes apart in the banks
  extern __shared__ float4 smem4[];
  float* s_q = reinterpret_cast<float*>(smem4);  // [kRows][kLd]
  float* s_k = s_q + kRows * kLd;                // [kKeys][kLd]
  float* s_v = s_k + kKeys * kLd;                // [kKeys][kLd]
  float* s_p = s_v + kKeys * kLd;                // [kRows][kKeys + 1]
  __shared__ int s_seq[kRows];
  __shared__ int s_count;

  griddep_wait();
  griddep_launch_dependents();  // the own parts may start beside: all before this grid has completed

  const int H = a.pv.kv_heads, G = a.group, bs = a.pv.block_size;
  const int chunks = a.chunk_prefix[H];
  const int f = (int)blockIdx.x / chunks;
  const int ci = (int)blockIdx.x - f * chunks;
  int h = 0;
  while (a.chunk_prefix[h + 1] <= ci) ++h;
  const int c = ci - a.chunk_prefix[h];
  const int C = (a.g.nblk_prefix[h + 1] - a.g.nblk_prefix[h]) * bs;
  const int w = a.g.window[h];
  const int first = (int)blockIdx.y * a.seqs_per_cta;
  if (threadIdx.x == 0 && ci == 0 && first == 0 && a.prefix_lens[f] < 0) atomicOr(a.pv.err, HWKV_DEVERR_NEG_LENGTH);
  if (threadIdx.x < 32) {
    const int n = shared_members(a, f, first, a.seqs_per_cta, s_seq, threadIdx.x);
    if (threadIdx.x == 0) s_count = n;
  }
  __syncthreads();
  const int seqs = s_count;
  if (seqs == 0) return;
  const int rows = seqs * G;
  const int N = prefix_len(a, f);

  for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
    const int r = e / D, d = e - r * D;
    float x = 0.f;
    if (r < rows) x = load_in<T>(static_cast<const T*>(a.q) + (((int64_t)s_seq[r / G] * H + h) * G + r % G) * D + d);
    s_q[r * kLd + d] = x;
  }
  const int r = threadIdx.x >> 2, part = threadIdx.x & 3;
  const bool live = r < rows;
  const int s = live ? s_seq[r / G] : 0;
  const int n = live ? shared_len(a, s) : 0;
  // a key's age, counted from the prefix's last token, that the row still sees
  const int reach = live ? max(0, w - n) : 0;
  const float slope = SC && live ? slope_log2(a.score, h * G + r % G) : 0.f;
  float m = kNegInf, l = 0.f;
  float acc[D / 4];
#pragma unroll
  for (int i = 0; i < D / 4; ++i) acc[i] = 0.f;

  const int t_begin = c * a.split_tokens, t_end = min(C, t_begin + a.split_tokens);
  for (int t0 = t_begin; t0 < t_end; t0 += kKeys) {
    __syncthreads();  // the pass before has been read
    {
      // four threads bring a key's row and a value's, 16 bytes at a time
      const int key = (int)threadIdx.x >> 2, t = t0 + key;
      constexpr int V = 16 / (int)sizeof(T), kVec = D / V;  // elements of a vector, vectors of a row
      const T* from = nullptr;
      if (t < t_end && ring_age(N, t, C) < min(N, w)) {
        const int j = t / bs;
        const int32_t blk = a.pv.tbl[a.g.tbl_base + (int64_t)f * a.g.tbl_seq_stride + a.g.nblk_prefix[h] + j];
        if (blk < 0 || (int64_t)blk >= a.pv.total_blocks) {
          if (part == 0) atomicOr(a.pv.err, HWKV_DEVERR_BAD_BLOCK);
        } else {
          from = static_cast<const T*>(a.pv.pool) + ((int64_t)blk * 2 * bs + (t - j * bs)) * D;
        }
      }
      uint4 kx[kVec / 4], vx[kVec / 4];
#pragma unroll
      for (int i = 0; i < kVec / 4; ++i) {
        kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
        if (from != nullptr) {
          kx[i] = *reinterpret_cast<const uint4*>(from + (4 * i + part) * V);
          vx[i] = *reinterpret_cast<const uint4*>(from + (int64_t)bs * D + (4 * i + part) * V);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec / 4; ++i) {
        float k[V], v[V];
        const uint32_t kw[4] = {kx[i].x, kx[i].y, kx[i].z, kx[i].w}, vw[4] = {vx[i].x, vx[i].y, vx[i].z, vx[i].w};
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (sizeof(T) == 4) {
            k[e] = __uint_as_float(kw[e]);
            v[e] = __uint_as_float(vw[e]);
          } else {
            k[e] = __uint_as_float((e & 1) ? (kw[e >> 1] & 0xFFFF0000u) : (kw[e >> 1] << 16));
            v[e] = __uint_as_float((e & 1) ? (vw[e >> 1] & 0xFFFF0000u) : (vw[e >> 1] << 16));
          }
        }
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const int d = (4 * i + part) * V + e;
          *reinterpret_cast<float4*>(s_k + key * kLd + d) = make_float4(k[e], k[e + 1], k[e + 2], k[e + 3]);
          *reinterpret_cast<float4*>(s_v + key * kLd + d) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    __syncthreads();
    float sc[kKeys / 4];
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < kKeys / 4; ++j) sc[j] = 0.f;
    for (int d = 0; d < D; d += 4) {
      const float4 q = *reinterpret_cast<const float4*>(s_q + r * kLd + d);
#pragma unroll
      for (int j = 0; j < kKeys / 4; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(s_k + (4 * j + part) * kLd + d);
        sc[j] = fmaf(q.w, k.w, fmaf(q.z, k.z, fmaf(q.y, k.y, fmaf(q.x, k.x, sc[j]))));
      }
    }
#pragma unroll
    for (int j = 0; j < kKeys / 4; ++j) {
      const int t = t0 + 4 * j + part;
      const int age = t < t_end ? ring_age(N, t, C) : INT32_MAX;
      const bool seen = age < N && age < reach;
      const float x = SC ? scored_log2<sizeof(T) == 4>(a.score, a.scale_log2, sc[j], slope, (float)((uint32_t)age + (uint32_t)n))
                         : sc[j] * a.scale_log2;
      sc[j] = seen ? x : kNegInf;
      top = fmaxf(top, sc[j]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float mn = fmaxf(m, top);
    const float base = mn == kNegInf ? 0.f : mn;
    const float al = ex2(m - base);
    m = mn;
    l *= al;
#pragma unroll
    for (int j = 0; j < kKeys / 4; ++j) {
      const float p = ex2(sc[j] - base);
      l += p;
      s_p[r * (kKeys + 1) + 4 * j + part] = p;
    }
    __syncwarp();  // a row's four threads are of one warp
#pragma unroll
    for (int i = 0; i < D / 4; ++i) acc[i] *= al;
    for (int key = 0; key < kKeys; ++key) {
      const float p = s_p[r * (kKeys + 1) + key];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(s_v + key * kLd + 16 * i + 4 * part);
        acc[4 * i] = fmaf(p, v.x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(p, v.y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(p, v.z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(p, v.w, acc[4 * i + 3]);
      }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (!live) return;
  const int64_t slot = ((int64_t)s * chunks + ci) * G + r % G;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    *reinterpret_cast<float4*>(a.part_o + slot * D + 16 * i + 4 * part) =
        make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
  if (part == 0) reinterpret_cast<float2*>(a.part_ml)[slot] = make_float2(m, l);
}

template <int D>
constexpr int simt_smem() {
  return ((kRows + 2 * kKeys) * (D + 4) + kRows * (kKeys + 1)) * 4;
}

// The join, a CTA per (sequence, KV head): out = sum_i acc_i 2^(m_i - M) / sum_i l_i 2^(m_i - M) over the head's own
// partial and its prefix's, M = max_i m_i; nothing to attend to gives zeros.  A thread sums four columns of a head over every
// kSplit'th part, the states and sums of kAhead parts on their way at once; where a head has more
// threads than columns, their sums meet in shared memory.  The order of all sums is fixed.  Bound: two dependent loads and L2;
// 16 sequences of 8 heads, 78 partials: 5 us, 128 sequences of 8: 8.5.
constexpr int kAhead = 8;

template <typename T, int D, int threads>
__global__ void __launch_bounds__(threads, threads == 512 ? 1 : 768 / threads) shared_join_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int kV = D / 4;  // float4 columns of a head
  __shared__ float4 s_acc[threads];
  __shared__ float2 s_ml[threads];
  const int H = a.pv.kv_heads, G = a.group;
  const int s = (int)blockIdx.x / H, h = (int)blockIdx.x - s * H;
  const int64_t row = (int64_t)blockIdx.x * G;  // the first of the CTA's rows
  const int cols = G * kV;
  const int split = max(1, threads / cols);  // threads of a column
  const int e0 = split > 1 ? (int)threadIdx.x % cols : (int)threadIdx.x, k0 = split > 1 ? (int)threadIdx.x / cols : 0;
  griddep_wait();
  const int f = prefix_of(a, s, threadIdx.x == 0 && h == 0);
  int64_t part0 = 0, step = 0;  // partial rows of the first head
  int parts = 0;
  if (f >= 0 && a.tc) {
    // a record is there for every row that sees a key of the prefix
    const int4 rec = a.rec[blockIdx.x];
    if (min(prefix_len(a, f), a.g.window[h] - min(a.g.window[h], shared_len(a, s))) > 0) {
      // (one left by a launch that gave up a wait may say anything: it is read only within the partials)
      if (rec.x >= 0 && rec.y == 2 && rec.z >= 0 && rec.x + 2ll * rec.z < 2ll * a.slots + 2 && rec.w >= 0 && rec.w + G <= a.chain_rows) {
        part0 = (int64_t)rec.x * a.chain_rows + rec.w;
        step = (int64_t)rec.y * a.chain_rows;
        parts = rec.z;
      }
    }
  } else if (f >= 0) {
    const int chunks = a.chunk_prefix[H];
    part0 = ((int64_t)s * chunks + a.chunk_prefix[h]) * G;
    step = G;
    parts = a.chunk_prefix[h + 1] - a.chunk_prefix[h];
  }
  for (int c0 = 0; c0 < cols; c0 += threads) {  // more than one pass: heads of more columns than threads
    const int e = c0 + e0;
    const bool on = e < cols && k0 < split;
    const int g = on ? e / kV : 0, d = on ? e % kV : 0;
    float M = kNegInf, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // adds a part of state e and sums v, both at a reference of M already
    auto add = [&](float2 e, float4 v) {
      if (e.x == kNegInf) return;  // a part without a key: its sums may be anything
      const float x = ex2(e.x - M);
      L = fmaf(e.y, x, L);
      acc.x = fmaf(v.x, x, acc.x);
      acc.y = fmaf(v.y, x, acc.y);
      acc.z = fmaf(v.z, x, acc.z);
      acc.w = fmaf(v.w, x, acc.w);
    };
    auto raise = [&](float m) {
      if (m <= M) return;
      const float x = M == kNegInf ? 0.f : ex2(M - m);
      L *= x;
      acc = make_float4(acc.x * x, acc.y * x, acc.z * x, acc.w * x);
      M = m;
    };
    if (on) {
      const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + part0 + g;
      const float4* po = reinterpret_cast<const float4*>(a.part_o + (part0 + g) * D) + d;
      float2 own = make_float2(kNegInf, 0.f);
      float4 own_v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 == 0) {
        own = reinterpret_cast<const float2*>(a.own_ml)[row + g];
        own_v = reinterpret_cast<const float4*>(a.own_acc + (row + g) * D)[d];
        own.x += a.own_shift;
      }
      for (int i0 = k0; i0 < parts || i0 == k0; i0 += kAhead * split) {
        float2 st[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int i = i0 + j * split;
          st[j] = make_float2(kNegInf, 0.f);
          if (i < parts) {
            st[j] = ml[i * step];
            v[j] = po[i * step * kV];
          }
        }
        float m = kNegInf;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) m = fmaxf(m, st[j].x);
        if (i0 == k0) m = fmaxf(m, own.x);
        raise(m);
        if (i0 == k0) add(own, own_v);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) add(st[j], v[j]);
      }
    }
    if (split > 1) {
      s_acc[threadIdx.x] = acc;
      s_ml[threadIdx.x] = make_float2(M, L);
      __syncthreads();
      if (on && k0 == 0) {
        for (int k = 1; k < split; ++k) {
          const float2 e2 = s_ml[k * cols + e0];
          raise(e2.x);
          add(e2, s_acc[k * cols + e0]);
        }
      }
    }
    if (on && k0 == 0) {
      const float inv = L > 0.f ? 1.f / L : 0.f;
      T* out = static_cast<T*>(a.out) + (row + g) * D + 4 * d;
      if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(out) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      else *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
  }
}

template <typename T, int D, bool SC>
cudaError_t launch_simt(const SharedArgs& a, dim3 grid, cudaStream_t st) {
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(shared_simt_kernel<T, D, SC>, cudaFuncAttributeMaxDynamicSharedMemorySize, simt_smem<D>());
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)simt_smem<D>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_simt_kernel<T, D, SC>, a);
}

template <typename T, int D>
cudaError_t launch_simt(const SharedArgs& a, dim3 grid, cudaStream_t st) {
  return a.score.on ? launch_simt<T, D, true>(a, grid, st) : launch_simt<T, D, false>(a, grid, st);
}

template <typename T, int D, int threads>
cudaError_t launch_join(const SharedArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.pv.kv_heads));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_join_kernel<T, D, threads>, a);
}

// Few heads: more threads for each, which share its parts (96 heads of 8 queries and 22 parts: 10 us with 128 threads, 4.5 with 512;
// 1024 heads of 8 and 6 parts: 8.5 with 128, 10.8 with 256 of as many registers as 512 want).
template <typename T, int D>
cudaError_t launch_join(const SharedArgs& a, cudaStream_t st) {
  const int64_t ctas = (int64_t)a.num_seqs * a.pv.kv_heads;
  return ctas <= 200 ? launch_join<T, D, 512>(a, st) : ctas <= 800 ? launch_join<T, D, 256>(a, st) : launch_join<T, D, 128>(a, st);
}

}  // namespace

int shared_simt_seqs(int group) { return std::max(1, kRows / group); }

cudaError_t launch_shared_simt(const SharedArgs& a, int dtype, int chunks, cudaStream_t st) {
  const dim3 grid((unsigned)(a.num_prefixes * (int64_t)chunks), (unsigned)((a.num_seqs + a.seqs_per_cta - 1) / a.seqs_per_cta));
  const int D = a.pv.head_dim;
  cudaError_t e = cudaErrorInvalidValue;
  if (dtype == HWKV_F32) e = D == 128 ? launch_simt<float, 128>(a, grid, st) : launch_simt<float, 64>(a, grid, st);
  else if (dtype == HWKV_BF16) e = D == 128 ? launch_simt<__nv_bfloat16, 128>(a, grid, st) : launch_simt<__nv_bfloat16, 64>(a, grid, st);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_shared_join(const SharedArgs& a, bool f32, cudaStream_t st) {
  const bool wide = a.pv.head_dim == 128;
  const cudaError_t e = f32 ? (wide ? launch_join<float, 128>(a, st) : launch_join<float, 64>(a, st))
                            : (wide ? launch_join<__nv_bfloat16, 128>(a, st) : launch_join<__nv_bfloat16, 64>(a, st));
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace hwkv
