// Tile-level pieces of the stream-K decode kernel for 8-bit pools (hwkv_decode_q8.cu; HWKV_E4M3,
// hwkv_fp8.cuh): the loads of one 16-token tile with its two scales, the fused
// append, and one warp's work on a tile.
//
// With K = k_scale * Kc and V = v_scale * Vc for the codes Kc, Vc of a tile (one group of 16
// slots, so one pair of scales):
//   S = (Kc . Qn^T) * (k_scale * qs)       Qn = Q / qs, qs a power of two per query head
//   O = sum over tiles of (P * v_scale) . Vc
// Codes become fp16 exactly, one conversion instruction per two values, and feed
// mma.sync.m16n8k16 fp16 -> fp32.  fp16's range is kept in two exact ways.  Each query head is
// scaled by a power of two so its largest element lies in [2^14, 2^15) (the elements then lose
// nothing above 2^-39 of that largest one).  And P * v_scale is formed relative to a reference of its own:
// with m the integer reference maximum of the scores s (log2 units) and e the one of s + log2(v_scale) - m,
//   p = 2^(s - m)                            fp32, summed to l
//   p * v_scale = 2^e * 2^(s - m + log2(v_scale) - e)
// where the last factor, times 2^11, is what fp16 holds: the largest of a head lies in [2^11, 2^12), or up
// to 2^15.98 while a reference lags.  So a product of weight and scale keeps its 11 bits down to 2^-25 of its
// head's largest and is off by at most 2^-36 of that below, and a group whose scale is large but whose
// weight is not has no say in it.  (With the scale relative to the largest one met, whatever its weight, such a
// group 2^24 above the others put 12% into the result and one 2^37 above them erased it.)  m and e are
// integers, so no reference is rounded, and 2^e is exact where O leaves the warp.  The second exponential per
// weight costs up to 2% of a decode whose references seldom move and 6% where steep slopes move them at every
// stage (policy layer, uncapped 55.0 -> 55.1 us, biased 57.5 -> 62); a product by the power of two instead of it
// is slower (61 at cap 50 against 57).
// A dim or token index may be permuted freely inside a contraction: K's bytes are fed in the
// order ldmatrix delivers them, against queries loaded in the same order, and V's columns come
// out as dim pairs (2i, 2i + 1) in the accumulator's row halves, which publish() undoes.
#pragma once

#include "hwkv_decode_tile.cuh"
#include "hwkv_fp8.cuh"

namespace hwkv {
namespace {

// Byte offset of byte b of row r of a 16-row tile of codes, as TMA stores it: rows of D bytes,
// 128-byte swizzle for D = 128 (chunk ^ row % 8), 64-byte swizzle for D = 64 (chunk ^ row / 2 % 4).
template <int D>
__device__ __forceinline__ uint32_t swz_q8(int row, int b) {
  const int c = b >> 4;
  if constexpr (D == 128) return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4) + (b & 15));
  else return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4) + (b & 15));
}

// The copy of one tile whose table entry `blk` is in range, first row r0 of the block: K and V rows
// in one box of the 3-D map (head_dim, block_size rows, 2 * block + K/V).
template <int D>
__device__ __forceinline__ void issue_tile_q8(const CUtensorMap* tmap, int blk, int r0, uint32_t dst, uint64_t* bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(r0), "r"(2 * blk), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// Fused append: when the tile starting at slot t0 is the new token's group, the group is stored
// anew with the new row (GroupRecode), in shared memory and in the pool, with its scales.  No
// other CTA reads this tile, or its scales, in the launch.  A call of its own: it happens once per
// group and would only fill the tile loop's registers and instruction cache.
template <int D>
__device__ __noinline__ void patch_new_row_q8(const DecodeArgs& a, const int32_t* tbl, int s, int h, int pos, int C,
                                              int t0, int new_slot, uint32_t sK, float2* slot, int lane) {
  const float2 old = *slot;
  __syncwarp();
  const int bs = a.pv.block_size;
  const int jb = t0 / bs, r0 = t0 - jb * bs;
  const int32_t blk = tbl[jb];
  const bool blk_ok = blk >= 0 && (int64_t)blk < a.pv.total_blocks;
  const int64_t src = ((int64_t)s * a.pv.kv_heads + h) * D;
  auto ld = [&](uint32_t base) {
    return [base](int r, int c) {
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(base + swz_q8<D>(r, 16 * c)));
      return v;
    };
  };
  auto st = [&](uint32_t base, uint8_t* dst) {
    return [base, dst, blk_ok](int r, int c, uint4 v) {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(base + swz_q8<D>(r, 16 * c)), "r"(v.x), "r"(v.y),
                   "r"(v.z), "r"(v.w)
                   : "memory");
      if (blk_ok) *reinterpret_cast<uint4*>(dst + r * D + 16 * c) = v;
    };
  };
  GroupRecode<D> k, v;
  k.load(static_cast<const __nv_bfloat16*>(a.k_new) + src, t0, new_slot, pos, a.g.window[h], C, ld(sK), lane);
  v.load(static_cast<const __nv_bfloat16*>(a.v_new) + src, t0, new_slot, pos, a.g.window[h], C, ld(sK + kTile * D), lane);
  float mk = k.amax(old.x), mv = v.amax(old.y);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
  }
  uint8_t* rows = static_cast<uint8_t*>(a.pv.pool) + ((int64_t)(blk_ok ? blk : 0) * 2 * bs + r0) * D;
  const float2 now = make_float2(k.store(mk, old.x, st(sK, rows), lane),
                                 v.store(mv, old.y, st(sK + kTile * D, rows + (int64_t)bs * D), lane));
  if (lane == 0) {
    *slot = now;
    const int64_t group = (int64_t)blk * (bs / kScaleGroup) + r0 / kScaleGroup;
    if (blk_ok) *reinterpret_cast<float2*>(a.pv.scales + group * 2) = now;
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8-bit pools: the GQA group on the N side of mma.sync as for bf16, fp32 accumulators in units of
// 2^(er - kShift) per head.
template <int D, int GP, bool SC>
struct WarpState<E4m3, D, GP, SC> {
  static constexpr int NT = (GP + 7) / 8;
  static constexpr float kShift = 11.f;   // log2 of the factor P * v_scale carries over its reference
  static constexpr float kSlack = 4.98f;  // log2 of how far it, or a weight, may pass its reference: below fp16's end
  static constexpr float kNone = -3e38f;  // the reference before any score: finite, so differences are no NaN
  // 2^5 for the slack is taken out of sums and accumulators alike where they leave the warp, and the shift out
  // of the accumulators: weights are then at most 1, and no V that bf16 holds overflows by itself
  static constexpr float kTakeSum = 0x1p-5f, kTakeAcc = 0x1p-16f;
  uint32_t qf[NT][D / 16][2];
  float acc[D / 16][NT][4];
  float mx[NT][2];   // reference maximum of the scores (log2 units, an integer)
  float er[NT][2];   // reference of score + log2(V scale), less mx: an integer from -120 to 120
  float2 ls[NT];     // this lane's partial sums of 2^(score - mx)
  float qs[NT][2];  // the power of two taken out of each of the lane's heads (times |scale| log2(e) unless SC)
  float slope[NT][2];  // SC: of the lane's heads, log2 units

  // Q of the group, normalised: the lane holds q[g][16i + 4*q4 .. + 3], g = 8*nt + lane / 4
  __device__ __forceinline__ void begin(const DecodeArgs& a, const Group& gr, int G, int lane) {
    const int gq = lane >> 2, q4 = lane & 3;
    const int Hq = a.pv.kv_heads * G;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = 8 * nt + gq;
      const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)gr.s * Hq + gr.h * G + g) * D;
      uint2 raw[D / 16];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        raw[i] = g < G ? *reinterpret_cast<const uint2*>(qrow + 16 * i + 4 * q4) : make_uint2(0u, 0u);
        const float x0 = __uint_as_float(raw[i].x << 16), x1 = __uint_as_float(raw[i].x & 0xFFFF0000u);
        const float x2 = __uint_as_float(raw[i].y << 16), x3 = __uint_as_float(raw[i].y & 0xFFFF0000u);
        top = fmaxf(top, fmaxf(fmaxf(finite_abs(x0), finite_abs(x1)), fmaxf(finite_abs(x2), finite_abs(x3))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // top = f * 2^x, f in [1, 2): elements times 2^(14 - x); x is clamped so the factor is normal
      const int x = max((int)(__float_as_uint(top) >> 23) - 127, -112);
      // (a negative scale's sign goes into the elements: scores' factors stay positive)
      const float f = !SC && a.scale_log2 < 0.f ? -pow2i(14 - x) : pow2i(14 - x);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qf[nt][i][0] = pack_f16(__uint_as_float(raw[i].x << 16) * f, __uint_as_float(raw[i].x & 0xFFFF0000u) * f);
        qf[nt][i][1] = pack_f16(__uint_as_float(raw[i].y << 16) * f, __uint_as_float(raw[i].y & 0xFFFF0000u) * f);
      }
      // the accumulator's columns are heads 2 q4 and 2 q4 + 1
      const float inv = pow2i(x - 14);
      qs[nt][0] = __shfl_sync(0xffffffffu, inv, (2 * q4) * 4) * (SC ? 1.f : fabsf(a.scale_log2));
      qs[nt][1] = __shfl_sync(0xffffffffu, inv, (2 * q4 + 1) * 4) * (SC ? 1.f : fabsf(a.scale_log2));
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[j][nt][0] = acc[j][nt][1] = acc[j][nt][2] = acc[j][nt][3] = 0.f;
      mx[nt][0] = mx[nt][1] = kNone;
      er[nt][0] = er[nt][1] = 0.f;
      ls[nt] = make_float2(0.f, 0.f);
    }
    if constexpr (SC) load_slopes<NT>(a, gr, G, lane, slope);
  }

  // whether the tile at slot t0 holds slots outside the window (or the window's two ends)
  static __device__ __forceinline__ bool partly_resident(const Group& gr, int t0) {
    int first = t0 - gr.rs.first_slot;
    if (first < 0) first += gr.rs.C;
    return first + kTile > gr.rs.n;
  }

  // The raw scores s of M tiles capped, biased and in log2 units.  While no score of the warp
  // reaches the cap the polynomial alone serves, on packed pairs (a capped policy layer 65 -> 55 us when it
  // came; now 58, uncapped 55, past the cap 83).
  template <int M>
  __device__ __forceinline__ void score_tiles(const DecodeArgs& a, const Group& gr, const int (&t0)[M], float (&s)[M][NT][4],
                                              int gq) const {
    bool past = false;  // the cap; judged by the slots in the window alone where one outside seems to pass it
    if (a.score.capped) {
      auto passes = [&](bool all) {
        float top = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const bool v0 = all || slot_valid(gr.rs, t0[m] + gq), v1 = all || slot_valid(gr.rs, t0[m] + gq + 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, (e < 2 ? v0 : v1) ? fabsf(s[m][nt][e]) : 0.f);
        }
        return __any_sync(0xffffffffu, top * fabsf(a.score.cap_in) > 1.f) != 0;
      };
      past = !a.score.poly_on || (passes(true) && passes(false));
    }
    const float2 sl = make_float2(a.scale_log2, a.scale_log2);
    if (!a.score.capped) {
#pragma unroll
      for (int i = 0; i < M * NT * 2; ++i) {
        float* x = &s[i / (NT * 2)][i / 2 % NT][i % 2 * 2];
        const float2 y = fmul2(make_float2(x[0], x[1]), sl);
        x[0] = y.x, x[1] = y.y;
      }
    } else if (!past) {
#pragma unroll
      for (int i = 0; i < M * NT * 2; ++i) {
        float* x = &s[i / (NT * 2)][i / 2 % NT][i % 2 * 2];
        const float2 v = make_float2(x[0], x[1]), t = fmul2(v, v);
        float2 p = make_float2(a.score.poly[5], a.score.poly[5]);
#pragma unroll
        for (int k = 4; k >= 0; --k) p = ffma2(t, p, make_float2(a.score.poly[k], a.score.poly[k]));
        const float2 y = fmul2(v, p);
        x[0] = y.x, x[1] = y.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < M * NT * 4; ++i) {
        float& x = s[i / (NT * 4)][i / 4 % NT][i % 4];
        x = a.score.cap_out * tanh_f32<false>(x * a.score.cap_in);
      }
    }
    if (a.score.slopes != nullptr) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float d0 = -(float)slot_distance(gr.rs, t0[m] + gq), d1 = -(float)slot_distance(gr.rs, t0[m] + gq + 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 k = make_float2(slope[nt][0], slope[nt][1]);
          const float2 x = ffma2(k, make_float2(d0, d0), make_float2(s[m][nt][0], s[m][nt][1]));
          const float2 y = ffma2(k, make_float2(d1, d1), make_float2(s[m][nt][2], s[m][nt][3]));
          s[m][nt][0] = x.x, s[m][nt][1] = x.y, s[m][nt][2] = y.x, s[m][nt][3] = y.y;
        }
      }
    }
  }

  // M tiles at once: more work between the waits, one check of the maximum for all of them.
  // `slot[m]` and `sK[m]` are tile m's scales (K, V) and codes (V kTile * D bytes after K).  Returns true
  // when shared memory was written (the caller fences before TMA refills the stages).
  template <int M>
  __device__ __forceinline__ bool consume(const DecodeArgs& a, const Group& gr, const int (&t0)[M],
                                          const uint32_t (&sK)[M], const float2* (&slot)[M], int lane) {
    const int gq = lane >> 2;
    // ldmatrix lane roles: matrices 0, 1 are rows 0-7, 8-15 of a 16-byte chunk, matrices 2, 3 those of
    // the next; the swizzle xors the chunk index, so chunk i + {0, 1} of a tile is one xor away
    const uint32_t lane_off = swz_q8<D>((lane & 7) + ((lane >> 3) & 1) * 8, (lane >> 4) * 16);
    bool dirty = false;

    float s[M][NT][4];  // scores in log2 units (SC: raw until score_tiles)
    float ev[M];  // log2 of each tile's V scale
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float2 sc = *slot[m];
      // (a scale of 0, of a group never stored, has codes 0: any exponent serves)
      ev[m] = (float)max((int)(__float_as_uint(sc.y) >> 23) - 127, kMinScaleExp);
      constexpr bool kTwoChains = M * NT < 4;  // few scores at once: shorter accumulation chains
      float sb[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][nt][e] = sb[nt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
        uint32_t w[4], a0[4], a1[4];
        ldsm_x4(w, (sK[m] + lane_off) ^ (uint32_t)(16 * i));
        e4m3x4_to_f16(w[0], a0[0], a0[2]);
        e4m3x4_to_f16(w[1], a0[1], a0[3]);
        e4m3x4_to_f16(w[2], a1[0], a1[2]);
        e4m3x4_to_f16(w[3], a1[1], a1[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(s[m][nt], a0, qf[nt][i][0], qf[nt][i][1]);
          if constexpr (kTwoChains) mma_f16(sb[nt], a1, qf[nt][i + 1][0], qf[nt][i + 1][1]);
          else mma_f16(s[m][nt], a1, qf[nt][i + 1][0], qf[nt][i + 1][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (kTwoChains) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[m][nt][e] += sb[nt][e];
        }
        // rounded here, not in a multiply-add with the reference: a difference of two scores is then exact
        // where it counts, however large they are
        const float2 f = make_float2(qs[nt][0] * sc.x, qs[nt][1] * sc.x);
        const float2 x = fmul2(make_float2(s[m][nt][0], s[m][nt][1]), f);
        const float2 y = fmul2(make_float2(s[m][nt][2], s[m][nt][3]), f);
        s[m][nt][0] = x.x, s[m][nt][1] = x.y, s[m][nt][2] = y.x, s[m][nt][3] = y.y;
      }
    }
    if constexpr (SC) score_tiles<M>(a, gr, t0, s, gq);

#pragma unroll
    for (int m = 0; m < M; ++m) {
      // a tile with slots outside the window: their scores are masked, and their V rows zeroed, as
      // 0 times a NaN is not 0
      if (partly_resident(gr, t0[m])) {
        const bool v0 = slot_valid(gr.rs, t0[m] + gq), v1 = slot_valid(gr.rs, t0[m] + gq + 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[m][nt][e] = (e < 2 ? v0 : v1) ? s[m][nt][e] : kNegInf;
        const int r = lane >> 1;
        if (!slot_valid(gr.rs, t0[m] + r)) {
          for (int c = lane & 1; c < D / 16; c += 2)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sK[m] + kTile * D + swz_q8<D>(r, 16 * c)), "r"(0u)
                         : "memory");
        }
        __syncwarp();
        dirty = true;
      }
    }

    // The references move only when a weight, or its product with the V scale, passes its own by more than
    // 2^kSlack: seldom after a group's first tiles, so the common case reduces nothing over the warp and
    // rescales nothing.  (The products are judged by the tiles' largest scale: at worst a step in vain.)
    float ev_max = ev[0];
#pragma unroll
    for (int m = 1; m < M; ++m) ev_max = fmaxf(ev_max, ev[m]);
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = kNegInf;
#pragma unroll
        for (int m = 0; m < M; ++m) x = fmaxf(x, fmaxf(s[m][nt][c], s[m][nt][c + 2]));
        top[nt][c] = x;
        grow = grow || x - mx[nt][c] + fmaxf(ev_max - er[nt][c], 0.f) > kSlack;
      }
    if (__any_sync(0xffffffffu, grow)) {
      auto over_lanes = [](float v) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        return v;
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float n = fmaxf(mx[nt][c], floorf(over_lanes(top[nt][c])));
          float w = kNegInf;
#pragma unroll
          for (int m = 0; m < M; ++m) w = fmaxf(w, fmaxf(s[m][nt][c], s[m][nt][c + 2]) - n + ev[m]);
          const float fall = mx[nt][c] - n;  // at most 0, as is the accumulators' exponent
          const float e = fmaxf(er[nt][c] + fall, floorf(over_lanes(w)));
          const float al = ex2(fall), aa = ex2(er[nt][c] + fall - e);
          mx[nt][c] = n;
          er[nt][c] = e;
          (c ? ls[nt].y : ls[nt].x) *= al;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            acc[j][nt][c] *= aa;
            acc[j][nt][c + 2] *= aa;
          }
        }
    }

    uint32_t pb[M][NT][2];
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 nm = make_float2(-mx[nt][0], -mx[nt][1]);
        const float2 rel = make_float2(ev[m] + kShift - er[nt][0], ev[m] + kShift - er[nt][1]);
        const float2 x = fadd2(make_float2(s[m][nt][0], s[m][nt][1]), nm);
        const float2 y = fadd2(make_float2(s[m][nt][2], s[m][nt][3]), nm);
        ls[nt] = fadd2(ls[nt], fadd2(make_float2(ex2(x.x), ex2(x.y)), make_float2(ex2(y.x), ex2(y.y))));
        // exponentials of their own: a weight may be below fp32's range where its product with the scale is not
        const float2 xv = fadd2(x, rel), yv = fadd2(y, rel);
        const float2 pv = make_float2(ex2(xv.x), ex2(xv.y)), rv = make_float2(ex2(yv.x), ex2(yv.y));
        pb[m][nt][0] = movmatrix_trans(pack_f16(pv.x, pv.y));
        pb[m][nt][1] = movmatrix_trans(pack_f16(rv.x, rv.y));
      }
    }

#pragma unroll
    for (int j = 0; j < D / 16; j += 2) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        uint32_t w[4], a0[4], a1[4];
        ldsm_x4_trans(w, (sK[m] + kTile * D + lane_off) ^ (uint32_t)(16 * j));
        // bytes of a register: (token 2 q4, dims 2 gq, 2 gq + 1), (token 2 q4 + 1, the same dims)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __byte_perm(w[e], 0u, 0x3120);
        e4m3x4_to_f16(w[0], a0[0], a0[1]);
        e4m3x4_to_f16(w[1], a0[2], a0[3]);
        e4m3x4_to_f16(w[2], a1[0], a1[1]);
        e4m3x4_to_f16(w[3], a1[2], a1[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[j][nt], a0, pb[m][nt][0], pb[m][nt][1]);
          mma_f16(acc[j + 1][nt], a1, pb[m][nt][0], pb[m][nt][1]);
        }
      }
    }
    return dirty;
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        ls[nt].x += __shfl_xor_sync(0xffffffffu, ls[nt].x, off);
        ls[nt].y += __shfl_xor_sync(0xffffffffu, ls[nt].y, off);
      }
  }

  template <int SG>
  __device__ __forceinline__ void publish(int nt, int hh, int warp, int lane, float* sc_m, float* sc_l,
                                          float* sc_acc) const {
    const int gq = lane >> 2, q4 = lane & 3;
    const int c0 = 2 * q4 - hh * SG;  // this lane's first column within the pass
    if (c0 < 0 || c0 >= SG) return;
    if (gq == 0) {
      sc_m[warp * SG + c0] = mx[nt][0];
      sc_m[warp * SG + c0 + 1] = mx[nt][1];
      sc_l[warp * SG + c0] = ls[nt].x * kTakeSum;
      sc_l[warp * SG + c0 + 1] = ls[nt].y * kTakeSum;
    }
    const float u0 = pow2i((int)er[nt][0]) * kTakeAcc, u1 = pow2i((int)er[nt][1]) * kTakeAcc;
    float* wacc = sc_acc + warp * SG * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const int d = 16 * j + 2 * gq;
      *reinterpret_cast<float2*>(wacc + c0 * D + d) = make_float2(acc[j][nt][0] * u0, acc[j][nt][2] * u0);
      *reinterpret_cast<float2*>(wacc + (c0 + 1) * D + d) = make_float2(acc[j][nt][1] * u1, acc[j][nt][3] * u1);
    }
  }
};

}  // namespace
}  // namespace hwkv
