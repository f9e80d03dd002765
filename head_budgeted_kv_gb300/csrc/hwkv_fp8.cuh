// 8-bit storage of cache rows: e4m3 codes with one power-of-two scale per group of 16
// consecutive ring slots, for K and for V (HWKV_E4M3 pools).
//
// A group's value is code * 2^e with the smallest e >= -120 for which the largest finite
// magnitude of the group is at most 448 * 2^e, 448 being the largest e4m3 number; so the
// largest magnitude lies in (224, 448] * 2^e unless e is clamped.  A power of two costs e4m3
// nothing against an exact amax / 448 (a floating-point code's relative step does not depend on
// the scale) and makes both directions exact but for the one rounding to a code: scaling by 2^-e
// rounds nothing, and when a later token makes the group's scale anew (GroupRecode), the codes
// move by a power of two, which rounds only those that become subnormal.
// What is not finite is stored as NaN and does not count for the scale.
#pragma once

#include <cuda_fp16.h>

#include "hwkv_device.cuh"

namespace hwkv {

constexpr int kScaleGroup = 16;     // ring slots that share a scale
constexpr int kMinScaleExp = -120;  // smallest scale exponent (2^e and 2^-e stay normal fp32)

// The smallest e >= kMinScaleExp with amax <= 448 * 2^e, for a finite amax >= 0.  For a normal amax = f * 2^x with
// f in [1, 2): 448 = 1.75 * 2^8, so e = x - 8, one more when f > 1.75.  A subnormal amax reads
// as x = -127 and is clamped like every other x < -112.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExp);
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 1 / s for a power of two s in [2^-126, 2^126]
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

// |x| when it is finite, else 0 (x counts for a group's scale only when finite)
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_huge_valf() ? a : 0.f;
}

// two e4m3 codes (lo in the low byte), round to nearest even; what is not finite becomes NaN
// (the conversion itself would saturate an infinity to 448)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  const float nan = __uint_as_float(0x7FFFFFFFu);
  lo = fabsf(lo) < __builtin_huge_valf() ? lo : nan;
  hi = fabsf(hi) < __builtin_huge_valf() ? hi : nan;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// four codes to two pairs of fp16, exactly (bytes 0, 1 to `lo`, bytes 2, 3 to `hi`)
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }

// the four bytes' largest magnitude code that is not NaN, byte by byte against `best`
__device__ __forceinline__ uint32_t code_max4(uint32_t best, uint32_t x) {
  const uint32_t m = x & 0x7F7F7F7Fu;
  return __vmaxu4(best, m & ~__vcmpeq4(m, 0x7F7F7F7Fu));
}

// the value of the largest of four magnitude codes (codes order like their values)
__device__ __forceinline__ float code_max_value(uint32_t best) {
  const uint32_t b = max(max(best & 0xFFu, (best >> 8) & 0xFFu), max((best >> 16) & 0xFFu, best >> 24));
  uint32_t lo, hi;
  e4m3x4_to_f16(b, lo, hi);
  return half2_to_float2(lo).x;
}

// 16 codes times `factor`, rounded to codes again
__device__ __forceinline__ uint4 rescale_codes(uint4 c, float factor) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(w[i], lo, hi);
    const float2 a = half2_to_float2(lo), b = half2_to_float2(hi);
    w[i] = e4m3x2(a.x * factor, a.y * factor) | (e4m3x2(b.x * factor, b.y * factor) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bf16 values (two 16-byte vectors) as fp32
struct Row16 {
  float v[16];
};

__device__ __forceinline__ Row16 widen16(uint4 a, uint4 b) {
  Row16 r;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

__device__ __forceinline__ uint4 encode16(const Row16& r, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2(r.v[4 * i] * inv, r.v[4 * i + 1] * inv) | (e4m3x2(r.v[4 * i + 2] * inv, r.v[4 * i + 3] * inv) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 finite bf16 values (a 16-byte vector) times a power of two, as codes
__device__ __forceinline__ uint2 encode8_finite(uint4 a, float inv) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  uint16_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = fmul2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), make_float2(inv, inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[i]) : "f"(x.y), "f"(x.x));
  }
  return make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16), (uint32_t)c[2] | ((uint32_t)c[3] << 16));
}

// the same for any 8 values: what is not finite becomes NaN
__device__ __forceinline__ uint2 encode8(uint4 a, float inv) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// Storing a new token's row into one group (K or V) with the whole warp, scaling the group anew:
// the row at slot `new_slot` (position `pos`) is replaced; the stored values of the other slots of
// the group whose positions are in the window [pos + 1 - w, pos) are kept at the new scale, and every
// other slot becomes zero.  Three steps, so that K and V can take them side by side:
//   load     the chunks a lane owns (16 bytes of codes each), and its chunk of the new row;
//   amax     the largest finite magnitude this lane sees (to be maximised over the warp);
//   store    the chunks at the new scale.
template <int D>
struct GroupRecode {
  static constexpr int kChunks = D / 16;                   // 16-byte chunks of a row of codes
  static constexpr int kPer = kScaleGroup * kChunks / 32;  // chunks a lane owns: rows 32 / kChunks apart,
                                                           // so at most one is of the new row
  uint4 code[kPer];
  int kind[kPer];  // 0 zero, 1 kept, 2 the new row
  uint4 fresh[2];  // chunk lane % kChunks of the new row, bf16

  // t0: first slot of the group, C: ring capacity; ld(r, c): 16-byte chunk c of row r
  template <typename Ld>
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int t0, int new_slot, int pos, int w, int C, Ld ld,
                                       int lane) {
    const uint4* src = reinterpret_cast<const uint4*>(row + 16 * (lane % kChunks));
    fresh[0] = src[0];
    fresh[1] = src[1];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (lane + 32 * i) / kChunks;
      int age = new_slot - (t0 + r);
      if (age < 0) age += C;
      kind[i] = age == 0 ? 2 : (age < w && age <= pos ? 1 : 0);
      code[i] = make_uint4(0u, 0u, 0u, 0u);
      if (kind[i] == 1) code[i] = ld(r, lane % kChunks);
    }
  }

  __device__ __forceinline__ float amax(float old_scale) const {
    float m = 0.f;
    uint32_t best = 0u;
    bool owner = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      owner = owner || kind[i] == 2;
      best = code_max4(code_max4(code_max4(code_max4(best, code[i].x), code[i].y), code[i].z), code[i].w);
    }
    if (owner) {
      const Row16 x = widen16(fresh[0], fresh[1]);
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, finite_abs(x.v[e]));
    }
    return fmaxf(m, code_max_value(best) * old_scale);
  }

  // amax: over the warp; st(r, c, v) writes a chunk.  Returns the new scale.
  template <typename St>
  __device__ __forceinline__ float store(float amax, float old_scale, St st, int lane) {
    const float scale = pow2i(scale_exponent(amax)), inv = pow2_inverse(scale);
    // a kept code that is not 0 bounds this by 2^18; with none the product may overflow, and 0
    // times infinity must stay 0
    const float factor = fminf(old_scale * inv, 0x1p100f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint4 v = code[i];
      if (kind[i] == 2) v = encode16(widen16(fresh[0], fresh[1]), inv);
      else if (factor != 1.f) v = rescale_codes(v, factor);
      st((lane + 32 * i) / kChunks, lane % kChunks, v);
    }
    return scale;
  }
};

}  // namespace hwkv
