// What the kernels of rotary positions share: 16-byte vectors of a row as fp32, the turn of a pair, and
// its angle (hwkv_rope.cu for rows, hwkv_rope_q8.cu for rows stored in 8-bit pools).
#pragma once

#include "hwkv_device.cuh"

namespace hwkv {
namespace {

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

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = fmaf(x, c, -(y * s));
  b = fmaf(y, c, x * s);
}

// The cosine and sine of p F / 2^64 turns, times the magnitude (see hwkv_rope.cu for the arithmetic).
__device__ __forceinline__ void turn_angle(uint64_t turns, uint32_t p, float magnitude, float& cn, float& sn) {
  const float x = (float)(int32_t)((turns * (uint64_t)p) >> 32) * 0x1p-31f;  // half turns
  sincospif(x, &sn, &cn);
  cn *= magnitude;
  sn *= magnitude;
}

// The same from the nearest quarter turn: what is left is below an eighth of a turn, so that its fp32 value is off by 2^-26 rad,
// not 2^-23 (codes of 8 bits stand on the exact turned value, where fp32 and bf16 outputs round it away).
__device__ __forceinline__ void turn_angle_fine(uint64_t turns, uint32_t p, float magnitude, float& cn, float& sn) {
  const uint64_t t = turns * (uint64_t)p;
  const uint32_t quarter = (uint32_t)((t + (1ull << 61)) >> 62);      // modulo 4
  const int32_t rest = (int32_t)(uint32_t)((t << 2) >> 32);       // from there, 2^-33 half turns
  float s, c;
  sincospif((float)rest * 0x1p-33f, &s, &c);
  const float a = quarter & 1u ? -s : c, b = quarter & 1u ? c : s;    // (cos, sin) a quarter further for odd ones
  cn = (quarter & 2u ? -a : a) * magnitude;
  sn = (quarter & 2u ? -b : b) * magnitude;
}

}  // namespace
}  // namespace hwkv
