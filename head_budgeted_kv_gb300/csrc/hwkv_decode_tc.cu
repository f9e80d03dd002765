// The stream-K decode kernel (hwkv_decode_sk.cuh) for pools that hold the element type itself:
// tile work on the tensor cores for bf16, on the CUDA cores for fp32; and the choice between
// these instances and those for 8-bit pools (hwkv_decode_q8.cu).
#include "hwkv_decode_sk.cuh"

namespace hwkv {
namespace {

template <int D>
cudaError_t configure_dim(int dtype, int ctas_per_sm[kGroupPads]) {
  cudaError_t e;
  if (dtype == HWKV_F32) {  // fp32: one instance, up to 4 query heads per KV head
    ctas_per_sm[1] = ctas_per_sm[2] = 0;
    return configure_one<float, D, 4>(&ctas_per_sm[0]);
  }
  if ((e = configure_one<__nv_bfloat16, D, 4>(&ctas_per_sm[0])) != cudaSuccess) return e;
  if ((e = configure_one<__nv_bfloat16, D, 8>(&ctas_per_sm[1])) != cudaSuccess) return e;
  return configure_one<__nv_bfloat16, D, 16>(&ctas_per_sm[2]);
}

template <typename T, int D>
cudaError_t launch_dim(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if constexpr (sizeof(T) == 4) {
    return a.group <= 4 ? launch_one<T, D, 4>(a, tmap, ctas, st) : cudaErrorInvalidValue;
  } else {
    switch (decode_tc_group_pad(a.group)) {
      case 4: return launch_one<T, D, 4>(a, tmap, ctas, st);
      case 8: return launch_one<T, D, 8>(a, tmap, ctas, st);
      default: return launch_one<T, D, 16>(a, tmap, ctas, st);
    }
  }
}

}  // namespace

int decode_tc_group_pad(int group) { return group <= 4 ? 4 : group <= 8 ? 8 : 16; }

int decode_tc_pad_index(int group) { return group <= 4 ? 0 : group <= 8 ? 1 : 2; }

cudaError_t configure_decode_tc(int head_dim, int dtype, int ctas_per_sm[kGroupPads]) {
  if (dtype == HWKV_E4M3) return configure_decode_q8(head_dim, ctas_per_sm);
  if (head_dim == 128) return configure_dim<128>(dtype, ctas_per_sm);
  if (head_dim == 64) return configure_dim<64>(dtype, ctas_per_sm);
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_tc(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.elem_bytes == 1) return launch_decode_q8(a, tmap, ctas, st);
  if (a.score.on) return launch_decode_score(a, tmap, ctas, st);
  const bool f32 = a.pv.elem_bytes == 4;
  if (a.pv.head_dim == 128) return f32 ? launch_dim<float, 128>(a, tmap, ctas, st) : launch_dim<__nv_bfloat16, 128>(a, tmap, ctas, st);
  if (a.pv.head_dim == 64) return f32 ? launch_dim<float, 64>(a, tmap, ctas, st) : launch_dim<__nv_bfloat16, 64>(a, tmap, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace hwkv
