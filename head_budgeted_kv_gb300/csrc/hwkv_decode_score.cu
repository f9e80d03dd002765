// The stream-K decode kernel (hwkv_decode_sk.cuh) with capped or distance-biased scores, for bf16
// and fp32 pools (8-bit pools: hwkv_decode_q8.cuh).  A tile's scores change between the two
// products, cap * tanh(s / cap) - slope * distance per score, in registers: no more bytes move.
//
// Bound: HBM, as the plain instances (eight sequences at 32K, 445 MB: cap 50 75.5 us, uncapped 75; fp32, 890
// MB: cap 50, tanhf per score, 165 us, a bias 161, uncapped 155).
// Instances of their own, so that the plain ones keep their registers and their results.
#include "hwkv_decode_sk.cuh"

namespace hwkv {
namespace {

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.elem_bytes == 4)
    return a.group <= 4 ? launch_one<float, D, 4, true>(a, tmap, ctas, st) : cudaErrorInvalidValue;
  switch (decode_tc_group_pad(a.group)) {
    case 4: return launch_one<__nv_bfloat16, D, 4, true>(a, tmap, ctas, st);
    case 8: return launch_one<__nv_bfloat16, D, 8, true>(a, tmap, ctas, st);
    default: return launch_one<__nv_bfloat16, D, 16, true>(a, tmap, ctas, st);
  }
}

}  // namespace

cudaError_t launch_decode_score(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.head_dim == 128) return launch_dim<128>(a, tmap, ctas, st);
  if (a.pv.head_dim == 64) return launch_dim<64>(a, tmap, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace hwkv
