// The stream-K decode kernel for 8-bit pools (hwkv_decode_q8.cuh) with open results (see hwkv_decode_open.cu).
#include "hwkv_decode_q8.cuh"

namespace hwkv {
namespace {

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  switch (decode_tc_group_pad(a.group)) {
    case 4: return launch_one<D, 4, true, true>(a, tmap, ctas, st);
    case 8: return launch_one<D, 8, true, true>(a, tmap, ctas, st);
    default: return launch_one<D, 16, true, true>(a, tmap, ctas, st);
  }
}

}  // namespace

cudaError_t launch_decode_open_q8(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.head_dim == 128) return launch_dim<128>(a, tmap, ctas, st);
  if (a.pv.head_dim == 64) return launch_dim<64>(a, tmap, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace hwkv
