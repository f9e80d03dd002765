// The stream-K decode kernel for 8-bit pools (hwkv_decode_q8.cuh): plain and scored instances.
#include "hwkv_decode_q8.cuh"

namespace hwkv {
namespace {

template <int D>
cudaError_t configure_dim(int ctas_per_sm[kGroupPads]) {
  cudaError_t e;
  if ((e = configure_one<D, 4>(&ctas_per_sm[0])) != cudaSuccess) return e;
  if ((e = configure_one<D, 8>(&ctas_per_sm[1])) != cudaSuccess) return e;
  return configure_one<D, 16>(&ctas_per_sm[2]);
}

template <int D, bool SC>
cudaError_t launch_dim(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  switch (decode_tc_group_pad(a.group)) {
    case 4: return launch_one<D, 4, SC>(a, tmap, ctas, st);
    case 8: return launch_one<D, 8, SC>(a, tmap, ctas, st);
    default: return launch_one<D, 16, SC>(a, tmap, ctas, st);
  }
}

}  // namespace

cudaError_t configure_decode_q8(int head_dim, int ctas_per_sm[kGroupPads]) {
  if (head_dim == 128) return configure_dim<128>(ctas_per_sm);
  if (head_dim == 64) return configure_dim<64>(ctas_per_sm);
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_q8(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.head_dim == 128)
    return a.score.on ? launch_dim<128, true>(a, tmap, ctas, st) : launch_dim<128, false>(a, tmap, ctas, st);
  if (a.pv.head_dim == 64)
    return a.score.on ? launch_dim<64, true>(a, tmap, ctas, st) : launch_dim<64, false>(a, tmap, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace hwkv
