// The prefixes' keys of a decode behind shared prefixes on the tensor cores (hwkv_shared_tc.cuh), 8-bit pools.
#include "hwkv_shared_tc.cuh"

namespace hwkv {

cudaError_t launch_shared_tc_q8(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas,
                                cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;
  if (a.pv.head_dim == 128) e = launch<128, true>(a, pool_map, stage_map, ctas, st);
  else if (a.pv.head_dim == 64) e = launch<64, true>(a, pool_map, stage_map, ctas, st);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace hwkv
