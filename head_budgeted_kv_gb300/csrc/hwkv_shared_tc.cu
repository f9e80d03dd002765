// The prefixes' keys of a decode behind shared prefixes on the tensor cores (hwkv_shared_tc.cuh), bf16 pools.
#include "hwkv_shared_tc.cuh"

namespace hwkv {

int shared_tc_seqs(int group) { return kM / group; }

cudaError_t launch_shared_tc(const SharedArgs& a, const CUtensorMap* pool_map, const CUtensorMap* stage_map, int ctas, cudaStream_t st) {
  if (a.pv.elem_bytes == 1) return launch_shared_tc_q8(a, pool_map, stage_map, ctas, st);
  cudaError_t e = cudaErrorInvalidValue;
  if (a.pv.head_dim == 128) e = launch<128, false>(a, pool_map, stage_map, ctas, st);
  else if (a.pv.head_dim == 64) e = launch<64, false>(a, pool_map, stage_map, ctas, st);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace hwkv
