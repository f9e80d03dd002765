// The stream-K decode kernel (hwkv_decode_sk.cuh) with open results, for bf16 and fp32 pools (8-bit pools:
// hwkv_decode_open_q8.cu): the sequences' own part of a decode behind shared prefixes.  The scored form serves plain
// scores too (with instances for those, a call behind a 32K document takes 45.0 us, not 45.3, behind several prefixes 36.4, not 36.8, others
// the same).  Only the grid's last CTA waits for the prefixes' kernel, which so has ended when the
// join starts; had each CTA waited, those done would have held their SMs.
#include "hwkv_decode_sk.cuh"

namespace hwkv {
namespace {

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.elem_bytes == 4)
    return a.group <= 4 ? launch_one<float, D, 4, true, true>(a, tmap, ctas, st) : cudaErrorInvalidValue;
  switch (decode_tc_group_pad(a.group)) {
    case 4: return launch_one<__nv_bfloat16, D, 4, true, true>(a, tmap, ctas, st);
    case 8: return launch_one<__nv_bfloat16, D, 8, true, true>(a, tmap, ctas, st);
    default: return launch_one<__nv_bfloat16, D, 16, true, true>(a, tmap, ctas, st);
  }
}

}  // namespace

cudaError_t launch_decode_open(const DecodeArgs& a, const CUtensorMap* tmap, int ctas, cudaStream_t st) {
  if (a.pv.elem_bytes == 1) return launch_decode_open_q8(a, tmap, ctas, st);
  if (a.pv.head_dim == 128) return launch_dim<128>(a, tmap, ctas, st);
  if (a.pv.head_dim == 64) return launch_dim<64>(a, tmap, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace hwkv
