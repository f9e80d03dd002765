// What the kernels of a decode behind shared prefixes have in common: the sequences of a prefix, lengths, and
// the age of a ring slot.
#pragma once

#include "hwkv_device.cuh"

namespace hwkv {
namespace {

// Prefix of sequence s, or -1.  One that the pool does not hold counts as none (`flag`: it is recorded).
__device__ __forceinline__ int prefix_of(const SharedArgs& a, int s, bool flag) {
  const int f = a.prefix_of[s];
  if (f >= a.num_prefixes && flag) atomicOr(a.pv.err, HWKV_DEVERR_BAD_PREFIX);
  return f < 0 || f >= a.num_prefixes ? -1 : f;
}

// length of a prefix (the caller flags one below 0)
__device__ __forceinline__ int prefix_len(const SharedArgs& a, int f) { return max(0, a.prefix_lens[f]); }

// own length of sequence s after the append
__device__ __forceinline__ int shared_len(const SharedArgs& a, int s) { return max(0, a.lens[s] + a.len_add); }

// Distance of ring slot t's newest position from the last of N tokens, below C (the slot holds none when it is N or
// more).
__device__ __forceinline__ int ring_age(int N, int t, int C) {
  const int last = N > 0 ? (N - 1) % C : C - 1;
  const int d = last - t;
  return d < 0 ? d + C : d;
}

// The sequences behind prefix f, in order: those from the first'th, at most `most`, to seq[]; their number.  By one warp.
__device__ __forceinline__ int shared_members(const SharedArgs& a, int f, int first, int most, int* seq, int lane) {
  int seen = 0;
  for (int s0 = 0; s0 < a.num_seqs && seen < first + most; s0 += 32) {
    const int s = s0 + lane;
    const bool mine = s < a.num_seqs && a.prefix_of[s] == f;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    const int at = seen + __popc(all & ((1u << lane) - 1u)) - first;
    if (mine && at >= 0 && at < most) seq[at] = s;
    seen += __popc(all);
  }
  __syncwarp();
  return max(0, min(most, seen - first));
}

}  // namespace
}  // namespace hwkv
