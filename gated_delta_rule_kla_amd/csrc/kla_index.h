// kla_index.h -- index arithmetic of kernels at sizes near 2^31, apart from them so that a test on
// the host runs it too.
#pragma once

#include <hip/hip_runtime.h>

namespace kla {

// f(i) for the positions of [from, to) that thread `thread` of workgroup `block` of `blocks` (256
// threads each) takes: all threads of all workgroups side by side, as often as it takes.  In 64
// bits: the last step of a thread may end past 2^31.
template <class F>
__host__ __device__ __forceinline__ void each_position(int from, int to, int block, int blocks, int thread, F f) {
  for (long long i = from + block * 256LL + thread; i < to; i += blocks * 256LL) f(i);
}

// f(place) for the bits that are set, the lowest first.
template <class F>
__host__ __device__ __forceinline__ void each_bit(unsigned bits, F f) {
  for (; bits; bits &= bits - 1) f(__builtin_ctz(bits));
}

}  // namespace kla
