// Device code shared by the operators between the GEMVs of a decode step:
// where a token's sequence is found and how a paged cache is addressed.
#pragma once
#include <hip/hip_runtime.h>

#include "decode_index.hpp"

namespace sgemv_dev {

typedef uint32_t dword4 __attribute__((ext_vector_type(4)));

// The last sequence s of [0, count) with f(s) <= x, for f non-decreasing and
// f(0) <= x (0 otherwise): each step the wave's 64 lanes look at 64 places,
// so one round trip finds one of up to 64 sequences and two one of 4096.
template <class F>
__device__ __forceinline__ int wave_upper(int count, int x, F f) {
  const int lane = threadIdx.x & 63;
  Upper u(count);
  while (u.n > 1) u.narrow(__popcll(__ballot(u.in(lane) && f(u.place(lane)) <= x)));
  return __builtin_amdgcn_readfirstlane(u.lo);
}

}  // namespace sgemv_dev
