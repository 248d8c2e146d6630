// Device code shared by the operators between the GEMVs of a decode step:
// where a token's sequence is found and how a paged cache is addressed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgemv_dev {

typedef uint32_t dword4 __attribute__((ext_vector_type(4)));

// Sequences as the kernels see them (sgemv_seqs). Lengths live in device
// memory, where no host check reaches them, so every one is clamped before
// it is used: a bad one gives wrong numbers, never an access out of range.
struct SeqView {
  const int32_t* new_start;   // [count + 1] first new token of each sequence
  const int32_t* ctx_len;     // [count] tokens of each sequence, new ones included
  const int32_t* pages;       // [count][pages_per_seq]
  int64_t pages_stride;
  int32_t count, pages_per_seq, page_shift, n_pages, tokens;

  __device__ __forceinline__ int start(int s) const {
    const int v = new_start[s];
    return v < 0 ? 0 : v > tokens ? tokens : v;
  }
  // tokens of sequence s: no more than its row of the page table holds
  __device__ __forceinline__ int ctx(int s) const {
    const int64_t cap = (int64_t)pages_per_seq << page_shift;
    const int v = ctx_len[s];
    return v < 0 ? 0 : v > cap ? (int)cap : v;
  }
  __device__ __forceinline__ bool page_ok(int page) const { return (uint32_t)page < (uint32_t)n_pages; }
};

// The last sequence s of [0, count) with f(s) <= x, for f non-decreasing and
// f(0) <= x (0 otherwise): each step the wave's 64 lanes look at 64 places,
// so one round trip finds one of up to 64 sequences and two one of 4096.
template <class F>
__device__ __forceinline__ int wave_upper(int count, int64_t x, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = count;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lane * step;
    const bool in = at < n && f(lo + (at < n ? at : 0)) <= x;
    int below = __popcll(__ballot(in));
    below = below < 1 ? 1 : below;
    lo += (below - 1) * step;
    n = n - (below - 1) * step;
    n = n < step ? n : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace sgemv_dev
