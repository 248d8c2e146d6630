// Joins the parts of a split context.
#pragma once
#include "attend_device.hpp"

namespace sgemv_dev {

constexpr int kMaxSplits = 256, kJoinLanes = 256;

// How many parts the context of a row (token, query head) has; 0 for a row of
// no sequence. Lanes of a wave may have rows of different tokens.
template <bool WINDOW>
__device__ __forceinline__ int parts_of(const AttendParams& p, int64_t at, int tile_rows, int block) {
  const int all = p.heads * p.group, tok = (int)(at / all), hq = (int)(at % all);
  int lo = 0, n = p.seq.count;
  while (n > 1) {
    const int half = n / 2;
    const bool up = p.seq.start(lo + half) <= tok;
    lo = up ? lo + half : lo;
    n = up ? n - half : half;
  }
  Tile t;
  const int next = p.seq.start(lo + 1), ctx = p.seq.ctx(lo);
  t.s = lo;
  t.first = p.seq.start(lo);
  t.n = next - t.first;
  if (tok < t.first || tok >= next) return 0;
  t.rows = t.n * p.group;
  t.row0 = ((tok - t.first) * p.group + hq % p.group) / tile_rows * tile_rows;
  tile_keys<WINDOW>(p, tile_rows, block, ctx, 0, t);
  // key1 of split 0 is the length of a part (or all there is); a tile without
  // a key has no part, and its rows are zeros
  return t.key1 > 0 ? (t.keys + t.key1 - 1) / t.key1 : -1;
}
template <class T>
__device__ __forceinline__ void store_row(const AttendParams& p, int64_t at, int d, f32x4 x) {
  const int all = p.heads * p.group, tok = (int)(at / all), hq = (int)(at % all);
  *(dword2*)(p.out + tok * p.o_token + hq * p.o_head + d) = dword2{Half<T>::pack(x[0], x[1]), Half<T>::pack(x[2], x[3])};
}

// One workgroup a row. Groups of DP/4 lanes take the parts in turn, 4 columns a
// lane, and meet in LDS. Which part is added where is fixed by their number, so
// the result does not depend on the order in which they were computed.
// Bound by round trips: a row's first parts and all statistics are read before
// it is known how many there are (the workspace has room for `splits` of every
// row; what no part wrote is read and not used).
template <class T, int DP, bool WINDOW>
__global__ void __launch_bounds__(kJoinLanes) attend_join_kernel(AttendParams p, int tile_rows, int block) {
  constexpr int PER = DP / 4, GROUPS = kJoinLanes / PER, AHEAD = 4, STATS = (kMaxSplits + 63) / 64;
  __shared__ float weight[kMaxSplits];
  __shared__ __attribute__((aligned(16))) float sums[GROUPS][DP];
  __shared__ float total;
  const int64_t at = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int group = tid / PER, d = tid % PER * 4;
  const float* from = part_sums(p, at, 0) + (d < p.dim ? d : 0);
  f32x4 first[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = group + k * GROUPS;
    first[k] = *(const f32x4*)(from + (int64_t)(i < p.splits ? i : 0) * p.dim);
  }
  float m[STATS], l[STATS];
#pragma unroll
  for (int k = 0; k < STATS; ++k) {
    const int i = lane + 64 * k;
    const float* st = part_stats(p, at, i < p.splits ? i : 0);
    m[k] = st[0];
    l[k] = st[1];
  }
  const int parts = parts_of<WINDOW>(p, at, tile_rows, block);
  if (parts == 0) return;

  if (tid < 64) {
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int k = 0; k < STATS; ++k) {
      const bool there = lane + 64 * k < parts;
      m[k] = there ? m[k] : -__builtin_inff();
      l[k] = there ? l[k] : 0.0f;
      top = fmaxf(top, m[k]);
    }
    top = max_x32(max_x16(top));
#pragma unroll
    for (int x = 1; x < 16; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
#pragma unroll
    for (int k = 0; k < STATS; ++k) {
      const float by = m[k] == top ? 1.0f : exp2_fast(m[k] - top);
      weight[lane + 64 * k] = by;
      sum += by * l[k];
    }
    sum = sum_x32(sum_x16(sum));
#pragma unroll
    for (int x = 1; x < 16; x *= 2) sum += __shfl_xor(sum, x);
    if (lane == 0) total = sum;
  }
  __syncthreads();
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = group + k * GROUPS;
    if (i < parts) x += weight[i] * first[k];
  }
#pragma unroll 4
  for (int i = group + AHEAD * GROUPS; i < parts; i += GROUPS) x += weight[i] * *(const f32x4*)(from + (int64_t)i * p.dim);
  *(f32x4*)&sums[group][d] = x;
  __syncthreads();
  if (group == 0 && d < p.dim) {
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) x += *(const f32x4*)&sums[g][d];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    store_row<T>(p, at, d, x * inv);
  }
}

// Many rows with few parts each: DP/4 lanes a row, which read its statistics
// and its parts all at once, eight parts at a time.
template <class T, int DP, bool WINDOW>
__global__ void __launch_bounds__(kJoinLanes) attend_join_rows_kernel(AttendParams p, int tile_rows, int block) {
  constexpr int PER = DP / 4, ROWS = kJoinLanes / PER, AHEAD = 8;
  const int64_t rows = (int64_t)p.seq.tokens * p.heads * p.group, at = (int64_t)blockIdx.x * ROWS + threadIdx.x / PER;
  const int64_t mine = at < rows ? at : rows - 1;
  const int d = threadIdx.x % PER * 4;
  const float* from = part_sums(p, mine, 0) + (d < p.dim ? d : 0);
  const float* st = part_stats(p, mine, 0);
  float top = -__builtin_inff(), l = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  int parts = 0;
  for (int i0 = 0; i0 < p.splits; i0 += AHEAD) {
    float m[AHEAD], s[AHEAD];
    f32x4 v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k < p.splits ? i0 + k : 0;
      m[k] = st[2 * i];
      s[k] = st[2 * i + 1];
      v[k] = *(const f32x4*)(from + (int64_t)i * p.dim);
    }
    if (i0 == 0) parts = parts_of<WINDOW>(p, mine, tile_rows, block);
    float to = top;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) to = i0 + k < parts ? fmaxf(to, m[k]) : to;
    const float keep = top == to ? 1.0f : exp2_fast(top - to);
    l *= keep;
    x *= keep;
    top = to;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i0 + k < parts) {
        const float by = m[k] == top ? 1.0f : exp2_fast(m[k] - top);
        l += by * s[k];
        x += by * v[k];
      }
  }
  if (parts == 0 || at >= rows || d >= p.dim) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store_row<T>(p, at, d, x * inv);
}

}  // namespace sgemv_dev
