// Attention of new tokens over a paged cache: device code.
//
// Row (token i, query head hq) of a sequence with keys k_t and values v_t:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m),
// over the visible keys t, in one pass: m follows the running maximum of the
// scores, and what was summed under an older m is scaled down when it
// grows. Scores, m, the sum of the p_t and the output are kept in FP32; p_t is
// rounded to the cache's type for the second product, half a step of its own,
// as the result is once more. In FP16 that step is relative down to 2^-14 only,
// and what is below 2^-25 is gone, which adds up over a long context (131072
// slots under one key 25.1 powers of two above them: 0.0036 of the result), so m
// lies kLift below the maximum there and a row's largest weight is 2^kLift or
// more (a prompt of 8192, 32 heads: 563 us without, 567 with). The sum is that
// of the rounded p_t (a two-way dot product with ones, one operation for two of
// them), so that a weight that outweighs the others is off in both sums alike.
// That operation does not round to nearest (its sums were off by up to 2^-21):
// it adds up a block only.
//
// Both products run on the matrix cores, the first transposed (keys x rows),
// so that a lane holds scores of one row only: the row statistics are a
// reduction over the lane's own registers and one or two lane swaps, and the
// scores become the second product's operand without leaving the lane. That
// operand wants 8 keys in a row from each lane; the lane has runs of 4, so the
// keys of a step are numbered by where they are, and V is read in that order.
#pragma once
#include "decode_device.hpp"

namespace sgemv_dev {

struct AttendParams : TileView {
  int32_t heads;          // cache heads
  const uint16_t *k, *v, *q;
  uint16_t* out;
  int64_t k_head, v_head;
  uint32_t k_page, k_slot, v_page, v_slot;
  int64_t q_token, q_head, o_token, o_head;
  int32_t dim;
  int32_t slots;          // row tiles, empty ones included
  float scale2;           // scale * log2(e): scores in powers of two
  float* part;            // splits > 1: [row][split][dim] sums, then [row][split] of (m, sum of p)
  // a cache in 8 bits: k and v are codes, one byte each, and of every block of
  // 2^exp_shift slots and head there are the exponents (K's in the low byte, V's)
  const uint16_t* exps;   // [page][block][head]
  uint32_t exp_page;      // of them in a page
  int32_t exp_shift;
};
typedef void (*AttendFn)(AttendParams);

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));

template <class T> struct Half;
template <> struct Half<_Float16> {
  static constexpr float kLift = 7.0f;
  static __device__ __forceinline__ f32x4 mma16(dword4 a, dword4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma32(dword4 a, dword4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b}); }
  // c + both halves
  static __device__ __forceinline__ float sum(uint32_t u, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, u), f16x2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
  }
  static __device__ __forceinline__ float lo(uint32_t u) { return (float)__builtin_bit_cast(f16x2, u).x; }
  static __device__ __forceinline__ float hi(uint32_t u) { return (float)__builtin_bit_cast(f16x2, u).y; }
};
template <> struct Half<__bf16> {
  static constexpr float kLift = 0.0f;                  // its exponents are FP32's
  static __device__ __forceinline__ f32x4 mma16(dword4 a, dword4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma32(dword4 a, dword4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return __builtin_bit_cast(uint32_t, b16x2{(__bf16)a, (__bf16)b}); }
  static __device__ __forceinline__ float sum(uint32_t u, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b16x2, u), b16x2{(__bf16)1.0f, (__bf16)1.0f}, c, false);
  }
  static __device__ __forceinline__ float lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
  static __device__ __forceinline__ float hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }
};

// A cache in 8 bits. Keys and values are e4m3 codes times powers of two that a
// block of slots shares: e4m3 has 4 significant bits, so codes are exact in
// either 16-bit type, and the conversion takes a power of two along for nothing.
//   K: the few-row kernel multiplies the scores of a run of 4 keys by their
//   scale, exactly. V, and K in the many-row kernel: converted to multiples of
//   2^E, E the largest exponent that the wave's keys have had so far (what was
//   summed in units of an older E is scaled down when it grows).
// FP16 holds a code below 2^E exactly down to 2^-15 of it, BF16 any that count.
// Where exponents differ by more than kSpread the tile is summed again key by
// key in FP32, so that a row is as exact as its own keys allow whatever other
// rows of its tile see. Exponents up to kTiny do not count for that: FP16
// results below 2^-25 are 0 (values up to 448 2^-35); in BF16 they are those that
// an append gives to zeros. Of K those up to tiny_key() do not.
template <class T> struct Eight;
template <> struct Eight<_Float16> {
  static constexpr int kSpread = 15, kTiny = 127 - 35;
  static __device__ __forceinline__ uint32_t pair(uint32_t codes, float scale, bool high) {
    return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, true))
                : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, false));
  }
};
template <> struct Eight<__bf16> {
  static constexpr int kSpread = 60, kTiny = 127 - 96;
  static __device__ __forceinline__ uint32_t pair(uint32_t codes, float scale, bool high) {
    return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true))
                : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
  }
};
// The largest exponent (biased) of keys that no score can tell from zeros: 256
// products of a query up to 2^16 and a key up to 448 2^e, times scale2 < 2^(s + 1),
// stay below 2^-26 for e <= -60 - s. In BF16 no more than kTiny, which goes down
// with larger scales too (s > 36); 0 always, which keys that are not there have.
template <class T>
__device__ __forceinline__ int tiny_key(float scale2) {
  const int s = (int)(__builtin_bit_cast(uint32_t, scale2) >> 23) - 127, e = 127 - 60 - (s > 0 ? s : 0);
  return e < 0 ? 0 : e < Eight<T>::kTiny ? e : Eight<T>::kTiny;
}
// 8 codes as 8 halves
template <class T>
__device__ __forceinline__ dword4 eight(uint32_t lo, uint32_t hi, float scale) {
  return dword4{Eight<T>::pair(lo, scale, false), Eight<T>::pair(lo, scale, true), Eight<T>::pair(hi, scale, false),
                Eight<T>::pair(hi, scale, true)};
}
// 2^(e - to) for e <= to, which is never 0: under 2^-126 it makes no difference
__device__ __forceinline__ float below(int e, int to) {
  const int d = e - to + 127;
  return __builtin_bit_cast(float, (uint32_t)(d < 1 ? 1 : d) << 23);
}
// The factor of scores whose keys have the exponent e (biased): a normal number,
// so that -inf stays what it is.
__device__ __forceinline__ float score_scale(float scale2, int e) {
  const float x = __builtin_amdgcn_ldexpf(scale2, e - 127);
  return fminf(fmaxf(x, 0x1p-126f), 0x1.fffffep127f);
}

// What lanes read in the place of a key that is not there, as wide as a row:
// V's rows have to be zeros even where their weight is 0 (0 * NaN), K's may be
// anything.
static __device__ const dword4 kNothing[32] = {};

// Addresses as whole numbers, so that choosing between a key and nothing is a
// select and not a branch around a load, and loads know that they are global.
typedef uint64_t addr_t;
__device__ __forceinline__ addr_t addr(const void* p) { return (addr_t)p; }
// `a` where it is there. What `a` is computed from is hidden, or the compiler
// would branch around the arithmetic instead of selecting.
__device__ __forceinline__ addr_t or_nothing(bool there, addr_t a) {
  asm("" : "+v"(a));
  return there ? a : addr(kNothing);
}
template <class V>
__device__ __forceinline__ V load(addr_t a) { return *(const __attribute__((address_space(1))) V*)a; }

// Element `slot` rows into page `page` of a cache whose strides fit 32 bits.
__device__ __forceinline__ uint64_t element(int page, uint32_t page_stride, int slot, uint32_t slot_stride) {
  return (uint64_t)(uint32_t)page * page_stride + (uint64_t)(uint32_t)slot * slot_stride;
}

// m is raised only when a block's largest score, less kLift, passes it by more
// than this (in powers of two): the sums are then scaled down, a pass over the
// whole output, for a few blocks instead of most. Weights reach 2^8 at most, in
// FP16 2^15, as exact in either type as those around 1; those that FP16 rounds
// to 0 are under 2^-32 of the largest.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// max and sum with the lane 16 or 32 places away
struct Two { float a, b; };
__device__ __forceinline__ Two both_x32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = r[0], b = r[1];
  return Two{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Two both_x16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a = r[0], b = r[1];
  return Two{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float max_x32(float x) { const Two t = both_x32(x); return fmaxf(t.a, t.b); }
__device__ __forceinline__ float max_x16(float x) { const Two t = both_x16(x); return fmaxf(t.a, t.b); }
__device__ __forceinline__ float sum_x32(float x) { const Two t = both_x32(x); return t.a + t.b; }
__device__ __forceinline__ float sum_x16(float x) { const Two t = both_x16(x); return t.a + t.b; }
// the largest of a small whole number over the wave's groups of 16 lanes
__device__ __forceinline__ int top_of_groups(int x) {
  const float f = __builtin_bit_cast(float, x + 0x3f800000);   // as a float of the same order
  return __builtin_bit_cast(int, max_x32(max_x16(f))) - 0x3f800000;
}

// The tile of a workgroup. Up to 64 sequences: every lane reads one's lengths,
// so that one round trip to memory gives all there is to know.
template <int M, bool WINDOW = false>
__device__ __forceinline__ bool find_tile(const TileView& p, int block, int slot, int split, Tile& t) {
  const int count = p.seq.count;
  if (count <= 64) {
    const int lane = threadIdx.x & 63, i = lane < count ? lane : count - 1;
    const int first = p.seq.start(i), next = p.seq.start(i + 1), ctx = p.seq.ctx(i);
    const int holds = __popcll(__ballot(lane < count && slot_base(p, i, first, M) <= slot));
    const int s = holds < 1 ? 0 : holds - 1;
    return make_tile<WINDOW>(p, M, block, s, __builtin_amdgcn_readlane(first, s), __builtin_amdgcn_readlane(next, s),
                     __builtin_amdgcn_readlane(ctx, s), slot, split, t);
  }
  const int s = wave_upper(count, slot, [&](int i) { return slot_base(p, i, p.seq.start(i), M); });
  return make_tile<WINDOW>(p, M, block, s, p.seq.start(s), p.seq.start(s + 1), p.seq.ctx(s), slot, split, t);
}

__device__ __forceinline__ bool not_finite(float x) { return !(__builtin_fabsf(x) < __builtin_inff()); }

// Where a row's part of the sums goes when the context is split.
__device__ __forceinline__ float* part_sums(const AttendParams& p, int64_t row, int split) {
  return p.part + (row * p.splits + split) * p.dim;
}
__device__ __forceinline__ float* part_stats(const AttendParams& p, int64_t row, int split) {
  return p.part + (int64_t)p.seq.tokens * p.heads * p.group * p.splits * p.dim + (row * p.splits + split) * 2;
}

}  // namespace sgemv_dev
