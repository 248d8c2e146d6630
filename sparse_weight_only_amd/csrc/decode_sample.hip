// The choice of a token for each row of logits.
//
// With M a row's largest logit and p_v = exp((x_v - M) / T), the row keeps
//   the tokens of p_v >= min_p, of those the top_k largest, of those the fewest
//   largest whose sum reaches top_p of theirs
// (of equal logits the lower id counts as larger): all three take a first part of
// the order by value, so what is kept is given by its last token, the border:
// every token above its logit, and of its logit the first few. The token is
// then the first one, by id, up to which the kept p sum to more than u times
// their sum.
//
// A chosen token is a whole number, and 2^-24 off in a sum picks another one in
// one of some thousand rows. So exponents and exponentials are in 64 bits (a
// polynomial of degree 9 on half a power of two to each side, within 2^-45),
// and p is rounded to whole multiples of 2^-43, whose sums are exact and do not
// depend on their order.
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;

namespace {

constexpr int kLanes = 1024, kWaves = kLanes / 64;
constexpr int kUnit = 43;                            // p in units of 2^-43: 2^20 of them fit 64 bits
constexpr int kMostVocab = 1 << 20;
constexpr int kBins = 2048;                          // of a step of a search
constexpr int kMassBins = 512, kBinsPerPower = 16;   // of a wave's masses by value: 16 to a power of two
constexpr int kList = 8192;                          // tokens that are looked at one by one
constexpr int kMostK = 768;                          // see candidates()

struct SampleParams {
  const void* x;
  int64_t stride;
  const float *uniform, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* ids;
  float* logprob;
  int32_t vocab;
};

// Whole numbers in the order of the floats; both zeros the same, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  x = x != x ? -__builtin_inff() : x + 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kNever = 0x007fffffu;             // the key of -inf

// A token's place in its row's order by value, the largest first: of equal
// logits the lower id.
__device__ __forceinline__ uint64_t place_of(uint32_t key, uint32_t id) { return (uint64_t)key << 32 | (uint32_t)~id; }

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int from) {
  const uint32_t lo = __shfl((uint32_t)x, from), hi = __shfl((uint32_t)(x >> 32), from);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_prefix(uint64_t x) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t y = shfl64(x, lane - d);
    if (lane >= d) x += y;
  }
  return x;
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t x) {
#pragma unroll
  for (int d = 32; d; d /= 2) x += shfl64(x, (threadIdx.x & 63) ^ d);
  return x;
}

struct Shared {
  union {
    unsigned long long wave_mass[kWaves][kMassBins];
    struct {
      unsigned long long mass[kBins];
      uint32_t count[kBins];
    };
  };
  uint64_t list[kList];                              // places
  unsigned long long stretch[kWaves];                // sums of the kept p, by waves' stretches of the row
  uint64_t part[kWaves];
  uint32_t best[kWaves];
  uint64_t above, place;
  uint32_t bin_count;
  int bin, listed;
};

// The largest of a number over the workgroup.
__device__ __forceinline__ uint32_t block_max(Shared& s, uint32_t v) {
#pragma unroll
  for (int d = 32; d; d /= 2) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.best[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s.best[threadIdx.x & (kWaves - 1)];
#pragma unroll
  for (int d = kWaves / 2; d; d /= 2) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Exclusive prefix over the workgroup, and the sum in `all`.
__device__ __forceinline__ uint64_t block_prefix(Shared& s, uint64_t v, uint64_t& all) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint64_t inc = wave_prefix(v);
  __syncthreads();
  if (lane == 63) s.part[wave] = inc;
  __syncthreads();
  uint64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint64_t q = s.part[w];
    before += w < wave ? q : 0;
    total += q;
  }
  all = total;
  return before + inc - v;
}

// A row and what its weights follow from.
template <class T>
struct Row {
  static constexpr int PER = 16 / sizeof(T);         // logits of a lane and load
  typedef T Some __attribute__((ext_vector_type(PER), aligned(sizeof(T))));   // rows of any vocabulary: element alignment only
  const T* x;
  int vocab;
  float top;                                         // M
  float least;                                       // the smallest logit that min_p (or being a number) leaves
  double base, scale;                                // M and log2(e) / T
  double floor;                                      // of exponents: where M is infinite the others' do not count, and its own are 0

  // 2^((x - M) scale) in units of 2^-43, rounded; for x from `least` on.
  __device__ __forceinline__ uint64_t weight(float v) const {
    // no number (infinities less each other) becomes the floor
    const double z = __builtin_fmax(((double)v - base) * scale, floor);
    // the nearest whole number, in the low bits too
    const double big = z + 0x1.8p52, n = big - 0x1.8p52, f = z - n;
    double y = 0x1.b69b333333333p+19;                // 2^43 2^f
    y = fma(y, f, 0x1.63f1a66666666p+23);
    y = fma(y, f, 0x1.ffcb2e3333335p+26);
    y = fma(y, f, 0x1.43088c34ccccbp+30);
    y = fma(y, f, 0x1.5d87fea9ba666p+33);
    y = fma(y, f, 0x1.3b2ab72c33333p+36);
    y = fma(y, f, 0x1.c6b08d70374acp+38);
    y = fma(y, f, 0x1.ebfbdff813d86p+40);
    y = fma(y, f, 0x1.62e42fefa3a31p+42);
    y = fma(y, f, 0x1.000000000003fp+43);
    // times 2^n (n >= -1000: no subnormals)
    const uint64_t bits = __builtin_bit_cast(uint64_t, y) + ((uint64_t)__builtin_bit_cast(uint64_t, big) << 52);
    // 2^52 on top leaves the number in the low bits, rounded to a whole one
    return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, bits) + 0x1p52) & 0xfffffffffffffull;
  }
  // f(logit, id) for the ids of [a, b) by the lanes `lane` of n, and for a few
  // that are not there, as logits that are no numbers. AHEAD loads at a time:
  // as many as registers allow.
  template <int AHEAD, class F>
  __device__ __forceinline__ void each(int a, int b, int lane, int n, F f) const {
    for (int i = a + lane * PER; i < b; i += n * PER * AHEAD) {
      Some w[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int at = i + k * n * PER;
        if (at + PER <= b) {
          w[k] = *(const Some*)(x + at);
        } else {
#pragma unroll
          for (int e = 0; e < PER; ++e) w[k][e] = at + e < b ? x[at + e] : (T)__builtin_nanf("");
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
#pragma unroll
        for (int e = 0; e < PER; ++e) f((float)w[k][e], i + k * n * PER + e);
    }
  }
};

// Where the tokens that a search goes through come from: the row itself, or
// what has been listed of it. f(place, logit) for each.
template <class T>
struct FromRow {
  const Row<T>& row;
  template <class F>
  __device__ __forceinline__ void operator()(F f) const {
    row.template each<1>(0, row.vocab, threadIdx.x, kLanes, [&](float v, int id) {
      if (v >= row.least) f(place_of(key_of(v), id), v);
    });
  }
};
struct FromList {
  const Shared& s;
  int n;
  template <class F>
  __device__ __forceinline__ void operator()(F f) const {
    for (int i = threadIdx.x; i < n; i += kLanes) {
      const uint64_t p = s.list[i];
      f(p, of_key((uint32_t)(p >> 32)));
    }
  }
};

// The border among a source's places in [lo, hi], of which there is one at least:
// the last one in order such that those up to it, counted (MASS: weighed), reach
// `goal`, which all together do. A histogram of kBins intervals at a time.
template <bool MASS, class T, class S>
__device__ uint64_t find_border(Shared& s, const Row<T>& row, const S& source, uint64_t lo, uint64_t hi, uint64_t goal) {
  while (true) {
    const uint64_t span = hi - lo;
    const int bits = span ? 64 - __clzll((long long)span) : 0, shift = bits > 11 ? bits - 11 : 0;
    for (int i = threadIdx.x; i < kBins; i += kLanes) {
      if (MASS) s.mass[i] = 0;
      s.count[i] = 0;
    }
    __syncthreads();
    source([&](uint64_t p, float v) {
      if (p < lo || p > hi) return;
      const uint32_t bin = (uint32_t)((hi - p) >> shift);
      if (MASS) atomicAdd(&s.mass[bin], (unsigned long long)row.weight(v));
      atomicAdd(&s.count[bin], 1u);
    });
    __syncthreads();
    const int i0 = threadIdx.x * 2;
    const uint64_t a = MASS ? s.mass[i0] : s.count[i0], b = MASS ? s.mass[i0 + 1] : s.count[i0 + 1];
    uint64_t all;
    const uint64_t before = block_prefix(s, a + b, all);
    if (before < goal && before + a + b >= goal) {
      const int second = before + a < goal;
      s.bin = i0 + second;
      s.above = before + (second ? a : 0);
      s.bin_count = s.count[i0 + second];
    }
    __syncthreads();
    goal -= s.above;
    const uint64_t from = hi - ((uint64_t)s.bin << shift), rest = ((uint64_t)1 << shift) - 1;
    lo = from - lo > rest ? from - rest : lo;
    hi = from;
    const bool one = s.bin_count == 1;
    __syncthreads();
    if (lo == hi) return hi;
    if (one) {
      source([&](uint64_t p, float) {
        if (p >= lo && p <= hi) s.place = p;
      });
      __syncthreads();
      return s.place;
    }
  }
}

// goal of a sum: the least whole number that is `share` of `sum` or more, 1 at least
__device__ __forceinline__ uint64_t goal_of(float share, uint64_t sum) {
  const double want = (double)sum * (double)share;
  uint64_t goal = want > 0.0 ? (uint64_t)want : 0;
  goal += (double)goal < want;
  return goal < 1 ? 1 : goal > sum ? sum : goal;
}

template <class S>
__device__ __forceinline__ uint64_t count_of(Shared& s, const S& source) {
  uint64_t n = 0, all;
  source([&](uint64_t, float) { ++n; });
  block_prefix(s, n, all);
  return all;
}
template <class T, class S>
__device__ __forceinline__ uint64_t mass_from(Shared& s, const Row<T>& row, const S& source, uint64_t border) {
  uint64_t n = 0, all;
  source([&](uint64_t p, float v) { n += p >= border ? row.weight(v) : 0; });
  block_prefix(s, n, all);
  return all;
}

// One workgroup a row. Three ways to the border:
//  * top_k up to kMostK: at least k tokens are as large as the k-th largest of the
//    lanes' own largest logits, and hardly more; those are listed, and the rest
//    of the work is on the list;
//  * top_p: each wave sums the p of its stretch of the row by value, in bins of
//    1/16 power of two; the tokens of the bin that the border falls into are
//    listed;
//  * anything else (larger k, more tokens than the list takes): searches over the row.
// The token is then looked for in the stretch of the row, a sixteenth of it, that
// the sums of the kept p point at.
template <class T>
__global__ void __launch_bounds__(kLanes) sample_kernel(SampleParams p) {
  __shared__ Shared s;
  const int r = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  Row<T> row;
  row.x = (const T*)p.x + r * p.stride;
  row.vocab = p.vocab;
  const float t = p.temperature ? p.temperature[r] : 1.0f, u = p.uniform[r];
  const int k = p.top_k ? p.top_k[r] : 0;
  const float top_p = p.top_p ? p.top_p[r] : 1.0f, min_p = p.min_p ? p.min_p[r] : 0.0f;
  constexpr int PER = Row<T>::PER, W = 1;
  // a wave's stretch of the row, in whole steps of the wave
  const int stretch = (row.vocab + kWaves * 64 * PER - 1) / (kWaves * 64 * PER) * (64 * PER);
  const int from = wave * stretch < row.vocab ? wave * stretch : row.vocab, to = from + stretch < row.vocab ? from + stretch : row.vocab;

  float most = -__builtin_inff();
  row.template each<4>(from, to, lane, 64, [&](float v, int) { most = fmaxf(most, v); });
  const uint32_t mine = key_of(most), top_key = block_max(s, mine);
  if (top_key <= kNever) {
    if (tid == 0) {
      p.ids[r] = -1;
      if (p.logprob) p.logprob[r] = -__builtin_inff();
    }
    return;
  }
  row.top = of_key(top_key);
  if (!(t > 0.0f)) {
    uint32_t first = 0;                                // the lowest id, as the largest of its complements
    if (mine == top_key)
      row.template each<4 / (PER / 4)>(from, to, lane, 64, [&](float v, int id) {
        if (v == row.top && ~(uint32_t)id > first) first = ~(uint32_t)id;
      });
    first = ~block_max(s, first);
    if (tid == 0) {
      p.ids[r] = (int32_t)first;
      if (p.logprob) p.logprob[r] = 0.0f;
    }
    return;
  }
  const bool infinite = !(row.top < __builtin_inff());
  row.base = (double)row.top;
  row.scale = 1.4426950408889634074 / (double)t;
  row.floor = infinite ? 0.0 : -1000.0;
  row.least = infinite ? row.top : -0x1.fffffep127f;
  if (min_p > 0.0f && !infinite) {
    // the smallest logit of exponent log2(min_p) or more
    const double least = min_p < 1.0f ? log2((double)min_p) : 0.0;
    uint32_t key = kNever + 1, enough = top_key;
    while (key < enough) {
      const uint32_t mid = key + (enough - key) / 2;
      if (((double)of_key(mid) - row.base) * row.scale >= least) enough = mid;
      else key = mid + 1;
    }
    row.least = of_key(key);
  }
  const uint64_t lowest = place_of(key_of(row.least), ~0u), highest = place_of(top_key, 0);

  uint64_t border = lowest;                            // tokens from it on, in order, are kept
  bool summed = false;                                 // s.stretch holds the sums of what is kept
  const FromRow<T> whole{row};
  const auto search_row = [&] {
    // on the row itself
    if (k > 0 && count_of(s, whole) > (uint64_t)k) border = find_border<false>(s, row, whole, lowest, highest, k);
    if (top_p < 1.0f)
      border = find_border<true>(s, row, whole, border, highest, goal_of(top_p, mass_from(s, row, whole, border)));
  };
  // adds the kept tokens of the list to their stretches
  const auto sum_list = [&](int n) {
    for (int i = tid; i < n; i += kLanes) {
      const uint64_t q = s.list[i];
      if (q >= border) atomicAdd(&s.stretch[~(uint32_t)q / (uint32_t)stretch], (unsigned long long)row.weight(of_key((uint32_t)(q >> 32))));
    }
  };
  if (tid < kWaves) s.stretch[tid] = 0;
  if (tid == 0) s.listed = 0;
  if (k > 0 && k <= kMostK) {
    // a bound that at least k lanes' largest reach: the lower end of the bin of
    // the k-th largest, of kLanes bins between the smallest and the largest of them
    const uint32_t floor_key = key_of(row.least);
    uint32_t bound = floor_key;
    {
      const uint32_t low = ~block_max(s, ~mine);
      const float lo = fmaxf(of_key(low), -0x1.fffffep127f), by = (float)kLanes / (row.top - lo);
      s.count[tid] = 0;
      __syncthreads();
      const auto bin_of = [&](float v) {
        return (int)fminf(fmaxf((row.top - v) * by, 0.0f), kLanes - 1.0f);   // no number (0 by infinity): 0
      };
      const int b = bin_of(most);
      if (mine >= floor_key) atomicAdd(&s.count[b], 1u);
      __syncthreads();
      uint64_t all;
      const uint64_t c = s.count[tid], before = block_prefix(s, c, all);
      if (before < (uint64_t)k && before + c >= (uint64_t)k) s.bin = tid;
      if (all >= (uint64_t)k) {
        // the smallest of the bin's own
        __syncthreads();
        const int last = s.bin;
        bound = ~block_max(s, mine >= floor_key && b <= last ? ~mine : 0);
      }
    }
    __syncthreads();
    row.template each<4 / (PER / 4)>(from, to, lane, 64, [&](float v, int id) {
      if (!(v >= row.least)) return;
      const uint32_t key = key_of(v);
      if (key < bound) return;
      const int at = atomicAdd(&s.listed, 1);
      if (at < kList) s.list[at] = place_of(key, id);
    });
    __syncthreads();
    const int n = s.listed;
    if (n <= kList) {
      const FromList listed{s, n};
      const uint64_t bottom = place_of(bound, ~0u);
      border = bottom;
      if (n > k) border = find_border<false>(s, row, listed, bottom, highest, k);
      if (top_p < 1.0f)
        border = find_border<true>(s, row, listed, border, highest, goal_of(top_p, mass_from(s, row, listed, border)));
      sum_list(n);
      summed = true;
    } else {
      search_row();
    }
  } else if (k <= 0 && top_p < 1.0f) {
    const float by = fminf(kBinsPerPower * (float)row.scale, 1e30f);
    const auto bin_of = [&](float v) {
      return (int)fminf(fmaxf((row.top - v) * by, 0.0f), kMassBins - 1.0f);  // no number (of infinite logits): 0
    };
    for (int i = lane; i < kMassBins; i += 64) s.wave_mass[wave][i] = 0;
    row.template each<W>(from, to, lane, 64, [&](float v, int) {
      if (v >= row.least) atomicAdd(&s.wave_mass[wave][bin_of(v)], (unsigned long long)row.weight(v));
    });
    __syncthreads();
    uint64_t in_bin = 0, all;
    if (tid < kMassBins)
#pragma unroll
      for (int w = 0; w < kWaves; ++w) in_bin += s.wave_mass[w][tid];
    const uint64_t before = block_prefix(s, in_bin, all), goal = goal_of(top_p, all);
    if (before < goal && before + in_bin >= goal) {
      s.bin = tid;
      s.above = before;
    }
    __syncthreads();
    const int last = s.bin;
    const uint64_t rest = goal - s.above;
    uint64_t larger = 0;
    for (int i = lane; i < last; i += 64) larger += s.wave_mass[wave][i];
    larger = wave_sum(larger);
    row.template each<4 / (PER / 4)>(from, to, lane, 64, [&](float v, int id) {
      if (!(v >= row.least) || bin_of(v) != last) return;
      const int at = atomicAdd(&s.listed, 1);
      if (at < kList) s.list[at] = place_of(key_of(v), id);
    });
    __syncthreads();
    const int n = s.listed;
    if (n <= kList) {
      if (lane == 0) s.stretch[wave] = larger;
      uint32_t hi = 0, lo = 0;                         // the list's largest key, and its smallest's complement
      for (int i = tid; i < n; i += kLanes) {
        const uint32_t key = (uint32_t)(s.list[i] >> 32);
        hi = key > hi ? key : hi;
        lo = ~key > lo ? ~key : lo;
      }
      hi = block_max(s, hi);
      lo = ~block_max(s, lo);
      border = find_border<true>(s, row, FromList{s, n}, place_of(lo, ~0u), place_of(hi, 0), rest);
      sum_list(n);
      summed = true;
    } else {
      search_row();
    }
  } else if (k > 0 || top_p < 1.0f) {
    search_row();
  }

  const auto kept = [&](float v, int id) { return v >= row.least && place_of(key_of(v), id) >= border; };
  if (!summed) {
    uint64_t sum = 0;
    row.template each<W>(from, to, lane, 64, [&](float v, int id) { sum += kept(v, id) ? row.weight(v) : 0; });
    sum = wave_sum(sum);
    if (lane == 0) s.stretch[wave] = sum;
  }
  __syncthreads();
  // the stretch of the token, by every wave for itself
  uint64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all += s.stretch[w];
  const double at = (double)(u > 0.0f ? u : 0.0f) * (double)all;
  uint64_t goal = at < (double)all ? (uint64_t)at : all - 1;
  goal = goal < all ? goal : all - 1;
  uint64_t run = 0;
  int chosen = 0;
  while (run + s.stretch[chosen] <= goal) run += s.stretch[chosen++];
  // and in it, again by waves and then step by step of the one
  const int a = chosen * stretch, piece = (stretch / (64 * PER) + kWaves - 1) / kWaves * (64 * PER);
  const int end = a + stretch < row.vocab ? a + stretch : row.vocab;
  const int pa = a + wave * piece < end ? a + wave * piece : end, pb = pa + piece < end ? pa + piece : end;
  uint64_t sum = 0;
  row.template each<1>(pa, pb, lane, 64, [&](float v, int id) { sum += kept(v, id) ? row.weight(v) : 0; });
  sum = wave_sum(sum);
  if (lane == 0) s.part[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) run += s.part[w];
  if (goal < run || goal >= run + sum) return;
  for (int i = pa; i < pb; i += 64 * PER) {
    uint64_t w[PER], of_lane = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int id = i + lane * PER + e;
      const float v = id < pb ? (float)row.x[id] : __builtin_nanf("");
      w[e] = kept(v, id) ? row.weight(v) : 0;
      of_lane += w[e];
    }
    const uint64_t inc = wave_prefix(of_lane), step = shfl64(inc, 63);
    if (goal < run + step) {
      uint64_t upto = run + inc - of_lane;
      if (goal >= upto && goal < run + inc) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          if (goal >= upto && goal < upto + w[e]) {
            p.ids[r] = i + lane * PER + e;
            if (p.logprob) p.logprob[r] = (float)log((double)w[e] / (double)all);
          }
          upto += w[e];
        }
      }
      return;
    }
    run += step;
  }
}

}  // namespace

extern "C" int sgemv_sample(const sgemv_sampling* g, void* hip_stream) {
  if (!g || g->rows < 0 || g->vocab < 1) return SGEMV_EINVAL;
  if (g->dtype != SGEMV_F16 && g->dtype != SGEMV_BF16 && g->dtype != SGEMV_F32) return SGEMV_EINVAL;
  if (g->rows > 65535 || g->vocab > kMostVocab) return SGEMV_ESIZE;
  if (g->rows > 1 && g->x_stride < 0) return SGEMV_EINVAL;
  if (g->rows == 0) return SGEMV_OK;
  if (!g->x || !g->uniform || !g->ids) return SGEMV_EINVAL;
  if ((uintptr_t)g->x % (g->dtype == SGEMV_F32 ? 4 : 2)) return SGEMV_EALIGN;
  for (const void* q : {(const void*)g->uniform, (const void*)g->temperature, (const void*)g->top_k, (const void*)g->top_p,
                        (const void*)g->min_p, (const void*)g->ids, (const void*)g->logprob})
    if ((uintptr_t)q % 4) return SGEMV_EALIGN;
  SampleParams p;
  memset(&p, 0, sizeof p);
  p.x = g->x;
  p.stride = g->rows > 1 ? g->x_stride : 0;
  p.uniform = g->uniform;
  p.temperature = g->temperature;
  p.top_k = g->top_k;
  p.top_p = g->top_p;
  p.min_p = g->min_p;
  p.ids = g->ids;
  p.logprob = g->logprob;
  p.vocab = g->vocab;
  (void)hipGetLastError();
  const dim3 grid((uint32_t)g->rows), block(kLanes);
  if (g->dtype == SGEMV_F32) hipLaunchKernelGGL(sample_kernel<float>, grid, block, 0, (hipStream_t)hip_stream, p);
  else if (g->dtype == SGEMV_F16) hipLaunchKernelGGL(sample_kernel<_Float16>, grid, block, 0, (hipStream_t)hip_stream, p);
  else hipLaunchKernelGGL(sample_kernel<__bf16>, grid, block, 0, (hipStream_t)hip_stream, p);
  return hipGetLastError() == hipSuccess ? SGEMV_OK : SGEMV_EHIP;
}
