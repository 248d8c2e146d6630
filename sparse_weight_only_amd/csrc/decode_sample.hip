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
#include <type_traits>

#include "decode_internal.hpp"
#include "launch_util.hpp"
#include "sample_bound.hpp"

using namespace sgemv;

namespace {

using sgemv_dev::KeyBins;
using sgemv_dev::LogitBins;
using sgemv_dev::key_of;
using sgemv_dev::of_key;

constexpr int kLanes = sgemv_dev::kSampleLanes, kWaves = sgemv_dev::kSampleWaves;
constexpr uint32_t kNever = sgemv_dev::kNeverKey;
constexpr int kUnit = 43;                            // p in units of 2^-43: 2^20 of them fit 64 bits
constexpr int kMostVocab = 1 << 20;
constexpr int kBins = 2048;                          // of a step of a search
constexpr int kMassBins = 512, kBinsPerPower = 16;   // of a wave's masses by value: 16 to a power of two
constexpr int kHeld = 32;                            // logits that a lane may hold
typedef float floats __attribute__((ext_vector_type(kHeld)));
constexpr int kList = 8192;                          // tokens that are looked at one by one: 64 KiB of places
// The k-th largest of the lanes' own largest is a bound: where logits come in no
// order and every lane has some, 1024 ln(1024 / (1024 - k)) of a row are above it,
// 1420 for 768. From there on the searches over the row are hardly slower (1 x
// 32000: top_k 50 8.2 us, 768 18.6, 1000 30.2).
constexpr int kMostK = 768;

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

// A token's place in its row's order by value, the largest first: of equal
// logits the lower id.
__device__ __forceinline__ uint64_t place_of(uint32_t key, uint32_t id) { return (uint64_t)key << 32 | (uint32_t)~id; }

// What a lane gets of x by a data-parallel move (0 where it gets nothing).
template <int MOVE, int ROWS = 0xf>
__device__ __forceinline__ uint32_t moved(uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, MOVE, ROWS, 0xf, true); }
template <int MOVE, int ROWS = 0xf>
__device__ __forceinline__ uint64_t moved(uint64_t x) { return (uint64_t)moved<MOVE, ROWS>((uint32_t)(x >> 32)) << 32 | moved<MOVE, ROWS>((uint32_t)x); }
constexpr int kShift1 = 0x111, kShift2 = 0x112, kShift4 = 0x114, kShift8 = 0x118;       // from the lane so many places down, in rows of 16
constexpr int kLast15 = 0x142, kLast31 = 0x143;                                        // the last lane of the row below, of the lower half
constexpr int kPair = 0xb1, kQuad = 0x4e, kHalf = 0x141, kMirror = 0x140;              // lanes 1 and 2 away; mirrored in 8, in 16

template <class X>
__device__ __forceinline__ X wave_prefix(X x) {      // inclusive
  x += moved<kShift1>(x);
  x += moved<kShift2>(x);
  x += moved<kShift4>(x);
  x += moved<kShift8>(x);
  x += moved<kLast15, 0xa>(x);
  x += moved<kLast31, 0xc>(x);
  return x;
}
__device__ __forceinline__ uint32_t read_lane(uint32_t x, int i) { return (uint32_t)__builtin_amdgcn_readlane((int)x, i); }
__device__ __forceinline__ uint64_t read_lane(uint64_t x, int i) { return (uint64_t)read_lane((uint32_t)(x >> 32), i) << 32 | read_lane((uint32_t)x, i); }
template <class X>
__device__ __forceinline__ X last_lane(X x) { return read_lane(x, 63); }
__device__ __forceinline__ uint64_t wave_sum(uint64_t x) { return last_lane(wave_prefix(x)); }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  const auto up = [&](uint32_t y) { x = y > x ? y : x; };
  up(moved<kShift1>(x));
  up(moved<kShift2>(x));
  up(moved<kShift4>(x));
  up(moved<kShift8>(x));
  up(moved<kLast15, 0xa>(x));
  up(moved<kLast31, 0xc>(x));
  return last_lane(x);
}
// The sum over 4, 8 or 16 neighbouring lanes, in each of them.
template <class X>
__device__ __forceinline__ X near_sum(X x, int lanes) {
  x += moved<kPair>(x);
  x += moved<kQuad>(x);
  if (lanes > 4) x += moved<kHalf>(x);
  if (lanes > 8) x += moved<kMirror>(x);
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
  uint32_t best[2][kWaves];
  uint64_t above, place;
  uint32_t bin_count;
  int bin, listed;
};

// The largest of two numbers each over the workgroup.
__device__ __forceinline__ void block_max(Shared& s, uint32_t& u, uint32_t& v) {
  u = wave_max(u);
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    s.best[0][threadIdx.x >> 6] = u;
    s.best[1][threadIdx.x >> 6] = v;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    u = s.best[0][w] > u ? s.best[0][w] : u;
    v = s.best[1][w] > v ? s.best[1][w] : v;
  }
}

// Exclusive prefix over the workgroup, and the sum in `all`.
template <class X>
__device__ __forceinline__ X block_prefix(Shared& s, X v, X& all) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const X inc = wave_prefix(v);
  __syncthreads();
  if (lane == 63) s.part[wave] = inc;
  __syncthreads();
  // each row of 16 lanes goes through the waves' sums
  X sums = (X)s.part[lane & (kWaves - 1)];
  sums += moved<kShift1>(sums);
  sums += moved<kShift2>(sums);
  sums += moved<kShift4>(sums);
  sums += moved<kShift8>(sums);
  all = last_lane(sums);
  const X before = wave ? read_lane(sums, wave - 1) : 0;
  return before + inc - v;
}

// A row and what its weights follow from.
template <class T, int PER_>
struct Row {
  static constexpr int PER = PER_;                   // logits of a lane and load, at most a row's
  typedef T Some __attribute__((ext_vector_type(PER), aligned(sizeof(T))));   // rows of any vocabulary: element alignment only
  const T* x;
  int vocab;
  float top;                                         // M
  float least;                                       // the smallest logit that min_p (or being a number) leaves
  double base, scale;                                // M and log2(e) / T
  double floor;                                      // of exponents: where M is infinite the others' do not count, and its own are 0

  // y f + c. Left to itself the compiler moves every coefficient into the
  // registers of the sum first, which is a third of the polynomial's time.
  static __device__ __forceinline__ double step(double y, double f, double c) {
    double r;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(y), "v"(f), "s"(c));
    return r;
  }
  // 2^((x - M) scale) in units of 2^-43, rounded; for x from `least` on.
  __device__ __forceinline__ uint64_t weight(float v) const {
    // no number (infinities less each other) becomes the floor
    const double z = __builtin_fmax(((double)v - base) * scale, floor);
    // the nearest whole number, in the low bits too
    const double big = z + 0x1.8p52, n = big - 0x1.8p52, f = z - n;
    double y = 0x1.b69b333333333p+19;                // 2^43 2^f
    y = step(y, f, 0x1.63f1a66666666p+23);
    y = step(y, f, 0x1.ffcb2e3333335p+26);
    y = step(y, f, 0x1.43088c34ccccbp+30);
    y = step(y, f, 0x1.5d87fea9ba666p+33);
    y = step(y, f, 0x1.3b2ab72c33333p+36);
    y = step(y, f, 0x1.c6b08d70374acp+38);
    y = step(y, f, 0x1.ebfbdff813d86p+40);
    y = step(y, f, 0x1.62e42fefa3a31p+42);
    y = step(y, f, 0x1.000000000003fp+43);
    // times 2^n (n >= -1000: no subnormals)
    const uint64_t bits = __builtin_bit_cast(uint64_t, y) + ((uint64_t)__builtin_bit_cast(uint64_t, big) << 52);
    // 2^52 on top leaves the number in the low bits, rounded to a whole one
    return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, bits) + 0x1p52) & 0xfffffffffffffull;
  }
  // The PER logits from `at` on of those before `end`. A load that would pass the
  // end comes back to it, without a branch, which would wait for every load.
  __device__ __forceinline__ Some load(int at, int end) const { return *(const Some*)(x + (end - PER < at ? end - PER : at)); }
  // f(logits, first id) for PER ids at a time of [a, b), by the lanes `lane` of n;
  // those that a load past the end brings once more, or that are none, as no numbers.
  // AHEAD loads of a lane are on their way at any time. One body for all of them:
  // a row of a workgroup's own is gone through a few times, each time by other
  // code, which costs more to fetch than to execute where it is long.
  template <int AHEAD, class F>
  __device__ __forceinline__ void each(int a, int b, int lane, int n, F f) const {
    const int step = n * PER;
    int at = a + lane * PER;
    if (a >= b) return;
    Some w[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) w[k] = load(at + k * step, b);
    for (int i = a; i < b; i += AHEAD * step) {
      float v[AHEAD][PER];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
#pragma unroll
        for (int e = 0; e < PER; ++e) v[k][e] = (float)w[k][e];
        w[k] = load(at + (k + AHEAD) * step, b);
      }
      if (i + AHEAD * step > b) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
          for (int e = 0; e < PER; ++e) v[k][e] = b - PER + e >= at + k * step || at + k * step <= b - PER ? v[k][e] : __builtin_nanf("");
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int id = at + k * step;
        f(v[k], id < b - PER ? id : b - PER);
      }
      at += AHEAD * step;
    }
  }
};

// Where the tokens that a search goes through come from: the row itself, or
// what has been listed of it. f(place, logit) for each.
template <class R>
struct FromRow {
  const R& row;
  template <class F>
  __device__ __forceinline__ void operator()(F f) const {
    row.template each<1>(0, row.vocab, threadIdx.x, kLanes, [&](const float (&v)[R::PER], int id) {
#pragma unroll
      for (int e = 0; e < R::PER; ++e)
        if (v[e] >= row.least) f(place_of(key_of(v[e]), id + e), v[e]);
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

// goal of a sum: the least whole number that is `share` of `sum` or more, 1 at least
__device__ __forceinline__ uint64_t goal_of(float share, uint64_t sum) {
  const double want = (double)sum * (double)share;
  uint64_t goal = want > 0.0 ? (uint64_t)want : 0;
  goal += (double)goal < want;
  return goal < 1 ? 1 : goal > sum ? sum : goal;
}

// the sum that a random number stands for: the token is the first to pass it
__device__ __forceinline__ uint64_t chosen_of(float u, uint64_t all) {
  const double at = (double)(u > 0.0f ? u : 0.0f) * (double)all;
  const uint64_t goal = at < (double)all ? (uint64_t)at : all - 1;
  return goal < all ? goal : all - 1;
}

template <class S>
__device__ __forceinline__ uint64_t count_of(Shared& s, const S& source) {
  uint64_t n = 0, all;
  source([&](uint64_t, float) { ++n; });
  block_prefix(s, n, all);
  return all;
}
template <class R, class S>
__device__ __forceinline__ uint64_t mass_from(Shared& s, const R& row, const S& source, uint64_t border) {
  uint64_t n = 0, all;
  source([&](uint64_t p, float v) { n += p >= border ? row.weight(v) : 0; });
  block_prefix(s, n, all);
  return all;
}

// Tokens that are compared each with each, 4 to 16 lanes a token: 64 comparisons a
// lane at most, in place of a histogram's barriers (1 x 32000, top_k 50: 18 -> 12.6
// us, 16 x 32000 with top_p: 35 -> 25).
constexpr int kPairs = 256;

// Up to kPairs places, each with all: for the lane that a token is with (one of 4
// to 16 neighbours) its place and weight, its rank and the weight of those larger;
// `there` is false in the others. Weights stay in s.mass.
struct Token {
  uint64_t place, weight, above;
  uint32_t rank;
  bool there;
};
__device__ __forceinline__ int lanes_of(int n) { return n <= 64 ? 16 : n <= 128 ? 8 : 4; }
template <class R>
__device__ __forceinline__ Token compare_all(Shared& s, const R& row, const uint64_t* places, int n) {
  const int tid = threadIdx.x;
  if (tid < n) s.mass[tid] = row.weight(of_key((uint32_t)(places[tid] >> 32)));
  __syncthreads();
  const int lanes = lanes_of(n), mine = tid / lanes, at = mine < n ? mine : n - 1;
  Token t{places[at], s.mass[at], 0, 0, mine < n && tid % lanes == 0};
  for (int j = tid % lanes; j < n; j += lanes) {
    const bool larger = places[j] > t.place;
    t.rank += larger;
    t.above += larger ? s.mass[j] : 0;
  }
  t.rank = near_sum(t.rank, lanes);
  t.above = near_sum(t.above, lanes);
  return t;
}

// The border among a source's places in [lo, hi], of which there is one at least:
// the last one in order such that those up to it, counted (MASS: weighed), reach
// `goal`, which all together do. A histogram of kBins intervals, of the one with
// the border again where it holds too many to compare.
template <bool MASS, class R, class S>
__device__ uint64_t find_border(Shared& s, const R& row, const S& source, uint64_t lo, uint64_t hi, uint64_t goal) {
  for (int round = 0; round < 6; ++round) {            // 64 bits, 11 a round
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
    const int n = s.bin_count;
    __syncthreads();
    if (lo == hi) return hi;
    if (n <= kPairs) {
      uint64_t* near = (uint64_t*)s.count;
      if (threadIdx.x == 0) s.bin = 0;
      __syncthreads();
      source([&](uint64_t p, float) {
        if (p >= lo && p <= hi) near[atomicAdd(&s.bin, 1)] = p;
      });
      __syncthreads();
      const Token t = compare_all(s, row, near, n);
      const uint64_t above = MASS ? t.above : t.rank, weight = MASS ? t.weight : 1;
      if (t.there && above < goal && above + weight >= goal) s.place = t.place;
      __syncthreads();
      return s.place;
    }
  }
  return hi;
}

// One workgroup a row. Ways to what is kept:
//  * top_k up to kMostK: at least k tokens are as large as the k-th largest of the
//    lanes' own largest logits, and hardly more; those are listed, and up to 64
//    lanes' more, since the k-th is looked for by counting (sample_bound.hpp).
//    Lanes without a logit, which many lengths and masks leave, do not count (1 x
//    50257 in 16 bits, top_k 50: 11 us, 44 with all of the row listed); tokens
//    of -1e9 in place of -inf cost two counts more (1 x 32000, 90 % of them: 11.4
//    us, 9.1 without). All are listed where fewer than k lanes have any. With min_p
//    alone those that it leaves are.
//  * top_p without them, or more than the list takes: each wave sums the p of its
//    stretch of the row by value, in bins of 1/16 power of two; the tokens of the
//    bin that the border falls into are listed.
//  * anything else: searches over the row.
// Up to kPairs listed tokens are compared each with each, of more the border is
// searched for with histograms. The token is then, if all that is kept was
// compared, among them; otherwise it is looked for in the stretch of the row, a
// sixteenth of it, that the sums of the kept p point at.
//
// HELD, for rows that fit: what a lane reads of its wave's stretch stays in its
// registers, and the row is read once (1 x 32000 among other calls, top_k 50 and
// top_p: 10.3 -> 9.2 us).
//
// A row is bound by its round trips where there are few: 1 x 32000 takes 4.0 us
// for the largest logit, 6.6 with min_p, 8.2 with top_k 50, 8.8 with top_p behind
// it, 18 with top_p alone. Of 256 rows of 128003, one a compute unit, 29 us are
// the pass over the logits (131 MB at 4.5 TB/s), 43 top_k, 50 min_p; top_p alone,
// 80, is bound by the vector units: 26 us of 64-bit weights with an LDS atomic
// each. Its rows are read 2.8 times: for the largest, the masses and the list,
// and the list's pass takes 15 to 20 us although few of it are listed.
// Searches over the row, which is what is left for top_k over 768 and flat rows,
// take 120 there.
//
// LIGHT and HEAVY loads of a lane are on their way: 4 where a logit takes a few
// operations, 2 of 16 bytes of FP32 where it takes a weight. With more the loops,
// each gone through a few times, take longer to fetch than what they wait less.
template <class T, int PER, bool HELD>
__global__ void __launch_bounds__(kLanes) sample_kernel(SampleParams p) {
  __shared__ Shared s;
  const int r = blockIdx.x, tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  Row<T, PER> row;
  row.x = (const T*)p.x + r * p.stride;
  row.vocab = p.vocab;
  const float t = p.temperature ? p.temperature[r] : 1.0f, u = p.uniform[r];
  const int k = p.top_k ? p.top_k[r] : 0;
  const float top_p = p.top_p ? p.top_p[r] : 1.0f, min_p = p.min_p ? p.min_p[r] : 0.0f;
  constexpr int LIGHT = 4, HEAVY = PER == 1 ? 2 : 8 / PER;   // loads on their way
  // a wave's stretch of the row, in whole steps of the wave
  const int stretch = sgemv_dev::stretch_of(row.vocab, PER);
  const int from = wave * stretch < row.vocab ? wave * stretch : row.vocab, to = from + stretch < row.vocab ? from + stretch : row.vocab;
  if (tid < kWaves) s.stretch[tid] = 0;
  if (tid == 0) s.listed = 0;
  s.count[tid] = 0;

  float most = -__builtin_inff();
  floats held = {};
  constexpr int LOADS = kHeld / PER;
  if constexpr (HELD) {
    typename Row<T, PER>::Some w[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) w[k] = row.load(from + (k * 64 + lane) * PER, to);
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int at = from + (k * 64 + lane) * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float v = at <= to - PER || to - PER + e >= at ? (float)w[k][e] : __builtin_nanf("");
        held[k * PER + e] = v;
        most = fmaxf(most, v);
      }
    }
  } else {
    row.template each<LIGHT>(from, to, lane, 64, [&](const float (&v)[PER], int) {
#pragma unroll
      for (int e = 0; e < PER; ++e) most = fmaxf(most, v[e]);
    });
  }
  // f(logits, first id) for what the lane has of the wave's stretch
  const auto own = [&](auto ahead, auto f) {
    if constexpr (HELD) {
#pragma unroll 1
      for (int k = 0; k < LOADS; ++k) {
        const int at = from + (k * 64 + lane) * PER;
        float v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = held[k * PER + e];
        f(v, at < to - PER ? at : to - PER);
      }
    } else {
      row.template each<decltype(ahead)::value>(from, to, lane, 64, f);
    }
  };
  const std::integral_constant<int, LIGHT> light{};
  const std::integral_constant<int, HEAVY> heavy{};
  row.scale = 1.4426950408889634074 / (double)t;
  const double log_p = min_p > 0.0f && min_p < 1.0f ? log2((double)min_p) : 0.0;
  const uint32_t mine = key_of(most);
  uint32_t top_key = mine, low_key = sgemv_dev::low_part(mine);   // of the lanes' largest the largest and the smallest
  block_max(s, top_key, low_key);
  low_key = ~low_key;
  if (top_key <= kNever) {
    if (tid == 0) {
      p.ids[r] = -1;
      if (p.logprob) p.logprob[r] = -__builtin_inff();
    }
    return;
  }
  row.top = of_key(top_key);
  if (!(t > 0.0f)) {
    uint32_t first = 0, none = 0;                      // the lowest id, as the largest of its complements
    if (mine == top_key)
      own(std::integral_constant<int, 1>{}, [&](const float (&v)[PER], int id) {
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (v[e] == row.top && ~(uint32_t)(id + e) > first) first = ~(uint32_t)(id + e);
      });
    block_max(s, first, none);
    if (tid == 0) {
      p.ids[r] = (int32_t)~first;
      if (p.logprob) p.logprob[r] = 0.0f;
    }
    return;
  }
  const bool infinite = !(row.top < __builtin_inff());
  row.base = (double)row.top;
  row.floor = infinite ? 0.0 : -1000.0;
  row.least = infinite ? row.top : -0x1.fffffep127f;
  const bool some = min_p > 0.0f && !infinite;
  if (some) {
    // the smallest logit of exponent log2(min_p) or more: from where it should be
    // outwards in growing steps, then halving
    const auto enough = [&](uint32_t key) { return ((double)of_key(key) - row.base) * row.scale >= log_p; };
    const double about = row.base + log_p / row.scale;
    uint32_t yes = top_key, no = kNever;               // no logit at all is not enough
    uint32_t key = about > -0x1.fffffep127 ? key_of((float)about) : kNever + 1;
    key = key > top_key ? top_key : key;
    for (uint32_t step = 1; yes - no > 1; step *= 8) {
      if (enough(key)) {
        yes = key;
        if (no != kNever) break;
        key = yes - no > step ? yes - step : no + 1;
      } else {
        no = key;
        if (yes != top_key) break;
        key = yes - no > step ? no + step : yes - 1;
      }
      if (step >= 1u << 27) break;
    }
    while (yes - no > 1) {
      const uint32_t mid = no + (yes - no) / 2;
      if (enough(mid)) yes = mid;
      else no = mid;
    }
    row.least = of_key(yes);
  }
  // lists the tokens from `bound` on that are wanted; how many there are, or more
  // than the list takes
  const auto list = [&](float bound, auto wanted) {
    bool full = false;                                 // to this lane's knowledge; a held row is soon through
    own(light, [&](const float (&v)[PER], int id) {
      // most lanes have none: one look at the largest
      float top = v[0];
#pragma unroll
      for (int e = 1; e < PER; ++e) top = fmaxf(top, v[e]);
      if (!(top >= bound) || (!HELD && full)) return;
      uint32_t bits = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) bits |= (uint32_t)(v[e] >= bound && wanted(v[e])) << e;
      if (!bits) return;
      int at = atomicAdd(&s.listed, __popc(bits));
      if (!HELD) full = at >= kList;
      while (bits) {
        const int e = __ffs(bits) - 1;
        bits &= bits - 1;
        float one = v[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) one = i == e ? v[i] : one;
        if (at < kList) s.list[at] = place_of(key_of(one), id + e);
        ++at;
      }
    });
    __syncthreads();
    return s.listed;
  };
  int n = kList + 1;                                   // listed tokens; too many for the list: none
  uint64_t rest = 0;                                   // of those listed, the sum that the kept ones reach, where the larger ones are not listed
  const bool by_count = k > 0 && k <= kMostK;
  if (by_count || (some && k <= 0)) {
    float bound = row.least;
    if (by_count) {
      // the interval of the k-th largest of the lanes' largest; none where not so many lanes have any
      bool here = most >= row.least;
      const auto find = [&](int at, int need) {
        if (here) atomicAdd(&s.count[at], 1u);
        __syncthreads();
        uint32_t all;
        const uint32_t c = s.count[tid], before = block_prefix(s, c, all);
        s.count[tid] = 0;
        if (before < (uint32_t)need && before + c >= (uint32_t)need) {
          s.bin = tid;
          s.above = before;
          s.bin_count = c;
        }
        __syncthreads();
      };
      if (tid == 0) s.bin = kLanes;
      const LogitBins bins(row.top, fmaxf(of_key(low_key), row.least));
      int at = bins.bin(most), need = k;
      find(at, need);
      if (s.bin < kLanes) {
        bound = fmaxf(bound, bins.lower(s.bin));
        if (s.bin_count > (uint32_t)sgemv_dev::kCrowd) {
          here &= at == s.bin;
          need -= (int)s.above;
          uint32_t hi = here ? mine : 0, lo = here ? ~mine : 0;
          block_max(s, hi, lo);
          KeyBins keys(hi, ~lo);
          for (int round = 0; round < sgemv_dev::kKeyRounds; ++round) {
            at = here ? keys.bin(mine) : 0;
            find(at, need);
            here &= at == s.bin;
            need -= (int)s.above;
            keys.narrow(s.bin);
            if (s.bin_count <= (uint32_t)sgemv_dev::kCrowd || keys.low == keys.top) break;
          }
          bound = fmaxf(bound, of_key(keys.low));
        }
      }
    }
    n = list(bound, [](float) { return true; });
  }
  if (n > kList && k <= 0 && top_p < 1.0f) {
    const float by = fminf(kBinsPerPower * (float)row.scale, 1e30f);
    const auto bin_of = [&](float v) { return (int)fminf(fmaxf((row.top - v) * by, 0.0f), kMassBins - 1.0f); };  // no number (of infinite logits): 0
    __syncthreads();
    if (tid == 0) s.listed = 0;
    for (int i = lane; i < kMassBins; i += 64) s.wave_mass[wave][i] = 0;
    own(heavy, [&](const float (&v)[PER], int) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        // without branches, so that one weight's latencies are the others' time
        uint64_t w = row.weight(v[e]);
        asm("" : "+v"(w));
        atomicAdd(&s.wave_mass[wave][bin_of(v[e])], (unsigned long long)(v[e] >= row.least ? w : 0));
      }
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
    rest = goal - s.above;
    uint64_t larger = 0;
    for (int i = lane; i < last; i += 64) larger += s.wave_mass[wave][i];
    larger = wave_sum(larger);
    const float least_of = last, past = last < kMassBins - 1 ? last + 1.0f : __builtin_nanf("");
    n = list(row.least, [&](float v) {
      const float y = (row.top - v) * by;
      return !(y < least_of) && !(y >= past);
    });
    if (n <= kList && lane == 0) s.stretch[wave] = larger;
  }

  uint64_t border = place_of(key_of(row.least), ~0u);  // tokens from it on, in order, are kept
  bool summed = false;                                 // s.stretch holds the sums of what is kept
  if (n <= kPairs) {
    const Token one = compare_all(s, row, s.list, n);
    bool kept = one.there;
    if (!rest) {
      // all that is kept is here: the token among them, by their ids
      uint64_t all, before = 0;
      if (k > 0) kept &= one.rank < (uint32_t)k;
      block_prefix(s, kept ? one.weight : 0, all);
      if (top_p < 1.0f) {
        kept &= one.above < goal_of(top_p, all);
        block_prefix(s, kept ? one.weight : 0, all);
      }
      const int lanes = lanes_of(n);
      if (one.there && !kept) s.mass[tid / lanes] = 0;
      __syncthreads();
      const uint64_t goal = chosen_of(u, all);
      const uint32_t id = ~(uint32_t)one.place;
      for (int j = tid % lanes; j < n; j += lanes) before += ~(uint32_t)s.list[j] < id ? s.mass[j] : 0;
      before = near_sum(before, lanes);
      if (kept && before <= goal && goal < before + one.weight) {
        p.ids[r] = (int32_t)id;
        if (p.logprob) p.logprob[r] = (float)log((double)one.weight / (double)all);
      }
      return;
    }
    kept &= one.above < rest;
    if (kept && one.above + one.weight >= rest) s.place = one.place;
    if (kept) atomicAdd(&s.stretch[~(uint32_t)one.place / (uint32_t)stretch], (unsigned long long)one.weight);
    __syncthreads();
    border = s.place;
    summed = true;
  } else if (n <= kList) {
    const FromList listed{s, n};
    uint32_t hi_key = 0, lo_key = 0;
    for (int i = tid; i < n; i += kLanes) {
      const uint32_t key = (uint32_t)(s.list[i] >> 32);
      hi_key = key > hi_key ? key : hi_key;
      lo_key = ~key > lo_key ? ~key : lo_key;
    }
    block_max(s, hi_key, lo_key);
    const uint64_t hi = place_of(hi_key, 0);
    border = place_of(~lo_key, ~0u);
    if (!rest && k > 0 && n > k) border = find_border<false>(s, row, listed, border, hi, k);
    if (top_p < 1.0f)
      border = find_border<true>(s, row, listed, border, hi, rest ? rest : goal_of(top_p, mass_from(s, row, listed, border)));
    for (int i = tid; i < n; i += kLanes) {
      const uint64_t q = s.list[i];
      if (q >= border) atomicAdd(&s.stretch[~(uint32_t)q / (uint32_t)stretch], (unsigned long long)row.weight(of_key((uint32_t)(q >> 32))));
    }
    summed = true;
  } else if (k > 0 || top_p < 1.0f) {
    const FromRow<Row<T, PER>> whole{row};
    const uint64_t hi = place_of(top_key, 0);
    if (k > 0 && count_of(s, whole) > (uint64_t)k) border = find_border<false>(s, row, whole, border, hi, k);
    if (top_p < 1.0f) border = find_border<true>(s, row, whole, border, hi, goal_of(top_p, mass_from(s, row, whole, border)));
  }

  // the weights of the kept ones of [a, b), 64 ids at a time: f(weight, first id)
  const auto each_kept = [&](int a, int b, auto f) {
    T next = a + lane < b ? row.x[a + lane] : (T)__builtin_nanf("");
    for (int i = a; i < b; i += 64) {
      const float v = (float)next;
      const int id = i + lane, ahead = id + 64;
      if (ahead < b) next = row.x[ahead];
      const bool kept = id < b && v >= row.least && place_of(key_of(v), id) >= border;
      if (f(kept ? row.weight(v) : 0, i)) return;
    }
  };
  if (!summed) {
    uint64_t sum = 0;
    own(heavy, [&](const float (&v)[PER], int id) {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (v[e] >= row.least && place_of(key_of(v[e]), id + e) >= border) sum += row.weight(v[e]);
    });
    sum = wave_sum(sum);
    if (lane == 0) s.stretch[wave] = sum;
  }
  __syncthreads();
  // the stretch of the token, by every wave for itself
  uint64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all += s.stretch[w];
  const uint64_t goal = chosen_of(u, all);
  uint64_t run = 0;
  int chosen = 0;
  while (run + s.stretch[chosen] <= goal) run += s.stretch[chosen++];
  // and in it, again by waves and then step by step of the one
  const int a = chosen * stretch, piece = stretch / kWaves;
  const int end = a + stretch < row.vocab ? a + stretch : row.vocab;
  const int pa = a + wave * piece < end ? a + wave * piece : end, pb = pa + piece < end ? pa + piece : end;
  uint64_t sum = 0;
  each_kept(pa, pb, [&](uint64_t w, int) {
    sum += w;
    return false;
  });
  sum = wave_sum(sum);
  if (lane == 0) s.part[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) run += s.part[w];
  if (goal < run || goal >= run + sum) return;
  each_kept(pa, pb, [&](uint64_t w, int first) {
    const uint64_t upto = run + wave_prefix(w);
    if (goal < upto && goal >= upto - w) {
      p.ids[r] = first + lane;
      if (p.logprob) p.logprob[r] = (float)log((double)w / (double)all);
    }
    run = last_lane(upto);
    return goal < run;
  });
}

typedef void (*SampleFn)(SampleParams);
template <class T>
SampleFn pick(int vocab) {
  constexpr int PER = 16 / sizeof(T);
  // lanes hold what 16 of their waves' stretches, in whole steps, come to
  return vocab < PER ? sample_kernel<T, 1, false> : vocab <= kLanes * kHeld ? sample_kernel<T, PER, true> : sample_kernel<T, PER, false>;
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
  // rows of fewer logits than a load takes: one by one
  const SampleFn fn = g->dtype == SGEMV_F32 ? pick<float>(g->vocab) : g->dtype == SGEMV_F16 ? pick<_Float16>(g->vocab) : pick<__bf16>(g->vocab);
  hipLaunchKernelGGL(fn, grid, block, 0, (hipStream_t)hip_stream, p);
  return hipGetLastError() == hipSuccess ? SGEMV_OK : SGEMV_EHIP;
}
