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
constexpr int kPer = 4;                              // logits of a lane and step
constexpr int kBins = 2048;
constexpr int kUnit = 43;                            // p in units of 2^-43: 2^20 of them fit 64 bits
constexpr int kMostVocab = 1 << 20;

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

template <class T>
using Four = T __attribute__((ext_vector_type(4), aligned(sizeof(T))));   // rows of any vocabulary: element alignment only

// 2^z for z <= 0, in units of 2^-43, rounded
__device__ __forceinline__ uint64_t weight(double z) {
  const double n = rint(z), f = z - n;
  double y = 0x1.b69b333333333p-24;
  y = fma(y, f, 0x1.63f1a66666666p-20);
  y = fma(y, f, 0x1.ffcb2e3333335p-17);
  y = fma(y, f, 0x1.43088c34ccccbp-13);
  y = fma(y, f, 0x1.5d87fea9ba666p-10);
  y = fma(y, f, 0x1.3b2ab72c33333p-7);
  y = fma(y, f, 0x1.c6b08d70374acp-5);
  y = fma(y, f, 0x1.ebfbdff813d86p-3);
  y = fma(y, f, 0x1.62e42fefa3a31p-1);
  y = fma(y, f, 0x1.000000000003fp+0);
  // 2^52 on top leaves the number in the low bits, rounded to a whole one
  const double at = n < -1000.0 ? 0.0 : ldexp(y, (int)n + kUnit);
  return __builtin_bit_cast(uint64_t, at + 0x1p52) & 0xfffffffffffffull;
}

// Whole numbers in the order of the floats; both zeros the same, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  x = x != x ? -__builtin_inff() : x + 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kNever = 0x007fffffu;             // the key of -inf

// sums and prefixes over the workgroup; `at`: LDS of kWaves entries
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

// A row and its workgroup.
template <class T>
struct Row {
  const T* x;
  int vocab;
  uint32_t top;                                      // key of M
  double scale;                                      // log2(e) / T
  double least;                                      // log2(min_p), or -inf

  __device__ __forceinline__ double power(uint32_t key) const {
    // M itself first: infinite logits have no difference
    return key == top ? 0.0 : ((double)of_key(key) - (double)of_key(top)) * scale;
  }
  __device__ __forceinline__ bool eligible(uint32_t key) const { return key > kNever && (key == top || power(key) >= least); }
  // f(key, id) for the ids of [a, b), a multiple of 4, by the lanes `lane` of n
  template <class F>
  __device__ __forceinline__ void each(int a, int b, int lane, int n, F f) const {
    for (int i = a + lane * kPer; i < b; i += n * kPer) {
      if (i + kPer <= b) {
        const Four<T> w = *(const Four<T>*)(x + i);
#pragma unroll
        for (int e = 0; e < kPer; ++e) f(key_of((float)w[e]), i + e);
      } else {
        for (int e = i; e < b; ++e) f(key_of((float)x[e]), e);
      }
    }
  }
};

struct Shared {
  uint32_t count[kBins];
  unsigned long long mass[kBins];
  uint64_t part[kWaves + 1];
  uint32_t best[kWaves];
  int bin, found;
  uint64_t above;
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

// The border in a row's order by value: the smallest key such that the eligible
// keys from it on, counted (MASS: weighed), reach `want`, what lies above it, and
// `sum`, all of the eligible keys from `floor` on. want(sum) is asked once.
// A histogram of kBins intervals of keys at a time, so three rounds at most.
struct Border {
  uint32_t key;
  uint64_t above, sum;
  bool found;                                        // not: all together do not reach it
};
template <bool MASS, class T, class W>
__device__ Border find_border(Shared& s, const Row<T>& row, uint32_t floor, W want) {
  uint32_t hi = row.top, lo = floor;
  Border r{lo, 0, 0, true};
  uint64_t goal = 0;
  bool first = true;
  while (true) {
    const uint32_t span = hi - lo;
    const int bits = 32 - __clz((int)span), shift = span == 0 ? 0 : bits > 11 ? bits - 11 : 0;
    for (int i = threadIdx.x; i < kBins; i += kLanes) {
      if (MASS) s.mass[i] = 0;
      else s.count[i] = 0;
    }
    __syncthreads();
    row.each(0, row.vocab, threadIdx.x, kLanes, [&](uint32_t key, int) {
      if (key < lo || key > hi || !row.eligible(key)) return;
      const uint32_t bin = (hi - key) >> shift;
      if (MASS) atomicAdd(&s.mass[bin], (unsigned long long)weight(row.power(key)));
      else atomicAdd(&s.count[bin], 1u);
    });
    __syncthreads();
    const int i0 = threadIdx.x * 2;
    const uint64_t a = MASS ? s.mass[i0] : s.count[i0], b = MASS ? s.mass[i0 + 1] : s.count[i0 + 1];
    uint64_t all;
    const uint64_t before = block_prefix(s, a + b, all);
    if (first) {
      r.sum = all;
      goal = want(all);
      first = false;
      if (goal > all) {
        r.found = false;
        return r;
      }
    }
    const uint64_t need = goal - r.above;              // at least 1, and no more than `all`
    if (before < need && before + a >= need) {
      s.bin = i0;
      s.above = before;
    } else if (before + a < need && before + a + b >= need) {
      s.bin = i0 + 1;
      s.above = before + a;
    }
    __syncthreads();
    r.above += s.above;
    const uint32_t from = hi - ((uint32_t)s.bin << shift), rest = (1u << shift) - 1;
    hi = from;
    lo = from - lo > rest ? from - rest : lo;
    __syncthreads();
    if (shift == 0) {
      r.key = hi;
      return r;
    }
  }
}

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

  uint32_t most = 0;
  row.each(0, row.vocab, tid, kLanes, [&](uint32_t key, int) { most = key > most ? key : most; });
  row.top = block_max(s, most);
  if (row.top <= kNever) {
    if (tid == 0) {
      p.ids[r] = -1;
      if (p.logprob) p.logprob[r] = -__builtin_inff();
    }
    return;
  }
  if (!(t > 0.0f)) {
    uint32_t first = 0;                                // the lowest id, as the largest of its negatives
    row.each(0, row.vocab, tid, kLanes, [&](uint32_t key, int id) {
      const uint32_t v = ~(uint32_t)id;
      if (key == row.top && v > first) first = v;
    });
    first = ~block_max(s, first);
    if (tid == 0) {
      p.ids[r] = (int32_t)first;
      if (p.logprob) p.logprob[r] = 0.0f;
    }
    return;
  }
  row.scale = 1.4426950408889634074 / (double)t;
  row.least = min_p > 0.0f ? min_p < 1.0f ? log2((double)min_p) : 0.0 : -__builtin_inf();

  // what is kept: keys above `key`, and the first `ties` of `key`
  uint32_t key = kNever + 1;
  uint64_t ties = ~0ull;
  if (k > 0) {
    const Border b = find_border<false>(s, row, key, [&](uint64_t) { return (uint64_t)k; });
    if (b.found) {
      key = b.key;
      ties = k - b.above;
    }
  }
  if (top_p < 1.0f) {
    // of the tokens with the border's logit the histogram weighs all; those past
    // the border come off the sum that the share is taken of
    uint64_t extra = 0;
    if (ties != ~0ull) {
      uint64_t same = 0;
      row.each(0, row.vocab, tid, kLanes, [&](uint32_t x, int) { same += x == key; });
      uint64_t all;
      block_prefix(s, same, all);
      extra = (all - ties) * weight(row.power(key));
    }
    const Border b = find_border<true>(s, row, key, [&](uint64_t sum) {
      const double want = (double)(sum - extra) * (double)(top_p > 0.0f ? top_p : 0.0f);
      uint64_t goal = (uint64_t)want;
      goal += (double)goal < want;
      return goal < 1 ? 1 : goal;
    });
    if (b.found) {
      // as many of the border's logit as it takes, all of one weight
      double want = (double)(b.sum - extra) * (double)(top_p > 0.0f ? top_p : 0.0f);
      uint64_t goal = (uint64_t)want;
      goal += (double)goal < want;
      goal = goal < 1 ? 1 : goal;
      const uint64_t w = weight(row.power(b.key)), some = w ? (goal - b.above + w - 1) / w : 1;
      if (b.key > key || some < ties) ties = some;
      key = b.key;
    }
  }

  // Running sums by id: each wave has a stretch of the row.
  const int stretch = (row.vocab + kWaves * 256 - 1) / (kWaves * 256) * 256;
  const int a = wave * stretch < row.vocab ? wave * stretch : row.vocab, b = a + stretch < row.vocab ? a + stretch : row.vocab;
  const uint64_t tie_weight = weight(row.power(key));
  uint64_t sum = 0, same = 0;
  row.each(a, b, lane, 64, [&](uint32_t x, int) {
    if (x > key && row.eligible(x)) sum += weight(row.power(x));
    same += x == key && row.eligible(x);
  });
  uint64_t same_all, all;
#pragma unroll
  for (int d = 32; d; d /= 2) {
    sum += shfl64(sum, lane ^ d);
    same += shfl64(same, lane ^ d);
  }
  const uint64_t ties_before = block_prefix(s, lane == 0 ? same : 0, same_all);
  const uint64_t wave_ties_before = shfl64(ties_before, 0);
  const uint64_t left = ties > wave_ties_before ? ties - wave_ties_before : 0, mine = same < left ? same : left;
  const uint64_t wave_sum = sum + mine * tie_weight;
  const uint64_t lane_before = block_prefix(s, lane == 0 ? wave_sum : 0, all);
  const uint64_t before = shfl64(lane_before, 0);
  double at = (double)(u > 0.0f ? u : 0.0f) * (double)all;
  uint64_t goal = at < (double)all ? (uint64_t)at : all - 1;
  goal = goal < all ? goal : all - 1;
  if (!(before <= goal && goal < before + wave_sum)) return;
  // this wave's stretch holds the token: 256 ids at a time
  uint64_t run = before, ties_left = left;
  for (int i = a; i < b; i += 256) {
    uint64_t w[kPer];
    bool tie[kPer];
    uint32_t n_same = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int id = i + lane * kPer + e;
      const uint32_t x = id < b ? key_of((float)row.x[id]) : 0;
      const bool ok = row.eligible(x);
      tie[e] = x == key && ok;
      w[e] = x > key && ok ? weight(row.power(x)) : 0;
      n_same += tie[e];
    }
    const uint64_t same_inc = wave_prefix(n_same);
    uint64_t rank = same_inc - n_same, lane_sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (tie[e]) w[e] = rank++ < ties_left ? tie_weight : 0;
      lane_sum += w[e];
    }
    const uint64_t inc = wave_prefix(lane_sum);
    const uint64_t step = shfl64(inc, 63), step_ties = shfl64(same_inc, 63);
    if (goal < run + step) {
      uint64_t upto = run + inc - lane_sum;
      if (goal >= upto && goal < run + inc) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (goal >= upto && goal < upto + w[e]) {
            p.ids[r] = i + lane * kPer + e;
            if (p.logprob) p.logprob[r] = (float)log((double)w[e] / (double)all);
          }
          upto += w[e];
        }
      }
      return;
    }
    run += step;
    ties_left = ties_left > step_ties ? ties_left - step_ties : 0;
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
