// Penalties for repeated tokens, biases and grammar masks on logits.
//
// For token v of a row, with `seen` whether v is in the row's history and n how
// often behind its prompt:
//   l <- seen ? (l > 0 ? l / repetition : l * repetition) : l
//   l <- l - frequency n - presence [n > 0]
//   l <- l + bias(v)
//   l <- -inf where the row's mask bit v is 0
// in FP32, rounded once to the output's type.
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;

namespace {

constexpr int kLanes = 256;
constexpr int kPer = 4;                              // logits of a lane and step
constexpr int kSteps = 4;
constexpr int kPart = kLanes * kPer * kSteps;        // vocabulary entries of a workgroup

struct LogitsParams {
  const void* x;
  void* out;
  int64_t x_stride, out_stride;
  const int32_t *hist_start, *hist_ids, *prompt_len;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_start, *bias_ids;
  const float* bias_values;
  const uint32_t* masks;
  const int32_t* mask_row;
  int64_t n_hist, n_bias, mask_stride;
  int32_t vocab, n_masks;
};

template <class T>
using Four = T __attribute__((ext_vector_type(4), aligned(sizeof(T))));   // rows of any vocabulary: element alignment only

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t most) { return v < 0 ? 0 : v > most ? most : v; }

// f(entry, place) for the ids of a list that fall into the part; eight ids of
// a lane are on their way at once.
template <class F>
__device__ __forceinline__ void each_id(const int32_t* ids, int64_t a, int64_t b, int v0, int n, F f) {
  constexpr int AHEAD = 8;
  for (int64_t i0 = a + threadIdx.x; i0 < b; i0 += kLanes * AHEAD) {
    int32_t id[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t i = i0 + k * kLanes;
      id[k] = ids[i < b ? i : b - 1];
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t i = i0 + k * kLanes;
      const uint32_t at = (uint32_t)id[k] - (uint32_t)v0;
      if (i < b && at < (uint32_t)n) f(at, i);
    }
  }
}

// Workgroup (c, b): entries c kPart .. of row b. The counts of its entries are
// kept in LDS: every lane walks the history and counts the ids that fall into
// the part (whole numbers, so the order of the atomics does not matter). Of a
// bias id given twice the later place wins, by an atomic maximum of the places;
// then the winners put their values where the places were.
// Bound by memory for a batch, by its round trips for one row: everything that
// does not wait for something else is asked for at the start.
template <class TI, class TO, bool HIST, bool BIAS>
__global__ void __launch_bounds__(kLanes) logits_kernel(LogitsParams p) {
  __shared__ uint32_t count[HIST ? kPart : 1];       // bit 31: in the prompt; below: how often behind it
  __shared__ uint32_t place[BIAS ? kPart : 1];       // place in the row's bias list + 1, then the bias
  const int tid = threadIdx.x, row = blockIdx.y;
  const int v0 = blockIdx.x * kPart;
  const int n = p.vocab - v0 < kPart ? p.vocab - v0 : kPart;
  const TI* x = (const TI*)p.x + row * p.x_stride + v0;
  TO* out = (TO*)p.out + row * p.out_stride + v0;

  int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
  int prompt = 0, m = -1;
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (HIST) {
    h0 = p.hist_start[row];
    h1 = p.hist_start[row + 1];
    if (p.prompt_len) prompt = p.prompt_len[row];
    if (p.repetition) rep = p.repetition[row];
    if (p.frequency) freq = p.frequency[row];
    if (p.presence) pres = p.presence[row];
  }
  if (BIAS) {
    b0 = p.bias_start[row];
    b1 = p.bias_start[row + 1];
  }
  if (p.masks) m = p.mask_row ? p.mask_row[row] : row;
  float l[kSteps][kPer];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int at = (s * kLanes + tid) * kPer;
    if (at + kPer <= n) {
      const Four<TI> w = *(const Four<TI>*)(x + at);
#pragma unroll
      for (int e = 0; e < kPer; ++e) l[s][e] = (float)w[e];
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) l[s][e] = at + e < n ? (float)x[at + e] : 0.0f;
    }
  }
  uint32_t allowed[kSteps];
  const bool masked = (uint32_t)m < (uint32_t)p.n_masks;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int at = (s * kLanes + tid) * kPer;
    allowed[s] = masked && at < n ? p.masks[m * p.mask_stride + ((v0 + at) >> 5)] >> (at & 31) : ~0u;
  }
  if (HIST || BIAS) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (HIST) *(sgemv_dev::dword4*)&count[(s * kLanes + tid) * kPer] = sgemv_dev::dword4{0, 0, 0, 0};
      if (BIAS) *(sgemv_dev::dword4*)&place[(s * kLanes + tid) * kPer] = sgemv_dev::dword4{0, 0, 0, 0};
    }
    __syncthreads();
  }
  if (HIST) {
    h0 = clamp64(h0, p.n_hist);
    h1 = clamp64(h1, p.n_hist);
    const int64_t behind = h0 + prompt;
    each_id(p.hist_ids, h0, h1, v0, n, [&](uint32_t at, int64_t i) {
      if (i < behind) atomicOr(&count[at], 0x80000000u);
      else atomicAdd(&count[at], 1u);
    });
  }
  if (BIAS) {
    b0 = clamp64(b0, p.n_bias);
    b1 = clamp64(b1, p.n_bias);
    // the first kLanes entries, most often all of them, stay with their lanes
    const int64_t i = b0 + tid;
    uint32_t at = ~0u, value = 0;
    if (i < b1) {
      at = (uint32_t)p.bias_ids[i] - (uint32_t)v0;
      value = __builtin_bit_cast(uint32_t, p.bias_values[i]);
      if (at < (uint32_t)n) atomicMax(&place[at], (uint32_t)tid + 1u);
    }
    each_id(p.bias_ids, b0 + kLanes, b1, v0, n, [&](uint32_t v, int64_t k) { atomicMax(&place[v], (uint32_t)(k - b0) + 1u); });
    __syncthreads();
    // who won is known to everybody before the first place is overwritten
    bool won = at < (uint32_t)n && place[at] == (uint32_t)tid + 1u;
    if (b1 - b0 <= kLanes) {
      __syncthreads();
      if (won) place[at] = value;
    } else {
      // a long list: values are looked up from the places, entry by entry
      uint32_t w[kSteps][kPer];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < kPer; ++e) w[s][e] = place[(s * kLanes + tid) * kPer + e];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (w[s][e]) w[s][e] = __builtin_bit_cast(uint32_t, p.bias_values[b0 + w[s][e] - 1]);
          place[(s * kLanes + tid) * kPer + e] = w[s][e];
        }
    }
  }
  if (HIST || BIAS) __syncthreads();
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int at = (s * kLanes + tid) * kPer;
    if (at >= n) break;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      float y = l[s][e];
      if (HIST) {
        const uint32_t w = count[at + e], c = w & 0x7fffffffu;
        if (w) y = y > 0.0f ? y / rep : y * rep;
        if (c) y = y - freq * (float)c - pres;
      }
      if (BIAS) y += __builtin_bit_cast(float, place[at + e]);
      l[s][e] = allowed[s] >> e & 1u ? y : -__builtin_inff();
    }
    if (at + kPer <= n) {
      Four<TO> w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[e] = (TO)l[s][e];
      *(Four<TO>*)(out + at) = w;
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (at + e < n) out[at + e] = (TO)l[s][e];
    }
  }
}

typedef void (*LogitsFn)(LogitsParams);
template <class TI, class TO>
LogitsFn pick(bool hist, bool bias) {
  return hist ? bias ? logits_kernel<TI, TO, true, true> : logits_kernel<TI, TO, true, false>
              : bias ? logits_kernel<TI, TO, false, true> : logits_kernel<TI, TO, false, false>;
}

}  // namespace

extern "C" int sgemv_adjust_logits(const sgemv_logits* g, void* hip_stream) {
  if (!g || g->rows < 0 || g->vocab < 1) return SGEMV_EINVAL;
  if (g->dtype != SGEMV_F16 && g->dtype != SGEMV_BF16 && g->dtype != SGEMV_F32) return SGEMV_EINVAL;
  if (g->out_dtype != g->dtype && g->out_dtype != SGEMV_F32) return SGEMV_EINVAL;
  const bool hist = g->hist_start || g->hist_ids, bias = g->bias_start || g->bias_ids || g->bias_values;
  if (hist && (!g->hist_start || (!g->hist_ids && g->n_hist > 0) || g->n_hist < 0 || g->n_hist > INT32_MAX)) return SGEMV_EINVAL;
  if (!hist && (g->prompt_len || g->repetition || g->frequency || g->presence)) return SGEMV_EINVAL;
  if (bias && (!g->bias_start || g->n_bias < 0 || g->n_bias > INT32_MAX || (g->n_bias > 0 && (!g->bias_ids || !g->bias_values)))) return SGEMV_EINVAL;
  const int64_t words = (g->vocab + 31) / 32;
  if (g->masks ? (g->n_masks < 1 || (g->n_masks > 1 && g->mask_stride < words)) : (g->n_masks != 0 || g->mask_row != nullptr)) return SGEMV_EINVAL;
  if (g->masks && !g->mask_row && g->n_masks != g->rows) return SGEMV_EINVAL;
  if (g->rows > 65535) return SGEMV_ESIZE;
  if (g->rows > 1 && (g->x_stride < 0 || g->out_stride < g->vocab)) return SGEMV_EINVAL;
  if (g->rows == 0) return SGEMV_OK;
  if (!g->x || !g->out) return SGEMV_EINVAL;
  const uintptr_t si = g->dtype == SGEMV_F32 ? 4 : 2, so = g->out_dtype == SGEMV_F32 ? 4 : 2;
  if (g->x == g->out && (si != so || (g->rows > 1 && g->x_stride != g->out_stride))) return SGEMV_EINVAL;
  if ((uintptr_t)g->x % si || (uintptr_t)g->out % so) return SGEMV_EALIGN;
  for (const void* q : {(const void*)g->hist_start, (const void*)g->hist_ids, (const void*)g->prompt_len, (const void*)g->repetition,
                        (const void*)g->frequency, (const void*)g->presence, (const void*)g->bias_start, (const void*)g->bias_ids,
                        (const void*)g->bias_values, (const void*)g->masks, (const void*)g->mask_row})
    if ((uintptr_t)q % 4) return SGEMV_EALIGN;
  LogitsParams p;
  memset(&p, 0, sizeof p);
  p.x = g->x;
  p.out = g->out;
  p.x_stride = g->rows > 1 ? g->x_stride : 0;
  p.out_stride = g->rows > 1 ? g->out_stride : 0;
  p.hist_start = g->hist_start;
  p.hist_ids = g->hist_ids;
  p.prompt_len = g->prompt_len;
  p.repetition = g->repetition;
  p.frequency = g->frequency;
  p.presence = g->presence;
  p.bias_start = g->bias_start;
  p.bias_ids = g->bias_ids;
  p.bias_values = g->bias_values;
  p.masks = g->masks;
  p.mask_row = g->mask_row;
  p.n_hist = g->n_hist;
  p.n_bias = g->n_bias;
  p.mask_stride = g->n_masks > 1 ? g->mask_stride : 0;
  p.vocab = g->vocab;
  p.n_masks = g->n_masks;
  LogitsFn fn = g->dtype == SGEMV_F32   ? pick<float, float>(hist, bias)
                : g->dtype == SGEMV_F16 ? (so == 4 ? pick<_Float16, float>(hist, bias) : pick<_Float16, _Float16>(hist, bias))
                                        : (so == 4 ? pick<__bf16, float>(hist, bias) : pick<__bf16, __bf16>(hist, bias));
  (void)hipGetLastError();
  const dim3 grid((uint32_t)(((int64_t)g->vocab + kPart - 1) / kPart), (uint32_t)g->rows);
  hipLaunchKernelGGL(fn, grid, dim3(kLanes), 0, (hipStream_t)hip_stream, p);
  return hipGetLastError() == hipSuccess ? SGEMV_OK : SGEMV_EHIP;
}
