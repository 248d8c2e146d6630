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

// Bias entries that a lane holds, 512 in all; longer lists go through the table
// (256 x 128003 logits without histories, the table's time first: 300 entries a
// row 35.8 and 36.1 us, 600 38.3 and 47.1, 1000 40.6 and 64.6).
constexpr int kShort = 2;
// Bias entries of a part that the lanes go through, each of them all; more go
// through the table too (64 rows, 300 entries in one part: 7.1 and 17.6 us).
constexpr int kListed = 256;

// The first two steps for one logit: w is its word of counts.
__device__ __forceinline__ float penalised(float y, uint32_t w, float rep, float freq, float pres) {
  const uint32_t c = w & 0x7fffffffu;
  if (w) y = y > 0.0f ? y / rep : y * rep;
  if (c) y = y - freq * (float)c - pres;
  return y;
}

// Workgroup (c, b): entries c kPart .. of row b. The counts of its entries are
// kept in LDS: every lane walks the history and counts the ids that fall into
// the part (whole numbers, so the order of the atomics does not matter).
// A bias list has few entries in a part (300 in 32 parts, say). The lanes that
// hold them work out those logits themselves and write them once the part has
// been written: of an id given twice the entry with the earlier place does, which
// each lane knows from the part's entries in LDS (their order there does not
// matter). A longer list, or more entries in one part, goes through a table of
// places instead, by an atomic maximum of the places from the end, in the words
// of the counts (a table of
// its own for every list cost a third of the waves of a compute unit: 93 us
// for 256 x 128003 logits with 300 entries a row, 63 without any).
// Bound by memory for a batch, by its round trips for one row: everything that
// does not wait for something else is asked for at the start.
template <class TI, class TO, bool HIST, bool BIAS>
__global__ void __launch_bounds__(kLanes) logits_kernel(LogitsParams p) {
  __shared__ uint32_t count[HIST || BIAS ? kPart : 1];   // bit 31: in the prompt; below: how often behind it
  __shared__ uint32_t listed[BIAS ? kListed : 1];        // bias entries of the part: entry << 16 | place
  __shared__ int n_listed;
  const int tid = threadIdx.x, row = blockIdx.y;
  const int v0 = blockIdx.x * kPart;
  const int n = p.vocab - v0 < kPart ? p.vocab - v0 : kPart;
  const TI* x = (const TI*)p.x + row * p.x_stride + v0;
  TO* out = (TO*)p.out + row * p.out_stride + v0;

  int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
  int prompt = 0, m = -1;
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (BIAS) {
    b0 = p.bias_start[row];
    b1 = p.bias_start[row + 1];
  }
  if (HIST) {
    h0 = p.hist_start[row];
    h1 = p.hist_start[row + 1];
    if (p.prompt_len) prompt = p.prompt_len[row];
    if (p.repetition) rep = p.repetition[row];
    if (p.frequency) freq = p.frequency[row];
    if (p.presence) pres = p.presence[row];
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
  const bool masked = (uint32_t)m < (uint32_t)p.n_masks;
  const uint32_t* mask = masked ? p.masks + m * p.mask_stride + (v0 >> 5) : nullptr;
  uint32_t allowed[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int at = (s * kLanes + tid) * kPer;
    allowed[s] = masked && at < n ? mask[at >> 5] >> (at & 31) : ~0u;
  }
  if (HIST || BIAS) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) *(sgemv_dev::dword4*)&count[(s * kLanes + tid) * kPer] = sgemv_dev::dword4{0, 0, 0, 0};
    if (BIAS && tid == 0) n_listed = 0;
    __syncthreads();
  }
  uint32_t mine[kShort];                                 // entries of the part that this lane holds; n or more: none
  float value[kShort], logit[kShort];
  uint32_t bit[kShort];
  bool table = false;
  if (BIAS) {
    b0 = clamp64(b0, p.n_bias);
    b1 = clamp64(b1, p.n_bias);
    table = b1 - b0 > kShort * kLanes;
#pragma unroll
    for (int k = 0; k < kShort; ++k) {
      const int64_t i = b0 + k * kLanes + tid;
      mine[k] = !table && i < b1 ? (uint32_t)p.bias_ids[i] - (uint32_t)v0 : ~0u;
    }
#pragma unroll
    for (int k = 0; k < kShort; ++k) {
      bit[k] = 1u;
      if (mine[k] < (uint32_t)n) {
        const int to = atomicAdd(&n_listed, 1);
        if (to < kListed) listed[to] = mine[k] << 16 | (uint32_t)(k * kLanes + tid);
        value[k] = p.bias_values[b0 + k * kLanes + tid];
        logit[k] = (float)x[mine[k]];
        if (masked) bit[k] = mask[mine[k] >> 5] >> (mine[k] & 31) & 1u;
      }
    }
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
  if (HIST || BIAS) __syncthreads();
  if (HIST) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const sgemv_dev::dword4 w = *(const sgemv_dev::dword4*)&count[(s * kLanes + tid) * kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) l[s][e] = penalised(l[s][e], w[e], rep, freq, pres);
    }
  }
  if (BIAS && (table || n_listed > kListed)) {
    table = true;
    __syncthreads();                                     // all counts have been read
#pragma unroll
    for (int s = 0; s < kSteps; ++s) *(sgemv_dev::dword4*)&count[(s * kLanes + tid) * kPer] = sgemv_dev::dword4{0, 0, 0, 0};
    __syncthreads();
    each_id(p.bias_ids, b0, b1, v0, n, [&](uint32_t v, int64_t i) { atomicMax(&count[v], (uint32_t)(b1 - i)); });
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const sgemv_dev::dword4 w = *(const sgemv_dev::dword4*)&count[(s * kLanes + tid) * kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (w[e]) l[s][e] += p.bias_values[b1 - w[e]];
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int at = (s * kLanes + tid) * kPer;
    if (at >= n) break;
#pragma unroll
    for (int e = 0; e < kPer; ++e) l[s][e] = allowed[s] >> e & 1u ? l[s][e] : -__builtin_inff();
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
  if (BIAS && !table && n_listed > 0) {
    // the part has been written, by every wave, before an entry is written again
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShort; ++k) {
      if (mine[k] >= (uint32_t)n) continue;
      bool first = true;
      const uint32_t me = mine[k] << 16 | (uint32_t)(k * kLanes + tid);
      for (int i = 0; i < n_listed; ++i) first &= listed[i] >> 16 != mine[k] || listed[i] >= me;
      if (!first) continue;
      float y = logit[k];
      if (HIST) y = penalised(y, count[mine[k]], rep, freq, pres);
      out[mine[k]] = (TO)(bit[k] ? y + value[k] : -__builtin_inff());
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
