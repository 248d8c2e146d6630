// The append of new tokens, with their rotary positions, to a cache in 8 bits.
//
// A block of B slots, a head and one of K and V share a power of two 2^e; with
// A the largest finite magnitude among the block's new values,
//   e(A) = the least e with A <= 448 2^e (448 is e4m3's largest), -96 <= e <= 120
//   e'   = e(A), or the larger of it and e where the block holds older tokens
//   new codes e4m3(x 2^-e'), older ones e4m3(c 2^(e - e')) where e' > e.
// A power of two, not A / 448: codes are floating-point numbers, which a power
// of two leaves alone, so a block's exponent may grow while tokens come in and
// older codes stay what they were (but for the smallest, which lose bits).
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;

namespace {

using sgemv_dev::SeqView;
using sgemv_dev::dword2;
using sgemv_dev::dword4;

constexpr int kMostLanes = 1024;              // of a workgroup: 256 columns and 128 new tokens
constexpr int kHold = 4;                     // tokens of a lane
constexpr int kLeast = 127 - 96, kMost = 127 + 120;

struct RowsView {
  uint16_t* p;
  int64_t token, head;
};
struct CodesView {
  uint8_t* p;
  int64_t page, slot, head;
};

struct Append8Params {
  SeqView seq;
  RowsView q, q_out, k, v;
  CodesView kc, vc;
  uint8_t* scales;
  const double* turns;                       // [rot / 2], or null: nothing is rotated
  const int32_t* positions;                  // [tokens], or null: a token's slot
  float magnitude;
  int32_t nq, nkv, chunks;                   // heads; 8-column chunks of a head
  int32_t rot, interleaved;
  int32_t block_shift;                       // log2 of B
  int32_t sines;                             // angles that a block may need
  int32_t lanes, per, groups;                // of a workgroup: lanes, heads; lanes that share a head's tokens
};

template <class T>
__device__ __forceinline__ float to_f(uint16_t u) { return (float)__builtin_bit_cast(T, u); }
template <class T>
__device__ __forceinline__ uint16_t from_f(float f) { return __builtin_bit_cast(uint16_t, (T)f); }

// The biased exponent that A, as the bits of a float, needs.
__device__ __forceinline__ int exponent_of(uint32_t a) {
  // A = f 2^x with f in [1, 2): 448 = 1.75 2^8. Subnormal A are below all of it.
  const int e = (int)(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u);
  return e < kLeast ? kLeast : e > kMost ? kMost : e;
}

// 8 values as codes of the biased exponent e. `odd`: some are not finite.
__device__ __forceinline__ dword2 codes_of(const float (&v)[8], int e, bool odd) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __builtin_amdgcn_ldexpf(v[4 * i + k], 127 - e);
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    u = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], u, true);
    if (odd) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!(__builtin_fabsf(v[4 * i + k]) < __builtin_inff())) u = (u & ~(0xff << 8 * k)) | 0x7f << 8 * k;
    }
    w[i] = (uint32_t)u;
  }
  return dword2{w[0], w[1]};
}

// How a chunk of 8 columns finds the others of its pairs: in a chunk of its own
// (halves of a multiple of 8 columns), within itself (interleaved, in whole
// chunks), or column by column.
enum Pairing { kApart, kWithin, kAnyhow };

// Workgroup (u, y): block u of those that new tokens fall into, heads y per ...
// of the list q0 .. q(nq-1), k0 .. k(nkv-1), v0 .. v(nkv-1); q goes along, its
// tokens being those of the block's slots. A lane has one chunk of 8 columns of
// one head in up to 4 of the block's tokens, from the load to the store, so
// that every row is read once: the values stay in registers while the block's
// largest magnitude is found in LDS. A rotated chunk reads its partner's columns
// beside its own (from the same cache lines as the lane that has them).
// Bound by memory: a batch of 5 prompts of up to 4001 tokens, 96 heads of 128
// columns, blocks of 16, takes 150 us at 3.8 TB/s of the rows read and written
// (copies reach 4.7 to 4.9). 16 single tokens: 5.0 us, the launch and two round
// trips (a sequence's lengths and page, then its rows). The rows' loads are asked
// for before the sines are worked out, which then cost nothing up to blocks of
// 32; larger ones (64: 237 us, 128: 264) work out more of them in each workgroup
// for fewer heads, and a rotated width whose halves are no whole chunks goes
// column by column (40 of 128: 190).
//
// Blocks are numbered without a pass over the sequences: sequence s, whose
// first new token is a, has the numbers from floor(a / B) + 2 s on; n tokens fall
// into at most floor(n / B) + 2 blocks. What is left over is empty.
template <class T, Pairing PAIRING>
__global__ void __launch_bounds__(kMostLanes) append8_kernel(Append8Params p) {
  extern __shared__ float2 trig[];                         // [token of the block][pair], then
  uint32_t* top = (uint32_t*)(trig + p.sines);             // [head] the largest magnitude
  const int tid = threadIdx.x, unit = blockIdx.x;
  const SeqView& sq = p.seq;
  int s, a, b, ctx;
  const auto base = [&](int start, int i) { return (start >> p.block_shift) + 2 * i; };
  if (sq.count <= 64) {
    const int lane = tid & 63, i = lane < sq.count ? lane : sq.count - 1;
    const int from = sq.start(i), to = sq.start(i + 1), all = sq.ctx(i);
    const int holds = __popcll(__ballot(lane < sq.count && base(from, i) <= unit));
    s = holds < 1 ? 0 : holds - 1;
    a = __builtin_amdgcn_readlane(from, s);
    b = __builtin_amdgcn_readlane(to, s);
    ctx = __builtin_amdgcn_readlane(all, s);
  } else {
    s = sgemv_dev::wave_upper(sq.count, unit, [&](int i) { return base(sq.start(i), i); });
    a = sq.start(s);
    b = sq.start(s + 1);
    ctx = sq.ctx(s);
  }
  const int skip = unit - base(a, s), B = 1 << p.block_shift;
  if (b <= a || skip < 0) return;
  const int first_slot = ctx - (b - a);                    // below 0 where the sequence is shorter than its new tokens
  const int block = (first_slot >> p.block_shift) + skip;
  if ((int64_t)block * B >= ctx) return;
  const int start = block * B;
  const int lo = first_slot > start ? first_slot : start, hi = ctx < start + B ? ctx : start + B;
  const int n = hi - lo, tok0 = a + (lo - first_slot), older = lo - start;
  int page = -1;
  if (block >= 0) page = sq.pages[s * sq.pages_stride + (start >> sq.page_shift)];
  const bool store = block >= 0 && sq.page_ok(page);

  const int chunk = tid % p.chunks, rest = tid / p.chunks, mine = rest % p.per, group = rest / p.per, first = chunk * 8;
  const int h = blockIdx.y * p.per + mine;
  const bool in = group < p.groups && h < p.nq + 2 * p.nkv;
  const bool is_q = in && h < p.nq, is_k = in && !is_q && h < p.nq + p.nkv, is_v = in && h >= p.nq + p.nkv;
  const int hh = is_q ? h : is_k ? h - p.nq : is_v ? h - p.nq - p.nkv : 0;
  const int pairs = p.rot / 2;
  const bool turned = (is_q || is_k) && first < p.rot;
  const bool work = is_q || (in && store);

  float x[kHold][8];
  {
    const RowsView& src = is_q ? p.q : is_k ? p.k : p.v;
    const uint16_t* from = src.p + hh * src.head;
    const int partner = first < pairs ? first + pairs : first - pairs;
    dword4 own[kHold], other[PAIRING == kWithin ? 1 : kHold];
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int at = j * p.groups + group;
      own[j] = dword4{0, 0, 0, 0};
      if (PAIRING != kWithin) other[j] = dword4{0, 0, 0, 0};
      if (j * p.groups >= n) break;
      if (!work || at >= n) continue;
      const uint16_t* row = from + (int64_t)(tok0 + at) * src.token;
      own[j] = *(const dword4*)(row + first);
      if (PAIRING == kApart && turned) other[j] = *(const dword4*)(row + partner);
      if (PAIRING == kAnyhow && turned) {
        uint16_t y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = first + e;
          y[e] = d < p.rot ? row[p.interleaved ? d ^ 1 : d < pairs ? d + pairs : d - pairs] : 0;
        }
        other[j] = *(const dword4*)y;
      }
    }
    if (p.rot > 0 && tid < p.lanes / pairs * pairs) {
      const int j = tid % pairs;
      const double turns = p.turns[j];
      for (int at = tid / pairs; at < n; at += p.lanes / pairs) {
        const int pos = p.positions ? p.positions[tok0 + at] : lo + at;
        const double rev = (double)pos * turns;
        float sn, cs;
        sincospif(2.0f * (float)(rev - rint(rev)), &sn, &cs);
        trig[at * pairs + j] = float2{cs * p.magnitude, sn * p.magnitude};
      }
    }
    top[tid] = 0;
    // every row has been read, by every lane, before any is written (q_out may be q)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const bool low = first < pairs;                        // kApart: of the whole chunk
    const float sign = low ? -1.0f : 1.0f;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int at = j * p.groups + group;
      if (j * p.groups >= n) break;
      uint16_t u[8], w[8];
      *(dword4*)u = own[j];
      if (PAIRING != kWithin) *(dword4*)w = other[j];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = to_f<T>(u[e]);
      if (!turned || at >= n) continue;
      const float2* t = trig + at * pairs;
      if (PAIRING == kApart) {
        t += low ? first : first - pairs;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 c = t[e];
          x[j][e] = x[j][e] * c.x + to_f<T>(w[e]) * (sign * c.y);
        }
      } else if (PAIRING == kWithin) {
        t += first / 2;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 c = t[e / 2];
          const float a0 = x[j][e], b0 = x[j][e + 1];
          x[j][e] = a0 * c.x - b0 * c.y;
          x[j][e + 1] = b0 * c.x + a0 * c.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = first + e;
          if (d >= p.rot) continue;
          const bool one = p.interleaved ? !(d & 1) : d < pairs;
          const float2 c = t[p.interleaved ? d >> 1 : one ? d : d - pairs];
          x[j][e] = x[j][e] * c.x + to_f<T>(w[e]) * (one ? -c.y : c.y);
        }
      }
    }
  }

  if (is_q) {
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int at = j * p.groups + group;
      if (j * p.groups >= n) break;
      if (at >= n) continue;
      uint16_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = from_f<T>(x[j][e]);
      *(dword4*)(p.q_out.p + (int64_t)(tok0 + at) * p.q_out.token + hh * p.q_out.head + first) = *(const dword4*)y;
    }
  }

  const int64_t in_page = start & ((1 << sq.page_shift) - 1);
  const int64_t blocks_of_page = (int64_t)1 << (sq.page_shift - p.block_shift);
  uint8_t* scale = p.scales + ((page * blocks_of_page + (in_page >> p.block_shift)) * p.nkv + hh) * 2 + is_v;
  const bool write = (is_k || is_v) && store;
  int was = 0;
  if (write && older) was = *scale;
  bool odd = false;                                        // some of the lane's values are not finite
  if (write) {
    float most = 0.0f, none = 0.0f;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      if (j * p.groups >= n) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        most = fmaxf(most, __builtin_fabsf(x[j][e]));
        none = __builtin_fmaf(x[j][e], 0.0f, none);        // not a number after one that is not finite
      }
    }
    odd = none != 0.0f;
    if (odd) {
      most = 0.0f;
#pragma unroll
      for (int j = 0; j < kHold; ++j) {
        if (j * p.groups >= n) break;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (__builtin_fabsf(x[j][e]) < __builtin_inff()) most = fmaxf(most, __builtin_fabsf(x[j][e]));
      }
    }
    atomicMax(&top[mine], __builtin_bit_cast(uint32_t, most));
  }
  // `was` has been read, by every lane, before it is written
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (!write) return;
  int e = exponent_of(top[mine]);
  if (older && was > e) e = was;
  const CodesView& to = is_k ? p.kc : p.vc;
  uint8_t* row0 = to.p + page * to.page + in_page * to.slot + hh * to.head + first;
  if (older && e > was) {
    const int by = was - e;
    for (int r = group; r < older; r += p.groups) {
      uint8_t* row = row0 + r * to.slot;
      const dword2 c = *(const dword2*)row;
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto f0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), f1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_ldexpf(f0[0], by), __builtin_amdgcn_ldexpf(f0[1], by), 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_ldexpf(f1[0], by), __builtin_amdgcn_ldexpf(f1[1], by), u, true);
      }
      *(dword2*)row = dword2{w[0], w[1]};
    }
  }
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int at = j * p.groups + group;
    if (j * p.groups >= n) break;
    if (at >= n) continue;
    *(dword2*)(row0 + (older + at) * to.slot) = codes_of(x[j], e, odd);
  }
  if (group == 0 && chunk == 0) *scale = (uint8_t)e;
}

typedef void (*Append8Fn)(Append8Params);
template <class T>
Append8Fn pick(Pairing pairing) {
  return pairing == kApart ? append8_kernel<T, kApart> : pairing == kWithin ? append8_kernel<T, kWithin> : append8_kernel<T, kAnyhow>;
}

int check_rope(const sgemv_rope_t* r, int dim) {
  if (r->rot_dim < 2 || r->rot_dim > dim || r->rot_dim % 2 || !r->turns) return SGEMV_EINVAL;
  if (r->interleaved != 0 && r->interleaved != 1) return SGEMV_EINVAL;
  if (!(r->magnitude > 0.0f) || r->magnitude > 3.0e38f) return SGEMV_EINVAL;
  return (uintptr_t)r->turns % 8 ? SGEMV_EALIGN : SGEMV_OK;
}

RowsView view(const sgemv_rows* r) { return RowsView{(uint16_t*)r->data, r->tokens > 1 ? r->token_stride : 0, r->heads > 1 ? r->head_stride : 0}; }

}  // namespace

extern "C" int sgemv_append8(const sgemv_cache8* cache, const sgemv_seqs* seqs, const sgemv_rope_t* rope, const int32_t* positions_dev,
                             const sgemv_rows* q, const sgemv_rows* q_out, const sgemv_rows* k, const sgemv_rows* v, void* hip_stream) {
  if (!k || !v || !q != !q_out || (q && !rope)) return SGEMV_EINVAL;
  int rc = check_cache8(cache, true);
  if (rc) return rc;
  rc = check_seqs(seqs);
  if (rc) return rc;
  for (const sgemv_rows* r : {k, v}) {
    rc = check_rows(r, false);
    if (rc) return rc;
    if (r->tokens != k->tokens || r->heads != cache->heads || r->head_dim != cache->head_dim || r->dtype != k->dtype) return SGEMV_EINVAL;
  }
  if (q) {
    rc = check_rows(q, false);
    if (rc) return rc;
    rc = check_rows(q_out, true);
    if (rc) return rc;
    for (const sgemv_rows* r : {q, q_out})
      if (r->tokens != k->tokens || r->heads != q->heads || r->head_dim != k->head_dim || r->dtype != k->dtype) return SGEMV_EINVAL;
  }
  if (rope) {
    rc = check_rope(rope, k->head_dim);
    if (rc) return rc;
  }
  if ((uintptr_t)positions_dev % 4) return SGEMV_EALIGN;
  if (k->tokens >= (1 << 24)) return SGEMV_ESIZE;
  if (seqs->count == 0 || k->tokens == 0) return SGEMV_OK;
  Append8Params p;
  memset(&p, 0, sizeof p);
  p.seq = seq_view(seqs, cache, k->tokens);
  if (q) {
    p.q = view(q);
    p.q_out = view(q_out);
    p.nq = q->heads;
  }
  p.k = view(k);
  p.v = view(v);
  p.nkv = k->heads;
  p.kc = CodesView{(uint8_t*)cache->k, cache->pages > 1 ? cache->k_page : 0, cache->k_slot, cache->heads > 1 ? cache->k_head : 0};
  p.vc = CodesView{(uint8_t*)cache->v, cache->pages > 1 ? cache->v_page : 0, cache->v_slot, cache->heads > 1 ? cache->v_head : 0};
  p.scales = cache->scales;
  p.positions = positions_dev;
  if (rope) {
    p.turns = rope->turns;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.magnitude = rope->magnitude;
  }
  const int B = cache->scale_slots;
  p.block_shift = ilog2(B);
  p.chunks = k->head_dim / 8;
  const int most = B < k->tokens ? B : k->tokens;                // new tokens of a block
  p.groups = (most + kHold - 1) / kHold;
  // four waves, or as many as a head takes (a batch of prompts of up to 4001
  // tokens, 96 heads of 128 columns, blocks of 16: 149 us with 4 tokens a lane and
  // 4 waves, 164 with 8 waves; 179 with 2 tokens; 191 with 8, 184 of them and 8 waves;
  // 16 waves for blocks of more than 16: 32 slots 157 -> 166, 64 and 128 within 1 %.
  // Sines of a quarter of the block at a time take less LDS, but a barrier each:
  // 64 slots 237 -> 199, 16 of them 150 -> 162)
  p.lanes = p.chunks * p.groups > 256 ? (p.chunks * p.groups + 63) / 64 * 64 : 256;
  p.per = p.lanes / p.chunks / p.groups;
  const int64_t units = (k->tokens >> p.block_shift) + 2 * (int64_t)seqs->count;
  const int heads = p.nq + 2 * p.nkv;
  if (units * p.lanes > (int64_t)UINT32_MAX) return SGEMV_ESIZE;  // lanes of a grid axis fit 32 bits
  p.sines = most * (p.rot / 2);
  const int64_t lds = (int64_t)p.sines * 8 + p.lanes * 4;
  const Pairing pairing = !rope || (!rope->interleaved && rope->rot_dim % 16 == 0) ? kApart
                          : rope->interleaved && rope->rot_dim % 8 == 0          ? kWithin
                                                                                 : kAnyhow;
  const Append8Fn fn = k->dtype == SGEMV_F16 ? pick<_Float16>(pairing) : pick<__bf16>(pairing);
  (void)hipGetLastError();
  if (ensure_lds((const void*)fn, lds)) return SGEMV_EHIP;
  const dim3 grid((uint32_t)units, (uint32_t)((heads + p.per - 1) / p.per));
  hipLaunchKernelGGL(fn, grid, dim3(p.lanes), (uint32_t)lds, (hipStream_t)hip_stream, p);
  return hipGetLastError() == hipSuccess ? SGEMV_OK : SGEMV_EHIP;
}
