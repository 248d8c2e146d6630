// Rotary positions, and the append of new tokens to a paged cache.
//
// A pair (a, b) of a head's rotated columns at position pos turns by
// theta = 2 pi pos f_j:  (a, b) <- m (a cos - b sin, a sin + b cos).
// The frequencies f_j come in turns per position and 64 bits: pos f_j minus
// the nearest whole number is the angle left over, to 2^-53 of pos f_j turns,
// so a position of a million is as exact as position one (in 32 bits its
// angle would be off by up to 0.03 of a turn). Only the fraction goes to 32
// bits, for the sine, the cosine and the products; q and k are rounded once.
#include "decode_internal.hpp"

using namespace sgemv;

namespace {

using sgemv_dev::SeqView;
using sgemv_dev::dword4;

constexpr int kLanes = 256;
constexpr int kMaxPairs = 128;   // head_dim <= 256

struct RowsView {
  uint16_t* p;
  int64_t token, head;
};

struct RopeParams {
  SeqView seq;
  RowsView q, q_out, k, v;       // q: heads to rotate into q_out; k, v: heads for the cache
  RowsView kc, vc;               // cache: token = slot stride
  int64_t k_page, v_page;
  const double* turns;           // [rot / 2], or null: nothing is rotated
  const int32_t* positions;      // [tokens], or null: a token's slot
  float magnitude;
  int32_t nq, nkv, chunks;       // heads; 8-column chunks of a head
  int32_t rot, interleaved;
  int32_t per_pass, passes;      // heads per pass of the workgroup, passes per workgroup
};

template <class T>
__device__ __forceinline__ float to_f(uint16_t u) { return (float)__builtin_bit_cast(T, u); }
template <class T>
__device__ __forceinline__ uint16_t from_f(float f) { return __builtin_bit_cast(uint16_t, (T)f); }

// Workgroup (t, y): token t, passes y * passes ... of the head list
// q0 .. q(nq-1), k0 .. k(nkv-1), v0 .. v(nkv-1). In a pass each lane holds one
// 16-byte chunk of one head; a rotated chunk finds its partners in LDS, where
// the pass's heads are staged, so any even `rot` and both pairings go the same
// way and q_out may be q itself (all of a pass is read before it is written).
// Bound by memory, one token by the round trips to it: the rows do not wait
// for the token's sequence, and of up to 64 sequences every lane reads one's
// lengths, so the page is the second round trip and the stores follow it. The
// sines of a token are computed once per workgroup, meanwhile.
template <class T>
__global__ void __launch_bounds__(kLanes) rope_kernel(RopeParams p) {
  __shared__ float cs[kMaxPairs], sn[kMaxPairs];
  __shared__ __attribute__((aligned(16))) uint16_t stage[2][kLanes * 8];
  const int tok = blockIdx.x, tid = threadIdx.x;
  const int mine = tid / p.chunks, chunk = tid - mine * p.chunks, first = chunk * 8;
  const int heads = p.nq + 2 * p.nkv, head0 = blockIdx.y * p.passes * p.per_pass + mine;
  const auto fetch = [&](int h) {
    dword4 x = {0, 0, 0, 0};
    if (mine < p.per_pass && h < heads) {
      const bool is_q = h < p.nq, is_k = h < p.nq + p.nkv;
      const RowsView& src = is_q ? p.q : is_k ? p.k : p.v;
      x = *(const dword4*)(src.p + tok * src.token + (is_q ? h : is_k ? h - p.nq : h - p.nq - p.nkv) * src.head + first);
    }
    return x;
  };
  dword4 next = fetch(head0);
  const int pairs = p.rot / 2;
  const double turns = tid < pairs ? p.turns[tid] : 0.0;

  int pos = 0, slot = -1, page = -1;
  if (p.positions) pos = p.positions[tok];
  if (p.nkv > 0) {
    const SeqView& q = p.seq;
    int s, a, b, ctx;
    if (q.count <= 64) {
      const int lane = tid & 63, i = lane < q.count ? lane : q.count - 1;
      const int from = q.start(i), to = q.start(i + 1), all = q.ctx(i);
      const int holds = __popcll(__ballot(lane < q.count && from <= tok));
      s = holds < 1 ? 0 : holds - 1;
      a = __builtin_amdgcn_readlane(from, s);
      b = __builtin_amdgcn_readlane(to, s);
      ctx = __builtin_amdgcn_readlane(all, s);
    } else {
      s = sgemv_dev::wave_upper(q.count, tok, [&](int i) { return q.start(i); });
      a = q.start(s);
      b = q.start(s + 1);
      ctx = q.ctx(s);
    }
    if (tok < a || tok >= b) return;                       // of no sequence
    slot = ctx - (b - tok);
    if (slot >= 0) page = q.pages[s * q.pages_stride + (slot >> q.page_shift)];
    if (!p.positions) pos = slot;
  }
  if (tid < pairs) {
    const double rev = (double)pos * turns;
    const float frac = (float)(rev - rint(rev));
    float s, c;
    sincospif(2.0f * frac, &s, &c);
    cs[tid] = c * p.magnitude;
    sn[tid] = s * p.magnitude;
  }
  const bool store = slot >= 0 && p.seq.page_ok(page);
  const int64_t in_page = slot & ((1 << p.seq.page_shift) - 1);
  for (int pass = 0; pass < p.passes; ++pass) {
    const int h = head0 + pass * p.per_pass;
    dword4 x = next;
    uint16_t* part = stage[pass & 1];
    *(dword4*)(part + tid * 8) = x;
    if (pass + 1 < p.passes) next = fetch(h + p.per_pass);
    __syncthreads();                                       // two parts: nobody still reads the one written next
    const bool is_q = h < p.nq, is_k = !is_q && h < p.nq + p.nkv;
    if (mine >= p.per_pass || h >= heads || (!is_q && !store)) continue;
    if ((is_q || is_k) && first < p.rot) {
      const uint16_t* head = part + (tid - chunk) * 8;
      uint16_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = first + e;
        y[e] = head[d];
        if (d < p.rot) {
          const bool low = p.interleaved ? !(d & 1) : d < pairs;
          const int j = p.interleaved ? d >> 1 : low ? d : d - pairs;
          const int other = p.interleaved ? d ^ 1 : low ? d + pairs : d - pairs;
          const float u = to_f<T>(y[e]), w = to_f<T>(head[other]);
          y[e] = from_f<T>(low ? u * cs[j] - w * sn[j] : w * sn[j] + u * cs[j]);
        }
      }
      x = *(const dword4*)y;
    }
    const int hh = is_q ? h : is_k ? h - p.nq : h - p.nq - p.nkv;
    uint16_t* dst = is_q ? p.q_out.p + tok * p.q_out.token + hh * p.q_out.head
                         : is_k ? p.kc.p + page * p.k_page + in_page * p.kc.token + hh * p.kc.head
                                : p.vc.p + page * p.v_page + in_page * p.vc.token + hh * p.vc.head;
    *(dword4*)(dst + first) = x;
  }
}

int launch(RopeParams& p, int tokens, int dim, int dtype, void* stream) {
  if (tokens == 0 || p.nq + 2 * p.nkv == 0) return SGEMV_OK;
  p.chunks = dim / 8;
  p.per_pass = kLanes / p.chunks;
  const int all = (p.nq + 2 * p.nkv + p.per_pass - 1) / p.per_pass;
  // few tokens: a workgroup for each pass, for the latency of one; many: one
  // workgroup a token, so that its sines are computed once (32 heads of q, k and
  // v; as many workgroups as there are passes, or one a token: 16 tokens 4.4 and
  // 10.3 us, 512 tokens 10.7 and 12.6, 9.6 in between, 4096 tokens 59 and 44)
  int groups = all;
  while (groups > 1 && (int64_t)groups * tokens > 2048) groups = (groups + 1) / 2;
  p.passes = (all + groups - 1) / groups;
  groups = (all + p.passes - 1) / p.passes;
  if (tokens >= (1 << 24)) return SGEMV_ESIZE;   // lanes of a grid axis fit 32 bits
  (void)hipGetLastError();
  const dim3 grid((uint32_t)tokens, (uint32_t)groups);
  if (dtype == SGEMV_F16) hipLaunchKernelGGL(rope_kernel<_Float16>, grid, dim3(kLanes), 0, (hipStream_t)stream, p);
  else hipLaunchKernelGGL(rope_kernel<__bf16>, grid, dim3(kLanes), 0, (hipStream_t)stream, p);
  return hipGetLastError() == hipSuccess ? SGEMV_OK : SGEMV_EHIP;
}

RowsView view(const sgemv_rows* r) { return RowsView{(uint16_t*)r->data, r->tokens > 1 ? r->token_stride : 0, r->heads > 1 ? r->head_stride : 0}; }

int check_rope(const sgemv_rope_t* r, int dim) {
  if (r->rot_dim < 2 || r->rot_dim > dim || r->rot_dim % 2 || !r->turns) return SGEMV_EINVAL;
  if (r->interleaved != 0 && r->interleaved != 1) return SGEMV_EINVAL;
  if (!(r->magnitude > 0.0f) || r->magnitude > 3.0e38f) return SGEMV_EINVAL;
  return (uintptr_t)r->turns % 8 ? SGEMV_EALIGN : SGEMV_OK;
}

void set_rope(RopeParams& p, const sgemv_rope_t* r) {
  p.turns = r->turns;
  p.rot = r->rot_dim;
  p.interleaved = r->interleaved;
  p.magnitude = r->magnitude;
}

// Both of q and q_out, equal in shape.
int check_pair(const sgemv_rows* a, const sgemv_rows* b) {
  int rc = check_rows(a, false);
  if (rc) return rc;
  rc = check_rows(b, true);
  if (rc) return rc;
  return a->tokens != b->tokens || a->heads != b->heads || a->head_dim != b->head_dim || a->dtype != b->dtype ? SGEMV_EINVAL : SGEMV_OK;
}

}  // namespace

extern "C" int sgemv_rope(const sgemv_rope_t* rope, const int32_t* positions_dev, const sgemv_rows* x, const sgemv_rows* out,
                          void* hip_stream) {
  if (!rope || !x || !out) return SGEMV_EINVAL;
  int rc = check_pair(x, out);
  if (rc) return rc;
  rc = check_rope(rope, x->head_dim);
  if (rc) return rc;
  if (x->tokens > 0 && !positions_dev) return SGEMV_EINVAL;
  if ((uintptr_t)positions_dev % 4) return SGEMV_EALIGN;
  RopeParams p;
  memset(&p, 0, sizeof p);
  p.q = view(x);
  p.q_out = view(out);
  p.nq = x->heads;
  p.positions = positions_dev;
  set_rope(p, rope);
  return launch(p, x->tokens, x->head_dim, x->dtype, hip_stream);
}

extern "C" int sgemv_append(const sgemv_cache* cache, const sgemv_seqs* seqs, const sgemv_rope_t* rope, const int32_t* positions_dev,
                            const sgemv_rows* q, const sgemv_rows* q_out, const sgemv_rows* k, const sgemv_rows* v, void* hip_stream) {
  if (!k || !v || !q != !q_out || (q && !rope)) return SGEMV_EINVAL;
  int rc = check_cache(cache, true);
  if (rc) return rc;
  rc = check_seqs(seqs);
  if (rc) return rc;
  for (const sgemv_rows* r : {k, v}) {
    rc = check_rows(r, false);
    if (rc) return rc;
    if (r->tokens != k->tokens || r->heads != cache->heads || r->head_dim != cache->head_dim || r->dtype != cache->dtype) return SGEMV_EINVAL;
  }
  if (q) {
    rc = check_pair(q, q_out);
    if (rc) return rc;
    if (q->tokens != k->tokens || q->head_dim != k->head_dim || q->dtype != k->dtype) return SGEMV_EINVAL;
  }
  if (rope) {
    rc = check_rope(rope, k->head_dim);
    if (rc) return rc;
  }
  if ((uintptr_t)positions_dev % 4) return SGEMV_EALIGN;
  if (seqs->count == 0) return SGEMV_OK;
  RopeParams p;
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
  p.kc = RowsView{(uint16_t*)cache->k, cache->k_slot, cache->heads > 1 ? cache->k_head : 0};
  p.vc = RowsView{(uint16_t*)cache->v, cache->v_slot, cache->heads > 1 ? cache->v_head : 0};
  p.k_page = cache->pages > 1 ? cache->k_page : 0;
  p.v_page = cache->pages > 1 ? cache->v_page : 0;
  p.positions = positions_dev;
  if (rope) set_rope(p, rope);
  return launch(p, k->tokens, k->head_dim, k->dtype, hip_stream);
}
