// sgemv_attend, sgemv_attend_window, sgemv_attend8 and their plans: host checks
// and the launches of the attention.
#include "attend_few.hpp"
#include "attend_join.hpp"
#include "attend_kernels.hpp"
#include "attend_many.hpp"
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;
using sgemv_dev::AttendFn;
using sgemv_dev::AttendParams;

namespace {

constexpr int kCus = 256;
using sgemv_dev::kMaxSplits;

// A cache of either kind and how it is looked at. Strides are of elements: two
// bytes each, or one in 8 bits.
struct Cache {
  const void *k, *v;
  const int64_t *k_stride, *v_stride;   // page, slot, head
  int pages, page_size, heads, head_dim;
  const void* exps;                     // in 8 bits
  int dtype, scale_slots;               // of 16 bits; in 8 bits
  int window, sinks;                    // 0: all that is before a token
};

constexpr int kMostSlots = 1 << 30;     // a window of more is one of all slots

int look(const sgemv_cache* c, int32_t window, int32_t sinks, Cache* out) {
  const int rc = check_cache(c, false);
  if (rc) return rc;
  *out = Cache{c->k, c->v, &c->k_page, &c->v_page, c->pages, c->page_size, c->heads, c->head_dim, nullptr, c->dtype, 0,
               window < kMostSlots ? window : kMostSlots, sinks < kMostSlots ? sinks : kMostSlots};
  return SGEMV_OK;
}

int look(const sgemv_cache8* c, int32_t window, int32_t sinks, Cache* out) {
  const int rc = check_cache8(c, false);
  if (rc) return rc;
  *out = Cache{c->k, c->v, &c->k_page, &c->v_page, c->pages, c->page_size, c->heads, c->head_dim, c->scales, -1, c->scale_slots,
               window < kMostSlots ? window : kMostSlots, sinks < kMostSlots ? sinks : kMostSlots};
  return SGEMV_OK;
}

struct Shape {
  bool few, halves;
  int dp, tile_rows, block, waves, splits;
  int64_t lds, slots, grid, workspace;
};

// Which kernel, and in how many parts the context is split: from the sizes on
// the host alone. Lengths in device memory never change what is launched.
int make_shape(const Cache* c, const sgemv_seqs* s, int32_t tokens, int32_t heads, int32_t max_ctx, Shape* out) {
  const int group = heads / c->heads;
  Shape h;
  h.dp = c->head_dim <= 64 ? 64 : c->head_dim <= 128 ? 128 : 256;
  const int64_t rows = (int64_t)tokens * group;
  int64_t ctx = (int64_t)s->pages_per_seq * c->page_size;
  if (max_ctx > 0 && max_ctx < ctx) ctx = max_ctx;
  // through a window the keys of a sequence's tiles: the sinks, the window and a
  // slot for each further token, however long the context
  if (c->window > 0 && (int64_t)c->sinks + c->window + tokens / s->count < ctx) ctx = (int64_t)c->sinks + c->window + tokens / s->count;
  // Up to 16 rows a sequence on average: a tile of 16 that reads K and V
  // straight from memory (12 rows, 4 sequences of up to 6000 slots, 8 heads:
  // 20.5 us, 25.5 as a tile of 128). Up to 128 rows the same, a few tiles each
  // for itself, over short contexts, where the larger kernel's start and end
  // weigh more (96 rows over 300 slots: 9.7 against 15.2 us, over 6000: 61.6
  // against 31.9; 48 rows: 11.9 against 13.6, and 39.5 against 27.8). In 8 bits
  // the tiles read half as much and the larger kernel converts on top: up to 4096
  // (4 x 108 rows, 8 heads, over 2000 slots: 19.4 against 30.9 us, over 4000: 31.9
  // against 33.3; 1 x 128 rows over 4000: 16.9 against 26.5). Through a window in
  // 16 bits up to 2048 (4 x 96 rows, a window of 1000: 16.1 against 24.3, of 2000:
  // 25.8 against 25.5, of 3000: 35.3 against 27.7; 1 x 128, of 2000: 15.8, 22.5).
  // All these leave compute units without work. Where sequences and heads fill the
  // chip tiles of 16 rows stay ahead over 8 bits up to 32 rows (16 and 64 sequences,
  // 32 heads, 2000 slots: 85 against 106 us, 387 against 424) but not with 108, whose
  // keys they read and convert seven times (4, 16 and 64 sequences: 73 against 49,
  // 264 against 129, 1044 against 525; 64 over 500: 505 against 216): the rule does
  // not look at that.
  const int64_t near = c->exps ? 4096 : c->window > 0 ? 2048 : 1024;
  h.few = rows <= (int64_t)16 * s->count || (rows <= (int64_t)128 * s->count && ctx <= near);
  h.waves = !h.few ? sgemv_dev::kManyWaves : h.dp == 256 ? sgemv_dev::kFewWaves<256> : sgemv_dev::kFewWaves<128>;
  h.halves = !h.few && h.dp < 256 && rows <= (int64_t)128 * s->count;
  h.tile_rows = h.few ? 16 : h.halves ? sgemv_dev::kManyRows<true> : sgemv_dev::kManyRows<false>;
  h.block = h.few || h.dp == 256 ? 32 : 64;
  h.lds = h.few ? 0 : h.dp == 64 ? sgemv_dev::kManyLds<64> : h.dp == 128 ? sgemv_dev::kManyLds<128> : sgemv_dev::kManyLds<256>;
  h.slots = rows / h.tile_rows + s->count;
  int64_t tiles = (rows + h.tile_rows - 1) / h.tile_rows;
  const int64_t each = s->count < tokens ? s->count : tokens;
  tiles = tiles < each ? each : tiles;
  // Workgroups to aim for: one a compute unit, as a workgroup has eight waves
  // and up to 128 KiB of LDS; two of the 64-column kernel fit (chunks of 777
  // over 9001 and 440 over 4550: 71 us, 76 with one). More parts than that
  // only add to what is joined (131071 slots, 8 heads: 100 us with 256, 102
  // with 512, 107 with 1024). A part has two blocks at least in the few-row
  // kernel (700 slots, 32 heads: 10.0 us with parts of 64, 11.0 of 128, 12.8
  // of 256), four in the other (8 heads, 27 rows over 1500 slots: 15.4 us with
  // parts of 256, 14.0 of 128, 22.2 of 512; 300 rows over 2000: 27.9, 28.3 and
  // 32.1; 64 tokens of 32 heads sharing 8 over 4000: 30.4, 28.9 and 32.2).
  const int64_t want = (!h.few && h.dp == 64 ? 2 : 1) * kCus / (tiles * c->heads);
  const int64_t most = ctx / (h.few ? 64 : 256);
  int64_t splits = want < most ? want : most;
  splits = splits < 1 ? 1 : splits > kMaxSplits ? kMaxSplits : splits;
  h.splits = (int)splits;
  h.workspace = splits > 1 ? (int64_t)tokens * heads * splits * (c->head_dim + 2) * 4 : 0;
  h.grid = h.slots * c->heads * splits;
  if (h.grid * h.waves * 64 > (int64_t)UINT32_MAX) return SGEMV_ESIZE;   // lanes of a grid axis fit 32 bits
  if (splits > 1 && (int64_t)tokens * heads * 256 > (int64_t)UINT32_MAX) return SGEMV_ESIZE;
  *out = h;
  return SGEMV_OK;
}

int check(const Cache* c, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx) {
  const int rc = check_seqs(seqs);
  if (rc) return rc;
  // the kernels' page and slot strides, and eight slots' bytes, fit 32 bits
  for (const int64_t* d : {c->k_stride, c->v_stride})
    if ((c->pages > 1 && d[0] > INT32_MAX) || d[1] > INT32_MAX / 16) return SGEMV_ESIZE;
  if (tokens < 0 || heads < 1 || heads > 65535 || heads % c->heads || max_ctx < 0) return SGEMV_EINVAL;
  return (int64_t)tokens * heads > (1 << 30) ? SGEMV_ESIZE : SGEMV_OK;
}

int plan(const Cache* c, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx, sgemv_attend_plan_t* out) {
  const int rc = check(c, seqs, tokens, heads, max_ctx);
  if (rc) return rc;
  sgemv_attend_plan_t q;
  memset(&q, 0, sizeof q);
  if (tokens > 0 && seqs->count > 0) {
    Shape h;
    const int rs = make_shape(c, seqs, tokens, heads, max_ctx, &h);
    if (rs) return rs;
    q.workspace_bytes = h.workspace;
    q.grid = h.grid;
    q.lds_bytes = h.lds;
    q.block = 64 * h.waves;
    q.tile_rows = h.tile_rows;
    q.block_keys = h.block;
    q.splits = h.splits;
  }
  *out = q;
  return SGEMV_OK;
}

AttendFn pick(const Cache* c, const Shape& h, bool bf16) {
  using namespace sgemv_dev;
  if (h.few) {
    if (c->exps) return c->window ? get_attend_few<true, true>(bf16, c->head_dim) : get_attend_few<true, false>(bf16, c->head_dim);
    return c->window ? get_attend_few<false, true>(bf16, c->head_dim) : get_attend_few<false, false>(bf16, c->head_dim);
  }
  if (c->exps) return c->window ? get_attend_many<true, true>(bf16, c->head_dim, h.halves) : get_attend_many<true, false>(bf16, c->head_dim, h.halves);
  return c->window ? get_attend_many<false, true>(bf16, c->head_dim, h.halves) : get_attend_many<false, false>(bf16, c->head_dim, h.halves);
}

int attend(const Cache* c, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale, const uint32_t* tree_dev,
           int32_t tree_words, int32_t max_ctx, void* workspace_dev, int64_t workspace_bytes, void* hip_stream) {
  int rc = check(c, seqs, q->tokens, q->heads, max_ctx);
  if (rc) return rc;
  if (q->tokens != out->tokens || q->heads != out->heads || q->head_dim != out->head_dim || q->dtype != out->dtype) return SGEMV_EINVAL;
  if (q->head_dim != c->head_dim || (c->dtype >= 0 && q->dtype != c->dtype)) return SGEMV_EINVAL;
  if (!(scale > 0.0f) || scale > 1.0e30f || tree_words < 0 || (tree_words > 0 && !tree_dev)) return SGEMV_EINVAL;
  if ((uintptr_t)tree_dev % 4) return SGEMV_EALIGN;
  if (q->tokens == 0 || seqs->count == 0) return SGEMV_OK;
  Shape h;
  rc = make_shape(c, seqs, q->tokens, q->heads, max_ctx, &h);
  if (rc) return rc;
  if (h.workspace > 0) {
    if (!workspace_dev) return SGEMV_EINVAL;
    if (workspace_bytes < h.workspace) return SGEMV_ESIZE;
    if ((uintptr_t)workspace_dev % 16) return SGEMV_EALIGN;
  }
  AttendParams p;
  memset(&p, 0, sizeof p);
  p.seq = seq_view(seqs, c, q->tokens);
  p.k = (const uint16_t*)c->k;
  p.v = (const uint16_t*)c->v;
  p.q = (const uint16_t*)q->data;
  p.out = (uint16_t*)out->data;
  p.k_page = c->pages > 1 ? (uint32_t)c->k_stride[0] : 0;
  p.v_page = c->pages > 1 ? (uint32_t)c->v_stride[0] : 0;
  p.k_slot = (uint32_t)c->k_stride[1];
  p.v_slot = (uint32_t)c->v_stride[1];
  p.k_head = c->heads > 1 ? c->k_stride[2] : 0;
  p.v_head = c->heads > 1 ? c->v_stride[2] : 0;
  p.q_token = q->tokens > 1 ? q->token_stride : 0;
  p.q_head = q->heads > 1 ? q->head_stride : 0;
  p.o_token = out->tokens > 1 ? out->token_stride : 0;
  p.o_head = out->heads > 1 ? out->head_stride : 0;
  p.tree = tree_dev;
  p.tree_words = tree_words;
  p.group = q->heads / c->heads;
  p.window = c->window;
  p.sinks = c->sinks;
  p.heads = c->heads;
  p.dim = q->head_dim;
  p.splits = h.splits;
  p.slots = (int32_t)h.slots;
  p.scale2 = scale * 1.44269504088896340736f;
  p.part = (float*)workspace_dev;
  if (c->exps) {
    p.exps = (const uint16_t*)c->exps;
    p.exp_shift = ilog2(c->scale_slots);
    p.exp_page = (uint32_t)(c->page_size >> p.exp_shift) * (uint32_t)c->heads;
  }
  const bool bf16 = q->dtype == SGEMV_BF16;
  const AttendFn fn = pick(c, h, bf16);
  (void)hipGetLastError();
  if (ensure_lds((const void*)fn, h.lds)) return SGEMV_EHIP;
  hipLaunchKernelGGL(fn, dim3((uint32_t)h.grid), dim3(64 * h.waves), (uint32_t)h.lds, (hipStream_t)hip_stream, p);
  if (hipGetLastError() != hipSuccess) return SGEMV_EHIP;
  if (h.splits > 1) {
    const int64_t rows = (int64_t)q->tokens * q->heads;
    // a workgroup a row while that fills the chip a few times over at most,
    // then DP/4 lanes a row (128 rows of 31 parts: 9.8 us of both kernels, 12.8
    // the other way; 1024 of 15: 23.3 and 23.4; 4096 of 16: 40.8 and 37.8)
    const bool many = rows >= 4 * kCus;
    const int64_t grid = many ? (rows * (h.dp / 4) + sgemv_dev::kJoinLanes - 1) / sgemv_dev::kJoinLanes : rows;
    hipLaunchKernelGGL(sgemv_dev::get_attend_join(bf16, p.dim, many, c->window > 0), dim3((uint32_t)grid), dim3(sgemv_dev::kJoinLanes), 0,
                       (hipStream_t)hip_stream, p, h.tile_rows, h.block);
    if (hipGetLastError() != hipSuccess) return SGEMV_EHIP;
  }
  return SGEMV_OK;
}

// Both entry points of a kind of cache. window 0: none, without sinks.
bool window_ok(int32_t window, int32_t sinks) { return window >= 0 && sinks >= 0 && (window > 0 || sinks == 0); }

template <class C>
int plan_of(const C* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t window, int32_t sinks, int32_t max_ctx,
            sgemv_attend_plan_t* out) {
  if (!out || !window_ok(window, sinks)) return SGEMV_EINVAL;
  Cache c;
  const int rc = look(cache, window, sinks, &c);
  return rc ? rc : plan(&c, seqs, tokens, heads, max_ctx, out);
}

template <class C>
int attend_of(const C* cache, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale, const uint32_t* tree_dev,
              int32_t tree_words, int32_t window, int32_t sinks, int32_t max_ctx, void* workspace_dev, int64_t workspace_bytes,
              void* hip_stream) {
  int rc = check_rows(q, false);
  if (rc) return rc;
  rc = check_rows(out, true);
  if (rc) return rc;
  if (!window_ok(window, sinks)) return SGEMV_EINVAL;
  Cache c;
  rc = look(cache, window, sinks, &c);
  return rc ? rc : attend(&c, seqs, q, out, scale, tree_dev, tree_words, max_ctx, workspace_dev, workspace_bytes, hip_stream);
}

}  // namespace

extern "C" int sgemv_attend_plan(const sgemv_cache* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx,
                                 sgemv_attend_plan_t* out) {
  return plan_of(cache, seqs, tokens, heads, 0, 0, max_ctx, out);
}

extern "C" int sgemv_attend(const sgemv_cache* cache, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale,
                            const uint32_t* tree_dev, int32_t tree_words, int32_t max_ctx, void* workspace_dev, int64_t workspace_bytes,
                            void* hip_stream) {
  return attend_of(cache, seqs, q, out, scale, tree_dev, tree_words, 0, 0, max_ctx, workspace_dev, workspace_bytes, hip_stream);
}

extern "C" int sgemv_attend_window_plan(const sgemv_cache* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t window,
                                        int32_t sinks, int32_t max_ctx, sgemv_attend_plan_t* out) {
  return plan_of(cache, seqs, tokens, heads, window, sinks, max_ctx, out);
}

extern "C" int sgemv_attend_window(const sgemv_cache* cache, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale,
                                   const uint32_t* tree_dev, int32_t tree_words, int32_t window, int32_t sinks, int32_t max_ctx,
                                   void* workspace_dev, int64_t workspace_bytes, void* hip_stream) {
  return attend_of(cache, seqs, q, out, scale, tree_dev, tree_words, window, sinks, max_ctx, workspace_dev, workspace_bytes, hip_stream);
}

extern "C" int sgemv_attend8_plan(const sgemv_cache8* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t window,
                                  int32_t sinks, int32_t max_ctx, sgemv_attend_plan_t* out) {
  return plan_of(cache, seqs, tokens, heads, window, sinks, max_ctx, out);
}

extern "C" int sgemv_attend8(const sgemv_cache8* cache, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale,
                             const uint32_t* tree_dev, int32_t tree_words, int32_t window, int32_t sinks, int32_t max_ctx,
                             void* workspace_dev, int64_t workspace_bytes, void* hip_stream) {
  return attend_of(cache, seqs, q, out, scale, tree_dev, tree_words, window, sinks, max_ctx, workspace_dev, workspace_bytes, hip_stream);
}
