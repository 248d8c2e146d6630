// sgemv_attend_plan / sgemv_attend: host checks and the launches of the attention.
#include "attend_kernels.hpp"
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;
using sgemv_dev::AttendParams;

namespace {

constexpr int kCus = 256;
constexpr int kMaxSplits = 256;

struct Shape {
  bool few;
  int dp, tile_rows, block, waves, splits;
  int64_t lds, slots, workspace;
};

// Which kernel, and in how many parts the context is split: from the sizes on
// the host alone. Lengths in device memory never change what is launched.
int make_shape(const sgemv_cache* c, const sgemv_seqs* s, int32_t tokens, int32_t heads, int32_t max_ctx, Shape* out) {
  const int group = heads / c->heads;
  Shape h;
  h.dp = c->head_dim <= 64 ? 64 : c->head_dim <= 128 ? 128 : 256;
  const int64_t rows = (int64_t)tokens * group;
  h.few = rows <= (int64_t)32 * s->count;
  h.waves = h.few || h.dp == 256 ? 4 : 8;
  h.tile_rows = h.few ? 16 : 32 * h.waves;
  h.block = h.few ? 32 : 64;
  h.lds = h.few ? 0 : (int64_t)2 * 2 * 64 * h.dp * 2;
  h.slots = rows / h.tile_rows + s->count;
  int64_t ctx = (int64_t)s->pages_per_seq * c->page_size;
  if (max_ctx > 0 && max_ctx < ctx) ctx = max_ctx;
  int64_t tiles = (rows + h.tile_rows - 1) / h.tile_rows;
  const int64_t each = s->count < tokens ? s->count : tokens;
  if (tiles < each) tiles = each;
  const int64_t want = 2 * kCus / (tiles * c->heads);
  const int64_t most = ctx / 256;
  int64_t splits = want < most ? want : most;
  splits = splits < 1 ? 1 : splits > kMaxSplits ? kMaxSplits : splits;
  h.splits = (int)splits;
  h.workspace = splits > 1 ? (int64_t)tokens * heads * splits * (c->head_dim + 2) * 4 : 0;
  if (h.slots * c->heads * splits * h.waves * 64 > (int64_t)UINT32_MAX) return SGEMV_ESIZE;
  *out = h;
  return SGEMV_OK;
}

int check(const sgemv_cache* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx) {
  int rc = check_cache(cache, false);
  if (rc) return rc;
  rc = check_seqs(seqs);
  if (rc) return rc;
  if (tokens < 0 || heads < 1 || heads > 65535 || heads % cache->heads || max_ctx < 0) return SGEMV_EINVAL;
  return (int64_t)tokens * heads > (1 << 30) ? SGEMV_ESIZE : SGEMV_OK;
}

}  // namespace

extern "C" int sgemv_attend_plan(const sgemv_cache* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx,
                                 sgemv_attend_plan_t* out) {
  if (!out) return SGEMV_EINVAL;
  const int rc = check(cache, seqs, tokens, heads, max_ctx);
  if (rc) return rc;
  sgemv_attend_plan_t q;
  memset(&q, 0, sizeof q);
  if (tokens > 0 && seqs->count > 0) {
    Shape h;
    const int rs = make_shape(cache, seqs, tokens, heads, max_ctx, &h);
    if (rs) return rs;
    q.workspace_bytes = h.workspace;
    q.grid = h.slots * cache->heads * h.splits;
    q.lds_bytes = h.lds;
    q.block = 64 * h.waves;
    q.tile_rows = h.tile_rows;
    q.block_keys = h.block;
    q.splits = h.splits;
  }
  *out = q;
  return SGEMV_OK;
}

extern "C" int sgemv_attend(const sgemv_cache* cache, const sgemv_seqs* seqs, const sgemv_rows* q, const sgemv_rows* out, float scale,
                            const uint32_t* tree_dev, int32_t tree_words, int32_t max_ctx, void* workspace_dev, int64_t workspace_bytes,
                            void* hip_stream) {
  int rc = check_rows(q, false);
  if (rc) return rc;
  rc = check_rows(out, true);
  if (rc) return rc;
  rc = check(cache, seqs, q->tokens, q->heads, max_ctx);
  if (rc) return rc;
  if (q->tokens != out->tokens || q->heads != out->heads || q->head_dim != out->head_dim || q->dtype != out->dtype) return SGEMV_EINVAL;
  if (q->head_dim != cache->head_dim || q->dtype != cache->dtype) return SGEMV_EINVAL;
  if (!(scale > 0.0f) || scale > 1.0e30f || tree_words < 0 || (tree_words > 0 && !tree_dev)) return SGEMV_EINVAL;
  if ((uintptr_t)tree_dev % 4) return SGEMV_EALIGN;
  if (q->tokens == 0 || seqs->count == 0) return SGEMV_OK;
  Shape h;
  rc = make_shape(cache, seqs, q->tokens, q->heads, max_ctx, &h);
  if (rc) return rc;
  if (h.workspace > 0) {
    if (!workspace_dev) return SGEMV_EINVAL;
    if (workspace_bytes < h.workspace) return SGEMV_ESIZE;
    if ((uintptr_t)workspace_dev % 16) return SGEMV_EALIGN;
  }
  AttendParams p;
  memset(&p, 0, sizeof p);
  p.seq = seq_view(seqs, cache, q->tokens);
  p.k = (const uint16_t*)cache->k;
  p.v = (const uint16_t*)cache->v;
  p.q = (const uint16_t*)q->data;
  p.out = (uint16_t*)out->data;
  p.k_page = cache->pages > 1 ? cache->k_page : 0;
  p.v_page = cache->pages > 1 ? cache->v_page : 0;
  p.k_slot = cache->k_slot;
  p.v_slot = cache->v_slot;
  p.k_head = cache->heads > 1 ? cache->k_head : 0;
  p.v_head = cache->heads > 1 ? cache->v_head : 0;
  p.q_token = q->tokens > 1 ? q->token_stride : 0;
  p.q_head = q->heads > 1 ? q->head_stride : 0;
  p.o_token = out->tokens > 1 ? out->token_stride : 0;
  p.o_head = out->heads > 1 ? out->head_stride : 0;
  p.tree = tree_dev;
  p.tree_words = tree_words;
  p.group = q->heads / cache->heads;
  p.heads = cache->heads;
  p.dim = q->head_dim;
  p.splits = h.splits;
  p.slots = (int32_t)h.slots;
  p.scale2 = scale * 1.44269504088896340736f;
  p.part = (float*)workspace_dev;
  const bool bf16 = q->dtype == SGEMV_BF16;
  sgemv_dev::AttendFn fn = h.few ? sgemv_dev::get_attend_few(bf16, h.dp) : sgemv_dev::get_attend_many(bf16, h.dp);
  (void)hipGetLastError();
  if (ensure_lds((const void*)fn, h.lds)) return SGEMV_EHIP;
  hipLaunchKernelGGL(fn, dim3((uint32_t)(h.slots * cache->heads * h.splits)), dim3(64 * h.waves), (uint32_t)h.lds, (hipStream_t)hip_stream, p);
  if (hipGetLastError() != hipSuccess) return SGEMV_EHIP;
  if (h.splits > 1) {
    const int64_t rows = (int64_t)q->tokens * q->heads;
    hipLaunchKernelGGL(sgemv_dev::get_attend_join(bf16), dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, (hipStream_t)hip_stream, p,
                       h.tile_rows, h.block);
    if (hipGetLastError() != hipSuccess) return SGEMV_EHIP;
  }
  return SGEMV_OK;
}
