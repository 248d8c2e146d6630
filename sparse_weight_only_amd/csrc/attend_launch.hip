// sgemv_attend_plan / sgemv_attend: host checks and the launches of the attention.
#include "attend_few.hpp"
#include "attend_join.hpp"
#include "attend_kernels.hpp"
#include "attend_many.hpp"
#include "decode_internal.hpp"
#include "launch_util.hpp"

using namespace sgemv;
using sgemv_dev::AttendParams;

namespace {

constexpr int kCus = 256;
using sgemv_dev::kMaxSplits;

struct Shape {
  bool few, halves;
  int dp, tile_rows, block, waves, splits;
  int64_t lds, slots, grid, workspace;
};

// Which kernel, and in how many parts the context is split: from the sizes on
// the host alone. Lengths in device memory never change what is launched.
int make_shape(const sgemv_cache* c, const sgemv_seqs* s, int32_t tokens, int32_t heads, int32_t max_ctx, Shape* out) {
  const int group = heads / c->heads;
  Shape h;
  h.dp = c->head_dim <= 64 ? 64 : c->head_dim <= 128 ? 128 : 256;
  const int64_t rows = (int64_t)tokens * group;
  int64_t ctx = (int64_t)s->pages_per_seq * c->page_size;
  if (max_ctx > 0 && max_ctx < ctx) ctx = max_ctx;
  // Up to 16 rows a sequence on average: a tile of 16 that reads K and V
  // straight from memory (12 rows, 4 sequences of up to 6000 slots, 8 heads:
  // 20.5 us, 25.5 as a tile of 128). Up to 128 rows the same, a few tiles each
  // for itself, over short contexts, where the larger kernel's start and end
  // weigh more (96 rows over 300 slots: 9.7 against 15.2 us, over 6000: 61.6
  // against 31.9; 48 rows: 11.9 against 13.6, and 39.5 against 27.8).
  h.few = rows <= (int64_t)16 * s->count || (rows <= (int64_t)128 * s->count && ctx <= 1024);
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

int check(const sgemv_cache* cache, const sgemv_seqs* seqs, int32_t tokens, int32_t heads, int32_t max_ctx) {
  int rc = check_cache(cache, false);
  if (rc) return rc;
  rc = check_seqs(seqs);
  if (rc) return rc;
  // the kernels' page and slot strides, and eight slots' bytes, fit 32 bits
  for (const int64_t* d : {&cache->k_page, &cache->v_page})
    if ((cache->pages > 1 && d[0] > INT32_MAX) || d[1] > INT32_MAX / 16) return SGEMV_ESIZE;
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
  p.k_page = cache->pages > 1 ? (uint32_t)cache->k_page : 0;
  p.v_page = cache->pages > 1 ? (uint32_t)cache->v_page : 0;
  p.k_slot = (uint32_t)cache->k_slot;
  p.v_slot = (uint32_t)cache->v_slot;
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
  sgemv_dev::AttendFn fn = h.few ? sgemv_dev::get_attend_few(bf16, p.dim) : sgemv_dev::get_attend_many(bf16, p.dim, h.halves);
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
    hipLaunchKernelGGL(sgemv_dev::get_attend_join(bf16, p.dim, many), dim3((uint32_t)grid), dim3(sgemv_dev::kJoinLanes), 0,
                       (hipStream_t)hip_stream, p, h.tile_rows, h.block);
    if (hipGetLastError() != hipSuccess) return SGEMV_EHIP;
  }
  return SGEMV_OK;
}
