// Host checks shared by the operators between the GEMVs of a decode step.
#pragma once
#include "decode_device.hpp"
#include "internal.hpp"

namespace sgemv {

inline bool half_type(int dtype) { return dtype == SGEMV_F16 || dtype == SGEMV_BF16; }
inline bool valid_dim(int d) { return d >= 8 && d <= 256 && d % 8 == 0; }

// A stride between n things of `least` elements that the kernels reach with
// 16-byte accesses; one thing has no stride to check. `least` 0: things that
// are only read may overlap.
inline bool stride_ok(int64_t stride, int64_t n, int64_t least) {
  return n <= 1 || (stride >= least && stride % 8 == 0 && stride <= INT64_MAX / 4 / n);
}

// Packed rows of tokens x heads x columns.
inline int check_rows(const sgemv_rows* r, bool written) {
  if (!r) return SGEMV_EINVAL;
  if (r->tokens < 0 || r->heads < 1 || r->heads > 65535 || !valid_dim(r->head_dim) || !half_type(r->dtype)) return SGEMV_EINVAL;
  if ((int64_t)r->tokens * r->heads > (1 << 30)) return SGEMV_ESIZE;   // rows are counted in 32 bits
  const int64_t least = written ? r->head_dim : 0;
  if (!stride_ok(r->token_stride, r->tokens, least) || !stride_ok(r->head_stride, r->heads, least)) return SGEMV_EINVAL;
  if (r->tokens > 0 && !r->data) return SGEMV_EINVAL;
  if ((uintptr_t)r->data % 16) return SGEMV_EALIGN;
  return SGEMV_OK;
}

inline int check_cache(const sgemv_cache* c, bool written) {
  if (!c) return SGEMV_EINVAL;
  if (c->pages < 0 || c->heads < 1 || c->heads > 65535 || !valid_dim(c->head_dim) || !half_type(c->dtype)) return SGEMV_EINVAL;
  if (c->page_size < 8 || c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return SGEMV_EINVAL;
  const int64_t least = written ? c->head_dim : 0;
  for (const int64_t* s : {&c->k_page, &c->v_page}) {
    if (!stride_ok(s[0], c->pages, least) || !stride_ok(s[1], c->page_size, least) || !stride_ok(s[2], c->heads, least)) return SGEMV_EINVAL;
  }
  if (c->pages > 0 && (!c->k || !c->v)) return SGEMV_EINVAL;
  if ((uintptr_t)c->k % 16 || (uintptr_t)c->v % 16) return SGEMV_EALIGN;
  return SGEMV_OK;
}

// A cache in 8 bits: 16 codes to a 16-byte access.
inline bool stride16_ok(int64_t stride, int64_t n, int64_t least) { return n <= 1 || (stride_ok(stride, n, least) && stride % 16 == 0); }

inline int check_cache8(const sgemv_cache8* c, bool written) {
  if (!c) return SGEMV_EINVAL;
  if (c->pages < 0 || c->heads < 1 || c->heads > 65535 || !valid_dim(c->head_dim) || c->head_dim % 16) return SGEMV_EINVAL;
  if (c->page_size < 8 || c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return SGEMV_EINVAL;
  if (c->scale_slots < 8 || c->scale_slots > 128 || (c->scale_slots & (c->scale_slots - 1)) || c->scale_slots > c->page_size) return SGEMV_EINVAL;
  const int64_t least = written ? c->head_dim : 0;
  for (const int64_t* s : {&c->k_page, &c->v_page}) {
    if (!stride16_ok(s[0], c->pages, least) || !stride16_ok(s[1], c->page_size, least) || !stride16_ok(s[2], c->heads, least)) return SGEMV_EINVAL;
  }
  if (c->pages > 0 && (!c->k || !c->v || !c->scales)) return SGEMV_EINVAL;
  if ((int64_t)(c->page_size / c->scale_slots) * c->heads > INT32_MAX) return SGEMV_ESIZE;
  if ((uintptr_t)c->k % 16 || (uintptr_t)c->v % 16 || (uintptr_t)c->scales % 2) return SGEMV_EALIGN;
  return SGEMV_OK;
}

inline int check_seqs(const sgemv_seqs* s) {
  if (!s || s->count < 0 || s->pages_per_seq < 0) return SGEMV_EINVAL;
  if (s->count == 0) return SGEMV_OK;
  if (!s->new_start || !s->ctx_len || (s->pages_per_seq > 0 && !s->pages)) return SGEMV_EINVAL;
  if (s->count > 1 && (s->pages_stride < 0 || s->pages_stride > INT64_MAX / 8 / s->count)) return SGEMV_EINVAL;
  if ((uintptr_t)s->new_start % 4 || (uintptr_t)s->ctx_len % 4 || (uintptr_t)s->pages % 4) return SGEMV_EALIGN;
  return SGEMV_OK;
}

template <class Cache>
sgemv_dev::SeqView seq_view(const sgemv_seqs* s, const Cache* c, int32_t tokens) {
  sgemv_dev::SeqView v;
  v.new_start = s->new_start;
  v.ctx_len = s->ctx_len;
  v.pages = s->pages;
  v.pages_stride = s->count > 1 ? s->pages_stride : 0;
  v.count = s->count;
  v.page_shift = ilog2(c->page_size);
  // slots are counted in 32 bits: pages past 2^30 slots are out of reach
  const int32_t most = (1 << 30) >> v.page_shift;
  v.pages_per_seq = s->pages_per_seq < most ? s->pages_per_seq : most;
  v.n_pages = c->pages;
  v.tokens = tokens;
  return v;
}

}  // namespace sgemv
