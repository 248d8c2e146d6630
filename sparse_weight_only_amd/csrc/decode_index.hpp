// Where the operators between the GEMVs find their tokens, keys and pages:
// plain arithmetic, compiled into the kernels and, for its tests, for the CPU.
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define SGEMV_BOTH __host__ __device__ __forceinline__
#else
#define SGEMV_BOTH inline
#endif

namespace sgemv_dev {

// Sequences as the kernels see them (sgemv_seqs). Lengths live in device
// memory, where no host check reaches them, so every one is clamped before
// it is used: a bad one gives wrong numbers, never an access out of range.
struct SeqView {
  const int32_t* new_start;   // [count + 1] first new token of each sequence
  const int32_t* ctx_len;     // [count] tokens of each sequence, new ones included
  const int32_t* pages;       // [count][pages_per_seq]
  int64_t pages_stride;
  int32_t count, pages_per_seq, page_shift, n_pages, tokens;

  SGEMV_BOTH int start(int s) const {
    const int v = new_start[s];
    return v < 0 ? 0 : v > tokens ? tokens : v;
  }
  // tokens of sequence s: no more than its row of the page table holds
  SGEMV_BOTH int ctx(int s) const {
    const int64_t cap = (int64_t)pages_per_seq << page_shift;
    const int v = ctx_len[s];
    return v < 0 ? 0 : v > cap ? (int)cap : v;
  }
  SGEMV_BOTH bool page_ok(int page) const { return (uint32_t)page < (uint32_t)n_pages; }
};

// A search for the last place of [0, count) that a condition holds for, given
// that it holds up to some place: 64 lanes look at 64 places at a time.
struct Upper {
  int lo, n;
  SGEMV_BOTH explicit Upper(int count) : lo(0), n(count) {}
  SGEMV_BOTH int step() const { return (n + 63) >> 6; }
  SGEMV_BOTH bool in(int lane) const { return lane * step() < n; }
  SGEMV_BOTH int place(int lane) const { return in(lane) ? lo + lane * step() : lo; }
  // `holds`: how many lanes it holds for
  SGEMV_BOTH void narrow(int holds) {
    const int s = step(), skip = (holds < 1 ? 0 : holds - 1) * s;
    lo += skip;
    n = n - skip < s ? n - skip : s;
  }
};

// The rows of a tile are (new token, query head of the group) pairs of one
// sequence and cache head: row r is token r / group, head r % group, so a
// tile of a shared head reads its keys once for the whole group.
//
// Tiles of M rows are numbered without a pass over the sequences: sequence s
// has the slots from floor(start(s) group / M) + s on, at least as many as its
// tiles, since floor(a + b) - floor(a) + 1 >= ceil(b); what is left over is
// empty. floor(tokens group / M) + count slots in all.
struct TileView {
  SeqView seq;
  const uint32_t* tree;   // [tokens][tree_words], or null: a token sees the slots up to its own
  int32_t tree_words;
  int32_t group;          // query heads per cache head
  int32_t splits;         // parts of the context
};

struct Tile {
  int s, first, n;          // sequence, its first new token, its new tokens
  int old;                  // slot of its first new token
  int row0, rows;           // first row of the tile, rows of the sequence
  int end, full;            // keys any row sees, keys every row sees
  int key0, key1;           // this split's part of [0, end)
  const int32_t* pages;
};

// First slot of sequence s, whose first new token is `first`. tokens x heads
// is at most 2^30, so rows fit 32 bits without a sign.
SGEMV_BOTH int slot_base(const TileView& p, int s, int first, int m) {
  return (int)((uint32_t)first * (uint32_t)p.group / (uint32_t)m) + s;
}

// The keys of the tile at `row0` of sequence t.s, and split `split` of them in
// whole blocks of `block` keys.
SGEMV_BOTH void tile_keys(const TileView& p, int m, int block, int ctx, int split, Tile& t) {
  t.old = ctx - t.n;
  if (p.tree) {
    t.end = ctx;
    t.full = t.old;
  } else {
    const int last = t.row0 + m < t.rows ? (t.row0 + m - 1) / p.group : t.n - 1;
    t.end = t.old + last + 1;
    t.full = t.old + t.row0 / p.group + 1;
  }
  t.end = t.end < 0 ? 0 : t.end > ctx ? ctx : t.end;
  const int blocks = (t.end + block - 1) / block;
  const int per = (blocks + p.splits - 1) / p.splits * block;
  const int64_t k0 = (int64_t)split * per;
  t.key0 = k0 < t.end ? (int)k0 : t.end;
  t.key1 = k0 + per < t.end ? (int)(k0 + per) : t.end;
}

// The tile of `slot`, which lies in sequence s with new tokens first .. next - 1
// and ctx tokens in all; false for an empty slot.
SGEMV_BOTH bool make_tile(const TileView& p, int m, int block, int s, int first, int next, int ctx, int slot, int split, Tile& t) {
  t.s = s;
  t.first = first;
  t.n = next - first;
  t.rows = t.n * p.group;
  const int64_t at = slot - slot_base(p, s, first, m);
  if (t.n <= 0 || at < 0 || at * m >= t.rows) return false;
  t.row0 = (int)at * m;
  t.pages = p.seq.pages + s * p.seq.pages_stride;
  tile_keys(p, m, block, ctx, split, t);
  return true;
}

// Bit b: whether key kb + b lies before the end and new token `i` of the tile's
// sequence sees it, by its slot or by its words of the tree.
SGEMV_BOTH uint32_t seen_bits(const TileView& p, const Tile& t, int i, int kb) {
  int n;
  uint32_t bits = ~0u;
  if (p.tree) {
    // the words of this row, from new token kb - old on; older keys are seen
    const int at = kb - t.old;
    const uint32_t* w = p.tree + (int64_t)(t.first + i) * p.tree_words;
    const int w0 = at >> 5, sh = at & 31;      // rounds down for at < 0 too
    const uint32_t a = w0 < 0 ? ~0u : w0 < p.tree_words ? w[w0] : 0u;
    const uint32_t b = w0 + 1 < 0 ? ~0u : w0 + 1 < p.tree_words ? w[w0 + 1] : 0u;
    bits = sh ? (a >> sh) | (b << (32 - sh)) : a;
    n = t.end - kb;
  } else {
    n = t.old + i + 1 - kb;
    n = n < t.end - kb ? n : t.end - kb;
  }
  return n >= 32 ? bits : n <= 0 ? 0u : bits & ((1u << n) - 1u);
}

// The same for a token that may have no slot: in a sequence shorter than its
// new tokens the first of them lie below slot 0 and see no key, whatever their
// words of the tree say. Such a tile has `full` at 0 or less, so all of its
// blocks are masked.
SGEMV_BOTH uint32_t visible_bits(const TileView& p, const Tile& t, int i, int kb) {
  return t.old + i < 0 ? 0u : seen_bits(p, t, i, kb);
}

}  // namespace sgemv_dev
