// Which keys a new token sees, run on the CPU under the sanitizers: sequences
// shorter and longer than their new tokens, with and without a tree, against
// the definition key by key. Prints "ok", or what failed.
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <random>

#include "../../sparse_weight_only_amd/csrc/decode_index.hpp"

using namespace sgemv_dev;

int main() {
  std::mt19937 rng(11);
  const auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int set = 0; set < 3000; ++set) {
    const int n = pick(1, 70), ctx = pick(0, set % 2 ? 150 : n), group = pick(1, 5), words = pick(0, 3);
    const int32_t start[2] = {0, n}, len[1] = {ctx};
    const std::unique_ptr<int32_t[]> pages(new int32_t[19]());
    const std::unique_ptr<uint32_t[]> tree(new uint32_t[(size_t)n * words]);
    for (int i = 0; i < n * words; ++i) tree[i] = rng();
    TileView p;
    p.seq = SeqView{start, len, pages.get(), 19, 1, 19, 3, 1, n};
    p.tree = set % 3 ? tree.get() : nullptr;
    p.tree_words = words;
    p.group = group;
    p.splits = 1;
    for (int slot = 0; slot < n * group / 16 + 1; ++slot) {
      Tile t;
      if (!make_tile(p, 16, 32, 0, 0, n, p.seq.ctx(0), slot, 0, t)) continue;
      for (int r = t.row0; r < t.rows && r < t.row0 + 16; ++r) {
        const int i = r / group, own = ctx - n + i;
        for (int key = 0; key < ctx + 40; ++key) {
          const int j = key - (ctx - n);
          bool want = own >= 0 && key < ctx;                     // a token below slot 0 has no key
          if (p.tree) want = want && (j < 0 || (j < 32 * words && (tree[(size_t)i * words + j / 32] >> (j % 32) & 1)));
          else want = want && key <= own;
          const bool got = visible_bits(p, t, i, key & ~31) >> (key & 31) & 1;
          // blocks that end at `full` are not masked
          const bool masked = (key & ~31) + 32 > t.full;
          if (got != want || (!masked && key < t.end && !want)) {
            printf("failed: set %d, n %d, ctx %d, token %d, key %d: %d\n", set, n, ctx, i, key, got);
            return 1;
          }
        }
      }
    }
  }
  printf("ok\n");
  return 0;
}
