// Which keys a tile of a windowed attention goes through and which of them a new
// token sees, run on the CPU under the sanitizers: random windows, sinks, trees
// and splits against the definition slot by slot. Prints "ok", or what failed.
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <random>
#include <vector>

#include "../../sparse_weight_only_amd/csrc/decode_index.hpp"

using namespace sgemv_dev;

#define REQUIRE(c)                                                                  \
  do {                                                                              \
    if (!(c)) { printf("failed: %s (line %d, set %d)\n", #c, __LINE__, set); exit(1); } \
  } while (0)

int main() {
  std::mt19937 rng(5);
  const auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int set = 0; set < 4000; ++set) {
    const int n = pick(1, set % 3 ? 6 : 90), ctx = pick(0, set % 5 ? 600 : n), group = pick(1, 5), words = pick(0, 4);
    const int per = (ctx + 7) / 8;
    const int32_t start[2] = {0, n}, len[1] = {ctx};
    const std::unique_ptr<int32_t[]> pages(new int32_t[per]());
    const std::unique_ptr<uint32_t[]> tree(new uint32_t[(size_t)n * words]);
    for (int i = 0; i < n * words; ++i) tree[i] = rng() & rng();
    TileView p;
    p.seq = SeqView{start, len, pages.get(), per, 1, per, 3, 1, n};
    p.tree = set % 2 ? tree.get() : nullptr;
    p.tree_words = words;
    p.group = group;
    p.splits = pick(1, 4);
    p.window = set % 11 == 0 ? 1 << 30 : pick(1, set % 4 ? 120 : 700);
    p.sinks = set % 13 == 0 ? 1 << 30 : set % 4 == 1 ? 0 : pick(0, 90);
    for (const auto& mb : {std::pair<int, int>{16, 32}, {128, 64}, {256, 64}, {256, 32}}) {
      const int m = mb.first, block = mb.second;
      for (int slot = 0; slot < n * group / m + 1; ++slot) {
        int at_key = 0;
        for (int split = 0; split < p.splits; ++split) {
          Tile t;
          if (!make_tile<true>(p, m, block, 0, 0, n, p.seq.ctx(0), slot, split, t)) break;
          REQUIRE(t.gap0 % block == 0 && t.gap % block == 0 && t.gap >= 0 && t.keys >= 0 && t.keys <= t.end && t.end <= ctx);
          REQUIRE(split == 0 ? t.key0 == 0 : t.key0 == at_key);
          at_key = t.key1;
          if (split == p.splits - 1) REQUIRE(t.key1 == t.keys);
          Tile j = t;
          tile_keys<true>(p, m, block, p.seq.ctx(0), 0, j);
          const int part = j.key1, parts = part > 0 ? (j.keys + part - 1) / part : 0;
          REQUIRE(parts <= p.splits && (t.key0 < t.key1) == (split < parts));
          for (int v = t.key0; v < t.key1; ++v) {
            REQUIRE(slot_of<true>(t, v) >= 0 && slot_of<true>(t, v) < ctx);
            (void)pages[slot_of<true>(t, v) >> 3];
          }
          if (split) continue;
          // each row sees each of its slots once, under some key number
          for (int r = t.row0; r < t.rows && r < t.row0 + m; ++r) {
            const int i = r / group, own = ctx - n + i, from = window_from(p, t, i);
            int path = 0;
            for (int b = 0; p.tree && b < n && b < 32 * words; ++b) path += tree[(size_t)i * words + b / 32] >> (b % 32) & 1;
            std::vector<int> seen(ctx, 0);
            for (int kb = 0; kb < t.keys; kb += 32) {
              const int at = slot_of<true>(t, kb);
              const uint32_t bits = visible_bits(p, t, i, at) & window_bits(p.sinks, from, at);
              const bool masked = needs_mask<true>(p, t, slot_of<true>(t, kb / block * block), block);
              for (int b = 0; b < 32; ++b) {
                if (kb + b >= t.keys) { REQUIRE(!(bits >> b & 1)); continue; }
                REQUIRE(slot_of<true>(t, kb + b) == at + b);
                if (bits >> b & 1) ++seen[at + b];
                else REQUIRE(masked);
              }
            }
            for (int k = 0; k < ctx; ++k) {
              const int64_t old = ctx - n, b = k - old;
              bool want = own >= 0;
              if (p.tree) want = want && (b < 0 ? (k >= old + path - (int64_t)p.window || k < p.sinks)
                                                : (b < 32 * words && (tree[(size_t)i * words + b / 32] >> (b % 32) & 1)));
              else want = want && k <= own && (k > (int64_t)own - p.window || k < p.sinks);
              REQUIRE(seen[k] == (want ? 1 : 0));
            }
          }
        }
      }
    }
  }
  printf("ok\n");
  return 0;
}
