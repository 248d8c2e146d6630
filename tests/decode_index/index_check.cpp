// Where the decode-step operators find tokens, keys and pages, run on the CPU
// under the address and undefined-behaviour sanitizers: random sequences, good
// ones and ones with anything in their arrays, each array exactly as long as
// its contract says. Prints "ok" and the number of sequences sets, or what failed.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <memory>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "../../sparse_weight_only_amd/csrc/decode_index.hpp"

using namespace sgemv_dev;

#define REQUIRE(c)                                                                  \
  do {                                                                              \
    if (!(c)) { printf("failed: %s (line %d, set %d)\n", #c, __LINE__, set); exit(1); } \
  } while (0)

static int set = 0;
static std::mt19937 rng(7);
static int pick(int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); }

// the search as a wave makes it
template <class F>
static int upper(int count, int64_t x, F f) {
  Upper u(count);
  for (int rounds = 0; u.n > 1; ++rounds) {
    REQUIRE(rounds < 8);
    int holds = 0;
    for (int lane = 0; lane < 64; ++lane) holds += u.in(lane) && f(u.place(lane)) <= x;
    u.narrow(holds);
  }
  return u.lo;
}

int main() {
  for (set = 0; set < 1500; ++set) {
    const bool bad = set % 2;
    const int count = set % 7 == 0 ? pick(60, 300) : pick(1, 9), group = pick(1, 9), shift = pick(3, 6), per = pick(0, 6), pages = pick(0, 12);
    std::vector<int> n(count);
    int tokens = 0;
    for (int& v : n) { v = pick(0, 3) ? pick(0, set % 5 ? 12 : 60) : 0; tokens += v; }
    const int lead = pick(0, 2), trail = pick(0, 2);
    std::unique_ptr<int32_t[]> start(new int32_t[count + 1]), ctx(new int32_t[count]), table(new int32_t[(size_t)count * per]);
    start[0] = lead;
    for (int s = 0; s < count; ++s) start[s + 1] = start[s] + n[s];
    tokens += lead + trail;
    for (int s = 0; s < count; ++s) ctx[s] = n[s] + pick(0, (per << shift) + 3);
    for (int i = 0; i < count * per; ++i) table[i] = pages ? pick(0, pages - 1) : 0;
    const int words = pick(0, 3);
    std::unique_ptr<uint32_t[]> tree(new uint32_t[(size_t)tokens * words]);
    for (int i = 0; i < tokens * words; ++i) tree[i] = rng();
    if (bad) {
      auto any = [&] { const int k = pick(0, 4); return k == 0 ? INT32_MIN : k == 1 ? INT32_MAX : k == 2 ? -pick(1, 50) : pick(0, 100); };
      for (int i = 0; i < 3; ++i) {
        start[pick(0, count)] = any();
        ctx[pick(0, count - 1)] = any();
        if (per) table[pick(0, count * per - 1)] = any();
      }
    }
    TileView p;
    p.seq = SeqView{start.get(), ctx.get(), table.get(), per, count, per, shift, pages, tokens};
    p.tree = set % 3 ? nullptr : tree.get();
    p.tree_words = words;
    p.group = group;
    p.splits = pick(1, 5);
    for (const auto& mb : {std::pair<int, int>{16, 32}, {128, 64}, {256, 64}, {256, 32}}) {
      const int m = mb.first, block = mb.second;
      const int slots = (int)((int64_t)tokens * group / m + count);
      std::map<std::pair<int, int>, int> rows_seen;   // (token, head of the group) -> tiles
      for (int slot = 0; slot < slots; ++slot) {
        const int s = upper(count, slot, [&](int i) { return slot_base(p, i, p.seq.start(i), m); });
        REQUIRE(s >= 0 && s < count);
        int at_key = 0;
        for (int split = 0; split < p.splits; ++split) {
          Tile t;
          if (!make_tile(p, m, block, s, p.seq.start(s), p.seq.start(s + 1), p.seq.ctx(s), slot, split, t)) break;
          REQUIRE(t.row0 >= 0 && t.row0 < t.rows && t.first >= 0 && t.first + t.n <= tokens);
          REQUIRE(t.key0 <= t.key1 && t.key1 <= t.end && t.end <= per << shift);
          REQUIRE(split == 0 ? t.key0 == 0 : t.key0 == at_key);
          at_key = t.key1;
          if (split == p.splits - 1) REQUIRE(t.key1 == t.end);
          // the join finds the same parts from split 0 alone
          Tile j = t;
          tile_keys(p, m, block, p.seq.ctx(s), 0, j);
          const int len = j.key1, parts = len > 0 ? (j.end + len - 1) / len : 0;
          REQUIRE(parts <= p.splits && (t.key0 < t.key1) == (split < parts));
          int sum = 0;
          for (int key = t.key0; key < t.key1; ++key) sum += p.seq.page_ok(t.pages[key >> shift]);
          REQUIRE(sum >= 0);
          if (split) continue;
          for (int r = t.row0; r < t.rows && r < t.row0 + m; ++r) {
            ++rows_seen[{t.first + r / group, r % group}];
            const int i = r / group;
            for (int kb = 0; kb < t.end + 32; kb += 32) {
              const uint32_t bits = seen_bits(p, t, i, kb);
              for (int b = 0; b < 32; ++b) {
                const int key = kb + b, new_j = key - t.old;
                bool want = key < t.end;
                if (p.tree) want = want && (new_j < 0 || (new_j < 32 * words && (tree[(size_t)(t.first + i) * words + new_j / 32] >> (new_j % 32) & 1)));
                else want = want && key <= t.old + i;
                REQUIRE((bits >> b & 1) == want);
                if (key < t.full && key < t.end) REQUIRE(want);
              }
            }
          }
        }
      }
      if (!bad) {
        REQUIRE((int)rows_seen.size() == (tokens - lead - trail) * group);
        for (const auto& e : rows_seen) REQUIRE(e.second == 1);
      }
      for (int tok = 0; tok < tokens; ++tok) {         // as the append and the join find a token's sequence
        const int s = upper(count, tok, [&](int i) { return (int64_t)p.seq.start(i); });
        const int a = p.seq.start(s), b = p.seq.start(s + 1);
        if (!bad) REQUIRE((tok >= a && tok < b) == (tok >= lead && tok < tokens - trail));
        if (tok < a || tok >= b) continue;
        const int slot = p.seq.ctx(s) - (b - tok);
        REQUIRE(slot < per << shift);
        if (slot >= 0) p.seq.page_ok(table[(size_t)s * per + (slot >> shift)]);
      }
    }
  }
  printf("ok %d\n", set);
  return 0;
}
