// How many logits of a row are listed for its top_k, run on the CPU under the
// sanitizers: rows of many lengths and both widths of a load, with masks of -inf,
// NaN, large negative numbers and min_p, each lane's largest logit as the kernel's
// lanes have it. At least k lanes reach the bound, and no more than kCrowd below
// the k-th of them. Prints "ok", or what failed.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../sparse_weight_only_amd/csrc/sample_bound.hpp"

using namespace sgemv_dev;

static int failures = 0;

static void check(const char* what, const std::vector<float>& x, int per, int k, float least = -0x1.fffffep127f) {
  const int vocab = (int)x.size(), stretch = stretch_of(vocab, per);
  std::vector<float> most(kSampleLanes, -INFINITY);
  for (int id = 0; id < vocab; ++id) {
    float& lane = most.at(id / stretch * 64 + id % stretch / per % 64);
    lane = fmaxf(lane, x[id]);
  }
  uint32_t top = 0, low = 0;
  for (float m : most) top = std::max(top, key_of(m)), low = std::max(low, low_part(key_of(m)));
  if (top <= kNeverKey) return;
  if (of_key(top) == INFINITY) least = INFINITY;

  std::vector<char> here(kSampleLanes);
  std::vector<int> at(kSampleLanes);
  int with = 0, bin, before, crowd;
  for (int i = 0; i < kSampleLanes; ++i) with += here[i] = most[i] >= least;
  const auto find = [&](int need, auto bin_of) {
    std::vector<int> count(kSampleLanes);
    for (int i = 0; i < kSampleLanes; ++i)
      if (here[i]) ++count.at(at[i] = bin_of(most[i]));
    for (bin = before = 0; before + count.at(bin) < need;) before += count[bin++];
    crowd = count[bin];
  };
  float bound = least;
  int need = k;
  if (with >= k) {
    const LogitBins logits(of_key(top), fmaxf(of_key(~low), least));
    find(need, [&](float m) { return logits.bin(m); });
    bound = fmaxf(bound, logits.lower(bin));
    const auto border = [&] {
      need -= before;
      for (int i = 0; i < kSampleLanes; ++i) here[i] = here[i] && at[i] == bin;
    };
    if (crowd > kCrowd) {
      border();
      uint32_t hi = 0, lo = 0;
      for (int i = 0; i < kSampleLanes; ++i)
        if (here[i]) hi = std::max(hi, key_of(most[i])), lo = std::max(lo, ~key_of(most[i]));
      KeyBins keys(hi, ~lo);
      for (int round = 0; round < kKeyRounds; ++round) {
        find(need, [&](float m) { return keys.bin(key_of(m)); });
        border();
        keys.narrow(bin);
        if (crowd <= kCrowd || keys.low == keys.top) break;
      }
      bound = fmaxf(bound, of_key(keys.low));
    }
  }
  std::vector<float> order = most;
  std::sort(order.begin(), order.end(), std::greater<float>());
  int lanes = 0, ideal = 0, listed = 0;
  for (float m : most) lanes += m >= bound, ideal += m >= fmaxf(order[k - 1], least);
  for (float v : x) listed += v >= bound;
  if (!(bound >= least && (with < k ? bound == least : lanes >= k && lanes <= ideal + kCrowd) && listed >= std::min(k, with)) && ++failures <= 20)
    printf("failed: %s, %d logits, %d a load, k %d: %d of %d lanes from the bound on (%d from the k-th), %d listed\n", what, vocab, per, k, lanes, with,
           ideal, listed);
}

int main() {
  std::mt19937 rng(7);
  std::normal_distribution<float> normal(0.0f, 2.0f);
  std::uniform_real_distribution<float> uniform(0.0f, 1.0f);
  const int sizes[] = {1, 7, 999, 4097, 8191, 8193, 30522, 32000, 32761, 32768, 33000, 36000, 49408, 50021, 50257, 50304, 51200, 65024, 92416, 100277,
                       128003, 151643, 200001};
  for (int vocab : sizes)
    for (int per : {4, 8}) {
      if (vocab < per) continue;
      std::vector<float> plain(vocab);
      for (float& v : plain) v = normal(rng);
      const auto masked = [&](float share, float with) {
        std::vector<float> y = plain;
        for (float& v : y) v = uniform(rng) < share ? with : v;
        return y;
      };
      std::vector<float> half = plain, steps = plain, ties = plain, pad = plain;
      for (int i = 0; i < vocab / 2; ++i) half[i] = -INFINITY;
      for (int i = 0; i < vocab; ++i) {
        if (i % 3 == 0) steps[i] = -powf(10.0f, (float)(i % 38));
        ties[i] = roundf(plain[i]);
        if (i > vocab - vocab / 30) pad[i] = -0x1.fffffep127f;
      }
      std::vector<float> spread(vocab);                  // a third of all powers of two, of either sign
      for (float& v : spread) v = ldexpf(normal(rng), (int)(rng() % 80) - 40);
      const float inf = INFINITY, worst = -0x1.fffffep127f;
      std::vector<float> infinite = plain, far = plain;
      for (int i = 0; i < vocab; i += 1 + vocab / 90) infinite[i] = inf;
      for (float& v : far) v += 1e6f;
      for (int k : {1, 2, 50, 300, 768}) {
        check("as they come", plain, per, k);
        check("half of them never", half, per, k);
        check("90 % never", masked(0.9f, -inf), per, k);
        check("99 % never", masked(0.99f, -inf), per, k);
        check("90 % NaN", masked(0.9f, NAN), per, k);
        check("90 % of -1e9", masked(0.9f, -1e9f), per, k);
        check("90 % of -65504", masked(0.9f, -65504.0f), per, k);
        check("90 % of the least number", masked(0.9f, worst), per, k);
        check("a padded end", pad, per, k);
        check("-10^0 to -10^37", steps, per, k);
        check("of all magnitudes", spread, per, k);
        check("min_p", plain, per, k, 3.0f);
        check("min_p behind a mask", masked(0.9f, -1e9f), per, k, 0.5f);
        check("equal ones", ties, per, k);
        check("all the same", std::vector<float>(vocab, -3.5f), per, k);
        check("zeros of both signs", std::vector<float>(vocab, -0.0f), per, k);
        check("infinite", infinite, per, k);
        check("all infinite", std::vector<float>(vocab, inf), per, k);
        check("far from 0", far, per, k);
        check("both ends", [&] { auto y = masked(0.5f, worst); y[0] = -worst; return y; }(), per, k);
      }
    }
  if (failures) return printf("failed: %d rows\n", failures), 1;
  printf("ok\n");
}
