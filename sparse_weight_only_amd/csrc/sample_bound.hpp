// Which logits of a row are listed for its top_k: plain arithmetic, compiled into
// the kernel and, for its tests, for the CPU.
#pragma once
#include <math.h>
#include <stdint.h>

#include "decode_index.hpp"

namespace sgemv_dev {

constexpr int kSampleLanes = 1024, kSampleWaves = kSampleLanes / 64;
constexpr int kMostListed = 8192;

// Whole numbers in the order of the floats; both zeros the same, NaN as -inf.
SGEMV_BOTH uint32_t key_of(float x) {
  x = x != x ? -__builtin_inff() : x + 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return b >> 31 ? ~b : b | 0x80000000u;
}
SGEMV_BOTH float of_key(uint32_t k) { return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kNeverKey = 0x007fffffu;          // the key of -inf

// A wave's stretch of the row, in whole steps of the wave: 64 lanes, `per` logits each.
SGEMV_BOTH int stretch_of(int vocab, int per) { return (vocab + kSampleWaves * 64 * per - 1) / (kSampleWaves * 64 * per) * (64 * per); }

// What a lane's largest logit adds to the search for the smallest of them, as
// the largest of complements. A lane without a logit adds nothing.
SGEMV_BOTH uint32_t low_part(uint32_t key) { return key > kNeverKey ? ~key : 0; }

// At least k of a row's logits are as large as the k-th largest of the lanes' own
// largest, so a bound just below that one leaves k of them and hardly more. It
// is found by counting the lanes' largest in kSampleLanes intervals, the largest
// first: LogitBins of equal width between the largest and the smallest of them,
// and where the interval with the k-th holds more than kCrowd (one lane that has
// only tokens of -1e9 makes all others one interval) KeyBins, of that interval
// alone and in the order of the floats, whatever their magnitudes.
constexpr int kCrowd = 64, kKeyRounds = 4;           // 32 bits, 10 a round

struct LogitBins {
  float hi, lo, by;
  SGEMV_BOTH LogitBins(float top, float low) : hi(top), lo(low), by((float)kSampleLanes / (top - low)) {}
  // no number (0 by infinity, infinities less each other): 0
  SGEMV_BOTH int bin(float x) const { return (int)fminf(fmaxf((hi - x) * by, 0.0f), kSampleLanes - 1.0f); }
  // A logit that all lanes of intervals up to `at` reach: one of a later interval
  // (bin() never falls where x does), or the smallest of all.
  SGEMV_BOTH float lower(int at) const {
    if (at >= kSampleLanes - 1) return lo;
    float x = hi - (at + 1.0f) / by;
    for (uint32_t step = 1; x > lo && bin(x) <= at; step *= 2) x = step < 1u << 20 ? of_key(key_of(x) - step) : lo;
    return fmaxf(x, lo);
  }
};

struct KeyBins {
  uint32_t top, low;
  int shift;
  SGEMV_BOTH KeyBins(uint32_t top_, uint32_t low_) { set(top_, low_); }
  SGEMV_BOTH void set(uint32_t top_, uint32_t low_) {
    top = top_;
    low = low_;
    const uint32_t span = top - low;
    const int bits = span ? 32 - __builtin_clz(span) : 0;
    shift = bits > 10 ? bits - 10 : 0;
  }
  SGEMV_BOTH int bin(uint32_t key) const { return (int)((top - key) >> shift); }
  // on to the keys of interval `at`, to be split in their turn
  SGEMV_BOTH void narrow(int at) {
    const uint32_t from = top - ((uint32_t)at << shift), rest = (1u << shift) - 1;
    set(from, from - low > rest ? from - rest : low);
  }
};

}  // namespace sgemv_dev
