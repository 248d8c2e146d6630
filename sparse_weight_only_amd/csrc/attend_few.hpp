// Attention of few rows (one token, a few candidates) over a paged cache.
#pragma once
#include <type_traits>

#include "attend_device.hpp"

namespace sgemv_dev {

constexpr int kFewRows = 16, kFewBlock = 32;
// eight waves, or as many as 256 columns leave registers for
template <int DP> constexpr int kFewWaves = DP == 256 ? 4 : 8;

// One workgroup: a tile of 16 rows and one split of its keys; its waves take
// blocks of 32 keys in turn and meet in LDS at the end. Bound by reading K and
// V once: the operands come straight from memory, 16 bytes a lane, in the order
// the matrix cores want them, with the next block's loads in flight (a wave has
// 32 KiB of 128-column K and V in registers, a compute unit 256 KiB).
//   K (16 keys x 32 columns): lane r + 16 g has key r, columns 8 g ..;
//   V^T (16 columns x 32 keys): lane r + 16 g has the keys of group g and the
//   columns DP/16 r .., so a load is again one row's run, and a step for
//   column c of each run is put together from two rows at a time (v_perm).
// One row over 131071 slots of 8 heads of 128 columns: 95 us with its join, of
// which 5 join; 5.65 TB/s, where plain reads reach 6.3 to 6.5. 16 rows of 32
// heads each, token-major, where a head's rows are 256 bytes at strides of
// 8 KiB: 4.7 TB/s (5.3 head-major).
//
// EIGHT: the cache holds codes of 8 bits. A lane's 16 bytes of K are then 16
// columns, 8 for each of two steps, so the columns of q go by them; the codes of
// two of V's rows are put together before they are converted. A block's scale of
// K goes to the scores (one factor for 4 keys), that of V into the conversion,
// which takes it for nothing; sums are in units of the largest so far. Half the
// bytes, and 382 vector instructions for a wave's 32 keys: with the same 128
// columns, one row over 131071 slots of 8 heads takes 53 us with its join (head-major;
// 5.1 TB/s), 16 rows of 32 heads over up to 2500 slots 58 (3.6 TB/s;
// head-major 47: a head's row is 128 bytes in 4 KiB else, and reads of 128 bytes
// reach less). Tried: three blocks in flight (58.2 -> 59.5, 53.4 -> 54.5), two
// workgroups a compute unit with one block each (58.2 -> 65.9), 4 waves (60), all
// heads of a token in one XCD (59.3).
//
// WINDOW: key numbers leave out what no row of the tile sees. 16 rows of 8 heads
// of 4 over a window of 4096 and 4 sinks of 60000 slots: 52.4 us and 4.8 of join,
// 5.1 TB/s of the keys that are seen, as without a window over as many.
template <class T, int DP, bool WHOLE, bool EIGHT, bool WINDOW>
struct Few {
  using Elem = std::conditional_t<EIGHT, uint8_t, uint16_t>;
  static constexpr int W = kFewWaves<DP>;
  static constexpr int KC = DP / 32;      // K steps: 16-byte pieces of a key in a lane
  static constexpr int VC = DP / 16;      // columns of V in a lane = 16-column tiles of the output
  static constexpr int VD = VC / 2;       // dwords of them

  struct Block {
    dword4 k[2][EIGHT ? KC / 2 : KC];
    uint32_t v[8][EIGHT ? VD / 2 : VD];
    uint32_t there;                       // bit b: key b of the block exists
    uint32_t e[EIGHT ? 2 : 1];            // EIGHT: the exponents of the lane's runs of 4 keys, K's and V's
  };
  struct Rows { int k[2], v[2]; };        // page of the lane's keys: K rows, V runs of 4

  const AttendParams& p;
  const Tile& t;
  const Elem *kh, *vh;                    // this head's K and V
  const uint16_t* eh;                     // EIGHT: its exponents
  int r, g;                               // lane = r + 16 g
  dword4 q[KC];
  f32x4 o[VC];
  float m, l;                             // where the weights are 1 (kLift below the maximum), and this lane's share of the sum
  int unit, least;                        // EIGHT: exponent that `o` is in units of, and the least that counts of the lane's runs (biased)
  int from;                               // WINDOW: the first slot behind the sinks that the lane's row sees

  __device__ __forceinline__ Few(const AttendParams& p_, const Tile& t_, int head) : p(p_), t(t_) {
    const int lane = threadIdx.x & 63;
    r = lane & 15;
    g = lane >> 4;
    kh = (const Elem*)p.k + head * p.k_head;
    vh = (const Elem*)p.v + head * p.v_head;
    eh = EIGHT ? p.exps + head : nullptr;
    // rows past the sequence repeat its last one and are not stored
    const int row = t.row0 + r < t.rows ? t.row0 + r : t.rows - 1;
    const uint16_t* qr = p.q + (int64_t)(t.first + row / p.group) * p.q_token + (int64_t)(head * p.group + row % p.group) * p.q_head;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const int d = EIGHT ? 64 * (c / 2) + 16 * g + 8 * (c % 2) : 32 * c + 8 * g;
      q[c] = columns<dword4>(addr(qr), d);
    }
    from = WINDOW ? window_from(p, t, row / p.group) : 0;
  }

  // columns d .. of a row; zeros past the head's own where it is narrower than DP
  template <class V, class E = uint16_t>
  __device__ __forceinline__ V columns(addr_t row, int d) const {
    return load<V>(WHOLE ? row + sizeof(E) * d : or_nothing(d < p.dim, row + sizeof(E) * d));
  }
  __device__ __forceinline__ int slot(int key) const { return slot_of<WINDOW>(t, key); }
  // a key past the end looks up the last one's page
  __device__ __forceinline__ int page_of(int key) const { return t.pages[slot(key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift]; }
  __device__ __forceinline__ Rows lookup(int kb) const {
    Rows w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.k[i] = page_of(kb + 16 * i + r);
      w.v[i] = page_of(kb + 16 * i + 4 * g);   // pages hold at least 8 slots: a run of 4 lies in one
    }
    return w;
  }
  __device__ __forceinline__ void fetch(int kb, const Rows& w, Block& b) const {
    const int in_page = (1 << p.seq.page_shift) - 1;
    uint32_t there = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = kb + 16 * i + r;
      const bool ok = key < t.key1 && p.seq.page_ok(w.k[i]);
      there |= (uint32_t)(__ballot(ok) & 0xffffu) << (16 * i);
      const addr_t row = or_nothing(ok, addr(kh + element(w.k[i], p.k_page, slot(key) & in_page, p.k_slot)));
#pragma unroll
      for (int c = 0; c < (EIGHT ? KC / 2 : KC); ++c) b.k[i][c] = columns<dword4, Elem>(row, EIGHT ? 64 * c + 16 * g : 32 * c + 8 * g);
    }
    b.there = there;
    if constexpr (EIGHT) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // a run that is not there, or that no row sees, has no exponents
        const int key = kb + 16 * i + 4 * g, at = slot(key);
        const bool ok = key < t.key1 && p.seq.page_ok(w.v[i]) && (!WINDOW || at < p.sinks || at + 3 >= t.low);
        const uint64_t block = (uint64_t)(uint32_t)w.v[i] * p.exp_page + (uint64_t)(uint32_t)((at & in_page) >> p.exp_shift) * (uint32_t)p.heads;
        b.e[i] = load<uint16_t>(or_nothing(ok, addr(eh + block)));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = kb + 16 * (j / 4) + 4 * g + j % 4;
      const bool ok = key < t.key1 && p.seq.page_ok(w.v[j / 4]);
      const addr_t row = or_nothing(ok, addr(vh + element(w.v[j / 4], p.v_page, slot(key) & in_page, p.v_slot)));
      if constexpr (EIGHT) {
        if constexpr (VC == 4) {
          b.v[j][0] = columns<uint32_t, Elem>(row, 4 * r);
        } else if constexpr (VC == 8) {
          const dword2 x = columns<dword2, Elem>(row, 8 * r);
          b.v[j][0] = x.x;
          b.v[j][1] = x.y;
        } else {
          const dword4 x = columns<dword4, Elem>(row, 16 * r);
#pragma unroll
          for (int e = 0; e < 4; ++e) b.v[j][e] = x[e];
        }
      } else if constexpr (VC == 4) {
        const dword2 x = columns<dword2>(row, 4 * r);
        b.v[j][0] = x.x;
        b.v[j][1] = x.y;
      } else {
#pragma unroll
        for (int u = 0; u < VC / 8; ++u) {
          const dword4 x = columns<dword4>(row, VC * r + 8 * u);
#pragma unroll
          for (int e = 0; e < 4; ++e) b.v[j][4 * u + e] = x[e];
        }
      }
    }
  }

  // bit b: whether row r sees key b of the block at kb
  __device__ __forceinline__ uint32_t visible(int kb) const {
    const int row = t.row0 + r < t.rows ? t.row0 + r : t.rows - 1;
    const uint32_t bits = visible_bits(p, t, row / p.group, slot(kb));
    return WINDOW ? bits & window_bits(p.sinks, from, slot(kb)) : bits;
  }
  // scores of the block's keys 16 i + 4 g + e for row r, -inf where not seen
  // (EIGHT: in units of the keys' own scales)
  __device__ __forceinline__ void scores(int kb, const Block& b, float (&s)[8]) const {
    f32x4 a[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      if constexpr (EIGHT) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const dword4 x = b.k[i][c / 2];
          a[i] = Half<T>::mma16(c % 2 ? eight<T>(x[2], x[3], 1.0f) : eight<T>(x[0], x[1], 1.0f), q[c], a[i]);
        }
      } else {
        a[0] = Half<T>::mma16(b.k[0][c], q[c], a[0]);
        a[1] = Half<T>::mma16(b.k[1][c], q[c], a[1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = a[e / 4][e % 4];
    if (needs_mask<WINDOW>(p, t, slot(kb), kFewBlock) || b.there != ~0u) {
      const uint32_t bits = visible(kb) & b.there;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(bits >> (16 * (e / 4) + 4 * g + e % 4) & 1u)) s[e] = -__builtin_inff();
    }
  }

  // factors that take the scores of the lane's two runs to powers of two
  __device__ __forceinline__ void factors(const Block& b, float (&by)[2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) by[i] = EIGHT ? score_scale(p.scale2, (int)(b.e[EIGHT ? i : 0] & 255u)) : p.scale2;
  }
  // EIGHT: sees to it that `o` is in units that the block's values do not exceed
  __device__ __forceinline__ void raise(const Block& b, int (&ev)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ev[i] = (int)(b.e[EIGHT ? i : 0] >> 8);
      least = ev[i] > Eight<T>::kTiny && ev[i] < least ? ev[i] : least;
    }
    const int top = ev[0] > ev[1] ? ev[0] : ev[1];
    if (__any(top > unit)) {
      const int to = top_of_groups(top > unit ? top : unit);
      const float by = below(unit, to);
#pragma unroll
      for (int c = 0; c < VC; ++c) o[c] *= by;
      unit = to;
    }
  }

  __device__ __forceinline__ void add(int kb, const Block& b) {
    float s[8], sc[2];
    scores(kb, b, s);
    factors(b, sc);
    float top;
    if constexpr (EIGHT) {
      top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) * sc[0], fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])) * sc[1]);
      top = max_x32(max_x16(top)) - Half<T>::kLift;
    } else {
      top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
      top = __builtin_fmaf(max_x32(max_x16(top)), p.scale2, -Half<T>::kLift);
    }
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top), by = m == to ? 1.0f : exp2_fast(m - to);
      l *= by;
#pragma unroll
      for (int c = 0; c < VC; ++c) o[c] *= by;
      m = to;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
    dword4 pb;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pb[e] = Half<T>::pack(exp2_fast(__builtin_fmaf(s[2 * e], sc[e / 2], -base)), exp2_fast(__builtin_fmaf(s[2 * e + 1], sc[e / 2], -base)));
      sum = Half<T>::sum(pb[e], sum);
    }
    l += sum;
    if constexpr (EIGHT) {
      int ev[2];
      raise(b, ev);
      const float by[2] = {below(ev[0], unit), below(ev[1], unit)};
#pragma unroll
      for (int u = 0; u < VD / 2; ++u) {
        // columns 4 u .. of two keys at a time
        dword4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = __builtin_amdgcn_perm(b.v[2 * j + 1][u], b.v[2 * j][u], 0x05010400u);
          const uint32_t hi = __builtin_amdgcn_perm(b.v[2 * j + 1][u], b.v[2 * j][u], 0x07030602u);
          x[0][j] = Eight<T>::pair(lo, by[j / 2], false);
          x[1][j] = Eight<T>::pair(lo, by[j / 2], true);
          x[2][j] = Eight<T>::pair(hi, by[j / 2], false);
          x[3][j] = Eight<T>::pair(hi, by[j / 2], true);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) o[4 * u + c] = Half<T>::mma16(x[c], pb, o[4 * u + c]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < VD; ++u) {
        dword4 lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = __builtin_amdgcn_perm(b.v[2 * j + 1][u], b.v[2 * j][u], 0x05040100u);
          hi[j] = __builtin_amdgcn_perm(b.v[2 * j + 1][u], b.v[2 * j][u], 0x07060302u);
        }
        o[2 * u] = Half<T>::mma16(lo, pb, o[2 * u]);
        o[2 * u + 1] = Half<T>::mma16(hi, pb, o[2 * u + 1]);
      }
    }
  }

  // The same sums again, key by key, each row adding the keys it sees and no
  // other: a matrix product adds 0 * v for the others, which is not 0 where v
  // is infinite or not a number. Only for a tile whose sums are not finite
  // (EIGHT: or whose exponents lie too far apart; `o` is in units of 1 then).
  __device__ __forceinline__ void add_seen_only(int kb) {
    Block b;
    fetch(kb, lookup(kb), b);
    float s[8], sc[2];
    scores(kb, b, s);
    factors(b, sc);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    // a key that is seen may have a score of -inf too
    const uint32_t bits = visible(kb) & b.there;
    for (int key = 0; key < kFewBlock; ++key) {
      // the lane that holds this key's score for row r
      const int from = r + 16 * (key / 4 % 4), e = key % 4;
      const float s0 = e == 0 ? s[0] : e == 1 ? s[1] : e == 2 ? s[2] : s[3];
      const float s1 = e == 0 ? s[4] : e == 1 ? s[5] : e == 2 ? s[6] : s[7];
      const float sk = __shfl(key < 16 ? s0 : s1, from);
      const float scale2 = EIGHT ? __shfl(key < 16 ? sc[0] : sc[1], from) : p.scale2;
      const int ev = EIGHT ? __shfl((int)((key < 16 ? b.e[0] : b.e[EIGHT ? 1 : 0]) >> 8), from) - 127 : 0;
      if (!(b.there >> key & 1u)) continue;
      const int at = slot(kb + key), page = t.pages[at >> p.seq.page_shift];
      const Elem* vr = vh + element(page, p.v_page, at & ((1 << p.seq.page_shift) - 1), p.v_slot);
      if (!(bits >> key & 1u)) continue;
      const float pk = exp2_fast(__builtin_fmaf(sk, scale2, -base));
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
#pragma unroll
        for (int u = 0; u < VD; ++u) {
          const int d = (4 * g + e4) * VC + 2 * u;
          if (d >= p.dim) continue;
          if constexpr (EIGHT) {
            const uint32_t w = Eight<T>::pair(load<uint16_t>(addr(vr + d)), 1.0f, false);
            o[2 * u][e4] += pk * __builtin_amdgcn_ldexpf(Half<T>::lo(w), ev);
            o[2 * u + 1][e4] += pk * __builtin_amdgcn_ldexpf(Half<T>::hi(w), ev);
          } else {
            const uint32_t w = load<uint32_t>(addr(vr + d));
            o[2 * u][e4] += pk * Half<T>::lo(w);
            o[2 * u + 1][e4] += pk * Half<T>::hi(w);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < VC; ++c) o[c] = f32x4{0, 0, 0, 0};
  }

  __device__ __forceinline__ void walk(int wave) {
    m = -__builtin_inff();
    l = 0.0f;
    unit = 0;
    least = 255;
    clear();
    constexpr int step = kFewBlock * W;
    int kb = t.key0 + wave * kFewBlock;
    if (kb < t.key1) {
      Block a, b;
      // pages are looked up two blocks ahead, before the loads of the next
      // block: loads return in order, so one that was issued later could not
      // be waited for without waiting for that block too
      Rows w = lookup(kb), next = lookup(kb + step);
      fetch(kb, w, a);
      while (true) {
        w = lookup(kb + 2 * step);
        fetch(kb + step, next, b);
        add(kb, a);
        if ((kb += step) >= t.key1) break;
        next = lookup(kb + 2 * step);
        fetch(kb + step, w, a);
        add(kb, b);
        if ((kb += step) >= t.key1) break;
      }
      bool bad = false;
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= not_finite(o[c][e]);
      if (EIGHT) bad |= unit - least > Eight<T>::kSpread;
      if (__any(bad)) {
        clear();
        unit = 127;
        for (kb = t.key0 + wave * kFewBlock; kb < t.key1; kb += step) add_seen_only(kb);
      }
      if (EIGHT) {
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][e] = __builtin_amdgcn_ldexpf(o[c][e], unit - 127);
      }
    }
    l = sum_x32(sum_x16(l));
  }
};

template <class T, int DP, bool WHOLE, bool EIGHT, bool WINDOW>
__global__ void __launch_bounds__(64 * kFewWaves<DP>, DP == 256 ? 1 : 2) attend_few_kernel(AttendParams p) {
  constexpr int VC = DP / 16, W = kFewWaves<DP>;
  __shared__ float sums[W][kFewRows][DP + 4];
  __shared__ float stat_m[W][kFewRows], stat_l[W][kFewRows];
  const int id = blockIdx.x, head = id % p.heads, split = id / p.heads % p.splits, slot = id / p.heads / p.splits;
  Tile t;
  if (!find_tile<kFewRows, WINDOW>(p, kFewBlock, slot, split, t)) return;
  if (p.splits > 1 && t.key0 >= t.key1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  {
    Few<T, DP, WHOLE, EIGHT, WINDOW> f(p, t, head);
    f.walk(wave);
    if (f.g == 0) {
      stat_m[wave][f.r] = f.m;
      stat_l[wave][f.r] = f.l;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int c = 0; c < VC; c += 4)
        *(f32x4*)&sums[wave][f.r][(4 * f.g + e) * VC + c] = f32x4{f.o[c][e], f.o[c + 1][e], f.o[c + 2][e], f.o[c + 3][e]};
  }
  __syncthreads();
  // 4 W lanes a row
  constexpr int PER = 4 * W;
  const int row = threadIdx.x / PER, at_row = threadIdx.x % PER, r = t.row0 + row;
  if (r >= t.rows) return;
  float top = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < W; ++w) top = fmaxf(top, stat_m[w][row]);
  float by[W], l = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    // a wave without a visible key has sums of zero (or, seeing keys whose
    // scores are not numbers, sums that have to stay so)
    by[w] = stat_m[w][row] == top ? 1.0f : exp2_fast(stat_m[w][row] - top);
    l += by[w] * stat_l[w][row];
  }
  const int tok = t.first + r / p.group, hq = head * p.group + r % p.group;
  const int64_t at = (int64_t)tok * p.heads * p.group + hq;
  if (p.splits > 1 && at_row == 0) {
    float* st = part_stats(p, at, split);
    st[0] = top;
    st[1] = l;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  for (int d = at_row * 4; d < p.dim; d += PER * 4) {
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w) x += by[w] * *(const f32x4*)&sums[w][row][d];
    if (p.splits > 1)
      *(f32x4*)(part_sums(p, at, split) + d) = x;
    else
      *(dword2*)(p.out + tok * p.o_token + hq * p.o_head + d) = dword2{Half<T>::pack(x[0] * inv, x[1] * inv), Half<T>::pack(x[2] * inv, x[3] * inv)};
  }
}

}  // namespace sgemv_dev
