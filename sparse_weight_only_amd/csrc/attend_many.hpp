// Attention of many rows (a chunk of a prompt) over a paged cache.
#pragma once
#include <type_traits>

#include "attend_device.hpp"

namespace sgemv_dev {

constexpr int kManyWaves = 8, kManyStages = 4;
template <bool HALVES> constexpr int kManyRows = 32 * kManyWaves / (HALVES ? 2 : 1);
template <int DP> constexpr int kManyBlock = DP == 256 ? 32 : 64;
template <int DP> constexpr int kManyLds = kManyStages * 2 * kManyBlock<DP> * DP * 2;   // K and V of each stage

// One workgroup: a tile of 32 rows a wave and one split of its keys, in blocks
// of 64 (32 for the widest heads) that all waves share through LDS. Bound by
// the matrix cores and, as much, by the exponentials and what is around them
// on the vector units, which one wave cannot keep busy together. So the waves
// take turns: while waves 0..3, one on each SIMD, are at the products (of the
// last block's weights with V, of q with the next block's K), waves 4..7 are
// at the softmax, and the other way round, a barrier at each change.
//
// HALVES, for tiles of up to 128 rows: waves 4..7 have the rows of waves 0..3
// and every wave half of a block's keys; the two meet in LDS at the end.
//
// K and V go from memory straight to LDS, two blocks ahead (a block is computed
// in less time than its loads take). The loads are issued and waited for here,
// not by the compiler, which would wait for all of them before any LDS read.
// Every fetch is the same number of loads, past the end too, so that a wait
// for all but the last so many is a wait for the block at hand. Rows of a stage
// are 2 DP bytes; the 16-byte pieces of a row are stored in an order that depends on
// the key (K: xor of the piece with the key; V: of the piece's group of four),
// so that the lanes of an operand read, which are at the same columns of
// different keys, fall on different banks. V's operand, 4 keys of one column a
// lane, is read with the transposing LDS load: of its 16 lanes, lane 4 i + j
// names key i's columns 4 j .., and lane c gets column c of the 4 keys.
//
// EIGHT: the cache holds codes of 8 bits. They come through registers, a
// block or two ahead, are converted once for all waves and written to the same
// places of LDS (every wave converting what it reads would take as many vector
// operations as its softmax). Each wave brings 8 keys of a block (4 of the
// widest), which share their exponents; of the block's others it reads the
// exponents alone, so that all waves agree on the units. The conversion adds a
// third to the vector instructions: a prompt of 8192 and 32 heads of 128 columns
// takes 616 us where 16 bits take 594 (matrix cores busy 40 % and 54 % of the
// time), 4096 and 16 heads 140 against 112, of 64 columns 93 and 82, of 256 345 and
// 217. Full tiles of 64 columns spill 12 to 21 registers and 256 columns 29 to 44
// (none in 16 bits) around the exact pass, which is inlined.
// WINDOW: key numbers leave out what no row of the tile sees. Two prompts of up to
// 6001 tokens and 16 heads of 64 columns through a window of 1024: 84 us, 458
// TFLOP/s of what is seen, which is what this width reaches without a window.
template <class T, int DP, bool WHOLE, bool HALVES, bool EIGHT, bool WINDOW>
struct Many {
  using Elem = std::conditional_t<EIGHT, uint8_t, uint16_t>;
  static constexpr int W = kManyWaves, ST = kManyStages, B = kManyBlock<DP>;
  static constexpr int KC = DP / 16, OT = DP / 32;
  static constexpr int NS = B / 32 / (HALVES ? 2 : 1), KS = 2 * NS;   // 32-key and 16-key steps of a wave in a block
  static constexpr int PIECES = DP / 8;                  // 16-byte pieces of a row
  static constexpr int ROWS = 64 / PIECES;               // rows that one load of a wave fills
  static constexpr int LOADS = B / ROWS / W;             // loads of a wave, for K and for V
  static constexpr int STAGE = B * DP;                   // elements of K or V in a stage

  static __device__ __forceinline__ int k_mix(int key) { return DP == 64 ? key >> 1 & 7 : key & 15; }
  static __device__ __forceinline__ int v_mix(int key) { return DP == 64 ? (key >> 1 & 1) * 4 : (key & 3) * 4; }

  const AttendParams& p;
  const Tile& t;
  const Elem *kh, *vh;
  const uint16_t* eh;                                    // EIGHT: the head's exponents
  uint32_t lds;                                          // LDS address of the stages
  const uint16_t* lds_p;
  int lane, wave, c, h;                                  // lane = c + 32 h: row c of the wave
  int part;                                              // HALVES: which half of a block's keys, 0 or 1; else 0
  int row0, row;                                         // the wave's first row; the lane's, clamped to the sequence
  dword4 q[KC];
  f32x16 s[NS];                                          // scores of a block: key 32 i + (8 a + 4 h + e) at s[i][4 a + e]
  dword4 w[KS];                                          // weights of a block, as the second product takes them
  f32x16 o[OT];
  float m, l;
  int from;                                              // WINDOW: the first slot behind the sinks that the row sees
  // EIGHT (exponents are biased): what `o` is in units of; the largest of K and
  // of V so far, which is what LDS holds a block in units of; the least that count
  int unit, k_top, v_top, k_least, v_least;
  int k_tiny;                                            // and up to where those of K do not

  __device__ __forceinline__ Many(const AttendParams& p_, const Tile& t_, int head, uint16_t* lds_) : p(p_), t(t_), lds_p(lds_) {
    lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds_;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c = lane & 31;
    h = lane >> 5;
    kh = (const Elem*)p.k + head * p.k_head;
    vh = (const Elem*)p.v + head * p.v_head;
    eh = EIGHT ? p.exps + head : nullptr;
    part = HALVES ? wave / (W / 2) : 0;
    row0 = t.row0 + 32 * (HALVES ? wave % (W / 2) : wave);
    row = row0 + c < t.rows ? row0 + c : t.rows - 1;
    const uint16_t* qr = p.q + (int64_t)(t.first + row / p.group) * p.q_token + (int64_t)(head * p.group + row % p.group) * p.q_head;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int d = 16 * i + 8 * h;
      q[i] = load<dword4>(or_nothing(WHOLE || d < p.dim, addr(qr + d)));
    }
    from = WINDOW ? window_from(p, t, row / p.group) : 0;
  }

  __device__ __forceinline__ int slot(int key) const { return slot_of<WINDOW>(t, key); }

  // Pages of the rows that this wave fetches of the block at kb (past the end:
  // the last key's). The rows of one load lie in one page (pages hold at least
  // 8 slots), so this is scalar work.
  struct Pages { int at[LOADS]; };
  __device__ __forceinline__ Pages lookup(int kb) const {
    const __attribute__((address_space(4))) int32_t* table = (const __attribute__((address_space(4))) int32_t*)(uint64_t)t.pages;
    Pages w;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int key = kb + (i * W + wave) * ROWS;
      w.at[i] = table[__builtin_amdgcn_readfirstlane(slot(key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift)];
    }
    return w;
  }
  // starts the loads of the block at kb into a stage; `w` from lookup(kb)
  __device__ __forceinline__ void fetch(int kb, const Pages& w, int stage) const {
    const int in_page = (1 << p.seq.page_shift) - 1;
    const uint32_t ks = lds + stage * 2 * STAGE * 2, vs = ks + STAGE * 2;
    const int row = lane / PIECES, piece = lane % PIECES;
    const bool full = WHOLE && kb + B <= t.key1;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int first = (i * W + wave) * ROWS, key = first + row;
      const int dk = (piece ^ k_mix(key)) * 8, dv = (piece ^ v_mix(key)) * 8;
      const int pg = w.at[i], at = (slot(kb) + first) & in_page;
      const bool ok = p.seq.page_ok(pg);
      const addr_t kr = addr(kh + element(pg, p.k_page, at, p.k_slot)), vr = addr(vh + element(pg, p.v_page, at, p.v_slot));
      const uint32_t ko = 2 * (row * p.k_slot + dk), vo = 2 * (row * p.v_slot + dv);
      if (full && ok) {
        to_lds(kr, ko, ks + first * DP * 2);
        to_lds(vr, vo, vs + first * DP * 2);
      } else {
        const bool in = ok && kb + key < t.key1;
        to_lds(or_nothing(in && (WHOLE || dk < p.dim), kr + ko), ks + first * DP * 2);
        to_lds(or_nothing(in && (WHOLE || dv < p.dim), vr + vo), vs + first * DP * 2);
      }
    }
  }
  // 16 bytes a lane from memory to LDS: lane i's go to `to` + 16 i. No register
  // receives anything; walk() waits.
  static __device__ __forceinline__ void to_lds(uint64_t base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
  }
  static __device__ __forceinline__ void to_lds(addr_t from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
  }

  // which keys of the block at kb exist; `sound`: no page of the tile is missing
  __device__ __forceinline__ uint64_t there(int kb, bool sound) const {
    const int n = t.key1 - kb;
    uint64_t bits = n >= 64 ? ~0ull : (1ull << n) - 1;
    if (!sound) {
      const int key = kb + lane;
      bits &= __ballot(p.seq.page_ok(t.pages[slot(key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift]));
    }
    return B == 64 ? bits : bits | ~0ull << 32;
  }
  __device__ __forceinline__ bool pages_sound() const {
    const int last = slot(t.key1 - 1) >> p.seq.page_shift;
    bool ok = true;
#pragma unroll 4
    for (int i = (slot(t.key0) >> p.seq.page_shift) + lane; i <= last; i += 64) {
      // pages that a window leaves out altogether may have been given back
      if (WINDOW && (int64_t)i << p.seq.page_shift >= t.gap0 && (int64_t)(i + 1) << p.seq.page_shift <= (int64_t)t.gap0 + t.gap) continue;
      ok &= p.seq.page_ok(t.pages[i]);
    }
    return __all(ok);
  }

  // bit b: whether the lane's row sees key number kb + b
  __device__ __forceinline__ uint32_t visible(int kb) const {
    const uint32_t bits = visible_bits(p, t, row / p.group, slot(kb));
    return WINDOW ? bits & window_bits(p.sinks, from, slot(kb)) : bits;
  }
  // -inf for the keys of the block at kb that the lane's row does not see
  __device__ __forceinline__ void mask(int kb, uint64_t there) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int at = 32 * (i + part);
      const uint32_t bits = (visible(kb + at) & (uint32_t)(there >> at)) >> (4 * h);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!(bits >> (8 * (e / 4) + e % 4) & 1u)) s[i][e] = -__builtin_inff();
    }
  }

  // LDS addresses of operands: kept in registers over the whole walk, as the
  // compiler would, or put together where they are used, a vector operation
  // each that is hidden from it. The latter where registers are short (256
  // columns spilled: 327 us, 220 without, for 4096 x 4096 and 16 heads) or the
  // vector units wait for the matrix cores anyway (64 columns: 74 against
  // 80 us; halves: 33.8 against 35.0); with 128 columns and full tiles the
  // operations cost more than they free (685 against 572 us for a prompt of
  // 8192 and 32 heads).
  static __device__ __forceinline__ uint32_t fresh(uint32_t x) {
    if constexpr (DP != 128 || HALVES) asm volatile("" : "+v"(x));
    return x;
  }

  // s = the scores of the block in a stage
  __device__ __forceinline__ void first_product(int stage) {
    const uint32_t row = lds + stage * 4 * STAGE + (32 * part + c) * DP * 2;
    const uint32_t mix = fresh((h ^ k_mix(c)) * 16);       // of piece 2 j + h: (32 j) ^ mix
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = f32x16{};
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int i = 0; i < NS; ++i) s[i] = Half<T>::mma32(lds_load((32 * j ^ mix) + row + 32 * i * DP * 2), q[j], s[i]);
  }

  // w = the weights of the block at kb from its scores, and m and the sum with
  // it
  __device__ __forceinline__ void softmax(int kb, uint64_t there, float scale2) {
    if (needs_mask<WINDOW>(p, t, slot(kb), B) || there != ~0ull) mask(kb, there);
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 16 * NS; ++e) top = fmaxf(top, s[e / 16][e % 16]);
    top = __builtin_fmaf(max_x32(top), scale2, -Half<T>::kLift);
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top), by = m == to ? 1.0f : exp2_fast(m - to);
      l *= by;
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i] *= by;
      m = to;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16 * NS; e += 2) {
      const float a = exp2_fast(__builtin_fmaf(s[e / 16][e % 16], scale2, -base));
      const float b = exp2_fast(__builtin_fmaf(s[e / 16][e % 16 + 1], scale2, -base));
      const uint32_t ab = Half<T>::pack(a, b);
      sum[e / 2 % 2] = Half<T>::sum(ab, sum[e / 2 % 2]);
      w[e / 8][e % 8 / 2] = ab;
    }
    l += sum[0] + sum[1];
  }

  // o += the weights times V of the block in a stage
  __device__ __forceinline__ void second_product(int stage) {
    const int key = 4 * h + (lane & 15) / 4;
    const uint32_t row = lds + stage * 4 * STAGE + 2 * STAGE + (32 * part + key) * DP * 2 + 8 * (lane & 1);
    const uint32_t mix = fresh((v_mix(key) ^ (2 * (lane >> 4 & 1) + (lane >> 1 & 1))) * 16);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        const uint32_t at = (64 * i ^ mix) + row + 16 * k * DP * 2;
        const dword2 x = transposed(at), y = transposed(at + 8 * DP * 2);
        o[i] = Half<T>::mma32(dword4{x.x, x.y, y.x, y.y}, w[k], o[i]);
      }
  }

  // The products of a step: o += weights V of one block, s = scores of the
  // next. A wave has its SIMD's matrix core for itself here, so the LDS reads
  // of an operand are put DEPTH products before the one that takes it (left
  // alone, the compiler waits for each read where it is used).
  __device__ __forceinline__ void products(int stage, int next) {
    constexpr int DEPTH = DP == 256 ? 2 : 4, SECOND = KS * OT, FIRST = NS * KC;
    second_product(stage);
    first_product(next);
    __builtin_amdgcn_sched_group_barrier(LDS_READ, 2 * DEPTH, 0);
#pragma unroll
    for (int n = 0; n < SECOND + FIRST; ++n) {
      __builtin_amdgcn_sched_group_barrier(MATRIX, 1, 0);
      if (n + DEPTH < SECOND) __builtin_amdgcn_sched_group_barrier(LDS_READ, 2, 0);
      else if (n + DEPTH < SECOND + FIRST) __builtin_amdgcn_sched_group_barrier(LDS_READ, 1, 0);
    }
  }
  static constexpr int MATRIX = 0x008, LDS_READ = 0x100;

  static __device__ __forceinline__ dword4 lds_load(uint32_t at) { return *(const __attribute__((address_space(3))) dword4*)at; }
  // 4 keys of one column: see above
  static __device__ __forceinline__ dword2 transposed(uint32_t at) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(dword2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
  }

  // The sums again, each row adding the keys it sees and no other (a matrix
  // product adds 0 * v for the others, which is not 0 where v is infinite or
  // not a number). From memory, 32 keys at a time; only for a wave whose sums
  // are not finite.
  __device__ __forceinline__ void walk_seen_only() {
    const int in_page = (1 << p.seq.page_shift) - 1;
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] = f32x16{};
    const float base = m == -__builtin_inff() ? 0.0f : m;
    for (int kb = t.key0 + 32 * part; kb < t.key1; kb += HALVES ? 64 : 32) {
      const int mine = kb + c, at = slot(mine);
      const int page = mine < t.key1 ? t.pages[at >> p.seq.page_shift] : -1;
      const bool ok = p.seq.page_ok(page);
      const uint32_t there = (uint32_t)__ballot(ok);
      const Elem* kr = kh + element(page, p.k_page, at & in_page, p.k_slot);
      f32x16 x = f32x16{};
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int d = 16 * j + 8 * h;
        x = Half<T>::mma32(load<dword4>(or_nothing(ok && (WHOLE || d < p.dim), addr(kr + d))), q[j], x);
      }
      const uint32_t bits = visible(kb) & there;
      for (int key = 0; key < 32; ++key) {
        // this key's score for row c, from the half that holds it
        const int e = key / 8 * 4 + key % 4;
        float sk = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sk = i == e ? x[i] : sk;
        sk = __shfl(sk, c + 32 * (key / 4 % 2));
        const int pg = __shfl(page, key);
        if (!(there >> key & 1u)) continue;
        const Elem* vr = vh + element(pg, p.v_page, slot(kb + key) & in_page, p.v_slot);
        const float pk = exp2_fast(__builtin_fmaf(sk, p.scale2, -base));
        if (bits >> key & 1u) {
#pragma unroll
          for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const int d = 32 * i + 8 * a + 4 * h;
              if (d >= p.dim) continue;
              const dword2 v = load<dword2>(addr(vr + d));
              o[i][4 * a] += pk * Half<T>::lo(v.x);
              o[i][4 * a + 1] += pk * Half<T>::hi(v.x);
              o[i][4 * a + 2] += pk * Half<T>::lo(v.y);
              o[i][4 * a + 3] += pk * Half<T>::hi(v.y);
            }
        }
      }
    }
  }

  // ---- EIGHT
  static constexpr int CP = DP == 64 ? 8 : 16;           // codes of a lane's piece
  static constexpr int ROW_LANES = DP / CP;
  static constexpr int WAVE_KEYS = 64 / ROW_LANES;       // keys of a block that a wave brings
  static constexpr int GROUPS = B / 8;                   // 8 keys in a row share their page and their exponents
  using Piece = std::conditional_t<DP == 64, dword2, dword4>;
  // blocks that are on their way in registers: as many as those leave room for
  static constexpr int DEEP = DP == 128 ? 2 : 1;
  struct Raw {
    Piece k, v;
    uint32_t e;                                          // exponents of group lane % GROUPS
    int keys;                                            // how many of the wave's keys there are
  };
  struct Units { int k, v; };                            // what a stage holds K and V in units of

  // the page of group lane % GROUPS of the block at kb (past the end: of the last key)
  __device__ __forceinline__ int lookup8(int kb) const {
    const int key = kb + 8 * (lane % GROUPS);
    return t.pages[slot(key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift];
  }
  __device__ __forceinline__ addr_t exps_at(int page, int at) const {
    const int in_page = (1 << p.seq.page_shift) - 1;
    return addr(eh + ((uint64_t)(uint32_t)page * p.exp_page + (uint64_t)(uint32_t)((at & in_page) >> p.exp_shift) * (uint32_t)p.heads));
  }
  // Starts the loads of the block at kb; `pages` from lookup8(kb). Keys behind the
  // end lie in the last key's page, and those of a page that is not there are read
  // from the first one: convert() leaves them out.
  __device__ __forceinline__ void fetch8(int kb, int pages, Raw& x) const {
    const int in_page = (1 << p.seq.page_shift) - 1;
    const int first = wave * WAVE_KEYS, key = lane / ROW_LANES, d = lane % ROW_LANES * CP, column = WHOLE || d < p.dim ? d : 0;
    const int pg = __builtin_amdgcn_readlane(pages, first / 8), at = (slot(kb) + first) & in_page;
    const bool ok = p.seq.page_ok(pg);
    x.keys = ok ? t.key1 - kb - first : 0;
    const int page = ok ? pg : 0;
    x.k = load<Piece>(addr(kh + element(page, p.k_page, at, p.k_slot)) + (uint32_t)(key * p.k_slot + column));
    x.v = load<Piece>(addr(vh + element(page, p.v_page, at, p.v_slot)) + (uint32_t)(key * p.v_slot + column));
    // a group that is not there, or that no row sees, has no exponents
    const int gk = kb + 8 * (lane % GROUPS), ga = slot(gk);
    const bool there = gk < t.key1 && p.seq.page_ok(pages) && (!WINDOW || ga < p.sinks || ga + 7 >= t.low);
    x.e = load<uint16_t>(or_nothing(there, exps_at(pages, ga)));
  }
  // converts a block that has come into a stage
  __device__ __forceinline__ Units convert(Raw& x, int stage) {
    const int key = lane / ROW_LANES, d = lane % ROW_LANES * CP;
    {
      const int ek = x.e & 255u, ev = x.e >> 8;
      const bool news = ek > k_top || ev > v_top || (ek > k_tiny && ek < k_least) || (ev > Eight<T>::kTiny && ev < v_least);
      if (__any(news)) {
#pragma unroll 1
        for (int g = 0; g < GROUPS; ++g) {
          const int e = __builtin_amdgcn_readlane(x.e, g), gk = e & 255, gv = e >> 8;
          k_top = gk > k_top ? gk : k_top;
          v_top = gv > v_top ? gv : v_top;
          k_least = gk > k_tiny && gk < k_least ? gk : k_least;
          v_least = gv > Eight<T>::kTiny && gv < v_least ? gv : v_least;
        }
      }
    }
    if (!WHOLE || x.keys < WAVE_KEYS) {
      const bool in = key < x.keys && (WHOLE || d < p.dim);
#pragma unroll
      for (int u = 0; u < CP / 4; ++u) {
        x.k[u] = in ? x.k[u] : 0;
        x.v[u] = in ? x.v[u] : 0;
      }
    }
    const int mine = __builtin_amdgcn_readlane(x.e, wave * WAVE_KEYS / 8);
    const float by_k = below(mine & 255, k_top), by_v = below(mine >> 8, v_top);
    const int row = wave * WAVE_KEYS + key, piece = d / 8;
    const uint32_t ks = lds + stage * 4 * STAGE + row * DP * 2, vs = ks + STAGE * 2;
    const uint32_t k_at = fresh((piece ^ k_mix(row)) * 16), v_at = fresh((piece ^ v_mix(row)) * 16);   // of piece + u: u * 16 ^ k_at
#pragma unroll
    for (int u = 0; u < CP / 8; ++u) {
      lds_store(ks + (k_at ^ u * 16), eight<T>(x.k[2 * u], x.k[2 * u + 1], by_k));
      lds_store(vs + (v_at ^ u * 16), eight<T>(x.v[2 * u], x.v[2 * u + 1], by_v));
    }
    return Units{k_top, v_top};
  }
  static __device__ __forceinline__ void lds_store(uint32_t at, dword4 x) { *(__attribute__((address_space(3))) dword4*)at = x; }
  // takes the sums to the units of a block
  __device__ __forceinline__ void take(int to) {
    if (to == unit) return;
    const float by = below(unit, to);
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] *= by;
    unit = to;
  }

  // All of it again, in FP32 from the keys' own scales: scores, the maximum and
  // the sums, each row adding the keys it sees and no other. Only for a wave
  // whose sums are not finite or whose exponents lie too far apart.
  __device__ __forceinline__ void walk_seen_only8() {
    const int in_page = (1 << p.seq.page_shift) - 1;
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] = f32x16{};
    m = -__builtin_inff();
    l = 0.0f;
    unit = 127;
    for (int kb = t.key0 + 32 * part; kb < t.key1; kb += HALVES ? 64 : 32) {
      const int mine = kb + c, at = slot(mine);
      const int page = mine < t.key1 ? t.pages[at >> p.seq.page_shift] : -1;
      const bool ok = p.seq.page_ok(page);
      const uint32_t there = (uint32_t)__ballot(ok);
      const uint32_t e = load<uint16_t>(or_nothing(ok, exps_at(page, at)));
      const Elem* kr = kh + element(page, p.k_page, at & in_page, p.k_slot);
      f32x16 x = f32x16{};
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int d = 16 * j + 8 * h;
        const dword2 w8 = load<dword2>(or_nothing(ok && (WHOLE || d < p.dim), addr(kr + d)));
        x = Half<T>::mma32(eight<T>(w8.x, w8.y, 1.0f), q[j], x);
        if (j % 2) __builtin_amdgcn_sched_barrier(0);      // or all loads are issued first, into registers that are not there
      }
      const uint32_t bits = visible(kb) & there, own = bits >> (4 * h);
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float by = score_scale(p.scale2, __builtin_amdgcn_readlane(e, i / 4 * 8) & 255);
        x[i] = own >> (8 * (i / 4) + i % 4) & 1u ? x[i] * by : -__builtin_inff();
        top = fmaxf(top, x[i]);
      }
      top = max_x32(top);
      const float to = fmaxf(m, top), by = m == to ? 1.0f : exp2_fast(m - to);
      l *= by;
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i] *= by;
      m = to;
      const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = exp2_fast(x[i] - base);
        if (own >> (8 * (i / 4) + i % 4) & 1u) l += x[i];
      }
      for (int key = 0; key < 32; ++key) {
        const int n = key / 8 * 4 + key % 4;
        float pk = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) pk = i == n ? x[i] : pk;
        pk = __shfl(pk, c + 32 * (key / 4 % 2));
        const int pg = __shfl(page, key), ev = (int)(__shfl(e, key) >> 8) - 127;
        if (!(there >> key & 1u)) continue;
        const Elem* vr = vh + element(pg, p.v_page, slot(kb + key) & in_page, p.v_slot);
        if (bits >> key & 1u) {
#pragma unroll
          for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const int d = 32 * i + 8 * a + 4 * h;
              if (d >= p.dim) continue;
              const uint32_t w4 = load<uint32_t>(addr(vr + d));
              const uint32_t lo = Eight<T>::pair(w4, 1.0f, false), hi = Eight<T>::pair(w4, 1.0f, true);
              o[i][4 * a] += pk * __builtin_amdgcn_ldexpf(Half<T>::lo(lo), ev);
              o[i][4 * a + 1] += pk * __builtin_amdgcn_ldexpf(Half<T>::hi(lo), ev);
              o[i][4 * a + 2] += pk * __builtin_amdgcn_ldexpf(Half<T>::lo(hi), ev);
              o[i][4 * a + 3] += pk * __builtin_amdgcn_ldexpf(Half<T>::hi(hi), ev);
              __builtin_amdgcn_sched_barrier(0);
            }
        }
      }
    }
  }

  // As walk() below; a wave's loads need no wait of their own.
  __device__ __forceinline__ void walk8() {
    m = -__builtin_inff();
    l = 0.0f;
    unit = k_top = v_top = 0;
    k_least = v_least = 255;
    k_tiny = tiny_key<T>(p.scale2);
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] = f32x16{};
    if (t.key0 >= t.key1 || p.seq.n_pages == 0) return;
    const bool live = row0 < t.rows;
    const int blocks = (t.key1 - t.key0 + B - 1) / B;
    Raw even, odd;                                       // blocks on their way, by their numbers
    Units before = {0, 0}, now, next = {0, 0};           // of blocks i - 1, i, i + 1
    int pages;
    {
      const int a = lookup8(t.key0), b = lookup8(t.key0 + B), d = DEEP == 2 ? lookup8(t.key0 + 2 * B) : 0;
      fetch8(t.key0, a, even);
      if (DEEP == 2) fetch8(t.key0 + B, b, odd);
      pages = lookup8(t.key0 + (DEEP + 1) * B);
      now = convert(even, 0);
      fetch8(t.key0 + DEEP * B, DEEP == 2 ? d : b, even);
    }
    const bool sound = pages_sound();
    // block i + 1 into LDS, block i + 1 + DEEP on its way, the pages of the one
    // after that (asked for first: loads return in order)
    const auto ahead = [&](int i, Raw& r_) {
      Raw& r = DEEP == 2 ? r_ : even;
      const int later = lookup8(t.key0 + (i + 2 + DEEP) * B);
      next = convert(r, (i + 1) % ST);
      fetch8(t.key0 + (i + 1 + DEEP) * B, pages, r);
      pages = later;
    };
    const auto begin = [&] { change_over<63>(); };
    const auto change = [&] { change_over<63>(); };
    const auto weigh = [&](int i, const Units& u) {
      softmax(t.key0 + i * B, there(t.key0 + i * B, sound), score_scale(p.scale2, u.k));
    };
    const auto shift = [&] {
      before = now;
      now = next;
    };
    if (!live) {
      const auto step = [&](int i, Raw& r) {
        begin();
        ahead(i, r);
        change();
      };
      for (int i = 0; i <= blocks; i += 2) {
        step(i, odd);
        if (i < blocks) step(i + 1, even);
      }
    } else if (wave < W / 2) {
      begin();
      first_product(0);
      change();
      ahead(0, odd);
      weigh(0, now);
      shift();
      const auto step = [&](int i, Raw& r) {
        begin();
        take(before.v);
        products((i - 1) % ST, i % ST);
        change();
        ahead(i, r);
        weigh(i, now);
        shift();
      };
      for (int i = 1; i < blocks; i += 2) {
        step(i, even);
        if (i + 1 < blocks) step(i + 1, odd);
      }
      begin();
      take(before.v);
      second_product((blocks - 1) % ST);
      change();
    } else {
      begin();
      ahead(0, odd);
      change();
      first_product(0);
      shift();
      const auto step = [&](int i, Raw& r) {
        begin();
        ahead(i, r);
        weigh(i - 1, before);
        change();
        take(before.v);
        products((i - 1) % ST, i % ST);
        shift();
      };
      for (int i = 1; i < blocks; i += 2) {
        step(i, even);
        if (i + 1 < blocks) step(i + 1, odd);
      }
      begin();
      weigh(blocks - 1, before);
      change();
      take(before.v);
      second_product((blocks - 1) % ST);
    }
    if (live) {
      bool bad = k_top - k_least > Eight<T>::kSpread || v_top - v_least > Eight<T>::kSpread;
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) bad |= not_finite(o[i][e]);
      if (__any(bad)) walk_seen_only8();
      l = sum_x32(l);
      const int by = unit - 127;
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = __builtin_amdgcn_ldexpf(o[i][e], by);
    }
    if (HALVES) join_halves(live);
  }

  // HALVES: the second half's sums go to the first's waves, a lane's values 64 floats apart
  __device__ __forceinline__ void join_halves(bool live) {
    float* x = (float*)lds_p + (wave % (W / 2)) * (16 * OT + 2) * 64 + lane;
    __syncthreads();
    if (part == 1 && live) {
      x[0] = m;
      x[64] = l;
#pragma unroll
      for (int i = 0; i < 16 * OT; ++i) x[(i + 2) * 64] = o[i / 16][i % 16];
    }
    __syncthreads();
    if (part == 0 && live) {
      const float m1 = x[0], to = fmaxf(m, m1);
      const float by0 = m == to ? 1.0f : exp2_fast(m - to), by1 = m1 == to ? 1.0f : exp2_fast(m1 - to);
      l = by0 * l + by1 * x[64];
#pragma unroll
      for (int i = 0; i < 16 * OT; ++i) o[i / 16][i % 16] = by0 * o[i / 16][i % 16] + by1 * x[(i + 2) * 64];
      m = to;
    }
  }

  // Waits for all but the last LATER loads and for the wave's LDS reads, then
  // for all waves.
  template <int LATER>
  static __device__ __forceinline__ void change_over() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void walk() {
    m = -__builtin_inff();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] = f32x16{};
    if (t.key0 >= t.key1) return;
    const bool live = row0 < t.rows;                      // a wave without rows still loads its share of K and V
    const int blocks = (t.key1 - t.key0 + B - 1) / B;
    {
      const Pages a = lookup(t.key0), b = lookup(t.key0 + B);
      fetch(t.key0, a, 0);
      fetch(t.key0 + B, b, 1);
    }
    Pages pages = lookup(t.key0 + 2 * B);
    const bool sound = pages_sound();
    // Step i: waves 0..3 are at the products while waves 4..7 are at the softmax
    // of block i - 1, then waves 0..3 at the softmax of block i while waves 4..7
    // are at the products. The stage of block i - 1 is read for the last time
    // in the second half of step i, so block i + 2 takes that of block i - 2.
    // The two orders are written out apart, the first and the last step too:
    // all waves pass the same number of barriers.
    // A wave starts its loads of block i + 2 with its softmax, so that they do
    // not hold up its products.
    const auto ahead = [&](int i) {
      fetch(t.key0 + (i + 2) * B, pages, (i + 2) % ST);
      pages = lookup(t.key0 + (i + 3) * B);
    };
    // block i is there: only the loads of block i + 1 may still be on their way
    const auto begin = [&] { change_over<2 * LOADS>(); };
    const auto change = [&] { change_over<63>(); };
    const auto weigh = [&](int i) { softmax(t.key0 + i * B, there(t.key0 + i * B, sound), p.scale2); };
    if (!live) {
      for (int i = 0; i <= blocks; ++i) {
        begin();
        ahead(i);
        change();
      }
    } else if (wave < W / 2) {
      begin();
      first_product(0);
      change();
      ahead(0);
      weigh(0);
      for (int i = 1; i < blocks; ++i) {
        begin();
        products((i - 1) % ST, i % ST);
        change();
        ahead(i);
        weigh(i);
      }
      begin();
      second_product((blocks - 1) % ST);
      change();
    } else {
      begin();
      ahead(0);
      change();
      first_product(0);
      for (int i = 1; i < blocks; ++i) {
        begin();
        ahead(i);
        weigh(i - 1);
        change();
        products((i - 1) % ST, i % ST);
      }
      begin();
      weigh(blocks - 1);
      change();
      second_product((blocks - 1) % ST);
    }
    // nothing may still be on its way to LDS when the workgroup gives it up
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (live) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) bad |= not_finite(o[i][e]);
      if (__any(bad)) walk_seen_only();
      l = sum_x32(l);
    }
    if (HALVES) join_halves(live);
  }

  __device__ __forceinline__ void store(int head, int split) const {
    const int r = row0 + c;
    if (r >= t.rows || part) return;
    const int tok = t.first + r / p.group, hq = head * p.group + r % p.group;
    const int64_t at = (int64_t)tok * p.heads * p.group + hq;
    if (p.splits > 1) {
      if (h == 0) {
        float* st = part_stats(p, at, split);
        st[0] = m;
        st[1] = l;
      }
      float* to = part_sums(p, at, split);
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int d = 32 * i + 8 * a + 4 * h;
          if (d < p.dim) *(f32x4*)(to + d) = f32x4{o[i][4 * a], o[i][4 * a + 1], o[i][4 * a + 2], o[i][4 * a + 3]};
        }
      return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* to = p.out + tok * p.o_token + hq * p.o_head;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int d = 32 * i + 8 * a + 4 * h;
        if (d < p.dim)
          *(dword2*)(to + d) = dword2{Half<T>::pack(o[i][4 * a] * inv, o[i][4 * a + 1] * inv),
                                      Half<T>::pack(o[i][4 * a + 2] * inv, o[i][4 * a + 3] * inv)};
      }
  }
};

template <class T, int DP, bool WHOLE, bool HALVES, bool EIGHT, bool WINDOW>
__global__ void __launch_bounds__(64 * kManyWaves, DP == 64 ? 4 : 2) attend_many_kernel(AttendParams p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t many_lds[];
  const int id = blockIdx.x, head = id % p.heads, split = id / p.heads % p.splits;
  // the last rows of a prompt see the most keys: they go first
  const int slot = p.slots - 1 - id / p.heads / p.splits;
  Tile t;
  if (!find_tile<kManyRows<HALVES>, WINDOW>(p, kManyBlock<DP>, slot, split, t)) return;
  if (p.splits > 1 && t.key0 >= t.key1) return;
  Many<T, DP, WHOLE, HALVES, EIGHT, WINDOW> f(p, t, head, many_lds);
  if constexpr (EIGHT) f.walk8();
  else f.walk();
  f.store(head, split);
}

}  // namespace sgemv_dev
