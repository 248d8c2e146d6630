// Attention of many rows (a chunk of a prompt) over a paged cache.
#pragma once
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
template <class T, int DP, bool WHOLE, bool HALVES>
struct Many {
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
  const uint16_t *kh, *vh;
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

  __device__ __forceinline__ Many(const AttendParams& p_, const Tile& t_, int head, uint16_t* lds_) : p(p_), t(t_), lds_p(lds_) {
    lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds_;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c = lane & 31;
    h = lane >> 5;
    kh = p.k + head * p.k_head;
    vh = p.v + head * p.v_head;
    part = HALVES ? wave / (W / 2) : 0;
    row0 = t.row0 + 32 * (HALVES ? wave % (W / 2) : wave);
    row = row0 + c < t.rows ? row0 + c : t.rows - 1;
    const uint16_t* qr = p.q + (int64_t)(t.first + row / p.group) * p.q_token + (int64_t)(head * p.group + row % p.group) * p.q_head;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int d = 16 * i + 8 * h;
      q[i] = load<dword4>(or_nothing(WHOLE || d < p.dim, addr(qr + d)));
    }
  }

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
      w.at[i] = table[__builtin_amdgcn_readfirstlane((key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift)];
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
      const int pg = w.at[i], slot = (kb + first) & in_page;
      const bool ok = p.seq.page_ok(pg);
      const addr_t kr = addr(kh + element(pg, p.k_page, slot, p.k_slot)), vr = addr(vh + element(pg, p.v_page, slot, p.v_slot));
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
      bits &= __ballot(p.seq.page_ok(t.pages[(key < t.key1 ? key : t.key1 - 1) >> p.seq.page_shift]));
    }
    return B == 64 ? bits : bits | ~0ull << 32;
  }
  __device__ __forceinline__ bool pages_sound() const {
    const int last = (t.key1 - 1) >> p.seq.page_shift;
    bool ok = true;
#pragma unroll 4
    for (int i = (t.key0 >> p.seq.page_shift) + lane; i <= last; i += 64) ok &= p.seq.page_ok(t.pages[i]);
    return __all(ok);
  }

  // -inf for the keys of the block at kb that the lane's row does not see
  __device__ __forceinline__ void mask(int kb, uint64_t there) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int at = 32 * (i + part);
      const uint32_t bits = (visible_bits(p, t, row / p.group, kb + at) & (uint32_t)(there >> at)) >> (4 * h);
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
  __device__ __forceinline__ void softmax(int kb, uint64_t there) {
    if (kb + B > t.full || there != ~0ull) mask(kb, there);
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 16 * NS; ++e) top = fmaxf(top, s[e / 16][e % 16]);
    top = __builtin_fmaf(max_x32(top), p.scale2, -Half<T>::kLift);
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
      const float a = exp2_fast(__builtin_fmaf(s[e / 16][e % 16], p.scale2, -base));
      const float b = exp2_fast(__builtin_fmaf(s[e / 16][e % 16 + 1], p.scale2, -base));
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
      const int mine = kb + c;
      const int page = mine < t.key1 ? t.pages[mine >> p.seq.page_shift] : -1;
      const bool ok = p.seq.page_ok(page);
      const uint32_t there = (uint32_t)__ballot(ok);
      const uint16_t* kr = kh + element(page, p.k_page, mine & in_page, p.k_slot);
      f32x16 x = f32x16{};
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int d = 16 * j + 8 * h;
        x = Half<T>::mma32(load<dword4>(or_nothing(ok && (WHOLE || d < p.dim), addr(kr + d))), q[j], x);
      }
      const uint32_t bits = visible_bits(p, t, row / p.group, kb) & there;
      for (int key = 0; key < 32; ++key) {
        // this key's score for row c, from the half that holds it
        const int e = key / 8 * 4 + key % 4;
        float sk = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sk = i == e ? x[i] : sk;
        sk = __shfl(sk, c + 32 * (key / 4 % 2));
        const int pg = __shfl(page, key);
        if (!(there >> key & 1u)) continue;
        const uint16_t* vr = vh + element(pg, p.v_page, (kb + key) & in_page, p.v_slot);
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
    const auto weigh = [&](int i) { softmax(t.key0 + i * B, there(t.key0 + i * B, sound)); };
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
    if (HALVES) {
      // the second half's sums, a lane's values 64 floats apart
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

template <class T, int DP, bool WHOLE, bool HALVES>
__global__ void __launch_bounds__(64 * kManyWaves, DP == 64 ? 4 : 2) attend_many_kernel(AttendParams p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t many_lds[];
  const int id = blockIdx.x, head = id % p.heads, split = id / p.heads % p.splits;
  // the last rows of a prompt see the most keys: they go first
  const int slot = p.slots - 1 - id / p.heads / p.splits;
  Tile t;
  if (!find_tile<kManyRows<HALVES>>(p, kManyBlock<DP>, slot, split, t)) return;
  if (p.splits > 1 && t.key0 >= t.key1) return;
  Many<T, DP, WHOLE, HALVES> f(p, t, head, many_lds);
  f.walk();
  f.store(head, split);
}

}  // namespace sgemv_dev
