// Attention of many rows (a chunk of a prompt) over a paged cache.
#pragma once
#include "attend_device.hpp"

namespace sgemv_dev {

constexpr int kManyBlock = 64;
template <int DP> constexpr int kManyWaves = DP == 256 ? 4 : 8;
template <int DP> constexpr int kManyRows = 32 * kManyWaves<DP>;
template <int DP> constexpr int kManyLds = 2 * 2 * kManyBlock * DP * 2;   // two stages of K and V

// One workgroup: a tile of 32 rows a wave and one split of its keys, in blocks
// of 64 that all waves share through LDS. Bound by the matrix cores, then by
// LDS reads (each operand read feeds one 32-row step) and the exponentials.
//
// The next block's K and V go from memory straight to the other LDS stage
// while this one is computed; one barrier a block. Rows of a stage are 2 DP
// bytes; the 16-byte pieces of a row are stored in an order that depends on
// the key (K: xor of the piece with the key; V: of the piece's group of four),
// so that the lanes of an operand read, which are at the same columns of
// different keys, fall on different banks. V's operand, 4 keys of one column a
// lane, is read with the transposing LDS load: of its 16 lanes, lane 4 i + j
// names key i's columns 4 j .., and lane c gets column c of the 4 keys.
template <class T, int DP>
struct Many {
  static constexpr int W = kManyWaves<DP>, KC = DP / 16, OT = DP / 32;
  static constexpr int PIECES = DP / 8;                  // 16-byte pieces of a row
  static constexpr int ROWS = 64 / PIECES;               // rows that one load of a wave fills
  static constexpr int LOADS = kManyBlock / ROWS / W;    // loads of a wave, for K and for V
  static constexpr int STAGE = kManyBlock * DP;          // elements of K or V in a stage

  static __device__ __forceinline__ int k_mix(int key) { return DP == 64 ? key >> 1 & 7 : key & 15; }
  static __device__ __forceinline__ int v_mix(int key) { return DP == 64 ? (key >> 1 & 1) * 4 : (key & 3) * 4; }

  const AttendParams& p;
  const Tile& t;
  const uint16_t *kh, *vh;
  uint16_t* lds;
  int lane, wave, c, h;                                  // lane = c + 32 h: row c of the wave
  int row;                                               // of the sequence, clamped to it
  dword4 q[KC];
  f32x16 o[OT];
  float m, l;

  __device__ __forceinline__ Many(const AttendParams& p_, const Tile& t_, int head, uint16_t* lds_) : p(p_), t(t_), lds(lds_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c = lane & 31;
    h = lane >> 5;
    kh = p.k + head * p.k_head;
    vh = p.v + head * p.v_head;
    row = t.row0 + 32 * wave + c;
    row = row < t.rows ? row : t.rows - 1;
    const uint16_t* qr = p.q + (int64_t)(t.first + row / p.group) * p.q_token + (int64_t)(head * p.group + row % p.group) * p.q_head;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int d = 16 * i + 8 * h;
      q[i] = d < p.dim ? *(const dword4*)(qr + d) : dword4{0, 0, 0, 0};
    }
  }

  // page of key kb + lane, -1 past the end
  __device__ __forceinline__ int lookup(int kb) const {
    const int key = kb + lane;
    return key < t.key1 ? t.pages[key >> p.seq.page_shift] : -1;
  }
  // starts the loads of the block at kb into a stage; `page` from lookup(kb)
  __device__ __forceinline__ void load(int kb, int page, int stage) const {
    const int in_page = (1 << p.seq.page_shift) - 1;
    page = p.seq.page_ok(page) ? page : -1;
    uint16_t* ks = lds + stage * 2 * STAGE;
    uint16_t* vs = ks + STAGE;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int first = (i * W + wave) * ROWS, key = first + lane / PIECES, piece = lane % PIECES;
      const int pg = __shfl(page, key);
      const int64_t slot = (kb + key) & in_page;
      const int dk = (piece ^ k_mix(key)) * 8, dv = (piece ^ v_mix(key)) * 8;
      const void* ka = pg >= 0 && dk < p.dim ? (const void*)(kh + pg * p.k_page + slot * p.k_slot + dk) : (const void*)kNothing;
      const void* va = pg >= 0 && dv < p.dim ? (const void*)(vh + pg * p.v_page + slot * p.v_slot + dv) : (const void*)kNothing;
      to_lds(ka, ks + first * DP);
      to_lds(va, vs + first * DP);
    }
  }
  // 16 bytes a lane from memory to LDS: lane i's go to `to` + 16 i bytes
  static __device__ __forceinline__ void to_lds(const void* from, uint16_t* to) {
    __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)const_cast<void*>(from),
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
  }

  // scores of keys kb + 32 i + (8 a + 4 h + e) at s[i][4 a + e]
  __device__ __forceinline__ void mask(int kb, uint64_t there, f32x16 (&s)[2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t bits = (seen_bits(p, t, row / p.group, kb + 32 * i) & (uint32_t)(there >> (32 * i))) >> (4 * h);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!(bits >> (8 * (e / 4) + e % 4) & 1u)) s[i][e] = -__builtin_inff();
    }
  }

  __device__ __forceinline__ void add(int kb, uint64_t there, int stage) {
    const uint16_t* ks = lds + stage * 2 * STAGE;
    const uint16_t* vs = ks + STAGE;
    f32x16 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s[i] = f32x16{};
      const int key = 32 * i + c;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const dword4 a = *(const dword4*)(ks + key * DP + (((2 * j + h) ^ k_mix(key)) * 8));
        s[i] = Half<T>::mma32(a, q[j], s[i]);
      }
    }
    if (kb + kManyBlock > t.full || there != ~0ull) mask(kb, there, s);
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e / 16][e % 16]);
    top = max_x32(top) * p.scale2;
    if (__any(top > m)) {
      const float to = fmaxf(m, top), by = m == to ? 1.0f : exp2_fast(m - to);
      l *= by;
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i] *= by;
      m = to;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float x = exp2_fast(__builtin_fmaf(s[e / 16][e % 16], p.scale2, -base));
      s[e / 16][e % 16] = x;
      l += x;
    }
#pragma unroll
    for (int ks16 = 0; ks16 < 4; ++ks16) {
      const f32x16& pr = s[ks16 / 2];
      const int e0 = 8 * (ks16 % 2);
      const dword4 pb = {Half<T>::pack(pr[e0], pr[e0 + 1]), Half<T>::pack(pr[e0 + 2], pr[e0 + 3]),
                         Half<T>::pack(pr[e0 + 4], pr[e0 + 5]), Half<T>::pack(pr[e0 + 6], pr[e0 + 7])};
      const int key = 16 * ks16 + 4 * h + (lane & 15) / 4;
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        const int piece = 4 * i + 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
        const dword2 x = transposed(vs + key * DP + ((piece ^ v_mix(key)) * 8) + 4 * (lane & 1));
        const dword2 y = transposed(vs + (key + 8) * DP + ((piece ^ v_mix(key + 8)) * 8) + 4 * (lane & 1));
        o[i] = Half<T>::mma32(dword4{x.x, x.y, y.x, y.y}, pb, o[i]);
      }
    }
  }
  static __device__ __forceinline__ dword2 transposed(const uint16_t* a) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(dword2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<uint16_t*>(a)));
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
    for (int kb = t.key0; kb < t.key1; kb += 32) {
      const int mine = kb + c;
      const int page = mine < t.key1 ? t.pages[mine >> p.seq.page_shift] : -1;
      const bool ok = p.seq.page_ok(page);
      const uint32_t there = (uint32_t)__ballot(ok);
      const uint16_t* kr = kh + page * p.k_page + (mine & in_page) * p.k_slot;
      f32x16 s = f32x16{};
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int d = 16 * j + 8 * h;
        s = Half<T>::mma32(*(ok && d < p.dim ? (const dword4*)(kr + d) : kNothing), q[j], s);
      }
      const uint32_t bits = seen_bits(p, t, row / p.group, kb) & there;
      for (int key = 0; key < 32; ++key) {
        // this key's score for row c, from the half that holds it
        const int e = key / 8 * 4 + key % 4;
        float sk = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sk = i == e ? s[i] : sk;
        sk = __shfl(sk, c + 32 * (key / 4 % 2));
        const int pg = __shfl(page, key);
        if (!(there >> key & 1u)) continue;
        const uint16_t* vr = vh + pg * p.v_page + ((kb + key) & in_page) * p.v_slot;
        const float pk = exp2_fast(__builtin_fmaf(sk, p.scale2, -base));
        if (bits >> key & 1u) {
#pragma unroll
          for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const int d = 32 * i + 8 * a + 4 * h;
              if (d >= p.dim) continue;
              const dword2 v = *(const dword2*)(vr + d);
              o[i][4 * a] += pk * Half<T>::lo(v.x);
              o[i][4 * a + 1] += pk * Half<T>::hi(v.x);
              o[i][4 * a + 2] += pk * Half<T>::lo(v.y);
              o[i][4 * a + 3] += pk * Half<T>::hi(v.y);
            }
        }
      }
    }
  }

  __device__ __forceinline__ void walk() {
    m = -__builtin_inff();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i] = f32x16{};
    if (t.key0 >= t.key1) return;
    int page = lookup(t.key0);
    uint64_t there = __ballot(p.seq.page_ok(page));
    load(t.key0, page, 0);
    page = lookup(t.key0 + kManyBlock);
    int stage = 0;
    for (int kb = t.key0; kb < t.key1; kb += kManyBlock, stage ^= 1) {
      // this block's loads are done, and nobody reads the other stage any more
      __syncthreads();
      const uint64_t now = there;
      if (kb + kManyBlock < t.key1) {
        there = __ballot(p.seq.page_ok(page));
        load(kb + kManyBlock, page, stage ^ 1);
        page = lookup(kb + 2 * kManyBlock);
      }
      add(kb, now, stage);
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) bad |= not_finite(o[i][e]);
    if (__any(bad)) walk_seen_only();
    l = sum_x32(l);
  }

  __device__ __forceinline__ void store(int head, int split) const {
    const int r = t.row0 + 32 * wave + c;
    if (r >= t.rows) return;
    const int tok = t.first + r / p.group, hq = head * p.group + r % p.group;
    const int64_t at = (int64_t)tok * p.heads * p.group + hq;
    if (p.splits > 1) {
      if (t.key0 >= t.key1) return;
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

template <class T, int DP>
__global__ void __launch_bounds__(64 * kManyWaves<DP>, DP == 256 ? 1 : 2) attend_many_kernel(AttendParams p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t many_lds[];
  const int id = blockIdx.x, head = id % p.heads, split = id / p.heads % p.splits;
  // the last rows of a prompt see the most keys: they go first
  const int slot = p.slots - 1 - id / p.heads / p.splits;
  Tile t;
  if (!find_tile(p, kManyRows<DP>, kManyBlock, slot, split, t)) return;
  Many<T, DP> f(p, t, head, many_lds);
  f.walk();
  f.store(head, split);
}

// Joins the parts of a split context: one wave a row. The parts are added in
// the order of the context, whatever order they were computed in.
template <class T>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendParams p, int tile_rows, int block) {
  const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, hq_all = p.heads * p.group;
  if (at >= (int64_t)p.seq.tokens * hq_all) return;
  const int tok = (int)(at / hq_all), hq = (int)(at % hq_all);
  Tile t;
  t.s = wave_upper(p.seq.count, tok, [&](int i) { return (int64_t)p.seq.start(i); });
  t.first = p.seq.start(t.s);
  t.n = p.seq.start(t.s + 1) - t.first;
  if (tok < t.first || tok >= t.first + t.n) return;
  t.rows = t.n * p.group;
  t.row0 = ((tok - t.first) * p.group + hq % p.group) / tile_rows * tile_rows;
  tile_keys(p, tile_rows, block, 0, t);
  // key1 of split 0 is the length of a part (or all there is)
  const int per = t.key1, parts = per > 0 ? (t.end + per - 1) / per : 0;

  float top = -__builtin_inff(), l = 0.0f;
  for (int i = lane; i < parts; i += 64) top = fmaxf(top, part_stats(p, at, i)[0]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  float x[4] = {0, 0, 0, 0};
  const int d0 = lane * 4;
  for (int i = 0; i < parts; ++i) {
    const float* st = part_stats(p, at, i);
    const float m = st[0], by = m == top ? 1.0f : exp2_fast(m - top);
    l += by * st[1];
    if (d0 < p.dim) {
      const f32x4 v = *(const f32x4*)(part_sums(p, at, i) + d0);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += by * v[e];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (d0 < p.dim)
    *(dword2*)(p.out + tok * p.o_token + hq * p.o_head + d0) =
        dword2{Half<T>::pack(x[0] * inv, x[1] * inv), Half<T>::pack(x[2] * inv, x[3] * inv)};
}

}  // namespace sgemv_dev
