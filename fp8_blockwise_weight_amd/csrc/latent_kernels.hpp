// Device code of the latent cache (gfx950): appending latents and rotated key
// channels to pages, and attention over them in the absorbed form, where every
// head reads the same latent as its key and as its value.
#pragma once

#include "kv_kernels.hpp"

namespace fp8bq {

constexpr int kRope = 64;   // rotated channels

typedef __attribute__((ext_vector_type(8))) int32_t i32x8;
typedef __attribute__((ext_vector_type(2))) int32_t i32x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) short s16x2;

struct LatentCache {
  uint8_t* c;      // e4m3 [pages, S, L]
  uint16_t* r;     // BF16 [pages, S, 64]
  float* scale;    // fp32 [pages, S], powers of two
  int32_t pages;
  int32_t log_s;   // S = 1 << log_s, 16 .. 256
};

struct LatentTokens {
  const uint16_t* c;    // BF16 rows
  const uint16_t* r;
  uint16_t* r_out;      // or null
  const uint16_t* q;    // or null
  uint16_t* q_out;
  const float* cos;     // fp32 [positions, 32], or null: nothing is rotated
  const float* sin;
  int64_t c_tok, r_tok, r_out_tok, q_tok, q_head, o_tok, o_head;  // strides in elements
  int64_t positions;
  int32_t tokens;
  int32_t heads;        // of q; 0 without
  int32_t interleaved;
};

// ------------------------------------------------------------------ append
//
// A token's latent is a block of its own, as [1, L] blocks of a weight are, so
// that nothing stored earlier changes when tokens arrive.  Its scale is the
// smallest power of two with 448 s >= max|x|: codes are floats themselves, and
// a finer scale would only move values between binades, while a power of two
// is an exponent that the matrix instruction takes beside its operand.
//
// kWaves waves share a token: 64 lanes hold its latent, 8 channels each (L =
// 512; half the lanes at 256), the others, or all of them later, turn 16
// channels at a time of the key and of the queries.  Bound by memory: 17,633
// tokens with 128 query heads, 616 MB, 134 us, 4.6 TB/s (a copy reaches 4.9);
// steps by their launch, 5.5 us of 10.
template <int L, int kWaves>
__global__ __launch_bounds__(kThreads) void latent_append(LatentCache c, KvBatch bt, LatentTokens t) {
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t row = kWaves == 4 ? blockIdx.x : blockIdx.x * 4 + wave;
  if (row >= t.tokens) return;
  int32_t b = row, n = 1, row0 = row;
  if (bt.starts) {
    b = kv_find(bt.count, row, [&](int32_t i) { return (int64_t)kv_clamp(bt.starts[i], t.tokens); });
    row0 = kv_clamp(bt.starts[b], t.tokens);
    n = kv_clamp(bt.starts[b + 1], t.tokens) - row0;
    if (row < row0 || row >= row0 + n) return;
  }
  const int64_t at = (int64_t)bt.lens[b] - n + (row - row0);
  if (at < 0 || at >= INT32_MAX || (t.cos && at >= t.positions)) return;
  const int32_t pos = (int32_t)at, slot = pos & ((1 << c.log_s) - 1);
  int32_t page = pos < kv_capacity(bt, c.log_s) ? bt.table[(int64_t)b * bt.stride + (pos >> c.log_s)] : -1;
  if (page >= c.pages) page = -1;
  const int64_t place = ((int64_t)max(page, 0) << c.log_s) + slot;

  if ((kWaves == 1 || wave == 0) && page >= 0) {
    u32x4 x = {0, 0, 0, 0};
    if (lane < L / 8) x = __builtin_nontemporal_load((const u32x4*)(t.c + row * t.c_tok + 8 * lane));
    float most = __uint_as_float((uint32_t)halves_max(fold_abs(x)) << 16);
    most = wave_max(most);
    const float s = kv_fit_scale(most), inv = kv_inverse(s);
    if (lane < L / 8) *(u32x2*)(c.c + place * L + 8 * lane) = quant8(x, inv);
    if (lane == 0) c.scale[place] = s;
  }
  // Units of 16 channels: those of the key first.
  const int32_t units = 4 * (t.heads + 1);
  const int32_t half = t.cos ? kRope / 2 : 0;
  for (int32_t i = kWaves == 1 ? lane : threadIdx.x; i < units; i += 64 * kWaves) {
    const int32_t u = i & 3, head = (i >> 2) - 1;
    KvTurn turn;
    turn.turn = half > 0;
    if (turn.turn) {
      const f32x4* cp = (const f32x4*)(t.cos + (int64_t)pos * half + 8 * u);
      const f32x4* sp = (const f32x4*)(t.sin + (int64_t)pos * half + 8 * u);
      turn.cs[0] = cp[0];
      turn.cs[1] = cp[1];
      turn.sn[0] = sp[0];
      turn.sn[1] = sp[1];
    }
    int32_t ca, cb;
    unit_channels(u, half, t.interleaved, ca, cb);
    const uint16_t* from = head < 0 ? t.r + row * t.r_tok : t.q + row * t.q_tok + head * t.q_head;
    const u32x4 lo = __builtin_nontemporal_load((const u32x4*)(from + ca));
    const u32x4 hi = __builtin_nontemporal_load((const u32x4*)(from + cb));
    float y[16];
    unit_rotate(lo, hi, turn, t.interleaved, y);
    bf16x8 ya, yb;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ya[e] = (__bf16)y[e];
      yb[e] = (__bf16)y[8 + e];
    }
    auto put = [&](uint16_t* to) {
      *(u32x4*)(to + ca) = __builtin_bit_cast(u32x4, ya);
      *(u32x4*)(to + cb) = __builtin_bit_cast(u32x4, yb);
    };
    if (head >= 0) {
      put(t.q_out + row * t.o_tok + head * t.o_head);
    } else {
      if (page >= 0) put(c.r + place * kRope);
      if (t.r_out) put(t.r_out + row * t.r_out_tok);
    }
  }
}

// --------------------------------------------------------------- attention

struct LatentQuery {
  KvQuery k;             // k.q: the absorbed channels; k.group: heads
  const uint16_t* r;     // the rotated channels
  int64_t r_tok, r_head;
  int32_t subs;          // row tiles that share keys, side by side on one XCD
};

// 16 bytes a lane, or 4, from memory into LDS, past the registers: lane i's go to
// lds + 16 i, lds + 4 i.  Written as assembly because the compiler, which cannot
// tell one buffer from another, waits for all of them before any read of LDS.
// The place is an operand in m0, not written here, so that the compiler knows
// what m0 holds; it may come right before, and the load wants a state between.
__device__ __forceinline__ void lds_load16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void lds_load4(const void* at, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(lds), "v"(at) : "memory");
}
// What this wave has loaded lies in LDS, what it reads from LDS it has read,
// and so it is for every wave.
__device__ __forceinline__ void lds_arrived() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ void lds_written() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}

// Two values as the sum of two codes.
//
// The matrix units multiply e4m3 by e4m3 at twice the rate of BF16.  A latent
// is stored in e4m3; a query or a weight is split into the code nearest to it
// and the code nearest to what is left, both with power-of-two scales that the
// instruction applies.  Together they hold 8 bits, as BF16 does (4 bits each,
// the rest is at most half a step of the first), so the product costs what
// BF16's does, but latents go from LDS to the matrix units as they are: half
// the bytes, and nothing to widen.
//
// `hi` is the code of x / s, `lo` of (x - hi s) / (s / 32): with |x| < 256 s
// the rest is at most 8 s.
constexpr int kLoShift = 5;
__device__ __forceinline__ void split2(float x, float y, float s, uint32_t& hi, uint32_t& lo, bool upper) {
  const float t = s * (1.0f / (1 << kLoShift));
  s16x2 h = __builtin_bit_cast(s16x2, hi), l = __builtin_bit_cast(s16x2, lo);
  if (upper) {
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, x, y, s, true);
    const f32x2 back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(__builtin_bit_cast(uint32_t, h), s, true);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, x - back[0], y - back[1], t, true);
  } else {
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, x, y, s, false);
    const f32x2 back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(__builtin_bit_cast(uint32_t, h), s, false);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, x - back[0], y - back[1], t, false);
  }
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, l);
}

// Biased exponent of the scale that brings values up to `most` below 256,
// with room for the rest's scale below it.
__device__ __forceinline__ int32_t split_exponent(float most) {
  return max((int32_t)((__float_as_uint(most) >> 23) & 255) - 7, 1 + kLoShift);
}
__device__ __forceinline__ float exponent_scale(int32_t e) { return __uint_as_float((uint32_t)e << 23); }

// By how much (log2) a maximum passes that of the sums before they follow.  Sums
// stay below 2^27 times the largest scale, 2^60, the largest code, 448, and 2^31
// keys: 2^126.8, where a float ends at 2^128.  Scaling sums is what costs: 96
// sequences at 16 heads take 116.5 us with 27, 145 with 12 (in steps of 12 of the
// waves' maxima, too), 121 where sums follow either wave's maximum at once, which
// moves in steps of 24.
constexpr float kRise = 27.0f;

template <int kSelA, int kSelB>
__device__ __forceinline__ f32x16 mfma_codes(const i32x8& a, const i32x8& b, const f32x16& c, int32_t sa, int32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, kSelA, sa, kSelB, sb);
}

// Sums stay in accumulation registers a0 .. a127 from the first product to the
// last, by name.  Left to itself the compiler moves all of them to other
// registers and back in every tile, for the sake of the path that scales them
// once in a while (96 sequences at 16 heads: 245 us for what then took 150).  So
// every use is assembly: the
// products (which need two cycles behind whatever vector instruction wrote their
// operands), scaling and reading (behind the wait that a product's result needs).
template <int I>
struct Acc;
#define FP8BQ_ACC_MUL(n) \
  "v_accvgpr_read_b32 %1, a" #n "\n\ts_nop 1\n\tv_mul_f32_e32 %1, %1, %2\n\ts_nop 1\n\tv_accvgpr_write_b32 a" #n ", %1\n\t"
#define FP8BQ_ACC(I, R, n0, n1, n2, n3, n4, n5, n6, n7, n8, n9, n10, n11, n12, n13, n14, n15)                        \
  template <>                                                                                                        \
  struct Acc<I> {                                                                                                    \
    static __device__ __forceinline__ void clear(f32x16& o) {                                                        \
      o = f32x16{};                                                                                                  \
      asm volatile("" : "+{" R "}"(o));                                                                              \
    }                                                                                                                \
    static __device__ __forceinline__ void add_hi(f32x16& o, const i32x8& a, const i32x8& b, int32_t sa, int32_t sb) { \
      asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 " R ", %1, %2, " R ", %3, %4 op_sel_hi:[0,0,0]"        \
                   : "+{" R "}"(o)                                                                                   \
                   : "v"(a), "v"(b), "v"(sa), "v"(sb));                                                              \
    }                                                                                                                \
    static __device__ __forceinline__ void add_lo(f32x16& o, const i32x8& a, const i32x8& b, int32_t sa, int32_t sb) { \
      asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 " R ", %1, %2, " R                                   \
                   ", %3, %4 op_sel:[0,1,0] op_sel_hi:[0,0,0]"                                                       \
                   : "+{" R "}"(o)                                                                                   \
                   : "v"(a), "v"(b), "v"(sa), "v"(sb));                                                              \
    }                                                                                                                \
    static __device__ __forceinline__ void scale(f32x16& o, float g) {                                               \
      float t;                                                                                                       \
      asm volatile(FP8BQ_ACC_MUL(n0) FP8BQ_ACC_MUL(n1) FP8BQ_ACC_MUL(n2) FP8BQ_ACC_MUL(n3) FP8BQ_ACC_MUL(n4)         \
                   FP8BQ_ACC_MUL(n5) FP8BQ_ACC_MUL(n6) FP8BQ_ACC_MUL(n7) FP8BQ_ACC_MUL(n8) FP8BQ_ACC_MUL(n9)         \
                   FP8BQ_ACC_MUL(n10) FP8BQ_ACC_MUL(n11) FP8BQ_ACC_MUL(n12) FP8BQ_ACC_MUL(n13) FP8BQ_ACC_MUL(n14)    \
                   FP8BQ_ACC_MUL(n15)                                                                                \
                   : "+{" R "}"(o), "=&v"(t)                                                                         \
                   : "v"(g));                                                                                        \
    }                                                                                                                \
  };
FP8BQ_ACC(0, "a[0:15]", 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15)
FP8BQ_ACC(1, "a[16:31]", 16, 17, 18, 19, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30, 31)
FP8BQ_ACC(2, "a[32:47]", 32, 33, 34, 35, 36, 37, 38, 39, 40, 41, 42, 43, 44, 45, 46, 47)
FP8BQ_ACC(3, "a[48:63]", 48, 49, 50, 51, 52, 53, 54, 55, 56, 57, 58, 59, 60, 61, 62, 63)
FP8BQ_ACC(4, "a[64:79]", 64, 65, 66, 67, 68, 69, 70, 71, 72, 73, 74, 75, 76, 77, 78, 79)
FP8BQ_ACC(5, "a[80:95]", 80, 81, 82, 83, 84, 85, 86, 87, 88, 89, 90, 91, 92, 93, 94, 95)
FP8BQ_ACC(6, "a[96:111]", 96, 97, 98, 99, 100, 101, 102, 103, 104, 105, 106, 107, 108, 109, 110, 111)
FP8BQ_ACC(7, "a[112:127]", 112, 113, 114, 115, 116, 117, 118, 119, 120, 121, 122, 123, 124, 125, 126, 127)
#undef FP8BQ_ACC
#undef FP8BQ_ACC_MUL
// The wait, before the compiler may move sums anywhere (an operand of each, so
// that moves come behind it), and once more before they are products' operands.
template <int N>
__device__ __forceinline__ void acc_wait(f32x16 (&o)[N]) {
  static_assert(N == 4 || N == 8, "the channels of a wave");
  if constexpr (N == 8) {
    asm volatile("s_nop 15\n\ts_nop 15"
                 : "+{a[0:15]}"(o[0]), "+{a[16:31]}"(o[1]), "+{a[32:47]}"(o[2]), "+{a[48:63]}"(o[3]),
                   "+{a[64:79]}"(o[4]), "+{a[80:95]}"(o[5]), "+{a[96:111]}"(o[6]), "+{a[112:127]}"(o[7]));
  } else {
    asm volatile("s_nop 15\n\ts_nop 15"
                 : "+{a[0:15]}"(o[0]), "+{a[16:31]}"(o[1]), "+{a[32:47]}"(o[2]), "+{a[48:63]}"(o[3]));
  }
}
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

// A tile of 64 keys in LDS: rows of L codes, whose 16-byte chunks are exchanged
// within 16 of them (XOR), rows of 64 BF16 rotated channels, exchanged within 8,
// and the scales.
//
// Key m of a 32-key product is key 32 u + 16 ((m / 4) % 2) + 4 (m / 8) + m % 4 of
// the tile, as in kv_attend_tiles.  The scores' product reads 16 bytes of 16
// such rows at one column, the weighted sum's 8 neighbouring rows at two
// columns: with twice the row's place in 8, plus its bit 4, both fall on
// different banks.
__device__ __forceinline__ int32_t code_turn(int32_t key) { return ((key & 7) << 1) | ((key >> 4) & 1); }
__device__ __forceinline__ int32_t rope_turn(int32_t key) { return ((key >> 1) & 3) | (((key >> 4) & 1) << 2); }

template <int L, int W>
struct LatentTile {
  static constexpr bool kDeep = W == 4;
  static constexpr int kSlots = kDeep ? 3 : 2;
  static constexpr int kCodes = 64 * L, kRopes = kDeep ? 64 * 2 * kRope : 0;
  static constexpr int kBytes = kCodes + kRopes + 256;
};

// The weights of 32 rows and 32 keys, as two terms, in the order in which the
// product takes them; the maximum they are taken from, the scale's exponent.
struct LatentWeights {
  u32x4 hi[64], lo[64];
  float m[32];
  int32_t e[32];
};

// f(std::integral_constant<int, i>) for i = 0 .. N - 1.
template <int N, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// The absorbed form: for 32 query rows, tile by tile of 64 keys, scores Q C, the
// weights with a running maximum, and the weighted sum of the same C, which is
// read from memory and from LDS's loads once.
//
// W waves, two of them for 32 rows: each makes the scores and weights of every
// other 32 keys, the weights go through LDS, and each sums half the channels: 32
// rows of 512 sums and their queries as codes fill what two waves hold of
// registers.  One wave to a SIMD, so nothing hides a wait but the wave's own
// order: operands are read a step ahead, the next tile's loads are issued
// between products, and with four waves the sums run a tile behind the scores,
// with that tile's weights between their products.  Two waves alone (two
// workgroups to a CU) take turns instead.
//
// What bounds it: up to 32 rows the loads (96 sequences of up to 16,384
// tokens, 16 heads, 512 MB: 116 us, 4.4 TB/s, of which loading alone takes 98);
// from 64 rows on the products and what is not hidden between them, 2.2 us a tile
// of 64 rows by 64 keys (60 sequences of up to 12,000 tokens, 128 heads, 103
// GFLOP: 130 us, of which 32 are the queries' splitting, the sums' writing and
// the join).  One wave with all channels of 32 rows, without the exchange,
// takes 2.0 us for that but 24 us more around it.
template <int L, int W>
__global__ __launch_bounds__(64 * W, 1) void latent_attend(LatentCache c, KvBatch bt, LatentQuery lq) {
  constexpr int R = 16 * W, N = 64 * W;
  constexpr int kJ = L / 64;              // 64-channel pieces of the scores
  constexpr int kO = L / 64;              // 32-channel tiles of a wave's sums
  using Tile = LatentTile<L, W>;
  constexpr bool kDeep = Tile::kDeep;
  constexpr int kSlots = Tile::kSlots;
  __shared__ __align__(1024) uint8_t lds[kSlots * Tile::kBytes];
  __shared__ LatentWeights ex[kDeep ? 2 : 1][W];
  __shared__ u32x4 turned[W / 2][4][64];   // the queries' rotated channels: registers are scarce
  const KvQuery& p = lq.k;
  const int32_t cap = kv_capacity(bt, c.log_s);
  const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the factor below is positive
  const float factor = fmaxf(fabsf(p.scale), kTiny);
  const int32_t wave = __builtin_amdgcn_readfirstlane((int32_t)threadIdx.x >> 6);
  const int32_t part = wave & 1;                             // which keys, which channels
  const uint32_t lds0 = lds_address(lds);
  // Workgroups go round the eight XCDs: those of one share follow each other on one.
  const int32_t turn_of = blockIdx.x >> 3, sub = turn_of % lq.subs;
  KvShares<0> shares(bt, p, cap, (turn_of / lq.subs) * 8 + (blockIdx.x & 7));
  KvWork wk;
  while (shares.next(wk)) {
    int32_t tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // as in kv_attend_rows
    const int32_t lane = tid & 63, col = lane & 31, half = lane >> 5;
    wk.first += sub * R;
    if (wk.first >= wk.count) continue;
    const KvSeen see = kv_seen<R>(wk, p, cap);
    const int32_t r_in = (wave >> 1) * 32 + col, r_mine = wk.first + r_in;
    const bool live = r_mine < wk.count;
    const int32_t tok_mine = live ? r_mine / p.group : 0;
    const int64_t head = live ? r_mine - tok_mine * p.group : 0;
    const int64_t row = wk.row0 + tok_mine;
    const int32_t row_hi = live ? min(wk.pos0 + tok_mine + 1, cap) : 0;
    const int32_t last = see.tile1 - 1;

    // Pages of a tile's runs of 16 tokens (runs that nobody sees: that of the
    // last token), the same in every lane; -1 where the table's entry is no page.
    // 64 entries of the table lie in a register, a lane each: loaded one tile at a
    // time, even two tiles ahead, they were waited for in every tile.
    const int32_t* table = bt.table + (int64_t)wk.b * bt.stride;
    int32_t held = INT32_MIN / 2, entries = 0;
    struct Pages {
      int32_t of[4];
    };
    auto entry_of = [&](int32_t tile, int32_t r) { return min(tile * kKeyTile + 16 * r, see.see_hi - 1) >> c.log_s; };
    auto pages = [&](int32_t tile) {
      if (entry_of(tile, 3) - held >= 64) {
        held = entry_of(tile, 0);
        entries = table[min(held + lane, entry_of(last, 3))];
        asm volatile("" : "+v"(entries));   // waited for here
      }
      Pages x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t pg = lane_of(entries, entry_of(tile, r) - held);
        x.of[r] = (uint32_t)pg < (uint32_t)c.pages ? pg : -1;
      }
      return x;
    };
    auto bad = [](const Pages& x) { return (x.of[0] | x.of[1] | x.of[2] | x.of[3]) < 0; };
    auto pick = [](const Pages& x, int32_t r) {
      const int32_t a = r & 1 ? x.of[1] : x.of[0], b = r & 1 ? x.of[3] : x.of[2];
      return r & 2 ? b : a;
    };
    auto place_of = [&](const Pages& x, int32_t tile, int32_t run) {
      return ((int64_t)max(pick(x, run), 0) << c.log_s) + ((tile * kKeyTile + 16 * run) & ((1 << c.log_s) - 1));
    };
    // A wave stages 4 / W runs of 16 tokens, in kPieces instructions: one takes
    // 1024 / L tokens' codes, or the rotated channels of 8, or all scales (which
    // every wave loads, so that there is no branch).
    constexpr int kKeys = 1024 / L, kRuns = 4 / W, kPerRun = 16 / kKeys + (kDeep ? 2 : 0), kPieces = kRuns * kPerRun + 1;
    const int32_t k_in = lane / (L / 16), r_in8 = lane >> 3;
    struct Stage {
      const uint8_t* code[kRuns];
      const uint8_t* rope[kRuns];
      const float* scale;
      uint32_t to;
    };
    auto plan = [&](int32_t tile, int32_t slot, const Pages& x) {
      Stage g;
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const int64_t place = place_of(x, tile, wave * kRuns + i);
        g.code[i] = c.c + place * L;
        g.rope[i] = (const uint8_t*)(c.r + place * kRope);
      }
      g.scale = c.scale + place_of(x, tile, lane >> 4) + (lane & 15);
      g.to = lds0 + slot * Tile::kBytes;
      return g;
    };
    auto piece = [&](const Stage& g, auto which) {
      constexpr int n = decltype(which)::value;
      if constexpr (n == kPieces - 1) {
        lds_load4(g.scale, g.to + Tile::kCodes + Tile::kRopes);
      } else if constexpr (n < kPieces - 1) {
        constexpr int i = n / kPerRun, at = n - i * kPerRun;
        const int32_t run = wave * kRuns + i;
        if constexpr (at < 16 / kKeys) {
          constexpr int k = at * kKeys;
          const uint32_t off = k_in * L + ((lane % (L / 16)) ^ code_turn(16 * run + k + k_in)) * 16;
          lds_load16(g.code[i] + k * L, off, g.to + (16 * run + k) * L);
        } else {
          constexpr int k = (at - 16 / kKeys) * 8;
          const uint32_t off = r_in8 * 128 + ((lane & 7) ^ rope_turn(16 * run + k + r_in8)) * 16;
          lds_load16(g.rope[i] + k * 128, off, g.to + Tile::kCodes + (16 * run + k) * 128);
        }
      }
    };
    // Key that is row `col` of this wave's scores.
    const int32_t key = 32 * part + 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
    // Its rotated channels, where they do not go through LDS.
    u32x4 rope[kDeep ? 1 : 4];
    auto fetch_rope = [&](int32_t tile, const Pages& x) {
      if constexpr (!kDeep) {
        const uint16_t* from = c.r + (place_of(x, tile, key >> 4) + (key & 15)) * kRope + 8 * half;
#pragma unroll
        for (int j = 0; j < 4; ++j) rope[j] = *(const u32x4*)(from + 16 * j);
      }
    };
    // What nobody sees counts as zeros, whatever is there.
    auto clear = [&](uint8_t* to, int32_t tile, const Pages& x) {
      for (int32_t i = tid; i < 64 * (L / 16); i += N) {
        const int32_t k = i / (L / 16);
        if (pick(x, k >> 4) < 0 || tile * kKeyTile + k >= see.see_hi) *(u32x4*)(to + 16 * i) = u32x4{0, 0, 0, 0};
      }
      if (tid < 64 && (pick(x, tid >> 4) < 0 || tile * kKeyTile + tid >= see.see_hi)) {
        *(float*)(to + Tile::kCodes + Tile::kRopes + 4 * tid) = 1.0f;
      }
      lds_written();
    };

    Pages now;
    lds_written();   // LDS is free of the row tile before
    if (see.tile0 <= last) {
      now = pages(see.tile0);
      const Stage g = plan(see.tile0, 0, now);
      unrolled<kPieces>([&](auto n) { piece(g, n); });
      fetch_rope(see.tile0, now);
    }

    // The queries, as codes and as what is left.  Each wave of a pair splits half
    // the channels, with a scale for its half of a row, and both take both from
    // LDS, out of slots that are not filled yet.
    i32x8 qh[kJ], ql[kJ];
    int32_t q_scale[2];
    {
      constexpr int kH = kJ / 2;
      static_assert((W / 2) * 2 * kH * 4 * 64 * 16 <= (kSlots - 1) * Tile::kBytes, "behind the first slot");
      // (rows beyond the last one read the sequence's first, for nothing)
      const uint16_t* src = p.q + row * p.q_tok + head * p.q_head + 64 * kH * part + 32 * half;
      const uint16_t* rot = lq.r + row * lq.r_tok + head * lq.r_head + 8 * half;
      u32x4 x[kH][4], y[4];
      uint32_t most = 0, most_r = 0;
#pragma unroll
      for (int j = 0; j < kH; ++j) {
#pragma unroll
        for (int z = 0; z < 4; ++z) x[j][z] = *(const u32x4*)(src + 64 * j + 8 * z);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *(const u32x4*)(rot + 16 * j);
#pragma unroll
      for (int j = 0; j < kH; ++j) {
#pragma unroll
        for (int z = 0; z < 4; ++z) most = pk_max_u16(most, fold_abs(x[j][z]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) most_r = pk_max_u16(most_r, fold_abs(y[j]));
      // What is not a number counts as the largest that is: it becomes a code that
      // is none anyway.
      const bool odd = __ballot(halves_max(pk_max_u16(most, most_r)) >= 0x7F80u) != 0;
      const float top = half_max(__uint_as_float(min(halves_max(most), 0x7F7Fu) << 16));
      const int32_t e = split_exponent(top);
      const float es = exponent_scale(e);
      if (odd || flip != 0) {
        const auto clean = [&](u32x4 v) { return kv_no_infinity(v ^ u32x4{flip, flip, flip, flip}); };
#pragma unroll
        for (int j = 0; j < kH; ++j) {
#pragma unroll
          for (int z = 0; z < 4; ++z) x[j][z] = clean(x[j][z]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = clean(y[j]);
      }
      u32x4* pass = (u32x4*)(lds + Tile::kBytes) + (wave & ~1) * kH * 4 * 64 + lane;
#pragma unroll
      for (int j = 0; j < kH; ++j) {
        u32x4 h[2], l[2];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t a = 0, b = 0;
            split2(bf_lo(x[j][z][2 * w]), bf_hi(x[j][z][2 * w]), es, a, b, false);
            split2(bf_lo(x[j][z][2 * w + 1]), bf_hi(x[j][z][2 * w + 1]), es, a, b, true);
            h[z >> 1][2 * (z & 1) + w] = a;
            l[z >> 1][2 * (z & 1) + w] = b;
          }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          pass[((part * kH + j) * 4 + z) * 64] = h[z];
          pass[((part * kH + j) * 4 + 2 + z) * 64] = l[z];
        }
      }
      if (part == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turned[wave >> 1][j][lane] = y[j];
      }
      if (half == 0) ex[0][wave].e[col] = e;
      lds_written();
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const u32x4 h = pass[(j * 4 + z) * 64], l = pass[(j * 4 + 2 + z) * 64];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            qh[j][4 * z + w] = (int32_t)h[w];
            ql[j][4 * z + w] = (int32_t)l[w];
          }
        }
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int32_t of = ex[0][(wave & ~1) + z].e[col];
        q_scale[z] = of | ((of - kLoShift) << 8);
      }
    }

    f32x16 o[kO];
    unrolled<kO>([&](auto i) { Acc<decltype(i)::value>::clear(o[decltype(i)::value]); });
    // The maximum that weights are taken from, a whole number, so that changes of
    // it are exact: of this wave's keys, and of the sums.
    float m = -INFINITY, ref = -INFINITY, l = 0.0f;

    // Places in a tile that this lane reads: chunk 0, from which the others are
    // an exchange away (places of tiles are multiples of 256).
    static_assert(Tile::kBytes % 256 == 0, "an XOR with less than 256 stays in its row");
    const uint32_t k_at = key * L + ((2 * half) ^ code_turn(key)) * 16;
    const uint32_t r_at = Tile::kCodes + key * 128 + (half ^ rope_turn(key)) * 16;
    // Channel 32 i + (lane mod 32) of this wave's half, 8 keys to a read.
    const int32_t v_key = 16 * half + ((lane & 15) >> 1), v_bit = (lane >> 4) & 1;
    const uint32_t v_at = v_key * L + ((2 * part * kO + v_bit) ^ code_turn(v_key)) * 16 + 8 * (lane & 1);
    const int32_t k0 = 32 * part + 16 * half;   // the 16 keys of a lane's scores

    // Scores, operands read two pieces ahead, the next tile's loads in between:
    // one wave to a SIMD, nothing else hides what it waits for.  Each step is
    // held where it is written.
    auto lds_of = [&](const uint8_t* from) { return (uint32_t)(from - lds); };
    auto scores = [&](const uint8_t* from, const Stage& g, auto staging, auto&& at_end) {
      constexpr int kAhead = 1, kSteps = kJ + 2, kEach = kDeep ? (kPieces + kSteps - 1) / kSteps : 5;
      u32x4 a[kAhead + 1][2];
      bf16x8 ra[2], rq[2];
      const uint32_t k_now = k_at + lds_of(from), r_now = r_at + lds_of(from);
      const auto read = [&](int j) {
#pragma unroll
        for (int y = 0; y < 2; ++y) a[j % (kAhead + 1)][y] = *(const u32x4*)(lds + (k_now ^ ((4 * (j & 3) + y) * 16)) + (j >> 2) * 256);
      };
      const auto read_rope = [&](int j) {
        if constexpr (kDeep) {
          ra[j & 1] = *(const bf16x8*)(lds + (r_now ^ (2 * j * 16)));
        } else {
          ra[j & 1] = __builtin_bit_cast(bf16x8, rope[j]);
        }
        rq[j & 1] = __builtin_bit_cast(bf16x8, turned[wave >> 1][j][lane]);
      };
      const int32_t ks = (__float_as_uint(*(const float*)(from + Tile::kCodes + Tile::kRopes + 4 * key)) >> 23) & 255;
      read(0);
      f32x16 s = {};
      __builtin_amdgcn_sched_barrier(0);
      unrolled<kJ>([&](auto step) {
        constexpr int j = decltype(step)::value;
        if constexpr (j + kAhead < kJ) read(j + kAhead);
        if constexpr (j + kAhead == kJ) {
          read_rope(0);
          read_rope(1);
        }
        const u32x4 x = a[j % (kAhead + 1)][0], y = a[j % (kAhead + 1)][1];
        const i32x8 k = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
        s = mfma_codes<0, 0>(k, qh[j], s, ks, q_scale[2 * j / kJ]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(staging)::value) {
          unrolled<kEach>([&](auto z) { piece(g, std::integral_constant<int, kEach * j + decltype(z)::value>{}); });
        }
        __builtin_amdgcn_sched_barrier(0);
        s = mfma_codes<0, 1>(k, ql[j], s, ks, q_scale[2 * j / kJ]);
        __builtin_amdgcn_sched_barrier(0);
      });
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ra[0], rq[0], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ra[1], rq[1], s, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      read_rope(2);
      read_rope(3);
      if constexpr (decltype(staging)::value) {
        unrolled<2 * kEach>([&](auto z) { piece(g, std::integral_constant<int, kEach * kJ + decltype(z)::value>{}); });
      }
      __builtin_amdgcn_sched_barrier(0);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ra[0], rq[0], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ra[1], rq[1], s, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      at_end();
      return s;
    };
    auto hide = [&](f32x16& s, int32_t tile, const Pages& x) {
      const int32_t hi = pick(x, k0 >> 4) >= 0 ? row_hi - tile * kKeyTile - k0 : 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = e < hi ? s[e] : -INFINITY;
    };
    // Weights of this wave's keys, written for both waves: in 16 parts, one
    // behind each product of the sums.
    struct Weigh {
      f32x16 s;
      float top, was, base, most, sum, ws;
      f32x4 scale[2];
      int32_t e;
      u32x4 hi, lo;
    };
    auto weigh = [&](Weigh& x, const uint8_t* from, LatentWeights& to, auto which) {
      constexpr int n = decltype(which)::value;
      // scales of four keys, two parts ahead
      if constexpr (n == 1 || n == 3 || n == 5 || n == 7) {
        x.scale[(n >> 1) & 1] = *(const f32x4*)(from + Tile::kCodes + Tile::kRopes + 4 * k0 + 16 * (n >> 1));
      }
      if constexpr (n == 0) {
        x.top = x.s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) x.top = fmaxf(x.top, x.s[e]);
        asm volatile("" : "+v"(x.top));
      } else if constexpr (n == 1) {
        x.top = half_max(x.top) * factor;
        // The maximum is a whole number at or above all scores: its changes scale
        // the sum of weights exactly.
        x.was = m;
        m = x.top > m ? __builtin_ceilf(x.top) : m;
        asm volatile("" : "+v"(m));
      } else if constexpr (n == 2) {
        l *= x.was == m ? 1.0f : __builtin_amdgcn_exp2f(x.was - m);
        x.base = m == -INFINITY ? 0.0f : m;
        x.most = x.sum = 0.0f;
        asm volatile("" : "+v"(l), "+v"(x.base));
      } else if constexpr (n < 11) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          constexpr int e0 = 2 * (n - 3);
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x.s[e0 + z], factor, -x.base));
          x.sum += w;
          x.s[e0 + z] = w * x.scale[(e0 >> 2) & 1][(e0 & 3) + z];
        }
        x.most = fmaxf(fmaxf(x.most, x.s[2 * (n - 3)]), x.s[2 * (n - 3) + 1]);
        asm volatile("" : "+v"(x.most), "+v"(x.sum));
      } else if constexpr (n == 11) {
        l += x.sum;
        x.e = split_exponent(half_max(x.most));
        x.ws = exponent_scale(x.e);
        asm volatile("" : "+v"(x.ws));
      } else {
        constexpr int y = n - 12;
        uint32_t a = 0, b = 0;
        split2(x.s[4 * y], x.s[4 * y + 1], x.ws, a, b, false);
        split2(x.s[4 * y + 2], x.s[4 * y + 3], x.ws, a, b, true);
        asm volatile("" : "+v"(a), "+v"(b));
        x.hi[y] = a;
        x.lo[y] = b;
        if constexpr (n == 15) {
          to.hi[lane] = x.hi;
          to.lo[lane] = x.lo;
          if (half == 0) {
            to.m[col] = m;
            to.e[col] = x.e;
          }
        }
      }
    };
    // Both waves' weights, and what they are taken from.
    struct Both {
      i32x8 h, l;
      float m0, m1;
      int32_t e, scale;
    };
    auto gather = [&](const LatentWeights* w) {
      const LatentWeights& w0 = w[wave & ~1];
      const LatentWeights& w1 = w[wave | 1];
      Both x;
      x.m0 = w0.m[col];
      x.m1 = w1.m[col];
      // The second 16 bytes of both halves, the odd wave's, have the upper half's scale.
      x.e = (half ? w1 : w0).e[col];
      const u32x4 h0 = w0.hi[lane], h1 = w1.hi[lane], l0 = w0.lo[lane], l1 = w1.lo[lane];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x.h[y] = (int32_t)h0[y];
        x.h[4 + y] = (int32_t)h1[y];
        x.l[y] = (int32_t)l0[y];
        x.l[4 + y] = (int32_t)l1[y];
      }
      return x;
    };
    auto follow = [&](Both& x) {
      // The sums are taken from a maximum of both waves', which weights pass by
      // 2^kRise at most; until then their scale goes with them.
      const float top = fmaxf(x.m0, x.m1), was = ref;
      const bool rise = top > ref + kRise;
      ref = rise ? top : ref;
      // sums without a maximum yet are zeros, or no numbers
      if (__builtin_expect(__ballot(rise && was > -INFINITY) != 0, 0)) {
        const float g = rise && was > -INFINITY ? __builtin_amdgcn_exp2f(was - ref) : 1.0f;
        acc_wait(o);
        unrolled<kO>([&](auto i) { Acc<decltype(i)::value>::scale(o[decltype(i)::value], g); });
        acc_wait(o);
      }
      // Weights without a maximum are zeros or no numbers.
      const float mm = half ? x.m1 : x.m0;
      const float by = mm == -INFINITY ? 0.0f : fmaxf(mm - ref, -256.0f);
      const int32_t e = min(max(x.e + (int32_t)by, kLoShift), 254);
      x.scale = e | ((e - kLoShift) << 8);
    };
    // The weighted sums of a tile, and between its products what `between` does
    // in 16 parts.
    auto add = [&](const uint8_t* from, const Both& x, auto&& between) {
      constexpr int kAhead = 1, kParts = 8 / kO;
      i32x8 v[kAhead + 1];
      const uint32_t v_now = v_at + lds_of(from);
      const auto read = [&](int i) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2*)(lds + (v_now ^ (2 * i * 16)) + (32 * (y >> 1) + 8 * (y & 1)) * L));
          v[i % (kAhead + 1)][2 * y] = t[0];
          v[i % (kAhead + 1)][2 * y + 1] = t[1];
        }
      };
      read(0);
      __builtin_amdgcn_sched_barrier(0);
      unrolled<kO>([&](auto step) {
        constexpr int i = decltype(step)::value;
        Acc<i>::add_hi(o[i], v[i % (kAhead + 1)], x.h, 127, x.scale);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (i + kAhead < kO) read(i + kAhead);
        unrolled<kParts>([&](auto z) { between(std::integral_constant<int, 2 * kParts * i + decltype(z)::value>{}); });
        __builtin_amdgcn_sched_barrier(0);
        Acc<i>::add_lo(o[i], v[i % (kAhead + 1)], x.l, 127, x.scale);
        __builtin_amdgcn_sched_barrier(0);
        unrolled<kParts>(
            [&](auto z) { between(std::integral_constant<int, 2 * kParts * i + kParts + decltype(z)::value>{}); });
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    const auto nothing = [](auto) {};

    if (see.tile0 <= last) {
      int32_t slot = 0, tile = see.tile0;
      // kEdge: tiles that not every row sees all of, or the last one; kFirst: no
      // sums are due yet.
      const auto step = [&](auto first, auto edge) {
        constexpr bool kFirst = decltype(first)::value, kEdge = decltype(edge)::value;
        const int32_t after = slot + 1 == kSlots ? 0 : slot + 1, ahead = slot == 0 ? kSlots - 1 : slot - 1;
        uint8_t* from = lds + slot * Tile::kBytes;
        lds_arrived();
        const Pages mine = now;
        if constexpr (kEdge) {
          if (bad(mine) || (tile + 1) * kKeyTile > see.see_hi) clear(from, tile, mine);
        }
        now = pages(min(tile + 1, last));
        Both x;
        const auto at_end = [&] {
          if constexpr (kDeep && !kFirst) x = gather(ex[(tile + 1) & 1]);
        };
        Weigh w;
        if constexpr (kEdge) {
          if (tile < last) {
            const Stage g = plan(tile + 1, after, now);
            unrolled<kPieces>([&](auto n) { piece(g, n); });
          }
          w.s = scores(from, Stage{}, std::false_type{}, at_end);
          if (tile < last) fetch_rope(tile + 1, now);
          hide(w.s, tile, mine);
        } else {
          w.s = scores(from, plan(tile + 1, after, now), std::true_type{}, at_end);
          fetch_rope(tile + 1, now);
        }
        if constexpr (kDeep) {
          // The products of the tile before, and between them this tile's weights.
          const auto part_of = [&](auto n) { weigh(w, from, ex[tile & 1][wave], n); };
          if constexpr (kFirst) {
            unrolled<16>(part_of);
          } else {
            follow(x);
            add(lds + ahead * Tile::kBytes, x, part_of);
          }
        } else {
          unrolled<16>([&](auto n) { weigh(w, from, ex[0][wave], n); });
          lds_written();
          x = gather(ex[0]);
          follow(x);
          add(from, x, nothing);
        }
        slot = after;
        ++tile;
      };
      if constexpr (kDeep) step(std::true_type{}, std::true_type{});
      while (tile <= last) {
        while (tile < last && (tile + 1) * kKeyTile <= see.all_hi && !bad(now)) step(std::false_type{}, std::false_type{});
        step(std::false_type{}, std::true_type{});
      }
      if constexpr (kDeep) {
        lds_written();
        Both x = gather(ex[last & 1]);
        follow(x);
        add(lds + (slot == 0 ? kSlots - 1 : slot - 1) * Tile::kBytes, x, nothing);
      }
      acc_wait(o);
    }

    // The pair's sums, over one maximum.
    l += __shfl_xor(l, 32);
    lds_written();
    if (half == 0) {
      ex[0][wave].m[col] = m;
      ex[0][wave].e[col] = __float_as_int(l);
    }
    lds_written();
    {
      const LatentWeights& w0 = ex[0][wave & ~1];
      const LatentWeights& w1 = ex[0][wave | 1];
      const float f0 = w0.m[col] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(w0.m[col] - ref);
      const float f1 = w1.m[col] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(w1.m[col] - ref);
      l = __int_as_float(w0.e[col]) * f0 + __int_as_float(w1.e[col]) * f1;
    }
    const bool writes = live && half == 0 && part == 0;
    const int64_t item = row * p.group + head;
    const int32_t in_share = sub * R + r_in;
    if (wk.parts > 1) {
      const int64_t at = (int64_t)wk.slot * p.tile_rows + in_share;
      if (live) {
        float* to = p.part + at * L + 32 * kO * part + 4 * half;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            *(f32x4*)(to + 32 * i + 8 * e) = f32x4{acc_read(o[i][4 * e]), acc_read(o[i][4 * e + 1]),
                                                   acc_read(o[i][4 * e + 2]), acc_read(o[i][4 * e + 3])};
          }
        }
      }
      if (writes) p.part_ml[at] = kv_part_ml(ref, l);
    } else {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (live) {
        uint16_t* to = p.out + row * p.o_tok + head * p.o_head + 32 * kO * part + 4 * half;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            *(bf16x4*)(to + 32 * i + 8 * e) =
                bf16x4{(__bf16)(acc_read(o[i][4 * e]) * inv), (__bf16)(acc_read(o[i][4 * e + 1]) * inv),
                       (__bf16)(acc_read(o[i][4 * e + 2]) * inv), (__bf16)(acc_read(o[i][4 * e + 3]) * inv)};
          }
        }
      }
      if (writes && p.lse) p.lse[item] = l == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
    if (writes && wk.begin && p.rows) p.rows[item] = int2{wk.slot * p.tile_rows + in_share, wk.parts};
  }
}

}  // namespace fp8bq
