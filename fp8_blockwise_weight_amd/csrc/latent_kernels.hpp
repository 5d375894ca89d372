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
// channels at a time of the key and of the queries.
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
};

// 16 bytes a lane (4 with kWord) from memory into LDS, past the registers: lane
// i's go to lds + 16 i.  Written as assembly because the compiler, which cannot
// tell one buffer from another, waits for all of them before any read of LDS.
__device__ __forceinline__ void lds_load16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void lds_load16_at(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(at) : "memory");
}
__device__ __forceinline__ void lds_load4(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(at) : "memory");
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

template <int kSelA, int kSelB>
__device__ __forceinline__ f32x16 mfma_codes(const i32x8& a, const i32x8& b, const f32x16& c, int32_t sa, int32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, kSelA, sa, kSelB, sb);
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

template <int L, int W, int S>
struct LatentTile {
  static constexpr bool kRopeStaged = !(W == 2);
  static constexpr int kCodes = 64 * L, kRopes = kRopeStaged ? 64 * 2 * kRope : 0;
  static constexpr int kBytes = kCodes + kRopes + 256;
};

// W waves; S of them share 32 query rows.  With S = 1 a wave makes all scores of
// its rows and all channels of their sums.  With S = 2 it makes those of every
// other 32 keys, the weights go through LDS, and each wave sums half the
// channels.
template <int L, int W, int S>
__global__ __launch_bounds__(64 * W, 1) void latent_attend(LatentCache c, KvBatch bt, LatentQuery lq) {
  constexpr int R = 32 * W / S, N = 64 * W;
  constexpr int kJ = L / 64;              // 64-channel pieces of the scores
  constexpr int kU = 2 / S;               // 32-key blocks of a wave's scores
  constexpr int kO = L / 32 / S;          // 32-channel tiles of a wave's sums
  using Tile = LatentTile<L, W, S>;
  constexpr bool kRopeStaged = Tile::kRopeStaged;
  struct Weights {                        // of 32 rows and 32 keys
    u32x4 hi[64], lo[64];
    float m[32];
    int32_t e[32];
  };
  __shared__ __align__(1024) uint8_t lds[2 * Tile::kBytes];
  __shared__ Weights ex[S == 2 ? W : 1];
  const KvQuery& p = lq.k;
  const int32_t cap = kv_capacity(bt, c.log_s);
  const float scale = fabsf(p.scale);
  const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the factor below is positive
  const int32_t wave = __builtin_amdgcn_readfirstlane((int32_t)threadIdx.x >> 6);
  const int32_t part = S == 2 ? wave & 1 : 0;                // which keys, which channels
  const int32_t lds0 = (int32_t)lds_address(lds);
  KvShares<R> shares(bt, p, cap, blockIdx.x);
  KvWork wk;
  while (shares.next(wk)) {
    int32_t tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // as in kv_attend_rows
    const int32_t lane = tid & 63, col = lane & 31, half = lane >> 5;
    const KvSeen see = kv_seen<R>(wk, p, cap);
    const int32_t r_in = (wave / S) * 32 + col, r_mine = wk.first + r_in;
    const bool live = r_mine < wk.count;
    const int32_t tok_mine = live ? r_mine / p.group : 0;
    const int64_t head = live ? r_mine - tok_mine * p.group : 0;
    const int64_t row = wk.row0 + tok_mine;
    const int32_t row_hi = live ? min(wk.pos0 + tok_mine + 1, cap) : 0;

    // Pages of a tile's runs of 16 tokens, the same in every lane; -1 where the
    // table's entry is no page or none of the tokens is seen.
    const FP8BQ_CONSTANT int32_t* table =
        (const FP8BQ_CONSTANT int32_t*)(uintptr_t)(bt.table + (int64_t)wk.b * bt.stride);
    struct Pages {
      int32_t of[4];
    };
    auto pages = [&](int32_t tile) {
      Pages x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t t0 = tile * kKeyTile + 16 * r;
        int32_t pg = -1;
        if (t0 < see.see_hi) pg = table[t0 >> c.log_s];
        pg = __builtin_amdgcn_readfirstlane(pg);
        x.of[r] = pg >= 0 && pg < c.pages ? pg : -1;
      }
      return x;
    };
    auto pick = [](const Pages& x, int32_t r) {
      const int32_t a = r & 1 ? x.of[1] : x.of[0], b = r & 1 ? x.of[3] : x.of[2];
      return r & 2 ? b : a;
    };
    // A wave stages 4 / W runs of 16 tokens.
    auto stage = [&](int32_t tile, int32_t slot, const Pages& x) {
      const uint32_t to = lds0 + slot * Tile::kBytes;
#pragma unroll
      for (int i = 0; i < 4 / W; ++i) {
        const int32_t run = wave * (4 / W) + i, t0 = tile * kKeyTile + 16 * run;
        const int64_t place = ((int64_t)max(pick(x, run), 0) << c.log_s) + (t0 & ((1 << c.log_s) - 1));
        const uint8_t* from = c.c + place * L;
        constexpr int kKeys = 1024 / L;   // of an instruction
#pragma unroll
        for (int k = 0; k < 16; k += kKeys) {
          const int32_t key = 16 * run + k + lane / (L / 16);
          const uint32_t off = (lane / (L / 16)) * L + ((lane % (L / 16)) ^ code_turn(key)) * 16;
          lds_load16(from + k * L, off, to + (16 * run + k) * L);
        }
        if constexpr (kRopeStaged) {
          const uint8_t* rope = (const uint8_t*)(c.r + place * kRope);
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            const int32_t key = 16 * run + k + (lane >> 3);
            const uint32_t off = (lane >> 3) * 128 + ((lane & 7) ^ rope_turn(key)) * 16;
            lds_load16(rope + k * 128, off, to + Tile::kCodes + (16 * run + k) * 128);
          }
        }
      }
      if (wave == 0) {
        const int32_t run = lane >> 4, t0 = tile * kKeyTile + 16 * run;
        const int64_t place = ((int64_t)max(pick(x, run), 0) << c.log_s) + (t0 & ((1 << c.log_s) - 1)) + (lane & 15);
        lds_load4(c.scale + place, to + Tile::kCodes + Tile::kRopes);
      }
    };
    // Rotated channels of this wave's own keys, where they do not go through LDS.
    u32x4 rope[kRopeStaged ? 1 : 4];
    auto fetch_rope = [&](int32_t tile, const Pages& x) {
      if constexpr (!kRopeStaged) {
        const int32_t key = 32 * part + 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
        const int32_t t0 = tile * kKeyTile + (key & ~15);
        const int64_t place = ((int64_t)max(pick(x, key >> 4), 0) << c.log_s) + (t0 & ((1 << c.log_s) - 1)) + (key & 15);
#pragma unroll
        for (int j = 0; j < 4; ++j) rope[j] = *(const u32x4*)(c.r + place * kRope + 16 * j + 8 * half);
      }
    };

    const int32_t last = see.tile1 - 1;
    Pages now, next;
    lds_written();   // LDS is free of the row tile before
    if (see.tile0 <= last) {
      now = pages(see.tile0);
      stage(see.tile0, 0, now);
      next = pages(min(see.tile0 + 1, last));
    }

    // The queries, as codes and as what is left: one scale for a row.
    i32x8 qh[kJ], ql[kJ];
    bf16x8 qr[4];
    int32_t q_scale;
    {
      const uint16_t* src = p.q + row * p.q_tok + head * p.q_head + 32 * half;
      u32x4 x[kJ][4];
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          x[j][y] = *(const u32x4*)(src + 64 * j + 8 * y);
          if (!live) x[j][y] = u32x4{0, 0, 0, 0};
          x[j][y] = kv_no_infinity(x[j][y] ^ u32x4{flip, flip, flip, flip});
          most = pk_max_u16(most, fold_abs(x[j][y]));
        }
      }
      // what is not a number has the largest magnitude; it becomes a code that is none under any scale
      const float top = half_max(__uint_as_float(min(halves_max(most), 0x7F7Fu) << 16));
      const int32_t e = split_exponent(top);
      q_scale = e | ((e - kLoShift) << 8);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t h = 0, l = 0;
            split2(bf_lo(x[j][y][2 * z]), bf_hi(x[j][y][2 * z]), exponent_scale(e), h, l, false);
            split2(bf_lo(x[j][y][2 * z + 1]), bf_hi(x[j][y][2 * z + 1]), exponent_scale(e), h, l, true);
            qh[j][2 * y + z] = (int32_t)h;
            ql[j][2 * y + z] = (int32_t)l;
          }
        }
      }
      const uint16_t* rot = lq.r + row * lq.r_tok + head * lq.r_head + 8 * half;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 y = *(const u32x4*)(rot + 16 * j);
        if (!live) y = u32x4{0, 0, 0, 0};
        qr[j] = __builtin_bit_cast(bf16x8, kv_no_infinity(y ^ u32x4{flip, flip, flip, flip}));
      }
    }

    f32x16 o[kO];
#pragma unroll
    for (int i = 0; i < kO; ++i) o[i] = f32x16{};
    // The maximum that weights are taken from, a whole number, so that changes of
    // it are exact: of this wave's keys, and of the sums (S = 2).
    float m = -INFINITY, ref = -INFINITY, l = 0.0f;

    if (see.tile0 <= last) fetch_rope(see.tile0, now);
    for (int32_t tile = see.tile0; tile <= last; ++tile) {
      const int32_t slot = (tile - see.tile0) & 1;
      const uint8_t* from = lds + slot * Tile::kBytes;
      const float* scales = (const float*)(from + Tile::kCodes + Tile::kRopes);
      lds_arrived();
      u32x4 rope_now[kRopeStaged ? 1 : 4];
      if constexpr (!kRopeStaged) {
#pragma unroll
        for (int j = 0; j < 4; ++j) rope_now[j] = rope[j];
      }
      const int32_t t0 = tile * kKeyTile;
      const bool bad = (now.of[0] | now.of[1] | now.of[2] | now.of[3]) < 0;
      if (bad || t0 + kKeyTile > see.see_hi) {
        // what nobody sees counts as zeros, whatever is there
        uint8_t* to = lds + slot * Tile::kBytes;
        for (int32_t i = tid; i < 64 * (L / 16); i += N) {
          const int32_t key = i / (L / 16);
          if (pick(now, key >> 4) < 0 || t0 + key >= see.see_hi) *(u32x4*)(to + 16 * i) = u32x4{0, 0, 0, 0};
        }
        if (tid < 64 && (pick(now, tid >> 4) < 0 || t0 + tid >= see.see_hi)) {
          *(float*)(to + Tile::kCodes + Tile::kRopes + 4 * tid) = 1.0f;
        }
        lds_written();
      }
      const Pages mine = now;
      if (tile < last) {
        stage(tile + 1, slot ^ 1, next);
        fetch_rope(tile + 1, next);
        now = next;
        next = pages(min(tile + 2, last));
      }

      // scores
      f32x16 s[kU];
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        const int32_t u = S == 2 ? part : v;
        const int32_t key = 32 * u + 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
        const uint8_t* krow = from + key * L;
        const int32_t turn = code_turn(key);
        const int32_t ks = (__float_as_uint(scales[key]) >> 23) & 255;
        s[v] = f32x16{};
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const u32x4 a = *(const u32x4*)(krow + ((4 * j + 2 * half) ^ turn) * 16);
          const u32x4 b = *(const u32x4*)(krow + ((4 * j + 2 * half + 1) ^ turn) * 16);
          const i32x8 k = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
          s[v] = mfma_codes<0, 0>(k, qh[j], s[v], ks, q_scale);
          s[v] = mfma_codes<0, 1>(k, ql[j], s[v], ks, q_scale);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4 a;
          if constexpr (kRopeStaged) {
            a = *(const u32x4*)(from + Tile::kCodes + key * 128 + ((2 * j + half) ^ rope_turn(key)) * 16);
          } else {
            a = rope_now[j];
          }
          s[v] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), qr[j], s[v], 0, 0, 0);
        }
      }
      if (bad || t0 + kKeyTile > see.all_hi) {
        asm volatile("");   // a branch
#pragma unroll
        for (int v = 0; v < kU; ++v) {
          const int32_t k0 = 32 * (S == 2 ? part : v) + 16 * half;
          const int32_t hi = pick(mine, k0 >> 4) >= 0 ? row_hi - t0 - k0 : 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) s[v][e] = e < hi ? s[v][e] : -INFINITY;
        }
      }
      // weights
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < kU; ++v) {
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[v][e]);
      }
      const float factor = fmaxf(scale, kTiny);
      top = half_max(top) * factor;
      if (__ballot(top > m + 8.0f) != 0) {
        const float to = fmaxf(m, __builtin_ceilf(top));
        const float g = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        l *= g;
        if constexpr (S == 1) {
#pragma unroll
          for (int i = 0; i < kO; ++i) o[i] *= g;
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      uint32_t wh[kU][4], wl[kU][4];
      int32_t we[kU];
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        const int32_t k0 = 32 * (S == 2 ? part : v) + 16 * half;
        float w[16], most = 0.0f;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f32x4 sc = *(const f32x4*)(scales + k0 + 4 * y);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 4 * y + z;
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[v][e], factor, -base));
            l += x;
            w[e] = x * __uint_as_float(__float_as_uint(sc[z]) & 0x7F800000u);
            most = fmaxf(most, w[e]);
          }
        }
        we[v] = split_exponent(half_max(most));
        const float ws = exponent_scale(we[v]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          wh[v][y] = wl[v][y] = 0;
          split2(w[4 * y], w[4 * y + 1], ws, wh[v][y], wl[v][y], false);
          split2(w[4 * y + 2], w[4 * y + 3], ws, wh[v][y], wl[v][y], true);
        }
      }
      i32x8 ph, pl;
      int32_t p_scale;
      if constexpr (S == 1) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            ph[4 * v + y] = (int32_t)wh[v][y];
            pl[4 * v + y] = (int32_t)wl[v][y];
          }
        }
        p_scale = half ? we[1] : we[0];
      } else {
        Weights& to = ex[wave];
        to.hi[lane] = u32x4{wh[0][0], wh[0][1], wh[0][2], wh[0][3]};
        to.lo[lane] = u32x4{wl[0][0], wl[0][1], wl[0][2], wl[0][3]};
        if (half == 0) {
          to.m[col] = m;
          to.e[col] = we[0];
        }
        lds_written();
        const Weights& w0 = ex[wave & ~1];
        const Weights& w1 = ex[wave | 1];
        const float m0 = w0.m[col], m1 = w1.m[col], both = fmaxf(m0, m1);
        if (__ballot(both > ref + 8.0f) != 0) {
          const float to_ref = fmaxf(ref, both);
          const float g = to_ref == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ref - to_ref);
          ref = to_ref;
#pragma unroll
          for (int i = 0; i < kO; ++i) o[i] *= g;
        }
        const u32x4 h0 = w0.hi[lane], h1 = w1.hi[lane], l0 = w0.lo[lane], l1 = w1.lo[lane];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          ph[y] = (int32_t)h0[y];
          ph[4 + y] = (int32_t)h1[y];
          pl[y] = (int32_t)l0[y];
          pl[4 + y] = (int32_t)l1[y];
        }
        // weights of a block without a maximum are zeros or no numbers
        const float mm = half ? m1 : m0;
        const float by = mm == -INFINITY ? 0.0f : fmaxf(mm - ref, -256.0f);
        p_scale = min(max((half ? w1.e[col] : w0.e[col]) + (int32_t)by, kLoShift), 254);
      }
      p_scale |= (p_scale - kLoShift) << 8;

      // the weighted sum
#pragma unroll
      for (int i = 0; i < kO; ++i) {
        const int32_t tile_of = i + part * kO;
        i32x8 v;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int32_t key = 32 * (y >> 1) + 16 * half + 8 * (y & 1) + ((lane & 15) >> 1);
          const int32_t chunk = 2 * tile_of + ((lane >> 4) & 1);
          const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(
              from + key * L + (chunk ^ code_turn(key)) * 16 + 8 * (lane & 1)));
          v[2 * y] = x[0];
          v[2 * y + 1] = x[1];
        }
        o[i] = mfma_codes<0, 0>(v, ph, o[i], 127, p_scale);
        o[i] = mfma_codes<0, 1>(v, pl, o[i], 127, p_scale);
      }
    }

    l += __shfl_xor(l, 32);
    if constexpr (S == 2) {
      // the pair's sums, over one maximum
      lds_written();
      Weights& to = ex[wave];
      if (half == 0) {
        to.m[col] = m;
        to.e[col] = __float_as_int(l);
      }
      lds_written();
      const Weights& w0 = ex[wave & ~1];
      const Weights& w1 = ex[wave | 1];
      const float f0 = w0.m[col] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(w0.m[col] - ref);
      const float f1 = w1.m[col] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(w1.m[col] - ref);
      l = __int_as_float(w0.e[col]) * f0 + __int_as_float(w1.e[col]) * f1;
      m = ref;
    }
    const bool writes = live && half == 0 && part == 0;
    const int64_t item = row * p.group + head;
    if (wk.parts > 1) {
      const int64_t at = (int64_t)wk.slot * R + r_in;
      if (live) {
        float* to = p.part + at * L + 32 * kO * part + 4 * half;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            *(f32x4*)(to + 32 * i + 8 * e) = f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
          }
        }
      }
      if (writes) p.part_ml[at] = kv_part_ml(m, l);
    } else {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (live) {
        uint16_t* to = p.out + row * p.o_tok + head * p.o_head + 32 * kO * part + 4 * half;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            *(bf16x4*)(to + 32 * i + 8 * e) =
                bf16x4{(__bf16)(o[i][4 * e] * inv), (__bf16)(o[i][4 * e + 1] * inv), (__bf16)(o[i][4 * e + 2] * inv),
                       (__bf16)(o[i][4 * e + 3] * inv)};
          }
        }
      }
      if (writes && p.lse) p.lse[item] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
    if (writes && wk.begin && p.rows) p.rows[item] = int2{wk.slot * R + r_in, wk.parts};
  }
}

}  // namespace fp8bq
