// Device code of the blockwise e4m3 key/value cache (gfx950): appending
// rotated tokens to paged blocks, and attention over them.
//
// A page of S tokens holds, for each key/value head, two e4m3 blocks with one
// fp32 descale each, as fp8bq_quantize lays out a weight's tiles:
//   k  [S, D]  a token's channels side by side
//   v  [D, S]  a channel's tokens side by side
// Both products of attention then read their 8-bit operand in 16-byte loads
// in the order the matrix instruction wants it: the scores contract over
// channels (rows of k), the weighted sum over tokens (rows of v).  With v
// token-major, every lane would gather the 8 tokens of an operand byte by
// byte, or transpose each tile through LDS on every read; the transposition
// is paid once instead, when a token is stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace fp8bq {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;

// Memory that no kernel writes while it is read so (scalar loads).
#define FP8BQ_CONSTANT __attribute__((address_space(4)))

struct KvCache {
  uint8_t* k;      // e4m3 [pages, heads, S, D]
  uint8_t* v;      // e4m3 [pages, heads, D, S]
  float* ks;       // fp32 [pages, heads]
  float* vs;
  int32_t pages;
  int32_t heads;
  int32_t log_s;   // S = 1 << log_s, 16 .. 256
};

struct KvBatch {
  const int32_t* table;   // [count, max_pages], rows `stride` apart
  const int32_t* lens;    // [count]
  const int32_t* starts;  // [count + 1], or null: one token each
  int64_t stride;
  int32_t count;
  int32_t max_pages;
};

struct KvTokens {
  const uint16_t* k;    // BF16 rows
  const uint16_t* v;
  const uint16_t* q;    // or null
  uint16_t* q_out;
  const float* cos;     // fp32 [positions, half]
  const float* sin;
  int64_t k_tok, k_head, v_tok, v_head, q_tok, q_head, o_tok, o_head;  // strides in elements
  int64_t positions;    // rows of cos / sin (a limit only where half > 0)
  int32_t tokens;
  int32_t group;        // query heads per key/value head
  int32_t half;         // rotated channel pairs
  int32_t interleaved;
};

// Positions stay below 2^31 - 1024, so that a tile's end is in 32 bits; a
// whole number of pages of any size.
__device__ __forceinline__ int32_t kv_capacity(const KvBatch& bt, int32_t log_s) {
  return (int32_t)min((int64_t)bt.max_pages << log_s, (int64_t)INT32_MAX - 1023);
}

// ------------------------------------------------------------------ append
//
// s = the smallest power of two with 448 s >= max|x| (448 = 1.75 * 2^8), not
// amax / 448 as for weights: a page's maximum grows while tokens arrive, and
// every growth takes the stored codes along.  With a ratio of powers of two
// that is a change of exponent, exact except below the smallest normal code;
// with any other ratio each growth would round every earlier token again.

__device__ __forceinline__ float kv_fit_scale(float amax) {
  const uint32_t bits = __float_as_uint(fmaxf(amax, kEps));   // normal: kEps > 2^-126
  return __uint_as_float(((bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0)) << 23);
}

// 1 / s, rounded to fp32: exact for the powers of two that appends make.  A
// page that something else has filled can have another scale, which stays
// while it is large enough; a change of exponent would not be its inverse.
__device__ __forceinline__ float kv_inverse(float s) { return 1.0f / s; }

__device__ __forceinline__ int32_t kv_clamp(int32_t v, int32_t hi) {
  return v < 0 ? 0 : (v > hi ? hi : v);
}

// Four codes times `ratio`, rounded to codes again.
__device__ __forceinline__ uint32_t kv_recode4(uint32_t w, float ratio) {
  const f32x4 x = dq4(w, ratio);
  return cvt4(clamp448(x.x), clamp448(x.y), clamp448(x.z), clamp448(x.w));
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// The largest b in [0, n) with f(b) <= w for a non-decreasing f (0 if none),
// 64 values of f at a time: one round of loads for up to 64 sequences, two
// for up to 4096.  The same in every lane.
template <typename F>
__device__ __forceinline__ int32_t kv_find(int32_t n, int64_t w, F&& f) {
  const int32_t lane = threadIdx.x & 63;
  int32_t lo = 0, span = n;
  while (span > 1) {
    const int32_t step = (span + 63) >> 6;
    const int32_t at = lane * step;
    const bool below = at < span && f(lo + at) <= w;
    const int32_t c = __popcll(__ballot(below));
    if (c == 0) return lo;
    lo += (c - 1) * step;
    span = min(step, span - (c - 1) * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Channels of pair p: (p, p + half) or (2p, 2p + 1) where it is rotated, and
// (2p, 2p + 1) behind the rotated ones.
__device__ __forceinline__ void pair_channels(int32_t p, int32_t half, int32_t interleaved, int32_t& a,
                                              int32_t& b) {
  const bool split = p < half && !interleaved;
  a = split ? p : 2 * p;
  b = split ? p + half : 2 * p + 1;
}

__device__ __forceinline__ float bf16_up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t bf16_down(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// One token for every sequence: a wave for each (sequence, key/value head),
// lanes over channel pairs.  There is nothing to reuse.  One sequence, 32 + 8 +
// 8 heads of 128, takes the chain of dependent loads (length -> page -> scale)
// and the launch, 4 us.  256 sequences take 8.3 in pages of 64; 6.6 in pages
// of 16, where the channels' bytes of v share cache lines, and 7.6 without
// queries, which are loaded and stored in turn behind the keys.
//
// That is without growth.  A page that grows is recoded by its one wave, a
// round trip to memory after another: the last slot of a page of 64 tokens of
// 128 channels 18 us (47 where all 2048 blocks grow at once), of 256 tokens of
// 256 channels 71 (267).  Some page grows in most steps of a large batch: the
// 256 sequences with new random tokens at each step take 19 us, 11 of equal
// magnitudes, which let no page grow (pages of 16: 15 and 9).
template <int D>
__global__ __launch_bounds__(kThreads) void kv_append_step(KvCache c, KvBatch bt, KvTokens t) {
  constexpr int kP = (D / 2 + 63) / 64;   // pairs of a lane
  const int32_t lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (int64_t)bt.count * c.heads) return;
  const int32_t b = (int32_t)(item / c.heads), h = (int32_t)(item - (int64_t)b * c.heads);
  const int32_t pos = max(bt.lens[b], 0) - 1;
  if (pos < 0 || (t.half > 0 && pos >= t.positions)) return;
  const int32_t S = 1 << c.log_s, slot = pos & (S - 1), j = pos >> c.log_s;
  const int32_t page = pos < kv_capacity(bt, c.log_s) ? bt.table[(int64_t)b * bt.stride + j] : -1;
  const bool stored = page >= 0 && page < c.pages;

  float kx[kP], ky[kP], cs[kP], sn[kP];
  uint32_t vw[kP];
  float ka = 0.0f, va = 0.0f;
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int32_t p = lane + 64 * i;
    cs[i] = 1.0f;
    sn[i] = 0.0f;
    if (p < t.half) {
      cs[i] = t.cos[(int64_t)pos * t.half + p];
      sn[i] = t.sin[(int64_t)pos * t.half + p];
    }
    kx[i] = ky[i] = 0.0f;
    vw[i] = 0;
    if (p < D / 2) {
      int32_t ca, cb;
      pair_channels(p, t.half, t.interleaved, ca, cb);
      const uint16_t* kr = t.k + b * t.k_tok + h * t.k_head;
      const float x = bf16_up(kr[ca]), y = bf16_up(kr[cb]);
      kx[i] = p < t.half ? x * cs[i] - y * sn[i] : x;
      ky[i] = p < t.half ? y * cs[i] + x * sn[i] : y;
      vw[i] = *(const uint32_t*)(t.v + b * t.v_tok + h * t.v_head + 2 * p);
      ka = fmaxf(ka, fmaxf(fabsf(kx[i]), fabsf(ky[i])));
      va = fmaxf(va, fmaxf(fabsf(bf_lo(vw[i])), fabsf(bf_hi(vw[i]))));
    }
  }
  if (stored) {
    const int64_t block = (int64_t)page * c.heads + h;
    float k_was = slot ? c.ks[block] : 0.0f, v_was = slot ? c.vs[block] : 0.0f;
    const float k_fit = kv_fit_scale(wave_max(ka)), v_fit = kv_fit_scale(wave_max(va));
    const float k_s = slot ? fmaxf(k_was, k_fit) : k_fit, v_s = slot ? fmaxf(v_was, v_fit) : v_fit;
    uint8_t* kb = c.k + block * S * D;
    uint8_t* vb = c.v + block * S * D;
    const float kr = kv_inverse(k_s), vr = kv_inverse(v_s);
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int32_t p = lane + 64 * i;
      if (p >= D / 2) continue;
      int32_t ca, cb;
      pair_channels(p, t.half, t.interleaved, ca, cb);
      const uint32_t kc = cvt4(clamp448(kx[i] * kr), clamp448(ky[i] * kr), 0.0f, 0.0f);
      kb[slot * D + ca] = (uint8_t)kc;
      kb[slot * D + cb] = (uint8_t)(kc >> 8);
      const uint32_t vc = cvt4(clamp448(bf_lo(vw[i]) * vr), clamp448(bf_hi(vw[i]) * vr), 0.0f, 0.0f);
      vb[(2 * p) * S + slot] = (uint8_t)vc;
      vb[(2 * p + 1) * S + slot] = (uint8_t)(vc >> 8);
    }
    if (lane == 0) {
      c.ks[block] = k_s;
      c.vs[block] = v_s;
    }
    // Growth takes the earlier tokens along: whole 16-token runs of a channel
    // as vectors, the run the new byte lies in byte by byte (only its earlier
    // bytes), so that no two stores of the wave overlap.
    if (slot > 0 && k_s > k_was) {
      const float ratio = k_was * kr;
      for (int32_t i = lane; i < slot * (D / 16); i += 64) {
        u32x4* at = (u32x4*)kb + i;
        u32x4 w = *at;
        for (int x = 0; x < 4; ++x) w[x] = kv_recode4(w[x], ratio);
        *at = w;
      }
    }
    if (slot > 0 && v_s > v_was) {
      const float ratio = v_was * vr;
      const int32_t runs = slot >> 4, rest = slot & 15;
      for (int32_t d = lane; d < D; d += 64) {
        for (int32_t r = 0; r < runs; ++r) {
          u32x4* at = (u32x4*)(vb + d * S) + r;
          u32x4 w = *at;
          for (int x = 0; x < 4; ++x) w[x] = kv_recode4(w[x], ratio);
          *at = w;
        }
        for (int32_t x = 0; x < rest; ++x) {
          uint8_t* at = vb + d * S + (slot & ~15) + x;
          *at = (uint8_t)kv_recode4(*at, ratio);
        }
      }
    }
  }
  if (t.q == nullptr) return;
  for (int32_t g = 0; g < t.group; ++g) {
    const uint16_t* qr = t.q + b * t.q_tok + ((int64_t)h * t.group + g) * t.q_head;
    uint16_t* qo = t.q_out + b * t.o_tok + ((int64_t)h * t.group + g) * t.o_head;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int32_t p = lane + 64 * i;
      if (p >= D / 2) continue;
      int32_t ca, cb;
      pair_channels(p, t.half, t.interleaved, ca, cb);
      const float x = bf16_up(qr[ca]), y = bf16_up(qr[cb]);
      qo[ca] = bf16_down(p < t.half ? x * cs[i] - y * sn[i] : x);
      qo[cb] = bf16_down(p < t.half ? y * cs[i] + x * sn[i] : y);
    }
  }
}

// 16 channels of a row, in two runs of 8 at channels a and b: both halves of
// 8 rotated pairs, or 16 channels side by side.
__device__ __forceinline__ void unit_channels(int32_t u, int32_t half, int32_t interleaved, int32_t& a,
                                              int32_t& b) {
  const bool split = 8 * u < half && !interleaved;
  a = split ? 8 * u : 16 * u;
  b = split ? half + 8 * u : 16 * u + 8;
}

// The bytes lo .. hi - 1 of 16, as a mask.
__device__ __forceinline__ u32x4 kv_bytes(int32_t lo, int32_t hi) {
  u32x4 keep;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t w = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) w |= 4 * e + y >= lo && 4 * e + y < hi ? 0xFFu << (8 * y) : 0u;
    keep[e] = w;
  }
  return keep;
}

// cos and sin of a unit's 8 pairs.
struct KvTurn {
  f32x4 cs[2], sn[2];
  bool turn;
};

__device__ __forceinline__ KvTurn kv_turn(const KvTokens& t, int64_t pos, int32_t u) {
  KvTurn w;
  w.turn = 8 * u < t.half;
  if (w.turn) {
    const f32x4* cp = (const f32x4*)(t.cos + pos * t.half + 8 * u);
    const f32x4* sp = (const f32x4*)(t.sin + pos * t.half + 8 * u);
    w.cs[0] = cp[0];
    w.cs[1] = cp[1];
    w.sn[0] = sp[0];
    w.sn[1] = sp[1];
  }
  return w;
}

// The 16 values of a unit (read as two 16-byte words), rotated.
__device__ __forceinline__ void unit_rotate(u32x4 lo, u32x4 hi, const KvTurn& w, int32_t interleaved, float (&x)[16]) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(lo[i]);
    x[2 * i + 1] = bf_hi(lo[i]);
    x[8 + 2 * i] = bf_lo(hi[i]);
    x[8 + 2 * i + 1] = bf_hi(hi[i]);
  }
  if (!w.turn) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float cs = w.cs[i >> 2][i & 3], sn = w.sn[i >> 2][i & 3];
    const float a = interleaved ? x[2 * (i & 3) + 8 * (i >> 2)] : x[i];
    const float b = interleaved ? x[2 * (i & 3) + 1 + 8 * (i >> 2)] : x[8 + i];
    y[i] = a * cs - b * sn;
    y[8 + i] = b * cs + a * sn;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = interleaved ? y[i] : y[2 * i];
    x[2 * i + 1] = interleaved ? y[8 + i] : y[2 * i + 1];
  }
}

// 16 tokens of two channels of v as codes: two 16-byte words.
__device__ __forceinline__ void run_codes(const uint32_t (&pairs)[16], float r, u32x4 (&out)[2]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    out[0][x] = cvt4(clamp448(bf_lo(pairs[4 * x]) * r), clamp448(bf_lo(pairs[4 * x + 1]) * r),
                     clamp448(bf_lo(pairs[4 * x + 2]) * r), clamp448(bf_lo(pairs[4 * x + 3]) * r));
    out[1][x] = cvt4(clamp448(bf_hi(pairs[4 * x]) * r), clamp448(bf_hi(pairs[4 * x + 1]) * r),
                     clamp448(bf_hi(pairs[4 * x + 2]) * r), clamp448(bf_hi(pairs[4 * x + 3]) * r));
  }
}

// Sequences with any number of new tokens: a workgroup for each (page that a
// sequence writes, key/value head), which owns the block's scale: no other
// workgroup touches it, so there are no atomics and the result does not
// depend on any order.  Slot w of the grid belongs to the sequence with
// floor(starts[b] / S) + 2 b <= w, which leaves every sequence at least as
// many slots as its tokens can span pages.  Heads run fastest over the grid:
// the workgroups that share the rows of a projection's output run together.
//
// Streaming work, bound by HBM: a thread holds its part of a page in registers
// between the maximum and the codes, so that each input is read once (pages of
// more than kHoldK * 256 units are read a second time, out of the caches); it
// takes 16 channels of a token of k, with the rotation's row, which the
// group's queries share, and 16 tokens of two channels of v, whose codes are
// two 16-byte stores.  Rows of k and q pass the caches by (91 -> 83 us for
// 17,633 tokens of 32 + 8 + 8 heads of 128: 4.9 TB/s, as a large copy); codes,
// whose stores are parts of cache lines, do not (107 us).  A workgroup for k
// and one for v of their own measured slower (105 us).
template <int D>
__global__ __launch_bounds__(kThreads, 3) void kv_append_pages(KvCache c, KvBatch bt, KvTokens t) {
  constexpr int kU = D / 16;
  constexpr int kHoldK = 2, kHoldV = 1;
  constexpr int kQ = 2;   // queries loaded at a time
  __shared__ float red[8];
  const int32_t tid = threadIdx.x;
  const int32_t w = blockIdx.x / c.heads, h = blockIdx.x - w * c.heads;
  const int32_t S = 1 << c.log_s;
  auto first_slot = [&](int32_t b) {
    return (int64_t)(kv_clamp(bt.starts[b], t.tokens) >> c.log_s) + 2 * (int64_t)b;
  };
  const int32_t b = kv_find(bt.count, w, first_slot);
  const int64_t j0 = w - first_slot(b);
  const int32_t row0 = kv_clamp(bt.starts[b], t.tokens);
  const int32_t n = kv_clamp(bt.starts[b + 1], t.tokens) - row0;
  if (j0 < 0 || n <= 0) return;
  const int64_t len = bt.lens[b], start = len - n;
  const int64_t begin = start < 0 ? 0 : start;
  const int64_t j = (begin >> c.log_s) + j0;
  const int64_t lo = max(begin, j << c.log_s);
  int64_t hi = min(len, (j + 1) << c.log_s);
  if (t.half > 0) hi = min(hi, t.positions);
  if (lo >= hi) return;
  const int32_t page = lo < kv_capacity(bt, c.log_s) ? bt.table[(int64_t)b * bt.stride + j] : -1;
  const bool stored = page >= 0 && page < c.pages;
  const int32_t held = (int32_t)(lo - (j << c.log_s));   // earlier tokens in the page
  const int32_t count = (int32_t)(hi - lo);
  const int64_t row = row0 + (lo - start);               // input row of the first token
  const int64_t block = (int64_t)max(page, 0) * c.heads + h;
  const float k_was = held && stored ? c.ks[block] : 0.0f, v_was = held && stored ? c.vs[block] : 0.0f;

  // Unit i of the page's new tokens: of k, and of the queries of the group,
  // which are done with it.
  auto rotate_k = [&](int32_t i, float (&x)[16], bool queries) {
    const int32_t tok = i / kU, u = i - tok * kU;
    int32_t ca, cb;
    unit_channels(u, t.half, t.interleaved, ca, cb);
    const KvTurn turn = kv_turn(t, lo + tok, u);
    const uint16_t* kp = t.k + (row + tok) * t.k_tok + h * t.k_head;
    const u32x4 ka = __builtin_nontemporal_load((const u32x4*)(kp + ca)), kz = __builtin_nontemporal_load((const u32x4*)(kp + cb));
    if (queries) {
      const uint16_t* qp = t.q + (row + tok) * t.q_tok + (int64_t)h * t.group * t.q_head;
      uint16_t* to = t.q_out + (row + tok) * t.o_tok + (int64_t)h * t.group * t.o_head;
      for (int32_t g0 = 0; g0 < t.group; g0 += kQ) {
        u32x4 qa[kQ], qz[kQ];
#pragma unroll
        for (int g = 0; g < kQ; ++g) {
          const int64_t at = min(g0 + g, t.group - 1) * t.q_head;
          qa[g] = __builtin_nontemporal_load((const u32x4*)(qp + at + ca));
          qz[g] = __builtin_nontemporal_load((const u32x4*)(qp + at + cb));
        }
#pragma unroll
        for (int g = 0; g < kQ; ++g) {
          if (g0 + g >= t.group) continue;
          float y[16];
          unit_rotate(qa[g], qz[g], turn, t.interleaved, y);
          bf16x8 ya, yz;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ya[e] = (__bf16)y[e];
            yz[e] = (__bf16)y[8 + e];
          }
          __builtin_nontemporal_store(__builtin_bit_cast(u32x4, ya), (u32x4*)(to + (g0 + g) * t.o_head + ca));
          __builtin_nontemporal_store(__builtin_bit_cast(u32x4, yz), (u32x4*)(to + (g0 + g) * t.o_head + cb));
        }
      }
    }
    unit_rotate(ka, kz, turn, t.interleaved, x);
  };
  // 16 tokens of the channels 2 p, 2 p + 1 of v, zeros for those that are not new.
  const int32_t r0 = held >> 4, runs = ((held + count + 15) >> 4) - r0;
  auto pairs_v = [&](int32_t i, uint32_t (&pairs)[16]) {
    const int32_t a = 16 * (r0 + i / (D / 2)) - held, p = i % (D / 2);
    const uint16_t* src = t.v + row * t.v_tok + h * t.v_head + 2 * p;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      pairs[e] = a + e >= 0 && a + e < count ? *(const uint32_t*)(src + (int64_t)(a + e) * t.v_tok) : 0u;
    }
  };

  float kx[kHoldK][16];
  uint32_t vx[kHoldV][16];
  float ka = 0.0f;
  uint32_t va = 0;
  const bool queries = t.q != nullptr;
#pragma unroll
  for (int y = 0; y < kHoldK; ++y) {
    const int32_t i = tid + y * kThreads;
    if (i < count * kU) {
      rotate_k(i, kx[y], queries);
#pragma unroll
      for (int e = 0; e < 16; ++e) ka = fmaxf(ka, fabsf(kx[y][e]));
    }
  }
  for (int32_t i = tid + kHoldK * kThreads; i < count * kU; i += kThreads) {
    float x[16];
    rotate_k(i, x, queries);
#pragma unroll
    for (int e = 0; e < 16; ++e) ka = fmaxf(ka, fabsf(x[e]));
  }
#pragma unroll
  for (int y = 0; y < kHoldV; ++y) {
    const int32_t i = tid + y * kThreads;
    if (stored && i < runs * (D / 2)) {
      pairs_v(i, vx[y]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) vx[y][e] = 0;
    }
  }
  if (!stored) return;
#pragma unroll
  for (int y = 0; y < kHoldV; ++y) {
#pragma unroll
    for (int e = 0; e < 16; ++e) va = pk_max_u16(va, vx[y][e] & 0x7FFF7FFFu);
  }
  for (int32_t i = tid + kHoldV * kThreads; i < runs * (D / 2); i += kThreads) {
    uint32_t x[16];
    pairs_v(i, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) va = pk_max_u16(va, x[e] & 0x7FFF7FFFu);
  }
  ka = wave_max(ka);
  const float vm = wave_max(__uint_as_float(halves_max(va) << 16));
  if ((tid & 63) == 0) {
    red[tid >> 6] = ka;
    red[4 + (tid >> 6)] = vm;
  }
  __syncthreads();
  const float k_fit = kv_fit_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  const float v_fit = kv_fit_scale(fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7])));
  const float k_s = held ? fmaxf(k_was, k_fit) : k_fit, v_s = held ? fmaxf(v_was, v_fit) : v_fit;
  const float kr = kv_inverse(k_s), vr = kv_inverse(v_s);
  if (tid == 0) {
    c.ks[block] = k_s;
    c.vs[block] = v_s;
  }
  uint8_t* kb = c.k + block * S * D;
  uint8_t* vb = c.v + block * S * D;

  auto store_k = [&](int32_t i, const float (&x)[16]) {
    const int32_t tok = i / kU, u = i - tok * kU;
    int32_t ca, cb;
    unit_channels(u, t.half, t.interleaved, ca, cb);
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = clamp448(x[e] * kr);
    uint8_t* to = kb + (held + tok) * D;
    *(u32x2*)(to + ca) = u32x2{cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7])};
    *(u32x2*)(to + cb) = u32x2{cvt4(y[8], y[9], y[10], y[11]), cvt4(y[12], y[13], y[14], y[15])};
  };
  const bool v_grown = held > 0 && v_s > v_was;
  const float v_ratio = v_was * vr;
  // Runs that hold only some new tokens are read, merged and written back.
  auto store_v = [&](int32_t i, const uint32_t (&pairs)[16]) {
    const int32_t r = r0 + i / (D / 2), p = i % (D / 2), a = 16 * r - held;
    u32x4 out[2];
    run_codes(pairs, vr, out);
    u32x4* at[2] = {(u32x4*)(vb + (2 * p) * S) + r, (u32x4*)(vb + (2 * p + 1) * S) + r};
    if (a < 0 || a + 16 > count) {
      const u32x4 is_new = kv_bytes(-a, count - a), before = kv_bytes(0, -a);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const u32x4 was = *at[y];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t again = v_grown ? kv_recode4(was[x], v_ratio) : was[x];
          out[y][x] = (out[y][x] & is_new[x]) | (again & before[x]) | (was[x] & ~(is_new[x] | before[x]));
        }
      }
    }
    *at[0] = out[0];
    *at[1] = out[1];
  };
#pragma unroll
  for (int y = 0; y < kHoldK; ++y) {
    const int32_t i = tid + y * kThreads;
    if (i < count * kU) store_k(i, kx[y]);
  }
#pragma unroll
  for (int y = 0; y < kHoldV; ++y) {
    const int32_t i = tid + y * kThreads;
    if (i < runs * (D / 2)) store_v(i, vx[y]);
  }
  for (int32_t i = tid + kHoldK * kThreads; i < count * kU; i += kThreads) {
    float x[16];
    rotate_k(i, x, false);
    store_k(i, x);
  }
  for (int32_t i = tid + kHoldV * kThreads; i < runs * (D / 2); i += kThreads) {
    uint32_t x[16];
    pairs_v(i, x);
    store_v(i, x);
  }
  // Growth takes the earlier tokens along; those in the first new run of v
  // have gone with it.
  if (held > 0 && k_s > k_was) {
    const float ratio = k_was * kr;
    for (int32_t i = tid; i < held * kU; i += kThreads) {
      u32x4* at = (u32x4*)kb + i;
      u32x4 x = *at;
      for (int e = 0; e < 4; ++e) x[e] = kv_recode4(x[e], ratio);
      *at = x;
    }
  }
  if (v_grown) {
    for (int32_t i = tid; i < r0 * D; i += kThreads) {
      u32x4* at = (u32x4*)(vb + (i % D) * S) + i / D;
      u32x4 x = *at;
      for (int e = 0; e < 4; ++e) x[e] = kv_recode4(x[e], v_ratio);
      *at = x;
    }
  }
}

// --------------------------------------------------------------- attention

struct KvQuery {
  const uint16_t* q;   // BF16 rows
  uint16_t* out;
  float* lse;          // fp32 [tokens, query heads], or null
  float* part;         // partial sums [heads, slots, R, D], or null: no splits
  float2* part_ml;     // their maxima and sums [heads, slots, R]
  int2* rows;          // first slot and count of each query row's partials
  int64_t q_tok, q_head, o_tok, o_head;
  int32_t tokens;
  int32_t group;
  int32_t window;      // 0: none
  int32_t slots;       // places for partial sums per key/value head
  int32_t target;      // work items per head that splitting aims at; 0: no splits
  int32_t jump;        // second and later slots of a row tile: first + jump + 1, ...
  int32_t min_tiles;   // least key tiles of a split
  int32_t tile_rows;   // rows of a row tile where R below is 0
  int32_t extra;       // what starting and ending a row tile counts for in a share, in tiles
  float scale;         // of the scores, times log2(e)
};

// Rows of a row tile: R, or with R = 0 what the call says.
template <int R>
__device__ __forceinline__ int32_t kv_tile_rows(const KvQuery& p) {
  return R > 0 ? R : p.tile_rows;
}

constexpr int kKeyTile = 64;
// Least factor of a score: a masked one, minus infinity, stays that.
constexpr float kTiny = 1.17549435e-38f;
// Least scale of v, 2^-64: its logarithm is taken, and weights times it stay
// normal numbers.
constexpr float kLeastVScale = 5.421010862427522e-20f;
// The work of one workgroup: a tile of query rows of a sequence and a range
// of its key tiles.
struct KvWork {
  int32_t b, n, row0;       // sequence, its query tokens, their first row
  int32_t first, count;     // first query row (token * group + head in group) of the tile; rows of the sequence
  int32_t pos0;             // position of the sequence's first query token
  int32_t tile0, tile1;     // key tiles
  int32_t parts, slot;      // how many work items share the row tile's keys, and where this one's sums go
  bool begin;               // whether this one has the first of them
};

// Sum over lanes 0 .. i, for every lane i (data-parallel moves, no LDS).
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
  auto from = [](T x, auto ctrl, auto rows) {
    auto move = [](int y) {
      return __builtin_amdgcn_update_dpp(0, y, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    };
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(T, move(__builtin_bit_cast(int, x)));
    } else {
      return (T)(((uint64_t)(uint32_t)move((int)(x >> 32)) << 32) | (uint32_t)move((int)x));
    }
  };
  using std::integral_constant;
  v += from(v, integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});   // row_shr:1
  v += from(v, integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // last lane of the row before
  v += from(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // last lane of the first half
  return v;
}

__device__ __forceinline__ int32_t lane_of(int32_t v, int32_t lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int64_t lane_of(int64_t v, int32_t lane) {
  return (int64_t)(((uint64_t)(uint32_t)lane_of((int32_t)(v >> 32), lane) << 32) | (uint32_t)lane_of((int32_t)v, lane));
}

// The first position that a query at pos - 1 sees.
__device__ __forceinline__ int32_t kv_low(int32_t end, int32_t window) {
  return window > 0 ? max(max(end, 0) - window, 0) : 0;
}

// A sequence of the call: its rows, and its key tiles as far as any of its
// queries sees them.
struct KvSeq {
  int32_t row0, n, len, rtiles, tile0, tiles;
};

template <int R>
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& bt, const KvQuery& p, int32_t cap, int32_t b) {
  KvSeq s{0, 0, 0, 0, 0, 0};
  if (b >= bt.count) return s;
  s.len = max(bt.lens[b], 0);
  if (bt.starts) {
    s.row0 = kv_clamp(bt.starts[b], p.tokens);
    s.n = max(kv_clamp(bt.starts[b + 1], p.tokens) - s.row0, 0);
  } else {
    s.row0 = b;
    s.n = 1;
  }
  const uint32_t rows = (uint32_t)kv_tile_rows<R>(p);
  s.rtiles = (int32_t)(((uint32_t)s.n * (uint32_t)p.group + rows - 1) / rows);   // at most 2^25 rows
  const int32_t hi = min(s.len, cap), lo = kv_low(s.len - s.n + 1, p.window);
  if (s.n > 0 && hi > lo) {
    s.tile0 = lo / kKeyTile;
    s.tiles = (hi + kKeyTile - 1) / kKeyTile - s.tile0;
  }
  return s;
}

__device__ __forceinline__ KvSeq lane_of(const KvSeq& s, int32_t lane) {
  return KvSeq{lane_of(s.row0, lane), lane_of(s.n, lane), lane_of(s.len, lane),
               lane_of(s.rtiles, lane), lane_of(s.tile0, lane), lane_of(s.tiles, lane)};
}

// Every wave reads the batch's lengths and finds its work by itself, in one of
// two ways.  Grids depend on the number of sequences and query tokens alone,
// so a captured launch stays right, and balanced, as the lengths grow.
//
// kv_plan, for workgroups that do one item each: sequence b has
// ceil(rows / R) row tiles of ceil(key tiles / chunk) splits each, with one
// chunk for the whole batch such that about `target` items come out of it.
template <int R>
__device__ __forceinline__ bool kv_plan(const KvBatch& bt, const KvQuery& p, int32_t cap, int32_t w, KvWork& k) {
  const int32_t lane = threadIdx.x & 63;
  KvSeq mine = kv_seq<R>(bt, p, cap, lane);
  int32_t chunk = INT32_MAX;
  if (p.target > 0) {
    // fp32 is enough, with room for its rounding: the chunk may only be too
    // long, never so short that there are more items than slots
    float total = (float)mine.rtiles * (float)mine.tiles;
    for (int32_t b = 64; b < bt.count; b += 64) {
      const KvSeq s = kv_seq<R>(bt, p, cap, b + lane);
      total += (float)s.rtiles * (float)s.tiles;
    }
    total = __int_as_float(lane_of(__float_as_int(wave_scan(total)), 63));
    const float per = __builtin_ceilf(total * 1.0001f / (float)p.target);
    chunk = max((int32_t)fminf(per, 1e9f), p.min_tiles);
  }
  int64_t before = 0;
  for (int32_t b0 = 0; b0 < bt.count; b0 += 64) {
    if (b0 > 0) mine = kv_seq<R>(bt, p, cap, b0 + lane);
    const int32_t splits = max(1, (int32_t)(((int64_t)mine.tiles + chunk - 1) / chunk));
    const int32_t items = (int32_t)min((int64_t)mine.rtiles * splits, (int64_t)1 << 24);
    const int32_t sum = wave_scan(items);
    const uint64_t past = __ballot(before + sum > w);
    if (past != 0) {
      const int32_t at = __ffsll((unsigned long long)past) - 1;
      const KvSeq s = lane_of(mine, at);
      const int32_t of = lane_of(splits, at);
      const int32_t local = (int32_t)(w - before) - (lane_of(sum, at) - lane_of(items, at));
      const int32_t rtile = local / of, split = local - rtile * of;
      k.b = b0 + at;
      k.row0 = s.row0;
      k.n = s.n;
      k.pos0 = s.len - s.n;
      k.parts = of;
      k.begin = split == 0;
      // the last rows see the most keys: they go first
      k.first = (s.rtiles - 1 - rtile) * R;
      k.count = s.n * p.group;
      k.tile0 = s.tile0 + min((int64_t)split * chunk, (int64_t)s.tiles);
      k.tile1 = s.tile0 + min((int64_t)(split + 1) * chunk, (int64_t)s.tiles);
      k.slot = w;
      return true;
    }
    before += lane_of(sum, 63);
  }
  return false;
}

// KvShares, for a grid that the chip holds at once: the key tiles of all row
// tiles, one after another, are cut into `target` equal shares.  A workgroup
// goes through its share row tile by row tile; only the first and the last of
// them can continue in a neighbour's.  Everyone ends at the same time whatever
// the lengths are, and nothing is started twice.  The partial sums of a row
// tile that begins in share i are slot i, those of it in a later share j slot
// target + j.  With a target of 0 (short tables) every workgroup has one whole
// row tile.
template <int R>
struct KvShares {
  const KvBatch& bt;
  const KvQuery& p;
  int32_t cap, index;
  int64_t at, end, share;   // this share's tiles (row tiles: target 0), counted over the whole batch
  int32_t b, rtile, t;      // the next one's sequence, row tile and tile
  KvSeq s;

  // Units of a row tile: one that sees nothing is written, too.
  __device__ __forceinline__ int32_t units(const KvSeq& s) const { return p.target == 0 ? 1 : max(s.tiles, 1) + p.extra; }
  __device__ __forceinline__ int64_t weight(const KvSeq& s) const { return (int64_t)s.rtiles * units(s); }

  __device__ __forceinline__ KvShares(const KvBatch& bt_, const KvQuery& p_, int32_t cap_, int32_t index_)
      : bt(bt_), p(p_), cap(cap_), index(index_), at(0), end(0), share(1), b(0), rtile(0), t(0) {
    const int32_t lane = threadIdx.x & 63;
    KvSeq mine = kv_seq<R>(bt, p, cap, lane);
    if (p.target == 0) {
      at = index;
      end = at + 1;
    } else {
      int64_t total = lane_of(wave_scan(weight(mine)), 63);
      for (int32_t b0 = 64; b0 < bt.count; b0 += 64) {
        total += lane_of(wave_scan(weight(kv_seq<R>(bt, p, cap, b0 + lane))), 63);
      }
      share = (int64_t)__builtin_ceil((double)total / (double)p.target);
      if (share * p.target < total) ++share;
      share = lane_of(max(share, (int64_t)p.min_tiles), 0);
      at = index * share;
      end = min(at + share, total);
      if (at >= end) return;
    }
    int64_t before = 0;
    for (int32_t b0 = 0; b0 < bt.count; b0 += 64) {
      if (b0 > 0) mine = kv_seq<R>(bt, p, cap, b0 + lane);
      const int64_t w = weight(mine), sum = wave_scan(w);
      const uint64_t past = __ballot(before + sum > at);
      if (past != 0) {
        const int32_t which = __ffsll((unsigned long long)past) - 1;
        s = lane_of(mine, which);
        b = b0 + which;
        const int64_t off = at - (before + lane_of(sum, which) - lane_of(w, which));
        const int32_t tiles = units(s);
        rtile = off < tiles ? 0 : (int32_t)(off / tiles);
        t = (int32_t)(off - (int64_t)rtile * tiles);
        return;
      }
      before += lane_of(sum, 63);
    }
    end = at;   // beyond the last one
  }

  __device__ __forceinline__ bool next(KvWork& k) {
    if (at >= end) return false;
    // the next sequence that has rows, 64 at a time
    while (rtile >= s.rtiles) {
      if (++b >= bt.count) return false;
      const KvSeq mine = kv_seq<R>(bt, p, cap, b + (threadIdx.x & 63));
      const uint64_t has = __ballot(mine.rtiles > 0);
      const int32_t which = has != 0 ? __ffsll((unsigned long long)has) - 1 : 63;
      s = lane_of(mine, which);
      b += which;
      rtile = 0;
    }
    const int32_t tiles = units(s);
    const int32_t take = (int32_t)min((int64_t)(tiles - t), end - at);
    k.b = b;
    k.row0 = s.row0;
    k.n = s.n;
    k.pos0 = s.len - s.n;
    k.first = rtile * kv_tile_rows<R>(p);
    k.count = s.n * p.group;
    k.tile0 = s.tile0 + max(t - p.extra, 0);
    k.tile1 = s.tile0 + (p.target == 0 ? s.tiles : min(max(t + take - p.extra, 0), s.tiles));
    k.begin = t == 0;
    k.parts = 1;
    if (t > 0 || t + take < tiles) {
      k.parts = 1 + (int32_t)((at - t + tiles - 1) / share) - (int32_t)((at - t) / share);
    }
    k.slot = k.begin ? index : p.target + index;
    at += take;
    t = 0;
    ++rtile;
    return true;
  }
};

// What the query rows of a work item see: some of them keys see_lo ..
// see_hi - 1, all of them all_lo .. all_hi - 1; and the tiles to visit.
struct KvSeen {
  int32_t see_lo, see_hi, all_lo, all_hi, tile0, tile1;
};

template <int R>
__device__ __forceinline__ KvSeen kv_seen(const KvWork& k, const KvQuery& p, int32_t cap) {
  const int32_t first = k.pos0 + k.first / p.group + 1;
  const int32_t last = k.pos0 + min(k.first + R - 1, k.count - 1) / p.group + 1;
  KvSeen s;
  s.see_hi = min(last, cap);
  s.all_hi = min(first, cap);
  s.see_lo = kv_low(first, p.window);
  s.all_lo = kv_low(last, p.window);
  s.tile0 = max(k.tile0, s.see_lo / kKeyTile);
  s.tile1 = min(k.tile1, (max(s.see_hi, 0) + kKeyTile - 1) / kKeyTile);
  return s;
}

// Eight codes (two dwords) as BF16, exactly.
__device__ __forceinline__ bf16x8 kv_widen(uint32_t a, uint32_t b) {
  const bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

// Infinite queries as NaN (the exponent's carry sets the top bit of the
// mantissa).  A row with either is then NaN as its scores are, each of them: an
// infinity alone can give -inf for every key, which is what a row that sees
// nothing has, and whose sums are zeros.
__device__ __forceinline__ u32x4 kv_no_infinity(u32x4 x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] |= (((x[e] & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u) >> 9;
  return x;
}

// Maximum and sum of a part of a row's keys.  A sum that is NaN may have no
// maximum; with infinity for one, joining the parts keeps it (passing over
// those without a maximum there costs nothing, adding them up 1 us in 12).
__device__ __forceinline__ float2 kv_part_ml(float m, float l) { return float2{l != l ? INFINITY : m, l}; }

// The largest part of D channels, in equal parts of whole 16s, within `most`.
constexpr int kv_part(int d, int most) {
  int parts = 1;
  while (d / parts > most || d % (16 * parts) != 0) ++parts;
  return d / parts;
}

// Waves of kv_attend_rows that a SIMD holds: what its registers allow without
// spilling (a spill of four registers at D = 256 took a 91 us call to 107).
constexpr int kv_rows_per_simd(int d, int nt) { return nt > 1 ? 1 : (d == 64 ? 4 : (d == 128 ? 3 : 2)); }

// Few query rows: R = 16 NT rows of a sequence (tokens times the query heads
// that share a key head) in each of four waves, which take every fourth key
// tile of the workgroup's range and join their sums at its end.
//
// Scores are computed transposed, S^T = K Q^T, a tile of 64 keys as four
// 16x16x32 products per 32 channels.  Row m of product t is given token
// 16 (m / 4) + 4 t + m % 4, so that lane group g (16 lanes) ends up with the
// 16 consecutive tokens 16 g .. 16 g + 15 of its query row: one page, one pair
// of scales, and exactly the operand order of O^T = V^T P^T, whose lanes read
// 16 tokens of a channel in one load.  No key or value goes through LDS, which
// holds the queries and, at the end, the sums of the four waves; softmax
// needs one exchange across the four lane groups per tile.
//
// Codes are widened to BF16 exactly and multiplied there (BF16 products with
// fp32 sums); scales enter in fp32, k's with the score, v's with the weight,
// which is then rounded to BF16 once (relative 2^-8 at most, its sum is not).
//
// Bound by HBM.  One token each of 128 sequences of up to 16384, 32 heads over
// 8 of 128: 351 us, 6.2 TB/s; one sequence of 131071: 44 us, 6.2 TB/s, and 5
// for the join; 48 sequences under a window of 4096, heads of 256: 83 us, 4.6 TB/s,
// where 256 registers leave two waves per SIMD.  Reads pass the caches by
// (NT hints: 61 -> 57 us for the one sequence), as each byte is read once.
template <int D, int NT>
__global__ __launch_bounds__(kThreads, kv_rows_per_simd(D, NT)) void kv_attend_rows(KvCache c, KvBatch bt, KvQuery p) {
  constexpr int R = 16 * NT;
  constexpr int kI = D / 64;    // 64-channel pieces
  constexpr int kDt = D / 16;   // 16-channel tiles of the output
  constexpr int kPart = kv_part(D, 2048 / R);   // channels that are joined at a time: 8 per thread at most
  // the queries, later the waves' sums
  constexpr int kSums = 4 * R * (kPart + 4), kQueries = R * (D + 8) / 2;
  __shared__ __align__(16) float lds[kSums > kQueries ? kSums : kQueries];
  __shared__ float lds_m[4][R], lds_l[4][R];
  const int32_t w_item = blockIdx.x / c.heads, h = blockIdx.x - w_item * c.heads;
  const int32_t S = 1 << c.log_s, cap = kv_capacity(bt, c.log_s);
  const float scale = fabsf(p.scale);
  const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the factor below is positive
  KvShares<R> shares(bt, p, cap, w_item);
  KvWork wk;
  while (shares.next(wk)) {
    // Hidden from the compiler, which would keep what follows from it in
    // registers across row tiles and spill others for that.
    int32_t tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int32_t lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t col = lane & 15, grp = lane >> 4, k_run = col >> 2;
    const KvSeen see = kv_seen<R>(wk, p, cap);
    const int32_t* table = bt.table + (int64_t)wk.b * bt.stride;
    // Page of a run of 16 tokens, -1 where none of them is seen or the table's
    // entry is no page.
    auto page_at = [&](int32_t tile, int32_t run) {
      const int32_t t0 = min(tile, see.tile1 - 1) * kKeyTile + 16 * run;
      int32_t pg = -1;
      if (t0 < see.see_hi && t0 + 16 > see.see_lo) pg = table[t0 >> c.log_s];
      return pg >= 0 && pg < c.pages ? pg : -1;
    };
    u32x4 xk[4][kI], xv[kDt];
    float ks, vs;
    auto load_k = [&](int32_t tile, int32_t pk, int32_t pv) {
      const int32_t tk = tile * kKeyTile + 16 * k_run;
      const int64_t kblock = (int64_t)max(pk, 0) * c.heads + h, vblock = (int64_t)max(pv, 0) * c.heads + h;
      const uint8_t* kp = c.k + kblock * S * D + ((tk & (S - 1)) + (col & 3)) * D + 16 * grp;
#pragma unroll
      for (int i = 0; i < kI; ++i) {
#pragma unroll
        for (int t = 0; t < 4; ++t) xk[t][i] = __builtin_nontemporal_load((const u32x4*)(kp + t * 4 * D + 64 * i));
      }
      ks = c.ks[vblock];
      vs = c.vs[vblock];
    };
    // Not past the cache: a page row of v longer than a tile is read in pieces
    // of half a cache line, whose other half the next tile's wave wants.
    auto load_v = [&](int32_t tile, int32_t pv) {
      const int32_t tv = tile * kKeyTile + 16 * grp;
      const int64_t vblock = (int64_t)max(pv, 0) * c.heads + h;
      const uint8_t* vp = c.v + vblock * S * D + (int64_t)col * S + (tv & (S - 1));
#pragma unroll
      for (int i = 0; i < kDt; ++i) {
        xv[i] = *(const u32x4*)(vp + i * 16 * S);
      }
    };

    int32_t tile = see.tile0 + wave;
    int32_t pk = -1, pv = -1, pk_next = -1, pv_next = -1;
    if (tile < see.tile1) {
      pk = page_at(tile, k_run);
      pv = page_at(tile, grp);
      load_k(tile, pk, pv);
      pk_next = page_at(tile + 4, k_run);
      pv_next = page_at(tile + 4, grp);
    }
    // The queries in LDS, where all waves read them: row pitch 2 D + 16 bytes.
    uint16_t* q_lds = (uint16_t*)lds;
    for (int32_t i = tid; i < R * (D / 8); i += kThreads) {
      const int32_t rr = i / (D / 8), ch = i - rr * (D / 8), r = wk.first + rr;
      u32x4 x = {0, 0, 0, 0};
      if (r < wk.count) {
        const int32_t tok = r / p.group, g = r - tok * p.group;
        x = *(const u32x4*)(p.q + (wk.row0 + tok) * p.q_tok + ((int64_t)h * p.group + g) * p.q_head + 8 * ch);
        x = kv_no_infinity(x ^ u32x4{flip, flip, flip, flip});
      }
      *(u32x4*)(q_lds + rr * (D + 8) + 8 * ch) = x;
    }
    f32x4 o[NT][kDt];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.0f;
#pragma unroll
      for (int i = 0; i < kDt; ++i) o[nt][i] = f32x4{0, 0, 0, 0};
    }
    __syncthreads();

    // One tile at a time: its values' loads are in flight during the softmax,
    // the next one's keys when the others compute.  Two or three workgroups
    // to a CU keep more than enough bytes in flight; loading further ahead
    // measured no gain, and its registers cost a workgroup.
    for (; tile < see.tile1; tile += 4) {
      const int32_t pk_after = page_at(tile + 8, k_run), pv_after = page_at(tile + 8, grp);
      const bool ok = pv >= 0;
      const float f = ok ? fmaxf(ks * scale, kTiny) : 1.0f, vw = ok ? fmaxf(vs, kLeastVScale) : 0.0f;
      const int32_t t0 = tile * kKeyTile;
      f32x4 s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int t = 0; t < 4; ++t) s[nt][t] = f32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        bf16x8 q[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            q[nt][y] = *(const bf16x8*)(q_lds + (nt * 16 + col) * (D + 8) + 64 * i + 16 * grp + 8 * y);
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const bf16x8 a = kv_widen(xk[t][i][0], xk[t][i][1]), b = kv_widen(xk[t][i][2], xk[t][i][3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[nt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[nt][0], s[nt][t], 0, 0, 0);
            s[nt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, q[nt][1], s[nt][t], 0, 0, 0);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // the values' registers are the keys'
      load_v(tile, pv);
      const bool edge = __ballot(!ok) != 0 || t0 < see.all_lo || t0 + kKeyTile > see.all_hi;
      const int32_t run = t0 + 16 * grp;
      if (edge) {
        int32_t r = wk.first + col;
        asm volatile("" : "+v"(r));   // few tiles are edges: no registers for this across the others
#pragma unroll
        for (int nt = 0; nt < NT; ++nt, r += 16) {
          const int32_t last = wk.pos0 + r / p.group + 1;
          const int32_t lo = kv_low(last, p.window) - run, hi = ok && r < wk.count ? min(last, cap) - run : 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) s[nt][e >> 2][e & 3] = e >= lo && e < hi ? s[nt][e >> 2][e & 3] : -INFINITY;
        }
      }
      bf16x8 w[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = s[nt][0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[nt][e >> 2][e & 3]);
        top *= f;
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // sums are rescaled only when a maximum has grown by more than 2^8
        if (__ballot(top > m[nt] + 8.0f) != 0) {
          const float now = fmaxf(m[nt], top);
          const float x = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[nt] - now);
          m[nt] = now;
          l[nt] *= x;
#pragma unroll
          for (int i = 0; i < kDt; ++i) o[nt][i] *= x;
        }
        const float base = m[nt] == -INFINITY ? 0.0f : -m[nt];
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float pe = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][e >> 2][e & 3], f, base));
          sum += pe;
          w[nt][e >> 3][e & 7] = (__bf16)(pe * vw);
        }
        l[nt] += sum;
      }
      if (edge) {
        // What nobody sees counts as code 0, whatever is there.
        const u32x4 keep = kv_bytes(see.see_lo - run, ok ? see.see_hi - run : 0);
#pragma unroll
        for (int i = 0; i < kDt; ++i) xv[i] &= keep;
      }
#pragma unroll
      for (int i = 0; i < kDt; ++i) {
        const bf16x8 a = kv_widen(xv[i][0], xv[i][1]), b = kv_widen(xv[i][2], xv[i][3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w[nt][0], o[nt][i], 0, 0, 0);
          o[nt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, w[nt][1], o[nt][i], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (tile + 4 < see.tile1) load_k(tile + 4, pk_next, pv_next);
      pv = pv_next;
      pk_next = pk_after;
      pv_next = pv_after;
    }

    // Join the four waves: common maximum, then their sums one after another.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor(l[nt], 16);
      l[nt] += __shfl_xor(l[nt], 32);
      if (grp == 0) {
        lds_m[wave][nt * 16 + col] = m[nt];
        lds_l[wave][nt * 16 + col] = l[nt];
      }
    }
    __syncthreads();
    float f[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = -INFINITY;
      for (int w = 0; w < 4; ++w) top = fmaxf(top, lds_m[w][nt * 16 + col]);
      f[nt] = m[nt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[nt] - top);
    }
    // Of each thread: 8 channels of one row, in every part.
    const int32_t rr = tid / (kPart / 8), ch = (tid % (kPart / 8)) * 8, r = wk.first + rr;
    const bool mine = rr < R && r < wk.count;
    const int32_t tok = mine ? r / p.group : 0, g = mine ? r - tok * p.group : 0;
    const int64_t head = (int64_t)h * p.group + g, row = wk.row0 + tok, all = (int64_t)c.heads * p.group;
    const int64_t slot = (int64_t)h * p.slots + wk.slot;
    float top = -INFINITY, sum = 0.0f;
    if (mine) {
      for (int w = 0; w < 4; ++w) top = fmaxf(top, lds_m[w][rr]);
      // a wave without a maximum has a sum of zero, or NaN, which stays
      for (int w = 0; w < 4; ++w) {
        sum += lds_l[w][rr] * (lds_m[w][rr] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lds_m[w][rr] - top));
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int part = 0; part < D / kPart; ++part) {
      if (part > 0) __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < kPart / 16; ++i) {
          *(f32x4*)&lds[(wave * R + nt * 16 + col) * (kPart + 4) + i * 16 + 4 * grp] = o[nt][part * (kPart / 16) + i] * f[nt];
        }
      }
      __syncthreads();
      if (!mine) continue;
      f32x4 a = *(const f32x4*)&lds[rr * (kPart + 4) + ch], z = *(const f32x4*)&lds[rr * (kPart + 4) + ch + 4];
      for (int w = 1; w < 4; ++w) {
        a += *(const f32x4*)&lds[(w * R + rr) * (kPart + 4) + ch];
        z += *(const f32x4*)&lds[(w * R + rr) * (kPart + 4) + ch + 4];
      }
      const int32_t d = part * kPart + ch;
      if (wk.parts > 1) {
        f32x4* to = (f32x4*)(p.part + (slot * R + rr) * D + d);
        to[0] = a;
        to[1] = z;
      } else {
        bf16x8 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = (__bf16)(a[e] * inv);
          y[4 + e] = (__bf16)(z[e] * inv);
        }
        *(bf16x8*)(p.out + row * p.o_tok + head * p.o_head + d) = y;
      }
    }
    if (mine && ch == 0) {
      if (wk.parts > 1) {
        p.part_ml[slot * R + rr] = kv_part_ml(top, sum);
      } else if (p.lse) {
        p.lse[row * all + head] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
      }
      if (wk.begin && p.rows) p.rows[row * all + head] = int2{wk.slot * R + rr, wk.parts};
    }
    __syncthreads();   // LDS is free for the next row tile
  }
}

// The larger of a lane's value and that of its counterpart in the other half.
__device__ __forceinline__ float half_max(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}

// Many query rows: each of W waves holds 32 rows, and all of them share the
// key tiles, which the workgroup stages in LDS as codes, as they lie in the
// cache: staged as BF16 they would be widened once and not W times, but LDS's
// traffic doubles (prompts below 318 -> 332 us).  The loads of the next tile
// are under way in registers while the current one is computed.  Four waves
// have three buffers, so that one barrier a tile, between the two products,
// is enough; two waves have two, for the sake of four workgroups per CU
// (36 rows a sequence, 32 sequences of up to 8192: 52 us against 68).
//
// The products are the 32x32x16 ones, scores again transposed.  Key row m of a
// 32-key product is token 16 ((m / 4) % 2) + 4 (m / 8) + m % 4, which leaves
// lane half x with the 16 consecutive tokens 16 x .. 16 x + 15 of its query
// row, the order in which V^T P^T takes them.  16-byte LDS chunks are
// exchanged (XOR with the row) so that neighbouring lanes, which read rows at
// one column, fall on different banks: with row / 2 for rows of 128 bytes and
// row / 4 for rows of 64, conflicts went from 37% of LDS's cycles to none.
//
// Neither matrix units nor VALU are busy throughout: a wave's products, softmax
// and products follow one another, and overlap only with the other phases of
// the SIMD's other wave, as chance has it.  VALU work per score (the
// exponential at a quarter rate, and the widening of codes) is the smaller part
// of the distance to the matrix rate (below), but what can be is kept out of
// the inner loop: k's scale and the softmax scale are one factor per 16 tokens inside the
// fused multiply-add in front of the exponential; v's scale enters there too,
// as its logarithm; sums and maxima are only rescaled when a row's maximum
// has grown by more than 2^8; and a page that holds a whole tile (kOne) makes
// its addresses and scales uniform (307 -> 294 us).
//
// Two prompts of 4096, 32 heads over 8 of 128: 295 to 307 us on different
// cards, 895 to 934 TFLOP/s of the 1360 of a large matrix product (202 us);
// 500 tokens over 32768: 293 to 305 us with the join.
// Matrix units busy 40% of the cycles, VALU issue 64%, waits 21% of a wave's
// time; a copy without any exponential and widening took 285 us where this one
// took 311: 26 us of the 109 above the matrix rate.  64 rows a wave, to widen half as often, spills (586 us).
template <int D, int W, bool kOne>
__global__ __launch_bounds__(64 * W, D <= 128 ? 2 : 1) void kv_attend_tiles(KvCache c, KvBatch bt, KvQuery p) {
  constexpr int R = 32 * W, kN = 64 * W;
  constexpr int kC = D / 16;            // 16-byte chunks of a key row
  constexpr int kM = D / 32;            // 32-channel tiles of the output
  constexpr int kLoads = 4 * D / kN;    // chunks that a thread stages of k, and of v
  constexpr int kBuf = 128 * D;         // bytes of a staged tile: k, then v
  constexpr int kBufs = D <= 128 && W == 4 ? 3 : 2;
  __shared__ __align__(16) uint8_t lds[kBufs * kBuf];
  const int32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t col = lane & 31, half = lane >> 5;
  const int32_t w_item = blockIdx.x / c.heads, h = blockIdx.x - w_item * c.heads;
  const int32_t log_s = c.log_s, S = 1 << log_s, cap = kv_capacity(bt, log_s);
  KvWork wk;
  if (!kv_plan<R>(bt, p, cap, w_item, wk)) return;
  const KvSeen see = kv_seen<R>(wk, p, cap);

  const int32_t r_mine = wk.first + wave * 32 + col;
  const bool live = r_mine < wk.count;
  const int32_t tok_mine = live ? r_mine / p.group : 0;
  const int64_t head = (int64_t)h * p.group + (live ? r_mine - tok_mine * p.group : 0);
  const int64_t row = wk.row0 + tok_mine;
  const int32_t row_hi = live ? min(wk.pos0 + tok_mine + 1, cap) : 0;
  const int32_t row_lo = kv_low(wk.pos0 + tok_mine + 1, p.window);
  bf16x8 q[2 * kM];
  {
    const uint16_t* src = p.q + row * p.q_tok + head * p.q_head + 16 * half;
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the factor below is positive
    uint32_t most = 0;
#pragma unroll
    for (int s = 0; s < 2 * kM; ++s) {
      u32x4 x = *(const u32x4*)(src + 32 * (s >> 1) + 8 * (s & 1));
      x ^= u32x4{flip, flip, flip, flip};
      if (!live) x = u32x4{0, 0, 0, 0};
      most = pk_max_u16(most, fold_abs(x));
      q[s] = __builtin_bit_cast(bf16x8, x);
    }
    if (__ballot(halves_max(most) >= 0x7F80u) != 0) {
#pragma unroll
      for (int s = 0; s < 2 * kM; ++s) q[s] = __builtin_bit_cast(bf16x8, kv_no_infinity(__builtin_bit_cast(u32x4, q[s])));
    }
  }
  const float scale = fabsf(p.scale);
  f32x16 o[kM];
#pragma unroll
  for (int i = 0; i < kM; ++i) o[i] = f32x16{};
  float m = -INFINITY, l = 0.0f;

  // Pages of a tile's four runs of 16 tokens, the same in every lane; -1 where
  // the table's entry is no page or none of the tokens is seen.  A page of 64
  // tokens or more (kOne) holds the whole tile.
  const FP8BQ_CONSTANT int32_t* table =
      (const FP8BQ_CONSTANT int32_t*)(uintptr_t)(bt.table + (int64_t)wk.b * bt.stride);
  constexpr int kRuns = kOne ? 1 : 4;
  struct Pages {
    int32_t of[kRuns];
  };
  auto pages = [&](int32_t tile) {
    Pages x;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int32_t t0 = tile * kKeyTile + 16 * r;
      int32_t pg = -1;
      if (kOne || (t0 < see.see_hi && t0 + 16 > see.see_lo)) pg = table[t0 >> log_s];
      pg = __builtin_amdgcn_readfirstlane(pg);
      x.of[r] = pg >= 0 && pg < c.pages ? pg : -1;
    }
    return x;
  };
  auto pick = [](const Pages& x, int32_t r) {
    if constexpr (kOne) return x.of[0];
    const int32_t a = r & 1 ? x.of[1 % kRuns] : x.of[0], b = r & 1 ? x.of[3 % kRuns] : x.of[2 % kRuns];
    return r & 2 ? b : a;
  };

  // Where a thread stages its chunks, and reads its operands: byte `at` of row
  // `row`, whose 16-byte chunks are exchanged with the row.  What a constant
  // adds to (32 rows, 8 or 4 chunks) leaves the exchange as it is.
  auto swizzle = [](int32_t row, int32_t ch, int32_t chunks) {
    return (row * chunks + (ch ^ (chunks % 8 == 0 ? (row >> 1) & 7 : (row >> 2) & 3))) * 16;
  };
  constexpr int kAts = kC % 8 == 0 ? 4 : 2;
  int32_t k_at[kAts], v_at[2];
#pragma unroll
  for (int i = 0; i < kAts; ++i) k_at[i] = swizzle(col, 2 * i + half, kC);
#pragma unroll
  for (int u = 0; u < 2; ++u) v_at[u] = 64 * D + swizzle(col, 2 * u + half, 4);
  const int32_t v_off = ((tid >> 2) << log_s) + 16 * (tid & 3);

  u32x4 kr[kLoads], vr[kLoads];
  struct Scales {
    float k[2], v[2];   // of the lane's two runs (kOne: the same for all)
  };
  auto fetch = [&](int32_t tile, const Pages& x, Scales& sc) {
    if constexpr (kOne) {
      const int32_t in_page = (tile * kKeyTile) & (S - 1);   // 0 unless a page is longer than a tile
      const int64_t block = (int64_t)max(x.of[0], 0) * c.heads + h, at = block * (D << log_s);
      const uint8_t* kp = c.k + (at + in_page * D);
      const uint8_t* vp = c.v + (at + in_page);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        kr[i] = *(const u32x4*)(kp + (uint32_t)(16 * tid + 16 * i * kN));
        vr[i] = *(const u32x4*)(vp + (uint32_t)(v_off + ((i * kN / 4) << log_s)));
      }
      sc.k[0] = sc.k[1] = ((const FP8BQ_CONSTANT float*)(uintptr_t)c.ks)[block];
      sc.v[0] = sc.v[1] = ((const FP8BQ_CONSTANT float*)(uintptr_t)c.vs)[block];
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int32_t at = tid + i * kN, tok = at / kC, ch = at - tok * kC;
        const int64_t kb = ((int64_t)max(pick(x, tok >> 4), 0) * c.heads + h) << log_s;
        kr[i] = *(const u32x4*)(c.k + (kb + (tok & (S - 1))) * D + 16 * ch);
        const int32_t dim = at >> 2, run = at & 3;
        const int64_t vb = ((int64_t)max(pick(x, run), 0) * c.heads + h) * D + dim;
        vr[i] = *(const u32x4*)(c.v + (vb << log_s) + ((16 * run) & (S - 1)));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t at = (int64_t)max(pick(x, 2 * u + half), 0) * c.heads + h;
        sc.k[u] = c.ks[at];
        sc.v[u] = c.vs[at];
      }
    }
  };
  auto bad = [](const Pages& x) {
    int32_t any = x.of[0];
#pragma unroll
    for (int r = 1; r < kRuns; ++r) any |= x.of[r];
    return any < 0;
  };
  auto is_edge = [&](int32_t tile, const Pages& x) {
    const int32_t t0 = tile * kKeyTile;
    return bad(x) || t0 < see.all_lo || t0 + kKeyTile > see.all_hi;
  };
  auto put = [&](uint8_t* to, int32_t tile, const Pages& x) {
    if (is_edge(tile, x)) {
      // what nobody sees counts as code 0, whatever is there
      asm volatile("");   // a branch: not computed for the other tiles
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int32_t run = (tid + i * kN) & 3, t0 = tile * kKeyTile + 16 * run;
        vr[i] &= kv_bytes(see.see_lo - t0, pick(x, run) >= 0 ? see.see_hi - t0 : 0);
      }
    }
    int32_t first = tid;
    if constexpr (kLoads > 2) asm volatile("" : "+v"(first));   // computed here, not kept in registers
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int32_t at = first + i * kN, tok = at / kC;
      const int32_t lrow = (tok & 32) + 8 * ((tok >> 2) & 3) + 4 * ((tok >> 4) & 1) + (tok & 3);
      *(u32x4*)(to + swizzle(lrow, at - tok * kC, kC)) = kr[i];
      *(u32x4*)(to + 64 * D + swizzle(at >> 2, at & 3, 4)) = vr[i];
    }
  };

  auto compute = [&](const uint8_t* from, int32_t tile, const Pages& x, const Scales& sc, auto&& between) {
    f32x16 s[2];
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x16{};
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const u32x4 a = *(const u32x4*)(from + k_at[i % kAts] + 32 * u * D + i / kAts * 32 * kAts);
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kv_widen(a[0], a[1]), q[2 * i], s[u], 0, 0, 0);
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kv_widen(a[2], a[3]), q[2 * i + 1], s[u], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    between();
    float f[2], lv[2], back[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool ok = pick(x, 2 * u + half) >= 0;
      const float v = ok ? fmaxf(sc.v[u], kLeastVScale) : 1.0f;
      f[u] = ok ? fmaxf(sc.k[u] * scale, kTiny) : 1.0f;
      lv[u] = __builtin_amdgcn_logf(v);
      back[u] = __builtin_amdgcn_rcpf(v);
    }
    if (is_edge(tile, x)) {
      asm volatile("");
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int32_t t0 = tile * kKeyTile + 32 * u + 16 * half;
        const bool ok = pick(x, 2 * u + half) >= 0;
        const int32_t lo = row_lo - t0, hi = ok ? row_hi - t0 : 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[u][e] = e >= lo && e < hi ? s[u][e] : -INFINITY;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float t = s[u][0];
#pragma unroll
      for (int e = 1; e < 16; ++e) t = fmaxf(t, s[u][e]);
      top = fmaxf(top, t * f[u]);
    }
    top = half_max(top);
    if (__ballot(top > m + 8.0f) != 0) {
      const float now = fmaxf(m, top);
      const float g = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= g;
#pragma unroll
      for (int i = 0; i < kM; ++i) o[i] *= g;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    bf16x8 w[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float off = lv[u] - base;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float pe = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], f[u], off));
        sum += pe;
        w[u][e >> 3][e & 7] = (__bf16)pe;
      }
      l = __builtin_fmaf(sum, back[u], l);
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < kM; ++i) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const u32x4 a = *(const u32x4*)(from + v_at[u] + 32 * i * 64);
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kv_widen(a[0], a[1]), w[u][0], o[i], 0, 0, 0);
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kv_widen(a[2], a[3]), w[u][1], o[i], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
  };

  if (see.tile0 < see.tile1) {
    // Tiles go round through the buffers; all but one of those hold tiles that
    // are staged or computed, the last is being filled.
    constexpr int kAhead = kBufs - 1;
    const int32_t last = see.tile1 - 1;
    int32_t tile = see.tile0;
    Pages pg[kBufs];
    Scales sc[kBufs];
#pragma unroll
    for (int i = 0; i < kBufs; ++i) pg[i] = pages(min(tile + i, last));
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (tile + i <= last) {
        fetch(tile + i, pg[i], sc[i]);
        put(lds + i * kBuf, tile + i, pg[i]);
      }
    }
    if constexpr (kBufs == 3) __syncthreads();
    auto step = [&](auto which) {
      constexpr int kNow = decltype(which)::value, kNext = (kNow + kAhead) % kBufs;
      const bool more = tile + kAhead <= last;
      if (more) fetch(tile + kAhead, pg[kNext], sc[kNext]);
      // Whoever passes a tile's barrier has done with the buffer that is
      // filled next.  With three buffers what is read was written before the
      // barrier of a tile ago, and the barrier can stand between the products,
      // where nobody waits for it long (prompts, when it was put there: 317 -> 310 us).
      if constexpr (kBufs == 2) __syncthreads();
      compute(lds + kNow * kBuf, tile, pg[kNow], sc[kNow], [&] {
        if constexpr (kBufs == 3) __syncthreads();
      });
      if (more) put(lds + kNext * kBuf, tile + kAhead, pg[kNext]);
      pg[kNow] = pages(min(tile + kBufs, last));
      return ++tile <= last;
    };
    using std::integral_constant;
    if constexpr (kBufs == 3) {
      while (step(integral_constant<int, 0>{}) && step(integral_constant<int, 1>{}) && step(integral_constant<int, 2>{})) {
      }
    } else {
      while (step(integral_constant<int, 0>{}) && step(integral_constant<int, 1>{})) {
      }
    }
  }

  l += __shfl_xor(l, 32);
  const int64_t slot = (int64_t)h * p.slots + wk.slot;
  const int32_t rr = wave * 32 + col;
  const int64_t all = (int64_t)c.heads * p.group;
  if (wk.parts > 1) {
    if (live) {
      float* to = p.part + (slot * R + rr) * D + 4 * half;
#pragma unroll
      for (int i = 0; i < kM; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          *(f32x4*)(to + 32 * i + 8 * e) = f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
        }
      }
      if (half == 0) p.part_ml[slot * R + rr] = kv_part_ml(m, l);
    }
  } else {
    // Through LDS, so that a wave writes whole rows.
    constexpr int kRow = 2 * D + 16;   // bytes, a chunk of padding
    static_assert(8 * kRow * W <= 2 * kBuf, "a quarter of the wave's rows at a time");
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __syncthreads();
    uint8_t* mine = lds + wave * 8 * kRow;
#pragma unroll
    for (int part = 0; part < 4; ++part) {
      if ((col >> 3) == part) {
#pragma unroll
        for (int i = 0; i < kM; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bf16x4 y = {(__bf16)(o[i][4 * e] * inv), (__bf16)(o[i][4 * e + 1] * inv),
                              (__bf16)(o[i][4 * e + 2] * inv), (__bf16)(o[i][4 * e + 3] * inv)};
            *(bf16x4*)(mine + (col & 7) * kRow + 2 * (32 * i + 8 * e + 4 * half)) = y;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8 * (D / 8) / 64; ++i) {
        const int32_t at = lane + 64 * i, lr = at / (D / 8), ch = at - lr * (D / 8);
        const int32_t r = wk.first + wave * 32 + part * 8 + lr;
        if (r < wk.count) {
          const int32_t tok = r / p.group;
          const int64_t hd = (int64_t)h * p.group + (r - tok * p.group);
          *(u32x4*)(p.out + (wk.row0 + tok) * p.o_tok + hd * p.o_head + 8 * ch) =
              *(const u32x4*)(mine + lr * kRow + 16 * ch);
        }
      }
      __syncthreads();
    }
    if (live && half == 0 && p.lse) {
      p.lse[row * all + head] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
  }
  if (live && half == 0 && p.rows && wk.begin) p.rows[row * all + head] = int2{wk.slot * R + rr, wk.parts};
}

// Joins the partial sums of each query row whose keys were split, found
// through `rows` (first slot times R plus row in tile, and how many slots; the
// second is `jump` + 1 behind the first, the others follow it).  N waves share a row, each taking every Nth partial, all in
// flight at once: with few rows of many splits, as one long sequence has, one
// wave per row would add up its partials one round trip after another.
// Latency alone: 5 us for 32 rows of some 60 partials, 8 for 4608 rows, 12 for
// 16000.
template <int D, int N>
__global__ __launch_bounds__(N == 1 ? 256 : 64 * N) void kv_attend_join(KvBatch bt, KvQuery p, int32_t heads,
                                                                        int32_t R) {
  constexpr int kV = D / 64;
  __shared__ float acc_of[N][D], sum_of[N], top_of[N];
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t item = N == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int32_t part = N == 1 ? 0 : wave;
  const int32_t all = heads * p.group;
  if (item >= (int64_t)p.tokens * all) return;
  const int64_t row = item / all;
  const int32_t head = (int32_t)(item - row * all);
  // rows that belong to no sequence stay as they are
  if (bt.starts && (row < kv_clamp(bt.starts[0], p.tokens) || row >= kv_clamp(bt.starts[bt.count], p.tokens))) return;
  const int2 at = p.rows[item];
  const int32_t slot0 = at.x / R, rr = at.x - slot0 * R;
  if (at.y <= 1 || at.x < 0 || slot0 >= p.slots) return;
  const int32_t n = min(at.y, max(p.slots - slot0 - p.jump, 1));
  const int64_t base = ((int64_t)(head / p.group) * p.slots + slot0) * R + rr;
  float top = -INFINITY, sum = 0.0f, acc[kV] = {};
  for (int32_t i0 = part; i0 < n; i0 += 8 * N) {
    float2 ml[8];
    float x[8][kV];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int32_t i = min(i0 + j * N, n - 1);
      const int64_t e = base + (int64_t)(i + (i > 0 ? p.jump : 0)) * R;
      ml[j] = p.part_ml[e];
      const float* src = p.part + e * D + lane * kV;
#pragma unroll
      for (int y = 0; y < kV; ++y) x[j][y] = src[y];
    }
    float now = top;
#pragma unroll
    for (int j = 0; j < 8; ++j) now = fmaxf(now, ml[j].x);
    if (now == -INFINITY) continue;
    const float keep = __builtin_amdgcn_exp2f(top - now);
    top = now;
    sum *= keep;
#pragma unroll
    for (int y = 0; y < kV; ++y) acc[y] *= keep;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = i0 + j * N < n ? __builtin_amdgcn_exp2f(ml[j].x - now) : 0.0f;
      sum += ml[j].y * f;
#pragma unroll
      for (int y = 0; y < kV; ++y) acc[y] += x[j][y] * f;
    }
  }
  if constexpr (N > 1) {
    if (lane == 0) {
      top_of[wave] = top;
      sum_of[wave] = sum;
    }
#pragma unroll
    for (int y = 0; y < kV; ++y) acc_of[wave][lane * kV + y] = acc[y];
    __syncthreads();
    if (wave != 0) return;
    for (int w = 0; w < N; ++w) top = fmaxf(top, top_of[w]);
    sum = 0.0f;
#pragma unroll
    for (int y = 0; y < kV; ++y) acc[y] = 0.0f;
    for (int w = 0; w < N; ++w) {
      const float f = top_of[w] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top_of[w] - top);
      sum += sum_of[w] * f;
#pragma unroll
      for (int y = 0; y < kV; ++y) acc[y] += acc_of[w][lane * kV + y] * f;
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* to = p.out + row * p.o_tok + head * p.o_head + lane * kV;
#pragma unroll
  for (int x = 0; x < kV; ++x) to[x] = bf16_down(acc[x] * inv);
  if (lane == 0 && p.lse) {
    p.lse[item] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
  }
}

}  // namespace fp8bq
