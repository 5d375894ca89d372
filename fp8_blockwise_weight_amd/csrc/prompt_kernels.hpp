// Device code of attention in the expanded form (gfx950): every head has keys
// and values of its own, and one rotated key, which the heads share.
#pragma once

#include "latent_kernels.hpp"

namespace fp8bq {

typedef __attribute__((ext_vector_type(4))) short s16x4;

struct PromptQuery {
  const uint16_t* q;       // BF16 [tokens, heads, D + 64]
  const uint16_t* k;       // BF16 [keys, heads, D]
  const uint16_t* r;       // BF16 [keys, 64]
  const uint16_t* v;       // BF16 [keys, heads, D]
  uint16_t* out;           // BF16 [tokens, heads, D]
  float* lse;              // fp32 [tokens, heads], or null
  const int32_t* q_at;     // [count + 1]
  const int32_t* k_at;     // [count + 1]
  int64_t q_tok, q_head, k_tok, k_head, r_tok, v_tok, v_head, o_tok, o_head;
  int32_t tokens, keys, heads, count;
  float scale;             // of the scores, times log2(e)
};

// The scores of 64 keys, their softmax with a running maximum, the weighted sum
// of the values: both products on the matrix units, K Q and V W, so that a lane
// holds one query's scores and its weights are operands where they lie.  A wave
// holds 32 queries; four of them share the tiles in LDS, which loads put there
// past the registers while the tile before is worked on, and two such workgroups
// share a CU: one's products run while the other takes exponentials, and the
// priority that a wave has within its products keeps them taking turns.  What
// bounds it: a wave reads the whole tile, 40 KB, for 32 rows, which keeps LDS
// busy for as long as the products take.
//
// Two prompts of 4096 tokens, 32 heads of 128 channels, 344 GFLOP: 322 us, 1070
// TFLOP/s (335 to 350 on other cards; a large BF16 matrix product reaches 1330);
// beside it operands read when they were wanted 335, without the priorities 333,
// a lane's place in a tile worked out for every load 349.  Waves of 64 queries,
// one to a SIMD, with the weights of 32 keys between the products of the next,
// halve LDS's traffic and take 520: a wave alone does not keep both units busy.
//
// A workgroup takes R = 128 query tokens of one head.  Slot w of the grid
// belongs to the sequence with floor(q_at[b] / R) + b <= w, which leaves every
// sequence as many slots as it has row tiles, whatever the offsets are.
//
// With K = 2 a workgroup has as many waves again, which take every other tile, out
// of an LDS of their own, and whose sums are joined at the end: half the tiles in
// a row, on the whole of a CU.
template <int D, int K>
__global__ __launch_bounds__(256 * K, 2) void latent_prompt(PromptQuery p) {
  constexpr int W = 4, R = 32 * W;
  constexpr int kJ = D / 16, kO = D / 32;
  constexpr int kC = D / 8;                       // 16-byte chunks of a row
  constexpr int kK = 64 * 2 * D, kR = 64 * 2 * kRope;
  constexpr int kBytes = 2 * kK + kR;             // keys, rotated keys, values
  __shared__ __align__(1024) uint8_t all_lds[K * 2 * kBytes];
  const int32_t tid = threadIdx.x & (64 * W - 1), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t turn = K == 1 ? 0 : __builtin_amdgcn_readfirstlane((int32_t)threadIdx.x / (64 * W));
  uint8_t* lds = all_lds + turn * 2 * kBytes;
  const int32_t col = lane & 31, half = lane >> 5;
  const int32_t w_item = blockIdx.x / p.heads, h = blockIdx.x - w_item * p.heads;
  const auto q_row = [&](int32_t i) { return kv_clamp(p.q_at[i], p.tokens); };
  const auto k_row = [&](int32_t i) { return kv_clamp(p.k_at[i], p.keys); };
  const auto first_slot = [&](int32_t i) { return (int64_t)(q_row(i) / R) + i; };
  const int32_t b = kv_find(p.count, w_item, first_slot);
  const int32_t row0 = __builtin_amdgcn_readfirstlane(q_row(b));
  const int32_t n = __builtin_amdgcn_readfirstlane(q_row(b + 1)) - row0;
  const int32_t key0 = __builtin_amdgcn_readfirstlane(k_row(b));
  const int32_t keys = max(__builtin_amdgcn_readfirstlane(k_row(b + 1)) - key0, 0);
  const int32_t tiles = (max(n, 0) + R - 1) / R;
  const int64_t local = w_item - (__builtin_amdgcn_readfirstlane((int32_t)(row0 / R)) + (int64_t)b);
  if (local < 0 || local >= tiles) return;
  const int32_t first = (tiles - 1 - (int32_t)local) * R;   // the last rows see the most keys: they go first
  const int32_t r_mine = first + wave * 32 + col;
  const bool live = r_mine < n;
  const int64_t row = row0 + min(r_mine, n - 1);
  const int64_t before = (int64_t)keys - n;                 // keys in front of the first query's own
  const int32_t row_hi = live ? (int32_t)max(before + r_mine + 1, (int64_t)0) : 0;
  const int32_t see_hi = (int32_t)max(before + min(first + R, n), (int64_t)0);
  const int32_t all_hi = (int32_t)max(before + first + 1, (int64_t)0);
  const int32_t last = (see_hi + kKeyTile - 1) / kKeyTile - 1;

  const uint32_t lds0 = lds_address(lds);
  const uint8_t* kp = (const uint8_t*)(p.k + key0 * p.k_tok + h * p.k_head);
  const uint8_t* rp = (const uint8_t*)(p.r + key0 * p.r_tok);
  const uint8_t* vp = (const uint8_t*)(p.v + key0 * p.v_tok + h * p.v_head);
  // 16-byte chunks are exchanged within a row so that what is read at a time,
  // one chunk of 16 keys or four chunks of four, falls on different banks.
  const auto turn_k = [](int32_t key) { return kC == 16 ? key & 15 : (key >> 1) & 7; };
  const auto turn_r = [](int32_t key) { return (key >> 1) & 7; };
  const auto turn_v = [](int32_t key) { return kC == 16 ? (key & 3) << 2 : ((key >> 1) & 1) << 2; };
  // A row's place in a tile goes with the lane, for every instruction of a wave
  // the same (16 or 32 rows on, the exchange is): what advances is the base, in
  // scalar registers.  Of the last tile, keys behind the last one that is seen
  // count as that one.
  constexpr int kKeys = 64 / kC;                  // of an instruction
  const int32_t key_in = wave * kKeys + lane / kC, r_in8 = wave * 8 + (lane >> 3);
  const int32_t k_pitch = (int32_t)p.k_tok * 2, v_pitch = (int32_t)p.v_tok * 2, r_pitch = (int32_t)p.r_tok * 2;
  const int32_t k_off = ((lane % kC) ^ turn_k(key_in)) * 16, v_off = ((lane % kC) ^ turn_v(key_in)) * 16;
  const int32_t r_off = ((lane & 7) ^ turn_r(r_in8)) * 16;
  const uint32_t k_in = key_in * k_pitch + k_off, v_in = key_in * v_pitch + v_off, r_in = r_in8 * r_pitch + r_off;
  const auto stage = [&](int32_t tile, int32_t slot) {
    const uint32_t to = lds0 + slot * kBytes;
    const int32_t t0 = tile * kKeyTile, end = see_hi - 1 - t0;
    const uint8_t* kb = kp + t0 * (p.k_tok * 2);
    const uint8_t* vb = vp + t0 * (p.v_tok * 2);
    const uint8_t* rb = rp + t0 * (p.r_tok * 2);
    const bool whole = end >= kKeyTile - 1;
#pragma unroll
    for (int i = 0; i < 64 / kKeys / W; ++i) {
      const int32_t k0 = i * W * kKeys, at = to + (k0 + wave * kKeys) * 2 * D;
      if (whole) {
        lds_load16(kb + k0 * (int64_t)k_pitch, k_in, at);
        lds_load16(vb + k0 * (int64_t)v_pitch, v_in, at + kK + kR);
      } else {
        const int32_t key = min(k0 + key_in, end);
        lds_load16(kb, key * k_pitch + k_off, at);
        lds_load16(vb, key * v_pitch + v_off, at + kK + kR);
      }
    }
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      const int32_t k0 = i * W * 8, at = to + kK + (k0 + wave * 8) * 128;
      if (whole) {
        lds_load16(rb + k0 * (int64_t)r_pitch, r_in, at);
      } else {
        lds_load16(rb, min(k0 + r_in8, end) * r_pitch + r_off, at);
      }
    }
  };
  if (turn <= last) stage(turn, 0);

  bf16x8 q[kJ + 4];
  {
    const uint16_t* src = p.q + row * p.q_tok + h * p.q_head + 8 * half;
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the factor below is positive
#pragma unroll
    for (int j = 0; j < kJ + 4; ++j) {
      u32x4 x = *(const u32x4*)(src + 16 * j) ^ u32x4{flip, flip, flip, flip};
      q[j] = __builtin_bit_cast(bf16x8, kv_no_infinity(x));
    }
  }
  const float factor = fmaxf(fabsf(p.scale), kTiny);
  f32x16 o[kO];
#pragma unroll
  for (int i = 0; i < kO; ++i) o[i] = f32x16{};
  float m = -INFINITY, l = 0.0f;

  const int32_t rounds = (last + K) / K;   // the same for all waves, as they wait for each other
  for (int32_t round = 0; round < rounds; ++round) {
    const int32_t tile = round * K + turn, slot = round & 1, t0 = tile * kKeyTile;
    uint8_t* from = lds + slot * kBytes;
    lds_arrived();
    if ((round + 1) * K * kKeyTile > see_hi) {
      // values that nobody sees count as zeros, whatever is there
      for (int32_t i = tid; i < 64 * kC; i += 64 * W) {
        if (t0 + i / kC >= see_hi) *(u32x4*)(from + kK + kR + 16 * i) = u32x4{0, 0, 0, 0};
      }
      lds_written();
    }
    if (tile + K <= last) stage(tile + K, slot ^ 1);
    if (K > 1 && tile > last) break;             // only in the last round
    __builtin_amdgcn_s_setprio(1);
    f32x16 s[2];
    s[0] = f32x16{};
    s[1] = f32x16{};
    {
      // operands of 16 channels, two steps ahead
      bf16x8 ring[4][2];
      const auto get = [&](int j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int32_t key = 32 * u + col;
          ring[j & 3][u] = j < kJ ? *(const bf16x8*)(from + key * 2 * D + ((2 * j + half) ^ turn_k(key)) * 16)
                                  : *(const bf16x8*)(from + kK + key * 128 + ((2 * (j - kJ) + half) ^ turn_r(key)) * 16);
        }
      };
      get(0);
      get(1);
      __builtin_amdgcn_sched_barrier(0);
      unrolled<kJ + 4>([&](auto step) {
        constexpr int j = decltype(step)::value;
        if constexpr (j + 2 < kJ + 4) get(j + 2);
        s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j & 3][0], q[j], s[0], 0, 0, 0);
        s[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j & 3][1], q[j], s[1], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    __builtin_amdgcn_s_setprio(0);
    if (t0 + kKeyTile > all_hi) {
      asm volatile("");   // a branch
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int32_t hi = row_hi - t0 - 32 * u - 4 * half;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[u][e] = 8 * (e >> 2) + (e & 3) < hi ? s[u][e] : -INFINITY;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[u][e]);
    }
    top = half_max(top) * factor;
    if (__ballot(top > m + 8.0f) != 0) {
      const float to = fmaxf(m, top);
      const float g = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= g;
#pragma unroll
      for (int i = 0; i < kO; ++i) o[i] *= g;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    bf16x8 w[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], factor, -base));
        l += x;
        w[2 * u + (e >> 3)][e & 7] = (__bf16)x;
      }
    }
    __builtin_amdgcn_s_setprio(1);
    // Lane half x holds, of each 16 keys, 4 x .. 4 x + 3 and 8 + 4 x .. 8 + 4 x + 3.
    {
      bf16x8 ring[4];   // three steps ahead
      const auto get = [&](int n) {
        s16x4 x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int32_t key = 16 * (n / kO) + 8 * y + 4 * half + ((lane & 15) >> 2);
          const int32_t chunk = 4 * (n % kO) + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
          x[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
              from + kK + kR + key * 2 * D + (chunk ^ turn_v(key)) * 16 + 8 * (lane & 1)));
        }
        const auto both = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
        ring[n & 3] = __builtin_bit_cast(bf16x8, both);
      };
      get(0);
      get(1);
      get(2);
      unrolled<4 * kO>([&](auto step) {
        constexpr int n = decltype(step)::value;
        if constexpr (n + 3 < 4 * kO) get(n + 3);
        o[n % kO] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[n & 3], w[n / kO], o[n % kO], 0, 0, 0);
        // (the first of them among the weights' instructions, as they come)
        if constexpr (n >= kO) __builtin_amdgcn_sched_barrier(0);
      });
    }
    __builtin_amdgcn_s_setprio(0);
  }
  if constexpr (K == 2) {
    constexpr int kSums = 16 * kO;
    static_assert(W * (kSums + 2) * 64 * 4 <= (int)sizeof(all_lds), "sums on their way");
    float* pass = (float*)all_lds + wave * (kSums + 2) * 64 + lane;
    lds_written();   // nobody reads tiles any more
    if (turn == 1) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) pass[i * 64] = o[i >> 4][i & 15];
      pass[kSums * 64] = m;
      pass[(kSums + 1) * 64] = l;
    }
    lds_written();
    if (turn == 1) return;
    const float m1 = pass[kSums * 64], to = fmaxf(m, m1);
    // sums without a maximum are zeros, or no numbers
    const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
    const float f1 = m1 == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m1 - to);
#pragma unroll
    for (int i = 0; i < kSums; ++i) o[i >> 4][i & 15] = o[i >> 4][i & 15] * f + pass[i * 64] * f1;
    l = l * f + pass[(kSums + 1) * 64] * f1;
    m = to;
  }
  l += __shfl_xor(l, 32);
  if (!live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* to = p.out + row * p.o_tok + h * p.o_head + 4 * half;
#pragma unroll
  for (int i = 0; i < kO; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *(bf16x4*)(to + 32 * i + 8 * e) =
          bf16x4{(__bf16)(o[i][4 * e] * inv), (__bf16)(o[i][4 * e + 1] * inv), (__bf16)(o[i][4 * e + 2] * inv),
                 (__bf16)(o[i][4 * e + 3] * inv)};
    }
  }
  if (half == 0 && p.lse) {
    p.lse[row * p.heads + h] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
  }
}

}  // namespace fp8bq
