// Host side of the latent cache: the fp8bq_latent_* calls of include/fp8bq.h.
// Every argument check runs before the first HIP call; the calls enqueue on
// the caller's stream and neither allocate nor wait.

#include <algorithm>

#include "latent_kernels.hpp"
#include "prompt_kernels.hpp"

namespace {

constexpr int32_t kLatentMaxHeads = 1024;
constexpr int64_t kPromptMaxStride = int64_t{1} << 23;   // of keys and values, elements
// What a row tile of the absorbed form costs beyond its key tiles, in key tiles
// (queries split, sums written): shares of 96 sequences x 16 heads, 60 x 128 and
// 64 x 40 heads with drafts come out at 126, 139 and 59 us without it, 120, 133
// and 51 with 3, 119, 127 and 52 with 5.
constexpr int32_t kLatentExtra = 4;

// The buffers of a cache.
struct LatentBuffers {
  const void* at[3];
  uint64_t bytes[3];
};

LatentBuffers latent_buffers(const fp8bq_latent_cache& c) {
  const uint64_t places = static_cast<uint64_t>(c.num_pages) * static_cast<uint64_t>(c.page_size);
  return LatentBuffers{{c.c, c.r, c.scale},
                       {places * static_cast<uint64_t>(c.latent_dim), places * 2 * fp8bq::kRope, places * 4}};
}

bool latent_cache_ok(const fp8bq_latent_cache* c) {
  if (c == nullptr || kv_log2_page(c->page_size) < 0 || (c->latent_dim != 256 && c->latent_dim != 512)) return false;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || !c->c || !c->r || !c->scale) return false;
  if (!kv_aligned(c->c, 16) || !kv_aligned(c->r, 16) || !kv_aligned(c->scale, 4)) return false;
  const LatentBuffers b = latent_buffers(*c);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j) {
      if (overlap(b.at[i], b.bytes[i], b.at[j], b.bytes[j])) return false;
    }
  }
  return true;
}

bool latent_apart(const fp8bq_latent_cache& c, const void* p, uint64_t bytes) {
  const LatentBuffers b = latent_buffers(c);
  for (int i = 0; i < 3; ++i) {
    if (bytes > 0 && overlap(p, bytes, b.at[i], b.bytes[i])) return false;
  }
  return true;
}

bool latent_heads_ok(int32_t heads, int64_t tokens) {
  return heads >= 1 && heads <= kLatentMaxHeads && tokens <= kKvMaxRows / heads;
}

// Rows that a call reads or writes, `dim` values each.
struct LatentRows {
  KvRows rows;
  int32_t dim;
  uint64_t extent(int64_t tokens) const { return kv_extent(tokens, rows.tok, rows.heads, rows.head, dim); }
  bool ok() const { return kv_rows_ok(rows.p, rows.tok, rows.head); }
  bool distinct(int64_t tokens) const { return kv_distinct(tokens, rows.tok, rows.heads, rows.head, dim); }
};

// Whether written rows share no element with others: by their extents, or as
// slices of one tensor, token by token or head by head.
bool latent_rows_apart(const LatentRows& a, const LatentRows& b, int64_t tokens) {
  if (!overlap(a.rows.p, a.extent(tokens), b.rows.p, b.extent(tokens))) return true;
  const int64_t off = (static_cast<int64_t>(reinterpret_cast<intptr_t>(b.rows.p)) -
                       static_cast<int64_t>(reinterpret_cast<intptr_t>(a.rows.p))) / 2;
  auto beside = [&](int64_t out, int64_t in_a, int64_t in_b) {
    if (out <= 0) return false;
    const int64_t d = (off % out + out) % out;
    return d >= in_a && d + in_b <= out;
  };
  const int64_t a_in = (a.rows.heads - 1) * a.rows.head + a.dim, b_in = (b.rows.heads - 1) * b.rows.head + b.dim;
  if (a.rows.tok == b.rows.tok && beside(a.rows.tok, a_in, b_in)) return true;
  return a.rows.head == b.rows.head && a.rows.heads > 1 && b.rows.heads > 1 &&
         beside(a.rows.head, (tokens - 1) * a.rows.tok + a.dim, (tokens - 1) * b.rows.tok + b.dim);
}

bool latent_same(const LatentRows& a, const LatentRows& b, int64_t tokens) {
  return a.rows.p == b.rows.p && (tokens == 1 || a.rows.tok == b.rows.tok) &&
         (a.rows.heads == 1 || a.rows.head == b.rows.head);
}

fp8bq::LatentCache latent_device(const fp8bq_latent_cache& c) {
  return fp8bq::LatentCache{static_cast<uint8_t*>(c.c), static_cast<uint16_t*>(c.r), c.scale,
                            static_cast<int32_t>(c.num_pages), kv_log2_page(c.page_size)};
}

// How an absorbed call is cut up, from the shapes alone.
struct LatentShape {
  int32_t rows;        // query rows of a workgroup
  int32_t subs;        // workgroups that take the same keys for rows side by side
  int32_t grid;
  int32_t target;      // shares that the key tiles are cut into; 0: one for each row tile
  int32_t slots;
  size_t rows_at, ml_at, bytes;   // workspace: partial sums at 0, then these
};

// Figures below: us of a step over L = 512, 8000 tokens a sequence where not said.
LatentShape latent_shape(const fp8bq_latent_cache& c, const fp8bq_kv_batch& b, int32_t heads, int64_t tokens) {
  LatentShape s;
  // One pair of waves, two workgroups to a CU, as long as a sequence's rows fit in
  // it, else two pairs that share the keys: 96 sequences of 16 rows 116 and 139, of
  // 32 rows 125 and 131; 60 of 40 rows 106 and 91, of 64 rows 113 and 99.
  // Where rows need more workgroups than one, these take the same keys side by
  // side on one XCD, whose cache serves all but the first: 60 sequences of 128
  // rows 155 -> 151, 30 of 256 rows 144 -> 140.  All of this goes by the mean, so
  // that one long chunk among single tokens leaves most of the workgroups beside
  // them idle: 31 sequences with a token each and one with 512 take 242 at 16 heads
  // (calls of their own: 47 and 163), 1087 at 128 (91 and 942).
  const int64_t per_seq = ceil_div(tokens * heads, b.count);
  s.rows = per_seq <= 32 ? 32 : 64;
  s.subs = per_seq <= 64 ? 1 : (per_seq <= 128 ? 2 : 4);
  const int64_t row_tiles = tokens * heads / (s.rows * s.subs) + b.count;
  const int64_t key_tiles = ceil_div(static_cast<int64_t>(b.max_pages) * c.page_size, 64);
  // One round of workgroups, but no more (in eights, one for each XCD) than there
  // can be key tiles to share: one sequence of 777 tokens takes 3 MB of workspace
  // instead of 64, and is cut up as before, a tile to a share.
  const int64_t units = row_tiles * (key_tiles + kLatentExtra);
  s.target = static_cast<int32_t>(std::min<int64_t>((s.rows == 32 ? 512 : 256) / s.subs, ceil_div(units, 8) * 8));
  // Short tables leave nothing to cut up: without shares, their partial sums and
  // the join, steps at 200 tokens (4 tiles) of 96 sequences take 18 instead of 24
  // at 16 heads and 24 instead of 53 at 128, one sequence 17.1 instead of 16.5; at
  // 500 tokens (8 tiles) 96 sequences 26 either way, one 24 instead of 17.
  if (key_tiles <= 4) s.target = 0;
  s.grid = static_cast<int32_t>(s.target ? s.target : ceil_div(row_tiles, 8) * 8) * s.subs;
  s.slots = 2 * s.target;
  s.ml_at = s.rows_at = s.bytes = 0;
  if (s.target == 0) return s;
  const size_t n = static_cast<size_t>(s.slots) * static_cast<size_t>(s.rows * s.subs);
  s.ml_at = n * static_cast<size_t>(c.latent_dim) * 4;
  s.rows_at = s.ml_at + n * 8;
  s.bytes = s.rows_at + static_cast<size_t>(tokens) * static_cast<size_t>(heads) * 8;
  return s;
}

template <int L>
void latent_launch(const LatentShape& s, const fp8bq::LatentCache& c, const fp8bq::KvBatch& b,
                   const fp8bq::LatentQuery& q, int64_t rows, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.grid));
  if (s.rows == 32) {
    hipLaunchKernelGGL((fp8bq::latent_attend<L, 2>), grid, dim3(128), 0, st, c, b, q);
  } else {
    hipLaunchKernelGGL((fp8bq::latent_attend<L, 4>), grid, dim3(256), 0, st, c, b, q);
  }
  if (s.target == 0) return;
  if (rows <= 1024) {   // as for the key/value cache
    hipLaunchKernelGGL((fp8bq::kv_attend_join<L, 8>), dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, b, q.k, 1,
                       s.rows * s.subs);
  } else {
    hipLaunchKernelGGL((fp8bq::kv_attend_join<L, 1>), dim3(static_cast<unsigned>(ceil_div(rows, 4))), dim3(256), 0, st,
                       b, q.k, 1, s.rows * s.subs);
  }
}

}  // namespace

extern "C" {

int fp8bq_latent_append(const fp8bq_latent_cache* cache, const fp8bq_kv_batch* batch, const fp8bq_latent_tokens* t,
                        void* stream) {
  if (!latent_cache_ok(cache) || t == nullptr || !kv_batch_ok(batch, t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (!latent_heads_ok(t->q ? t->q_heads : 1, t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (batch->count == 0 || t->tokens == 0) return FP8BQ_OK;
  const LatentRows in[3] = {{{t->c, t->c_token_stride, 1, 0}, cache->latent_dim},
                            {{t->r, t->r_token_stride, 1, 0}, fp8bq::kRope},
                            {{t->q, t->q_token_stride, t->q_heads, t->q_head_stride}, fp8bq::kRope}};
  const LatentRows out[2] = {{{t->r_out, t->r_out_token_stride, 1, 0}, fp8bq::kRope},
                             {{t->q_out, t->q_out_token_stride, t->q_heads, t->q_out_head_stride}, fp8bq::kRope}};
  const int ins = t->q ? 3 : 2;
  const bool has[2] = {t->r_out != nullptr, t->q != nullptr};
  if (!kv_apart(*batch, cache->c, latent_buffers(*cache).bytes[0]) ||
      !kv_apart(*batch, cache->r, latent_buffers(*cache).bytes[1]) ||
      !kv_apart(*batch, cache->scale, latent_buffers(*cache).bytes[2])) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  for (int i = 0; i < ins; ++i) {
    if (!in[i].ok() || !latent_apart(*cache, in[i].rows.p, in[i].extent(t->tokens))) return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  for (int o = 0; o < 2; ++o) {
    if (!has[o]) continue;
    if (!out[o].ok() || !out[o].distinct(t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
    const uint64_t bytes = out[o].extent(t->tokens);
    if (!latent_apart(*cache, out[o].rows.p, bytes) || !kv_apart(*batch, out[o].rows.p, bytes)) {
      return FP8BQ_ERR_INVALID_ARGUMENT;
    }
    for (int i = 0; i < ins; ++i) {
      const bool own = i == o + 1 && latent_same(out[o], in[i], t->tokens);   // r_out in r's place, q_out in q's
      if (!own && !latent_rows_apart(out[o], in[i], t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
    }
  }
  if (has[0] && has[1] && !latent_rows_apart(out[0], out[1], t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if ((t->cos == nullptr) != (t->sin == nullptr)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (t->cos) {
    if (!kv_aligned(t->cos, 16) || !kv_aligned(t->sin, 16) || t->positions < 0) return FP8BQ_ERR_INVALID_ARGUMENT;
    // saturated: no buffer is that long
    const uint64_t rows = static_cast<uint64_t>(t->positions < (int64_t{1} << 48) ? t->positions : int64_t{1} << 48);
    const uint64_t turns = rows * 4 * (fp8bq::kRope / 2);
    for (const float* at : {t->cos, t->sin}) {
      if (turns == 0) continue;
      if (!latent_apart(*cache, at, turns)) return FP8BQ_ERR_INVALID_ARGUMENT;
      for (int o = 0; o < 2; ++o) {
        if (has[o] && overlap(out[o].rows.p, out[o].extent(t->tokens), at, turns)) return FP8BQ_ERR_INVALID_ARGUMENT;
      }
    }
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  const fp8bq::LatentCache c = latent_device(*cache);
  const fp8bq::KvBatch b = kv_device(*batch);
  fp8bq::LatentTokens d;
  d.c = static_cast<const uint16_t*>(t->c);
  d.r = static_cast<const uint16_t*>(t->r);
  d.r_out = static_cast<uint16_t*>(t->r_out);
  d.q = static_cast<const uint16_t*>(t->q);
  d.q_out = static_cast<uint16_t*>(t->q_out);
  d.cos = t->cos;
  d.sin = t->sin;
  d.c_tok = t->c_token_stride;
  d.r_tok = t->r_token_stride;
  d.r_out_tok = t->r_out_token_stride;
  d.q_tok = t->q_token_stride;
  d.q_head = t->q_head_stride;
  d.o_tok = t->q_out_token_stride;
  d.o_head = t->q_out_head_stride;
  d.positions = t->positions;
  d.tokens = static_cast<int32_t>(t->tokens);
  d.heads = t->q ? t->q_heads : 0;
  d.interleaved = t->interleaved != 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto launch = [&](auto dim) {
    constexpr int L = decltype(dim)::value;
    // Four waves to a token from 24 heads on, below that one: 17,000 tokens with 8,
    // 16, 24, 32 and 128 heads take 22, 26, 28, 35 and 116 us with four, 18, 25,
    // 30, 37 and 121 with one; 96 tokens 12 to 13 either way.
    if (d.heads >= 24) {
      hipLaunchKernelGGL((fp8bq::latent_append<L, 4>), dim3(static_cast<unsigned>(t->tokens)), dim3(fp8bq::kThreads), 0,
                         st, c, b, d);
    } else {
      hipLaunchKernelGGL((fp8bq::latent_append<L, 1>), dim3(static_cast<unsigned>(ceil_div(t->tokens, 4))),
                         dim3(fp8bq::kThreads), 0, st, c, b, d);
    }
  };
  if (cache->latent_dim == 512) {
    launch(std::integral_constant<int, 512>{});
  } else {
    launch(std::integral_constant<int, 256>{});
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

size_t fp8bq_latent_attention_workspace_bytes(const fp8bq_latent_cache* cache, const fp8bq_kv_batch* batch,
                                              int32_t q_heads, int64_t tokens) {
  if (!cache || !batch || kv_log2_page(cache->page_size) < 0 || (cache->latent_dim != 256 && cache->latent_dim != 512) ||
      batch->count < 1 || batch->count > kKvMaxBatch || batch->max_pages < 0 || tokens < 1 ||
      !latent_heads_ok(q_heads, tokens)) {
    return 0;
  }
  return latent_shape(*cache, *batch, q_heads, tokens).bytes;
}

int fp8bq_latent_attention(const fp8bq_latent_cache* cache, const fp8bq_kv_batch* batch, const fp8bq_latent_query* q,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!latent_cache_ok(cache) || q == nullptr || !kv_batch_ok(batch, q->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (!latent_heads_ok(q->q_heads, q->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  const float scale = q->scale * 1.4426950408889634f;   // for exp2
  if (!(scale - scale == 0.0f)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (batch->count == 0 || q->tokens == 0) return FP8BQ_OK;
  const LatentRows qc{{q->q, q->q_token_stride, q->q_heads, q->q_head_stride}, cache->latent_dim};
  const LatentRows qr{{q->q_rope, q->q_rope_token_stride, q->q_heads, q->q_rope_head_stride}, fp8bq::kRope};
  const LatentRows out{{q->out, q->out_token_stride, q->q_heads, q->out_head_stride}, cache->latent_dim};
  if (!qc.ok() || !qr.ok() || !out.ok() || !out.distinct(q->tokens) || !kv_aligned(q->lse, 4)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const LatentShape s = latent_shape(*cache, *batch, q->q_heads, q->tokens);
  if (s.bytes > 0 && (workspace == nullptr || workspace_bytes < s.bytes || !kv_aligned(workspace, 16))) {
    return FP8BQ_ERR_WORKSPACE;
  }
  // Queries are still read while partial sums and finished rows are written.
  const uint64_t lse_bytes = q->lse ? 4 * static_cast<uint64_t>(q->tokens) * static_cast<uint64_t>(q->q_heads) : 0;
  struct {
    const void* p;
    uint64_t bytes;
  } const written[3] = {{q->out, out.extent(q->tokens)}, {q->lse, lse_bytes}, {workspace, s.bytes}};
  for (int i = 0; i < 3; ++i) {
    if (written[i].bytes == 0) continue;
    if (!latent_apart(*cache, written[i].p, written[i].bytes) || !kv_apart(*batch, written[i].p, written[i].bytes)) {
      return FP8BQ_ERR_INVALID_ARGUMENT;
    }
    for (int j = 0; j < i; ++j) {
      if (written[j].bytes > 0 && overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes)) {
        return FP8BQ_ERR_INVALID_ARGUMENT;
      }
    }
    if (i > 0 && (overlap(written[i].p, written[i].bytes, qc.rows.p, qc.extent(q->tokens)) ||
                  overlap(written[i].p, written[i].bytes, qr.rows.p, qr.extent(q->tokens)))) {
      return FP8BQ_ERR_INVALID_ARGUMENT;
    }
  }
  if (!latent_rows_apart(out, qc, q->tokens) || !latent_rows_apart(out, qr, q->tokens)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  const fp8bq::LatentCache c = latent_device(*cache);
  const fp8bq::KvBatch b = kv_device(*batch);
  fp8bq::LatentQuery d;
  char* ws = static_cast<char*>(workspace);
  const bool split = s.target > 0;
  d.k.q = static_cast<const uint16_t*>(q->q);
  d.k.out = static_cast<uint16_t*>(q->out);
  d.k.lse = q->lse;
  d.k.part = split ? reinterpret_cast<float*>(ws) : nullptr;
  d.k.part_ml = split ? reinterpret_cast<float2*>(ws + s.ml_at) : nullptr;
  d.k.rows = split ? reinterpret_cast<int2*>(ws + s.rows_at) : nullptr;
  d.k.q_tok = q->q_token_stride;
  d.k.q_head = q->q_head_stride;
  d.k.o_tok = q->out_token_stride;
  d.k.o_head = q->out_head_stride;
  d.k.tokens = static_cast<int32_t>(q->tokens);
  d.k.group = q->q_heads;
  d.k.window = 0;
  d.k.slots = s.slots;
  d.k.target = s.target;
  d.k.jump = s.target;
  d.k.min_tiles = 1;
  d.k.tile_rows = s.rows * s.subs;
  d.k.extra = kLatentExtra;
  d.subs = s.subs;
  d.k.scale = scale;
  d.r = static_cast<const uint16_t*>(q->q_rope);
  d.r_tok = q->q_rope_token_stride;
  d.r_head = q->q_rope_head_stride;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t rows = q->tokens * q->q_heads;
  if (cache->latent_dim == 512) {
    latent_launch<512>(s, c, b, d, rows, st);
  } else {
    latent_launch<256>(s, c, b, d, rows, st);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

int fp8bq_latent_prompt_attention(const fp8bq_latent_prompt* p, void* stream) {
  if (p == nullptr || p->tokens < 0 || p->keys < 0 || p->count < 0 || p->count > kKvMaxBatch) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if ((p->head_dim != 64 && p->head_dim != 128) || !latent_heads_ok(p->heads, p->tokens) ||
      p->keys > kKvMaxRows / p->heads || static_cast<int64_t>(p->count) * p->heads > kKvMaxBlocks) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const float scale = p->scale * 1.4426950408889634f;   // for exp2
  if (!(scale - scale == 0.0f)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (p->count == 0 || p->tokens == 0) return FP8BQ_OK;
  if (!p->query_start || !kv_aligned(p->query_start, 4) || !kv_aligned(p->key_start, 4) || !kv_aligned(p->lse, 4) ||
      (!p->key_start && p->keys != p->tokens)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const int32_t D = p->head_dim;
  const LatentRows q{{p->q, p->q_token_stride, p->heads, p->q_head_stride}, D + fp8bq::kRope};
  const LatentRows out{{p->out, p->out_token_stride, p->heads, p->out_head_stride}, D};
  const LatentRows in[3] = {{{p->k, p->k_token_stride, p->heads, p->k_head_stride}, D},
                            {{p->k_rope, p->k_rope_token_stride, 1, 0}, fp8bq::kRope},
                            {{p->v, p->v_token_stride, p->heads, p->v_head_stride}, D}};
  if (!q.ok() || !out.ok() || !out.distinct(p->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  // places of a tile's rows stay in 32 bits
  for (const int64_t pitch : {p->k_token_stride, p->k_rope_token_stride, p->v_token_stride}) {
    if (pitch >= kPromptMaxStride) return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const uint64_t out_bytes = out.extent(p->tokens);
  const uint64_t lse_bytes = p->lse ? 4 * static_cast<uint64_t>(p->tokens) * static_cast<uint64_t>(p->heads) : 0;
  const uint64_t starts = 4 * (static_cast<uint64_t>(p->count) + 1);
  // Other workgroups read while one writes: what is written lies apart from all else.
  const auto apart = [&](const void* at, uint64_t bytes) {
    return !overlap(at, bytes, p->out, out_bytes) && (lse_bytes == 0 || !overlap(at, bytes, p->lse, lse_bytes));
  };
  if (!latent_rows_apart(out, q, p->tokens) || (lse_bytes > 0 && (overlap(p->lse, lse_bytes, p->out, out_bytes) ||
                                                                  overlap(p->lse, lse_bytes, p->q, q.extent(p->tokens))))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!apart(p->query_start, starts) || (p->key_start && !apart(p->key_start, starts))) return FP8BQ_ERR_INVALID_ARGUMENT;
  for (const LatentRows& x : in) {
    if (p->keys == 0) break;
    if (!x.ok() || !apart(x.rows.p, x.extent(p->keys))) return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  fp8bq::PromptQuery d;
  d.q = static_cast<const uint16_t*>(p->q);
  d.k = static_cast<const uint16_t*>(p->k);
  d.r = static_cast<const uint16_t*>(p->k_rope);
  d.v = static_cast<const uint16_t*>(p->v);
  d.out = static_cast<uint16_t*>(p->out);
  d.lse = p->lse;
  d.q_at = p->query_start;
  d.k_at = p->key_start ? p->key_start : p->query_start;
  d.q_tok = p->q_token_stride;
  d.q_head = p->q_head_stride;
  d.k_tok = p->k_token_stride;
  d.k_head = p->k_head_stride;
  d.r_tok = p->k_rope_token_stride;
  d.v_tok = p->v_token_stride;
  d.v_head = p->v_head_stride;
  d.o_tok = p->out_token_stride;
  d.o_head = p->out_head_stride;
  d.tokens = static_cast<int32_t>(p->tokens);
  d.keys = static_cast<int32_t>(p->keys);
  d.heads = p->heads;
  d.count = p->count;
  d.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t slots = p->tokens / 128 + p->count;
  const dim3 grid(static_cast<unsigned>(slots * p->heads));
  // Where row tiles leave CUs idle (an eighth over, as slots count a tile too many
  // for most sequences), two sets of waves walk the keys of one: one prompt of 4096
  // at 8 heads of 128 (264 slots) 92 -> 75 us, 500 queries over 8000 keys at 32
  // heads (128) 171 -> 134.  Beyond it one set is faster mostly: four prompts of 700
  // at 16 heads (400) 28, with two 33; one of 4096 at 32 heads (1056) 178 and 188.
  // The number of slots does not tell how many tiles the longest row tile has, and
  // so it errs where that decides: nine prompts of 300 at 8 heads (240) take 14.1
  // with two sets, 13.5 with one; one of 4096 at 16 heads (528) 113 with one, 97
  // with two.
  const bool few = slots * p->heads <= 288;
  const auto launch = [&](auto dim) {
    constexpr int kDim = decltype(dim)::value;
    if (few) {
      hipLaunchKernelGGL((fp8bq::latent_prompt<kDim, 2>), grid, dim3(512), 0, st, d);
    } else {
      hipLaunchKernelGGL((fp8bq::latent_prompt<kDim, 1>), grid, dim3(256), 0, st, d);
    }
  };
  if (D == 128) {
    launch(std::integral_constant<int, 128>{});
  } else {
    launch(std::integral_constant<int, 64>{});
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

}  // extern "C"
