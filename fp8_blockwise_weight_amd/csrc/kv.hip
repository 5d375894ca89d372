// Host side of the blockwise e4m3 key/value cache: the fp8bq_kv_* calls of
// include/fp8bq.h.  Every argument check runs before the first HIP call;
// the calls enqueue on the caller's stream and neither allocate nor wait.

#include "kv_kernels.hpp"

namespace {

int kv_log2_page(int32_t page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    case 256: return 8;
    default: return -1;
  }
}

bool kv_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Grids and in-kernel row numbers stay in 32 bits.
constexpr int64_t kKvMaxRows = int64_t{1} << 25;   // query tokens x query heads
constexpr int32_t kKvMaxBatch = 1 << 20;
constexpr int64_t kKvMaxStride = int64_t{1} << 36;   // elements; extents stay in 64 bits
constexpr int64_t kKvMaxBlocks = int64_t{1} << 21;  // sequences x key/value heads

bool kv_cache_ok(const fp8bq_kv_cache* c) {
  if (c == nullptr || kv_log2_page(c->page_size) < 0) return false;
  if (c->head_dim < 64 || c->head_dim > 256 || c->head_dim % 64 != 0) return false;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->num_pages < 1 || c->num_pages > INT32_MAX) return false;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return false;
  if (!kv_aligned(c->k, 16) || !kv_aligned(c->v, 16) || !kv_aligned(c->k_scale, 4) ||
      !kv_aligned(c->v_scale, 4)) {
    return false;
  }
  const uint64_t blocks = static_cast<uint64_t>(c->num_pages) * static_cast<uint64_t>(c->kv_heads);
  const uint64_t codes = blocks * static_cast<uint64_t>(c->page_size) * static_cast<uint64_t>(c->head_dim);
  const void* at[4] = {c->k, c->v, c->k_scale, c->v_scale};
  const uint64_t size[4] = {codes, codes, 4 * blocks, 4 * blocks};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j) {
      if (overlap(at[i], size[i], at[j], size[j])) return false;
    }
  }
  return true;
}

bool kv_batch_ok(const fp8bq_kv_batch* b, int64_t tokens) {
  if (b == nullptr || b->count < 0 || b->count > kKvMaxBatch || b->max_pages < 0 || tokens < 0) return false;
  if (b->count == 0) return true;
  if (b->table_stride < b->max_pages || (b->max_pages > 0 && !b->block_table) || !b->seq_lens) return false;
  if (!kv_aligned(b->block_table, 4) || !kv_aligned(b->seq_lens, 4) || !kv_aligned(b->query_start, 4)) return false;
  return b->query_start != nullptr || tokens == b->count;
}

// Rows of 16-byte words: base and strides.
bool kv_rows_ok(const void* p, int64_t tok, int64_t head) {
  return p != nullptr && kv_aligned(p, 16) && tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0 &&
         tok < kKvMaxStride && head < kKvMaxStride;
}

// Whether such rows share no elements, as those must that are written.
bool kv_distinct(int64_t tokens, int64_t tok, int64_t heads, int64_t head, int32_t dim) {
  if ((heads > 1 && head < dim) || (tokens > 1 && tok < dim)) return false;
  return heads == 1 || tokens == 1 || tok >= (heads - 1) * head + dim || head >= (tokens - 1) * tok + dim;
}

// Bytes from the first to the last of such rows.
uint64_t kv_extent(int64_t tokens, int64_t tok, int64_t heads, int64_t head, int32_t dim) {
  return 2 * static_cast<uint64_t>((tokens - 1) * tok + (heads - 1) * head + dim);
}

// BF16 rows [tokens, heads, dim] of a call.
struct KvRows {
  const void* p;
  int64_t tok, heads, head;
};

// Whether rows share no element with others: by their extents, or interleaved
// with them token by token or head by head, as slices of one tensor are.
bool kv_rows_apart(const KvRows& a, const KvRows& b, int64_t tokens, int32_t dim) {
  if (!overlap(a.p, kv_extent(tokens, a.tok, a.heads, a.head, dim), b.p,
               kv_extent(tokens, b.tok, b.heads, b.head, dim))) {
    return true;
  }
  const int64_t off = (static_cast<int64_t>(reinterpret_cast<intptr_t>(b.p)) -
                       static_cast<int64_t>(reinterpret_cast<intptr_t>(a.p))) / 2;
  // pieces of `in_a` and `in_b` elements, the next ones `out` further on
  auto beside = [&](int64_t out, int64_t in_a, int64_t in_b) {
    if (out <= 0) return false;
    const int64_t d = (off % out + out) % out;
    return d >= in_a && d + in_b <= out;
  };
  return (a.tok == b.tok && beside(a.tok, (a.heads - 1) * a.head + dim, (b.heads - 1) * b.head + dim)) ||
         (a.head == b.head && beside(a.head, (tokens - 1) * a.tok + dim, (tokens - 1) * b.tok + dim));
}

// Whether output rows are their input's own, or apart from them.
bool kv_rows_same_or_apart(const KvRows& out, const KvRows& in, int64_t tokens, int32_t dim) {
  const bool same = out.p == in.p && (tokens == 1 || out.tok == in.tok) && (in.heads == 1 || out.head == in.head);
  return same || kv_rows_apart(out, in, tokens, dim);
}

// Whether a buffer that is written lies apart from all of the cache.
bool kv_apart(const fp8bq_kv_cache& c, const void* p, uint64_t bytes) {
  const uint64_t blocks = static_cast<uint64_t>(c.num_pages) * static_cast<uint64_t>(c.kv_heads);
  const uint64_t codes = blocks * static_cast<uint64_t>(c.page_size) * static_cast<uint64_t>(c.head_dim);
  return !overlap(p, bytes, c.k, codes) && !overlap(p, bytes, c.v, codes) &&
         !overlap(p, bytes, c.k_scale, 4 * blocks) && !overlap(p, bytes, c.v_scale, 4 * blocks);
}

// Whether a buffer that is written lies apart from the batch's arrays, which
// workgroups read at any time.
bool kv_apart(const fp8bq_kv_batch& b, const void* p, uint64_t bytes) {
  const uint64_t n = static_cast<uint64_t>(b.count), width = static_cast<uint64_t>(b.max_pages);
  const uint64_t table = width > 0 ? 4 * ((n - 1) * static_cast<uint64_t>(b.table_stride) + width) : 0;
  const auto hits = [&](const void* at, uint64_t size) { return bytes > 0 && size > 0 && overlap(p, bytes, at, size); };
  return !hits(b.block_table, table) && !hits(b.seq_lens, 4 * n) &&
         !hits(b.query_start, b.query_start ? 4 * (n + 1) : 0);
}

// The same for all of a cache that is written.
bool kv_apart(const fp8bq_kv_batch& b, const fp8bq_kv_cache& c) {
  const uint64_t blocks = static_cast<uint64_t>(c.num_pages) * static_cast<uint64_t>(c.kv_heads);
  const uint64_t codes = blocks * static_cast<uint64_t>(c.page_size) * static_cast<uint64_t>(c.head_dim);
  return kv_apart(b, c.k, codes) && kv_apart(b, c.v, codes) && kv_apart(b, c.k_scale, 4 * blocks) &&
         kv_apart(b, c.v_scale, 4 * blocks);
}

fp8bq::KvCache kv_device(const fp8bq_kv_cache& c) {
  fp8bq::KvCache d;
  d.k = static_cast<uint8_t*>(c.k);
  d.v = static_cast<uint8_t*>(c.v);
  d.ks = c.k_scale;
  d.vs = c.v_scale;
  d.pages = static_cast<int32_t>(c.num_pages);
  d.heads = c.kv_heads;
  d.log_s = kv_log2_page(c.page_size);
  return d;
}

fp8bq::KvBatch kv_device(const fp8bq_kv_batch& b) {
  return fp8bq::KvBatch{b.block_table, b.seq_lens, b.query_start, b.table_stride, b.count, b.max_pages};
}

// f(std::integral_constant<int, D>) for the cache's head_dim.
template <typename F>
void kv_for_dim(int32_t dim, F&& f) {
  switch (dim) {
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 128: f(std::integral_constant<int, 128>{}); break;
    case 192: f(std::integral_constant<int, 192>{}); break;
    default: f(std::integral_constant<int, 256>{}); break;
  }
}

// Key tiles, of those a row tile can see at most, up to which splitting them
// over workgroups does not pay: a few more tiles to each wave (1.5 to 2 us
// each) cost less than joining parts in a second launch.
constexpr int64_t kKvFew = 8, kKvWhole = 16, kKvWholeOfMany = 32;

// How an attention call is cut up: from the shapes alone, so that the
// workspace can be sized, and a launch captured, before any length is known.
//
// Rows of a workgroup, by the mean number of query rows per sequence (32
// sequences of 8192, 8 query heads to each of 4 key heads of 128):
//   up to 16   kv_attend_rows<16>: 16 rows 55.0 us, with <32> 56.6 (128
//              sequences: 339 against 361; half the registers go unused)
//   17 to 32   kv_attend_rows<32>: 24 rows 57.5, in tiles of 64 rows 64.2
//              (256 channels: 102 against 222); not so for few long sequences
//              (2 of 40000, 32 rows: 34.7 against 29.0), which the rule, that
//              goes by rows, does not tell apart
//   33 to 64   tiles of 64 rows: 64 rows 75, in tiles of 128 rows 94; above 128
//              channels, whose registers leave one wave per SIMD, twice
//              kv_attend_rows<32>: 64 rows of 256 channels 172, in tiles of 128
//              229 (but 100 sequences of 500, 80 and 71: tiles of 128 where
//              keys are few and row tiles many)
//   above      tiles of 128 rows (80 rows of 256 channels 232, in three of 32
//              262)
// Where key tiles are few, tiles of 64 rows are also taken for 17 to 32 rows
// of 128 channels, if workgroups of kv_attend_rows<32>, one to a CU, would take
// turns (100 sequences of 200 or 500, 24 rows: 22.0 -> 16.9, 27.7 -> 25.3), and
// for 129 to 192 rows, of which tiles of 128 would leave a quarter empty
// (100 sequences of 300 or 1000, 144 rows: 41 -> 35, 84 -> 76; of 8192, where
// keys are read from HBM, 162 -> 181, so not there).
// Keys are not split over workgroups where row tiles see few key tiles (a small
// window counts), or not many and there are many row tiles:
//   kv_attend_rows   one sequence of 1256: 14.9 split, 15.0 not; 16 of 2000:
//                    26.1 and 22.2; 8 of 2000: 18.2 and 22.0; 25 of 1256,
//                    16 heads to a key head of 64: 20.1 and 12.3
//   kv_attend_tiles  a prompt of 300 / 1000 / 2000: 21.3 / 45.8 / 70.1 split,
//                    14.8 / 32.7 / 62.3 not; 500 tokens over 2000: 43.5 and
//                    54.5; window of 30, 18 sequences: 26.6 and 13.0
// `resident` workgroups are what registers and LDS let the card hold at once
// and what was fastest: one sequence of 131071, rows of 16, 512: 52.8 us,
// 384: 61.6, 768: 55.4; drafted tokens in tiles of 64, 1024: 49.2, 768: 52.9,
// 1536: 58.8.
struct KvShape {
  int32_t group;       // query heads per key/value head
  int32_t rows;        // query rows (tokens x heads of a group) of a workgroup
  int32_t grid;        // workgroups per key/value head
  int32_t target;      // of these, how many splitting the keys aims at; 0: no splits
  int32_t slots;       // places for partial sums per key/value head
  int32_t jump;
  int32_t min_tiles;
  size_t rows_at, ml_at, bytes;   // workspace: partial sums at 0, then these
};

KvShape kv_shape(const fp8bq_kv_cache& c, const fp8bq_kv_batch& b, int32_t q_heads, int64_t tokens,
                 int32_t window) {
  KvShape s;
  s.group = q_heads / c.kv_heads;
  const int64_t per_seq = ceil_div(tokens * s.group, b.count);
  const auto row_tiles = [&](int32_t rows) { return tokens * s.group / rows + b.count; };   // of a head, at most
  const auto key_tiles = [&](int32_t rows) {   // of a row tile, at most
    const int64_t all = ceil_div(static_cast<int64_t>(b.max_pages) * c.page_size, 64);
    const int64_t seen = ceil_div(int64_t{window} + rows / s.group, 64) + 1;
    return window > 0 && seen < all ? seen : all;
  };
  s.rows = per_seq <= 16 ? 16 : (per_seq <= 32 ? 32 : (per_seq <= 64 && c.head_dim <= 128 ? 64 : 128));
  if (s.rows == 32 && c.head_dim == 128 && key_tiles(32) <= kKvFew && row_tiles(32) * c.kv_heads > 256) s.rows = 64;
  if (s.rows == 128 && c.head_dim > 128 && per_seq <= 64 &&
      (key_tiles(32) > kKvWhole || row_tiles(32) * c.kv_heads <= 256)) {
    s.rows = 32;
  }
  if (s.rows == 128 && c.head_dim <= 128 && per_seq > 128 && per_seq <= 192 && key_tiles(128) <= kKvWhole) s.rows = 64;
  const int64_t base = row_tiles(s.rows), tiles = key_tiles(s.rows), items = base * c.kv_heads;
  const int resident =
      s.rows == 16 ? (c.head_dim == 64 ? 768 : 512) : (s.rows == 64 ? 1024 : (s.rows == 128 ? 512 : 256));
  s.min_tiles = 4;
  s.target = static_cast<int32_t>(ceil_div(resident, c.kv_heads));
  if (s.rows <= 32) {
    if (tiles <= kKvWhole || (tiles <= kKvWholeOfMany && items >= 128)) s.target = 0;
    s.grid = s.target ? s.target : static_cast<int32_t>(base);
    s.slots = 2 * s.target;
    s.jump = s.target;
  } else {
    const int64_t few = c.head_dim <= 128 ? kKvFew : kKvFew / 2;   // a tile takes twice as long
    if (tiles <= few || items >= resident || (tiles <= kKvWholeOfMany && items >= resident / 2)) s.target = 0;
    s.grid = static_cast<int32_t>(base + s.target);
    s.slots = s.grid;
    s.jump = 0;
  }
  if (s.target == 0) {
    s.slots = s.jump = 0;
    s.ml_at = s.rows_at = s.bytes = 0;
    return s;
  }
  const size_t n = static_cast<size_t>(s.slots) * static_cast<size_t>(c.kv_heads) * static_cast<size_t>(s.rows);
  s.ml_at = n * static_cast<size_t>(c.head_dim) * 4;
  s.rows_at = s.ml_at + n * 8;
  s.bytes = s.rows_at + static_cast<size_t>(tokens) * static_cast<size_t>(q_heads) * 8;
  return s;
}

// A grid of `slots` workgroups per head stays below 2^32 work-items for
// count * kv_heads <= 2^21 (slots <= rows / 16 + count + 1024 / kv_heads + 1).
bool kv_heads_ok(int32_t q_heads, int32_t kv_heads, int32_t count, int64_t tokens) {
  return q_heads >= 1 && q_heads % kv_heads == 0 && tokens <= kKvMaxRows / q_heads &&
         static_cast<int64_t>(count) * kv_heads <= kKvMaxBlocks;
}

}  // namespace

extern "C" {

int fp8bq_kv_append(const fp8bq_kv_cache* cache, const fp8bq_kv_batch* batch, const fp8bq_kv_tokens* t,
                    void* stream) {
  if (!kv_cache_ok(cache) || t == nullptr || !kv_batch_ok(batch, t->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (t->rot_dim < 0 || t->rot_dim > cache->head_dim || t->rot_dim % 16 != 0) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (!kv_heads_ok(t->q ? t->q_heads : cache->kv_heads, cache->kv_heads, batch->count, t->tokens)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (batch->count == 0 || t->tokens == 0) return FP8BQ_OK;
  if (!kv_rows_ok(t->k, t->k_token_stride, t->k_head_stride) ||
      !kv_rows_ok(t->v, t->v_token_stride, t->v_head_stride)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (t->q && (!kv_rows_ok(t->q, t->q_token_stride, t->q_head_stride) ||
               !kv_rows_ok(t->q_out, t->q_out_token_stride, t->q_out_head_stride) ||
               !kv_distinct(t->tokens, t->q_out_token_stride, t->q_heads, t->q_out_head_stride, cache->head_dim))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const int32_t dim = cache->head_dim;
  if (!kv_apart(*batch, *cache) ||
      (t->q && !kv_apart(*batch, t->q_out,
                         kv_extent(t->tokens, t->q_out_token_stride, t->q_heads, t->q_out_head_stride, dim)))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!kv_apart(*cache, t->k, kv_extent(t->tokens, t->k_token_stride, cache->kv_heads, t->k_head_stride, dim)) ||
      !kv_apart(*cache, t->v, kv_extent(t->tokens, t->v_token_stride, cache->kv_heads, t->v_head_stride, dim)) ||
      (t->q && (!kv_apart(*cache, t->q, kv_extent(t->tokens, t->q_token_stride, t->q_heads, t->q_head_stride, dim)) ||
                !kv_apart(*cache, t->q_out,
                          kv_extent(t->tokens, t->q_out_token_stride, t->q_heads, t->q_out_head_stride, dim))))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (t->q) {
    const KvRows out{t->q_out, t->q_out_token_stride, t->q_heads, t->q_out_head_stride};
    if (!kv_rows_same_or_apart(out, KvRows{t->q, t->q_token_stride, t->q_heads, t->q_head_stride}, t->tokens, dim) ||
        !kv_rows_apart(out, KvRows{t->k, t->k_token_stride, cache->kv_heads, t->k_head_stride}, t->tokens, dim) ||
        !kv_rows_apart(out, KvRows{t->v, t->v_token_stride, cache->kv_heads, t->v_head_stride}, t->tokens, dim)) {
      return FP8BQ_ERR_INVALID_ARGUMENT;
    }
  }
  if (t->rot_dim > 0 && (!t->cos || !t->sin || !kv_aligned(t->cos, 16) || !kv_aligned(t->sin, 16) ||
                         t->positions < 0)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (t->rot_dim > 0 && t->positions > 0) {
    // saturated: no buffer is that long
    const uint64_t rows = static_cast<uint64_t>(t->positions < (int64_t{1} << 48) ? t->positions : int64_t{1} << 48);
    const uint64_t turns = rows * static_cast<uint64_t>(t->rot_dim) * 2;
    const uint64_t written = t->q ? kv_extent(t->tokens, t->q_out_token_stride, t->q_heads, t->q_out_head_stride, dim) : 0;
    for (const float* at : {t->cos, t->sin}) {
      if (!kv_apart(*cache, at, turns) || (t->q && overlap(t->q_out, written, at, turns))) {
        return FP8BQ_ERR_INVALID_ARGUMENT;
      }
    }
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  const fp8bq::KvCache c = kv_device(*cache);
  const fp8bq::KvBatch b = kv_device(*batch);
  fp8bq::KvTokens d;
  d.k = static_cast<const uint16_t*>(t->k);
  d.v = static_cast<const uint16_t*>(t->v);
  d.q = static_cast<const uint16_t*>(t->q);
  d.q_out = static_cast<uint16_t*>(t->q_out);
  d.cos = t->cos;
  d.sin = t->sin;
  d.k_tok = t->k_token_stride;
  d.k_head = t->k_head_stride;
  d.v_tok = t->v_token_stride;
  d.v_head = t->v_head_stride;
  d.q_tok = t->q_token_stride;
  d.q_head = t->q_head_stride;
  d.o_tok = t->q_out_token_stride;
  d.o_head = t->q_out_head_stride;
  d.positions = t->positions;
  d.tokens = static_cast<int32_t>(t->tokens);
  d.group = t->q ? t->q_heads / cache->kv_heads : 0;
  d.half = t->rot_dim / 2;
  d.interleaved = t->interleaved != 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  kv_for_dim(cache->head_dim, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (batch->query_start == nullptr) {
      const int64_t waves = static_cast<int64_t>(batch->count) * cache->kv_heads;
      hipLaunchKernelGGL(fp8bq::kv_append_step<D>, dim3(static_cast<unsigned>(ceil_div(waves, 4))),
                         dim3(fp8bq::kThreads), 0, st, c, b, d);
    } else {
      const int64_t slots = (t->tokens >> c.log_s) + 2 * static_cast<int64_t>(batch->count);
      hipLaunchKernelGGL(fp8bq::kv_append_pages<D>, dim3(static_cast<unsigned>(slots * cache->kv_heads)),
                         dim3(fp8bq::kThreads), 0, st, c, b, d);
    }
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

size_t fp8bq_kv_attention_workspace_bytes(const fp8bq_kv_cache* cache, const fp8bq_kv_batch* batch,
                                          int32_t q_heads, int64_t tokens) {
  if (!cache || !batch || cache->kv_heads < 1 || kv_log2_page(cache->page_size) < 0 || cache->head_dim < 1 ||
      batch->count < 1 || batch->max_pages < 0 || tokens < 1 ||
      !kv_heads_ok(q_heads, cache->kv_heads, batch->count, tokens)) {
    return 0;
  }
  return kv_shape(*cache, *batch, q_heads, tokens, 0).bytes;
}

int fp8bq_kv_attention(const fp8bq_kv_cache* cache, const fp8bq_kv_batch* batch, const fp8bq_kv_query* q,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!kv_cache_ok(cache) || q == nullptr || !kv_batch_ok(batch, q->tokens)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (!kv_heads_ok(q->q_heads, cache->kv_heads, batch->count, q->tokens) || q->window < 0) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const float scale = q->scale * 1.4426950408889634f;   // for exp2
  if (!(scale - scale == 0.0f)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (batch->count == 0 || q->tokens == 0) return FP8BQ_OK;
  if (!kv_rows_ok(q->q, q->q_token_stride, q->q_head_stride) ||
      !kv_rows_ok(q->out, q->out_token_stride, q->out_head_stride) || !kv_aligned(q->lse, 4) ||
      !kv_distinct(q->tokens, q->out_token_stride, q->q_heads, q->out_head_stride, cache->head_dim)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!kv_rows_same_or_apart(KvRows{q->out, q->out_token_stride, q->q_heads, q->out_head_stride},
                             KvRows{q->q, q->q_token_stride, q->q_heads, q->q_head_stride}, q->tokens,
                             cache->head_dim)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  // The workspace is sized without the window: a shape that wants more is not taken.
  KvShape s = kv_shape(*cache, *batch, q->q_heads, q->tokens, q->window);
  const KvShape all = kv_shape(*cache, *batch, q->q_heads, q->tokens, 0);
  if (s.bytes > all.bytes) s = all;
  if (s.bytes > 0 && (workspace == nullptr || workspace_bytes < s.bytes || !kv_aligned(workspace, 16))) {
    return FP8BQ_ERR_WORKSPACE;
  }
  const uint64_t out_bytes =
      kv_extent(q->tokens, q->out_token_stride, q->q_heads, q->out_head_stride, cache->head_dim);
  const uint64_t lse_bytes = q->lse ? 4 * static_cast<uint64_t>(q->tokens) * static_cast<uint64_t>(q->q_heads) : 0;
  // Queries are still read while partial sums and finished rows are written.
  const uint64_t q_bytes = kv_extent(q->tokens, q->q_token_stride, q->q_heads, q->q_head_stride, cache->head_dim);
  if (overlap(q->q, q_bytes, q->lse, lse_bytes) || (s.bytes > 0 && overlap(q->q, q_bytes, workspace, s.bytes))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!kv_apart(*cache, q->out, out_bytes) || !kv_apart(*cache, q->lse, lse_bytes) ||
      !kv_apart(*cache, workspace, s.bytes) || overlap(q->out, out_bytes, q->lse, lse_bytes) ||
      overlap(q->out, out_bytes, workspace, s.bytes) || overlap(q->lse, lse_bytes, workspace, s.bytes)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!kv_apart(*batch, q->out, out_bytes) || !kv_apart(*batch, q->lse, lse_bytes) ||
      !kv_apart(*batch, workspace, s.bytes)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  const fp8bq::KvCache c = kv_device(*cache);
  const fp8bq::KvBatch b = kv_device(*batch);
  fp8bq::KvQuery d;
  d.q = static_cast<const uint16_t*>(q->q);
  d.out = static_cast<uint16_t*>(q->out);
  d.lse = q->lse;
  char* ws = static_cast<char*>(workspace);
  const bool split = s.target > 0;
  d.part = split ? reinterpret_cast<float*>(ws) : nullptr;
  d.part_ml = split ? reinterpret_cast<float2*>(ws + s.ml_at) : nullptr;
  d.rows = split ? reinterpret_cast<int2*>(ws + s.rows_at) : nullptr;
  d.q_tok = q->q_token_stride;
  d.q_head = q->q_head_stride;
  d.o_tok = q->out_token_stride;
  d.o_head = q->out_head_stride;
  d.tokens = static_cast<int32_t>(q->tokens);
  d.group = s.group;
  d.window = q->window;
  d.slots = s.slots;
  d.target = s.target;
  d.jump = s.jump;
  d.min_tiles = s.min_tiles;
  d.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  kv_for_dim(cache->head_dim, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    const dim3 grid(static_cast<unsigned>(s.grid) * static_cast<unsigned>(cache->kv_heads));
    switch (s.rows) {
      case 16: hipLaunchKernelGGL((fp8bq::kv_attend_rows<D, 1>), grid, dim3(256), 0, st, c, b, d); break;
      case 32: hipLaunchKernelGGL((fp8bq::kv_attend_rows<D, 2>), grid, dim3(256), 0, st, c, b, d); break;
      case 64:
        if constexpr (D <= 128) {
          if (c.log_s >= 6) {
            hipLaunchKernelGGL((fp8bq::kv_attend_tiles<D, 2, true>), grid, dim3(128), 0, st, c, b, d);
          } else {
            hipLaunchKernelGGL((fp8bq::kv_attend_tiles<D, 2, false>), grid, dim3(128), 0, st, c, b, d);
          }
        }
        break;
      default:
        if (c.log_s >= 6) {
          hipLaunchKernelGGL((fp8bq::kv_attend_tiles<D, 4, true>), grid, dim3(256), 0, st, c, b, d);
        } else {
          hipLaunchKernelGGL((fp8bq::kv_attend_tiles<D, 4, false>), grid, dim3(256), 0, st, c, b, d);
        }
    }
    if (split) {
      const int64_t rows = q->tokens * q->q_heads;
      if (rows <= 1024) {
        hipLaunchKernelGGL((fp8bq::kv_attend_join<D, 8>), dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, b, d,
                           c.heads, s.rows);
      } else {
        hipLaunchKernelGGL((fp8bq::kv_attend_join<D, 1>), dim3(static_cast<unsigned>(ceil_div(rows, 4))), dim3(256), 0,
                           st, b, d, c.heads, s.rows);
      }
    }
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

}  // extern "C"
