// Host side of the calls on caches' pages: fp8bq_cache_fork and
// fp8bq_cache_compact of include/fp8bq.h.  Every argument check runs before the
// first HIP call; the calls enqueue on the caller's stream and neither allocate
// nor wait.

#include <algorithm>

#include "pages_kernels.hpp"

namespace {

constexpr int32_t kMaxPageBuffers = 4096;
// Bytes: a page of fewer is copied by one wave, with others of its number.  256
// bytes (a latent page's scales) by workgroups of their own: 8 layers' latents,
// 520 MB, 92 us for 88; 4 and 8 KB by a wave: 225 for 88, four forks of 27 layers 141
// for 14.
constexpr int64_t kSmallPage = 1024;

// A range of memory that a call reads or writes.
struct Range {
  uintptr_t at, end;
};

Range range_of(const void* p, uint64_t bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return Range{at, at + static_cast<uintptr_t>(bytes)};
}

// The buffers' ranges, in order.  (On the stack, 64 KB: nothing here may throw.)
struct Ranges {
  Range at[kMaxPageBuffers];
  int32_t count;
  const Range* begin() const { return at; }
  const Range* end() const { return at + count; }
};

// Fills them in, or gives false where something is wrong.
bool pages_ok(const fp8bq_pages* p, Ranges& all) {
  if (p == nullptr || kv_log2_page(p->page_size) < 0 || p->num_pages < 1 || p->num_pages > INT32_MAX) return false;
  if (p->count < 1 || p->count > kMaxPageBuffers || p->buffers == nullptr) return false;
  all.count = p->count;
  for (int32_t i = 0; i < p->count; ++i) {
    const fp8bq_page_buffer& x = p->buffers[i];
    if (!x.p || !kv_aligned(x.p, 4) || x.page_bytes < 4 || x.page_bytes > INT32_MAX || x.page_bytes % 4 != 0) return false;
    all.at[i] = range_of(x.p, static_cast<uint64_t>(p->num_pages) * static_cast<uint64_t>(x.page_bytes));
  }
  std::sort(all.at, all.at + all.count, [](const Range& a, const Range& b) { return a.at < b.at; });
  for (int32_t i = 1; i < all.count; ++i) {
    if (all.at[i].at < all.at[i - 1].end) return false;
  }
  return true;
}

// Whether a range lies apart from all buffers.
bool pages_apart(const Ranges& all, const void* p, uint64_t bytes) {
  if (bytes == 0) return true;
  const Range r = range_of(p, bytes);
  const Range* after = std::upper_bound(all.begin(), all.end(), r.at, [](uintptr_t v, const Range& x) { return v < x.at; });
  if (after != all.end() && after->at < r.end) return false;
  return after == all.begin() || (after - 1)->end <= r.at;
}

bool table_ok(const void* table, int64_t stride, int32_t count, int32_t max_pages) {
  return count >= 0 && count <= kKvMaxBatch && max_pages >= 0 && stride >= max_pages && stride < kKvMaxStride &&
         (max_pages == 0 || count == 0 || table != nullptr) && kv_aligned(table, 4);
}

uint64_t table_bytes(int64_t stride, int32_t count, int32_t max_pages) {
  if (count == 0 || max_pages == 0) return 0;
  return 4 * (static_cast<uint64_t>(count - 1) * static_cast<uint64_t>(stride) + static_cast<uint64_t>(max_pages));
}

// f(list) for runs of buffers that fit a launch's arguments, the first of them
// with the tables.
template <typename F>
void for_page_lists(const fp8bq_pages& p, F&& f) {
  fp8bq::PageList l;
  l.pages = static_cast<int32_t>(p.num_pages);
  l.log_s = kv_log2_page(p.page_size);
  for (int32_t at = 0; at < p.count; at += fp8bq::kPageBuffers) {
    const int32_t n = std::min(p.count - at, static_cast<int32_t>(fp8bq::kPageBuffers));
    l.count = l.large = l.chunks = 0;
    l.tables = at == 0;
    for (int pass = 0; pass < 2; ++pass) {
      for (int32_t i = at; i < at + n; ++i) {
        const fp8bq_page_buffer& x = p.buffers[i];
        const bool large = x.page_bytes >= kSmallPage && x.page_bytes % 16 == 0 && kv_aligned(x.p, 16);
        if (large != (pass == 0)) continue;
        l.p[l.count] = static_cast<uint8_t*>(x.p);
        l.bytes[l.count++] = static_cast<uint32_t>(x.page_bytes);
        if (large) l.chunks = std::max(l.chunks, static_cast<int32_t>(ceil_div(x.page_bytes, fp8bq::kPageChunk)));
      }
      if (pass == 0) l.large = l.count;
    }
    l.chunks = std::max(l.chunks, 1);
    f(l);
  }
}

}  // namespace

extern "C" {

int fp8bq_cache_fork(const fp8bq_pages* pages, int32_t* block_table, int64_t table_stride, int32_t count,
                     int32_t max_pages, int32_t* seq_lens, const int32_t* parents, const int32_t* children,
                     const int32_t* fresh, int32_t forks, void* stream) {
  Ranges all;
  if (!pages_ok(pages, all) || !table_ok(block_table, table_stride, count, max_pages)) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (forks < 0 || forks > kKvMaxBatch) return FP8BQ_ERR_INVALID_ARGUMENT;
  if (forks == 0 || count == 0) return FP8BQ_OK;
  if (!seq_lens || !parents || !children || !fresh || !kv_aligned(seq_lens, 4) || !kv_aligned(parents, 4) ||
      !kv_aligned(children, 4) || !kv_aligned(fresh, 4)) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const uint64_t n = 4 * static_cast<uint64_t>(forks), rows = table_bytes(table_stride, count, max_pages);
  const uint64_t lens = 4 * static_cast<uint64_t>(count);
  if (!pages_apart(all, block_table, rows) || !pages_apart(all, seq_lens, lens) ||
      (rows > 0 && overlap(block_table, rows, seq_lens, lens))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  for (const int32_t* x : {parents, children, fresh}) {
    if (!pages_apart(all, x, n) || (rows > 0 && overlap(block_table, rows, x, n)) || overlap(seq_lens, lens, x, n)) {
      return FP8BQ_ERR_INVALID_ARGUMENT;
    }
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  fp8bq::ForkBatch f{block_table, seq_lens, parents, children, fresh, table_stride, count, max_pages, forks};
  hipStream_t st = static_cast<hipStream_t>(stream);
  // Whatever the order of launches, copies read the parents' rows, which forks leave alone.
  for_page_lists(*pages, [&](const fp8bq::PageList& l) {
    const int32_t most = static_cast<int32_t>(kMaxGrid / l.chunks);   // forks of a launch
    for (int32_t at = 0; at < forks; at += most) {
      f.parents = parents + at;
      f.children = children + at;
      f.fresh = fresh + at;
      f.forks = std::min(most, forks - at);
      const dim3 grid(static_cast<unsigned>(l.chunks) * static_cast<unsigned>(f.forks),
                      static_cast<unsigned>(l.large + 1 + (l.tables ? 1 : 0)));
      hipLaunchKernelGGL(fp8bq::cache_fork, grid, dim3(fp8bq::kThreads), 0, st, l, f);
    }
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

size_t fp8bq_cache_compact_workspace_bytes(int64_t num_pages) {
  if (num_pages < 1 || num_pages > fp8bq::kCompactPages) return 0;
  return 4 * (4 + 3 * static_cast<size_t>(num_pages));
}

int fp8bq_cache_compact(const fp8bq_pages* pages, const int32_t* block_table, int64_t table_stride, int32_t count,
                        int32_t max_pages, const int32_t* seq_lens, int32_t* table_out, int64_t out_stride,
                        int32_t* used, void* workspace, size_t workspace_bytes, void* stream) {
  Ranges all;
  if (!pages_ok(pages, all) || !table_ok(block_table, table_stride, count, max_pages) ||
      !table_ok(table_out, out_stride, count, max_pages) || pages->num_pages > fp8bq::kCompactPages) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  if (!used || !kv_aligned(used, 4) || (count > 0 && (!seq_lens || !kv_aligned(seq_lens, 4)))) {
    return FP8BQ_ERR_INVALID_ARGUMENT;
  }
  const size_t need = fp8bq_cache_compact_workspace_bytes(pages->num_pages);
  if (workspace == nullptr || workspace_bytes < need || !kv_aligned(workspace, 16)) return FP8BQ_ERR_WORKSPACE;
  const uint64_t in = table_bytes(table_stride, count, max_pages), out = table_bytes(out_stride, count, max_pages);
  const uint64_t lens = 4 * static_cast<uint64_t>(count);
  const bool in_place = table_out == block_table && (count <= 1 || out_stride == table_stride);
  struct {
    const void* p;
    uint64_t bytes;
  } const list[5] = {{block_table, in}, {seq_lens, lens}, {table_out, out}, {used, 4}, {workspace, need}};
  for (int i = 0; i < 5; ++i) {
    if (!pages_apart(all, list[i].p, list[i].bytes)) return FP8BQ_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j) {
      // the table and the lengths are read only, and may share what they like
      if (i < 2 || list[i].bytes == 0 || list[j].bytes == 0 || (i == 2 && j == 0 && in_place)) continue;
      if (overlap(list[i].p, list[i].bytes, list[j].p, list[j].bytes)) return FP8BQ_ERR_INVALID_ARGUMENT;
    }
  }
  const int rc = device_check();
  if (rc != FP8BQ_OK) return rc;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const int64_t n = pages->num_pages;
  const fp8bq::CompactBatch f{block_table, seq_lens, table_out, used,         ws,    ws + 4,
                              ws + 4 + n,  ws + 4 + 2 * n, table_stride, out_stride, count, max_pages};
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(fp8bq::cache_compact_plan, dim3(1), dim3(fp8bq::kCompactThreads), 0, st, f,
                     static_cast<int32_t>(n), kv_log2_page(pages->page_size));
  for_page_lists(*pages, [&](const fp8bq::PageList& l) {
    const unsigned kinds = static_cast<unsigned>(l.large + 1 + (l.tables ? 1 : 0));
    // as many workgroups as the chip holds, few times over
    const unsigned each = static_cast<unsigned>(std::max<int64_t>(64, 8192 / kinds));
    hipLaunchKernelGGL(fp8bq::cache_compact_move, dim3(each, kinds), dim3(fp8bq::kThreads), 0, st, l, f);
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8BQ_OK : hip_failed(e);
}

}  // extern "C"
