// Device code for the pages of caches (gfx950): forking sequences and moving
// the pages in use to the front.
#pragma once

#include "kv_kernels.hpp"

namespace fp8bq {

// The buffers of a call, `large` ones first: pages of 16-byte words, copied
// kPageChunk bytes to a workgroup; the others, per-page scales and pages that
// are no such words, a wave each, by 4-byte words.
constexpr int kPageBuffers = 256;
constexpr int kPageChunk = 16384;
struct PageList {
  uint8_t* p[kPageBuffers];
  uint32_t bytes[kPageBuffers];   // of a page
  int32_t large, count;
  int32_t chunks;                 // of the largest page
  int32_t pages, log_s;
  int32_t tables;                 // whether this launch writes the tables
};

// One chunk of page `from` to page `to`; all loads before the stores.
__device__ __forceinline__ void copy_chunk(uint8_t* base, uint32_t bytes, int32_t chunk, int32_t from, int32_t to) {
  constexpr int kN = kPageChunk / 16 / kThreads;
  const int64_t at = (int64_t)chunk * kPageChunk;
  if (at >= bytes) return;
  const int32_t words = (int32_t)min((int64_t)kPageChunk, (int64_t)bytes - at) / 16;
  const u32x4* src = (const u32x4*)(base + (int64_t)from * bytes + at);
  u32x4* dst = (u32x4*)(base + (int64_t)to * bytes + at);
  u32x4 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int32_t w = threadIdx.x + i * kThreads;
    if (w < words) x[i] = src[w];
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int32_t w = threadIdx.x + i * kThreads;
    if (w < words) __builtin_nontemporal_store(x[i], &dst[w]);
  }
}

// The small buffers of a page, a wave each.
__device__ __forceinline__ void copy_small(const PageList& l, int32_t from, int32_t to) {
  const int32_t lane = threadIdx.x & 63;
  for (int32_t i = l.large + (threadIdx.x >> 6); i < l.count; i += kThreads / 64) {
    const uint32_t bytes = l.bytes[i];
    const uint32_t* src = (const uint32_t*)(l.p[i] + (int64_t)from * bytes);
    uint32_t* dst = (uint32_t*)(l.p[i] + (int64_t)to * bytes);
    for (uint32_t w = lane; w < bytes / 4; w += 64) dst[w] = src[w];
  }
}

struct ForkBatch {
  int32_t* table;
  int32_t* lens;
  const int32_t* parents;
  const int32_t* children;
  const int32_t* fresh;    // a page for each fork
  int64_t stride;
  int32_t count, max_pages, forks;
};

// A fork shares its parent's whole pages; a last page that is partly filled is
// copied, because both sequences go on writing into it.  Grid: x is (chunk,
// fork), so that forks of one parent, whose page is read for all of them, run
// next to each other; y a large buffer, or all small ones, or the tables.
// Bound by memory: 480 forks of 8 layers of keys and values, 520 MB, 107 us, 4.9
// TB/s, as a copy; few forks by the launch and the chain length, table, page (8
// us for 4 forks in 81 buffers).
__global__ __launch_bounds__(kThreads) void cache_fork(PageList l, ForkBatch f) {
  const int32_t chunk = blockIdx.x / f.forks, i = blockIdx.x - chunk * f.forks;
  const int32_t y = blockIdx.y;
  if (y >= l.large && chunk > 0) return;
  const int32_t a = f.parents[i], b = f.children[i];
  if (a < 0 || a >= f.count || b < 0 || b >= f.count || a == b) return;
  const int32_t len = max(f.lens[a], 0), S = 1 << l.log_s;
  const int32_t whole = min(len >> l.log_s, f.max_pages);   // pages that are shared
  const bool part = (len & (S - 1)) != 0 && whole < f.max_pages;
  int32_t to = f.fresh[i];
  if (to < 0 || to >= l.pages) to = -1;
  if (y == l.large + 1) {
    const int32_t* from = f.table + (int64_t)a * f.stride;
    int32_t* row = f.table + (int64_t)b * f.stride;
    for (int32_t j = threadIdx.x; j < f.max_pages; j += kThreads) {
      const int32_t pg = j <= whole ? from[j] : -1;
      const bool copied = j == whole && part && pg >= 0 && pg < l.pages;
      row[j] = j < whole ? pg : (copied ? to : -1);
    }
    if (threadIdx.x == 0) f.lens[b] = len;
    return;
  }
  if (!part || to < 0) return;
  const int32_t from = f.table[(int64_t)a * f.stride + whole];
  if (from < 0 || from >= l.pages || from == to) return;
  if (y < l.large) {
    copy_chunk(l.p[y], l.bytes[y], chunk, from, to);
  } else {
    copy_small(l, from, to);
  }
}

struct CompactBatch {
  const int32_t* table;
  const int32_t* lens;
  int32_t* out;            // [count, max_pages], rows out_stride apart; may be the table
  int32_t* used;           // [1]
  int32_t* moves;          // workspace: how many pages move,
  int32_t* holes;          //   to where,
  int32_t* movers;         //   from where,
  int32_t* name;           //   and the new number of each page in use
  int64_t stride, out_stride;
  int32_t count, max_pages;
};

constexpr int kCompactThreads = 1024;
constexpr int kCompactPages = 1 << 20;   // a bit each in LDS

// Which pages are in use, and where those behind the first `used` go: the k-th
// of them to the k-th free one before.  One workgroup, which marks pages in
// LDS: nothing to clear beforehand, no second launch in between.  Bound by its
// chain of round trips, 7 to 8 us for tables of some thousand entries.
__global__ __launch_bounds__(kCompactThreads) void cache_compact_plan(CompactBatch f, int32_t pages, int32_t log_s) {
  __shared__ uint32_t bits[kCompactPages / 32];
  __shared__ int32_t sums[kCompactThreads / 64], total_before;
  const int32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, S = 1 << log_s;
  const int32_t words = (pages + 31) / 32;
  for (int32_t i = tid; i < words; i += kCompactThreads) bits[i] = 0;
  __syncthreads();
  // a wave takes 64 lengths at a time, then eight rows at a time
  constexpr int kRows = 8;
  for (int32_t b0 = wave * 64; b0 < f.count; b0 += kCompactThreads) {
    int32_t n = 0;
    if (b0 + lane < f.count) {
      n = (int32_t)min(((int64_t)max(f.lens[b0 + lane], 0) + S - 1) >> log_s, (int64_t)f.max_pages);
    }
    uint64_t rest = __ballot(n > 0);
    while (rest != 0) {
      int32_t at[kRows], of[kRows], most = 0;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        at[r] = rest != 0 ? __ffsll((unsigned long long)rest) - 1 : 0;
        of[r] = rest != 0 ? lane_of(n, at[r]) : 0;
        rest &= rest - 1;
        most = max(most, of[r]);
      }
      for (int32_t j = lane; j < most; j += 64) {
        int32_t pg[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          pg[r] = j < of[r] ? f.table[(int64_t)(b0 + at[r]) * f.stride + j] : -1;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (pg[r] >= 0 && pg[r] < pages) atomicOr(&bits[pg[r] >> 5], 1u << (pg[r] & 31));
        }
      }
    }
  }
  __syncthreads();
  // Each thread's words, and the pages in use before them.
  const int32_t each = (words + kCompactThreads - 1) / kCompactThreads;
  const int32_t w0 = min(tid * each, words), w1 = min(w0 + each, words);
  int32_t mine = 0;
  for (int32_t w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int32_t sum = wave_scan(mine);
  if (lane == 63) sums[wave] = sum;
  __syncthreads();
  int32_t used = 0, before = sum - mine;
  for (int32_t w = 0; w < kCompactThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    used += sums[w];
  }
  // pages in use below number `used`
  int32_t seen = before;
  for (int32_t w = w0; w < w1; ++w) {
    if (used >= 32 * w && used < 32 * w + 32) total_before = seen + __popc(bits[w] & ((1u << (used & 31)) - 1));
    seen += __popc(bits[w]);
  }
  if (tid == 0 && used >= 32 * words) total_before = used;
  __syncthreads();
  const int32_t front = total_before, moves = used - front;
  for (int32_t w = w0; w < w1; ++w) {
    const uint32_t set = bits[w];
    const int32_t p0 = 32 * w, here = before;   // in use before this word
    before += __popc(set);
    if (p0 < used) {
      uint32_t free = ~set;
      if (used - p0 < 32) free &= (1u << (used - p0)) - 1;
      while (free != 0) {
        const int32_t x = __ffs(free) - 1;
        free &= free - 1;
        f.holes[p0 + x - here - __popc(set & ((1u << x) - 1))] = p0 + x;
      }
    }
    if (p0 + 32 > used) {
      uint32_t late = set;
      if (used > p0) late &= ~((1u << (used - p0)) - 1);
      while (late != 0) {
        const int32_t x = __ffs(late) - 1;
        late &= late - 1;
        const int32_t k = here + __popc(set & ((1u << x) - 1)) - front;
        f.movers[k] = p0 + x;
        f.name[p0 + x] = k;
      }
    }
  }
  if (tid == 0) {
    *f.used = used;
    *f.moves = moves;
  }
}

// Grid: x strides over (chunk, move), whose number only the device knows; y a
// large buffer, or all small ones, or the table.  Bound by memory: 8 layers of
// latents, 520 MB, 98 us.
__global__ __launch_bounds__(kThreads) void cache_compact_move(PageList l, CompactBatch f) {
  const int32_t y = blockIdx.y, moves = *f.moves;
  if (y == l.large + 1) {
    const int32_t used = *f.used, S = 1 << l.log_s;
    for (int32_t b = blockIdx.x; b < f.count; b += gridDim.x) {
      const int32_t n = (int32_t)min(((int64_t)max(f.lens[b], 0) + S - 1) >> l.log_s, (int64_t)f.max_pages);
      for (int32_t j = threadIdx.x; j < f.max_pages; j += kThreads) {
        int32_t pg = j < n ? f.table[(int64_t)b * f.stride + j] : -1;
        if (pg < 0 || pg >= l.pages) pg = -1;
        if (pg >= used) {
          const int32_t k = f.name[pg];
          pg = k >= 0 && k < moves ? f.holes[k] : -1;
        }
        f.out[(int64_t)b * f.out_stride + j] = pg;
      }
    }
    return;
  }
  if (y < l.large) {
    const uint32_t bytes = l.bytes[y];
    const int32_t chunks = (int32_t)((bytes + kPageChunk - 1) / kPageChunk);
    const int64_t items = (int64_t)moves * chunks;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
      const int32_t k = (int32_t)(i / chunks);
      copy_chunk(l.p[y], bytes, (int32_t)(i - (int64_t)k * chunks), f.movers[k], f.holes[k]);
    }
  } else {
    for (int32_t k = blockIdx.x; k < moves; k += gridDim.x) copy_small(l, f.movers[k], f.holes[k]);
  }
}

}  // namespace fp8bq
