// pages_kernel.cuh -- management of the pages of a K/V cache (sm_100a):
// appending rows, trimming, forking, compacting and copying.  Everything is
// decided on the device from the table, the lengths and the reference counts
// there, so the calls need no host copy of them and can be captured.
//
// What bounds it: moved rows are read once and written once, so the wide
// kernels are bound by HBM (600 MB of prompts written in 85 us, 1.25 GB of
// pages compacted in 189 us: 7.0 and 6.6 TB/s, at or above a plain copy's rate);
// the decisions (which page is free, which sequence gets it) are integer prefix
// sums over the sequences and over the reference counts, made by one CTA in a
// kernel before them and bound by L2 latency (6 us for 64 sequences, 9 us for 9400
// pages).  That one CTA reads 16384 counts a step, an append up to the last page it
// needs and a compaction all of them, twice; so in a pool that is nearly full they
// grow with it: a step of 64 sequences, appended and taken back, 8 us at 10000 pages of which
// 95% are in use, 17 at 100000, 48 at 400000; a compaction that moves nothing 7, 30, 107.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace attn {

constexpr int PG_PLAN_THREADS = 1024;   // the deciding kernels: one CTA
constexpr int PG_LIST = 4096;           // free pages kept in shared memory
constexpr int PG_FEW = 4;               // pages one thread hands out to a sequence
constexpr int PG_THREADS = 256;         // the moving kernels
constexpr int PG_ROWS = 64;             // new rows of one (sequence, K/V head) a CTA writes
constexpr int PG_CHUNK = PG_THREADS * 16 * 4;   // bytes of a page a CTA moves at a time
constexpr int STATUS_INVALID = -1;      // matches ATTN_ERR_INVALID_ARG
constexpr int STATUS_NO_PAGES = -6;     // matches ATTN_ERR_NO_PAGES

// The cache as the kernels see it (see attn_pages_t).
struct Pages {
  uint8_t* k;
  uint8_t* v;
  int* table;
  int* lens;
  int* refs;
  int n_pages, H_kv, page_size, page_shift, B, max_pages;
  int row_bytes;            // d * 2
  long long page_bytes;     // H_kv * page_size * d * 2
  int* status;
};

__device__ __forceinline__ void pg_report(const Pages& p, int code) { atomicCAS(p.status, 0, code); }

__device__ __forceinline__ bool pg_valid(const Pages& p, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
}

__device__ __forceinline__ int pg_count(const Pages& p, long long rows) {
  return static_cast<int>((rows + p.page_size - 1) >> p.page_shift);
}

// Exclusive prefix sum over the CTA's PG_PLAN_THREADS threads; `total` is the
// sum.  `part` holds 33 ints of shared memory.
__device__ __forceinline__ int pg_scan(int x, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
    const int own = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    part[lane] = w - own;
    if (lane == 31) part[32] = w;
  }
  __syncthreads();
  total = part[32];
  const int before = part[warp] + s - x;
  __syncthreads();   // the next call writes `part` again
  return before;
}

// Which of the 16 pages from `first` on have no reference (bit u: page first + u).
__device__ __forceinline__ uint32_t pg_zero_bits(const Pages& p, int first) {
  uint32_t bits = 0;
  if (first + 16 <= p.n_pages && (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0) {
    const int4* r4 = reinterpret_cast<const int4*>(p.refs + first);
    int4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] = r4[u];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      bits |= ((r[u].x <= 0 ? 1u : 0u) | (r[u].y <= 0 ? 2u : 0u) | (r[u].z <= 0 ? 4u : 0u) |
               (r[u].w <= 0 ? 8u : 0u)) << (4 * u);
  } else {
    for (int u = 0; u < 16; ++u)
      if (first + u < p.n_pages && p.refs[first + u] <= 0) bits |= 1u << u;
  }
  return bits;
}

// ------------------------------------------------------------ append

// What attn_pages_append's first kernel hands to its second, for each
// sequence: the position of its first new row, the rows it gets, and the page
// copied on write.
struct AppendPlan {
  int* start;
  int* count;
  int* from;      // a shared, partly filled last page, or -1
  int* to;        // its copy
  int* base;      // pages handed out to the sequences before this one
  int* need;
  int* free_list; // the lowest free pages, ascending
};

// One CTA.  A sequence needs a page for every page boundary its new rows
// reach, and one more when its last, partly filled page is also held by
// another sequence (copy on write).  The k-th page needed, in order of the
// sequences, is the k-th lowest page with no reference.  The first sequence
// that cannot be served and every later one that needs pages get none.
__global__ void __launch_bounds__(PG_PLAN_THREADS)
attn_pages_append_plan(const Pages p, const AppendPlan a, const int* counts, int n_new) {
  __shared__ int part[33], list_s[PG_LIST];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  int wanted = 0;
  for (int b0 = 0; b0 < p.B; b0 += PG_PLAN_THREADS) {
    const int b = b0 + t;
    int need = 0;
    if (b < p.B) {
      const int start = p.lens[b];
      int c = counts != nullptr ? counts[b] : n_new;
      int from = -1;
      if (c < 0 || c > n_new || start < 0 || static_cast<long long>(start) + c > cap) {
        pg_report(p, STATUS_INVALID);
        c = 0;
      } else if (c > 0 && (start & (p.page_size - 1)) != 0) {
        const int last = p.table[static_cast<size_t>(b) * p.max_pages + (start >> p.page_shift)];
        const int held = pg_valid(p, last) ? p.refs[last] : 0;
        if (held < 1) {          // no such page, or one that counts as free and may be handed out
          pg_report(p, STATUS_INVALID);
          c = 0;
        } else if (held > 1) {
          from = last;
        }
      }
      if (c > 0)
        need = pg_count(p, static_cast<long long>(start) + c) - pg_count(p, start) + (from >= 0 ? 1 : 0);
      a.start[b] = start;
      a.count[b] = c;
      a.from[b] = from;
      a.need[b] = need;
    }
    int total;
    const int before = pg_scan(need, part, total);
    if (b < p.B) a.base[b] = wanted + before;
    wanted += total;
  }
  // the lowest `wanted` free pages, 16 counts a thread and step; few of them
  // stay in shared memory
  int* list = wanted <= PG_LIST ? list_s : a.free_list;
  int found = 0;
  for (int c0 = 0; found < wanted && c0 < p.n_pages; c0 += PG_PLAN_THREADS * 16) {
    const int first = c0 + t * 16;
    uint32_t free_bits = pg_zero_bits(p, first);
    int total;
    int k = found + pg_scan(__popc(free_bits), part, total);
    for (; free_bits != 0 && k < wanted; free_bits &= free_bits - 1, ++k)
      list[k] = first + __ffs(free_bits) - 1;
    found += total;
  }
  __syncthreads();   // need, base, from and the list are this CTA's own writes
  // hand them out: a thread a sequence, a warp together for those of many pages
  const int lane = t & 31;
  for (int b0 = 0; b0 < p.B; b0 += PG_PLAN_THREADS) {
    const int b = b0 + t;
    int need = 0, base = 0, col0 = 0;
    if (b < p.B) {
      need = a.need[b];
      base = a.base[b];
      const int start = a.start[b], c = a.count[b], from = a.from[b];
      if (need > 0 && static_cast<long long>(base) + need > found) {
        pg_report(p, STATUS_NO_PAGES);
        a.count[b] = 0;
        a.from[b] = -1;
        need = 0;
      } else if (c > 0) {
        p.lens[b] = start + c;
        // column of the first page handed out: the copied one's, or the next free column
        col0 = from >= 0 ? start >> p.page_shift : pg_count(p, start);
        if (from >= 0) {
          a.to[b] = list[base];
          atomicSub(&p.refs[from], 1);
        }
      }
    }
    int* row = p.table + static_cast<size_t>(b) * p.max_pages + col0;
    if (need <= PG_FEW) {
#pragma unroll
      for (int j = 0; j < PG_FEW; ++j)
        if (j < need) {
          const int page = list[base + j];
          row[j] = page;
          p.refs[page] = 1;
        }
    }
    for (uint32_t many = __ballot_sync(0xffffffffu, need > PG_FEW); many != 0; many &= many - 1) {
      const int l = __ffs(many) - 1;
      const int n = __shfl_sync(0xffffffffu, need, l), first = __shfl_sync(0xffffffffu, base, l);
      int* to = reinterpret_cast<int*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), l));
      for (int j = lane; j < n; j += 32) {
        const int page = list[first + j];
        to[j] = page;
        p.refs[page] = 1;
      }
    }
  }
}

// Writes the new rows (blocks [0, n_tiles): PG_ROWS rows of one sequence and
// K/V head each) and copies the pages copied on write (the blocks after them:
// one sequence and K/V head each).  A thread has up to four 16-byte loads of K
// and four of V in flight.
__global__ void __launch_bounds__(PG_THREADS)
attn_pages_append_rows(const Pages p, const AppendPlan a, const uint8_t* k_new, const uint8_t* v_new,
                       int n_new, int row_tiles, long long n_tiles) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int vecs = p.row_bytes >> 4;             // 16-byte vectors of a row: 2, 4, 8 or 16
  const int vshift = 31 - __clz(vecs);
  const long long blk = blockIdx.x;
  if (blk < n_tiles) {
    const int tile = static_cast<int>(blk % row_tiles);
    const long long bh = blk / row_tiles;
    const int h = static_cast<int>(bh % p.H_kv), b = static_cast<int>(bh / p.H_kv);
    const int r0 = tile * PG_ROWS;
    const int c = a.count[b];
    if (r0 >= c) return;
    const int rows = min(PG_ROWS, c - r0), start = a.start[b];
    const int* row = p.table + static_cast<size_t>(b) * p.max_pages;
    const size_t src0 = (static_cast<size_t>(bh) * n_new + r0) * p.row_bytes;
    uint4 x[4], y[4];
    size_t to[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = threadIdx.x + u * PG_THREADS;
      const int r = i >> vshift, col = i & (vecs - 1);
      on[u] = r < rows;
      to[u] = 0;
      if (on[u]) {
        const size_t from = src0 + static_cast<size_t>(r) * p.row_bytes + col * 16;
        x[u] = *reinterpret_cast<const uint4*>(k_new + from);
        y[u] = *reinterpret_cast<const uint4*>(v_new + from);
        const int pos = start + r0 + r;
        const int page = row[pos >> p.page_shift];
        on[u] = pg_valid(p, page);
        to[u] = static_cast<size_t>(page) * p.page_bytes +
                (static_cast<size_t>(h) * p.page_size + (pos & (p.page_size - 1))) * p.row_bytes + col * 16;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (on[u]) {
        *reinterpret_cast<uint4*>(p.k + to[u]) = x[u];
        *reinterpret_cast<uint4*>(p.v + to[u]) = y[u];
      }
    }
    return;
  }
  const long long bh = blk - n_tiles;
  const int h = static_cast<int>(bh % p.H_kv), b = static_cast<int>(bh / p.H_kv);
  if (a.from[b] < 0) return;
  const int n = (a.start[b] & (p.page_size - 1)) * vecs;
  const size_t head = static_cast<size_t>(h) * p.page_size * p.row_bytes;
  const size_t src = static_cast<size_t>(a.from[b]) * p.page_bytes + head;
  const size_t dst = static_cast<size_t>(a.to[b]) * p.page_bytes + head;
  for (int i = threadIdx.x; i < n; i += PG_THREADS) {
    const uint4 x = *reinterpret_cast<const uint4*>(p.k + src + static_cast<size_t>(i) * 16);
    const uint4 y = *reinterpret_cast<const uint4*>(p.v + src + static_cast<size_t>(i) * 16);
    *reinterpret_cast<uint4*>(p.k + dst + static_cast<size_t>(i) * 16) = x;
    *reinterpret_cast<uint4*>(p.v + dst + static_cast<size_t>(i) * 16) = y;
  }
}

// ------------------------------------------------------------ trim

// One CTA a listed row.  Lowering the length with a compare-and-swap gives every
// entry of the list its own interval of pages, so a row that is listed twice ends
// at the smaller length and each of its pages is released once.  A length that
// cannot be right is looked at first and stays as it is, with the row's pages.
__global__ void __launch_bounds__(128)
attn_pages_trim_kernel(const Pages p, const int* rows, const int* new_lens) {
  __shared__ int old_s;
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = blockIdx.x;
  const int b = rows != nullptr ? rows[i] : i;
  const int n = new_lens != nullptr ? new_lens[i] : 0;
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  if (b < 0 || b >= p.B || n < 0) {
    if (threadIdx.x == 0) pg_report(p, STATUS_INVALID);
    return;
  }
  if (threadIdx.x == 0) {
    int old = p.lens[b];
    while (old > n && old <= cap) {
      const int seen = atomicCAS(&p.lens[b], old, n);
      if (seen == old) break;
      old = seen;              // another entry of the list lowered it
    }
    old_s = old;
  }
  __syncthreads();
  const int old = old_s;
  if (old < 0 || old > cap) {
    if (threadIdx.x == 0) pg_report(p, STATUS_INVALID);
    return;
  }
  int* row = p.table + static_cast<size_t>(b) * p.max_pages;
  const int end = pg_count(p, old);
  for (int c = pg_count(p, n) + threadIdx.x; c < end; c += blockDim.x) {
    const int page = row[c];
    row[c] = -1;
    if (!pg_valid(p, page)) {
      pg_report(p, STATUS_INVALID);
    } else if (atomicSub(&p.refs[page], 1) <= 0) {
      atomicAdd(&p.refs[page], 1);   // it had no reference: the counts do not fit the table
      pg_report(p, STATUS_INVALID);
    }
  }
}

// ------------------------------------------------------------ fork

// One CTA a fork: the child's row becomes the parent's, and every page gains
// a reference.  A fork whose child is listed earlier, whose parent is listed
// as a child, or whose child is not empty is skipped, so no CTA reads a row
// that another one writes.
__global__ void __launch_bounds__(128)
attn_pages_fork_kernel(const Pages p, const int* parents, const int* children, int n) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = blockIdx.x;
  const int from = parents[i], to = children[i];
  bool bad = from < 0 || from >= p.B || to < 0 || to >= p.B;
  for (int j = threadIdx.x; j < n && !bad; j += blockDim.x) {
    const int c = children[j];
    bad = c == from || (c == to && j < i);
  }
  bad = __syncthreads_or(bad);
  int len = 0;
  if (!bad) {
    len = p.lens[from];
    bad = p.lens[to] != 0 || len < 0 || len > (static_cast<long long>(p.max_pages) << p.page_shift);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) pg_report(p, STATUS_INVALID);
    return;
  }
  const int* src = p.table + static_cast<size_t>(from) * p.max_pages;
  int* dst = p.table + static_cast<size_t>(to) * p.max_pages;
  const int have = pg_count(p, len);
  for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
    const int page = c < have ? src[c] : -1;
    dst[c] = page;
    if (c < have) {
      if (pg_valid(p, page)) atomicAdd(&p.refs[page], 1);
      else pg_report(p, STATUS_INVALID);
    }
  }
  if (threadIdx.x == 0) p.lens[to] = len;
}

// ------------------------------------------------------------ compact

// What attn_pages_compact's first kernel hands to its second.
struct CompactPlan {
  int* n_moves;   // [1]
  int* n_live;    // [1]
  int* src;       // live pages at or past n_live, ascending
  int* dst;       // free pages below n_live, ascending
  int* map;       // [n_pages] a page's new index
};

// One CTA: counts the live pages, then ranks the live pages past that count
// and the free ones below it; both are as many, and the k-th moves to the k-th.
__global__ void __launch_bounds__(PG_PLAN_THREADS)
attn_pages_compact_plan(const Pages p, const CompactPlan a, int* n_live_out) {
  __shared__ int part[33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  int live = 0;
  for (int first = t * 16; first < p.n_pages; first += PG_PLAN_THREADS * 16)
    live += min(16, p.n_pages - first) - __popc(pg_zero_bits(p, first));
  for (int page = t; page < p.n_pages; page += PG_PLAN_THREADS) a.map[page] = page;
  int n_live;
  pg_scan(live, part, n_live);
  int moved = 0, filled = 0;
  for (int c0 = 0; c0 < p.n_pages; c0 += PG_PLAN_THREADS * 16) {
    const int first = c0 + t * 16;
    const int n = max(0, min(16, p.n_pages - first));
    const uint32_t all = (1u << n) - 1u, zero = pg_zero_bits(p, first);
    const int below = max(0, min(n, n_live - first));              // pages of these below n_live
    uint32_t dst = zero & ((1u << below) - 1u), src = ~zero & all & ~((1u << below) - 1u);
    // at most 16 a thread and 16384 a step: both counts fit one 32-bit scan
    int total;
    const int both = pg_scan(__popc(src) << 16 | __popc(dst), part, total);
    int s = moved + (both >> 16), d = filled + (both & 0xffff);
    for (; src != 0; src &= src - 1) a.src[s++] = first + __ffs(src) - 1;
    for (; dst != 0; dst &= dst - 1) a.dst[d++] = first + __ffs(dst) - 1;
    moved += total >> 16;
    filled += total & 0xffff;
  }
  __syncthreads();
  for (int i = t; i < moved; i += PG_PLAN_THREADS) a.map[a.src[i]] = a.dst[i];
  if (t == 0) {
    *a.n_moves = moved;
    *a.n_live = n_live;
    if (n_live_out != nullptr) *n_live_out = n_live;
  }
}

// Copies chunk `c` of page `src` to page `dst` (K chunks, then V chunks).
__device__ __forceinline__ void pg_move_chunk(const Pages& p, int src, int dst, int c, int chunks) {
  uint8_t* base = c < chunks ? p.k : p.v;
  const long long off = static_cast<long long>(c < chunks ? c : c - chunks) * PG_CHUNK;
  const uint8_t* from = base + static_cast<size_t>(src) * p.page_bytes + off;
  uint8_t* to = base + static_cast<size_t>(dst) * p.page_bytes + off;
  const long long left = p.page_bytes - off;
  uint4 x[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int at = (threadIdx.x + u * PG_THREADS) * 16;
    if (at < left) x[u] = __ldcs(reinterpret_cast<const uint4*>(from + at));
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int at = (threadIdx.x + u * PG_THREADS) * 16;
    if (at < left) __stcs(reinterpret_cast<uint4*>(to + at), x[u]);
  }
}

// Pages smaller than half a chunk: moves `first`, first + 1, ... of the lists, as many
// as fit a chunk (`per`), K and V.  Entries with a source below 0 are skipped; a bad
// one is reported (the compaction's plan has neither).
__device__ __forceinline__ void pg_move_small(const Pages& p, const int* src, const int* dst, long long first,
                                              long long n, int per) {
  const int pv = static_cast<int>(p.page_bytes >> 4);
  uint4 x[4];
  uint4* to[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int v = threadIdx.x + u * PG_THREADS;
    const int m = v / (2 * pv), in = v - m * 2 * pv;
    to[u] = nullptr;
    if (m < per && first + m < n) {
      const int s = src[first + m], d = dst[first + m];
      if (s >= 0 && pg_valid(p, s) && pg_valid(p, d)) {
        uint8_t* base = in < pv ? p.k : p.v;
        const int off = in < pv ? in : in - pv;
        x[u] = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<size_t>(s) * p.page_bytes) + off);
        to[u] = reinterpret_cast<uint4*>(base + static_cast<size_t>(d) * p.page_bytes) + off;
      } else if (s >= 0 && in == 0) {
        pg_report(p, STATUS_INVALID);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (to[u] != nullptr) __stcs(to[u], x[u]);
}

// Moves a CTA's chunk holds: 0 where a page has half a chunk or more, and its
// chunks are moved one by one.  Several small pages at once keep the loads in
// flight that one of 2 KB would not (18000 such pages, 4300 moved: 26.2 us a call one at a time, 19.5 so).
__host__ __device__ inline int pg_per_chunk(long long page_bytes) {
  return static_cast<int>(page_bytes * 2 <= PG_CHUNK ? PG_CHUNK / (2 * page_bytes) : 0);
}

// Moves the pages of the plan and writes the renumbered table and counts.
// The sources stay as they are (a source is never a destination), so the old
// table still reads the same rows until its pages are handed out again.
__global__ void __launch_bounds__(PG_THREADS)
attn_pages_compact_move(const Pages p, const CompactPlan a, int* table_out, int* refs_out,
                        int chunks) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int n_moves = *a.n_moves, n_live = *a.n_live;
  const long long tid = static_cast<long long>(blockIdx.x) * PG_THREADS + threadIdx.x;
  const long long threads = static_cast<long long>(gridDim.x) * PG_THREADS;
  for (long long i = tid; i < static_cast<long long>(p.B) * p.max_pages; i += threads) {
    const int page = p.table[i];
    table_out[i] = pg_valid(p, page) ? a.map[page] : page;
  }
  if (refs_out != p.refs) {
    for (long long i = tid; i < p.n_pages; i += threads) {
      const int r = p.refs[i];
      // moved pages' old and new places are written below
      if (i < n_live ? r > 0 : r <= 0) refs_out[i] = i < n_live ? r : 0;
    }
  }
  for (long long i = tid; i < n_moves; i += threads) {
    const int src = a.src[i], dst = a.dst[i];
    const int r = p.refs[src];
    refs_out[dst] = r;
    refs_out[src] = 0;
  }
  const int per = pg_per_chunk(p.page_bytes);
  if (per > 0) {
    for (long long m = static_cast<long long>(blockIdx.x) * per; m < n_moves; m += static_cast<long long>(gridDim.x) * per)
      pg_move_small(p, a.src, a.dst, m, n_moves, per);
    return;
  }
  const long long work = static_cast<long long>(n_moves) * 2 * chunks;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const long long i = w / (2 * chunks);
    pg_move_chunk(p, a.src[i], a.dst[i], static_cast<int>(w - i * 2 * chunks), chunks);
  }
}

// ------------------------------------------------------------ copy

__global__ void __launch_bounds__(PG_THREADS)
attn_pages_copy_kernel(const Pages p, const int* src, const int* dst, int n, int chunks) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int per = pg_per_chunk(p.page_bytes);
  if (per > 0) {
    for (long long m = static_cast<long long>(blockIdx.x) * per; m < n; m += static_cast<long long>(gridDim.x) * per)
      pg_move_small(p, src, dst, m, n, per);
    return;
  }
  const long long work = static_cast<long long>(n) * 2 * chunks;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const long long i = w / (2 * chunks);
    const int s = src[i], d = dst[i];
    if (s < 0) continue;               // an unused entry of the list
    if (!pg_valid(p, s) || !pg_valid(p, d)) {
      if (threadIdx.x == 0) pg_report(p, STATUS_INVALID);
      continue;
    }
    if (s != d) pg_move_chunk(p, s, d, static_cast<int>(w - i * 2 * chunks), chunks);
  }
}

}  // namespace attn
