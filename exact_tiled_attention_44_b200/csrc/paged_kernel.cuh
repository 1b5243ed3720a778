// paged_kernel.cuh -- a decoding step over a K/V cache of pages (sm_100a).
//
// What it computes: the N_q new query rows of every sequence b and query head
// attend to the lens[b] positions that the table lists for the sequence, under
// the forward's mask rule with row i at position lens[b] - N_q + i ("USAAIO
// Lesson 91", slide 31: every decoding step re-reads the whole cache; slide
// 32: the query heads of a group share one K/V head):
//     O = softmax(scale q K^T) V,   LSE = ln sum exp(scale q.k).
//
// Work split ("Building a FlashAttention-style tiled self-attention block in
// pure NumPy", "Extending It", item 6: split the sequence, then reduce the
// partial outputs): a group is one sequence, one K/V head and up to m of
// its (H / H_kv) * N_q query rows.  The kept 64-position tiles of all groups
// are laid end to end, by the lengths on the device, and cut into equal
// ranges, one for each CTA, so ragged lengths leave no CTA idle.  The part of
// a range inside one group is a run.  A group covered by one run is written
// out directly; the others leave (O_s, LSE_s) for every run in the workspace,
// and a second kernel merges them in the order of the runs:
//     LSE = ln sum_s exp(LSE_s),   O = sum_s exp(LSE_s - LSE) O_s.
//
// A prefix that the batch shares is one more set of groups, whose rows are
// the rows of all sequences and whose tiles come from the shared table; its
// partial results are merged with each sequence's own.
#pragma once

#include "attn_kernel.cuh"

namespace attn {

constexpr int PD_TILE = 64;             // positions of a tile
constexpr int PD_SLICE = 16;            // positions of a tile that a warp attends
constexpr int PD_WARPS = PD_TILE / PD_SLICE;
constexpr int PD_THREADS = 32 * (PD_WARPS + 1);   // and a warp that loads
constexpr int PD_MERGE = 128;           // threads of the merging kernels
constexpr int PD_LENS = 512;            // lengths kept in shared memory

struct PdParams {
  const void* q;
  void* o;
  float* lse;
  float* part_o;        // [2 * gridDim.x][m][D] results of runs of split groups
  float* part_lse;      // [2 * gridDim.x][m]
  float* own_o;         // with a shared prefix: [groups][m][D] results of groups with one run
  float* own_lse;       // [groups][m]
  const int* table;     // [B][max_pages], or the shared table
  const int* lens;
  int* status;
  unsigned long long watchdog_ns;
  int B, H, H_kv, N_q;
  int n_pages, max_pages, page_shift;
  int causal, window, n_sink;
  float scale_log2;     // scale * log2(e)
  int G;                // H / H_kv
  int R;                // G * N_q query rows of a sequence and K/V head
  int m;                // query rows of a group: 8 or 16, or (paged_tc_kernel.cuh) 128 or 256
  int tile_shift;       // log2 of the positions of a tile
  int row_tiles;        // groups of a sequence and K/V head (prefix: of a K/V head)
  int shared_tiles;     // whole tiles of the shared prefix
  int prefix;           // this launch attends the shared prefix
  int ranges;           // CTAs of the attending kernel
  int weight;           // prefix: time of a tile on one SM (see pd_prefix_ranges),
  int own_weight;       //   that of the sequences' own launch,
  int own_groups;       //   its groups a sequence
  int own_tile_shift;   //   and its tiles
  int own_shared_tiles; //   in the prefix
  int withhold_loads;   // test hook: no slice is loaded, so every wait runs out
};

// Shared memory of head dimension D and 8 NT rows a group: a ring of NST
// tiles (the slices of K, then those of V), a run's query rows, the exchange
// buffer of the epilogue, row statistics, the first sequences' lengths,
// barriers.
template <int D, int NT>
struct PdGeo {
  static_assert(D == 64 || D == 128, "the paged decoding kernel supports d = 64 and 128");
  static constexpr int M = 8 * NT;
  static constexpr int NST = D == 128 ? 3 : 6;
  static constexpr int NCH = D / 64;                    // 64-column chunks, 128-byte swizzle
  static constexpr int CHUNK_BYTES = PD_SLICE * 128;
  static constexpr int SLICE_BYTES = NCH * CHUNK_BYTES; // K (or V) of a slice
  static constexpr int HALF_BYTES = PD_WARPS * SLICE_BYTES;
  static constexpr int STAGE_BYTES = 2 * HALF_BYTES;
  static constexpr int RING_BYTES = NST * STAGE_BYTES;
  static constexpr int Q_LD = D * 2 + 16;               // bytes from row to row: no bank conflicts
  static constexpr int Q_OFF = RING_BYTES;
  static constexpr int X_ROWS = 512 / D;                // rows combined at a time
  static constexpr int X_LD = D + 4;                    // floats from row to row
  static constexpr int X_OFF = Q_OFF + M * Q_LD;        // float [PD_WARPS][X_ROWS][X_LD]
  static constexpr int STAT_OFF = X_OFF + PD_WARPS * X_ROWS * X_LD * 4;   // float [3][PD_WARPS][M]
  static constexpr int LENS_OFF = STAT_OFF + 3 * PD_WARPS * M * 4;
  static constexpr int BAR_OFF = LENS_OFF + PD_LENS * 4;   // full [NST], empty [NST], rows full, rows empty
  static constexpr int SCAN_OFF = BAR_OFF + (2 * NST + 2) * 8;   // int [PD_THREADS / 32 + 2]
  static constexpr int ABORT_OFF = SCAN_OFF + (PD_THREADS / 32 + 2) * 4;
  static constexpr int SMEM_BYTES = ABORT_OFF + 8;
  // two CTAs on an SM
  static_assert(2 * (SMEM_BYTES + 2048) <= 233472, "shared memory budget");
};

// ------------------------------------------------------------ work split

// The positions a sequence's rows may keep: tiles [0, sb) and [w0, ...) of len.
struct PdSeq {
  int len;      // positions (clamped to the table)
  int sb, w0;   // tiles [0, sb), then [w0, ...)
  int tiles;    // 0: nothing is kept (of the sequence's own positions)
};

// Lengths, table and query rows are read through L2: a launch behind a shared
// prefix, and the merging kernels before their wait, read them without a dependency
// wait of their own, so no line that L1 kept from before may serve them.
__device__ __forceinline__ int pd_len_of(const PdParams& p, int b) {
  return min(max(__ldcg(p.lens + b), 0), p.max_pages << p.page_shift);
}

// The same, from the lengths kept in shared memory (if there are any).
__device__ __forceinline__ int pd_len_of(const PdParams& p, int b, const int* lens_s) {
  return lens_s != nullptr && b < PD_LENS ? lens_s[b] : pd_len_of(p, b);
}

__device__ __forceinline__ PdSeq pd_seq(const PdParams& p, int len) {
  PdSeq s;
  if (p.prefix) {
    s.len = p.shared_tiles << p.tile_shift;
    s.sb = 0;
    s.w0 = 0;
    s.tiles = p.shared_tiles;
    return s;
  }
  s.len = len;
  const int tile = 1 << p.tile_shift;
  const int nt = (len + tile - 1) >> p.tile_shift;
  s.sb = 0;
  s.w0 = p.shared_tiles;
  if (p.window > 0) {
    const int first = len - p.N_q - p.window + 1;      // both below 2^30 + 1024
    s.sb = min((min(p.n_sink, len) + tile - 1) >> p.tile_shift, nt);
    s.w0 = max(first > 0 ? first >> p.tile_shift : 0, s.sb);
  }
  s.tiles = s.sb + max(0, nt - s.w0);
  return s;
}

// Lengths that do not fit the table are reported once, by one warp.
__device__ __forceinline__ void pd_report_lens(const PdParams& p) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) {
    const int n = __ldcg(p.lens + b);
    if (n < 0 || n > (p.max_pages << p.page_shift)) atomicCAS(p.status, 0, -1);
  }
}

// F tiles in `n` ranges: the first `more` ranges have one tile more than the
// other `each`.  With k > 0 every group of `tiles` tiles is cut into k ranges of
// its own instead.
struct PdCut {
  int n, each, more;
  int k, tiles;
};

__device__ __forceinline__ PdCut pd_cut(int F, int n) {
  PdCut c;
  c.n = min(F, n);
  c.each = F / max(c.n, 1);
  c.more = F - c.each * c.n;
  c.k = 0;
  c.tiles = 0;
  return c;
}

// A prefix's groups are all of one length, so where there are at least as many
// ranges (a run that begins in mid-range costs 18000 cycles, four tiles) no
// range holds parts of two.
__device__ __forceinline__ PdCut pd_cut_prefix(const PdParams& pre, int n) {
  const int groups = pre.H_kv * pre.row_tiles;
  PdCut c = pd_cut(groups * pre.shared_tiles, n);
  if (pre.m > 16 && n >= groups) {
    c.k = min(n / groups, pre.shared_tiles);
    c.tiles = pre.shared_tiles;
    c.n = c.k * groups;
  }
  return c;
}

__device__ __forceinline__ int pd_start(const PdCut& c, int i) {
  if (c.k > 0) {
    const int g = i / c.k;
    return g * c.tiles + (i - g * c.k) * c.tiles / c.k;
  }
  return i * c.each + min(i, c.more);
}

// The range that holds tile f.
__device__ __forceinline__ int pd_range_of(const PdCut& c, int f) {
  if (c.k > 0) {
    const int g = f / c.tiles;
    return g * c.k + ((f - g * c.tiles + 1) * c.k - 1) / c.tiles;
  }
  const int t = c.more * (c.each + 1);
  return f < t ? f / (c.each + 1) : c.more + (f - t) / c.each;
}

// The prefix is bound by the tensor cores and exponentials, the sequences' own
// positions by HBM, so the two launches share the SMs: the prefix takes the
// part of them that its work is of all (`own`: tiles of the other launch's
// groups), the other launch's CTAs the rest.  Weights: see paged_form.  A short
// prefix gets a quarter of the SMs even so: on fewer its row tiles come one after
// another, and the launch waits for them (256 rows over 2048 positions beside 64
// sequences of up to 8000, d = 64: 1 SM 184 us, 8 141, 18 136, 37 134, 74 136, all 143; d = 128 270,
// 222, 215, 214, 219, 228).  A prefix of few rows is bound by HBM itself and takes all.
__device__ __forceinline__ int pd_prefix_ranges(const PdParams& pre, int own) {
  if (pre.m <= 16) return pre.ranges;
  const long long a = static_cast<long long>(pre.shared_tiles) * pre.H_kv * pre.row_tiles * pre.weight;
  const long long b = static_cast<long long>(own) * pre.own_weight;
  return max(static_cast<int>(pre.ranges * a / (a + b)), pre.ranges / 4);
}

// Tiles of a sequence's own positions in the other launch.
__device__ __forceinline__ int pd_own_tiles(const PdParams& pre, int len) {
  return max(0, ((len + (1 << pre.own_tile_shift) - 1) >> pre.own_tile_shift) - pre.own_shared_tiles);
}

// The sum of x over the CTA's THREADS threads before this one, and of all.
// `part` holds THREADS / 32 + 2 ints of shared memory.
template <int THREADS>
__device__ __forceinline__ int pd_scan(int x, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int y = part[w];
    before += w < warp ? y : 0;
    total += y;
  }
  __syncthreads();
  return before + s - x;
}

// The tiles of all sequences (of one group of each) in order.  Every thread
// holds one of the first THREADS sequences; beyond them, the sums are made
// again when a tile is located.
struct PdSum {
  int total;
  int before, tiles;    // of sequence threadIdx.x
  int ranges;           // ranges of the tile space
};

// Also keeps the first PD_LENS lengths in shared memory when `lens_s` is given.
template <int THREADS>
__device__ __forceinline__ PdSum pd_sum(const PdParams& p, int* part, int* lens_s) {
  PdSum s;
  s.total = p.shared_tiles;
  s.before = 0;
  s.tiles = 0;
  s.ranges = p.ranges;
  int rest = 0, own = 0;
  for (int b = threadIdx.x; b < p.B; b += THREADS) {
    const int len = pd_len_of(p, b);
    if (lens_s != nullptr && b < PD_LENS) lens_s[b] = len;
    const int tiles = pd_seq(p, len).tiles;
    if (b < THREADS) s.tiles = tiles;
    else rest += tiles;
    if (p.prefix) own += pd_own_tiles(p, len);
  }
  if (p.prefix) {
    int total;
    pd_scan<THREADS>(own, part, total);
    s.ranges = pd_prefix_ranges(p, total * p.own_groups);
    return s;
  }
  s.before = pd_scan<THREADS>(s.tiles, part, s.total);
  if (p.B > THREADS) {
    int more;
    pd_scan<THREADS>(rest, part, more);
    s.total += more;
  }
  return s;
}

// The sequence that holds tile u of the sum of the sequences' tiles, and the
// tiles before it.  The last two ints of `part` pass them on.
template <int THREADS>
__device__ __forceinline__ void pd_locate(const PdParams& p, const PdSum& sum, int u, int* part, int& b_out,
                                          int& before_out) {
  b_out = 0;
  before_out = 0;
  if (p.prefix) return;
  int before = sum.before, tiles = sum.tiles, carry = 0;
  for (int b0 = 0;;) {
    if (before <= u && u < before + tiles) {
      part[THREADS / 32] = b0 + threadIdx.x;
      part[THREADS / 32 + 1] = before;
    }
    b0 += THREADS;
    if (b0 >= p.B) break;
    // the sum up to this chunk is the last thread's
    if (threadIdx.x == THREADS - 1) part[0] = before + tiles;
    __syncthreads();
    carry = part[0];
    __syncthreads();
    if (u < carry) break;
    const int b = b0 + threadIdx.x;
    tiles = b < p.B ? pd_seq(p, pd_len_of(p, b)).tiles : 0;
    int total;
    before = carry + pd_scan<THREADS>(tiles, part, total);
  }
  __syncthreads();
  b_out = part[THREADS / 32];
  before_out = part[THREADS / 32 + 1];
}

// A CTA's place in its range: the current run (tiles [i0, i_end) of group (b,
// h, rt)), and where the range goes on behind it.
struct PdWalk {
  int x, end;          // flattened start of the run; end of the range
  int base;            // flattened start of sequence b
  int b, h, rt;
  PdSeq s;
  int i0, i_end;
};

__device__ __forceinline__ void pd_run_here(const PdParams& p, PdWalk& w) {
  const int in = w.x - w.base;
  const int g = in / w.s.tiles;
  w.i0 = in - g * w.s.tiles;
  w.h = g / p.row_tiles;
  w.rt = g - w.h * p.row_tiles;
  w.i_end = min(w.i0 + w.end - w.x, w.s.tiles);
}

// The next run of the range, if there is one; it begins a group (of the next
// sequence that has tiles).
__device__ __forceinline__ bool pd_next_run(const PdParams& p, PdWalk& w, const int* lens_s) {
  w.x += w.i_end - w.i0;
  if (w.x >= w.end) return false;
  w.i0 = 0;
  if (++w.rt == p.row_tiles) {
    w.rt = 0;
    if (++w.h == p.H_kv) {
      w.h = 0;
      w.base = w.x;
      do {
        ++w.b;
        w.s = pd_seq(p, pd_len_of(p, w.b, lens_s));
      } while (w.s.tiles == 0);
    }
  }
  w.i_end = min(w.end - w.x, w.s.tiles);
  return true;
}

// First position of tile i.
__device__ __forceinline__ int pd_tile_key(const PdParams& p, const PdSeq& s, int i) {
  return (i < s.sb ? i : s.w0 + (i - s.sb)) << p.tile_shift;
}

// First position of warp `warp`'s slice of tile i.
__device__ __forceinline__ int pd_key(const PdSeq& s, int i, int warp) {
  return (i < s.sb ? i : s.w0 + (i - s.sb)) * PD_TILE + warp * PD_SLICE;
}

// Under a window, whether no row of the sequence keeps one of the n positions
// from key0 on: they are neither loaded nor looked up in the table.
__device__ __forceinline__ bool pd_gone(const PdParams& p, const PdSeq& s, int key0, int n = PD_SLICE) {
  return p.window > 0 && key0 >= p.n_sink && key0 + n - 1 < s.len - p.N_q - p.window + 1;
}

// ------------------------------------------------------------ warp pieces

__device__ __forceinline__ void pd_ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void pd_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit values, two of a row a lane.
__device__ __forceinline__ uint32_t pd_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c += a b, 16 x 8 x 16, fp32 accumulation.
template <bool BF16>
__device__ __forceinline__ void pd_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The rows of a run's group: row r of the tile is row r_first + r of the R
// rows of sequence w.b and K/V head w.h, or, in the prefix, of the B * R rows
// of that head.
__device__ __forceinline__ int pd_rows(const PdParams& p, const PdWalk& w) {
  return min(p.m, (p.prefix ? p.B * p.R : p.R) - w.rt * p.m);
}

// Index of row r in q, o and lse (r < pd_rows).
__device__ __forceinline__ size_t pd_row_index(const PdParams& p, const PdWalk& w, int r) {
  int b = w.b;
  r += w.rt * p.m;
  if (p.prefix) {
    b = r / p.R;
    r -= b * p.R;
  }
  return (static_cast<size_t>(b) * p.H + w.h * p.G) * p.N_q + r;
}

// The positions that row r (r < pd_rows) keeps: j <= hi, and j >= lo or j < n_sink.
__device__ __forceinline__ void pd_row_keeps(const PdParams& p, const PdWalk& w, int r, const int* lens_s,
                                             int& hi, int& lo) {
  int len = w.s.len;
  r += w.rt * p.m;
  if (p.prefix) {
    const int b = r / p.R;
    r -= b * p.R;
    len = pd_len_of(p, b, lens_s);
  }
  const int pos = len - p.N_q + (p.N_q == 1 ? 0 : r % p.N_q);
  hi = p.causal ? pos : len - 1;
  if (p.prefix) hi = min(hi, w.s.len - 1);
  lo = p.window > 0 ? pos - p.window + 1 : 0;
}

// ------------------------------------------------------------ loading warp

// 4-D tiled load of one box into shared memory; completes its bytes on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Rows of q into shared memory: untiled copies, 16-byte aligned and a
// multiple of 16 bytes long.
__device__ __forceinline__ void pd_copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void pd_sync_attending() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * PD_WARPS) : "memory");
}

// Up to PD_BATCH tiles of a run, and in lane 4 j + s the page of slice s of
// its j-th tile, if that slice is to be loaded.  The page is not looked at
// before its batch is loaded, so the table's latency is spent on the batch before.
constexpr int PD_BATCH = 32 / PD_WARPS;

struct PdBatch {
  PdWalk w;
  int i, n;
  bool have;
  int page;
};

__device__ __forceinline__ void pd_look_up(const PdParams& p, PdBatch& t, int lane) {
  t.n = min(PD_BATCH, t.w.i_end - t.i);
  t.have = false;
  const int j = lane / PD_WARPS;
  if (j < t.n) {
    const int key = pd_key(t.w.s, t.i + j, lane % PD_WARPS);
    t.have = key < t.w.s.len && !pd_gone(p, t.w.s, key);
    if (t.have)
      t.page = __ldcg(p.table + (p.prefix ? 0 : static_cast<size_t>(t.w.b) * p.max_pages) + (key >> p.page_shift));
  }
}

template <int D, int NT>
__device__ __forceinline__ void pd_load_role(const PdParams& p, const PdWalk& w0, const CUtensorMap* tmK,
                                          const CUtensorMap* tmV, uint32_t ring, uint32_t q_tile, uint32_t full,
                                          uint32_t empty, uint32_t q_full, uint32_t q_empty, const int* lens_s,
                                          int lane, volatile int* abort_flag) {
  using T = PdGeo<D, NT>;
  uint32_t stage = 0, phase = 1, q_phase = 1;           // parities of the empty barriers
  uint32_t issued = 0, q_issued = 0;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool x = mbar_try_wait(bar, par) || wait_slow(bar, par, abort_flag, p.status, p.watchdog_ns);
    return __all_sync(0xffffffffu, x);
  };
  // one batch is loaded while the next one's pages are looked up
  PdBatch t, next;
  t.w = w0;
  t.i = w0.i0;
  t.page = 0;
  pd_look_up(p, t, lane);
  bool fresh = true;                                    // t begins a run
  for (bool more = true; more && ok;) {
    next = t;
    next.i += t.n;
    const bool next_run = next.i >= next.w.i_end;
    if (next_run) {
      more = pd_next_run(p, next.w, lens_s);
      next.i = next.w.i0;
    }
    if (more) pd_look_up(p, next, lane);
    if (fresh) {
      ok = wait(q_empty, q_phase);
      if (!ok) break;
      q_phase ^= 1u;
      const int rows = pd_rows(p, t.w);
      if (elect_one()) mbar_arrive_expect_tx(q_full, rows * D * 2);
      __syncwarp();
      if (lane < rows)
        pd_copy_row(q_tile + lane * T::Q_LD, static_cast<const uint16_t*>(p.q) + pd_row_index(p, t.w, lane) * D, D * 2,
                    q_full);
      __syncwarp();
      ++q_issued;
    }
    // a bad entry's box lies outside the tensor and is filled with zeros
    const bool good = static_cast<unsigned>(t.page) < static_cast<unsigned>(p.n_pages);
    const int t_z = good ? t.page * p.H_kv + t.w.h : -1;
    if (t.have && !good) atomicCAS(p.status, 0, -1);
    const uint32_t t_have = __ballot_sync(0xffffffffu, t.have);
    for (int j = 0; j < t.n; ++j) {
      const uint32_t have = t_have >> (j * PD_WARPS) & ((1u << PD_WARPS) - 1);
      ok = wait(empty + 8 * stage, phase);
      if (!ok) break;
      const uint32_t bar = full + 8 * stage, dst = ring + stage * T::STAGE_BYTES;
      const int y0 = pd_tile_key(p, t.w.s, t.i + j) & ((1 << p.page_shift) - 1);
      int z[PD_WARPS];
#pragma unroll
      for (int s = 0; s < PD_WARPS; ++s) z[s] = __shfl_sync(0xffffffffu, t_z, j * PD_WARPS + s);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, __popc(have) * 2 * T::SLICE_BYTES);
#pragma unroll
        for (int s = 0; s < PD_WARPS; ++s) {
          if (!((have >> s) & 1u)) continue;
          const int y = (y0 + s * PD_SLICE) & ((1 << p.page_shift) - 1);
          tma_load_4d(dst + s * T::SLICE_BYTES, tmK, bar, 0, y, 0, z[s]);
          tma_load_4d(dst + T::HALF_BYTES + s * T::SLICE_BYTES, tmV, bar, 0, y, 0, z[s]);
        }
      }
      __syncwarp();
      ++issued;
      if (++stage == T::NST) {
        stage = 0;
        phase ^= 1u;
      }
    }
    t = next;
    fresh = next_run;
  }
  // after an expired wait, the copies still in flight
  if (!ok) {
    for (uint32_t i = issued > T::NST ? issued - T::NST : 0; i < issued; ++i)
      drain_wait(full + 8 * (i % T::NST), (i / T::NST) & 1u, p.watchdog_ns);
    if (q_issued > 0) drain_wait(q_full, (q_issued - 1) & 1u, p.watchdog_ns);
  }
}

// ------------------------------------------------------------ attending kernel

// PD_WARPS warps attend and one loads.  The loading warp looks up pages and
// brings tiles (and each run's query rows) through a ring of TMA loads, runs
// ahead of the others.  An attending warp takes slice `warp` of every tile of
// the range, with its own running (m, l, O) for the group's rows in registers;
// none waits for another before the end of a run, where their results are
// combined through shared memory.
//
// Bound: HBM (32 sequences of up to 16384 positions, 8 K/V heads, d = 128: 186
// us, 6.65 TB/s of K and V; 8 of up to 8192: 33.5 us, 4.9 TB/s, the rest being the
// chain of lengths, table and first tiles).  Two CTAs' rings keep 192 KB a SM in
// flight; three CTAs with rings of two tiles took 203 us.  With two attending
// warps on each scheduler the instructions of a slice bound the rate next,
// so they are kept few: the integer work of the loads is the loading warp's (in the
// attending warps it took half of a slice's 1300 cycles), and the products are
// taken transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync 16 x 8 x 16, 16
// positions or 16 columns by 8 query rows), so that up to 8 rows, the query heads
// of a K/V head at one new row each, cost half of what a 16-row tile of Q would;
// tcgen05's 128 rows would cost 16 times that and as many more exponentials.
template <int D, int NT, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_THREADS, 2)
attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PdParams p) {
  using T = PdGeo<D, NT>;
  constexpr int M = T::M;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* part = reinterpret_cast<int*>(smem + T::SCAN_OFF);
  int* lens_s = reinterpret_cast<int*>(smem + T::LENS_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::ABORT_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t ring = smem_addr(smem);
  const uint32_t full = smem_addr(smem) + T::BAR_OFF, empty = full + 8 * T::NST;
  const uint32_t q_full = empty + 8 * T::NST, q_empty = q_full + 8;
  const uint32_t q_tile = smem_addr(smem) + T::Q_OFF;
  float* xbuf = reinterpret_cast<float*>(smem + T::X_OFF);
  float* stat = reinterpret_cast<float*>(smem + T::STAT_OFF);
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::NST; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, PD_WARPS);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, PD_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // Behind a shared prefix the launch before is the prefix's, whose CTAs had
  // passed their dependency wait when this one was launched: what came before
  // that is complete, and nothing here reads what the prefix's launch writes.
  // So the two run side by side, and only the last CTA waits, at its end, so
  // that this launch is not complete before the other one.
  const bool late = p.shared_tiles > 0 && !p.prefix;
  if (!late) grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();

  const int HR = p.H_kv * p.row_tiles;
  const PdSum sum = pd_sum<PD_THREADS>(p, part, lens_s);
  const PdCut cut = p.prefix ? pd_cut_prefix(p, sum.ranges) : pd_cut(sum.total * HR, sum.ranges);
  if (static_cast<int>(blockIdx.x) >= cut.n) {
    if (warp == PD_WARPS) {
      pd_report_lens(p);
      if (late && blockIdx.x + 1 == gridDim.x) grid_dependency_wait();
    }
    return;
  }
  PdWalk w;
  const int f0 = pd_start(cut, blockIdx.x);
  w.x = f0;
  w.end = pd_start(cut, blockIdx.x + 1);
  pd_locate<PD_THREADS>(p, sum, w.x / HR, part, w.b, w.base);
  w.base *= HR;
  w.s = pd_seq(p, pd_len_of(p, w.b, lens_s));
  pd_run_here(p, w);

  if (warp == PD_WARPS) {
    if (!p.withhold_loads)   // failure-detection test: every wait on a tile runs out
      pd_load_role<D, NT>(p, w, &tmK, &tmV, ring, q_tile, full, empty, q_full, q_empty, lens_s, lane, abort_flag);
    pd_report_lens(p);
    if (late && blockIdx.x + 1 == gridDim.x) grid_dependency_wait();
    return;
  }

  // Fragments: lane 4 g + t holds positions g and g + 8 (of K's slice) or
  // columns g and g + 8 (of V's 16), and query rows 8 n + 2 t and 8 n + 2 t + 1.
  const int g = lane >> 2, t = lane & 3;
  // A scale of 0 (every kept logit 0, whatever the size of q . k) is run as 1
  // with Q as zeros: the maximum is then taken of real logits, not of 0 times the
  // minus infinity of masked ones.  A negative scale turns the signs of Q.
  const float c = p.scale_log2 != 0.f ? fabsf(p.scale_log2) : 1.f;
  const uint32_t q_sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  const uint32_t q_keep = p.scale_log2 != 0.f ? 0xffffffffu : 0u;
  // ldmatrix: lane -> row lane & 7 of 8 x 8 matrix lane / 8.  K: matrices
  // (positions 0-7, d 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15); V,
  // transposed: (0-7, 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15).  The four
  // column pairs of a 128-byte row, swizzled, are four offsets.
  const int mat = lane >> 3, mr = lane & 7;
  uint32_t k_off[4], v_off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    k_off[k] = ((mat & 1) * 8 + mr) * 128 + (((2 * k + (mat >> 1)) ^ mr) << 4);
    v_off[k] = ((mat >> 1) * 8 + mr) * 128 + (((2 * k + (mat & 1)) ^ mr) << 4);
  }
  constexpr uint32_t one2 = BF16 ? 0x3f803f80u : 0x3c003c00u;
  const uint32_t ones[4] = {one2, one2, one2, one2};
  uint32_t stage = 0, phase = 0, q_phase = 0;
  bool ok = true;
  // Whether the barrier's phase is over; after an expired wait the warp goes on
  // to the end without waiting, so that no barrier of the CTA is missed.
  auto wait = [&](uint32_t bar, uint32_t par) {
    if (ok) {
      ok = mbar_try_wait(bar, par) || wait_slow(bar, par, abort_flag, p.status, p.watchdog_ns);
      ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
  };

  for (bool more = true; more;) {
    uint32_t qf[D / 16][NT][2];
    wait(q_full, q_phase);
    q_phase ^= 1u;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t x[4];
        pd_ldsm(q_tile + (n * 8 + mr) * T::Q_LD + (4 * k + mat) * 16, x);
        qf[2 * k][n][0] = (x[0] & q_keep) ^ q_sign;
        qf[2 * k][n][1] = (x[1] & q_keep) ^ q_sign;
        qf[2 * k + 1][n][0] = (x[2] & q_keep) ^ q_sign;
        qf[2 * k + 1][n][1] = (x[3] & q_keep) ^ q_sign;
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty);
    // limits of this lane's rows, and the positions that some row keeps and
    // that all rows keep
    int hi[NT][2], lo[NT][2];
    int hi_max = -1, hi_min = INT_MAX, lo_min = INT_MAX, lo_max = INT_MIN;
    {
      const int n_rows = pd_rows(p, w);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e;
          hi[n][e] = -1;
          lo[n][e] = 0;
          if (r < n_rows) {
            pd_row_keeps(p, w, r, lens_s, hi[n][e], lo[n][e]);
            hi_max = max(hi_max, hi[n][e]);
            hi_min = min(hi_min, hi[n][e]);
            lo_min = min(lo_min, lo[n][e]);
            lo_max = max(lo_max, lo[n][e]);
          }
        }
      hi_max = __reduce_max_sync(0xffffffffu, hi_max);
      hi_min = __reduce_min_sync(0xffffffffu, hi_min);
      lo_min = __reduce_min_sync(0xffffffffu, lo_min);
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    }

    float acc[D / 16][NT][4];
    float lsum[NT][4];          // sums of the rounded weights, by the tensor cores
    float m[NT][2], le[NT][2];  // maximum (log2 units), sum of the exact weights
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) lsum[n][e] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      le[n][0] = le[n][1] = 0.f;
    }

    for (int i = w.i0; i < w.i_end; ++i) {
      const int key0 = pd_key(w.s, i, warp);
      const uint32_t ks = ring + stage * T::STAGE_BYTES + warp * T::SLICE_BYTES, vs = ks + T::HALF_BYTES;
      const uint32_t free_bar = empty + 8 * stage;
      wait(full + 8 * stage, phase);
      if (++stage == T::NST) {
        stage = 0;
        phase ^= 1u;
      }
      // a slice with no position that a row may keep was not loaded
      if (!ok || key0 >= w.s.len || pd_gone(p, w.s, key0)) {
        if (lane == 0) mbar_arrive(free_bar);
        continue;
      }
      // S^T in two chains of products: for 8 rows, the even and the odd steps of
      // d summed apart
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t kf[4];
        pd_ldsm(ks + (k >> 2) * T::CHUNK_BYTES + k_off[k & 3], kf);
#pragma unroll
        for (int n = 0; n < NT; ++n) pd_mma<BF16>(s[NT == 1 ? k & 1 : n], kf, qf[k][n][0], qf[k][n][1]);
      }
      bool up = false;
      if constexpr (NT == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][e] += s[1][e];
      }
      const bool masked = key0 + PD_SLICE - 1 > hi_min ||
                          (p.window > 0 && key0 < lo_max && key0 + PD_SLICE > p.n_sink);
      if (masked) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + g + (e >> 1) * 8;
            const bool keep = j <= hi[n][e & 1] && (p.window == 0 || j >= lo[n][e & 1] || j < p.n_sink);
            if (!keep) s[n][e] = -INFINITY;
          }
      }
      // lazy rescale: the stale maximum is kept until a row's grows by 2^8;
      // only then do the lanes that share a row agree on it
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) up |= fmaxf(s[n][e], s[n][e + 2]) * c > m[n][e] + RESCALE_THRESHOLD;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[n][e], s[n][e + 2]) * c;
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const bool grow = x > m[n][e] + RESCALE_THRESHOLD;
            const float a = grow ? (m[n][e] == -INFINITY ? 0.f : fast_exp2(m[n][e] - x)) : 1.f;
            if (grow) m[n][e] = x;
            le[n][e] *= a;
            lsum[n][e] *= a;
            lsum[n][e + 2] *= a;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              acc[k][n][e] *= a;
              acc[k][n][e + 2] *= a;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float r0 = m[n][0] == -INFINITY ? 0.f : -m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : -m[n][1];
        const float p0 = fast_exp2(fmaf(s[n][0], c, r0)), p1 = fast_exp2(fmaf(s[n][1], c, r1));
        const float p2 = fast_exp2(fmaf(s[n][2], c, r0)), p3 = fast_exp2(fmaf(s[n][3], c, r1));
        le[n][0] += p0 + p2;
        le[n][1] += p1 + p3;
        pf[n][0] = pd_transpose(pack2<BF16>(p0, p1));
        pf[n][1] = pd_transpose(pack2<BF16>(p2, p3));
        // O is divided by the sum of the weights as they are multiplied (16
        // bits), so that their rounding errors partly cancel
        pd_mma<BF16>(lsum[n], ones, pf[n][0], pf[n][1]);
      }
      // V rows that no row of the group keeps count as zeros: their weight is
      // 0, and 0 times what such a row holds could be NaN
      const bool holes = masked && (key0 + PD_SLICE - 1 > hi_max ||
                                    (p.window > 0 && key0 < lo_min && key0 + PD_SLICE > p.n_sink));
      if (!holes) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vf[4];
          pd_ldsm_t(vs + (k >> 2) * T::CHUNK_BYTES + v_off[k & 3], vf);
#pragma unroll
          for (int n = 0; n < NT; ++n) pd_mma<BF16>(acc[k][n], vf, pf[n][0], pf[n][1]);
        }
      } else {
        auto bits = [&](int j) {
          const bool k0 = j <= hi_max && (p.window == 0 || j >= lo_min || j < p.n_sink);
          const bool k1 = j + 1 <= hi_max && (p.window == 0 || j + 1 >= lo_min || j + 1 < p.n_sink);
          return (k0 ? 0xffffu : 0u) | (k1 ? 0xffff0000u : 0u);
        };
        const uint32_t first = bits(key0 + 2 * t), second = bits(key0 + 8 + 2 * t);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vf[4];
          pd_ldsm_t(vs + (k >> 2) * T::CHUNK_BYTES + v_off[k & 3], vf);
          vf[0] &= first;
          vf[1] &= first;
          vf[2] &= second;
          vf[3] &= second;
#pragma unroll
          for (int n = 0; n < NT; ++n) pd_mma<BF16>(acc[k][n], vf, pf[n][0], pf[n][1]);
        }
      }
      __syncwarp();   // every lane has read the slice
      if (lane == 0) mbar_arrive(free_bar);
    }

    // ---- the run's result: the warps' (m, l, O) combined
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = le[n][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          float* sw = stat + warp * M + 8 * n + 2 * t + e;
          sw[0] = m[n][e];
          sw[PD_WARPS * M] = x;
          sw[2 * PD_WARPS * M] = lsum[n][e];
        }
      }
    // where the result goes: the output, or for a split group the slot of the
    // range's first (0) or of another run (1), or else the group's own place
    const bool split = w.i_end - w.i0 != w.s.tiles;
    const bool direct = !split && !p.prefix && p.shared_tiles == 0;
    const int n_rows = pd_rows(p, w);
    size_t row;
    float* po = split ? p.part_o : p.own_o;
    float* pl = split ? p.part_lse : p.own_lse;
    if (direct)
      row = pd_row_index(p, w, 0);
    else if (split)
      row = (2 * static_cast<size_t>(blockIdx.x) + (w.x == f0 ? 0 : 1)) * M;
    else
      row = (static_cast<size_t>(w.b) * HR + w.h * p.row_tiles + w.rt) * M;
    more = pd_next_run(p, w, lens_s);

    constexpr int XR = T::X_ROWS;
#pragma unroll
    for (int r0 = 0; r0 < M; r0 += XR) {
      if (r0 >= n_rows) break;
      // rows [r0, r0 + XR) of this warp's O; rows 4 apart in bank and columns
      // side by side, so the stores of a warp hit every bank once
      if (XR == 8 || (t >> 1) == ((r0 >> 2) & 1)) {
        float* xw = xbuf + (warp * XR + ((2 * t) & (XR - 1))) * T::X_LD + g;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const float (&a)[4] = acc[k][r0 / 8];
          xw[16 * k] = a[0];
          xw[16 * k + T::X_LD] = a[1];
          xw[16 * k + 8] = a[2];
          xw[16 * k + 8 + T::X_LD] = a[3];
        }
      }
      pd_sync_attending();
      // this thread: four columns of one row
      const int xr = threadIdx.x / (D / 4), c4 = threadIdx.x % (D / 4), r = r0 + xr;
      if (r < n_rows) {
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) top = fmaxf(top, stat[v * M + r]);
        const float ref = top == -INFINITY ? 0.f : top;
        float l_exact = 0.f, l_round = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
          const float wt = fast_exp2(stat[v * M + r] - ref);
          l_exact = fmaf(wt, stat[(PD_WARPS + v) * M + r], l_exact);
          l_round = fmaf(wt, stat[(2 * PD_WARPS + v) * M + r], l_round);
          const float4 y = *reinterpret_cast<const float4*>(xbuf + (v * XR + xr) * T::X_LD + c4 * 4);
          o.x = fmaf(wt, y.x, o.x);
          o.y = fmaf(wt, y.y, o.y);
          o.z = fmaf(wt, y.z, o.z);
          o.w = fmaf(wt, y.w, o.w);
        }
        // a row without weights is set to 0 and not multiplied by it: its sums hold
        // 0 times every V row that another row of the group keeps, NaN if one is not finite
        const bool empty = l_exact == 0.f;
        const float inv = __fdividef(1.f, l_round);
        o.x = empty ? 0.f : o.x * inv;
        o.y = empty ? 0.f : o.y * inv;
        o.z = empty ? 0.f : o.z * inv;
        o.w = empty ? 0.f : o.w * inv;
        const size_t at = (row + r) * D + c4 * 4;
        if (!direct)
          *reinterpret_cast<float4*>(po + at) = o;
        else if constexpr (OUT_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) = o;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at) =
              make_uint2(pack2<BF16>(o.x, o.y), pack2<BF16>(o.z, o.w));
        if (c4 == 0) {
          const float z = empty ? -INFINITY : (top + __log2f(l_exact)) * 0.69314718055994531f;
          if (!direct) pl[row + r] = z;
          else if (p.lse != nullptr) p.lse[row + r] = z;
        }
      }
      pd_sync_attending();
    }
  }
}

// ------------------------------------------------------------ merge

// The partial results of one group: `n` slots from range c0 on, or the one
// of a group that one run covers.
struct PdParts {
  const float* o;
  const float* lse;
  int n;
  size_t row;       // row of the first part, in rows of m a slot or group
  size_t row_next;  // row of the second part; the others follow `step` apart
  int step;
};

// The parts of group `group`, whose tiles are [start, start + tiles).
__device__ __forceinline__ PdParts pd_parts(const PdParams& p, const PdCut& cut, int start, int tiles,
                                            size_t group, int row) {
  PdParts x;
  x.n = 0;
  if (tiles == 0) return x;
  const int c0 = pd_range_of(cut, start), c1 = pd_range_of(cut, start + tiles - 1);
  x.n = c1 - c0 + 1;
  if (x.n == 1) {
    x.o = p.own_o;
    x.lse = p.own_lse;
    x.row = group * p.m + row;
  } else {
    x.o = p.part_o;
    x.lse = p.part_lse;
    // the first part is its range's last run, the others their ranges' first
    x.row = (2 * static_cast<size_t>(c0) + (start != pd_start(cut, c0) ? 1 : 0)) * p.m + row;
  }
  x.row_next = 2 * (static_cast<size_t>(c0) + 1) * p.m + row;
  x.step = 2 * p.m;
  return x;
}

// The same of a row r further on in the group.
__device__ __forceinline__ PdParts pd_row_on(PdParts x, int r) {
  x.row += r;
  x.row_next += r;
  return x;
}

__device__ __forceinline__ size_t pd_part_row(const PdParts& x, int s) {
  return s == 0 ? x.row : x.row_next + static_cast<size_t>(s - 1) * x.step;
}

// A weighted sum of parts: max LSE_s, sum_s exp(LSE_s - max) and the same of
// four columns of O_s.
struct PdMix {
  float top, tot;
  float4 r;
};

__device__ __forceinline__ PdMix pd_no_parts() { return {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}; }

__device__ __forceinline__ void pd_scale(PdMix& x, float f) {
  x.tot *= f;
  x.r.x *= f;
  x.r.y *= f;
  x.r.z *= f;
  x.r.w *= f;
}

// Parts first, first + step, ... of `a`, then of `b` (b.n may be 0), of the
// columns 4 c4 .. 4 c4 + 3.  Eight parts' loads are in flight together.
template <int D>
__device__ __forceinline__ PdMix pd_mix(int c4, const PdParts& a, const PdParts& b, int first, int step) {
  constexpr int U = 8;
  const int n = a.n + b.n;
  PdMix x = pd_no_parts();
  for (int s0 = first; s0 < n; s0 += U * step) {
    float l[U];
    float4 y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * step;
      l[u] = -INFINITY;
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < n) {
        const PdParts& part = s < a.n ? a : b;
        const size_t row = pd_part_row(part, s < a.n ? s : s - a.n);
        l[u] = __ldcg(part.lse + row);
        y[u] = __ldcg(reinterpret_cast<const float4*>(part.o + row * D) + c4);
      }
    }
    float top = x.top;
    bool nan = top != top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nan |= l[u] != l[u];
      top = fmaxf(top, l[u]);
    }
    if (nan) top = NAN;                          // kept as the maximum, it reaches all that follows
    const float ref = top == -INFINITY ? 0.f : top;
    pd_scale(x, __expf(x.top - ref));              // 0 for the first parts
    x.top = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float wgt = __expf(l[u] - ref);
      x.tot += wgt;
      x.r.x = fmaf(wgt, y[u].x, x.r.x);
      x.r.y = fmaf(wgt, y[u].y, x.r.y);
      x.r.z = fmaf(wgt, y[u].z, x.r.z);
      x.r.w = fmaf(wgt, y[u].w, x.r.w);
    }
  }
  return x;
}

// x += y, both sums over parts.
__device__ __forceinline__ void pd_join(PdMix& x, PdMix y) {
  const float top = x.top != x.top || y.top != y.top ? NAN : fmaxf(x.top, y.top);
  const float ref = top == -INFINITY ? 0.f : top;
  pd_scale(x, __expf(x.top - ref));
  pd_scale(y, __expf(y.top - ref));
  x.top = top;
  x.tot += y.tot;
  x.r.x += y.r.x;
  x.r.y += y.r.y;
  x.r.z += y.r.z;
  x.r.w += y.r.w;
}

// Row `idx` of the output.
template <int D, bool BF16, bool OUT_F32>
__device__ __forceinline__ void pd_write_mix(const PdParams& p, size_t idx, int c4, PdMix x) {
  const bool none = x.top == -INFINITY;
  const float inv = __fdividef(1.f, x.tot);
  x.r.x = none ? 0.f : x.r.x * inv;
  x.r.y = none ? 0.f : x.r.y * inv;
  x.r.z = none ? 0.f : x.r.z * inv;
  x.r.w = none ? 0.f : x.r.w * inv;
  if constexpr (OUT_F32) {
    reinterpret_cast<float4*>(static_cast<float*>(p.o) + idx * D)[c4] = x.r;
  } else {
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + idx * D)[c4] =
        make_uint2(pack2<BF16>(x.r.x, x.r.y), pack2<BF16>(x.r.z, x.r.w));
  }
  if (c4 == 0 && p.lse != nullptr) p.lse[idx] = none ? -INFINITY : x.top + __logf(x.tot);
}

// The rows of sequence b, which keeps nothing: zeros and minus infinity.
template <int D, bool OUT_F32>
__device__ __forceinline__ void pd_write_empty(const PdParams& p, int b) {
  const size_t row0 = static_cast<size_t>(b) * p.H * p.N_q;
  const int rows = p.H * p.N_q;
  constexpr int VEC = D * (OUT_F32 ? 4 : 2) / 16;
  uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.o) + row0 * D * (OUT_F32 ? 4 : 2));
  for (int i = threadIdx.x; i < rows * VEC; i += PD_MERGE) o[i] = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse != nullptr)
    for (int i = threadIdx.x; i < rows; i += PD_MERGE) p.lse[row0 + i] = -INFINITY;
}

// Without a shared prefix: CTAs c, c + ranges, ... (`subs` of them) take the
// group that the boundary behind range c cuts, if any, and of it the share that
// falls to them among the boundaries that cut the same group.
//
// Both merging kernels may read the lengths before their dependency wait: every
// CTA of the attending kernel had passed its own when this one was launched,
// so what ran before that kernel is complete, and it writes no lengths.
template <int D, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_MERGE)
attn_paged_merge(const PdParams p, int subs) {
  __shared__ int part[PD_MERGE / 32 + 2];
  const int HR = p.H_kv * p.row_tiles;
  const PdSum sum = pd_sum<PD_MERGE>(p, part, nullptr);
  const PdCut cut = pd_cut(sum.total * HR, p.ranges);
  const int c = blockIdx.x % p.ranges, sub = blockIdx.x / p.ranges;
  PdWalk w;
  bool any = c + 1 < cut.n;
  int c_first = 0, cuts = 1, g_start = 0;
  if (any) {
    w.x = pd_start(cut, c + 1) - 1;
    w.end = w.x + 1;
    pd_locate<PD_MERGE>(p, sum, w.x / HR, part, w.b, w.base);
    w.base *= HR;
    w.s = pd_seq(p, pd_len_of(p, w.b));
    pd_run_here(p, w);
    g_start = w.x - w.i0;
    any = w.i0 + 1 < w.s.tiles;                   // else the group ends with the range
    c_first = pd_range_of(cut, g_start);
    cuts = pd_range_of(cut, g_start + w.s.tiles - 1) - c_first;
  }
  grid_dependency_wait();
  grid_launch_dependents();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (pd_len_of(p, b) == 0) pd_write_empty<D, OUT_F32>(p, b);
  if (!any) return;
  const int r_first = w.rt * p.m, n_rows = min(p.m, p.R - r_first);
  const size_t idx0 = (static_cast<size_t>(w.b) * p.H + w.h * p.G) * p.N_q + r_first;
  PdParts none;
  none.n = 0;
  // D / 4 threads a row.  Few rows of many parts: the CTA's SETS sets of
  // threads share a row's parts; else each takes rows of its own.
  constexpr int SETS = PD_MERGE / (D / 4);
  const int set = threadIdx.x / (D / 4), c4 = threadIdx.x % (D / 4);
  const int mine = (c - c_first) * subs + sub, takers = cuts * subs;
  const PdParts parts = pd_parts(p, cut, g_start, w.s.tiles, 0, 0);
  if (parts.n > 8 && n_rows <= 2 * takers) {
    __shared__ PdMix mix[PD_MERGE];
    for (int r = mine; r < n_rows; r += takers) {
      PdMix x = pd_mix<D>(c4, pd_row_on(parts, r), none, set, SETS);
      mix[threadIdx.x] = x;
      __syncthreads();
      if (set == 0) {
#pragma unroll
        for (int v = 1; v < SETS; ++v) pd_join(x, mix[v * (D / 4) + c4]);
        pd_write_mix<D, BF16, OUT_F32>(p, idx0 + r, c4, x);
      }
      __syncthreads();
    }
  } else {
    for (int r = mine * SETS + set; r < n_rows; r += takers * SETS)
      pd_write_mix<D, BF16, OUT_F32>(p, idx0 + r, c4, pd_mix<D>(c4, pd_row_on(parts, r), none, 0, 1));
  }
}

// Behind a shared prefix every row has parts of the prefix and of its own
// positions: D / 4 threads a row, rows in the order of the output.
template <int D, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_MERGE)
attn_paged_merge_shared(const PdParams p, const PdParams pre) {
  __shared__ int part[PD_MERGE / 32 + 2];
  constexpr int SETS = PD_MERGE / (D / 4);
  const int HR = p.H_kv * p.row_tiles;
  const int rows_b = p.H * p.N_q, rows = p.B * rows_b;
  const int row0 = static_cast<int>(static_cast<long long>(rows) * blockIdx.x / gridDim.x);
  const int row1 = static_cast<int>(static_cast<long long>(rows) * (blockIdx.x + 1) / gridDim.x);
  const int b0 = row0 / rows_b;
  int x = 0, all = 0, before, total;
  for (int i = threadIdx.x; i < p.B; i += PD_MERGE) {
    const int tiles = pd_seq(p, pd_len_of(p, i)).tiles;
    all += tiles;
    if (i < b0) x += tiles;
  }
  pd_scan<PD_MERGE>(x, part, before);
  pd_scan<PD_MERGE>(all, part, total);
  const PdCut cut = pd_cut(total * HR, p.ranges);
  const PdCut p_cut = pd_cut_prefix(pre, pd_prefix_ranges(pre, total * HR));
  int b = b0;
  PdSeq s = pd_seq(p, pd_len_of(p, b));
  const int set = threadIdx.x / (D / 4), c4 = threadIdx.x % (D / 4);
  grid_dependency_wait();
  grid_launch_dependents();
  for (int row = row0 + set; row < row1; row += SETS) {
    for (; row >= (b + 1) * rows_b; s = pd_seq(p, pd_len_of(p, b))) {
      before += s.tiles;
      ++b;
    }
    int r = row - b * rows_b;
    const int h = r / p.R;
    r -= h * p.R;                                 // of the R rows of (b, h)
    const int g = h * p.row_tiles + r / p.m;
    const int pr = b * p.R + r;                   // row of the prefix
    const int pg = h * pre.row_tiles + pr / pre.m;
    const PdParts a = pd_parts(pre, p_cut, pg * pre.shared_tiles, pre.shared_tiles, pg, pr % pre.m);
    const PdParts own = pd_parts(p, cut, before * HR + g * s.tiles, s.tiles, static_cast<size_t>(b) * HR + g, r % p.m);
    pd_write_mix<D, BF16, OUT_F32>(p, row, c4, pd_mix<D>(c4, a, own, 0, 1));
  }
}

}  // namespace attn
