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
// partial outputs): a group is one sequence, one K/V head and up to PD_M of
// its (H / H_kv) * N_q query rows.  The kept 128-position tiles of all groups
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

constexpr int PD_TILE = 128;            // positions of a tile
constexpr int PD_SLICE = 16;            // positions a warp loads and attends at a time
constexpr int PD_WARPS = PD_TILE / PD_SLICE;
constexpr int PD_THREADS = 32 * PD_WARPS;
constexpr int PD_M = 16;                // query rows of a group

struct PdParams {
  const void* q;
  void* o;
  float* lse;
  float* part_o;        // [2 * gridDim.x][PD_M][D] results of runs of split groups
  float* part_lse;      // [2 * gridDim.x][PD_M]
  float* own_o;         // with a shared prefix: [groups][PD_M][D] results of groups with one run
  float* own_lse;       // [groups][PD_M]
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
  int row_tiles;        // groups of a sequence and K/V head (prefix: of a K/V head)
  int shared_tiles;     // whole tiles of the shared prefix
  int prefix;           // this launch attends the shared prefix
  int ranges;           // CTAs of the attending kernel
  int withhold_loads;   // test hook: no slice is loaded, so every wait runs out
};

// Shared memory of head dimension D: a ring of PD_NST slices (K, then V) for
// each warp, the exchange buffer of the epilogue, row statistics, barriers.
template <int D>
struct PdGeo {
  static_assert(D == 64 || D == 128, "the paged decoding kernel supports d = 64 and 128");
  static constexpr int NST = D == 128 ? 3 : 5;
  static constexpr int NCH = D / 64;                    // 64-column chunks, 128-byte swizzle
  static constexpr int CHUNK_BYTES = PD_SLICE * 128;
  static constexpr int HALF_BYTES = NCH * CHUNK_BYTES;  // K (or V) of a slice
  static constexpr int STAGE_BYTES = 2 * HALF_BYTES;
  static constexpr int RING_BYTES = PD_WARPS * NST * STAGE_BYTES;
  static constexpr int X_OFF = RING_BYTES;              // [PD_WARPS][PD_M][64] float
  static constexpr int STAT_OFF = X_OFF + PD_WARPS * PD_M * 64 * 4;
  static constexpr int BAR_OFF = STAT_OFF + 3 * PD_WARPS * PD_M * 4;
  static constexpr int SCAN_OFF = BAR_OFF + PD_WARPS * NST * 8;   // long long [PD_WARPS + 2]
  static constexpr int ABORT_OFF = SCAN_OFF + (PD_WARPS + 2) * 8;
  static constexpr int SMEM_BYTES = ABORT_OFF + 8;
  static_assert(SMEM_BYTES + 1024 <= 232448, "shared memory budget");
};

// ------------------------------------------------------------ work split

// The positions a sequence's rows may keep: [0, 128 sb) and [128 w0, len).
struct PdSeq {
  int len;      // positions (clamped to the table)
  int sb, w0;   // tiles [0, sb), then [w0, ...)
  int tiles;    // at least 1, so that every group has a run
};

__device__ __forceinline__ PdSeq pd_seq(const PdParams& p, int b) {
  PdSeq s;
  if (p.prefix) {
    s.len = p.shared_tiles * PD_TILE;
    s.sb = 0;
    s.w0 = 0;
    s.tiles = p.shared_tiles;
    return s;
  }
  const int cap = p.max_pages << p.page_shift;
  s.len = min(max(p.lens[b], 0), cap);
  const int nt = (s.len + PD_TILE - 1) / PD_TILE;
  s.sb = 0;
  s.w0 = p.shared_tiles;
  if (p.window > 0) {
    const long long first = static_cast<long long>(s.len) - p.N_q - p.window + 1;
    s.sb = min((min(p.n_sink, s.len) + PD_TILE - 1) / PD_TILE, nt);
    s.w0 = max(first > 0 ? static_cast<int>(first) / PD_TILE : 0, s.sb);
  }
  s.tiles = max(1, s.sb + max(0, nt - s.w0));
  return s;
}

__host__ __device__ inline long long pd_start(long long c, long long F, int grid) { return c * F / grid; }

// The range that holds flattened tile f.
__host__ __device__ inline int pd_range_of(long long f, long long F, int grid) {
  int c = static_cast<int>(f * grid / F);
  while (c + 1 < grid && pd_start(c + 1, F, grid) <= f) ++c;
  while (c > 0 && pd_start(c, F, grid) > f) --c;
  return c;
}

// Sum of x over the CTA's PD_THREADS threads, and the sum over the threads before this one.
__device__ __forceinline__ long long pd_scan(long long x, long long* part, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < PD_WARPS; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  __syncthreads();
  return before + s - x;
}

// Tiles of all sequences (of one group of each).
__device__ __forceinline__ long long pd_total(const PdParams& p, long long* part) {
  if (p.prefix) return p.shared_tiles;
  long long x = 0, total;
  for (int b = threadIdx.x; b < p.B; b += PD_THREADS) x += pd_seq(p, b).tiles;
  pd_scan(x, part, total);
  return total;
}

// The sequence that holds tile u of the sum of the sequences' tiles, and the
// tiles before it.  `slot` holds two values of shared memory.
__device__ __forceinline__ void pd_locate(const PdParams& p, long long u, long long* part,
                                          long long* slot, int& b_out, long long& before_out) {
  if (p.prefix) {
    b_out = 0;
    before_out = 0;
    return;
  }
  long long carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += PD_THREADS) {
    const int b = b0 + threadIdx.x;
    const int tiles = b < p.B ? pd_seq(p, b).tiles : 0;
    long long total;
    const long long before = carry + pd_scan(tiles, part, total);
    if (before <= u && u < before + tiles) {
      slot[0] = b;
      slot[1] = before;
    }
    carry += total;
    if (u < carry) break;
  }
  __syncthreads();
  b_out = static_cast<int>(slot[0]);
  before_out = slot[1];
  __syncthreads();
}

// A CTA's place in its range: the current run (tiles [i, i_end) of group (b,
// h, rt)), and where the range goes on behind it.
struct PdWalk {
  long long x, end;    // flattened start of the run; end of the range
  long long base;      // flattened start of sequence b
  int b, h, rt;
  PdSeq s;
  int i0, i_end;
};

__device__ __forceinline__ void pd_run_here(const PdParams& p, PdWalk& w) {
  const long long in = w.x - w.base;
  const int g = static_cast<int>(in / w.s.tiles);
  w.i0 = static_cast<int>(in - static_cast<long long>(g) * w.s.tiles);
  w.h = g / p.row_tiles;
  w.rt = g - w.h * p.row_tiles;
  const long long left = w.end - w.x;
  w.i_end = static_cast<int>(left < w.s.tiles - w.i0 ? w.i0 + left : w.s.tiles);
}

// The next run of the range, if there is one.
__device__ __forceinline__ bool pd_next_run(const PdParams& p, PdWalk& w) {
  w.x += w.i_end - w.i0;
  if (w.x >= w.end) return false;
  const long long all = static_cast<long long>(w.s.tiles) * p.H_kv * p.row_tiles;
  if (w.x >= w.base + all) {
    w.base += all;
    w.s = pd_seq(p, ++w.b);
  }
  pd_run_here(p, w);
  return true;
}

// First position of warp `warp`'s slice of tile i, and whether any row of the
// sequence may keep a position of the slice (others are neither loaded nor
// looked up in the table).
__device__ __forceinline__ bool pd_slice(const PdParams& p, const PdSeq& s, int i, int warp, int& key0) {
  key0 = (i < s.sb ? i : s.w0 + (i - s.sb)) * PD_TILE + warp * PD_SLICE;
  if (key0 >= s.len) return false;
  if (p.window > 0 && key0 >= p.n_sink && key0 + PD_SLICE - 1 < s.len - p.N_q - p.window + 1) return false;
  return true;
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

// A query row of a group: its index in q, o and lse, and the positions it
// keeps: j <= hi, and j >= lo or j < n_sink.
struct PdRow {
  bool real;
  size_t idx;
  int hi, lo;
};

__device__ __forceinline__ PdRow pd_row(const PdParams& p, const PdWalk& w, int r_in_tile) {
  PdRow x;
  int b = w.b, r = w.rt * PD_M + r_in_tile;
  if (p.prefix) {
    b = r / p.R;
    r -= b * p.R;
    x.real = b < p.B;
  } else {
    x.real = r < p.R;
  }
  x.idx = 0;
  x.hi = -1;
  x.lo = 0;
  if (!x.real) return x;
  const int head = r / p.N_q, i = r - head * p.N_q;
  x.idx = (static_cast<size_t>(b) * p.H + w.h * p.G + head) * p.N_q + i;
  int len = w.s.len;
  if (p.prefix) len = min(max(p.lens[b], 0), p.max_pages << p.page_shift);
  const int pos = len - p.N_q + i;
  x.hi = p.causal ? pos : len - 1;
  if (p.prefix) x.hi = min(x.hi, w.s.len - 1);
  if (p.window > 0) x.lo = pos - p.window + 1;
  return x;
}

// ------------------------------------------------------------ attending kernel

// Each warp streams its own slices: slice `warp` of every tile of the range,
// through its own ring of TMA loads, with its own running (m, l, O) for the
// group's PD_M rows in registers (mma.sync 16 x 8 x 16; rows past R are
// padding).  No warp waits for another before the end of a run, where the
// eight results are combined through shared memory.  The next runs' slices are
// in flight meanwhile.
//
// Bound: HBM.  A slice is 16 rows of K and of V; 8 warps x PD_NST slices keep
// 192 KB a SM in flight.  The tensor work of 16 padded rows is small against
// that (rows are few: a group's query heads times new rows), so the
// instruction with the smallest M is taken; tcgen05's 128 rows would do
// eight times the work and exponentials.
template <int D, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_THREADS, 1)
attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PdParams p) {
  using T = PdGeo<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  long long* part = reinterpret_cast<long long*>(smem + T::SCAN_OFF);
  long long* slot = part + PD_WARPS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::ABORT_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t ring = smem_addr(smem) + warp * T::NST * T::STAGE_BYTES;
  const uint32_t bars = smem_addr(smem) + T::BAR_OFF + warp * T::NST * 8;
  float* xbuf = reinterpret_cast<float*>(smem + T::X_OFF);
  float* stat = reinterpret_cast<float*>(smem + T::STAT_OFF);
  if (lane == 0) {
    for (int s = 0; s < T::NST; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    if (warp == 0) {
      *abort_flag = 0;
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();

  // lengths that do not fit the table are reported once
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.B; b += PD_THREADS) {
      const int n = p.lens[b];
      if (n < 0 || n > (p.max_pages << p.page_shift)) atomicCAS(p.status, 0, -1);
    }
  }
  const int HR = p.H_kv * p.row_tiles;
  const long long F = pd_total(p, part) * HR;
  const int ranges = static_cast<int>(F < gridDim.x ? F : gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ranges) return;
  PdWalk w;
  const long long f0 = pd_start(blockIdx.x, F, ranges);
  w.x = f0;
  w.end = pd_start(blockIdx.x + 1, F, ranges);
  {
    long long before;
    pd_locate(p, w.x / HR, part, slot, w.b, before);
    w.base = before * HR;
  }
  w.s = pd_seq(p, w.b);
  pd_run_here(p, w);

  // ---- this warp's loads: the slice to load next, and its page
  PdWalk lw = w;
  int li = lw.i0 - 1, l_key0 = 0, l_page = 0;
  bool l_more = true;
  uint32_t loaded = 0;
  auto advance = [&]() {
    for (;;) {
      if (++li >= lw.i_end) {
        l_more = pd_next_run(p, lw);
        if (!l_more) return;
        li = lw.i0;
      }
      if (pd_slice(p, lw.s, li, warp, l_key0)) break;
    }
    const int col = l_key0 >> p.page_shift;
    l_page = p.table[(p.prefix ? 0 : static_cast<size_t>(lw.b) * p.max_pages) + col];
  };
  auto refill = [&]() {
    if (!l_more) return;
    const int st = loaded % T::NST;
    const uint32_t bar = bars + 8 * st;
    const uint32_t dst = ring + st * T::STAGE_BYTES;
    const bool good = static_cast<unsigned>(l_page) < static_cast<unsigned>(p.n_pages);
    // a bad page's box lies outside the tensor and is filled with zeros
    const int z = good ? l_page * p.H_kv + lw.h : -1;
    const int y = l_key0 & ((1 << p.page_shift) - 1);
    if (elect_one()) {
      if (!good) atomicCAS(p.status, 0, -1);
      if (!p.withhold_loads) {
        mbar_arrive_expect_tx(bar, T::STAGE_BYTES);
#pragma unroll
        for (int c = 0; c < T::NCH; ++c)
          tma_load_3d(dst + c * T::CHUNK_BYTES, &tmK, bar, c * 64, y, z);
#pragma unroll
        for (int c = 0; c < T::NCH; ++c)
          tma_load_3d(dst + T::HALF_BYTES + c * T::CHUNK_BYTES, &tmV, bar, c * 64, y, z);
      }
    }
    __syncwarp();
    ++loaded;
    advance();
  };
  advance();
  for (int s = 0; s < T::NST; ++s) refill();

  const int g = lane >> 2, t = lane & 3;
  // A scale of 0 (every kept logit 0) is run as 1e-30: the logits then stay
  // within 1e-25 of 0, every weight rounds to exactly 1 in fp32 as for 0.
  const float c = p.scale_log2 != 0.f ? p.scale_log2 : 1e-30f;
  // ldmatrix row addresses: lane -> row (lane & 7) of 8 x 8 matrix lane / 8.
  // K: matrices (rows 0-7, d 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15);
  // V, transposed: (0-7, 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15).
  const int mat = lane >> 3, mr = lane & 7;
  const uint32_t k_row = static_cast<uint32_t>((mat >> 1) * 8 + mr) * 128;
  const uint32_t v_row = static_cast<uint32_t>((mat & 1) * 8 + mr) * 128;
  const int k_col = mat & 1, v_col = mat >> 1;
  uint32_t done = 0, waited = 0;   // slices passed; slices whose loads have landed
  bool ok = true;

  for (bool more = true; more;) {
    // ---- the run's rows
    const PdRow row0 = pd_row(p, w, g), row1 = pd_row(p, w, g + 8);
    uint32_t qf[D / 16][4];
    {
      const uint32_t* q0 = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + row0.idx * D) + t;
      const uint32_t* q1 = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + row1.idx * D) + t;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][0] = row0.real ? q0[8 * k] : 0u;
        qf[k][1] = row1.real ? q1[8 * k] : 0u;
        qf[k][2] = row0.real ? q0[8 * k + 4] : 0u;
        qf[k][3] = row1.real ? q1[8 * k + 4] : 0u;
      }
    }
    // positions that some row keeps, and that all rows keep
    int hi_max = max(row0.hi, row1.hi);
    int hi_min = min(row0.real ? row0.hi : INT_MAX, row1.real ? row1.hi : INT_MAX);
    int lo_min = min(row0.real ? row0.lo : INT_MAX, row1.real ? row1.lo : INT_MAX);
    int lo_max = max(row0.real ? row0.lo : INT_MIN, row1.real ? row1.lo : INT_MIN);
    hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);

    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;
    float le0 = 0.f, le1 = 0.f, lr0 = 0.f, lr1 = 0.f;   // sums of exact and of rounded weights

    for (int i = w.i0; i < w.i_end; ++i) {
      int key0;
      if (!pd_slice(p, w.s, i, warp, key0)) continue;
      const int st = done % T::NST;
      if (ok) {
        const uint32_t par = (done / T::NST) & 1u;
        ok = mbar_try_wait(bars + 8 * st, par) ||
             wait_slow(bars + 8 * st, par, abort_flag, p.status, p.watchdog_ns);
        ok = __all_sync(0xffffffffu, ok);
      }
      ++done;
      if (!ok) continue;
      waited = done;
      const uint32_t ks = ring + st * T::STAGE_BYTES, vs = ks + T::HALF_BYTES;
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t kf[4];
        const int u = (k & 3) * 2 + k_col;   // 16-byte unit of the 128-byte chunk row
        pd_ldsm(ks + (k >> 2) * T::CHUNK_BYTES + k_row + ((u ^ mr) << 4), kf);
        pd_mma<BF16>(s[0], qf[k], kf[0], kf[1]);
        pd_mma<BF16>(s[1], qf[k], kf[2], kf[3]);
      }
      // log2 units
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] *= c;
      const bool masked = key0 + PD_SLICE - 1 > hi_min ||
                          (p.window > 0 && key0 < lo_max && key0 + PD_SLICE > p.n_sink);
      if (masked) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = key0 + n * 8 + 2 * t + e;
            const bool sink = p.window == 0 || j < p.n_sink;
            if (!(j <= row0.hi && (sink || j >= row0.lo))) s[n][e] = -INFINITY;
            if (!(j <= row1.hi && (sink || j >= row1.lo))) s[n][2 + e] = -INFINITY;
          }
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      // lazy rescale: the stale maximum is kept until a row's grows by 2^8
      const bool up0 = x0 > m0 + RESCALE_THRESHOLD, up1 = x1 > m1 + RESCALE_THRESHOLD;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float a0 = up0 ? (m0 == -INFINITY ? 0.f : fast_exp2(m0 - x0)) : 1.f;
        const float a1 = up1 ? (m1 == -INFINITY ? 0.f : fast_exp2(m1 - x1)) : 1.f;
        if (up0) m0 = x0;
        if (up1) m1 = x1;
        le0 *= a0; lr0 *= a0; le1 *= a1; lr1 *= a1;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          acc[n][0] *= a0; acc[n][1] *= a0;
          acc[n][2] *= a1; acc[n][3] *= a1;
        }
      }
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t pf[4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = fast_exp2(s[n][0] - r0), p1 = fast_exp2(s[n][1] - r0);
        const float p2 = fast_exp2(s[n][2] - r1), p3 = fast_exp2(s[n][3] - r1);
        pf[2 * n] = pack2<BF16>(p0, p1);
        pf[2 * n + 1] = pack2<BF16>(p2, p3);
        le0 += p0 + p1;
        le1 += p2 + p3;
        // O is divided by the sum of the weights as they are multiplied (16
        // bits), so that their rounding errors partly cancel
        lr0 += unpack_lo<BF16>(pf[2 * n]) + unpack_hi<BF16>(pf[2 * n]);
        lr1 += unpack_lo<BF16>(pf[2 * n + 1]) + unpack_hi<BF16>(pf[2 * n + 1]);
      }
      // V rows that no row of the group keeps count as zeros: their weight is
      // 0, and 0 times what such a row holds could be NaN
      uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
      const bool holes = masked && (key0 + PD_SLICE - 1 > hi_max ||
                                    (p.window > 0 && key0 < lo_min && key0 + PD_SLICE > p.n_sink));
      if (holes) {
        auto bits = [&](int j) {
          const bool k0 = j <= hi_max && (p.window == 0 || j >= lo_min || j < p.n_sink);
          const bool k1 = j + 1 <= hi_max && (p.window == 0 || j + 1 >= lo_min || j + 1 < p.n_sink);
          return (k0 ? 0xffffu : 0u) | (k1 ? 0xffff0000u : 0u);
        };
        keep_lo = bits(key0 + 2 * t);
        keep_hi = bits(key0 + 8 + 2 * t);
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t vf[4];
        const int u = (n & 3) * 2 + v_col;
        pd_ldsm_t(vs + (n >> 2) * T::CHUNK_BYTES + v_row + ((u ^ mr) << 4), vf);
        if (holes) {
          vf[0] &= keep_lo;
          vf[1] &= keep_hi;
          vf[2] &= keep_lo;
          vf[3] &= keep_hi;
        }
        pd_mma<BF16>(acc[2 * n], pf, vf[0], vf[1]);
        pd_mma<BF16>(acc[2 * n + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();   // every lane has read the stage
      refill();
    }

    // ---- the run's result: the eight warps' (m, l, O) combined
    le0 += __shfl_xor_sync(0xffffffffu, le0, 1);
    le1 += __shfl_xor_sync(0xffffffffu, le1, 1);
    lr0 += __shfl_xor_sync(0xffffffffu, lr0, 1);
    lr1 += __shfl_xor_sync(0xffffffffu, lr1, 1);
    le0 += __shfl_xor_sync(0xffffffffu, le0, 2);
    le1 += __shfl_xor_sync(0xffffffffu, le1, 2);
    lr0 += __shfl_xor_sync(0xffffffffu, lr0, 2);
    lr1 += __shfl_xor_sync(0xffffffffu, lr1, 2);
    if (t == 0) {
      float* sw = stat + warp * PD_M;
      sw[g] = m0;
      sw[g + 8] = m1;
      sw[PD_WARPS * PD_M + g] = le0;
      sw[PD_WARPS * PD_M + g + 8] = le1;
      sw[2 * PD_WARPS * PD_M + g] = lr0;
      sw[2 * PD_WARPS * PD_M + g + 8] = lr1;
    }
    // this thread's share of the result: 4 columns of every 64 of one row
    const int orow = threadIdx.x >> 4, oc = threadIdx.x & 15;
    const PdRow out = pd_row(p, w, orow);
    const long long g_start = w.x - w.i0;
    const int c_first = pd_range_of(g_start, F, ranges);
    const int c_last = pd_range_of(g_start + w.s.tiles - 1, F, ranges);
    const bool split = c_first != c_last;
    const bool direct = !split && !p.prefix && p.shared_tiles == 0;
    const long long group = static_cast<long long>(w.b) * HR + w.h * p.row_tiles + w.rt;
    // a split group's run: the range's first one in slot 0, another in slot 1
    float* po;
    float* pl;
    if (split) {
      const size_t sl = 2 * static_cast<size_t>(blockIdx.x) + (w.x == f0 ? 0 : 1);
      po = p.part_o + (sl * PD_M + orow) * D;
      pl = p.part_lse + sl * PD_M + orow;
    } else {
      po = p.own_o + (static_cast<size_t>(group) * PD_M + orow) * D;
      pl = p.own_lse + static_cast<size_t>(group) * PD_M + orow;
    }
    float wt[PD_WARPS], M = 0.f, le = 0.f, inv = 0.f;
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      float* xw = xbuf + warp * PD_M * 64;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        // 8-byte units of a row are swapped by the row, so that a half-warp's
        // stores hit every bank once
        const int u = (n * 4 + t) ^ ((g & 3) * 4);
        *reinterpret_cast<float2*>(xw + g * 64 + u * 2) = make_float2(acc[half * 8 + n][0], acc[half * 8 + n][1]);
        *reinterpret_cast<float2*>(xw + (g + 8) * 64 + u * 2) = make_float2(acc[half * 8 + n][2], acc[half * 8 + n][3]);
      }
      __syncthreads();
      if (half == 0) {
        M = -INFINITY;
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) M = fmaxf(M, stat[v * PD_M + orow]);
        const float mr_ = M == -INFINITY ? 0.f : M;
        float lr = 0.f;
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
          wt[v] = fast_exp2(stat[v * PD_M + orow] - mr_);
          le += wt[v] * stat[(PD_WARPS + v) * PD_M + orow];
          lr += wt[v] * stat[(2 * PD_WARPS + v) * PD_M + orow];
        }
        inv = le == 0.f ? 0.f : 1.f / lr;
      }
      if (out.real) {
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
          const float* xr = xbuf + (v * PD_M + orow) * 64;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 y = *reinterpret_cast<const float2*>(xr + (((2 * oc + e) ^ ((orow & 3) * 4)) * 2));
            o[2 * e] = fmaf(wt[v], y.x, o[2 * e]);
            o[2 * e + 1] = fmaf(wt[v], y.y, o[2 * e + 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= inv;
        const int col = half * 64 + oc * 4;
        if (!direct) {
          *reinterpret_cast<float4*>(po + col) = make_float4(o[0], o[1], o[2], o[3]);
        } else if constexpr (OUT_F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.o) + out.idx * D + col) =
              make_float4(o[0], o[1], o[2], o[3]);
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + out.idx * D + col) =
              make_uint2(pack2<BF16>(o[0], o[1]), pack2<BF16>(o[2], o[3]));
        }
        if (half == 0 && oc == 0) {
          const float z = le == 0.f ? -INFINITY : (M + log2f(le)) * 0.69314718055994531f;
          if (!direct) *pl = z;
          else if (p.lse != nullptr) p.lse[out.idx] = z;
        }
      }
      __syncthreads();
    }
    more = pd_next_run(p, w);
  }
  // after an expired wait, the copies still in flight
  if (!ok && !p.withhold_loads) {
    for (; waited < loaded; ++waited)
      drain_wait(bars + 8 * (waited % T::NST), (waited / T::NST) & 1u, p.watchdog_ns);
  }
}

// ------------------------------------------------------------ merge

// The partial results of one group: `n` slots from range c0 on, or the one
// of a group that one run covers.
struct PdParts {
  const float* o;
  const float* lse;
  int n, c0;
  size_t row;       // row of the first part, in rows of PD_M a slot or group
  size_t row_next;  // row of the second part; the others follow 2 * PD_M apart
};

// The parts of group `group`, whose tiles [start, start + tiles) lie in
// `ranges` ranges of F tiles.
__device__ __forceinline__ PdParts pd_parts(const PdParams& p, long long start, int tiles, long long F,
                                            int ranges, size_t group, int row) {
  PdParts x;
  const int c0 = pd_range_of(start, F, ranges), c1 = pd_range_of(start + tiles - 1, F, ranges);
  x.n = c1 - c0 + 1;
  x.c0 = c0;
  if (x.n == 1) {
    x.o = p.own_o;
    x.lse = p.own_lse;
    x.row = group * PD_M + row;
  } else {
    x.o = p.part_o;
    x.lse = p.part_lse;
    // the first part is its range's last run, the others their ranges' first
    x.row = (2 * static_cast<size_t>(c0) + (start != pd_start(c0, F, ranges) ? 1 : 0)) * PD_M + row;
  }
  x.row_next = 2 * (static_cast<size_t>(c0) + 1) * PD_M + row;
  return x;
}

__device__ __forceinline__ size_t pd_part_row(const PdParts& x, int s) {
  return s == 0 ? x.row : x.row_next + static_cast<size_t>(s - 1) * 2 * PD_M;
}

// Four columns of row `idx` of the output: the parts of `a`, then those of
// `b` (b.n may be 0), weighted by exp(LSE_s - max LSE).
template <int D, bool BF16, bool OUT_F32>
__device__ __forceinline__ void pd_merge_row(const PdParams& p, size_t idx, int c4, const PdParts& a,
                                             const PdParts& b) {
  const int n = a.n + b.n;
  float mx = -INFINITY;
  bool nan = false;
  for (int s = 0; s < n; ++s) {
    const float x = s < a.n ? __ldcg(a.lse + pd_part_row(a, s)) : __ldcg(b.lse + pd_part_row(b, s - a.n));
    nan |= x != x;
    mx = fmaxf(mx, x);
  }
  const float ref = mx == -INFINITY ? 0.f : mx;
  float tot = 0.f;
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < n; ++s) {
    const PdParts& x = s < a.n ? a : b;
    const size_t row = pd_part_row(x, s < a.n ? s : s - a.n);
    const float wgt = expf(__ldcg(x.lse + row) - ref);
    if (wgt == 0.f) continue;      // a part with no kept position, or far below the others
    const float4 y = __ldcg(reinterpret_cast<const float4*>(x.o + row * D) + c4);
    tot += wgt;
    r.x = fmaf(wgt, y.x, r.x);
    r.y = fmaf(wgt, y.y, r.y);
    r.z = fmaf(wgt, y.z, r.z);
    r.w = fmaf(wgt, y.w, r.w);
  }
  const bool none = mx == -INFINITY && !nan;
  const float inv = none ? 0.f : 1.f / tot;
  r.x *= inv;
  r.y *= inv;
  r.z *= inv;
  r.w *= inv;
  if constexpr (OUT_F32) {
    reinterpret_cast<float4*>(static_cast<float*>(p.o) + idx * D)[c4] = r;
  } else {
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + idx * D)[c4] =
        make_uint2(pack2<BF16>(r.x, r.y), pack2<BF16>(r.z, r.w));
  }
  if (c4 == 0 && p.lse != nullptr) p.lse[idx] = none ? -INFINITY : ref + logf(tot);
}

// Without a shared prefix: CTA c takes the group that the boundary behind
// range c cuts, if any, and of it the share that falls to it among the
// boundaries that cut the same group.
template <int D, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_THREADS)
attn_paged_merge(const PdParams p) {
  __shared__ long long part[PD_WARPS], slot[2];
  grid_dependency_wait();
  grid_launch_dependents();
  const int HR = p.H_kv * p.row_tiles;
  const long long F = pd_total(p, part) * HR;
  const int ranges = static_cast<int>(F < p.ranges ? F : p.ranges);
  const int c = blockIdx.x;
  if (c + 1 >= ranges) return;
  PdWalk w;
  w.x = pd_start(c + 1, F, ranges) - 1;
  w.end = w.x + 1;
  long long before;
  pd_locate(p, w.x / HR, part, slot, w.b, before);
  w.base = before * HR;
  w.s = pd_seq(p, w.b);
  pd_run_here(p, w);
  const long long g_start = w.x - w.i0;
  if (w.i0 + 1 == w.s.tiles) return;             // the group ends with the range
  const int c_first = pd_range_of(g_start, F, ranges);
  const int c_last = pd_range_of(g_start + w.s.tiles - 1, F, ranges);
  const int cuts = c_last - c_first;
  for (int x = (c - c_first) * PD_THREADS + threadIdx.x; x < PD_M * (D / 4); x += cuts * PD_THREADS) {
    const int r = x / (D / 4), c4 = x % (D / 4);
    const PdRow row = pd_row(p, w, r);
    if (!row.real) continue;
    PdParts none;
    none.n = 0;
    pd_merge_row<D, BF16, OUT_F32>(p, row.idx, c4, pd_parts(p, g_start, w.s.tiles, F, ranges, 0, r), none);
  }
}

// Behind a shared prefix: one CTA for each sequence, K/V head and row tile.
template <int D, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(PD_THREADS)
attn_paged_merge_shared(const PdParams p, const PdParams pre) {
  __shared__ long long part[PD_WARPS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int HR = p.H_kv * p.row_tiles;
  const int g = static_cast<int>(blockIdx.x % HR), b = static_cast<int>(blockIdx.x / HR);
  long long x = 0, before, all = 0;
  for (int i = threadIdx.x; i < p.B; i += PD_THREADS) {
    const int tiles = pd_seq(p, i).tiles;
    all += tiles;
    if (i < b) x += tiles;
  }
  long long total;
  pd_scan(x, part, before);
  pd_scan(all, part, total);
  const long long F = total * HR;
  const int ranges = static_cast<int>(F < p.ranges ? F : p.ranges);
  PdWalk w;
  w.b = b;
  w.s = pd_seq(p, b);
  w.base = before * HR;
  w.x = w.base + static_cast<long long>(g) * w.s.tiles;
  w.end = w.x + w.s.tiles;
  pd_run_here(p, w);
  const long long g_start = w.x;
  const long long pF = static_cast<long long>(pre.shared_tiles) * pre.H_kv * pre.row_tiles;
  const int p_ranges = static_cast<int>(pF < pre.ranges ? pF : pre.ranges);
  const size_t group = static_cast<size_t>(b) * HR + g;
  for (int i = threadIdx.x; i < PD_M * (D / 4); i += PD_THREADS) {
    const int r = i / (D / 4), c4 = i % (D / 4);
    const PdRow row = pd_row(p, w, r);
    if (!row.real) continue;
    const long long pr = static_cast<long long>(b) * p.R + w.rt * PD_M + r;     // row of the prefix
    const size_t pg = static_cast<size_t>(w.h) * pre.row_tiles + pr / PD_M;
    pd_merge_row<D, BF16, OUT_F32>(
        p, row.idx, c4,
        pd_parts(pre, static_cast<long long>(pg) * pre.shared_tiles, pre.shared_tiles, pF, p_ranges, pg,
                 static_cast<int>(pr % PD_M)),
        pd_parts(p, g_start, w.s.tiles, F, ranges, group, r));
  }
}

}  // namespace attn
