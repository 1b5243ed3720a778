// paged_tc_kernel.cuh -- the decoding step over a cache of pages for many
// query rows of one K/V head (sm_100a): a prefix that the batch shares, or many
// heads or new rows a sequence.
//
// What it computes and how the work is split: as paged_kernel.cuh, with 128-
// position tiles and groups of up to 128 or 256 query rows.
//
// How: the rows are the A operand of S = Q K^T on the 5th-generation tensor
// cores (tcgen05.mma, one row a TMEM lane); P is written over S in TMEM and O +=
// P V reads it from there.  K and V tiles come page by page, one TMA load each,
// through a ring of shared-memory stages.  A tile lies in groups of 8 rows, each
// the 64-column chunks of its rows one behind the other (swizzled), so that a
// page of any size is one box and the groups of a tile are evenly spaced.  Two softmax warpgroups work in turn, so that
// one's softmax runs beside the other's products:
//   PAIR   (groups of 256 rows) each takes 128 rows and every tile, so that a
//          tile loaded feeds two pairs of products;
//   else   (128 rows) they take the even and the odd tiles of a run, each with
//          its own (m, l, O), combined when the run ends.
// Rows lie on lane r / 4 of warp r % 4, which spreads few rows over all warps.
//
// Bound: a 128 x 128 tile costs 8.4 MFLOP and 16384 exponentials (0.75 us at the
// measured bf16 rate, 0.54 us at 16 a clock); reading it costs 64 KB, once
// for every 128 rows (256 in PAIR) from L2.  Measured: 4180 cycles for a tile of
// both warpgroups, of which a warpgroup's softmax takes 2400 and the products
// behind its P 1780 (P lies over S, so the next S waits for P V); a run costs
// 18000 cycles beside its tiles.  64 rows a K/V head, 8 sequences of up to 8192: 54
// us (172 MB of K and V); 512 rows over 16384 shared positions on all SMs: 62 us.
#pragma once

#include "paged_kernel.cuh"

namespace attn {

constexpr int PT_TILE = 128;

template <int D, bool PAIR>
struct PtGeo {
  static_assert(D == 64 || D == 128, "the paged decoding kernels support d = 64 and 128");
  using G = Geo<D>;                                     // 64-column chunks, 128-byte swizzle
  static constexpr int NST = D == 64 ? 4 : (PAIR ? 2 : 3);   // K/V ring stages
  static constexpr int M = PAIR ? 256 : 128;            // query rows of a group
  static constexpr int GROUP_BYTES = G::NCH * 1024;     // 8 rows of a K or V tile
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + (PAIR ? 2 : 1) * G::TILE_BYTES;
  static constexpr int V_OFF = K_OFF + NST * G::TILE_BYTES;
  static constexpr int STAT_OFF = V_OFF + NST * G::TILE_BYTES;   // float [3][128]
  static constexpr int BAR_OFF = STAT_OFF + 3 * 128 * 4;
  static constexpr int SCAN_OFF = BAR_OFF + 256;        // int [NUM_THREADS / 32 + 2], then the longest length
  static constexpr int SMEM_BYTES = SCAN_OFF + 64;
  static constexpr uint32_t S_COL0 = 0;                 // S_h at column 128 h
  static constexpr uint32_t O_COL0 = 256;               // O_h at column 256 + D h
  static_assert(SMEM_BYTES + 1024 <= 232448, "shared memory budget");
};

enum PtBar : int {
  P_K_FULL = 0, P_K_EMPTY = 4, P_V_FULL = 8, P_V_EMPTY = 12,   // [NST] each (at most 4)
  P_S_FULL = 16, P_P_FULL = 18, P_O_FULL = 20,                // [2] each
  P_Q_FULL = 22, P_HALF = 24, P_DRAIN = 25, P_COUNT = 26      // P_Q_FULL: [2]
};
constexpr int PT_TMEM_SLOT_OFF = 8 * P_COUNT;
constexpr int PT_ABORT_OFF = PT_TMEM_SLOT_OFF + 4;

// The positions j that some row of the run's sequence (prefix: of the batch)
// keeps: j < len, and j >= lo or j < n_sink.
struct PtUsed {
  int len, lo;
};

__device__ __forceinline__ PtUsed pt_used(const PdParams& p, const PdWalk& w, int longest) {
  PtUsed u;
  u.len = p.prefix ? min(w.s.len, longest) : w.s.len;
  u.lo = p.window > 0 ? w.s.len - p.N_q - p.window + 1 : 0;
  return u;
}

// The last kept position of a lane without a row, or whose row keeps nothing: past
// every position, and pt_kept's hi - key0 + 1 still fits 32 bits.
constexpr int kAllKept = INT_MAX - 1;

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t pt_low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Which of the 32 positions from key0 on a row keeps: j <= hi, and j >= lo or
// j < n_sink.
__device__ __forceinline__ uint32_t pt_kept(const PdParams& p, int key0, int hi, int lo) {
  uint32_t k = pt_low_bits(hi - key0 + 1);
  if (p.window > 0) k &= ~pt_low_bits(lo - key0) | pt_low_bits(p.n_sink - key0);
  return k;
}

// ------------------------------------------------------------ roles

// 5-D tiled load of one box into shared memory; completes its bytes on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int u, int w) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(w)
      : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}

template <int D, bool PAIR>
__device__ void pt_tma_role(const PdParams& p, PdWalk w, const CUtensorMap* tmK, const CUtensorMap* tmV,
                            uint32_t sbase, uint32_t bars, int lane, volatile int* abort_flag) {
  using T = PtGeo<D, PAIR>;
  using G = Geo<D>;
  if (p.withhold_loads) return;   // failure-detection test: every wait on a tile runs out
  const int box = min(1 << p.page_shift, PT_TILE);     // rows of one load
  const int boxes = PT_TILE / box;                      // a power of two, at most 8
  const int bshift = 31 - __clz(boxes);
  uint32_t stage = 0, ph = 1;                           // parity of the empty barriers
  uint32_t issued[2] = {0, 0};                          // tiles of K and of V
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool x = mbar_try_wait(bar, par) || wait_slow(bar, par, abort_flag, p.status, p.watchdog_ns);
    return __all_sync(0xffffffffu, x);
  };
  for (bool more = true; more && ok; more = pd_next_run(p, w, nullptr)) {
    const int* row = p.table + (p.prefix ? 0 : static_cast<size_t>(w.b) * p.max_pages);
    // the run's query rows are fetched into L2 ahead of the softmax warps, which
    // read them only when the run before is finished
    for (int r = lane; r < pd_rows(p, w); r += 32) {
      const char* q = static_cast<const char*>(p.q) + pd_row_index(p, w, r) * D * 2;
#pragma unroll
      for (int c = 0; c < D * 2; c += 128) prefetch_l2(q + c);
    }
    int l_base = -32, l_page = -1;                      // pages of 32 boxes, from tile l_base on
    for (int i = w.i0; i < w.i_end && ok; ++i) {
      if (i >= l_base + (32 >> bshift)) {
        l_base = i;
        const int li = i + (lane >> bshift);
        l_page = -1;
        if (li < w.i_end) {
          const int key = pd_tile_key(p, w.s, li) + (lane & (boxes - 1)) * box;
          // -1: not loaded at all; a bad entry becomes a box outside the tensor
          if (key < w.s.len && !pd_gone(p, w.s, key, box)) {
            const int page = __ldcg(row + (key >> p.page_shift));
            l_page = static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages) ? page : p.n_pages;
            if (l_page == p.n_pages) atomicCAS(p.status, 0, -1);
          }
        }
      }
      const int first = (i - l_base) << bshift;         // lane of the tile's first box
      const uint32_t have = __ballot_sync(0xffffffffu, l_page >= 0) >> first & ((1u << boxes) - 1);
      const int u0 = (pd_tile_key(p, w.s, i) & ((1 << p.page_shift) - 1)) >> 3;   // group of the page
      int z[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int page = __shfl_sync(0xffffffffu, l_page, (first + x) & 31);
        z[x] = page < p.n_pages ? page * p.H_kv + w.h : -1;
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = bars + 8 * ((kv ? P_V_FULL : P_K_FULL) + stage);
        const uint32_t dst = sbase + (kv ? T::V_OFF : T::K_OFF) + stage * G::TILE_BYTES;
        ok = ok && wait(bars + 8 * ((kv ? P_V_EMPTY : P_K_EMPTY) + stage), ph);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full, __popc(have) * box * D * 2);
          // boxes of one tile lie in different pages, or are one (u0 is then its place there)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if ((have >> x) & 1u) tma_load_5d(dst + x * box * D * 2, kv ? tmV : tmK, full, 0, 0, 0, x == 0 ? u0 : 0, z[x]);
        }
        __syncwarp();
        ++issued[kv];
      }
      if (++stage == T::NST) {
        stage = 0;
        ph ^= 1u;
      }
    }
  }
  // after an expired wait, the copies still in flight
  if (!ok) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      for (uint32_t i = issued[kv] > T::NST ? issued[kv] - T::NST : 0; i < issued[kv]; ++i)
        drain_wait(bars + 8 * ((kv ? P_V_FULL : P_K_FULL) + i % T::NST), (i / T::NST) & 1u, p.watchdog_ns);
  }
}

// Item k of a run of n tiles: warpgroup k & 1 with tile k (PAIR: tile k / 2,
// which both take).
template <int D, bool PAIR, bool BF16>
__device__ void pt_mma_role(const PdParams& p, PdWalk w, uint32_t tmem, uint32_t sbase, uint32_t bars,
                            volatile int* abort_flag) {
  using T = PtGeo<D, PAIR>;
  using G = Geo<D>;
  constexpr uint32_t idesc_qk = instr_desc(BF16, BM, PT_TILE, false);
  constexpr uint32_t idesc_pv = instr_desc(BF16, BM, D, true);
  uint32_t it = 0, q_ph = 0, p_ph[2] = {0, 0};
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool x = mbar_try_wait(bar, par) || wait_slow(bar, par, abort_flag, p.status, p.watchdog_ns);
    return __all_sync(0xffffffffu, x);
  };
  auto issue_s = [&](int h, int s) {
    const uint32_t qa = sbase + T::Q_OFF + (PAIR ? h : 0) * G::TILE_BYTES;
    const uint32_t ka = sbase + T::K_OFF + s * G::TILE_BYTES;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t in = ((kk * 16) % G::CW) * 2;
      mma_ss(tmem + T::S_COL0 + h * PT_TILE,
             smem_desc(qa + (kk * 16 / G::CW) * G::CHUNK_BYTES + in, 16, 8 * G::CB, G::LAYOUT),
             smem_desc(ka + (kk * 16 / G::CW) * 1024 + in, 16, T::GROUP_BYTES, G::LAYOUT), idesc_qk, kk > 0 ? 1u : 0u);
    }
  };
  auto issue_o = [&](int h, int s, bool acc) {
    const uint32_t va = sbase + T::V_OFF + s * G::TILE_BYTES;
#pragma unroll
    for (int kk = 0; kk < PT_TILE / 16; ++kk)
      mma_ts(tmem + T::O_COL0 + h * D, tmem + T::S_COL0 + h * PT_TILE + kk * 8,
             smem_desc(va + kk * 2 * T::GROUP_BYTES, 1024, T::GROUP_BYTES, G::LAYOUT), idesc_pv,
             (acc || kk > 0) ? 1u : 0u);
  };
  // S of item k, once its K tile (and, first, the warpgroup's rows) is there
  auto do_s = [&](int k) {
    const int h = k & 1;
    const uint32_t j = it + (PAIR ? k >> 1 : k);
    const int s = j % T::NST;
    if (!wait(bars + 8 * (P_K_FULL + s), (j / T::NST) & 1u)) return false;
    tc_fence_after_sync();
    if (elect_one()) {
      issue_s(h, s);
      mma_commit(bars + 8 * (P_S_FULL + h));
      if (!PAIR || h == 1) mma_commit(bars + 8 * (P_K_EMPTY + s));
    }
    __syncwarp();
    return true;
  };
  for (bool more = true; more && ok; more = pd_next_run(p, w, nullptr)) {
    const int n = w.i_end - w.i0, items = PAIR ? 2 * n : n;
    ok = wait(bars + 8 * P_Q_FULL, q_ph) && (!PAIR || wait(bars + 8 * (P_Q_FULL + 1), q_ph));
    if (!ok) break;
    q_ph ^= 1u;
    tc_fence_after_sync();
    for (int k = 0; k < items && k < 2 && ok; ++k) ok = do_s(k);
    for (int k = 0; k < items && ok; ++k) {
      const int h = k & 1;
      const uint32_t j = it + (PAIR ? k >> 1 : k);
      const int s = j % T::NST;
      ok = wait(bars + 8 * (P_V_FULL + s), (j / T::NST) & 1u) && wait(bars + 8 * (P_P_FULL + h), p_ph[h]);
      if (!ok) break;
      p_ph[h] ^= 1u;
      tc_fence_after_sync();
      if (elect_one()) {
        issue_o(h, s, k >= 2);
        if (k + 2 >= items) mma_commit(bars + 8 * (P_O_FULL + h));
        if (!PAIR || h == 1) mma_commit(bars + 8 * (P_V_EMPTY + s));
      }
      __syncwarp();
      // S_h of the next item overwrites P_h only after the P_h V just issued
      if (k + 2 < items) ok = do_s(k + 2);
    }
    it += n;
  }
  if (elect_one()) mma_commit(bars + 8 * P_DRAIN);
  __syncwarp();
  drain_wait(bars + 8 * P_DRAIN, 0, p.watchdog_ns);
}

template <int D, bool PAIR, bool BF16, bool OUT_F32>
__device__ void pt_softmax_role(const PdParams& p, PdWalk w, int f0, uint32_t tmem, uint8_t* smem,
                                uint32_t sbase, uint32_t bars, int h, int wq, int lane, int longest,
                                volatile int* abort_flag) {
  using T = PtGeo<D, PAIR>;
  using G = Geo<D>;
  const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t s_tmem = tmem + lane_base + T::S_COL0 + h * PT_TILE;
  const int L = wq * 32 + lane;                         // TMEM lane
  const int r = 4 * lane + wq + (PAIR ? h * 128 : 0);   // row of the group
  // A scale of 0 is run as 1 with Q as zeros, a negative one by the signs of Q
  // (see attn_paged_kernel)
  const float c = p.scale_log2 != 0.f ? fabsf(p.scale_log2) : 1.f;
  const uint32_t q_sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  float* stat = reinterpret_cast<float*>(smem + T::STAT_OFF);
  uint32_t it = 0, s_ph = 0, o_ph[2] = {0, 0}, half_ph = 0;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool x = mbar_try_wait(bar, par) || wait_slow(bar, par, abort_flag, p.status, p.watchdog_ns);
    return __all_sync(0xffffffffu, x);
  };
  for (bool more = true; more && ok; more = pd_next_run(p, w, nullptr)) {
    const int n = w.i_end - w.i0;
    const int rows = pd_rows(p, w);
    const bool real = r < rows;
    if (PAIR || h == 0) {
      // this lane's query row (zeros for lanes without one) into the Q tile, in
      // the K-major 128-byte swizzle of the S = Q K^T operand; the previous
      // run's products have all completed (its epilogue waited for the last P V)
      const uint32_t row_addr = sbase + T::Q_OFF + (PAIR ? h : 0) * G::TILE_BYTES + L * 128;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                        (real ? pd_row_index(p, w, r) : 0) * D);
#pragma unroll
      for (int u = 0; u < D / 8; ++u) {
        const uint4 x = real && p.scale_log2 != 0.f ? __ldcg(src + u) : make_uint4(0u, 0u, 0u, 0u);
        st_shared_v4(row_addr + (u / 8) * G::CHUNK_BYTES + (((u % 8) ^ (L & 7)) << 4), x.x ^ q_sign, x.y ^ q_sign,
                     x.z ^ q_sign, x.w ^ q_sign);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (P_Q_FULL + (PAIR ? h : 0)));
    }
    int hi = kAllKept, lo = 0;
    if (real) pd_row_keeps(p, w, r, nullptr, hi, lo);
    // a row that keeps nothing (its sequence is empty, or it lies before
    // position 0) masks no tile; its result is set at the end
    const bool none = hi < 0;
    if (none) {
      hi = kAllKept;
      lo = 0;
    }
    const int hi_min = __reduce_min_sync(0xffffffffu, hi);
    const int lo_max = __reduce_max_sync(0xffffffffu, lo);
    const PtUsed used = pt_used(p, w, longest);
    float m_run = -INFINITY, l_exact = 0.f, l_round = 0.f;
    bool first = true;
    for (int k = PAIR ? 0 : h; k < n; k += PAIR ? 1 : 2) {
      const int c0 = pd_tile_key(p, w.s, w.i0 + k);
      ok = wait(bars + 8 * (P_S_FULL + h), s_ph);
      if (!ok) break;
      s_ph ^= 1u;
      tc_fence_after_sync();
      // S is read twice, 64 columns at a time: for its maximum, then for P.
      // Held in registers at once, its 128 columns left too few for the rest
      // (spills: 3 us a tile instead of 1).  The loops here and in the epilogue
      // are not unrolled: each launch fetches the code anew, and a first tile
      // took 6000 cycles where a later one takes 2200.
      const bool masked = c0 + PT_TILE - 1 > hi_min ||
                          (p.window > 0 && c0 < lo_max && c0 + PT_TILE > p.n_sink);
      uint32_t sa[32], sb[32];
      const auto fetch = [&](int col) {
        tmem_ld_32x32b_x32_start(s_tmem + col, sa);
        tmem_ld_32x32b_x32_start(s_tmem + col + 32, sb);
        tmem_wait_ld_x32(sa);
        tmem_wait_ld_x32(sb);
        if (masked) {
          const uint32_t ka = pt_kept(p, c0 + col, hi, lo), kb = pt_kept(p, c0 + col + 32, hi, lo);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            sa[e] = (ka >> e) & 1u ? sa[e] : 0xff800000u;
            sb[e] = (kb >> e) & 1u ? sb[e] : 0xff800000u;
          }
        }
      };
      float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        fetch(64 * half);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          m0 = max3(m0, __uint_as_float(sa[e]), __uint_as_float(sa[e + 1]));
          m1 = max3(m1, __uint_as_float(sb[e]), __uint_as_float(sb[e + 1]));
        }
      }
      const float m_new = fmaxf(m_run, fmaxf(m0, m1) * c);
      // online softmax (log2 units), lazy rescale as in the forward kernel
      float alpha = 1.f;
      const bool rescale = m_new > m_run + RESCALE_THRESHOLD;
      if (rescale) {
        alpha = (m_run == -INFINITY) ? 0.f : fast_exp2(m_run - m_new);
        m_run = m_new;
      }
      const float mref = (m_run == -INFINITY) ? 0.f : m_run;
      const float2 cc2 = make_float2(c, c);
      const float2 nm2 = make_float2(-mref, -mref);
      float2 le = make_float2(0.f, 0.f), lr = make_float2(0.f, 0.f);
      // P of 32 columns into 16 columns at `col`: over columns of S already read
      const auto weights = [&](const uint32_t (&x32)[32], int col) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = make_float2(__uint_as_float(x32[2 * e]), __uint_as_float(x32[2 * e + 1]));
          const float2 a = fma2(x, cc2, nm2);
          const float2 pe = make_float2(fast_exp2(a.x), fast_exp2(a.y));
          pk[e] = pack2<BF16>(pe.x, pe.y);
          le = add2(le, pe);
          lr = add2(lr, make_float2(unpack_lo<BF16>(pk[e]), unpack_hi<BF16>(pk[e])));
        }
        tmem_st_32x32b_x16(s_tmem + col, pk);
      };
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        fetch(64 * half);
        weights(sa, 32 * half);
        weights(sb, 32 * half + 16);
      }
      l_exact = l_exact * alpha + (le.x + le.y);
      l_round = l_round * alpha + (lr.x + lr.y);
      if (!first && __any_sync(0xffffffffu, rescale)) {
        // O_h holds the earlier tiles (their P V completed before the S product
        // of this tile was issued)
        const uint32_t o_tmem = tmem + lane_base + T::O_COL0 + h * D;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t orr[32];
          tmem_ld_32x32b_x32(o_tmem + cc * 32, orr);
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
          tmem_st_32x32b_x32(o_tmem + cc * 32, orr);
        }
      }
      // V rows that no row keeps count as zeros: their weight is 0, and 0 times
      // what such a row holds (or what was in the stage before) could be NaN
      if (c0 + PT_TILE > used.len || (p.window > 0 && c0 < used.lo && c0 + PT_TILE > p.n_sink)) {
        const uint32_t j = it + k;
        const int s = j % T::NST;
        ok = wait(bars + 8 * (P_V_FULL + s), (j / T::NST) & 1u);
        if (!ok) break;
        const int key = c0 + L;
        if (!(key < used.len && (key >= used.lo || key < p.n_sink))) {
          const uint32_t v_row = sbase + T::V_OFF + s * G::TILE_BYTES + (L >> 3) * T::GROUP_BYTES + (L & 7) * 128;
#pragma unroll 1
          for (int u = 0; u < D / 8; ++u) st_shared_v4(v_row + (u / 8) * 1024 + (u % 8) * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (P_P_FULL + h));
      first = false;
    }
    it += n;
    if (!ok) break;
    if (!PAIR && h == 1) {
      // the second half's row statistics for the first warpgroup's combine
      if (n >= 2) {
        stat[L] = m_run;
        stat[128 + L] = l_exact;
        stat[256 + L] = l_round;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * P_HALF);
      }
      continue;
    }
    // ---- the run's result: combine the halves, write it
    ok = wait(bars + 8 * (P_O_FULL + h), o_ph[0]);
    if (!ok) break;
    o_ph[0] ^= 1u;
    const bool two = !PAIR && n >= 2;
    float m1 = -INFINITY, le1 = 0.f, lr1 = 0.f;
    if (two) {
      ok = wait(bars + 8 * (P_O_FULL + 1), o_ph[1]);
      if (!ok) break;
      o_ph[1] ^= 1u;
      ok = wait(bars + 8 * P_HALF, half_ph);
      if (!ok) break;
      half_ph ^= 1u;
      m1 = stat[L];
      le1 = stat[128 + L];
      lr1 = stat[256 + L];
    }
    tc_fence_after_sync();
    const float M = fmaxf(m_run, m1);
    const float ref = (M == -INFINITY) ? 0.f : M;
    const float a0 = (m_run == -INFINITY) ? 0.f : fast_exp2(m_run - ref);
    const float a1 = (m1 == -INFINITY) ? 0.f : fast_exp2(m1 - ref);
    const float lr_t = l_round * a0 + lr1 * a1;
    const float le_t = l_exact * a0 + le1 * a1;
    const bool empty = none || le_t == 0.f;
    const float inv = empty ? 0.f : __fdividef(1.f, lr_t);
    const float lse_nat = empty ? -INFINITY : (M + __log2f(le_t)) * 0.69314718055994531f;
    const bool split = w.i_end - w.i0 != w.s.tiles;
    const bool direct = !split && !p.prefix && p.shared_tiles == 0;
    const int HR = p.H_kv * p.row_tiles;
    size_t row = r;
    if (direct)
      row += pd_row_index(p, w, 0);
    else if (split)
      row += (2 * static_cast<size_t>(blockIdx.x) + (w.x == f0 ? 0 : 1)) * T::M;
    else
      row += (static_cast<size_t>(w.b) * HR + w.h * p.row_tiles + w.rt) * T::M;
    float* po = split ? p.part_o : p.own_o;
    float* pl = split ? p.part_lse : p.own_lse;
#pragma unroll 1
    for (int cc = 0; cc < D / 16; ++cc) {
      uint32_t o0[16], o1[16];
      tmem_ld_32x32b_x16(tmem + lane_base + T::O_COL0 + (PAIR ? h * D : 0) + cc * 16, o0);
      if (two) tmem_ld_32x32b_x16(tmem + lane_base + T::O_COL0 + D + cc * 16, o1);
      float o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        o[e] = empty ? 0.f : (__uint_as_float(o0[e]) * a0 + (two ? __uint_as_float(o1[e]) * a1 : 0.f)) * inv;
      if (real) {
        if (direct && !OUT_F32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + cc * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            dst[e] = make_uint4(pack2<BF16>(o[8 * e], o[8 * e + 1]), pack2<BF16>(o[8 * e + 2], o[8 * e + 3]),
                                pack2<BF16>(o[8 * e + 4], o[8 * e + 5]), pack2<BF16>(o[8 * e + 6], o[8 * e + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>((direct ? static_cast<float*>(p.o) : po) + row * D + cc * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    }
    if (real) {
      if (!direct) pl[row] = lse_nat;
      else if (p.lse != nullptr) p.lse[row] = lse_nat;
    }
    tc_fence_before_sync();
  }
}

template <int D, bool PAIR, bool BF16, bool OUT_F32>
__global__ void __launch_bounds__(NUM_THREADS, 1)
attn_paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PdParams p) {
  using T = PtGeo<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + T::BAR_OFF;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::BAR_OFF + PT_ABORT_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::BAR_OFF + PT_TMEM_SLOT_OFF);
  int* part = reinterpret_cast<int*>(smem + T::SCAN_OFF);
  int* longest_s = part + NUM_THREADS / 32 + 2;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::NST; ++s) {
      mbar_init(bars + 8 * (P_K_FULL + s), 1);
      mbar_init(bars + 8 * (P_K_EMPTY + s), 1);
      mbar_init(bars + 8 * (P_V_FULL + s), 1);
      mbar_init(bars + 8 * (P_V_EMPTY + s), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(bars + 8 * (P_S_FULL + h), 1);
      mbar_init(bars + 8 * (P_P_FULL + h), 4);   // one arrival a softmax warp
      mbar_init(bars + 8 * (P_O_FULL + h), 1);
      mbar_init(bars + 8 * (P_Q_FULL + h), 4);
    }
    mbar_init(bars + 8 * P_HALF, 4);
    mbar_init(bars + 8 * P_DRAIN, 1);
    *abort_flag = 0;
    *longest_s = 0;
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == TMA_WARP && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // The set-up above touches no global memory, so it may overlap the end of
  // the previous grid of the stream; nothing below runs before that grid is done.
  // (Behind a shared prefix: see attn_paged_kernel.)
  const bool late = p.shared_tiles > 0 && !p.prefix;
  if (!late) grid_dependency_wait();
  grid_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int HR = p.H_kv * p.row_tiles;
  const PdSum sum = pd_sum<NUM_THREADS>(p, part, nullptr);
  if (p.prefix) {
    int n = 0;
    for (int b = threadIdx.x; b < p.B; b += NUM_THREADS) n = max(n, pd_len_of(p, b));
    n = __reduce_max_sync(0xffffffffu, n);
    if (lane == 0) atomicMax(longest_s, n);
  }
  if (warp == NUM_THREADS / 32 - 1) pd_report_lens(p);
  const PdCut cut = p.prefix ? pd_cut_prefix(p, sum.ranges) : pd_cut(sum.total * HR, sum.ranges);
  const bool any = static_cast<int>(blockIdx.x) < cut.n;
  PdWalk w;
  const int f0 = any ? pd_start(cut, blockIdx.x) : 0;
  if (any) {
    w.x = f0;
    w.end = pd_start(cut, blockIdx.x + 1);
    pd_locate<NUM_THREADS>(p, sum, w.x / HR, part, w.b, w.base);
    w.base *= HR;
    w.s = pd_seq(p, pd_len_of(p, w.b));
    pd_run_here(p, w);
  }
  __syncthreads();
  const int longest = *longest_s;
  if (warp < 8) {
    regs_increase<SOFTMAX_REGS>();
    if (any)
      pt_softmax_role<D, PAIR, BF16, OUT_F32>(p, w, f0, tmem, smem, sbase, bars, warp / 4, warp % 4, lane,
                                              longest, abort_flag);
    tc_fence_before_sync();
    __syncthreads();
  } else {
    regs_decrease<CONTROL_REGS>();
    if (any) {
      if (warp == MMA_WARP) {
        pt_mma_role<D, PAIR, BF16>(p, w, tmem, sbase, bars, abort_flag);
      } else if (warp == TMA_WARP) {
        pt_tma_role<D, PAIR>(p, w, &tmK, &tmV, sbase, bars, lane, abort_flag);
      }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, TMEM_COLS);
      if (late && blockIdx.x + 1 == gridDim.x) grid_dependency_wait();
    }
  }
}

}  // namespace attn
