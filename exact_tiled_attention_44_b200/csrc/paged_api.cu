// paged_api.cu -- the decoding step over a K/V cache of pages:
// attn_decode_paged and its workspace query.
#include "host.h"
#include "paged_tc_kernel.cuh"

namespace attn_host {

namespace {

constexpr int kPagedMaxRows = 1024;   // (H / H_kv) * N_q

// Whether the kernels are built for d, and the rows of a K/V head and of the
// batch are within their limits (H a multiple of H_kv, nothing negative).
bool paged_sizes_taken(int B, int H, int H_kv, int N_q, int d) {
  const long long R = static_cast<long long>(H / H_kv) * N_q;
  return (d == 64 || d == 128) && R <= kPagedMaxRows && B * R <= INT32_MAX / 2 / H_kv;
}

constexpr int kSharedUnit = 128;      // the shared prefix is attended in whole tiles of this many positions

// How the `rows` query rows of a sequence (or, in a shared prefix, of the
// batch) and K/V head are attended: rows of a group, groups, positions of a
// tile, ranges of the tile space.  The ranges are one CTA (of
// attn_paged_tc_kernel) or two (of attn_paged_kernel) on each SM of a B200;
// fixed, so that the workspace can be sized without a device.
struct PagedForm {
  int m, row_tiles, tile_shift, ranges;
  int weight, own_weight;   // of a tile, in a prefix and in the launch beside it (see paged_form)
};

// Up to 16 rows attn_paged_kernel, whose products are of 8 rows, d = 128: at 4
// rows 8 sequences of up to 8192 take 33 us (with attn_paged_tc_kernel's 128-row
// products 42), 32 of up to 16384 186 (205), 256 of up to 256 46 (150), one of 517
// 7.8 (12.8); at 16 rows the first 47 (46), 64 of up to 256 39 (48).
//
// At d = 64, where a 128-row tile's softmax takes longer than HBM does, up to 32
// rows in two groups, unless `wide` (see paged_wide); at d = 128 two groups take 67
// us (47).
//
// The weights share out the SMs between a prefix and the sequences' own positions
// (pd_prefix_ranges): 100 cycles of an SM a tile, the own ones with their share of a
// run's fixed cost.  Swept at both d: us at 0.7, 1 and 1.5 times the own weight, for
// the rows of a sequence and of the prefix (16384 positions):
//   4 and 512: d = 64 89, 90, 91; d = 128 117, 117, 115
//   4 and 96: 51, 45, 50; 70, 61, 66
//   16 and 128: 53, 45, 48; 62, 63, 68 (at 7, as 8 rows have it: 50; 78)
//   64 and 1024: 124, 119, 119; 155, 139, 139 (at 21, as the prefix has it: 124; 155)
PagedForm paged_form(long long rows, int d, bool wide) {
  PagedForm f;
  f.m = rows <= 8 ? 8 : rows <= 16 || (d == 64 && rows <= 32 && !wide) ? 16 : rows <= 128 ? 128 : 256;
  f.row_tiles = static_cast<int>((rows + f.m - 1) / f.m);
  f.tile_shift = f.m <= 16 ? 6 : 7;
  f.ranges = f.m <= 16 ? 296 : 148;
  f.weight = f.m <= 128 ? 21 : 42;      // a prefix of 16 rows or fewer takes all SMs
  f.own_weight = f.m == 8 ? 7 : f.m == 16 ? (d == 64 ? 9 : 12) : f.m == 128 ? 25 : 42;
  return f;
}

// Whether, at d = 64, 17 to 32 rows are one group of attn_paged_tc_kernel and not
// two of attn_paged_kernel.  The second group reads a sequence's tiles again when the
// first is through with them: from L2 if the sequences are few or short, else from
// HBM.  The lengths are on the device, so what table, window and pages allow at most
// decides: 16384 positions a sequence, and 128 MB of K and V.  Two groups (one), us,
// at 32 rows of each of 8 K/V heads and tables as wide as the longest sequence:
//   65536 positions: 4 sequences 140 (112)
//   16384: 4 sequences (93 MB) 44.7 (46.6), 8 (172 MB) 73.5 (67.4), 16 115 (108), 32 (637 MB) 223 (190)
//   8192: 8 sequences 45.1 (46.9), 16 69.2 (69.6), 32 117 (117), 64 (630 MB) 229 (203)
//   4096: 64 sequences 132 (131), 128 224 (222); 2000: 32 47 (57), 256 (604 MB) 230 (250)
//   1000: 512 sequences 265 (307); 256: 64 45 (45), 256 98 (113)
// 20 rows differ from that by 5% at most.  Short sequences in wide tables pay what
// the 2000 and 256 show.  A prefix's length is known, and its tiles are those of one
// sequence: of 16384 positions (34 MB) 34 us (34), 32768 47.0 (49.8), 65536 (134 MB)
// 63.8 (55.1), 262144 197 (151).
constexpr long long kBeyondL2 = 128ll << 20;

bool paged_wide(const attn_pages_t* kv, int N_q, int window, int n_sink, int shared_len) {
  const long long cap = static_cast<long long>(kv->max_pages) * kv->page_size;
  const bool all_seen = window == 0 || window >= cap;
  const long long seen = all_seen ? cap - shared_len : static_cast<long long>(window) + n_sink + N_q;
  const long long each = seen < cap ? seen : cap, pool = static_cast<long long>(kv->n_pages) * kv->page_size;
  const long long all = kv->B * each < pool ? kv->B * each : pool;
  return each >= 16384 && all * kv->H_kv * kv->d * 4 >= kBeyondL2;
}

// Workspace of one attending launch over `groups` groups: two slots a range
// for the runs of split groups, and, behind or of a shared prefix, one result
// for each group that a single run covers.
struct PagedSpace {
  size_t part_o, part_lse, own_o, own_lse, end;
};

PagedSpace paged_space(size_t at, const PagedForm& f, size_t groups, int d) {
  const size_t rows = size_t(2) * f.ranges * f.m, own = groups * f.m;
  PagedSpace s;
  s.part_o = at;
  s.part_lse = s.part_o + rows * d * 4;
  s.own_o = round_up(s.part_lse + rows * 4, 256);
  s.own_lse = s.own_o + own * d * 4;
  s.end = round_up(s.own_lse + own * 4, 256);
  return s;
}

struct PagedPlan {
  bool shared;
  PagedForm form, prefix_form;
  PagedSpace own, prefix;
  size_t bytes;
};

PagedPlan paged_plan(int B, int H, int H_kv, int N_q, int d, int shared_len, bool wide) {
  PagedPlan pl{};
  const long long R = static_cast<long long>(H / H_kv) * N_q;
  pl.shared = shared_len >= kSharedUnit;
  const auto own = [&](const PagedForm& f) {
    return paged_space(0, f, pl.shared ? static_cast<size_t>(B) * H_kv * f.row_tiles : 0, d);
  };
  pl.form = paged_form(R, d, wide);
  pl.own = own(pl.form);
  // the workspace is sized without the table, for either form (a wide one's is no smaller)
  pl.own.end = own(paged_form(R, d, true)).end;
  pl.bytes = pl.own.end;
  if (pl.shared) {
    pl.prefix_form = paged_form(B * R, d, shared_len >= kBeyondL2 / (4ll * H_kv * d));
    pl.prefix = paged_space(pl.own.end, pl.prefix_form, static_cast<size_t>(H_kv) * pl.prefix_form.row_tiles, d);
    pl.bytes = pl.prefix.end;
  }
  return pl;
}

// 4-D view [z][d / 64][page_size][64] of the pages of one K/V head each (z =
// page * H_kv + head); one box is a slice of PD_SLICE rows, its 64-column
// chunks one behind the other, in the 128-byte swizzle.
int encode_pages(CUtensorMap* map, const void* base, bool bf16, int d, int page_size, int z) {
  const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(d / 64),
                              static_cast<cuuint64_t>(z)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, 128u, static_cast<cuuint64_t>(page_size) * d * 2};
  const cuuint32_t box[4] = {64u, attn::PD_SLICE, static_cast<cuuint32_t>(d / 64), 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// 5-D view [z][page_size / 8][d / 64][8][64] of the same; a box is as many
// groups of 8 rows as a page and a tile of attn_paged_tc_kernel have in common.
int encode_boxes(CUtensorMap* map, const void* base, bool bf16, int d, int page_size, int z) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t dims[5] = {64u, 8u, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(page_size / 8),
                              static_cast<cuuint64_t>(z)};
  const cuuint64_t strides[4] = {row, 128u, 8 * row, page_size * row};
  const int rows = page_size < attn::PT_TILE ? page_size : attn::PT_TILE;
  const cuuint32_t box[5] = {64u, 8u, static_cast<cuuint32_t>(d / 64), static_cast<cuuint32_t>(rows / 8), 1u};
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  const CUresult r = g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

int counted(cudaError_t e) {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Sets a kernel's shared memory on its first launch on the device; `regs`:
// the registers a thread it has to be launched with (it re-splits them).
template <typename Kern>
int prepare_kernel(DeviceState* st, Kern kern, uint32_t bit, int smem, int regs) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (st->paged_attr_set & bit) return ATTN_OK;
  if (regs > 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return ATTN_ERR_CUDA;
    if (fa.numRegs < regs) return ATTN_ERR_UNSUPPORTED;
  }
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  st->paged_attr_set |= bit;
  return ATTN_OK;
}

// One attending launch: the kernel for dp.m query rows a group.
template <int D, bool BF16, bool F32>
int attend(DeviceState* st, const attn::PdParams& dp, const attn_pages_t* kv, cudaStream_t stream) {
  alignas(64) CUtensorMap mk, mv;
  const int z = dp.n_pages * dp.H_kv;
  const auto encode = dp.m <= 16 ? encode_pages : encode_boxes;
  if (encode(&mk, kv->k, BF16, D, kv->page_size, z) != ATTN_OK ||
      encode(&mv, kv->v, BF16, D, kv->page_size, z) != ATTN_OK)
    return ATTN_ERR_CUDA;
  const auto go = [&](auto kern, int form, int smem, int regs, int threads) {
    const uint32_t bit = 1u << (form * 8 + (D == 128 ? 4 : 0) + (BF16 ? 2 : 0) + (F32 ? 1 : 0));
    const int rc = prepare_kernel(st, kern, bit, smem, regs);
    if (rc != ATTN_OK) return rc;
    return counted(launch_overlapped(kern, dp.ranges, threads, smem, stream, mk, mv, dp));
  };
  switch (dp.m) {
    case 8:
      return go(attn::attn_paged_kernel<D, 1, BF16, F32>, 0, attn::PdGeo<D, 1>::SMEM_BYTES + 1024, 0, attn::PD_THREADS);
    case 16:
      return go(attn::attn_paged_kernel<D, 2, BF16, F32>, 1, attn::PdGeo<D, 2>::SMEM_BYTES + 1024, 0, attn::PD_THREADS);
    case 128:
      return go(attn::attn_paged_tc_kernel<D, false, BF16, F32>, 2, attn::PtGeo<D, false>::SMEM_BYTES + 1024,
                attn::LAUNCH_REGS, attn::NUM_THREADS);
    default:
      return go(attn::attn_paged_tc_kernel<D, true, BF16, F32>, 3, attn::PtGeo<D, true>::SMEM_BYTES + 1024,
                attn::LAUNCH_REGS, attn::NUM_THREADS);
  }
}

template <int D, bool BF16, bool F32>
int launch_paged(DeviceState* st, const attn::PdParams& dp, const attn::PdParams* pre, const attn_pages_t* kv,
                 cudaStream_t stream) {
  int rc = ATTN_OK;
  if (pre != nullptr) rc = attend<D, BF16, F32>(st, *pre, kv, stream);
  if (rc == ATTN_OK) rc = attend<D, BF16, F32>(st, dp, kv, stream);
  if (rc != ATTN_OK) return rc;
  if (pre != nullptr) {
    // a CTA for as many rows as it takes at once, four CTAs on an SM at most
    const int at_once = attn::PD_MERGE / (D / 4), rows = dp.B * dp.H * dp.N_q;
    const int grid = (rows + at_once - 1) / at_once;
    return counted(launch_overlapped(attn::attn_paged_merge_shared<D, BF16, F32>, grid < 592 ? grid : 592,
                                     attn::PD_MERGE, 0, stream, dp, *pre));
  }
  // groups of many rows are merged by several CTAs a boundary
  const int subs = dp.m <= 16 ? 1 : dp.m / 16;
  return counted(launch_overlapped(attn::attn_paged_merge<D, BF16, F32>, dp.ranges * subs, attn::PD_MERGE, 0, stream,
                                   dp, subs));
}

}  // namespace

}  // namespace attn_host

using namespace attn_host;

extern "C" {

long long attn_decode_paged_workspace_bytes(int B, int H, int H_kv, int N_q, int d, int shared_len) {
  if (B < 0 || H < 0 || H_kv < 1 || N_q < 0 || d <= 0 || shared_len < 0) return -1;
  if (B == 0 || H == 0 || N_q == 0) return 0;
  if (H % H_kv != 0 || !paged_sizes_taken(B, H, H_kv, N_q, d)) return -1;
  return static_cast<long long>(paged_plan(B, H, H_kv, N_q, d, shared_len, false).bytes);
}

int attn_decode_paged(const void* q, const attn_pages_t* kv, void* o, float* lse, const int* shared_table,
                      int shared_len, void* workspace, long long workspace_bytes, int H, int N_q, int causal,
                      int window, int n_sink, float scale, int out_f32, void* stream) {
  int rc = validate_pages(kv, false);
  if (rc != ATTN_OK) return rc;
  if (H < 0 || N_q < 0 || shared_len < 0 || workspace_bytes < 0) return ATTN_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || (out_f32 != 0 && out_f32 != 1)) return ATTN_ERR_INVALID_ARG;
  if (window < 0 || n_sink < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (kv->B == 0 || H == 0 || N_q == 0) return ATTN_OK;
  const int B = kv->B, H_kv = kv->H_kv, d = kv->d;
  if (H % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if (window > 0 && !causal) return ATTN_ERR_UNSUPPORTED;
  if (!paged_sizes_taken(B, H, H_kv, N_q, d)) return ATTN_ERR_UNSUPPORTED;
  const long long R = static_cast<long long>(H / H_kv) * N_q;
  // the tiles of all groups are counted in 32 bits
  const long long most = static_cast<long long>(kv->max_pages) * kv->page_size;
  const long long tile_groups = (R + 15) / 16 * B * H_kv;
  if ((most + attn::PD_TILE) / attn::PD_TILE * tile_groups > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  if (kv->n_pages == 0) return ATTN_ERR_INVALID_ARG;
  if (q == nullptr || o == nullptr || workspace == nullptr) return ATTN_ERR_INVALID_ARG;
  if (shared_len > 0 && shared_table == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (lse != nullptr && !aligned16(lse)) ||
      !aligned_to(workspace, 256) || !aligned_to(shared_table, 4))
    return ATTN_ERR_MISALIGNED;
  const PagedPlan pl =
      paged_plan(B, H, H_kv, N_q, d, shared_len, paged_wide(kv, N_q, window, n_sink, shared_len));
  if (static_cast<size_t>(workspace_bytes) < pl.bytes) return ATTN_ERR_INVALID_ARG;
  // no output inside an input, the workspace or another output
  const size_t rows = static_cast<size_t>(B) * H * N_q;
  const size_t kv_bytes = static_cast<size_t>(kv->n_pages) * H_kv * kv->page_size * d * 2;
  const struct { const void* p; size_t n; } out[3] = {
      {o, rows * d * (out_f32 ? 4 : 2)}, {lse, lse != nullptr ? rows * 4 : 0}, {workspace, pl.bytes}};
  const struct { const void* p; size_t n; } in[6] = {
      {q, rows * d * 2}, {kv->k, kv_bytes}, {kv->v, kv_bytes},
      {kv->table, static_cast<size_t>(B) * kv->max_pages * 4}, {kv->lens, static_cast<size_t>(B) * 4},
      {shared_table, (static_cast<size_t>(shared_len) + kv->page_size - 1) / kv->page_size * 4}};
  for (int i = 0; i < 3; ++i) {
    if (out[i].n == 0) continue;
    for (int j = 0; j < 6; ++j)
      if (in[j].n != 0 && overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[j].n != 0 && overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const bool bf16 = kv->dtype == ATTN_BF16;
  attn::PdParams dp{};
  dp.q = q;
  dp.o = o;
  dp.lse = lse;
  dp.table = kv->table;
  dp.lens = kv->lens;
  dp.status = st->status;
  dp.watchdog_ns = g_watchdog_ns.load(std::memory_order_relaxed);
  dp.B = B;
  dp.H = H;
  dp.H_kv = H_kv;
  dp.N_q = N_q;
  dp.n_pages = kv->n_pages;
  dp.max_pages = kv->max_pages;
  for (dp.page_shift = 4; (1 << dp.page_shift) < kv->page_size;) ++dp.page_shift;
  dp.causal = causal;
  const long long cap = static_cast<long long>(kv->max_pages) << dp.page_shift;
  dp.window = window >= cap ? 0 : window;      // no row has that many positions before it
  dp.n_sink = dp.window > 0 ? (n_sink < cap ? n_sink : static_cast<int>(cap)) : 0;
  dp.scale_log2 = scale * 1.4426950408889634f;
  dp.G = H / H_kv;
  dp.R = static_cast<int>(R);
  dp.withhold_loads = take_withhold();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const auto place = [&](attn::PdParams& x, const PagedForm& f, const PagedSpace& s) {
    x.m = f.m;
    x.row_tiles = f.row_tiles;
    x.tile_shift = f.tile_shift;
    x.ranges = f.ranges;
    x.part_o = reinterpret_cast<float*>(ws + s.part_o);
    x.part_lse = reinterpret_cast<float*>(ws + s.part_lse);
    x.own_o = reinterpret_cast<float*>(ws + s.own_o);
    x.own_lse = reinterpret_cast<float*>(ws + s.own_lse);
  };
  place(dp, pl.form, pl.own);
  attn::PdParams pre = dp;
  // Whole tiles of the prefix are attended once whenever the caller names one.  That
  // costs a third launch and a merge of every row, and pays, at 4 rows of each of 8 K/V
  // heads, 500 positions of their own and d = 128, from about 1024 positions at 32
  // sequences on (22 us shared, 22 not; 4096: 25, 46) and at 128 (59, 62; 4096: 60,
  // 156; 128: 59, 35); at 8 not yet at 4096 (23, 19), nor at 2 (21, 12).  The header
  // says so, and leaves the choice to the caller.  A window moves with each
  // row, so under one (that masks anything: see dp.window) every sequence reads
  // its own pages
  const int units = static_cast<int>((shared_len < cap ? shared_len : cap) / kSharedUnit);
  const bool shared = units > 0 && dp.window == 0;
  if (shared) {
    pre.prefix = 1;
    pre.table = shared_table;
    place(pre, pl.prefix_form, pl.prefix);
    pre.shared_tiles = (units * kSharedUnit) >> pre.tile_shift;
    dp.shared_tiles = (units * kSharedUnit) >> dp.tile_shift;
    pre.weight = pl.prefix_form.weight;
    pre.own_weight = pl.form.own_weight;
    pre.own_groups = H_kv * dp.row_tiles;
    pre.own_tile_shift = dp.tile_shift;
    pre.own_shared_tiles = dp.shared_tiles;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const attn::PdParams* pp = shared ? &pre : nullptr;
  if (d == 128) {
    if (bf16) return out_f32 ? launch_paged<128, true, true>(st, dp, pp, kv, s)
                             : launch_paged<128, true, false>(st, dp, pp, kv, s);
    return out_f32 ? launch_paged<128, false, true>(st, dp, pp, kv, s)
                   : launch_paged<128, false, false>(st, dp, pp, kv, s);
  }
  if (bf16) return out_f32 ? launch_paged<64, true, true>(st, dp, pp, kv, s)
                           : launch_paged<64, true, false>(st, dp, pp, kv, s);
  return out_f32 ? launch_paged<64, false, true>(st, dp, pp, kv, s)
                 : launch_paged<64, false, false>(st, dp, pp, kv, s);
}

}  // extern "C"
