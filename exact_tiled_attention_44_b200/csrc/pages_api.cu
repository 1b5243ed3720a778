// pages_api.cu -- management of a paged K/V cache: attn_pages_append,
// attn_pages_trim, attn_pages_fork, attn_pages_compact, attn_pages_copy and
// their workspace queries.
#include "host.h"
#include "pages_kernel.cuh"

namespace attn_host {

namespace {

bool page_size_taken(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

}  // namespace

int validate_pages(const attn_pages_t* c, bool need_refs) {
  if (c == nullptr) return ATTN_ERR_INVALID_ARG;
  if (c->dtype != ATTN_BF16 && c->dtype != ATTN_FP16) return ATTN_ERR_INVALID_ARG;
  if (c->B < 0 || c->n_pages < 0 || c->max_pages < 0 || c->H_kv < 1 || c->d <= 0 || c->page_size <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (c->d != 16 && c->d != 32 && c->d != 64 && c->d != 128) return ATTN_ERR_UNSUPPORTED;
  const int ps = c->page_size;
  if (!page_size_taken(ps)) return ATTN_ERR_UNSUPPORTED;
  // page * H_kv + head, and sums of two positions, are 32-bit
  if (static_cast<long long>(c->n_pages) * c->H_kv > INT32_MAX ||
      static_cast<long long>(c->max_pages) * ps > (1 << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (c->n_pages > 0 && (c->k == nullptr || c->v == nullptr || (need_refs && c->refs == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (c->B > 0 && (c->lens == nullptr || (c->max_pages > 0 && c->table == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned_to(c->table, 4) || !aligned_to(c->lens, 4) ||
      !aligned_to(c->refs, 4))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

namespace {

int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

size_t page_bytes(const attn_pages_t* c) {
  return static_cast<size_t>(c->H_kv) * c->page_size * c->d * 2;
}

attn::Pages device_pages(const attn_pages_t* c, int* status) {
  attn::Pages p{};
  p.k = static_cast<uint8_t*>(c->k);
  p.v = static_cast<uint8_t*>(c->v);
  p.table = c->table;
  p.lens = c->lens;
  p.refs = c->refs;
  p.n_pages = c->n_pages;
  p.H_kv = c->H_kv;
  p.page_size = c->page_size;
  p.page_shift = shift_of(c->page_size);
  p.B = c->B;
  p.max_pages = c->max_pages;
  p.row_bytes = c->d * 2;
  p.page_bytes = static_cast<long long>(page_bytes(c));
  p.status = status;
  return p;
}

// The management calls need every array, and none of them inside another.
int validate_managed(const attn_pages_t* c) {
  int rc = validate_pages(c, true);
  if (rc != ATTN_OK) return rc;
  const size_t kv = page_bytes(c) * c->n_pages;
  const size_t tab = static_cast<size_t>(c->B) * c->max_pages * 4, len = static_cast<size_t>(c->B) * 4;
  const size_t ref = static_cast<size_t>(c->n_pages) * 4;
  const struct { const void* p; size_t n; } a[5] = {
      {c->k, kv}, {c->v, kv}, {c->table, tab}, {c->lens, len}, {c->refs, ref}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (a[i].n != 0 && a[j].n != 0 && overlaps(a[i].p, a[i].n, a[j].p, a[j].n))
        return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Whether `n` bytes at `ptr` touch any array of the cache.
bool touches(const attn_pages_t* c, const void* ptr, size_t n) {
  if (n == 0) return false;
  const size_t kv = page_bytes(c) * c->n_pages;
  return (kv != 0 && (overlaps(ptr, n, c->k, kv) || overlaps(ptr, n, c->v, kv) ||
                      overlaps(ptr, n, c->refs, static_cast<size_t>(c->n_pages) * 4))) ||
         (c->B > 0 && (overlaps(ptr, n, c->table, static_cast<size_t>(c->B) * c->max_pages * 4) ||
                       overlaps(ptr, n, c->lens, static_cast<size_t>(c->B) * 4)));
}

template <typename... Params, typename... Args>
int launch(void (*kern)(Params...), long long grid, int block, cudaStream_t s, Args&&... args) {
  const cudaError_t e = launch_overlapped(kern, static_cast<int>(grid), block, 0, s, std::forward<Args>(args)...);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Pages n_new rows can need at most: the boundaries they reach, and a copied page.
long long max_need(int n_new, int page_size) { return n_new / page_size + 2; }

// CTAs of the kernels that move whole pages: eight on every SM (the most that
// 256-thread CTAs reach), each looping over chunks.
long long mover_grid(const DeviceState* st, long long work) {
  const long long most = 8ll * st->sm_count;
  return work < 1 ? 1 : (work < most ? work : most);
}

}  // namespace

}  // namespace attn_host

using namespace attn_host;

extern "C" {

long long attn_pages_append_workspace_bytes(int B, int n_new, int page_size) {
  if (B < 0 || n_new < 0 || !page_size_taken(page_size)) return -1;
  if (B * max_need(n_new, page_size) > INT32_MAX) return -1;   // more pages than the call counts
  const long long ints = 6ll * B + B * max_need(n_new, page_size);
  return static_cast<long long>(round_up(static_cast<size_t>(ints) * 4, 256));
}

int attn_pages_append(const attn_pages_t* c, const void* k_new, const void* v_new, const int* counts,
                      int n_new, void* workspace, long long workspace_bytes, void* stream) {
  int rc = validate_managed(c);
  if (rc != ATTN_OK) return rc;
  if (n_new < 0 || workspace_bytes < 0) return ATTN_ERR_INVALID_ARG;
  if (c->B == 0 || n_new == 0) return ATTN_OK;
  if (k_new == nullptr || v_new == nullptr || workspace == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(workspace) || !aligned_to(counts, 4))
    return ATTN_ERR_MISALIGNED;
  const long long need = attn_pages_append_workspace_bytes(c->B, n_new, c->page_size);
  const long long bh = static_cast<long long>(c->B) * c->H_kv;
  const long long row_tiles = (static_cast<long long>(n_new) + attn::PG_ROWS - 1) / attn::PG_ROWS;
  if (need < 0 || bh > INT32_MAX || bh * (row_tiles + 1) > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  const size_t new_bytes = static_cast<size_t>(bh) * n_new * c->d * 2;
  if (touches(c, workspace, need) || touches(c, k_new, new_bytes) || touches(c, v_new, new_bytes) ||
      overlaps(workspace, need, k_new, new_bytes) || overlaps(workspace, need, v_new, new_bytes))
    return ATTN_ERR_INVALID_ARG;
  if (counts != nullptr) {
    const size_t n = static_cast<size_t>(c->B) * 4;
    if (touches(c, counts, n) || overlaps(workspace, need, counts, n)) return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const attn::Pages p = device_pages(c, st->status);
  int* w = static_cast<int*>(workspace);
  const size_t B = c->B;
  const attn::AppendPlan a{w, w + B, w + 2 * B, w + 3 * B, w + 4 * B, w + 5 * B, w + 6 * B};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch(attn::attn_pages_append_plan, 1, attn::PG_PLAN_THREADS, s, p, a, counts, n_new);
  if (rc != ATTN_OK) return rc;
  return launch(attn::attn_pages_append_rows, bh * (row_tiles + 1), attn::PG_THREADS, s, p, a,
                static_cast<const uint8_t*>(k_new), static_cast<const uint8_t*>(v_new), n_new,
                static_cast<int>(row_tiles), bh * row_tiles);
}

int attn_pages_trim(const attn_pages_t* c, const int* rows, const int* new_lens, int n, void* stream) {
  int rc = validate_managed(c);
  if (rc != ATTN_OK) return rc;
  if (n < 0 || (rows == nullptr && n > c->B)) return ATTN_ERR_INVALID_ARG;
  if (n == 0 || c->B == 0) return ATTN_OK;
  if (!aligned_to(rows, 4) || !aligned_to(new_lens, 4)) return ATTN_ERR_MISALIGNED;
  const size_t bytes = static_cast<size_t>(n) * 4;
  if ((rows != nullptr && touches(c, rows, bytes)) || (new_lens != nullptr && touches(c, new_lens, bytes)))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  return launch(attn::attn_pages_trim_kernel, n, 128, static_cast<cudaStream_t>(stream),
                device_pages(c, st->status), rows, new_lens);
}

int attn_pages_fork(const attn_pages_t* c, const int* parents, const int* children, int n, void* stream) {
  int rc = validate_managed(c);
  if (rc != ATTN_OK) return rc;
  if (n < 0) return ATTN_ERR_INVALID_ARG;
  if (n == 0 || c->B == 0) return ATTN_OK;
  if (parents == nullptr || children == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned_to(parents, 4) || !aligned_to(children, 4)) return ATTN_ERR_MISALIGNED;
  const size_t bytes = static_cast<size_t>(n) * 4;
  if (touches(c, parents, bytes) || touches(c, children, bytes)) return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  return launch(attn::attn_pages_fork_kernel, n, 128, static_cast<cudaStream_t>(stream),
                device_pages(c, st->status), parents, children, n);
}

long long attn_pages_compact_workspace_bytes(int n_pages) {
  if (n_pages < 0) return -1;
  return static_cast<long long>(round_up((3 * static_cast<size_t>(n_pages) + 4) * 4, 256));
}

int attn_pages_compact(const attn_pages_t* c, int* table_out, int* refs_out, int* n_live,
                       void* workspace, long long workspace_bytes, void* stream) {
  int rc = validate_managed(c);
  if (rc != ATTN_OK) return rc;
  if (workspace_bytes < 0 || workspace == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(workspace) || !aligned_to(table_out, 4) || !aligned_to(refs_out, 4) || !aligned_to(n_live, 4))
    return ATTN_ERR_MISALIGNED;
  const long long need = attn_pages_compact_workspace_bytes(c->n_pages);
  if (workspace_bytes < need || touches(c, workspace, need)) return ATTN_ERR_INVALID_ARG;
  const size_t tab = static_cast<size_t>(c->B) * c->max_pages * 4, ref = static_cast<size_t>(c->n_pages) * 4;
  if (table_out == nullptr) table_out = c->table;
  if (refs_out == nullptr) refs_out = c->refs;
  // a second table or array of counts lies apart from everything else
  const struct { const void* p; size_t n; bool own; } out[3] = {
      {table_out, tab, table_out == c->table}, {refs_out, ref, refs_out == c->refs}, {n_live, 4, n_live == nullptr}};
  for (int i = 0; i < 3; ++i) {
    if (out[i].own || out[i].n == 0) continue;
    if (touches(c, out[i].p, out[i].n) || overlaps(out[i].p, out[i].n, workspace, need))
      return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (!out[j].own && out[j].n != 0 && overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const attn::Pages p = device_pages(c, st->status);
  int* w = static_cast<int*>(workspace);
  const size_t n = c->n_pages;
  const attn::CompactPlan a{w, w + 1, w + 4, w + 4 + n, w + 4 + 2 * n};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch(attn::attn_pages_compact_plan, 1, attn::PG_PLAN_THREADS, s, p, a, n_live);
  if (rc != ATTN_OK) return rc;
  const int chunks = static_cast<int>((page_bytes(c) + attn::PG_CHUNK - 1) / attn::PG_CHUNK);
  const long long most = static_cast<long long>(n / 2) * 2 * chunks;   // no more than half the pages move
  const long long cells = (static_cast<long long>(c->B) * c->max_pages + static_cast<long long>(n)) / attn::PG_THREADS + 1;
  return launch(attn::attn_pages_compact_move, mover_grid(st, most > cells ? most : cells), attn::PG_THREADS, s,
                p, a, table_out, refs_out, chunks);
}

int attn_pages_copy(const attn_pages_t* c, const int* src, const int* dst, int n, void* stream) {
  int rc = validate_managed(c);
  if (rc != ATTN_OK) return rc;
  if (n < 0) return ATTN_ERR_INVALID_ARG;
  if (n == 0) return ATTN_OK;
  if (src == nullptr || dst == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned_to(src, 4) || !aligned_to(dst, 4)) return ATTN_ERR_MISALIGNED;
  const size_t bytes = static_cast<size_t>(n) * 4;
  if (touches(c, src, bytes) || touches(c, dst, bytes)) return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const int chunks = static_cast<int>((page_bytes(c) + attn::PG_CHUNK - 1) / attn::PG_CHUNK);
  const long long work = static_cast<long long>(n) * 2 * chunks;
  return launch(attn::attn_pages_copy_kernel, mover_grid(st, work), attn::PG_THREADS,
                static_cast<cudaStream_t>(stream), device_pages(c, st->status), src, dst, n, chunks);
}

}  // extern "C"
