// C ABI of the paged 8-bit key/value cache: argument checks, workspace layout, launches.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <climits>

#include "csa.h"
#include "paged.h"

using namespace csa;

namespace {

csa_status_t fail(csa_status_t st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(st, buf);
}

csa_status_t cuda_fail(cudaError_t e, const char* where) {
  return fail(CSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

csa_status_t need_ptr(const void* p, const char* name, size_t align = 16) {
  if (!p) return fail(CSA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align) return fail(CSA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
  return CSA_OK;
}

#define CSA_TRY(x)                     \
  do {                                 \
    csa_status_t _st = (x);            \
    if (_st != CSA_OK) return _st;     \
  } while (0)

constexpr int64_t kMaxPos = (int64_t)1 << 30;

csa_status_t check_gqa(const csa_gqa_t* L) {
  if (!L) return fail(CSA_ERR_INVALID_ARG, "layer is NULL");
  if (L->H < 1 || L->Hkv < 1 || L->H % L->Hkv) return fail(CSA_ERR_INVALID_ARG, "H=%d Hkv=%d", L->H, L->Hkv);
  if (L->Hkv > 1024 || L->H > 16384) return fail(CSA_ERR_UNSUPPORTED, "H=%d Hkv=%d (at most 16384, 1024)", L->H, L->Hkv);
  if (L->D != 64 && L->D != 128) return fail(CSA_ERR_UNSUPPORTED, "D=%d (64 or 128)", L->D);
  if (L->act_format != CSA_FMT_F32 && L->act_format != CSA_FMT_BF16)
    return fail(CSA_ERR_INVALID_ARG, "act_format=%d", L->act_format);
  if (L->window < 0 || L->first < 0) return fail(CSA_ERR_INVALID_ARG, "window=%d first=%d", L->window, L->first);
  if (L->first > 0 && L->window == 0) return fail(CSA_ERR_INVALID_ARG, "first=%d without a window", L->first);
  if (!(L->softmax_scale >= 0) || std::isinf(L->softmax_scale)) return fail(CSA_ERR_INVALID_ARG, "softmax_scale");
  if (L->reserved != 0) return fail(CSA_ERR_INVALID_ARG, "reserved must be 0");
  return CSA_OK;
}

csa_status_t check_table_shape(const csa_page_table_t* T) {
  if (!T) return fail(CSA_ERR_INVALID_ARG, "page table is NULL");
  if (T->B < 1) return fail(CSA_ERR_INVALID_ARG, "B=%d", T->B);
  if (T->page != 16 && T->page != 32 && T->page != 64 && T->page != 128)
    return fail(CSA_ERR_UNSUPPORTED, "page=%d (16, 32, 64 or 128)", T->page);
  if (T->table_cap < 1 || T->table_cap > INT_MAX) return fail(CSA_ERR_INVALID_ARG, "table_cap=%lld", (long long)T->table_cap);
  if (T->n_pages < 1 || T->n_pages > kMaxPos) return fail(CSA_ERR_INVALID_ARG, "n_pages=%lld", (long long)T->n_pages);
  return CSA_OK;
}

csa_status_t check_table(const csa_page_table_t* T, bool need_refs) {
  CSA_TRY(check_table_shape(T));
  CSA_TRY(need_ptr(T->table, "table", 4));                // a slice of rows is a table too
  if (need_refs || T->refs) CSA_TRY(need_ptr(T->refs, "refs"));
  return CSA_OK;
}

csa_status_t check_pool(const csa_page_pool_t* P) {
  if (!P) return fail(CSA_ERR_INVALID_ARG, "page pool is NULL");
  CSA_TRY(need_ptr(P->k, "pool.k"));
  CSA_TRY(need_ptr(P->v, "pool.v"));
  CSA_TRY(need_ptr(P->k_scale, "pool.k_scale"));
  CSA_TRY(need_ptr(P->v_scale, "pool.v_scale"));
  return CSA_OK;
}

csa_status_t check_stride(const csa_gqa_t* L, int64_t* stride, int64_t width, const char* name) {
  const int64_t esz = L->act_format == CSA_FMT_F32 ? 4 : 2;
  if (*stride == 0) *stride = width;
  if (*stride < width || *stride > ((int64_t)1 << 40) || *stride * esz % 16)
    return fail(CSA_ERR_INVALID_ARG, "%s=%lld (at least %lld, a multiple of 16 bytes)", name, (long long)*stride,
                (long long)width);
  return CSA_OK;
}

csa_status_t check_tokens(const int64_t* start, const int32_t* n_new, int32_t Tq) {
  CSA_TRY(need_ptr(start, "start", 8));
  if (n_new) CSA_TRY(need_ptr(n_new, "n_new", 4));
  if (Tq < 1 || Tq > (1 << 24)) return fail(CSA_ERR_INVALID_ARG, "Tq=%d", Tq);
  return CSA_OK;
}

PageArgs page_args(const csa_page_table_t* T) {
  PageArgs a;
  a.table = T->table;
  a.refs = T->refs;
  a.cap = T->table_cap;
  a.n_pages = T->n_pages;
  a.B = T->B;
  a.page = T->page;
  a.page_log2 = T->page == 16 ? 4 : T->page == 32 ? 5 : T->page == 64 ? 6 : 7;
  return a;
}

PoolArgs pool_args(const csa_page_pool_t* P) {
  PoolArgs a;
  a.k = static_cast<uint8_t*>(P->k);
  a.v = static_cast<uint8_t*>(P->v);
  a.ks = P->k_scale;
  a.vs = P->v_scale;
  return a;
}

TokenArgs token_args(const int64_t* start, const int32_t* n_new, int32_t Tq) {
  TokenArgs a;
  a.start = start;
  a.n_new = n_new;
  a.Tq = Tq;
  return a;
}

int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && known[dev].load(std::memory_order_relaxed) > 0)
    return known[dev].load(std::memory_order_relaxed);
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Checks shared by csa_paged_workspace_size and csa_paged_attend; fills the plan.
csa_status_t make_plan(const csa_gqa_t* L, const csa_page_table_t* T, int32_t Tq, int64_t n_max, PagedPlan* p) {
  CSA_TRY(check_gqa(L));
  CSA_TRY(check_table_shape(T));
  if (Tq < 1 || Tq > (1 << 24)) return fail(CSA_ERR_INVALID_ARG, "Tq=%d", Tq);
  if (n_max < 0 || n_max > kMaxPos || n_max > T->table_cap * T->page)
    return fail(CSA_ERR_INVALID_ARG, "n_max=%lld (at most the table's %lld tokens and 2^30)", (long long)n_max,
                (long long)(T->table_cap * T->page));
  const int64_t rows = (int64_t)Tq * (L->H / L->Hkv);
  if (rows > INT_MAX || (rows / 8 + 1) * T->B * L->Hkv > INT_MAX)
    return fail(CSA_ERR_UNSUPPORTED, "%lld query rows per KV head of %d sequences", (long long)rows, T->B);
  *p = paged_plan(L->act_format, T->B, L->H / L->Hkv, L->Hkv, L->D, Tq, num_sms());
  return CSA_OK;
}

// csa_paged_attend, or (join_only: no pool and no queries) its second launch alone.
csa_status_t attend(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T, const void* q,
                    int64_t q_stride, const float* sinks, const int64_t* start, const int32_t* n_new, int32_t Tq,
                    int64_t n_max, void* out, void* workspace, size_t ws_bytes, bool join_only, void* stream) {
  PagedPlan p;
  CSA_TRY(make_plan(L, T, Tq, n_max, &p));
  CSA_TRY(check_table(T, false));
  if (!join_only) {
    CSA_TRY(check_pool(pool));
    CSA_TRY(need_ptr(q, "q"));
    CSA_TRY(check_stride(L, &q_stride, (int64_t)L->H * L->D, "q_stride"));
  }
  if (sinks) CSA_TRY(need_ptr(sinks, "sinks", 4));
  CSA_TRY(check_tokens(start, n_new, Tq));
  CSA_TRY(need_ptr(out, "out"));
  if (!workspace) return fail(CSA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", p.total);
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(CSA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < p.total) return fail(CSA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, p.total);
  if (n_max == 0) return CSA_OK;
  PagedAttendArgs a;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.T = page_args(T);
  a.P = join_only ? PoolArgs{} : pool_args(pool);
  a.tok = token_args(start, n_new, Tq);
  a.H = L->H; a.Hkv = L->Hkv; a.G = L->H / L->Hkv; a.D = L->D; a.act_fmt = L->act_format;
  // no position is n_max or more: a longer window shows the same keys, and keeps the kernels' sums within int32
  a.window = L->window < n_max ? L->window : (int)n_max;
  a.first = L->first;
  a.scale_log2 = (L->softmax_scale > 0 ? L->softmax_scale : 1.0f / sqrtf((float)L->D)) * kLog2e;
  a.n_max = (int)n_max;
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride;
  a.sinks = sinks;
  a.out = static_cast<uint8_t*>(out);
  a.err = reinterpret_cast<int*>(ws);
  a.rb_max = p.rb_max;
  a.ctas = p.ctas;
  a.info = reinterpret_cast<int2*>(ws + p.info);
  a.part = reinterpret_cast<float*>(ws + p.part);
  const cudaError_t e = launch_paged_attend(a, p, join_only, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "paged attention launch");
}

}  // namespace

extern "C" {

csa_status_t csa_paged_append(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                              const void* k_new, const void* v_new, int64_t kv_stride, const int64_t* start,
                              const int32_t* n_new, int32_t Tq, void* stream) {
  CSA_TRY(check_gqa(L));
  CSA_TRY(check_table(T, false));
  CSA_TRY(check_pool(pool));
  CSA_TRY(need_ptr(k_new, "k_new"));
  CSA_TRY(need_ptr(v_new, "v_new"));
  CSA_TRY(check_stride(L, &kv_stride, (int64_t)L->Hkv * L->D, "kv_stride"));
  CSA_TRY(check_tokens(start, n_new, Tq));
  PagedAppendArgs a;
  a.T = page_args(T);
  a.P = pool_args(pool);
  a.tok = token_args(start, n_new, Tq);
  a.Hkv = L->Hkv; a.D = L->D; a.act_fmt = L->act_format;
  a.k_new = static_cast<const uint8_t*>(k_new);
  a.v_new = static_cast<const uint8_t*>(v_new);
  a.kv_stride = kv_stride;
  a.kmax = (int)pages_touched_max(Tq, T->page);
  if ((int64_t)T->B * a.kmax > INT_MAX / 2 / L->Hkv) return fail(CSA_ERR_UNSUPPORTED, "Tq=%d of %d sequences", Tq, T->B);
  cudaError_t e = page_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_paged_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "paged append launch");
}

size_t csa_paged_workspace_size(const csa_gqa_t* L, const csa_page_table_t* T, int32_t Tq, int64_t n_max) {
  PagedPlan p;
  return make_plan(L, T, Tq, n_max, &p) == CSA_OK ? p.total : 0;
}

csa_status_t csa_paged_attend(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                              const void* q, int64_t q_stride, const float* sinks, const int64_t* start,
                              const int32_t* n_new, int32_t Tq, int64_t n_max, void* out, void* workspace,
                              size_t ws_bytes, void* stream) {
  return attend(L, pool, T, q, q_stride, sinks, start, n_new, Tq, n_max, out, workspace, ws_bytes, false, stream);
}

csa_status_t csa_debug_paged_join(const csa_gqa_t* L, const csa_page_table_t* T, const float* sinks,
                                  const int64_t* start, const int32_t* n_new, int32_t Tq, int64_t n_max, void* out,
                                  void* workspace, size_t ws_bytes, void* stream) {
  return attend(L, nullptr, T, nullptr, 0, sinks, start, n_new, Tq, n_max, out, workspace, ws_bytes, true, stream);
}

csa_status_t csa_pages_fork(const csa_page_table_t* T, const int32_t* src, const int32_t* dst, int32_t n,
                            void* stream) {
  CSA_TRY(check_table(T, true));
  if (n < 0 || n > 4096) return fail(CSA_ERR_INVALID_ARG, "n=%d (0 to 4096)", n);
  if (n == 0) return CSA_OK;
  CSA_TRY(need_ptr(src, "src", 4));
  CSA_TRY(need_ptr(dst, "dst", 4));
  int* err = nullptr;
  cudaError_t e = page_error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_pages_fork(page_args(T), src, dst, n, err, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "page fork launch");
}

csa_status_t csa_pages_reserve(const csa_page_table_t* T, const int64_t* start, const int32_t* n_new, int32_t Tq,
                               int32_t* copy_src, int32_t* copy_dst, int32_t* missing, void* stream) {
  CSA_TRY(check_table(T, true));
  CSA_TRY(check_tokens(start, n_new, Tq));
  CSA_TRY(need_ptr(copy_src, "copy_src", 4));
  CSA_TRY(need_ptr(copy_dst, "copy_dst", 4));
  CSA_TRY(need_ptr(missing, "missing", 4));
  PagesReserveArgs a;
  a.T = page_args(T);
  a.tok = token_args(start, n_new, Tq);
  a.kmax = (int)pages_touched_max(Tq, T->page);
  if ((int64_t)T->B * a.kmax >= kMaxPos) return fail(CSA_ERR_UNSUPPORTED, "Tq=%d of %d sequences", Tq, T->B);
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.missing = missing;
  cudaError_t e = page_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_pages_reserve(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "page reserve launch");
}

csa_status_t csa_pages_free(const csa_page_table_t* T, const int64_t* keep, const int64_t* begin, int64_t first,
                            void* stream) {
  CSA_TRY(check_table(T, true));
  if (!keep && !begin) return fail(CSA_ERR_INVALID_ARG, "keep and begin are both NULL");
  if (keep) CSA_TRY(need_ptr(keep, "keep", 8));
  if (begin) CSA_TRY(need_ptr(begin, "begin", 8));
  if (first < 0) return fail(CSA_ERR_INVALID_ARG, "first=%lld", (long long)first);
  int* err = nullptr;
  cudaError_t e = page_error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_pages_free(page_args(T), keep, begin, first, err, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "page free launch");
}

csa_status_t csa_pages_compact(const csa_page_table_t* T, int32_t max_moves, int32_t* move_src, int32_t* move_dst,
                               int32_t* count, void* stream) {
  CSA_TRY(check_table(T, true));
  if (max_moves < 0 || max_moves > T->n_pages)
    return fail(CSA_ERR_INVALID_ARG, "max_moves=%d (0 to n_pages)", max_moves);
  if (max_moves > 0) {
    CSA_TRY(need_ptr(move_src, "move_src", 4));
    CSA_TRY(need_ptr(move_dst, "move_dst", 4));
  }
  CSA_TRY(need_ptr(count, "count", 4));
  PagesCompactArgs a;
  a.T = page_args(T);
  a.max_moves = max_moves;
  a.move_src = move_src;
  a.move_dst = move_dst;
  a.count = count;
  cudaError_t e = page_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_pages_compact(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "page compact launch");
}

csa_status_t csa_pages_copy(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                            const int32_t* src, const int32_t* dst, const int32_t* count, int32_t n, void* stream) {
  CSA_TRY(check_gqa(L));
  CSA_TRY(check_pool(pool));
  CSA_TRY(check_table_shape(T));
  if (n < 0) return fail(CSA_ERR_INVALID_ARG, "n=%d", n);
  if (n == 0) return CSA_OK;
  CSA_TRY(need_ptr(src, "src", 4));
  CSA_TRY(need_ptr(dst, "dst", 4));
  if (count) CSA_TRY(need_ptr(count, "count", 4));
  PagesCopyArgs a;
  a.P = pool_args(pool);
  a.n_pages = T->n_pages;
  a.page_bytes = (int64_t)L->Hkv * T->page * L->D;
  a.Hkv = L->Hkv;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.n = n;
  cudaError_t e = page_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "page error word");
  e = launch_pages_copy(a, num_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA_OK : cuda_fail(e, "page copy launch");
}

}  // extern "C"
