// C ABI of the paged caches (declared in include/jssa.h): host-side validation and the launch
// sequence of each entry point.  No entry point allocates, frees or synchronises.
#include <cstring>

#include "jssa.h"
#include "api_util.h"
#include "common.cuh"
#include "launch.h"

namespace jssa {
namespace {

constexpr int64_t kInt31 = (int64_t(1) << 31) - 1;

jssa_status check_paged(const jssa_paged_layout* L) {
  if (!L) return JSSA_ERR_INVALID_ARG;
  if (L->B < 1 || L->Hq < 1 || L->Hkv < 1 || L->d < 1 || L->page_size < 1 || L->n_pages < 1 || L->max_pages < 1)
    return JSSA_ERR_INVALID_ARG;
  if (L->Hq % L->Hkv != 0) return JSSA_ERR_INVALID_ARG;
  if (L->out_dtype != JSSA_OUT_F32 && L->out_dtype != JSSA_OUT_BF16) return JSSA_ERR_INVALID_ARG;
  const int64_t extent[3] = {L->n_pages, L->Hkv, L->page_size};
  for (const int64_t* st : {L->k_stride, L->v_stride})
    for (int i = 0; i < 3; ++i) {
      if (st[i] < 0 || st[i] % 8 || st[i] >= (int64_t(1) << 39)) return JSSA_ERR_INVALID_ARG;
      if (extent[i] > 1 && st[i] < L->d) return JSSA_ERR_INVALID_ARG;
    }
  if (L->B > 1024 || L->Hq > 65535 || L->Hq / L->Hkv > 128) return JSSA_ERR_UNSUPPORTED;
  if (L->d != 64 && L->d != 128 && L->d != 256) return JSSA_ERR_UNSUPPORTED;
  if (L->page_size % 16) return JSSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(L->max_pages) * L->page_size > (int64_t(1) << 30) ||
      static_cast<int64_t>(L->B) * L->max_pages > kInt31 ||
      static_cast<int64_t>(L->Hkv) * L->page_size * L->d >= (int64_t(1) << 34))
    return JSSA_ERR_UNSUPPORTED;
  return JSSA_OK;
}

struct PagedWorkspace {
  int* status;
  int32_t* counters;   // [num_sms], zero between calls; at the same place for every layout
  int32_t* growers;    // [n_pages, 2]
  int32_t* free_list;  // [n_pages]
  int32_t* map;        // [n_pages + 1]
  PagedCut* cuts;      // [num_sms]
  float2* part_ml;     // [2 num_sms][rows_cap]
  float* part_o;       // [2 num_sms][rows_cap][d]
  int rows_cap;
  size_t bytes;
};

jssa_status carve_paged(const jssa_paged_layout* L, int max_q_len, void* base, PagedWorkspace* w) {
  const int num_sms = num_sms_current();
  if (num_sms <= 0) return JSSA_ERR_CUDA;
  size_t off = 0;
  char* p = static_cast<char*>(base);
  auto take = [&](size_t n) {
    char* at = p ? p + off : nullptr;
    off += align_up(n);
    return at;
  };
  const size_t n = static_cast<size_t>(L->n_pages);
  w->status = reinterpret_cast<int*>(take(sizeof(int)));
  w->counters = reinterpret_cast<int32_t*>(take(num_sms * sizeof(int32_t)));
  w->growers = reinterpret_cast<int32_t*>(take(2 * n * sizeof(int32_t)));
  w->free_list = reinterpret_cast<int32_t*>(take(n * sizeof(int32_t)));
  w->map = reinterpret_cast<int32_t*>(take((n + 1) * sizeof(int32_t)));
  w->cuts = reinterpret_cast<PagedCut*>(take(num_sms * sizeof(PagedCut)));
  w->rows_cap = paged_attn_rows(L->d, L->Hq / L->Hkv, max_q_len);
  const size_t rows = static_cast<size_t>(2 * num_sms) * w->rows_cap;
  w->part_ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  w->part_o = reinterpret_cast<float*>(take(rows * L->d * sizeof(float)));
  w->bytes = off;
  return JSSA_OK;
}

jssa_status get_paged_ws(const jssa_paged_layout* L, int max_q_len, void* ws, size_t ws_bytes, PagedWorkspace* w) {
  if (!ws || !aligned(ws, kAlign)) return JSSA_ERR_WORKSPACE;
  const jssa_status st = carve_paged(L, max_q_len, ws, w);
  if (st != JSSA_OK) return st;
  return ws_bytes < w->bytes ? JSSA_ERR_WORKSPACE : JSSA_OK;
}

PagePool page_pool(const jssa_paged_layout* L, const void* K, const void* V) {
  PagePool p{};
  p.K = const_cast<void*>(K);
  memcpy(p.ks, L->k_stride, sizeof p.ks);
  p.V = const_cast<void*>(V);
  memcpy(p.vs, L->v_stride, sizeof p.vs);
  p.Hkv = L->Hkv;
  p.d = L->d;
  p.page_size = L->page_size;
  p.n_pages = L->n_pages;
  return p;
}

PageBook page_book(const jssa_paged_layout* L, int32_t* table, int32_t* ref, int32_t* seq_lens, int* status) {
  PageBook k{};
  k.table = table;
  k.ref = ref;
  k.seq_lens = seq_lens;
  k.B = L->B;
  k.max_pages = L->max_pages;
  k.page_size = L->page_size;
  k.n_pages = L->n_pages;
  k.status = status;
  return k;
}

bool ints(std::initializer_list<const void*> ps) {  // non-null int32 arrays
  for (const void* p : ps)
    if (!p || !aligned(p, 4)) return false;
  return true;
}

bool rows16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned(p, 16)) return false;
  return true;
}

}  // namespace
}  // namespace jssa

using namespace jssa;

extern "C" {

jssa_status jssa_paged_workspace_size(const jssa_paged_layout* L, int32_t max_q_len, size_t* bytes) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (!bytes || max_q_len < 0) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = carve_paged(L, max_q_len, nullptr, &w);
  if (st != JSSA_OK) return st;
  *bytes = w.bytes;
  return JSSA_OK;
}

jssa_status jssa_paged_append_kv(const jssa_paged_layout* L, const void* K_new, const void* V_new, int64_t new_stride,
                                 int64_t n_tokens, void* K, void* V, const int32_t* page_table,
                                 const int32_t* q_begin, const int32_t* seq_lens, void* workspace, size_t ws_bytes,
                                 void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (n_tokens < 0 || n_tokens > kInt31 || new_stride < static_cast<int64_t>(L->Hkv) * L->d || new_stride % 8 ||
      new_stride >= (int64_t(1) << 39))
    return JSSA_ERR_INVALID_ARG;
  if (n_tokens == 0) return JSSA_OK;
  if (!rows16({K_new, V_new, K, V}) || !ints({page_table, q_begin, seq_lens})) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  PagedAppendArgs a{};
  a.pool = page_pool(L, K, V);
  a.K_new = K_new;
  a.V_new = V_new;
  a.new_stride = new_stride;
  a.n_tokens = n_tokens;
  a.table = page_table;
  a.q_begin = q_begin;
  a.seq_lens = seq_lens;
  a.B = L->B;
  a.max_pages = L->max_pages;
  a.status = w.status;
  return cu(launch_paged_append(a, static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_paged_attn(const jssa_paged_layout* L, const void* Q, int64_t q_stride, int64_t n_tokens,
                            int32_t max_q_len, const void* K, const void* V, const int32_t* page_table,
                            const int32_t* q_begin, const int32_t* seq_lens, int32_t window, int32_t n_sinks,
                            float sm_scale, void* O, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (n_tokens < 0 || n_tokens > kInt31 || max_q_len < 0 || window < 0 || n_sinks < 0 ||
      q_stride < static_cast<int64_t>(L->Hq) * L->d || q_stride % 8 || q_stride >= (int64_t(1) << 39))
    return JSSA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || sm_scale > 2e38f) return JSSA_ERR_INVALID_ARG;  // its product with log2 e stays finite
  if (n_tokens == 0 || max_q_len == 0) return JSSA_OK;
  if (!rows16({Q, K, V, O}) || !ints({page_table, q_begin, seq_lens}) || (lse && !aligned(lse, 4)))
    return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, max_q_len, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  PagedAttnArgs a{};
  a.pool = page_pool(L, K, V);
  a.Q = Q;
  a.q_stride = q_stride;
  a.n_tokens = n_tokens;
  a.max_q_len = max_q_len;
  a.table = page_table;
  a.q_begin = q_begin;
  a.seq_lens = seq_lens;
  a.B = L->B;
  a.Hq = L->Hq;
  a.max_pages = L->max_pages;
  a.window = window;
  a.n_sinks = n_sinks;
  a.sm_scale = sm_scale;
  a.O = O;
  a.lse = lse;
  a.out_bf16 = (L->out_dtype == JSSA_OUT_BF16);
  a.status = w.status;
  a.part_o = w.part_o;
  a.part_ml = w.part_ml;
  a.counters = w.counters;
  a.cuts = w.cuts;
  a.rows_cap = w.rows_cap;
  const bool few = paged_few_rows(L->d, static_cast<int64_t>(max_q_len) * (L->Hq / L->Hkv));
  return cu((few ? launch_paged_few : launch_paged_attn)(a, num_sms_current(), static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_pages_fork(const jssa_paged_layout* L, const int32_t* src, const int32_t* dst, int32_t n,
                            int32_t* page_table, int32_t* ref_count, int32_t* seq_lens, void* workspace,
                            size_t ws_bytes, void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (n < 0 || n > 65535) return JSSA_ERR_INVALID_ARG;
  if (n == 0) return JSSA_OK;
  if (!ints({src, dst, page_table, ref_count, seq_lens})) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  return cu(launch_pages_fork(page_book(L, page_table, ref_count, seq_lens, w.status), src, dst, n,
                              static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_pages_reserve(const jssa_paged_layout* L, const int32_t* n_new, int32_t* page_table,
                               int32_t* ref_count, int32_t* seq_lens, int32_t* copy_src, int32_t* copy_dst,
                               void* workspace, size_t ws_bytes, void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (!ints({n_new, page_table, ref_count, seq_lens, copy_src, copy_dst})) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  return cu(launch_pages_reserve(page_book(L, page_table, ref_count, seq_lens, w.status), n_new, copy_src, copy_dst,
                                 w.growers, w.free_list, static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_pages_release(const jssa_paged_layout* L, const int32_t* ended, int32_t window, int32_t n_sinks,
                               int32_t* page_table, int32_t* ref_count, int32_t* seq_lens, void* workspace,
                               size_t ws_bytes, void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (window < 0 || n_sinks < 0) return JSSA_ERR_INVALID_ARG;
  if (!ints({page_table, ref_count, seq_lens}) || (ended && !aligned(ended, 4))) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  return cu(launch_pages_release(page_book(L, page_table, ref_count, seq_lens, w.status), ended, window, n_sinks,
                                 static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_pages_compact(const jssa_paged_layout* L, int32_t* page_table, int32_t* ref_count, int32_t* src,
                               int32_t* dst, int32_t max_moves, int32_t* n_moves, void* workspace, size_t ws_bytes,
                               void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (max_moves < 1) return JSSA_ERR_INVALID_ARG;
  if (!ints({page_table, ref_count, src, dst, n_moves})) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  return cu(launch_pages_compact(page_book(L, page_table, ref_count, nullptr, w.status), src, dst, max_moves, n_moves,
                                 w.map, static_cast<cudaStream_t>(stream)));
}

jssa_status jssa_pages_copy(const jssa_paged_layout* L, void* K, void* V, const int32_t* src, const int32_t* dst,
                            int32_t n, const int32_t* count, void* workspace, size_t ws_bytes, void* stream) {
  jssa_status st = check_paged(L);
  if (st != JSSA_OK) return st;
  if (n < 0) return JSSA_ERR_INVALID_ARG;
  if (n == 0) return JSSA_OK;
  if (!rows16({K, V}) || !ints({src, dst}) || (count && !aligned(count, 4))) return JSSA_ERR_INVALID_ARG;
  PagedWorkspace w{};
  st = get_paged_ws(L, 0, workspace, ws_bytes, &w);
  if (st != JSSA_OK) return st;
  return cu(launch_pages_copy(page_pool(L, K, V), src, dst, n, count, w.status, num_sms_current(),
                              static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
