// C ABI of the paged-cache operators (include/mtp.h): argument validation and dispatch. Every
// check is made before the device is touched.
#include <cmath>
#include <cstring>

#include "mtp.h"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

static bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

static bool overlap(const void* p, long long np, const void* q, long long nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + static_cast<uintptr_t>(nq) && b < a + static_cast<uintptr_t>(np);
}

static int log2_exact(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return (1 << s) == n ? s : -1;
}

// Multiprocessors of the current device.
static int sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    set_error("querying the device: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  if (*n > kMaxSms) *n = kMaxSms;
  return MTP_OK;
}

// Checks a caller's cache description and turns it into the kernels' form.
int make_cache(const mtp_paged_kv* kv, bool tables, Cache* c) {
  if (!kv || !kv->k || (tables && (!kv->block_table || !kv->ctx_len))) {
    set_error("the paged cache needs k%s", tables ? ", block_table and ctx_len" : "");
    return MTP_ERR_INVALID_ARG;
  }
  if (kv->dtype != MTP_DTYPE_BF16 && kv->dtype != MTP_DTYPE_F32) {
    set_error("dtype=%d is neither BF16 nor F32", kv->dtype);
    return MTP_ERR_INVALID_ARG;
  }
  const int vec = kv->dtype == MTP_DTYPE_BF16 ? 8 : 4, shift = kv->page_size > 0 ? log2_exact(kv->page_size) : -1;
  if (shift < 0 || kv->page_size > 256) {
    set_error("page_size=%d is not a power of two <= 256", kv->page_size);
    return MTP_ERR_UNSUPPORTED_SHAPE;
  }
  if (kv->head_dim < vec || kv->head_dim > 512 || kv->head_dim % vec || kv->n_kv_head < 1 || kv->n_kv_head > 1024) {
    set_error("head_dim=%d must be a multiple of %d in [%d, 512] and n_kv_head=%d in [1, 1024]", kv->head_dim, vec, vec,
              kv->n_kv_head);
    return MTP_ERR_UNSUPPORTED_SHAPE;
  }
  const long long tok = 1LL << 30;
  if (kv->n_pages < 1 || static_cast<long long>(kv->n_pages) * kv->page_size > tok ||
      (tables && (kv->max_pages < 1 || static_cast<long long>(kv->max_pages) * kv->page_size > tok ||
                  kv->table_stride < kv->max_pages))) {
    set_error("need n_pages >= 1, max_pages >= 1, both times page_size <= 2^30, and table_stride >= max_pages "
              "(n_pages=%d max_pages=%d page_size=%d table_stride=%lld)", kv->n_pages, kv->max_pages, kv->page_size,
              static_cast<long long>(kv->table_stride));
    return MTP_ERR_INVALID_ARG;
  }
  const int64_t s[3] = {kv->stride_page, kv->stride_t, kv->stride_h};
  for (int i = 0; i < 3; ++i)
    if (s[i] < kv->head_dim || s[i] % vec || s[i] > (1LL << 40)) {
      set_error("the cache's strides must be >= head_dim and multiples of %d elements (page %lld, token %lld, head %lld)",
                vec, static_cast<long long>(s[0]), static_cast<long long>(s[1]), static_cast<long long>(s[2]));
      return MTP_ERR_INVALID_ARG;
    }
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->codes, 16) || !aligned(kv->scales, 4) ||
      !aligned(kv->block_table, 4) || !aligned(kv->ctx_len, 4)) {
    set_error("k, v and codes must be 16-byte aligned (scales, block_table, ctx_len 4-byte)");
    return MTP_ERR_INVALID_ARG;
  }
  if ((kv->codes == nullptr) != (kv->scales == nullptr)) {
    set_error("codes and scales come together");
    return MTP_ERR_INVALID_ARG;
  }
  c->k = kv->k;
  c->v = kv->v == kv->k ? nullptr : kv->v;
  c->table = kv->block_table;
  c->ctx_len = kv->ctx_len;
  c->codes = reinterpret_cast<signed char*>(kv->codes);
  c->scales = kv->scales;
  c->sp = kv->stride_page;
  c->st = kv->stride_t;
  c->sh = kv->stride_h;
  c->table_stride = kv->table_stride;
  c->n_pages = kv->n_pages;
  c->pshift = shift;
  c->max_pages = tables ? kv->max_pages : 0;
  c->nkv = kv->n_kv_head;
  c->d = kv->head_dim;
  c->f32 = kv->dtype == MTP_DTYPE_F32 ? 1 : 0;
  return MTP_OK;
}

static int check_batch(const Cache& c, int B, int n_head) {
  if (B < 1 || B > 1 << 20 || n_head < 1 || n_head % c.nkv || n_head / c.nkv > 1024 ||
      static_cast<long long>(B) * n_head > 1 << 22) {
    set_error("need B >= 1, n_head a positive multiple of n_kv_head=%d and B * n_head <= 2^22 (B=%d n_head=%d)", c.nkv, B,
              n_head);
    return MTP_ERR_INVALID_ARG;
  }
  return MTP_OK;
}

int check_workspace(const void* ws, int64_t have, long long need) {
  if (need > 0 && (!ws || !aligned(ws, 16) || have < need)) {
    set_error("the workspace must be 16-byte aligned and hold %lld bytes (%lld given)", need,
              static_cast<long long>(have));
    return MTP_ERR_INVALID_ARG;
  }
  return MTP_OK;
}

}  // namespace pg
}  // namespace mtp

using namespace mtp;

extern "C" {

int mtp_page_plan(const int32_t* old_len, const int32_t* new_len, int32_t B, int32_t* block_table,
                  int64_t table_stride, int32_t max_pages, int32_t* free_ring, int32_t n_pages,
                  const int32_t* ring_state, int32_t page_size, int32_t max_tokens, int32_t* len_out,
                  int32_t* slot_map, int32_t* cu_new, int32_t* state_out, int32_t* status, void* stream) {
  set_error("%s", "");
  if (!old_len || !new_len || !block_table || !free_ring || !ring_state || !len_out || !cu_new || !state_out ||
      !status || (max_tokens > 0 && !slot_map)) {
    set_error("old_len, new_len, block_table, free_ring, ring_state, len_out, slot_map (max_tokens > 0), cu_new, "
              "state_out and status must be non-NULL");
    return MTP_ERR_INVALID_ARG;
  }
  if (len_out == old_len || len_out == new_len || state_out == ring_state) {
    set_error("len_out and state_out must be buffers of their own");
    return MTP_ERR_INVALID_ARG;
  }
  const int shift = page_size > 0 ? pg::log2_exact(page_size) : -1;
  if (shift < 0 || page_size > 256) {
    set_error("page_size=%d is not a power of two <= 256", page_size);
    return MTP_ERR_UNSUPPORTED_SHAPE;
  }
  const long long tok = 1LL << 30;
  if (B < 1 || B > pg::kPlanMaxB || max_pages < 1 || n_pages < 1 || max_tokens < 0 || max_tokens > tok ||
      static_cast<long long>(max_pages) * page_size > tok || static_cast<long long>(n_pages) * page_size > tok ||
      static_cast<long long>(B) * max_pages > INT32_MAX || table_stride < max_pages) {
    set_error("need 1 <= B <= 8192, max_pages, n_pages >= 1 with max_pages * page_size, n_pages * page_size and "
              "max_tokens <= 2^30, B * max_pages < 2^31 and table_stride >= max_pages (B=%d max_pages=%d n_pages=%d "
              "max_tokens=%d table_stride=%lld)", B, max_pages, n_pages, max_tokens, static_cast<long long>(table_stride));
    return MTP_ERR_INVALID_ARG;
  }
  if (!pg::aligned(slot_map, 16)) {
    set_error("slot_map must be 16-byte aligned");
    return MTP_ERR_INVALID_ARG;
  }
  int sms = 0;
  const int rc = pg::sm_count(&sms);
  if (rc) return rc;
  return run_page_plan(old_len, new_len, B, block_table, table_stride, max_pages, free_ring, n_pages, ring_state, shift,
                       max_tokens, len_out, slot_map, cu_new, state_out, status, sms, static_cast<cudaStream_t>(stream));
}

int mtp_page_append(const mtp_paged_kv* kv, const void* k_new, const void* v_new, int64_t row_stride_k,
                    int64_t row_stride_v, const int32_t* slot_map, int32_t T, void* stream) {
  set_error("%s", "");
  pg::Cache c;
  int rc = pg::make_cache(kv, false, &c);
  if (rc) return rc;
  if (T < 0 || T > 1 << 30 || (T > 0 && (!k_new || !slot_map || (c.v && !v_new)))) {
    set_error("need 0 <= T <= 2^30 and, for T > 0, k_new, slot_map and (a cache with a V) v_new");
    return MTP_ERR_INVALID_ARG;
  }
  if (!c.v && v_new && v_new != k_new) {
    set_error("v_new given, but the cache has V = K");
    return MTP_ERR_INVALID_ARG;
  }
  const int vec = c.f32 ? 4 : 8;
  const int64_t width = static_cast<int64_t>(c.nkv) * c.d;
  auto bad_row = [&](int64_t stride) { return stride < width || stride % vec || stride > (1LL << 40); };
  if (bad_row(row_stride_k) || (c.v && bad_row(row_stride_v)) ||
      !pg::aligned(k_new, 16) || !pg::aligned(v_new, 16) || !pg::aligned(slot_map, 4)) {
    set_error("new rows must be 16-byte aligned, n_kv_head * head_dim = %lld to 2^40 elements apart, in multiples of %d",
              static_cast<long long>(width), vec);
    return MTP_ERR_INVALID_ARG;
  }
  int sms = 0;
  if ((rc = pg::sm_count(&sms))) return rc;
  return run_page_append(c, k_new, v_new, row_stride_k, row_stride_v, slot_map, T, sms,
                         static_cast<cudaStream_t>(stream));
}

int mtp_paged_attention_workspace(const mtp_paged_kv* kv, int32_t B, int32_t n_head, int32_t n_list, int64_t* bytes) {
  set_error("%s", "");
  pg::Cache c;
  int rc = pg::make_cache(kv, true, &c);
  if (rc || (rc = pg::check_batch(c, B, n_head))) return rc;
  if (!bytes || n_list < 0) {
    set_error("need bytes and n_list >= 0 (n_list=%d)", n_list);
    return MTP_ERR_INVALID_ARG;
  }
  *bytes = paged_att_workspace(c, B, n_head, n_list);
  return MTP_OK;
}

int mtp_paged_attention(const mtp_paged_kv* kv, const float* q, int32_t B, int32_t n_head, int32_t window, float scale,
                        const int32_t* pages, int32_t n_list, float* out, float* lse, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  set_error("%s", "");
  pg::AttArgs a;
  memset(&a, 0, sizeof(a));
  int rc = pg::make_cache(kv, true, &a.c);
  if (rc || (rc = pg::check_batch(a.c, B, n_head))) return rc;
  if (!q || !out || !pg::aligned(q, 16) || !pg::aligned(out, 16) || !pg::aligned(lse, 4) || !pg::aligned(pages, 4)) {
    set_error("q and out must be non-NULL and 16-byte aligned");
    return MTP_ERR_INVALID_ARG;
  }
  const long long row_bytes = 4LL * B * n_head, q_bytes = row_bytes * a.c.d;
  if (pg::overlap(out, q_bytes, q, q_bytes) ||
      (lse && (pg::overlap(lse, row_bytes, q, q_bytes) || pg::overlap(lse, row_bytes, out, q_bytes)))) {
    set_error("out and lse must be buffers of their own");
    return MTP_ERR_INVALID_ARG;
  }
  const double s = scale > 0.f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(a.c.d));
  a.scale_log2 = static_cast<float>(s * 1.4426950408889634);
  if (window < 0 || !(scale >= 0.f) || !std::isfinite(a.scale_log2)) {
    set_error("need window >= 0 and a scale in [0, 2^127] (window=%d scale=%g)", window, static_cast<double>(scale));
    return MTP_ERR_INVALID_ARG;
  }
  if (pages ? (n_list < 1 || (static_cast<long long>(n_list) << a.c.pshift) > (1LL << 30)) : n_list != 0) {
    set_error("n_list=%d: at least 1 with pages, 0 without, n_list * page_size <= 2^30", n_list);
    return MTP_ERR_INVALID_ARG;
  }
  if ((rc = pg::check_workspace(workspace, workspace_bytes, paged_att_workspace(a.c, B, n_head, n_list)))) return rc;
  a.q = q;
  a.list = pages;
  a.n_list = n_list;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.nh = n_head;
  a.window = window;
  a.spin = pg::kSpin;
  a.skip = -1;
  int sms = 0;
  if ((rc = pg::sm_count(&sms))) return rc;
  return run_paged_att(a, workspace, sms, static_cast<cudaStream_t>(stream));
}

int mtp_page_select_workspace(const mtp_paged_kv* kv, int32_t B, int64_t* bytes) {
  set_error("%s", "");
  pg::Cache c;
  int rc = pg::make_cache(kv, true, &c);
  if (rc || (rc = pg::check_batch(c, B, c.nkv))) return rc;
  if (!bytes) {
    set_error("bytes must be non-NULL");
    return MTP_ERR_INVALID_ARG;
  }
  *bytes = page_select_workspace(c, B);
  return MTP_OK;
}

int mtp_page_select(const mtp_paged_kv* kv, const float* q, int32_t B, int32_t n_head, int32_t n_select,
                    int32_t keep_first, int32_t keep_last, int32_t* sel, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  set_error("%s", "");
  pg::Cache c;
  int rc = pg::make_cache(kv, true, &c);
  if (rc || (rc = pg::check_batch(c, B, n_head))) return rc;
  if (!c.codes || !q || !sel || !pg::aligned(q, 16) || !pg::aligned(sel, 4)) {
    set_error("q (16-byte aligned), sel and a cache with page summaries (codes, scales) are required");
    return MTP_ERR_INVALID_ARG;
  }
  if (n_head / c.nkv > 32) {
    set_error("at most 32 query heads per KV head (%d)", n_head / c.nkv);
    return MTP_ERR_UNSUPPORTED_SHAPE;
  }
  if (keep_first < 0 || keep_last < 1 || n_select < 1 || n_select > 1 << 24 ||
      static_cast<long long>(keep_first) + keep_last > n_select) {
    set_error("need keep_first >= 0, keep_last >= 1 and keep_first + keep_last <= n_select (%d, %d, %d)", keep_first,
              keep_last, n_select);
    return MTP_ERR_INVALID_ARG;
  }
  if ((rc = pg::check_workspace(workspace, workspace_bytes, page_select_workspace(c, B)))) return rc;
  int sms = 0;
  if ((rc = pg::sm_count(&sms))) return rc;
  return run_page_select(c, q, B, n_head, n_select, keep_first, keep_last, sel, workspace, sms,
                         static_cast<cudaStream_t>(stream));
}

}  // extern "C"
