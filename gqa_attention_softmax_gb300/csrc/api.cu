// C ABI of libsinkattn: argument validation, tensor-map encoding, launch
// selection. Every entry point checks its arguments on the host before any
// CUDA call and returns a status; nothing here allocates, frees or
// synchronises (except the diagnostic sinkattn_debug_status).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "internal.h"
#include "sinkattn.h"

namespace sinkattn {

static thread_local char g_last_error[512] = "";
static std::atomic<int> g_decode_kernel{SINKATTN_DECODE_AUTO};
static std::atomic<int> g_prefill_kernel{SINKATTN_PREFILL_AUTO};

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
}

int sm_count() {
  // host threads may call the library concurrently: entries are atomics (a
  // racing first fill stores the same value twice)
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 0 || dev >= 64) return 148;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

int make_rows_tmap(CUtensorMap* map, const void* base, uint64_t rows, int d, int box_rows,
                   int swizzle_bytes) {
  auto fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return SINKATTN_CUDA_ERROR;
  }
  if (rows == 0) rows = 1;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapSwizzle sw =
      swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

int make_rows_tmap_u8(CUtensorMap* map, const void* base, uint64_t rows, int d, int box_rows,
                      int swizzle_bytes) {
  auto fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return SINKATTN_CUDA_ERROR;
  }
  if (rows == 0) rows = 1;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapSwizzle sw = swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                               : swizzle_bytes == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_NONE;
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled (u8) failed (CUresult %d)", static_cast<int>(r));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

int make_q_tmap(CUtensorMap* map, const void* q, uint64_t total_q, int Hq, int d, int G, int QB) {
  auto fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return SINKATTN_CUDA_ERROR;
  }
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hq),
                              total_q > 0 ? total_q : 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(Hq) * d * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(QB)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled (q) failed (CUresult %d)", static_cast<int>(r));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

}  // namespace sinkattn

using namespace sinkattn;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_error("%s", buf);
  return status;
}

// Checks shared by every attention entry point.
int check_common(const void* q, const void* k, const void* v, int32_t Hq, int32_t Hkv,
                 int32_t d, float sm_scale, int32_t causal, int32_t window) {
  if (!q || !k || !v) return fail(SINKATTN_INVALID_ARG, "q, k and v must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v))
    return fail(SINKATTN_INVALID_ARG, "q, k and v must be 16-byte aligned");
  if (Hq <= 0 || Hkv <= 0) return fail(SINKATTN_INVALID_ARG, "head counts must be positive");
  if (Hq % Hkv != 0)
    return fail(SINKATTN_UNSUPPORTED, "num_qo_heads (%d) is not a multiple of num_kv_heads (%d)",
                Hq, Hkv);
  if (d != 64 && d != 128) return fail(SINKATTN_UNSUPPORTED, "head_dim %d is not 64 or 128", d);
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale))
    return fail(SINKATTN_INVALID_ARG, "sm_scale must be positive and finite");
  if (causal != 0 && causal != 1) return fail(SINKATTN_INVALID_ARG, "causal must be 0 or 1");
  if (window > 0 && !causal)
    return fail(SINKATTN_UNSUPPORTED, "a sliding window requires causal masking");
  return SINKATTN_OK;
}

// Paged KV: page pools [num_pages, Hkv, page_size, d] and per-sequence page lists.
struct PagedKv {
  const int32_t* page_indptr;
  const int32_t* page_indices;
  int32_t num_pages;
  int32_t page_size;
};

int check_paged(const PagedKv& pg, int32_t Hkv) {
  if (!pg.page_indptr || !pg.page_indices)
    return fail(SINKATTN_INVALID_ARG, "page_indptr and page_indices must be non-null");
  if (pg.page_size < 16 || pg.page_size > 256 || (pg.page_size & (pg.page_size - 1)))
    return fail(SINKATTN_UNSUPPORTED, "page_size %d is not a power of two in [16, 256]",
                pg.page_size);
  if (pg.num_pages < 1) return fail(SINKATTN_INVALID_ARG, "num_pages must be positive");
  if (static_cast<int64_t>(pg.num_pages) * Hkv * pg.page_size >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "page pools exceed 2^31 rows");
  return SINKATTN_OK;
}

void set_paged(AttnArgs* a, const PagedKv* pg) {
  a->page_size = pg ? pg->page_size : 0;
  a->num_pages = pg ? pg->num_pages : 0;
  a->page_indptr = pg ? pg->page_indptr : nullptr;
  a->page_indices = pg ? pg->page_indices : nullptr;
}

}  // namespace

extern "C" {

const char* sinkattn_status_string(int status) {
  switch (status) {
    case SINKATTN_OK: return "SINKATTN_OK";
    case SINKATTN_INVALID_ARG: return "SINKATTN_INVALID_ARG";
    case SINKATTN_UNSUPPORTED: return "SINKATTN_UNSUPPORTED";
    case SINKATTN_CUDA_ERROR: return "SINKATTN_CUDA_ERROR";
    case SINKATTN_TIMEOUT: return "SINKATTN_TIMEOUT";
    case SINKATTN_BAD_LENGTHS: return "SINKATTN_BAD_LENGTHS";
    case SINKATTN_OUT_OF_PAGES: return "SINKATTN_OUT_OF_PAGES";
    case SINKATTN_BAD_PAGES: return "SINKATTN_BAD_PAGES";
    default: return "SINKATTN_UNKNOWN_STATUS";
  }
}

const char* sinkattn_last_error(void) { return g_last_error; }

}  // extern "C"

namespace {

int prefill_impl(const void* q, const void* k, const void* v, const float* sinks,
                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, const PagedKv* pg,
                 int32_t batch, int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                 int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                 int32_t causal, int32_t window, void* out, float* lse, void* stream) {
  g_last_error[0] = '\0';
  int rc = check_common(q, k, v, num_qo_heads, num_kv_heads, head_dim, sm_scale, causal, window);
  if (rc) return rc;
  if (pg && (rc = check_paged(*pg, num_kv_heads))) return rc;
  if (!out || !aligned16(out)) return fail(SINKATTN_INVALID_ARG, "out must be non-null and 16-byte aligned");
  if (!cu_seqlens_q || !cu_seqlens_k) return fail(SINKATTN_INVALID_ARG, "cu_seqlens must be non-null");
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(SINKATTN_INVALID_ARG, "sizes must be non-negative");
  if (batch > 65535) return fail(SINKATTN_UNSUPPORTED, "batch %d exceeds 65535", batch);
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(SINKATTN_INVALID_ARG, "lse must be 4-byte aligned");
  if (max_seqlen_q > max_seqlen_k)
    return fail(SINKATTN_INVALID_ARG, "max_seqlen_q (%d) exceeds max_seqlen_k (%d)", max_seqlen_q,
                max_seqlen_k);
  if (static_cast<int64_t>(num_kv_heads) * batch * max_seqlen_k >= (int64_t{1} << 31) ||
      static_cast<int64_t>(total_q) * num_qo_heads >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "problem exceeds 2^31 rows");
  if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return SINKATTN_OK;

  AttnArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
  a.batch = batch; a.q_len = 0; a.max_q = max_seqlen_q; a.max_kv = max_seqlen_k;
  a.total_q = total_q;
  a.Hq = num_qo_heads; a.Hkv = num_kv_heads; a.d = head_dim;
  a.sm_scale = sm_scale; a.causal = causal; a.window = window; a.num_splits = 1;
  a.sinks = sinks; a.out = out; a.lse = lse;
  set_paged(&a, pg);
  if (num_qo_heads / num_kv_heads > 128)
    return fail(SINKATTN_UNSUPPORTED, "GQA group of %d heads exceeds 128", num_qo_heads / num_kv_heads);
  return launch_prefill_tc(a, g_prefill_kernel.load(std::memory_order_relaxed),
                           static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int sinkattn_prefill(const void* q, const void* k, const void* v, const float* sinks,
                     const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t batch,
                     int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                     int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                     float sm_scale, int32_t causal, int32_t window, void* out, float* lse,
                     void* stream) {
  return prefill_impl(q, k, v, sinks, cu_seqlens_q, cu_seqlens_k, nullptr, batch, total_q,
                      max_seqlen_q, max_seqlen_k, num_qo_heads, num_kv_heads, head_dim, sm_scale,
                      causal, window, out, lse, stream);
}

int sinkattn_prefill_paged(const void* q, const void* k_pages, const void* v_pages,
                           const float* sinks, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, const int32_t* page_indptr,
                           const int32_t* page_indices, int32_t num_pages, int32_t page_size,
                           int32_t batch, int32_t total_q, int32_t max_seqlen_q,
                           int32_t max_seqlen_k, int32_t num_qo_heads, int32_t num_kv_heads,
                           int32_t head_dim, float sm_scale, int32_t causal, int32_t window,
                           void* out, float* lse, void* stream) {
  const PagedKv pg{page_indptr, page_indices, num_pages, page_size};
  return prefill_impl(q, k_pages, v_pages, sinks, cu_seqlens_q, cu_seqlens_k, &pg, batch,
                      total_q, max_seqlen_q, max_seqlen_k, num_qo_heads, num_kv_heads, head_dim,
                      sm_scale, causal, window, out, lse, stream);
}

}  // extern "C"

namespace {

// Workspace of the backward pass: two arrays of a value per row, then the
// blocks' sums of the sinks' gradients.
size_t back_row_bytes(int32_t total_q, int32_t Hq) {
  return (static_cast<size_t>(total_q) * Hq * 4 + 255) & ~static_cast<size_t>(255);
}

}  // namespace

extern "C" {

int sinkattn_prefill_backward_workspace_bytes(int32_t total_q, int32_t num_qo_heads,
                                              size_t* bytes) {
  g_last_error[0] = '\0';
  if (!bytes) return fail(SINKATTN_INVALID_ARG, "bytes must be non-null");
  if (total_q < 0 || num_qo_heads <= 0) return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (static_cast<int64_t>(total_q) * num_qo_heads >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "problem exceeds 2^31 rows");
  *bytes = total_q == 0 ? 0
                        : 2 * back_row_bytes(total_q, num_qo_heads) + 256 +
                              static_cast<size_t>(back_sink_blocks(total_q, num_qo_heads)) * num_qo_heads * 4;
  return SINKATTN_OK;
}

int sinkattn_prefill_backward(const void* dout, const void* q, const void* k, const void* v,
                              const void* out, const float* lse, const float* sinks,
                              const float* dlse, const int32_t* cu_seqlens_q,
                              const int32_t* cu_seqlens_k, int32_t batch, int32_t total_q,
                              int32_t total_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                              int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                              float sm_scale, int32_t causal, int32_t window, void* dq, void* dk,
                              void* dv, float* dsinks, void* workspace, size_t workspace_bytes,
                              void* stream) {
  g_last_error[0] = '\0';
  if (batch < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(SINKATTN_INVALID_ARG, "sizes must be non-negative");
  const bool none = batch == 0 || total_k == 0;   // (each sequence has Lq <= Lk: no queries either)
  // an empty tensor has no address to check
  static const int unused __attribute__((aligned(16))) = 0;
  const bool no_q = none || total_q == 0;
  int rc = check_common(no_q ? &unused : q, none ? &unused : k, none ? &unused : v, num_qo_heads,
                        num_kv_heads, head_dim, sm_scale, causal, window);
  if (rc) return rc;
  if (batch > 65535) return fail(SINKATTN_UNSUPPORTED, "batch %d exceeds 65535", batch);
  if (num_kv_heads > 65535)
    return fail(SINKATTN_UNSUPPORTED, "num_kv_heads %d exceeds 65535", num_kv_heads);
  if (num_qo_heads / num_kv_heads > 128)
    return fail(SINKATTN_UNSUPPORTED, "GQA group of %d heads exceeds 128",
                num_qo_heads / num_kv_heads);
  if (max_seqlen_q > max_seqlen_k)
    return fail(SINKATTN_INVALID_ARG, "max_seqlen_q (%d) exceeds max_seqlen_k (%d)", max_seqlen_q,
                max_seqlen_k);
  if (static_cast<int64_t>(num_kv_heads) * total_k >= (int64_t{1} << 31) ||
      static_cast<int64_t>(total_q) * num_qo_heads >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "problem exceeds 2^31 rows");
  if ((sinks == nullptr) != (dsinks == nullptr))
    return fail(SINKATTN_INVALID_ARG, "sinks and dsinks must be both given or both NULL");
  if ((reinterpret_cast<uintptr_t>(sinks) | reinterpret_cast<uintptr_t>(dsinks) |
       reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dlse)) & 3u)
    return fail(SINKATTN_INVALID_ARG, "lse, dlse, sinks and dsinks must be 4-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (none) {
    if (dsinks && cudaMemsetAsync(dsinks, 0, sizeof(float) * num_qo_heads, s) != cudaSuccess)
      return fail(SINKATTN_CUDA_ERROR, "cudaMemsetAsync: %s", cudaGetErrorString(cudaGetLastError()));
    return SINKATTN_OK;
  }
  if (!dk || !dv || !aligned16(dk) || !aligned16(dv))
    return fail(SINKATTN_INVALID_ARG, "dk and dv must be non-null and 16-byte aligned");
  if (!cu_seqlens_q || !cu_seqlens_k ||
      ((reinterpret_cast<uintptr_t>(cu_seqlens_q) | reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u))
    return fail(SINKATTN_INVALID_ARG, "cu_seqlens must be non-null and 4-byte aligned");
  if (!no_q && (!dout || !out || !dq || !aligned16(dout) || !aligned16(out) || !aligned16(dq)))
    return fail(SINKATTN_INVALID_ARG, "dout, out and dq must be non-null and 16-byte aligned");
  if (!no_q && !lse) return fail(SINKATTN_INVALID_ARG, "lse must be non-null");
  size_t need = 0;
  if ((rc = sinkattn_prefill_backward_workspace_bytes(total_q, num_qo_heads, &need))) return rc;
  // (without queries it takes no bytes, and none are looked at)
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return fail(SINKATTN_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < need)
    return fail(SINKATTN_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  BackArgs a{};
  a.dout = dout; a.q = q; a.k = k; a.v = v; a.out = out;
  a.lse = lse; a.sinks = sinks; a.dlse = dlse;
  a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
  a.batch = batch; a.total_q = total_q; a.total_k = total_k;
  a.max_q = max_seqlen_q; a.max_kv = max_seqlen_k;
  a.Hq = num_qo_heads; a.Hkv = num_kv_heads; a.d = head_dim;
  a.sm_scale = sm_scale; a.causal = causal; a.window = window;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dsinks = dsinks;
  if (need > 0) {
    char* ws = static_cast<char*>(workspace);
    a.nlse = reinterpret_cast<float*>(ws);
    a.ndelta = reinterpret_cast<float*>(ws + back_row_bytes(total_q, num_qo_heads));
    a.sink_count = reinterpret_cast<int*>(ws + 2 * back_row_bytes(total_q, num_qo_heads));
    a.sink_part = reinterpret_cast<float*>(ws + 2 * back_row_bytes(total_q, num_qo_heads) + 256);
  }
  return launch_prefill_back(a, s);
}

}  // extern "C"

namespace {

// Validation shared by the split-KV decode entry points; fills `a` (without
// the output pointers). Returns SINKATTN_OK or the failing status.
int decode_args(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                int32_t batch, int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                int32_t window, int32_t num_splits, AttnArgs* a) {
  int rc = check_common(q, k, v, num_qo_heads, num_kv_heads, head_dim, sm_scale, causal, window);
  if (rc) return rc;
  if (!kv_indptr) return fail(SINKATTN_INVALID_ARG, "kv_indptr must be non-null");
  if (batch < 0 || max_kv_len < 0) return fail(SINKATTN_INVALID_ARG, "sizes must be non-negative");
  if (batch > 65535) return fail(SINKATTN_UNSUPPORTED, "batch %d exceeds 65535", batch);
  if (q_len < 1) return fail(SINKATTN_INVALID_ARG, "q_len must be at least 1");
  if (num_splits < 1) return fail(SINKATTN_INVALID_ARG, "num_splits must be at least 1");
  if (num_splits > 4096) return fail(SINKATTN_UNSUPPORTED, "num_splits %d exceeds 4096", num_splits);
  if (q_len > max_kv_len)
    return fail(SINKATTN_INVALID_ARG, "q_len (%d) exceeds max_kv_len (%d)", q_len, max_kv_len);
  if (num_qo_heads / num_kv_heads > 64)
    return fail(SINKATTN_UNSUPPORTED, "GQA group of %d heads exceeds 64", num_qo_heads / num_kv_heads);
  if (static_cast<int64_t>(num_kv_heads) * batch * max_kv_len >= (int64_t{1} << 31) ||
      static_cast<int64_t>(batch) * q_len * num_qo_heads * num_splits * head_dim >=
          (int64_t{1} << 40))
    return fail(SINKATTN_UNSUPPORTED, "problem too large");
  *a = AttnArgs{};
  a->q = q; a->k = k; a->v = v;
  a->cu_q = nullptr; a->cu_k = kv_indptr;
  a->batch = batch; a->q_len = q_len; a->max_q = q_len; a->max_kv = max_kv_len;
  a->Hq = num_qo_heads; a->Hkv = num_kv_heads; a->d = head_dim;
  a->sm_scale = sm_scale; a->causal = causal; a->window = window; a->num_splits = num_splits;
  return SINKATTN_OK;
}

// Partials with the selected kernel (a.part_acc / a.part_md set).
// FP8 KV: e4m3 K/V codes and their per-KV-head scales.
struct Fp8Kv {
  const float* k_scale;
  const float* v_scale;
};

int decode_kind() { return g_decode_kernel.load(std::memory_order_relaxed); }

int launch_partials(const AttnArgs& a, int kind, cudaStream_t stream) {
  if (a.kv_fp8) {   // tcgen05 up to 64 rows per tile at head_dim 128, else the warp-level kernel
    const bool tc8 = decode_tc_supported(a);
    if (kind == SINKATTN_DECODE_TCGEN05 && !tc8)
      return fail(SINKATTN_UNSUPPORTED,
                  "the tcgen05 FP8 decode needs head_dim 128 and at most 64 heads per group");
    if (kind == SINKATTN_DECODE_TCGEN05 || (kind == SINKATTN_DECODE_AUTO && tc8))
      return launch_decode_tc(a, stream);
    return a.part_slots > 0 ? launch_attn_mma_shared(a, stream) : launch_attn_mma(a, stream);
  }
  const bool tc_ok = decode_tc_supported(a);
  if (kind == SINKATTN_DECODE_TCGEN05 && !tc_ok)
    return fail(SINKATTN_UNSUPPORTED,
                "the tcgen05 decode kernel needs head_dim 128");
  if (kind == SINKATTN_DECODE_TCGEN05 || (kind == SINKATTN_DECODE_AUTO && tc_ok))
    return launch_decode_tc(a, stream);
  return a.part_slots > 0 ? launch_attn_mma_shared(a, stream) : launch_attn_mma(a, stream);
}

int decode_split_impl(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                      const PagedKv* pg, int32_t batch, int32_t q_len, int32_t max_kv_len,
                      int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                      float sm_scale, int32_t causal, int32_t window, int32_t num_splits,
                      float* part_acc, float* part_md, void* stream,
                      const Fp8Kv* f8 = nullptr) {
  g_last_error[0] = '\0';
  AttnArgs a;
  int rc = decode_args(q, k, v, kv_indptr, batch, q_len, max_kv_len, num_qo_heads, num_kv_heads,
                       head_dim, sm_scale, causal, window, num_splits, &a);
  if (rc) return rc;
  if (pg && (rc = check_paged(*pg, num_kv_heads))) return rc;
  if (!part_acc || !part_md || !aligned16(part_acc) || !aligned16(part_md))
    return fail(SINKATTN_INVALID_ARG, "partial buffers must be non-null and 16-byte aligned");
  if (f8) {
    if (!f8->k_scale || !f8->v_scale ||
        (reinterpret_cast<uintptr_t>(f8->k_scale) | reinterpret_cast<uintptr_t>(f8->v_scale)) & 3u)
      return fail(SINKATTN_INVALID_ARG, "k_scale and v_scale must be non-null and 4-byte aligned");
    a.kv_fp8 = 1;
    a.k_scale = f8->k_scale;
    a.v_scale = f8->v_scale;
  }
  if (batch == 0) return SINKATTN_OK;
  a.part_acc = part_acc; a.part_md = part_md;
  set_paged(&a, pg);
  return launch_partials(a, decode_kind(), static_cast<cudaStream_t>(stream));
}

int decode_impl(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                const PagedKv* pg, int32_t batch, int32_t q_len, int32_t max_kv_len,
                int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                int32_t causal, int32_t window, int32_t num_splits, const float* sinks,
                void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream,
                const Fp8Kv* f8 = nullptr) {
  g_last_error[0] = '\0';
  int rc;
  if (num_splits <= 0) {
    rc = sinkattn_decode_default_splits(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                        max_kv_len, &num_splits);
    if (rc) return rc;
  }
  size_t need = 0;
  rc = sinkattn_decode_workspace_bytes(batch, q_len, num_qo_heads, head_dim, num_splits, &need);
  if (rc) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(SINKATTN_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < need)
    return fail(SINKATTN_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  if (!out || !aligned16(out)) return fail(SINKATTN_INVALID_ARG, "out must be non-null and 16-byte aligned");
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(SINKATTN_INVALID_ARG, "lse must be 4-byte aligned");
  // More query rows per KV head than one 128-row tile holds (G x q_len > 128,
  // e.g. 16 MTP drafts of 16 heads): the split kernels would read every KV
  // tile once per 128-row block; the single-pass prefill kernel (decode
  // drafts are its queries, bottom-right causal) reads each once and needs
  // no partials. Only under the default kernel choice, bf16 KV.
  if (!f8 && batch > 0 && static_cast<int64_t>(num_qo_heads / num_kv_heads) * q_len > 128 &&
      g_decode_kernel.load(std::memory_order_relaxed) == SINKATTN_DECODE_AUTO &&
      (head_dim == 64 || head_dim == 128)) {
    AttnArgs a;
    rc = decode_args(q, k, v, kv_indptr, batch, q_len, max_kv_len, num_qo_heads, num_kv_heads,
                     head_dim, sm_scale, causal, window, num_splits, &a);
    if (rc) return rc;
    if (pg && (rc = check_paged(*pg, num_kv_heads))) return rc;
    if (static_cast<int64_t>(batch) * q_len >= (int64_t{1} << 31))
      return fail(SINKATTN_UNSUPPORTED, "too many query rows");
    set_paged(&a, pg);
    a.total_q = batch * q_len;
    a.sinks = sinks;
    a.out = out;
    a.lse = lse;
    return launch_prefill_tc(a, g_prefill_kernel.load(std::memory_order_relaxed),
                             static_cast<cudaStream_t>(stream));
  }
  const size_t slots = static_cast<size_t>(batch) * q_len * num_qo_heads * num_splits;
  float* part_acc = static_cast<float*>(workspace);
  float* part_md = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                            ((slots * head_dim * 4 + 255) & ~static_cast<size_t>(255)));
  rc = decode_split_impl(q, k, v, kv_indptr, pg, batch, q_len, max_kv_len, num_qo_heads,
                         num_kv_heads, head_dim, sm_scale, causal, window, num_splits, part_acc,
                         part_md, stream, f8);
  if (rc) return rc;
  if (batch == 0) return SINKATTN_OK;
  // the partials are this call's scratch: the merge may drop them from L2
  return launch_merge(part_acc, part_md, sinks, batch * q_len, num_qo_heads, head_dim,
                      num_splits, out, lse, static_cast<cudaStream_t>(stream), true);
}

// Whether the prefixes take the tcgen05 kernel, which works on row blocks of
// 256 (128 at least), or the warp-level one, which takes up to 64 rows at a
// time and re-reads the keys for each. Calls of one group behind 8192 keys,
// warp-level against tcgen05: 48 rows 19.8 and 20.4 us at d 64, 23.5 and 25.7
// at d 128; 64 rows 22.5 and 20.9, 37.5 and 25.6; behind 1024 keys 48 rows 13.2
// and 14.5, 15.3 and 18.3; 64 rows 14.0 and 14.9, 20.0 and 18.4.
// (A group's sequences come as one run of rows: 4 samples of 8 heads are 32.)
// Measured with bf16 pools; codes go by the same border.
bool prefix_on_tc(int kind, int64_t tokens, int G, int64_t groups) {
  if (kind != SINKATTN_DECODE_AUTO) return kind == SINKATTN_DECODE_TCGEN05;
  return tokens * G > 48 * groups;
}

// So few keys that every sequence reads its own: two launches instead of four,
// and what the sequences share comes from L2. By keys x KV heads x head_dim of
// the whole batch, in millions, us per call shared | not, 4 to 64 sequences: at
// d 64 2.2: 12.6 | 8.3, 4.4: 14.6 | 8.7, 8.5: 15 to 16.5 | 14.5 to 14.8, 9.7:
// 16.4 | 15.5, 17: 17.7 to 19.6 | 20.3 to 24.4; at d 128 4.4: 18.5 | 10.0, 9.7:
// 22.5 | 17.9, 17: 20.9 to 25.8 | 17.8 to 26.1. (bf16 pools; codes go by the same
// border. A window does not count here: with one of 128 behind 8192 keys, 64
// sequences at d 64 take 17.6 us shared and 20.0 each for itself, 4 16.3 and 9.1.)
bool few_keys(int kind, int64_t batch, int64_t max_prefix, int64_t max_suffix, int64_t Hkv,
              int64_t d) {
  // (one division at a time: the product of any sizes may pass 64 bits)
  return kind == SINKATTN_DECODE_AUTO && batch > 0 &&
         max_prefix + max_suffix <= (int64_t{10} << 20) / batch / Hkv / d;
}

// The default split counts under a choice of kernel.
int shared_splits(int kind, int32_t batch, int32_t q_len, int32_t num_qo_heads,
                  int32_t num_kv_heads, int32_t head_dim, int32_t num_groups,
                  int32_t max_prefix_len, int32_t max_suffix_len, int32_t* prefix_splits,
                  int32_t* num_splits) {
  g_last_error[0] = '\0';
  if (!prefix_splits || !num_splits)
    return fail(SINKATTN_INVALID_ARG, "prefix_splits and num_splits must be non-null");
  if (num_groups < 1 || max_prefix_len < 0) return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (batch < 0 || q_len < 1 || num_qo_heads <= 0 || num_kv_heads <= 0 || max_suffix_len < 0)
    return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (head_dim != 64 && head_dim != 128)
    return fail(SINKATTN_UNSUPPORTED, "head_dim %d is not 64 or 128", head_dim);
  if (few_keys(kind, batch, max_prefix_len, max_suffix_len, num_kv_heads, head_dim)) {
    *prefix_splits = 0;
    return sinkattn_decode_default_splits(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                          max_prefix_len + max_suffix_len, num_splits);
  }
  // Own keys: chunks of about 1024 keys while they are needed to fill the SMs
  // (the warp-level kernel's four blocks per SM twice over, the tcgen05
  // kernel's one block twice over). Each further chunk costs its partials: 64
  // sequences behind 8192 keys at d 64 take 33, 35 and 38 us in 1, 2 and 3
  // chunks with up to 1024 own keys, 76, 59 and 59 us with up to 4000; 16
  // sequences of up to 8000 own keys 96, 45, 40 and 37 us in 1, 3, 4 and 8.
  const int64_t items = std::max<int64_t>(1, static_cast<int64_t>(batch) * num_kv_heads);
  const int64_t fill = (head_dim == 64 ? 8 : 2) * static_cast<int64_t>(sm_count());
  *num_splits = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>((fill + items - 1) / items, (int64_t{max_suffix_len} + 1023) / 1024)));
  const int G = num_qo_heads / num_kv_heads;
  // (calls of 2^31 rows are refused: beyond, any answer does, within 64 bits)
  const int64_t tokens = std::min<int64_t>(static_cast<int64_t>(batch) * q_len, int64_t{1} << 31);
  if (G >= 1 && G <= 64 && prefix_on_tc(kind, tokens, G, num_groups)) {
    // partials that let the kernel deal its units out evenly (prefixes of
    // several groups about half as long as the longest), at most 16
    const int64_t tiles = (int64_t{max_prefix_len} + prefix_tile_keys(head_dim, false) - 1) /
                          prefix_tile_keys(head_dim, false);
    const int64_t bt = prefix_block_tokens(G);
    const double units = static_cast<double>(num_groups * ((tokens / num_groups + bt - 1) / bt)) *
                         num_kv_heads * (num_groups > 1 ? (tiles + 1) / 2 : tiles);
    const int64_t quota = static_cast<int64_t>(
        std::max(1.0, std::min(std::ceil(units / sm_count()), 0x1p40)));
    const int64_t n = tiles > 1 ? (tiles - 1 + quota - 1) / quota + 1 : 1;
    *prefix_splits = static_cast<int32_t>(std::min<int64_t>(n, 16));
    return SINKATTN_OK;
  }
  // the warp-level kernel's blocks of up to 64 query rows
  const int64_t blocks =
      std::min<int64_t>(num_groups + tokens * std::min(G, 64) / 64, int64_t{1} << 20);
  return sinkattn_decode_default_splits(static_cast<int32_t>(blocks), 1, num_qo_heads, num_kv_heads,
                                        head_dim, max_prefix_len, prefix_splits);
}

// Shared-prefix decode: the sequences' own keys and the groups' prefixes as
// two sets of partials of the same rows, folded by one merge.
size_t shared_plan_bytes(int64_t batch, int64_t q_len, int64_t groups) {
  return (shared_plan_ints(batch, q_len, groups) * 4 + 255) & ~static_cast<size_t>(255);
}

int decode_shared_impl(const void* q, const void* k_pages, const void* v_pages, const Fp8Kv* f8,
                       const int32_t* kv_indptr, const PagedKv& pg, const int32_t* group_indptr,
                       const int32_t* prefix_lens, int32_t num_groups, int32_t batch,
                       int32_t q_len, int32_t max_prefix_len, int32_t max_suffix_len,
                       int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                       float sm_scale, int32_t causal, int32_t window, int32_t prefix_splits,
                       int32_t num_splits, const float* sinks, void* workspace,
                       size_t workspace_bytes, void* out, float* lse, void* stream) {
  g_last_error[0] = '\0';
  if (!group_indptr || !prefix_lens)
    return fail(SINKATTN_INVALID_ARG, "group_indptr and prefix_lens must be non-null");
  if (num_groups < 1 || max_prefix_len < 0)
    return fail(SINKATTN_INVALID_ARG, "num_groups must be positive, max_prefix_len non-negative");
  if (num_groups > 65535) return fail(SINKATTN_UNSUPPORTED, "num_groups %d exceeds 65535", num_groups);
  int32_t ps = 0, ss = 0;
  const int kind = decode_kind();   // (read once: the passes of a call go by one choice)
  int rc = shared_splits(kind, batch, q_len, num_qo_heads, num_kv_heads, head_dim, num_groups,
                         max_prefix_len, max_suffix_len, &ps, &ss);
  if (rc) return rc;
  const bool alone = prefix_splits <= 0 &&
                     few_keys(kind, batch, max_prefix_len, max_suffix_len, num_kv_heads, head_dim);
  if (prefix_splits <= 0) prefix_splits = ps;
  if (num_splits <= 0) num_splits = ss;
  if (max_prefix_len == 0) prefix_splits = 0;   // nothing is shared
  AttnArgs a;
  rc = decode_args(q, k_pages, v_pages, kv_indptr, batch, q_len,
                   max_suffix_len + (alone ? max_prefix_len : 0), num_qo_heads, num_kv_heads,
                   head_dim, sm_scale, causal, window, num_splits, &a);
  if (rc) return rc;
  if ((rc = check_paged(pg, num_kv_heads))) return rc;
  if (f8) {
    if (!f8->k_scale || !f8->v_scale ||
        (reinterpret_cast<uintptr_t>(f8->k_scale) | reinterpret_cast<uintptr_t>(f8->v_scale)) & 3u)
      return fail(SINKATTN_INVALID_ARG, "k_scale and v_scale must be non-null and 4-byte aligned");
    a.kv_fp8 = 1;
    a.k_scale = f8->k_scale;
    a.v_scale = f8->v_scale;
  }
  if (static_cast<int64_t>(batch) * q_len * num_qo_heads >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "problem exceeds 2^31 rows");
  if (static_cast<int64_t>(max_prefix_len) + max_suffix_len >= (int64_t{1} << 31) ||
      static_cast<int64_t>(num_groups) * max_prefix_len >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "prefixes reach 2^31 keys");
  if (static_cast<int64_t>(prefix_splits) + num_splits > 4096)
    return fail(SINKATTN_UNSUPPORTED, "the splits exceed 4096 in all");
  const int slots = prefix_splits + num_splits;
  size_t need = 0;
  rc = sinkattn_decode_shared_workspace_bytes(batch, q_len, num_qo_heads, head_dim, num_groups,
                                              prefix_splits, num_splits, &need);
  if (rc) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(SINKATTN_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < need)
    return fail(SINKATTN_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  if (!out || !aligned16(out)) return fail(SINKATTN_INVALID_ARG, "out must be non-null and 16-byte aligned");
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(SINKATTN_INVALID_ARG, "lse must be 4-byte aligned");
  if (batch == 0) return SINKATTN_OK;
  set_paged(&a, &pg);
  const int G = num_qo_heads / num_kv_heads;
  const size_t rows = static_cast<size_t>(batch) * q_len;
  const bool tc = prefix_on_tc(kind, static_cast<int64_t>(rows), G, num_groups);
  // what a launch would refuse is refused here, before the first one
  const bool own_tc = kind != SINKATTN_DECODE_WARP && decode_tc_supported(a);
  if (kind == SINKATTN_DECODE_TCGEN05 && !own_tc)
    return fail(SINKATTN_UNSUPPORTED,
                "the tcgen05 shared-prefix decode needs head_dim 128 and bf16 pools");
  if (num_kv_heads > 65535)
    return fail(SINKATTN_UNSUPPORTED, "num_kv_heads %d exceeds 65535", num_kv_heads);
  // blocks of query tokens that a pass forms at most, and its work items
  auto blocks_of = [](int64_t n, int64_t per) { return (n + per - 1) / per; };
  const int tile = prefix_tile_keys(head_dim, f8 != nullptr);
  const int64_t prefix_items =
      tc ? (num_groups + static_cast<int64_t>(rows) / prefix_block_tokens(G)) * num_kv_heads *
               blocks_of(max_prefix_len, tile)
         : (num_groups + static_cast<int64_t>(rows) / attn_mma_block_tokens(G, rows)) * prefix_splits;
  const int64_t own_items =
      own_tc ? blocks_of(q_len, std::min(q_len, 128 / G)) * batch * num_kv_heads * num_splits
             : blocks_of(q_len, attn_mma_block_tokens(G, q_len)) * num_splits;
  if (std::max(prefix_items, own_items) >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "too many work items");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t plan_bytes = shared_plan_bytes(batch, q_len, num_groups);
  float* part_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan_bytes);
  float* part_md = reinterpret_cast<float*>(
      reinterpret_cast<char*>(part_acc) +
      ((rows * num_qo_heads * slots * head_dim * 4 + 255) & ~static_cast<size_t>(255)));
  a.part_acc = part_acc;
  a.part_md = part_md;
  if (alone) {
    if ((rc = launch_attn_mma(a, s))) return rc;
    const SharedCheck check{kv_indptr,    pg.page_indptr, group_indptr, prefix_lens,    num_groups,
                            pg.page_size, batch,          q_len,        max_prefix_len, max_suffix_len};
    return launch_merge_sparse(part_acc, part_md, sinks, static_cast<int32_t>(rows), num_qo_heads,
                               head_dim, slots, out, lse, &check, s);
  }

  SharedPlan plan;
  plan.own_seq = static_cast<int32_t*>(workspace);
  plan.own_len = plan.own_seq + batch;
  plan.own_page = plan.own_len + batch;
  plan.grp_q = plan.own_page + batch;
  plan.grp_k = plan.grp_q + num_groups + 1;
  plan.grp_pages = plan.grp_k + num_groups + 1;
  plan.grp_unit = plan.grp_pages + num_groups + 1;
  plan.quota = plan.grp_unit + num_groups + 1;
  plan.row_pos = plan.quota + 1;
  // (at d 128 a block of either pass fills its SM; bf16 figures, for codes too)
  SharedCost cost;
  cost.unit = head_dim == 64 ? 1.05f : 1.9f;
  cost.own_key = head_dim == 64 ? 0.35f / 64 * num_kv_heads : 0.f;
  cost.ramp = 4.f;
  cost.sms = sm_count();
  rc = launch_shared_plan(kv_indptr, pg.page_indptr, group_indptr, prefix_lens, num_groups,
                          pg.page_size, batch, q_len, max_prefix_len, max_suffix_len,
                          tc ? prefix_block_tokens(G) : attn_mma_block_tokens(G, rows),
                          tc ? prefix_tile_keys(head_dim, f8 != nullptr) : 0, num_kv_heads,
                          window, prefix_splits, cost, plan, s);
  if (rc) return rc;

  a.part_slots = slots;
  if (prefix_splits > 0) {
    AttnArgs pa = a;
    PagedKv shared = pg;
    shared.page_indptr = plan.grp_pages;
    set_paged(&pa, &shared);
    pa.cu_q = plan.grp_q;
    pa.cu_k = plan.grp_k;
    pa.batch = num_groups;
    pa.q_len = 0;
    pa.max_q = static_cast<int32_t>(rows);
    pa.max_kv = max_prefix_len;
    pa.total_q = static_cast<int32_t>(rows);
    pa.causal = 0;
    pa.num_splits = prefix_splits;
    pa.free_rows = 1;
    pa.row_pos = window > 0 ? plan.row_pos : nullptr;
    pa.blk = tc ? nullptr : plan.grp_unit;
    pa.chain = kChainWaitFirst | kChainFollow;
    if ((rc = tc ? launch_prefix_tc(pa, plan, s) : launch_attn_mma_shared(pa, s))) return rc;
  }
  PagedKv own = pg;
  own.page_indptr = plan.own_page;
  set_paged(&a, &own);
  a.cu_k = plan.own_len;
  a.seq = plan.own_seq;
  a.part_first = prefix_splits;
  // behind a prefix pass, the plan is complete (that pass waited for it)
  a.chain = prefix_splits > 0 ? kChainWaitLast : kChainWaitFirst;
  if ((rc = launch_partials(a, kind, s))) return rc;
  return launch_merge_sparse(part_acc, part_md, sinks, static_cast<int32_t>(rows), num_qo_heads,
                             head_dim, slots, out, lse, nullptr, s);
}

}  // namespace

extern "C" {

int sinkattn_decode_split(const void* q, const void* k, const void* v,
                          const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                          int32_t max_kv_len, int32_t num_qo_heads, int32_t num_kv_heads,
                          int32_t head_dim, float sm_scale, int32_t causal, int32_t window,
                          int32_t num_splits, float* part_acc, float* part_md, void* stream) {
  return decode_split_impl(q, k, v, kv_indptr, nullptr, batch, q_len, max_kv_len, num_qo_heads,
                           num_kv_heads, head_dim, sm_scale, causal, window, num_splits, part_acc,
                           part_md, stream);
}

int sinkattn_decode_split_paged(const void* q, const void* k_pages, const void* v_pages,
                                const int32_t* kv_indptr, const int32_t* page_indptr,
                                const int32_t* page_indices, int32_t num_pages, int32_t page_size,
                                int32_t batch, int32_t q_len, int32_t max_kv_len,
                                int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                float sm_scale, int32_t causal, int32_t window, int32_t num_splits,
                                float* part_acc, float* part_md, void* stream) {
  const PagedKv pg{page_indptr, page_indices, num_pages, page_size};
  return decode_split_impl(q, k_pages, v_pages, kv_indptr, &pg, batch, q_len, max_kv_len,
                           num_qo_heads, num_kv_heads, head_dim, sm_scale, causal, window,
                           num_splits, part_acc, part_md, stream);
}

int sinkattn_decode_split_fp8(const void* q, const void* k, const void* v,
                              const float* k_scale, const float* v_scale,
                              const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                              int32_t max_kv_len, int32_t num_qo_heads, int32_t num_kv_heads,
                              int32_t head_dim, float sm_scale, int32_t causal, int32_t window,
                              int32_t num_splits, float* part_acc, float* part_md, void* stream) {
  const Fp8Kv f8{k_scale, v_scale};
  return decode_split_impl(q, k, v, kv_indptr, nullptr, batch, q_len, max_kv_len, num_qo_heads,
                           num_kv_heads, head_dim, sm_scale, causal, window, num_splits, part_acc,
                           part_md, stream, &f8);
}

int sinkattn_decode_fp8(const void* q, const void* k, const void* v, const float* k_scale,
                        const float* v_scale, const int32_t* kv_indptr, int32_t batch,
                        int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                        int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                        int32_t window, int32_t num_splits, const float* sinks, void* workspace,
                        size_t workspace_bytes, void* out, float* lse, void* stream) {
  const Fp8Kv f8{k_scale, v_scale};
  return decode_impl(q, k, v, kv_indptr, nullptr, batch, q_len, max_kv_len, num_qo_heads,
                     num_kv_heads, head_dim, sm_scale, causal, window, num_splits, sinks,
                     workspace, workspace_bytes, out, lse, stream, &f8);
}

int sinkattn_decode_shared_paged(
    const void* q, const void* k_pages, const void* v_pages, const int32_t* kv_indptr,
    const int32_t* page_indptr, const int32_t* page_indices, const int32_t* group_indptr,
    const int32_t* prefix_lens, int32_t num_groups, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t q_len, int32_t max_prefix_len, int32_t max_suffix_len,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
    int32_t window, int32_t prefix_splits, int32_t num_splits, const float* sinks,
    void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream) {
  const PagedKv pg{page_indptr, page_indices, num_pages, page_size};
  return decode_shared_impl(q, k_pages, v_pages, nullptr, kv_indptr, pg, group_indptr, prefix_lens,
                            num_groups, batch, q_len, max_prefix_len, max_suffix_len, num_qo_heads,
                            num_kv_heads, head_dim, sm_scale, causal, window, prefix_splits,
                            num_splits, sinks, workspace, workspace_bytes, out, lse, stream);
}

int sinkattn_decode_shared_paged_fp8(
    const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
    const float* v_scale, const int32_t* kv_indptr, const int32_t* page_indptr,
    const int32_t* page_indices, const int32_t* group_indptr, const int32_t* prefix_lens,
    int32_t num_groups, int32_t num_pages, int32_t page_size, int32_t batch, int32_t q_len,
    int32_t max_prefix_len, int32_t max_suffix_len, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, float sm_scale, int32_t causal, int32_t window, int32_t prefix_splits,
    int32_t num_splits, const float* sinks, void* workspace, size_t workspace_bytes, void* out,
    float* lse, void* stream) {
  const PagedKv pg{page_indptr, page_indices, num_pages, page_size};
  const Fp8Kv f8{k_scale, v_scale};
  return decode_shared_impl(q, k_pages, v_pages, &f8, kv_indptr, pg, group_indptr, prefix_lens,
                            num_groups, batch, q_len, max_prefix_len, max_suffix_len, num_qo_heads,
                            num_kv_heads, head_dim, sm_scale, causal, window, prefix_splits,
                            num_splits, sinks, workspace, workspace_bytes, out, lse, stream);
}

int sinkattn_decode_shared_workspace_bytes(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                           int32_t head_dim, int32_t num_groups,
                                           int32_t prefix_splits, int32_t num_splits,
                                           size_t* bytes) {
  g_last_error[0] = '\0';
  if (num_groups < 1 || prefix_splits < 0) return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (static_cast<int64_t>(prefix_splits) + num_splits > 4096)
    return fail(SINKATTN_UNSUPPORTED, "the splits exceed 4096 in all");
  const int rc = sinkattn_decode_workspace_bytes(batch, q_len, num_qo_heads, head_dim,
                                                 prefix_splits + num_splits, bytes);
  if (rc) return rc;
  if (num_splits < 1) return fail(SINKATTN_INVALID_ARG, "bad sizes");
  *bytes += shared_plan_bytes(batch, q_len, num_groups);
  return SINKATTN_OK;
}

int sinkattn_decode_shared_default_splits(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                          int32_t num_kv_heads, int32_t head_dim,
                                          int32_t num_groups, int32_t max_prefix_len,
                                          int32_t max_suffix_len, int32_t* prefix_splits,
                                          int32_t* num_splits) {
  return shared_splits(decode_kind(), batch, q_len, num_qo_heads, num_kv_heads, head_dim, num_groups,
                       max_prefix_len, max_suffix_len, prefix_splits, num_splits);
}

int sinkattn_set_prefill_kernel(int kind) {
  g_last_error[0] = '\0';
  if (kind != SINKATTN_PREFILL_AUTO && kind != SINKATTN_PREFILL_ONE_BLOCK &&
      kind != SINKATTN_PREFILL_PERSISTENT)
    return fail(SINKATTN_INVALID_ARG, "unknown prefill kernel %d", kind);
  g_prefill_kernel.store(kind, std::memory_order_relaxed);
  return SINKATTN_OK;
}

int sinkattn_set_decode_kernel(int kind) {
  g_last_error[0] = '\0';
  if (kind != SINKATTN_DECODE_AUTO && kind != SINKATTN_DECODE_WARP &&
      kind != SINKATTN_DECODE_TCGEN05)
    return fail(SINKATTN_INVALID_ARG, "unknown decode kernel %d", kind);
  g_decode_kernel.store(kind, std::memory_order_relaxed);
  return SINKATTN_OK;
}

int sinkattn_merge(const float* part_acc, const float* part_md, const float* sinks, int32_t rows,
                   int32_t num_qo_heads, int32_t head_dim, int32_t num_splits, void* out,
                   float* lse, void* stream) {
  g_last_error[0] = '\0';
  if (!part_acc || !part_md || !out)
    return fail(SINKATTN_INVALID_ARG, "part_acc, part_md and out must be non-null");
  if (!aligned16(part_acc) || !aligned16(part_md) || !aligned16(out))
    return fail(SINKATTN_INVALID_ARG, "part_acc, part_md and out must be 16-byte aligned");
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(SINKATTN_INVALID_ARG, "lse must be 4-byte aligned");
  if (rows < 0 || num_qo_heads <= 0) return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (head_dim != 64 && head_dim != 128)
    return fail(SINKATTN_UNSUPPORTED, "head_dim %d is not 64 or 128", head_dim);
  if (num_splits < 1) return fail(SINKATTN_INVALID_ARG, "num_splits must be at least 1");
  return launch_merge(part_acc, part_md, sinks, rows, num_qo_heads, head_dim, num_splits, out,
                      lse, static_cast<cudaStream_t>(stream), false);
}

int sinkattn_decode_workspace_bytes(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                    int32_t head_dim, int32_t num_splits, size_t* bytes) {
  g_last_error[0] = '\0';
  if (!bytes) return fail(SINKATTN_INVALID_ARG, "bytes must be non-null");
  if (batch < 0 || q_len < 1 || num_qo_heads <= 0 || num_splits < 1)
    return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (head_dim != 64 && head_dim != 128)
    return fail(SINKATTN_UNSUPPORTED, "head_dim %d is not 64 or 128", head_dim);
  const size_t slots = static_cast<size_t>(batch) * q_len * num_qo_heads * num_splits;
  const size_t acc = (slots * head_dim * 4 + 255) & ~static_cast<size_t>(255);
  *bytes = acc + slots * 2 * 4;
  return SINKATTN_OK;
}

int sinkattn_decode_default_splits(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t max_kv_len,
                                   int32_t* num_splits) {
  g_last_error[0] = '\0';
  if (!num_splits) return fail(SINKATTN_INVALID_ARG, "num_splits must be non-null");
  if (batch < 0 || q_len < 1 || num_qo_heads <= 0 || num_kv_heads <= 0 || max_kv_len < 0)
    return fail(SINKATTN_INVALID_ARG, "bad sizes");
  if (head_dim != 64 && head_dim != 128)
    return fail(SINKATTN_UNSUPPORTED, "head_dim %d is not 64 or 128", head_dim);
  // Aim for ~4 work items per SM slot so variable lengths even out, but keep
  // each chunk at least 4 KV tiles long (shorter chunks mostly cost partials).
  const int64_t items = static_cast<int64_t>(batch) * num_kv_heads;
  const int64_t target = 8 * static_cast<int64_t>(sm_count());
  int64_t s = items > 0 ? (target + items - 1) / items : 1;
  const int kt = head_dim == 64 ? 64 : 32;
  const int64_t cap = max_kv_len / (4 * kt);
  if (s > cap) s = cap;
  if (s < 1) s = 1;
  if (s > 16) s = 16;
  *num_splits = static_cast<int32_t>(s);
  return SINKATTN_OK;
}

int sinkattn_decode(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                    int32_t batch, int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                    int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                    int32_t window, int32_t num_splits, const float* sinks, void* workspace,
                    size_t workspace_bytes, void* out, float* lse, void* stream) {
  return decode_impl(q, k, v, kv_indptr, nullptr, batch, q_len, max_kv_len, num_qo_heads,
                     num_kv_heads, head_dim, sm_scale, causal, window, num_splits, sinks,
                     workspace, workspace_bytes, out, lse, stream);
}

int sinkattn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                          const int32_t* kv_indptr, const int32_t* page_indptr,
                          const int32_t* page_indices, int32_t num_pages, int32_t page_size,
                          int32_t batch, int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                          int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                          int32_t window, int32_t num_splits, const float* sinks, void* workspace,
                          size_t workspace_bytes, void* out, float* lse, void* stream) {
  const PagedKv pg{page_indptr, page_indices, num_pages, page_size};
  return decode_impl(q, k_pages, v_pages, kv_indptr, &pg, batch, q_len, max_kv_len, num_qo_heads,
                     num_kv_heads, head_dim, sm_scale, causal, window, num_splits, sinks,
                     workspace, workspace_bytes, out, lse, stream);
}

int sinkattn_decode_fused(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                          int32_t batch, int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                          int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                          int32_t window, int32_t num_splits, const float* sinks, void* out,
                          float* lse, void* stream) {
  g_last_error[0] = '\0';
  int rc = check_common(q, k, v, num_qo_heads, num_kv_heads, head_dim, sm_scale, causal, window);
  if (rc) return rc;
  if (!kv_indptr) return fail(SINKATTN_INVALID_ARG, "kv_indptr must be non-null");
  if (!out || !aligned16(out)) return fail(SINKATTN_INVALID_ARG, "out must be non-null and 16-byte aligned");
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(SINKATTN_INVALID_ARG, "lse must be 4-byte aligned");
  if (batch < 0 || max_kv_len < 0) return fail(SINKATTN_INVALID_ARG, "sizes must be non-negative");
  if (batch > 65535) return fail(SINKATTN_UNSUPPORTED, "batch %d exceeds 65535", batch);
  if (q_len < 1) return fail(SINKATTN_INVALID_ARG, "q_len must be at least 1");
  if (q_len > max_kv_len)
    return fail(SINKATTN_INVALID_ARG, "q_len (%d) exceeds max_kv_len (%d)", q_len, max_kv_len);
  if (num_qo_heads / num_kv_heads > 64)
    return fail(SINKATTN_UNSUPPORTED, "GQA group of %d heads exceeds 64", num_qo_heads / num_kv_heads);
  if (static_cast<int64_t>(num_kv_heads) * batch * max_kv_len >= (int64_t{1} << 31))
    return fail(SINKATTN_UNSUPPORTED, "problem too large");
  if (num_splits <= 0) {
    rc = sinkattn_decode_default_splits(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                        max_kv_len, &num_splits);
    if (rc) return rc;
  }
  if (num_splits > 16)
    return fail(SINKATTN_UNSUPPORTED, "num_splits %d exceeds the 16 CTAs of a cluster", num_splits);
  if (batch == 0) return SINKATTN_OK;
  AttnArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.cu_q = nullptr; a.cu_k = kv_indptr;
  a.batch = batch; a.q_len = q_len; a.max_q = q_len; a.max_kv = max_kv_len;
  a.Hq = num_qo_heads; a.Hkv = num_kv_heads; a.d = head_dim;
  a.sm_scale = sm_scale; a.causal = causal; a.window = window; a.num_splits = num_splits;
  a.sinks = sinks; a.out = out; a.lse = lse;
  return launch_attn_mma_fused(a, static_cast<cudaStream_t>(stream));
}

int sinkattn_debug_status(void* stream, int* status) {
  g_last_error[0] = '\0';
  if (!status) return fail(SINKATTN_INVALID_ARG, "status must be non-null");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int a = 0, m = 0, t = 0, dt = 0, sh = 0, pg = 0, px = 0, ro = 0, pb = 0;
  if (read_status_attn_mma(s, &a) || read_status_merge(s, &m) || read_status_prefill_tc(s, &t) ||
      read_status_decode_tc(s, &dt) || read_status_shared(s, &sh) || read_status_pages(s, &pg) ||
      read_status_prefix_tc(s, &px) || read_status_rope(s, &ro) || read_status_prefill_back(s, &pb))
    return fail(SINKATTN_CUDA_ERROR, "reading the device status failed: %s",
                cudaGetErrorString(cudaGetLastError()));
  *status = a ? a : (dt ? dt : (t ? t : (m ? m : (px ? px : (sh ? sh : (pg ? pg : (pb ? pb : ro)))))));
  return SINKATTN_OK;
}

int sinkattn_debug_set_hooks(long long wait_limit_cycles, int skip_tile) {
  g_last_error[0] = '\0';
  if (skip_tile < -1) return fail(SINKATTN_INVALID_ARG, "skip_tile must be -1 or a tile index");
  if (set_hooks_attn_mma(wait_limit_cycles, skip_tile) ||
      set_hooks_prefill_tc(wait_limit_cycles, skip_tile) ||
      set_hooks_decode_tc(wait_limit_cycles, skip_tile) ||
      set_hooks_prefix_tc(wait_limit_cycles, skip_tile) ||
      set_hooks_pages(wait_limit_cycles, skip_tile) ||
      set_hooks_prefill_back(wait_limit_cycles, skip_tile))
    return fail(SINKATTN_CUDA_ERROR, "setting the test hooks failed: %s",
                cudaGetErrorString(cudaGetLastError()));
  return SINKATTN_OK;
}

}  // extern "C"
