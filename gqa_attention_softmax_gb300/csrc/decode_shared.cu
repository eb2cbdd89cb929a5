// Decode over a paged cache whose sequences share prefixes: the plan.
//
// With M the maximum over both parts, softmax over a sequence's keys splits
// into its group's prefix (keys 0 .. P - 1) and its own keys (P .. L - 1):
//   sum_j e^{l_j - M} v_j = sum_{j < P} ... + sum_{j >= P} ...,
// so the two parts are two sets of split-KV partials of the same rows, and the
// merge folds them with the sink once. The prefix part of all sequences of a
// group is one attention of (sequences x drafts x query heads) rows over the
// same P keys, read once; the own part is a split-KV decode whose page lists
// start behind the prefix. One small launch derives both parts' lengths and
// page-list starts from the caller's arrays, so the call needs no host copy.
#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_shared;

namespace {

struct PlanParams {
  const int32_t* kv_indptr;
  const int32_t* page_indptr;
  const int32_t* group_indptr;
  const int32_t* prefix_lens;
  int groups, page_size, batch, q_len, max_prefix, max_suffix, block_tokens, tile_keys, Hkv;
  SharedPlan out;
};

constexpr int kThreads = 1024;

// Inclusive sum over the block; *total gets the block's sum.
__device__ __forceinline__ int block_sum_scan(int v, int* total, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  int w = sums[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kThreads) shared_plan_kernel(const PlanParams p) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  grid_launch_dependents();   // the next launch sets itself up meanwhile, and waits for this one
  bool bad = false;
  // the keys of group g's prefix that can be used
  auto prefix_of = [&](int g, bool* wrong) -> int {
    const int len = p.prefix_lens[g];
    const bool ok = len >= 0 && len <= p.max_prefix && len % p.page_size == 0;
    if (!ok) *wrong = true;
    return ok ? len : 0;
  };
  // the groups have to cut the batch into runs, or none of them has rows
  bool broken = false;
  for (int g = tid; g < p.groups; g += kThreads) {
    const int b0 = p.group_indptr[g], b1 = p.group_indptr[g + 1];
    broken |= b0 < 0 || b1 < b0 || b1 > p.batch || (g == 0 && b0 != 0) ||
              (g == p.groups - 1 && b1 != p.batch);
  }
  broken = __syncthreads_or(broken);
  int run = 0, run_unit = 0, total;
  for (int base = 0; base < p.groups; base += kThreads) {
    const int g = base + tid;
    int len = 0, units = 0;
    if (g < p.groups && !broken) {
      const int b0 = p.group_indptr[g], b1 = p.group_indptr[g + 1];
      len = prefix_of(g, &bad);
      // the first sequence's list holds the prefix
      if (b1 > b0 && len > (p.page_indptr[b0 + 1] - p.page_indptr[b0]) * p.page_size) {
        bad = true;
        len = 0;
      }
      // row blocks x KV heads x key tiles (below 2^31: checked on the host)
      units = ((b1 - b0) * p.q_len + p.block_tokens - 1) / p.block_tokens * p.Hkv *
              ((len + p.tile_keys - 1) / p.tile_keys);
      p.out.grp_q[g] = b0 * p.q_len;
      p.out.grp_pages[g] = p.page_indptr[b0];
    } else if (g < p.groups) {
      p.out.grp_q[g] = p.batch * p.q_len;
      p.out.grp_pages[g] = p.page_indptr[p.batch];
    }
    const int upto = run + block_sum_scan(len, &total, sums);
    run += total;
    const int upto_unit = run_unit + block_sum_scan(units, &total, sums);
    run_unit += total;
    if (g < p.groups) {
      p.out.grp_k[g + 1] = upto;
      p.out.grp_unit[g + 1] = upto_unit;
    }
  }
  if (tid == 0) {
    p.out.grp_q[p.groups] = p.batch * p.q_len;
    p.out.grp_pages[p.groups] = p.page_indptr[p.batch];
    p.out.grp_unit[0] = 0;
  }
  if (tid == 0) p.out.grp_k[0] = p.out.kv[0] = 0;
  run = 0;
  for (int base = 0; base < p.batch; base += kThreads) {
    const int b = base + tid;
    int own = 0;
    if (b < p.batch) {
      int lo = 0, hi = broken ? 1 : p.groups;   // the group with group_indptr[g] <= b < group_indptr[g + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.group_indptr[mid] <= b) lo = mid;
        else hi = mid;
      }
      const int len = p.kv_indptr[b + 1] - p.kv_indptr[b];
      const int first = p.page_indptr[b], held = p.page_indptr[b + 1] - first;
      int prefix = broken ? 0 : prefix_of(lo, &bad);
      own = len - prefix;
      if (own < p.q_len || own > p.max_suffix || len > held * p.page_size) {
        bad = true;
        own = prefix = 0;
      }
      p.out.pages[b] = first + prefix / p.page_size;
      for (int t = 0; t < p.q_len; ++t) p.out.row_pos[b * p.q_len + t] = len - p.q_len + t;
      if (b == p.batch - 1) p.out.pages[p.batch] = p.page_indptr[p.batch];
    }
    const int upto = run + block_sum_scan(own, &total, sums);
    if (b < p.batch) p.out.kv[b + 1] = upto;
    run += total;
  }
  if (__syncthreads_or(bad || broken) && tid == 0) atomicExch(&g_status_shared, SINKATTN_BAD_LENGTHS);
}

}  // namespace

int launch_shared_plan(const int32_t* kv_indptr, const int32_t* page_indptr,
                       const int32_t* group_indptr, const int32_t* prefix_lens, int32_t groups,
                       int32_t page_size, int32_t batch, int32_t q_len, int32_t max_prefix,
                       int32_t max_suffix, int32_t block_tokens, int32_t tile_keys, int32_t Hkv,
                       const SharedPlan& plan, cudaStream_t stream) {
  const PlanParams p{kv_indptr,  page_indptr, group_indptr, prefix_lens, groups, page_size, batch,
                     q_len,      max_prefix,  max_suffix,   block_tokens, tile_keys, Hkv,   plan};
  shared_plan_kernel<<<1, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("shared-prefix plan launch: %s", cudaGetErrorString(e));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

int read_status_shared(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_shared, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  if (cudaMemcpyToSymbolAsync(g_status_shared, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
      cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn
