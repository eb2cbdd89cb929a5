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
// page-list starts from the caller's arrays, so the call needs no host copy: a
// block of 1024 threads, about 4 us of load, barrier and scan latency.
#include "chain.cuh"
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
  int groups, page_shift, batch, q_len, max_prefix, max_suffix, block_tokens, tile_keys, Hkv;
  int window;
  int splits;          // partials a row block may have
  float class_scale;   // own keys -> class
  SharedCost cost;
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

constexpr int kClasses = 64;   // of own lengths

__global__ void __launch_bounds__(kThreads, 1) shared_plan_kernel(const PlanParams p) {
  __shared__ int sums[32];
  __shared__ int count_s[kClasses], place_s[kClasses];
  __shared__ float own_s[32];
  __shared__ int longest_s;   // tiles of the longest prefix
  const int tid = threadIdx.x;
  grid_launch_dependents();   // the next launch sets itself up meanwhile, and waits for this one
  if (tid < kClasses) count_s[tid] = 0;
  if (tid == 0) longest_s = 0;
  // the first sequence of each thread: loads that depend on nothing
  int len0 = 0, page0 = 0, held0 = 0;
  if (tid < p.batch) {
    len0 = p.kv_indptr[tid + 1] - p.kv_indptr[tid];
    page0 = p.page_indptr[tid];
    held0 = p.page_indptr[tid + 1] - page0;
  }
  bool bad = false;
  // the keys of group g's prefix that can be used
  auto prefix_of = [&](int g, bool* wrong) -> int {
    const int len = p.prefix_lens[g];
    const bool ok = len >= 0 && len <= p.max_prefix && (len & ((1 << p.page_shift) - 1)) == 0;
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
      const int first = p.page_indptr[b0];
      // the first sequence's list holds the prefix
      if (b1 > b0 && len > (p.page_indptr[b0 + 1] - first) << p.page_shift) {
        bad = true;
        len = 0;
      }
      // row blocks x KV heads x key tiles (below 2^31: checked on the host)
      units = ((b1 - b0) * p.q_len + p.block_tokens - 1) / p.block_tokens;
      if (p.tile_keys > 0) {
        const int tiles = (len + p.tile_keys - 1) / p.tile_keys;
        units *= p.Hkv * tiles;
        if (b1 > b0) atomicMax(&longest_s, tiles);
      }
      p.out.grp_q[g] = b0 * p.q_len;
      p.out.grp_pages[g] = first;
    } else if (g < p.groups) {
      // all rows are the first group's, without a prefix
      if (g == 0 && p.tile_keys == 0) units = (p.batch * p.q_len + p.block_tokens - 1) / p.block_tokens;
      p.out.grp_q[g] = g == 0 ? 0 : p.batch * p.q_len;
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
  // The sequences: own keys and where their pages start. A sequence's class
  // goes by its length, longest first; the order within a class is whoever
  // comes first, which moves work between SMs and no result.
  struct Own {
    int len, page, kind;
  };
  auto own_of = [&](int b) -> Own {
    int lo = 0, hi = broken ? 1 : p.groups;   // the group with group_indptr[g] <= b < group_indptr[g + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.group_indptr[mid] <= b) lo = mid;
      else hi = mid;
    }
    const int len = b == tid ? len0 : p.kv_indptr[b + 1] - p.kv_indptr[b];
    const int first = b == tid ? page0 : p.page_indptr[b];
    const int held = b == tid ? held0 : p.page_indptr[b + 1] - first;
    int prefix = broken ? 0 : prefix_of(lo, &bad);
    int own = len - prefix;
    if (own < p.q_len || own > p.max_suffix || len > held << p.page_shift) {
      bad = true;
      own = prefix = 0;
    }
    const int kind = kClasses - 1 - min(kClasses - 1, static_cast<int>(static_cast<float>(own) * p.class_scale));
    return {own, first + (prefix >> p.page_shift), kind};
  };
  Own mine{};
  float keys = 0.f;   // own keys of the batch (for the quota only)
  for (int b = tid; b < p.batch; b += kThreads) {
    const Own o = own_of(b);
    if (b == tid) mine = o;
    atomicAdd(&count_s[o.kind], 1);
    keys += static_cast<float>(o.len);
    if (p.window > 0) {
      const int len = b == tid ? len0 : p.kv_indptr[b + 1] - p.kv_indptr[b];
      for (int t = 0; t < p.q_len; ++t) p.out.row_pos[b * p.q_len + t] = len - p.q_len + t;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) keys += __shfl_xor_sync(0xffffffffu, keys, off);
  if ((tid & 31) == 0) own_s[tid >> 5] = keys;
  __syncthreads();
  if (tid < 32) {   // where each class starts
    const int c0 = count_s[2 * tid], c1 = count_s[2 * tid + 1];
    int x = c0 + c1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (tid >= off) x += y;
    }
    place_s[2 * tid] = x - c0 - c1;
    place_s[2 * tid + 1] = x - c1;
  }
  __syncthreads();
  for (int b = tid; b < p.batch; b += kThreads) {
    const Own o = b == tid ? mine : own_of(b);
    const int at = atomicAdd(&place_s[o.kind], 1);
    p.out.own_seq[at] = b;
    p.out.own_len[at] = o.len;
    p.out.own_page[at] = o.page;
  }
  if (tid == 0) {
    p.out.grp_k[0] = 0;
    p.out.grp_q[p.groups] = p.batch * p.q_len;
    p.out.grp_pages[p.groups] = p.page_indptr[p.batch];
    p.out.grp_unit[0] = 0;
    // units of one thread block: an even share, or, where the own pass runs
    // beside the prefix, what keeps a block busy for as long as all work takes,
    // up to twice that (64 sequences behind 8192 keys, up to 1024 own keys:
    // 35.5 us with the even 10, 32.9 with 15; short prefixes lose by more)
    int quota = (run_unit + p.cost.sms - 1) / p.cost.sms;
    if (p.cost.own_key > 0.f) {
      float own = 0.f;
      for (int w = 0; w < 32; ++w) own += own_s[w];
      const float all = (static_cast<float>(run_unit) * p.cost.unit + own * p.cost.own_key) /
                        static_cast<float>(p.cost.sms);
      quota = max(quota, min(2 * quota, static_cast<int>((all - p.cost.ramp) / p.cost.unit)));
    }
    // a row block of T tiles meets at most ceil((T - 1) / quota) + 1 runs of units
    if (p.splits > 1) quota = max(quota, (longest_s - 1 + p.splits - 2) / (p.splits - 1));
    *p.out.quota = max(quota, 1);
  }
  if (__syncthreads_or(bad || broken) && tid == 0) atomicExch(&g_status_shared, SINKATTN_BAD_LENGTHS);
}

}  // namespace

int launch_shared_plan(const int32_t* kv_indptr, const int32_t* page_indptr,
                       const int32_t* group_indptr, const int32_t* prefix_lens, int32_t groups,
                       int32_t page_size, int32_t batch, int32_t q_len, int32_t max_prefix,
                       int32_t max_suffix, int32_t block_tokens, int32_t tile_keys, int32_t Hkv,
                       int32_t window, int32_t splits, const SharedCost& cost, const SharedPlan& plan,
                       cudaStream_t stream) {
  PlanParams p{};
  p.kv_indptr = kv_indptr;
  p.page_indptr = page_indptr;
  p.group_indptr = group_indptr;
  p.prefix_lens = prefix_lens;
  p.groups = groups;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.batch = batch;
  p.q_len = q_len;
  p.max_prefix = max_prefix;
  p.max_suffix = max_suffix;
  p.block_tokens = block_tokens;
  p.tile_keys = tile_keys;
  p.Hkv = Hkv;
  p.window = window;
  p.splits = splits;
  p.class_scale = static_cast<float>(kClasses) / (static_cast<float>(max_suffix) + 1.f);
  p.cost = cost;
  p.out = plan;
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
