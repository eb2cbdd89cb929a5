// Merge of split-KV partials with the sink counted exactly once: one warp
// per (row, query head) runs merge_row (merge_row.cuh).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "merge_row.cuh"

namespace sinkattn {

template <int D>
__global__ void __launch_bounds__(256)
    merge_kernel(const float* __restrict__ part_acc, const float* __restrict__ part_md,
                 const float* __restrict__ sinks, int n_rows, int Hq, int S,
                 __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int drop) {
  // Launched as a programmatic dependent of the partial kernel: wait until
  // that grid has completed and its writes are visible (immediate otherwise).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(n_rows) * Hq;
  const long long w0 = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w0 >= n) return;
  // newest rows first: the partial kernels finish the last sequences last,
  // so those partials are the ones still in L2
  const long long w = n - 1 - w0;
  const int h = static_cast<int>(w % Hq);
  const float* acc = part_acc + w * S * D;
  merge_row<D>(part_md + w * S * 2, acc, sinks ? sinks[h] : kNegInf, S, lane, out + w * D,
               lse != nullptr ? lse + w : nullptr);
  if (drop) {   // library-owned scratch: the row's accumulator lines are dead
    __syncwarp();
    const char* base = reinterpret_cast<const char*>(acc);
    for (int off = lane * 128; off < S * D * 4; off += 32 * 128)
      asm volatile("discard.global.L2 [%0], 128;" ::"l"(base + off) : "memory");
  }
}

__device__ int g_status_merge;

// Records SINKATTN_BAD_LENGTHS where the arrays of a shared-prefix call break a
// rule (the plan's own checks, for a call without one). Thread i has group i
// and sequence i.
__device__ __forceinline__ void check_shared(const SharedCheck& c, int i) {
  bool bad = false;
  if (i < c.groups) {
    const int b0 = c.group_indptr[i], b1 = c.group_indptr[i + 1], len = c.prefix_lens[i];
    const bool cut = b0 >= 0 && b1 >= b0 && b1 <= c.batch && (i > 0 || b0 == 0) &&
                     (i < c.groups - 1 || b1 == c.batch);
    bad = !cut || len < 0 || len > c.max_prefix || len % c.page_size != 0;
    if (cut && b1 > b0)
      bad |= len > static_cast<long long>(c.page_indptr[b0 + 1] - c.page_indptr[b0]) * c.page_size;
  }
  if (i < c.batch) {
    int lo = 0, hi = c.groups;   // the group with group_indptr[g] <= i < group_indptr[g + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.group_indptr[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int len = c.kv_indptr[i + 1] - c.kv_indptr[i];
    const long long own = static_cast<long long>(len) - c.prefix_lens[lo];
    bad |= own < c.q_len || own > c.max_suffix ||
           len > static_cast<long long>(c.page_indptr[i + 1] - c.page_indptr[i]) * c.page_size;
  }
  if (bad) atomicExch(&g_status_merge, SINKATTN_BAD_LENGTHS);
}

// The merge of shared-prefix decode: only the slots that hold keys are read, R
// rows per warp (R = 0: one row of more than 32 slots). Bound by two dependent
// reads per row and by HBM for partials that L2 no longer holds: 49152 rows of
// up to three partials at d 128 take 13.4 us (3.8 TB/s from cold).
template <int D, int R>
__global__ void __launch_bounds__(256)
    merge_sparse_kernel(const float* __restrict__ part_acc, const float* __restrict__ part_md,
                        const float* __restrict__ sinks, int n_rows, int Hq, int S,
                        __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                        const SharedCheck check) {
  const int beyond = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x) + check.blocks;
  if (beyond >= 0) {   // (reads nothing of the launch before)
    check_shared(check, beyond * 256 + static_cast<int>(threadIdx.x));
    return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(n_rows) * Hq;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if constexpr (R > 0) {
    if (w * R >= n) return;
    merge_rows_sparse<D, R>(part_md, part_acc, sinks, w * R,
                            static_cast<int>(min(static_cast<long long>(R), n - w * R)), Hq, S, lane,
                            out, lse);
  } else {
    if (w >= n) return;
    merge_row_sparse<D>(part_md + w * S * 2, part_acc + w * S * D,
                        sinks ? sinks[static_cast<int>(w % Hq)] : kNegInf, S, lane, out + w * D,
                        lse != nullptr ? lse + w : nullptr);
  }
}

int launch_merge_sparse(const float* part_acc, const float* part_md, const float* sinks,
                        int32_t rows, int32_t Hq, int32_t d, int32_t num_slots, void* out,
                        float* lse, const SharedCheck* check, cudaStream_t stream) {
  const long long n = static_cast<long long>(rows) * Hq;
  if (n == 0) return SINKATTN_OK;
  auto* o = static_cast<__nv_bfloat16*>(out);
  // Rows per warp as the slots allow, while every SM still gets its fill of
  // warps (49152 rows of 3 slots at d 128: 13.4 us with four rows a warp, 21.7
  // with one; 4096 rows of 11 at d 64: 6.8 with two, 6.1 with one).
  const int most = num_slots <= 8 ? 4 : num_slots <= 16 ? 2 : num_slots <= 32 ? 1 : 0;
  const int R = most > 1 && n / most < 64LL * sm_count() ? 1 : most;
  const unsigned blocks = static_cast<unsigned>((n + 8 * (R > 0 ? R : 1) - 1) / (8 * (R > 0 ? R : 1)));
  SharedCheck c = check ? *check : SharedCheck{};
  c.blocks = check ? (std::max(c.groups, c.batch) + 255) / 256 : 0;
  auto run = [&](auto kern) {
    return launch_chained(kern, dim3(blocks + c.blocks), 256, 0, stream, part_acc, part_md,
                          sinks, rows, Hq, num_slots, o, lse, c);
  };
  cudaError_t e;
  if (d == 64)
    e = R == 4   ? run(merge_sparse_kernel<64, 4>)
        : R == 2 ? run(merge_sparse_kernel<64, 2>)
        : R == 1 ? run(merge_sparse_kernel<64, 1>)
                 : run(merge_sparse_kernel<64, 0>);
  else
    e = R == 4   ? run(merge_sparse_kernel<128, 4>)
        : R == 2 ? run(merge_sparse_kernel<128, 2>)
        : R == 1 ? run(merge_sparse_kernel<128, 1>)
                 : run(merge_sparse_kernel<128, 0>);
  if (e != cudaSuccess) {
    set_error("merge kernel launch: %s", cudaGetErrorString(e));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

int launch_merge(const float* part_acc, const float* part_md, const float* sinks, int32_t rows,
                 int32_t Hq, int32_t d, int32_t num_splits, void* out, float* lse,
                 cudaStream_t stream, bool drop_partials) {
  const long long warps = static_cast<long long>(rows) * Hq;
  if (warps == 0) return SINKATTN_OK;
  const unsigned blocks = static_cast<unsigned>((warps + 7) / 8);
  auto* o = static_cast<__nv_bfloat16*>(out);
  // Programmatic stream serialisation: the launch may be processed while the
  // previous kernel on the stream (the partial kernel) drains its last CTAs;
  // the kernel's griddepcontrol.wait keeps the data dependency.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      d == 64 ? cudaLaunchKernelEx(&cfg, merge_kernel<64>, part_acc, part_md, sinks, rows, Hq,
                                   num_splits, o, lse, drop_partials ? 1 : 0)
              : cudaLaunchKernelEx(&cfg, merge_kernel<128>, part_acc, part_md, sinks, rows, Hq,
                                   num_splits, o, lse, drop_partials ? 1 : 0);
  if (e != cudaSuccess) {
    set_error("merge kernel launch: %s", cudaGetErrorString(e));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

int read_status_merge(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_merge, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  if (cudaMemcpyToSymbolAsync(g_status_merge, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
      cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn
