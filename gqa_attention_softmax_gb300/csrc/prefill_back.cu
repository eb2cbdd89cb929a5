// Backward pass of the varlen prefill with a per-head softmax sink (rules:
// sinkattn.h). With P = exp(l - lse) over the visible keys and delta = dout .
// out - dlse, dS = P (dout v^T - delta): dq = c dS k, dk = c dS^T q, dv = P^T
// dout, dsink = -sum exp(s - lse) delta.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_prefill_back;

namespace {

struct BackParams {
  const __nv_bfloat16 *dout, *q, *k, *v, *out;
  const float *lse, *sinks, *dlse;
  const int32_t *cu_q, *cu_k;
  int batch, total_q, total_k, max_q, max_kv, Hq, Hkv, G;
  float sm_scale;
  int causal, window;
  __nv_bfloat16 *dq, *dk, *dv;
  float *dsinks, *delta, *sink_part;
  int per;   // tokens of a block of the delta pass
};

__device__ __forceinline__ float dot8(uint4 x, uint4 y, float s) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
    s = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), s);
  }
  return s;
}

constexpr int kDeltaRows = 1024;   // rows (token, head) of a block of the delta pass at most
constexpr int kDeltaHeads = 256;   // heads of a block

// delta of p.per tokens and up to kDeltaHeads heads, d / 8 threads a row, and
// those rows' sum of the sinks' gradients, in the order of the tokens.
template <int D>
__global__ void __launch_bounds__(256) back_delta_kernel(const BackParams p) {
  constexpr int C = D / 8;
  __shared__ float term[kDeltaRows];
  const int h0 = blockIdx.y * kDeltaHeads;
  const int nh = min(kDeltaHeads, p.Hq - h0);
  const int t0 = blockIdx.x * p.per;
  const int total = min(p.total_q, p.cu_q[p.batch]);   // rows behind it are not read
  const int nt = min(p.per, total - t0);
  const int rows = max(nt, 0) * nh;
  const int c = threadIdx.x % C;
  for (int base = 0; base < rows; base += 256 / C) {
    const int r = base + threadIdx.x / C;
    float s = 0.f;
    long long at = 0;
    int h = 0;
    if (r < rows) {
      h = h0 + r % nh;
      at = static_cast<long long>(t0 + r / nh) * p.Hq + h;
      s = dot8(__ldcs(reinterpret_cast<const uint4*>(p.dout + at * D) + c),
               __ldcs(reinterpret_cast<const uint4*>(p.out + at * D) + c), 0.f);
    }
#pragma unroll
    for (int m = 1; m < C; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (r < rows && c == 0) {
      if (p.dlse) s -= p.dlse[at];
      p.delta[at] = s;
      // a row with no visible key and no sink has lse -inf, but then there are no sinks
      if (p.sinks) term[r] = -expf(p.sinks[h] - p.lse[at]) * s;
    }
  }
  if (!p.sinks) return;
  __syncthreads();
  if (threadIdx.x < nh) {
    float s = 0.f;
    for (int t = 0; t < nt; ++t) s += term[t * nh + threadIdx.x];
    p.sink_part[static_cast<long long>(blockIdx.x) * p.Hq + h0 + threadIdx.x] = s;
  }
}

// dsinks: the blocks' sums added in a fixed order, 32 heads a block.
__global__ void __launch_bounds__(256) back_sinks_kernel(const float* part, int blocks, int Hq,
                                                         float* dsinks) {
  __shared__ float s[8][32];
  const int h = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  float x = 0.f;
  if (h < Hq)
    for (int b = slice; b < blocks; b += 8) x += part[static_cast<long long>(b) * Hq + h];
  s[slice][threadIdx.x % 32] = x;
  __syncthreads();
  if (slice != 0 || h >= Hq) return;
  for (int j = 1; j < 8; ++j) x += s[j][threadIdx.x];
  dsinks[h] = x;
}

struct Seq {
  int q0, lq, k0, lk;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const BackParams& p, int b) {
  Seq s;
  s.q0 = p.cu_q[b];
  s.lq = p.cu_q[b + 1] - s.q0;
  s.k0 = p.cu_k[b];
  s.lk = p.cu_k[b + 1] - s.k0;
  s.ok = s.q0 >= 0 && s.k0 >= 0 && s.lq >= 0 && s.lk >= s.lq && s.lq <= p.max_q &&
         s.lk <= p.max_kv && s.q0 <= p.total_q - s.lq && s.k0 <= p.total_k - s.lk;
  return s;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// One warp a query row: block (x, y, z) has rows 8 x .. 8 x + 7 of head y of sequence z.
template <int D>
__global__ void __launch_bounds__(256) back_dq_kernel(const BackParams p) {
  constexpr int N = D / 32;
  const Seq s = load_seq(p, blockIdx.z);
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + threadIdx.x / 32, h = blockIdx.y;
  if (!s.ok) {
    if (threadIdx.x == 0) atomicExch(&g_status_prefill_back, SINKATTN_BAD_LENGTHS);
    return;
  }
  if (i >= s.lq) return;
  const long long at = static_cast<long long>(s.q0 + i) * p.Hq + h;
  const int pos = s.lk - s.lq + i;
  const int hi = p.causal ? pos + 1 : s.lk;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float q[N], g[N], acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = __bfloat162float(p.q[at * D + e * 32 + lane]);
    g[e] = __bfloat162float(p.dout[at * D + e * 32 + lane]);
    acc[e] = 0.f;
  }
  const float lse = p.lse[at], delta = p.delta[at];
  const long long row0 = static_cast<long long>(p.Hkv) * s.k0 + static_cast<long long>(h / p.G) * s.lk;
  for (int j = lo; j < hi; ++j) {
    float k[N], a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      k[e] = __bfloat162float(p.k[(row0 + j) * D + e * 32 + lane]);
      a = fmaf(q[e], k[e], a);
      b = fmaf(g[e], __bfloat162float(p.v[(row0 + j) * D + e * 32 + lane]), b);
    }
    const float ds = expf(warp_sum(a) * p.sm_scale - lse) * (warp_sum(b) - delta);
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    p.dq[at * D + e * 32 + lane] = __float2bfloat16_rn(acc[e] * p.sm_scale);
}

// One warp a key: block (x, y, z) has keys 8 x .. 8 x + 7 of KV head y of sequence z.
template <int D>
__global__ void __launch_bounds__(256) back_dkv_kernel(const BackParams p) {
  constexpr int N = D / 32;
  const Seq s = load_seq(p, blockIdx.z);
  const int lane = threadIdx.x & 31;
  const int j = blockIdx.x * 8 + threadIdx.x / 32, kh = blockIdx.y;
  if (!s.ok) {
    if (threadIdx.x == 0) atomicExch(&g_status_prefill_back, SINKATTN_BAD_LENGTHS);
    return;
  }
  if (j >= s.lk) return;
  const long long row = static_cast<long long>(p.Hkv) * s.k0 + static_cast<long long>(kh) * s.lk + j;
  float k[N], v[N], dk[N], dv[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    k[e] = __bfloat162float(p.k[row * D + e * 32 + lane]);
    v[e] = __bfloat162float(p.v[row * D + e * 32 + lane]);
    dk[e] = dv[e] = 0.f;
  }
  // queries that see key j: positions j .. j + window - 1 (causal)
  const int first = s.lk - s.lq;
  const int lo = p.causal ? max(0, j - first) : 0;
  const int hi = p.window > 0
                     ? static_cast<int>(max(0LL, min(static_cast<long long>(s.lq),
                                                     static_cast<long long>(j) - first + p.window)))
                     : s.lq;
  for (int i = lo; i < hi; ++i)
    for (int g = 0; g < p.G; ++g) {
      const long long at = static_cast<long long>(s.q0 + i) * p.Hq + kh * p.G + g;
      float q[N], o[N], a = 0.f, b = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        q[e] = __bfloat162float(p.q[at * D + e * 32 + lane]);
        o[e] = __bfloat162float(p.dout[at * D + e * 32 + lane]);
        a = fmaf(q[e], k[e], a);
        b = fmaf(o[e], v[e], b);
      }
      const float w = expf(warp_sum(a) * p.sm_scale - p.lse[at]);
      const float ds = w * (warp_sum(b) - p.delta[at]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dv[e] = fmaf(w, o[e], dv[e]);
        dk[e] = fmaf(ds, q[e], dk[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    p.dk[row * D + e * 32 + lane] = __float2bfloat16_rn(dk[e] * p.sm_scale);
    p.dv[row * D + e * 32 + lane] = __float2bfloat16_rn(dv[e]);
  }
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

template <int D>
int launch_back(const BackParams& p, cudaStream_t stream) {
  int rc;
  if (p.total_q > 0) {
    const int64_t blocks = back_blocks(p.total_q, p.Hq);
    back_delta_kernel<D><<<dim3(static_cast<unsigned>(blocks),
                                static_cast<unsigned>((p.Hq + kDeltaHeads - 1) / kDeltaHeads)),
                           256, 0, stream>>>(p);
    if ((rc = launched("delta"))) return rc;
    back_dq_kernel<D><<<dim3((p.max_q + 7) / 8, p.Hq, p.batch), 256, 0, stream>>>(p);
    if ((rc = launched("dq"))) return rc;
  }
  back_dkv_kernel<D><<<dim3((p.max_kv + 7) / 8, p.Hkv, p.batch), 256, 0, stream>>>(p);
  if ((rc = launched("dk, dv"))) return rc;
  if (!p.dsinks) return SINKATTN_OK;
  back_sinks_kernel<<<(p.Hq + 31) / 32, 256, 0, stream>>>(
      p.sink_part, static_cast<int>(back_blocks(p.total_q, p.Hq)), p.Hq, p.dsinks);
  return launched("dsinks");
}

}  // namespace

int back_block_tokens(int32_t Hq) {
  return std::max(1, kDeltaRows / std::min<int32_t>(Hq, kDeltaHeads));
}

int launch_prefill_back(const BackArgs& a, cudaStream_t stream) {
  BackParams p{};
  p.dout = static_cast<const __nv_bfloat16*>(a.dout);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.out = static_cast<const __nv_bfloat16*>(a.out);
  p.lse = a.lse; p.sinks = a.sinks; p.dlse = a.dlse;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k;
  p.batch = a.batch; p.total_q = a.total_q; p.total_k = a.total_k;
  p.max_q = a.max_q; p.max_kv = a.max_kv;
  p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv;
  p.sm_scale = a.sm_scale; p.causal = a.causal; p.window = a.window;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.dsinks = a.dsinks; p.delta = a.delta; p.sink_part = a.sink_part;
  p.per = back_block_tokens(a.Hq);
  return a.d == 64 ? launch_back<64>(p, stream) : launch_back<128>(p, stream);
}

int read_status_prefill_back(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_prefill_back, sizeof(int), 0,
                                cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_status_prefill_back, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                              s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn
