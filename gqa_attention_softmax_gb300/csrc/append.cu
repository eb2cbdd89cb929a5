// Writes new keys and values into the pages of a paged cache, as bf16 or as
// e4m3 codes under one scale per KV head (rules: sinkattn.h).
//
// One pass: each thread takes one 16-byte run of a pool row in K and the same
// run in V, so a row (head_dim elements of one head of one
// token) is written in full 16-byte lanes, and consecutive lanes read
// consecutive heads of the token. With codes a thread reads two 16-byte runs
// per pool instead of one.
//
// The code is the one nearest to the correctly rounded quotient x / s. 32 IEEE
// divisions a thread would take longer than its bytes, so the quotient comes
// from r = RN(1 / s) by one residual step, q0 = RN(x r), q = RN(q0 + r (x -
// q0 s)) with the residual exact in an fma: Markstein's theorem ("Computation
// of elementary functions on the IBM RISC System/6000", 1990) makes q the
// correctly rounded quotient where nothing over- or underflows. The residual's
// last bit is that of q0 s: with q0 >= 2^-11 (half the least quotient whose code
// is not zero) and s >= 2^-90 at least 2^(-11-23-90-23) = 2^-147, above fp32's
// 2^-149. Scales outside [2^-90, 2^100] (negative ones, whose zeros it would
// give the wrong sign) take IEEE divisions.
//
// 22000 tokens of 4 heads of 128 (68 MB) take 10.4 us as codes with all of it in
// L2, 17.6 from DRAM, where the bytes alone are 10 and the latency of the loads
// binds: 64 registers a thread leave 41 % of the warps resident, and 5 of the 12
// cycles from a warp's instruction to its next are a load's (issue slots 53 %,
// ALU 50 %).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sinkattn {

namespace {

struct AppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_stride, v_stride;   // elements between tokens
  const int32_t* slots;
  const float* k_scale;
  const float* v_scale;
  uint8_t* k_pages;
  uint8_t* v_pages;
  int tokens, Hkv, shift;         // page size = 1 << shift
  int per_block;                  // tokens of a thread block
  long long n_slots;
};

struct Scale {
  float s, r;   // the scale and RN(1 / s)
  bool plain;   // s is in the range of the residual step
};

__device__ __forceinline__ Scale make_scale(float s) {
  return {s, __frcp_rn(s), s >= 0x1p-90f && s <= 0x1p100f};
}

template <bool PLAIN>
__device__ __forceinline__ float quotient(float x, const Scale& c) {
  if constexpr (!PLAIN) return __fdiv_rn(x, c.s);
  const float q0 = x * c.r;
  // q0 s - x, and not x - q0 s: for x = -0 the first is +0 and the sum below -0 - 0,
  // where the second is +0 too and the sum -0 + 0 = +0 (a select for zeros instead: 10.4 -> 11.8 us)
  const float q = fmaf(-fmaf(q0, c.s, -x), c.r, q0);
  // (an infinity, or a value that saturates, stays as it is; so does NaN)
  return fabsf(q0) < 1024.f ? q : q0;
}

template <bool PLAIN>
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, const Scale& c) {
  const float x0 = quotient<PLAIN>(__uint_as_float(lo << 16), c);
  const float x1 = quotient<PLAIN>(__uint_as_float(lo & 0xffff0000u), c);
  const float x2 = quotient<PLAIN>(__uint_as_float(hi << 16), c);
  const float x3 = quotient<PLAIN>(__uint_as_float(hi & 0xffff0000u), c);
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x3), "f"(x2));
  return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
}

template <bool PLAIN>
__device__ __forceinline__ uint4 codes16_t(uint4 a, uint4 b, const Scale& c) {
  return make_uint4(codes4<PLAIN>(a.x, a.y, c), codes4<PLAIN>(a.z, a.w, c),
                    codes4<PLAIN>(b.x, b.y, c), codes4<PLAIN>(b.z, b.w, c));
}

// Sixteen bf16 (two 16-byte vectors) -> sixteen e4m3 codes of x / scale.
__device__ __forceinline__ uint4 codes16(uint4 a, uint4 b, float scale) {
  const Scale c = make_scale(scale);
  return c.plain ? codes16_t<true>(a, b, c) : codes16_t<false>(a, b, c);
}

// A block takes p.per_block tokens; a thread takes its runs kIlp at a time,
// with all loads of a step in flight before the first store.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  constexpr int EL = FP8 ? 16 : 8;         // elements of a thread's 16-byte run in a pool
  constexpr int RUNS = D / EL;
  constexpr int ROW = D * (FP8 ? 1 : 2);   // bytes of a pool row
  constexpr int kIlp = 2;
  const int per = p.Hkv * RUNS;
  const int tok0 = blockIdx.x * p.per_block;
  const int n = min(p.per_block, p.tokens - tok0) * per;
  for (int u0 = threadIdx.x; u0 < n; u0 += kIlp * 256) {
    uint4 k[kIlp], v[kIlp], k2[kIlp], v2[kIlp];
    int slot[kIlp], run[kIlp];
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      const int u = u0 + i * 256;
      slot[i] = -1;
      if (u >= n) continue;
      const int tok = tok0 + u / per;
      run[i] = u % per;
      slot[i] = p.slots[tok];
      const uint4* ks = reinterpret_cast<const uint4*>(p.k + tok * p.k_stride + run[i] * EL);
      const uint4* vs = reinterpret_cast<const uint4*>(p.v + tok * p.v_stride + run[i] * EL);
      k[i] = __ldcs(ks);
      v[i] = __ldcs(vs);
      if constexpr (FP8) {
        k2[i] = __ldcs(ks + 1);
        v2[i] = __ldcs(vs + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      if (slot[i] < 0 || slot[i] >= p.n_slots) continue;   // a padding token
      const int h = run[i] / RUNS, c = run[i] % RUNS;
      if constexpr (FP8) {
        k[i] = codes16(k[i], k2[i], p.k_scale[h]);
        v[i] = codes16(v[i], v2[i], p.v_scale[h]);
      }
      const long long row = ((static_cast<long long>(slot[i] >> p.shift) * p.Hkv + h) << p.shift) +
                            (slot[i] & ((1 << p.shift) - 1));
      *reinterpret_cast<uint4*>(p.k_pages + row * ROW + c * 16) = k[i];
      *reinterpret_cast<uint4*>(p.v_pages + row * ROW + c * 16) = v[i];
    }
  }
}

int refuse(int status, const char* text) {
  set_error("%s", text);
  return status;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
           int32_t tokens, const float* k_scale, const float* v_scale, bool fp8, void* k_pages,
           void* v_pages, int32_t num_pages, int32_t page_size, int32_t Hkv, int32_t d,
           void* stream) {
  set_error("%s", "");
  if (tokens < 0) return refuse(SINKATTN_INVALID_ARG, "tokens must be non-negative");
  if (!k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return refuse(SINKATTN_INVALID_ARG, "k_pages and v_pages must be non-null and 16-byte aligned");
  if (Hkv < 1 || num_pages < 1)
    return refuse(SINKATTN_INVALID_ARG, "num_kv_heads and num_pages must be positive");
  if (d != 64 && d != 128) return refuse(SINKATTN_UNSUPPORTED, "head_dim is not 64 or 128");
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return refuse(SINKATTN_UNSUPPORTED, "page_size is not a power of two in [16, 256]");
  if (static_cast<int64_t>(num_pages) * Hkv * page_size >= (int64_t{1} << 31))
    return refuse(SINKATTN_UNSUPPORTED, "page pools exceed 2^31 rows");
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return refuse(SINKATTN_INVALID_ARG, "k_scale and v_scale must be non-null and 4-byte aligned");
  if (tokens == 0) return SINKATTN_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !slots || !aligned(slots, 4))
    return refuse(SINKATTN_INVALID_ARG,
                  "k and v must be non-null and 16-byte aligned, slots 4-byte aligned");
  const int64_t width = static_cast<int64_t>(Hkv) * d;
  if (k_stride < width || v_stride < width || k_stride % 8 || v_stride % 8)
    return refuse(SINKATTN_INVALID_ARG,
                  "k_stride and v_stride must be multiples of 8 and at least num_kv_heads * head_dim");
  AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.tokens = tokens;
  p.Hkv = Hkv;
  while ((1 << p.shift) < page_size) ++p.shift;
  p.n_slots = static_cast<long long>(num_pages) * page_size;
  const int64_t per = width / (fp8 ? 16 : 8);   // runs of a token
  if (per > (1 << 20)) return refuse(SINKATTN_UNSUPPORTED, "more than 2^20 runs in a token");
  // two runs a thread, but one while that leaves SMs without a block (with the
  // reserve and the lists of the same tokens and a copy of the table: 22000
  // tokens as codes 23.2 us with two, 23.8 with one; 64 tokens 11.1 and 10.8)
  const int64_t blocks1 = (tokens * per + 255) / 256;
  const int64_t runs = blocks1 >= 8LL * sm_count() ? 512 : 256;
  p.per_block = static_cast<int>(std::max<int64_t>(1, runs / per));
  const unsigned blocks = static_cast<unsigned>((int64_t{tokens} + p.per_block - 1) / p.per_block);
  auto kern = d == 64 ? (fp8 ? append_kernel<64, true> : append_kernel<64, false>)
                      : (fp8 ? append_kernel<128, true> : append_kernel<128, false>);
  kern<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("append launch: %s", cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

}  // namespace
}  // namespace sinkattn

extern "C" {

int sinkattn_append_paged(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                          const int32_t* slots, int32_t tokens, void* k_pages, void* v_pages,
                          int32_t num_pages, int32_t page_size, int32_t num_kv_heads,
                          int32_t head_dim, void* stream) {
  return sinkattn::append(k, v, k_stride, v_stride, slots, tokens, nullptr, nullptr, false, k_pages,
                          v_pages, num_pages, page_size, num_kv_heads, head_dim, stream);
}

int sinkattn_append_paged_fp8(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                              const int32_t* slots, int32_t tokens, const float* k_scale,
                              const float* v_scale, void* k_pages, void* v_pages,
                              int32_t num_pages, int32_t page_size, int32_t num_kv_heads,
                              int32_t head_dim, void* stream) {
  return sinkattn::append(k, v, k_stride, v_stride, slots, tokens, k_scale, v_scale, true, k_pages,
                          v_pages, num_pages, page_size, num_kv_heads, head_dim, stream);
}

}  // extern "C"
