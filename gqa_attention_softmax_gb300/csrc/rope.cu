// Norm and position rotation of queries and keys, on the way from a fused
// projection's rows to the attention's layouts (q token-major, k and v ragged
// HND) or to the slots of a paged cache, and the gradients of the former
// (rules: sinkattn.h).
//
// A head's row x of d elements becomes y = R (w * x * rsqrt(mean x^2 + eps))
// (w: q_weight or k_weight; without one, no norm), where R turns pair i of the
// first r elements by the angle position * f_i and scales it by the attention
// factor. Backward: g = R^T dy, u = w * g, xh = x rs with rs = rsqrt(mean x^2 +
// eps), dx = rs (u - xh mean(u xh)), dw = sum of g xh over tokens and heads.
//
// Angles. The frequencies come as turns per position in units of 2^-64, so
// position * turns modulo 2^64 is the angle's fraction of a turn with an error
// of at most |position| 2^-65 turns, whatever the position; its upper 32 bits
// go to sincospif. A 32-bit product of position and frequency would be off by
// up to 2^-24 |position| radians instead.
//
// A thread holds eight elements of one head, four whole pairs, so that the
// rotation needs no exchange, and d / 8 threads hold a head. All heads of a
// token share its cosines: a block computes them once per token into shared
// memory. The mean squares and all arithmetic between the loads and the stores are
// 32-bit; each output is rounded once.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_rope;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;   // tokens of a block

enum Layout { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };
enum Kind { kPack = 0, kAppend = 1, kAppendFp8 = 2 };

struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;           // forward: the projection; backward: q, k before the norm
  long long q_stride, k_stride, v_stride;   // elements between tokens
  const int32_t* cu;                        // [batch + 1] (pack and backward)
  const int32_t* positions;                 // [tokens] or nullptr: the index in the sequence
  const unsigned long long* turns;          // [r / 2]
  const float *q_weight, *k_weight;         // [d] or nullptr
  float eps, factor;
  int tokens, batch, Hq, Hkv, r;
  uint32_t inv_heads;                       // ceil(2^32 / (Hq + 2 Hkv))
  int per_block, parts;                     // tokens of a block; blocks that share its heads
  __nv_bfloat16 *q_out, *k_out, *v_out;     // pack; append: q_out
  // append
  const int32_t* slots;
  const float *k_scale, *v_scale;
  uint8_t *k_pages, *v_pages;
  int shift;
  long long n_slots;
  // backward: dq [tokens, Hq, d], dk, dv ragged HND; gradients of the projection
  const __nv_bfloat16 *dq, *dk, *dv;
  __nv_bfloat16 *dq_in, *dk_in, *dv_in;
  long long dq_stride, dk_stride, dv_stride;
  float* part;                              // [blocks][2][d]
};

// What a block knows of each of its tokens.
struct Token {
  long long row;   // pack, backward: ragged row of KV head 0 (-1: none); append: pool row of it
  int step;        // rows from one KV head's to the next's
};

// Elements of thread c's four pairs: (first(e), second(e)), e = 0 .. 3; pair 4c + e.
template <int LAYOUT>
__device__ __forceinline__ int first_of(int c, int e, int r) {
  if constexpr (LAYOUT == kInterleaved) return 8 * c + 2 * e;
  if constexpr (LAYOUT == kHalf) return c < r / 8 ? 4 * c + e : 8 * c + e;
  const int i = 4 * c + e;
  return i < r / 2 ? i : 2 * i;   // past the rotated ones: elements (2i, 2i + 1), all at or above r
}
template <int LAYOUT>
__device__ __forceinline__ int second_of(int c, int e, int r) {
  if constexpr (LAYOUT == kInterleaved) return 8 * c + 2 * e + 1;
  if constexpr (LAYOUT == kHalf) return c < r / 8 ? r / 2 + 4 * c + e : 8 * c + 4 + e;
  const int i = 4 * c + e;
  return i < r / 2 ? i + r / 2 : 2 * i + 1;
}

// Thread c's eight elements of a row, as they lie: layout kInterleaved a0 b0 a1
// b1 .., the others a0 .. a3 b0 .. b3.
template <int LAYOUT>
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* row, int c, int r) {
  if constexpr (LAYOUT == kInterleaved) {
    return __ldcs(reinterpret_cast<const uint4*>(row + 8 * c));
  } else if constexpr (LAYOUT == kHalf) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + first_of<LAYOUT>(c, 0, r)));
    const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + second_of<LAYOUT>(c, 0, r)));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = s[first_of<LAYOUT>(c, e, r)];
      w[4 + e] = s[second_of<LAYOUT>(c, e, r)];
    }
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <int LAYOUT>
__device__ __forceinline__ void unpack(uint4 u, float (&a)[4], float (&b)[4]) {
  if constexpr (LAYOUT == kInterleaved) {
    a[0] = lo_f(u.x), b[0] = hi_f(u.x), a[1] = lo_f(u.y), b[1] = hi_f(u.y);
    a[2] = lo_f(u.z), b[2] = hi_f(u.z), a[3] = lo_f(u.w), b[3] = hi_f(u.w);
  } else {
    a[0] = lo_f(u.x), a[1] = hi_f(u.x), a[2] = lo_f(u.y), a[3] = hi_f(u.y);
    b[0] = lo_f(u.z), b[1] = hi_f(u.z), b[2] = lo_f(u.w), b[3] = hi_f(u.w);
  }
}

template <int LAYOUT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int c, int r, const float (&a)[4],
                                          const float (&b)[4]) {
  if constexpr (LAYOUT == kInterleaved) {
    *reinterpret_cast<uint4*>(row + 8 * c) =
        make_uint4(pack_bf16x2(a[0], b[0]), pack_bf16x2(a[1], b[1]), pack_bf16x2(a[2], b[2]),
                   pack_bf16x2(a[3], b[3]));
  } else if constexpr (LAYOUT == kHalf) {
    *reinterpret_cast<uint2*>(row + first_of<LAYOUT>(c, 0, r)) =
        make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    *reinterpret_cast<uint2*>(row + second_of<LAYOUT>(c, 0, r)) =
        make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      row[first_of<LAYOUT>(c, e, r)] = __float2bfloat16_rn(a[e]);
      row[second_of<LAYOUT>(c, e, r)] = __float2bfloat16_rn(b[e]);
    }
  }
}

// The e4m3 code nearest to the fp32 quotient x / s, two at a time.
__device__ __forceinline__ uint32_t codes2(float x0, float x1, float s) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(c)
      : "f"(__fdiv_rn(x1, s)), "f"(__fdiv_rn(x0, s)));
  return c;
}

template <int LAYOUT>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int r, const float (&a)[4],
                                            const float (&b)[4], float s) {
  if constexpr (LAYOUT == kInterleaved) {
    *reinterpret_cast<uint2*>(row + 8 * c) =
        make_uint2(codes2(a[0], b[0], s) | codes2(a[1], b[1], s) << 16,
                   codes2(a[2], b[2], s) | codes2(a[3], b[3], s) << 16);
  } else if constexpr (LAYOUT == kHalf) {
    *reinterpret_cast<uint32_t*>(row + first_of<LAYOUT>(c, 0, r)) =
        codes2(a[0], a[1], s) | codes2(a[2], a[3], s) << 16;
    *reinterpret_cast<uint32_t*>(row + second_of<LAYOUT>(c, 0, r)) =
        codes2(b[0], b[1], s) | codes2(b[2], b[3], s) << 16;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t two = codes2(a[e], b[e], s);
      row[first_of<LAYOUT>(c, e, r)] = static_cast<uint8_t>(two);
      row[second_of<LAYOUT>(c, e, r)] = static_cast<uint8_t>(two >> 8);
    }
  }
}

// Sum over the d / 8 threads of a head (warp-collective).
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int m = 1; m < D / 8; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ float sum_squares(const float (&a)[4], const float (&b)[4]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s = fmaf(a[e], a[e], fmaf(b[e], b[e], s));
  return s;
}

// The sequence of token t: the b with cu[b] <= t < cu[b + 1], or -1.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int batch, int t) {
  if (t < cu[0] || t >= cu[batch]) return -1;
  int lo = 0, hi = batch;   // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Cosine and sine of every pair of tokens tok0 .. tok0 + n - 1 into cs [n][d / 2]
// (1 and 0 past the rotated pairs), and where the tokens' rows lie.
template <int D, bool APPEND>
__device__ __forceinline__ void prepare_tokens(const RopeParams& p, int tok0, int n,
                                               float2 (*cs)[D / 2], Token* info, int* pos_s) {
  if (threadIdx.x < n) {
    const int t = tok0 + threadIdx.x;
    Token k{-1, 0};
    int pos = 0;
    if constexpr (APPEND) {
      pos = p.positions[t];
      const int slot = p.slots[t];
      if (slot >= 0 && slot < p.n_slots) {   // (a padding token writes no keys)
        k.row = ((static_cast<long long>(slot >> p.shift) * p.Hkv) << p.shift) +
                (slot & ((1 << p.shift) - 1));
        k.step = 1 << p.shift;
      }
    } else {
      const int b = sequence_of(p.cu, p.batch, t);
      if (b >= 0) {   // (rows behind the last sequence stay as they are)
        const int start = p.cu[b], end = p.cu[b + 1];
        if (start < 0 || end > p.tokens || t < start || t >= end) {
          atomicExch(&g_status_rope, SINKATTN_BAD_LENGTHS);
        } else {
          k.row = static_cast<long long>(p.Hkv) * start + (t - start);
          k.step = end - start;
          pos = p.positions ? p.positions[t] : t - start;
        }
      }
    }
    info[threadIdx.x] = k;
    pos_s[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < n * (D / 2); u += kThreads) {
    const int t = u / (D / 2), i = u % (D / 2);
    float2 v = make_float2(1.f, 0.f);
    if (i < p.r / 2) {
      const unsigned long long turn =
          p.turns[i] * static_cast<unsigned long long>(static_cast<long long>(pos_s[t]));
      // the upper 32 bits as a signed fraction: half turns in [-1, 1)
      const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      sincospif(x, &v.y, &v.x);
      v.x *= p.factor;
      v.y *= p.factor;
    }
    cs[t][i] = v;
  }
  __syncthreads();
}

// A block takes p.per_block tokens, or one of p.parts shares of their heads.
template <int D, int LAYOUT, int KIND>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int C = D / 8;                 // threads of a head
  constexpr int kIlp = 4;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ Token info[kMaxTokens];
  __shared__ int pos_s[kMaxTokens];
  const int tok0 = blockIdx.x / p.parts * p.per_block;
  const int n = min(p.per_block, p.tokens - tok0);
  prepare_tokens<D, KIND != kPack>(p, tok0, n, cs, info, pos_s);

  const int c = threadIdx.x % C;
  const int heads = p.Hq + 2 * p.Hkv;
  const int rows = n * heads;
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = first_of<LAYOUT>(c, e, p.r), j = second_of<LAYOUT>(c, e, p.r);
    wq[e] = p.q_weight ? p.q_weight[i] : 1.f;
    wq[4 + e] = p.q_weight ? p.q_weight[j] : 1.f;
    wk[e] = p.k_weight ? p.k_weight[i] : 1.f;
    wk[4 + e] = p.k_weight ? p.k_weight[j] : 1.f;
  }
  const bool any_norm = p.q_weight || p.k_weight;
  const int step = kThreads / C;
  const int part = blockIdx.x % p.parts;
  // (the trip count is the same for all threads: the head sums are warp-collective)
  for (int base = part * step * kIlp; base < rows; base += p.parts * step * kIlp) {
    uint4 raw[kIlp];
    int tok[kIlp], head[kIlp];
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      const int row = base + i * step + static_cast<int>(threadIdx.x) / C;
      tok[i] = -1;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (row >= rows) continue;
      const int t = static_cast<int>(__umulhi(row, p.inv_heads));
      const int h = row - t * heads;
      const long long g = tok0 + t;
      if (KIND == kPack && info[t].row < 0) continue;
      tok[i] = t;
      head[i] = h;
      if (h < p.Hq) raw[i] = load_row<LAYOUT>(p.q + g * p.q_stride + h * D, c, p.r);
      else if (info[t].row < 0) tok[i] = -1;
      else if (h < p.Hq + p.Hkv)
        raw[i] = load_row<LAYOUT>(p.k + g * p.k_stride + (h - p.Hq) * D, c, p.r);
      else
        raw[i] = load_row<kInterleaved>(p.v + g * p.v_stride + (h - p.Hq - p.Hkv) * D, c, p.r);
    }
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      float a[4], b[4];
      unpack<LAYOUT>(raw[i], a, b);
      float rs = 1.f;
      if (any_norm) rs = rsqrtf(head_sum<D>(sum_squares(a, b)) * (1.f / D) + p.eps);
      if (tok[i] < 0) continue;
      const int t = tok[i], h = head[i];
      const Token at = info[t];
      if (h >= p.Hq + p.Hkv) {
        const long long row = at.row + static_cast<long long>(h - p.Hq - p.Hkv) * at.step;
        if constexpr (KIND == kAppendFp8) {
          float x[4], y[4];
          unpack<kInterleaved>(raw[i], x, y);
          store_codes<kInterleaved>(p.v_pages + row * D, c, p.r, x, y,
                                    p.v_scale[h - p.Hq - p.Hkv]);
        } else {
          __nv_bfloat16* out = KIND == kPack ? p.v_out : reinterpret_cast<__nv_bfloat16*>(p.v_pages);
          *reinterpret_cast<uint4*>(out + row * D + 8 * c) = raw[i];
        }
        continue;
      }
      const bool is_q = h < p.Hq;
      if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] *= rs * (is_q ? wq[e] : wk[e]);
          b[e] *= rs * (is_q ? wq[4 + e] : wk[4 + e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // kHalf past the rotated pairs: cs holds 1 and 0
        const float2 w = cs[t][4 * c + e];
        const float x = a[e], y = b[e];
        a[e] = x * w.x - y * w.y;
        b[e] = y * w.x + x * w.y;
      }
      if (is_q) {
        store_row<LAYOUT>(p.q_out + (static_cast<long long>(tok0 + t) * p.Hq + h) * D, c, p.r, a, b);
      } else {
        const long long row = at.row + static_cast<long long>(h - p.Hq) * at.step;
        if constexpr (KIND == kAppendFp8)
          store_codes<LAYOUT>(p.k_pages + row * D, c, p.r, a, b, p.k_scale[h - p.Hq]);
        else
          store_row<LAYOUT>((KIND == kPack ? p.k_out : reinterpret_cast<__nv_bfloat16*>(p.k_pages)) +
                                row * D, c, p.r, a, b);
      }
    }
  }
}

// Gradients of the projection's rows; blocks walk over the groups of
// p.per_block tokens with the grid's stride and leave their sums of the
// weights' gradients in p.part.
template <int D, int LAYOUT, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_backward_kernel(const RopeParams p) {
  constexpr int C = D / 8;
  constexpr int kIlp = 2;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ Token info[kMaxTokens];
  __shared__ int pos_s[kMaxTokens];
  __shared__ float sums[kThreads][9];
  const int c = threadIdx.x % C;
  const int heads = p.Hq + 2 * p.Hkv;
  float wq[8], wk[8], sq[8], sk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = e < 4 ? first_of<LAYOUT>(c, e, p.r) : second_of<LAYOUT>(c, e - 4, p.r);
    wq[e] = NORM && p.q_weight ? p.q_weight[i] : 1.f;
    wk[e] = NORM && p.k_weight ? p.k_weight[i] : 1.f;
    sq[e] = sk[e] = 0.f;
  }
  const int step = kThreads / C;
  const int groups = (p.tokens + p.per_block - 1) / p.per_block;
  for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int tok0 = grp * p.per_block;
    const int n = min(p.per_block, p.tokens - tok0);
    __syncthreads();   // the group before has read cs and info
    prepare_tokens<D, false>(p, tok0, n, cs, info, pos_s);
    const int rows = n * heads;
    for (int base = 0; base < rows; base += step * kIlp) {
      uint4 raw[kIlp], xr[kIlp];
      int tok[kIlp], head[kIlp];
#pragma unroll
      for (int i = 0; i < kIlp; ++i) {
        const int row = base + i * step + static_cast<int>(threadIdx.x) / C;
        tok[i] = -1;
        head[i] = 0;
        raw[i] = xr[i] = make_uint4(0, 0, 0, 0);
        if (row >= rows) continue;
        const int t = static_cast<int>(__umulhi(row, p.inv_heads));
        const int h = row - t * heads;
        const long long g = tok0 + t;
        const Token at = info[t];
        if (at.row < 0) continue;
        tok[i] = t;
        head[i] = h;
        if (h < p.Hq) {
          raw[i] = load_row<LAYOUT>(p.dq + (g * p.Hq + h) * D, c, p.r);
          if (NORM && p.q_weight) xr[i] = load_row<LAYOUT>(p.q + g * p.q_stride + h * D, c, p.r);
        } else if (h < p.Hq + p.Hkv) {
          const int kh = h - p.Hq;
          raw[i] = load_row<LAYOUT>(p.dk + (at.row + static_cast<long long>(kh) * at.step) * D, c, p.r);
          if (NORM && p.k_weight) xr[i] = load_row<LAYOUT>(p.k + g * p.k_stride + kh * D, c, p.r);
        } else {
          const int kh = h - p.Hq - p.Hkv;
          raw[i] = load_row<kInterleaved>(
              p.dv + (at.row + static_cast<long long>(kh) * at.step) * D, c, p.r);
        }
      }
#pragma unroll
      for (int i = 0; i < kIlp; ++i) {
        const int t = max(tok[i], 0), h = head[i];
        const long long g = tok0 + t;
        const bool is_q = h < p.Hq;
        float a[4], b[4];
        unpack<LAYOUT>(raw[i], a, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 w = cs[t][4 * c + e];
          const float x = a[e], y = b[e];
          a[e] = x * w.x + y * w.y;
          b[e] = y * w.x - x * w.y;
        }
        if constexpr (NORM) {
          float x[4], y[4];
          unpack<LAYOUT>(xr[i], x, y);
          const float rs = rsqrtf(head_sum<D>(sum_squares(x, y)) * (1.f / D) + p.eps);
          float u[4], v[4], dot = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] *= rs;
            y[e] *= rs;
            u[e] = a[e] * (is_q ? wq[e] : wk[e]);
            v[e] = b[e] * (is_q ? wq[4 + e] : wk[4 + e]);
            dot = fmaf(u[e], x[e], fmaf(v[e], y[e], dot));
          }
          dot = head_sum<D>(dot) * (1.f / D);
          const bool normed = tok[i] >= 0 && h < p.Hq + p.Hkv &&
                              (is_q ? p.q_weight != nullptr : p.k_weight != nullptr);
          if (normed) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (is_q) {
                sq[e] = fmaf(a[e], x[e], sq[e]);
                sq[4 + e] = fmaf(b[e], y[e], sq[4 + e]);
              } else {
                sk[e] = fmaf(a[e], x[e], sk[e]);
                sk[4 + e] = fmaf(b[e], y[e], sk[4 + e]);
              }
              a[e] = rs * (u[e] - x[e] * dot);
              b[e] = rs * (v[e] - y[e] * dot);
            }
          }
        }
        if (tok[i] < 0) continue;
        if (is_q)
          store_row<LAYOUT>(p.dq_in + g * p.dq_stride + h * D, c, p.r, a, b);
        else if (h < p.Hq + p.Hkv)
          store_row<LAYOUT>(p.dk_in + g * p.dk_stride + (h - p.Hq) * D, c, p.r, a, b);
        else
          *reinterpret_cast<uint4*>(p.dv_in + g * p.dv_stride + (h - p.Hq - p.Hkv) * D + 8 * c) = raw[i];
      }
    }
  }
  if constexpr (NORM) {
    // the block's sums, over the threads that hold the same elements, in a fixed order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = which ? sk[e] : sq[e];
      __syncthreads();
      if (threadIdx.x < D) {
        const int cc = threadIdx.x / 8, e = threadIdx.x % 8;
        float s = 0.f;
        for (int j = 0; j < kThreads / C; ++j) s += sums[j * C + cc][e];
        const int el = e < 4 ? first_of<LAYOUT>(cc, e, p.r) : second_of<LAYOUT>(cc, e - 4, p.r);
        p.part[(static_cast<long long>(blockIdx.x) * 2 + which) * D + el] = s;
      }
    }
  }
}

// The weights' gradients: the blocks' sums added in a fixed order, 32 columns
// of the 2 d a block, eight threads a column.
__global__ void __launch_bounds__(256) rope_weights_kernel(const float* part, int blocks, int d,
                                                           float* dq_weight, float* dk_weight) {
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  float x = 0.f;
  for (int b = slice; b < blocks; b += 8) x += part[static_cast<long long>(b) * 2 * d + col];
  s[slice][threadIdx.x % 32] = x;
  __syncthreads();
  if (slice != 0) return;
  for (int j = 1; j < 8; ++j) x += s[j][threadIdx.x];
  float* out = col < d ? dq_weight : dk_weight;
  if (out) out[col % d] = x;
}

int refuse(int status, const char* text) {
  set_error("%s", text);
  return status;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks that all calls share, and the shared part of the parameters.
int rope_args(int32_t tokens, int32_t Hq, int32_t Hkv, int32_t d, const uint64_t* turns,
              int32_t rotary_dim, int32_t interleaved, float factor, const float* q_weight,
              const float* k_weight, float eps, RopeParams* p) {
  set_error("%s", "");
  if (tokens < 0) return refuse(SINKATTN_INVALID_ARG, "tokens must be non-negative");
  if (Hq < 1 || Hkv < 1) return refuse(SINKATTN_INVALID_ARG, "head counts must be positive");
  if (Hq > 4096 || Hkv > 4096) return refuse(SINKATTN_UNSUPPORTED, "more than 4096 heads");
  if (d != 64 && d != 128) return refuse(SINKATTN_UNSUPPORTED, "head_dim is not 64 or 128");
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 2)
    return refuse(SINKATTN_INVALID_ARG, "rotary_dim must be even and at most head_dim");
  if (interleaved != 0 && interleaved != 1)
    return refuse(SINKATTN_INVALID_ARG, "interleaved must be 0 or 1");
  if (!std::isfinite(factor)) return refuse(SINKATTN_INVALID_ARG, "attention_factor must be finite");
  if (rotary_dim > 0 && (!turns || !aligned(turns, 8)))
    return refuse(SINKATTN_INVALID_ARG, "turns must be non-null and 8-byte aligned");
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4))
    return refuse(SINKATTN_INVALID_ARG, "q_weight and k_weight must be 4-byte aligned");
  if ((q_weight || k_weight) && (!(eps >= 0.f) || !std::isfinite(eps)))
    return refuse(SINKATTN_INVALID_ARG, "eps must be non-negative and finite");
  *p = RopeParams{};
  p->tokens = tokens;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->r = rotary_dim;
  // row / heads is the upper half of row * inv_heads for the rows of a block: below 2^32 / heads
  const uint32_t heads = static_cast<uint32_t>(Hq) + 2 * Hkv;
  p->inv_heads = static_cast<uint32_t>(((uint64_t{1} << 32) + heads - 1) / heads);
  p->turns = reinterpret_cast<const unsigned long long*>(turns);
  p->factor = factor;
  p->q_weight = q_weight;
  p->k_weight = k_weight;
  p->eps = eps;
  return SINKATTN_OK;
}

// Rows of the projection, or of its gradient: `heads` rows of d elements per token.
int check_rows(const void* x, int64_t stride, int32_t heads, int32_t d) {
  if (!x || !aligned(x, 16))
    return refuse(SINKATTN_INVALID_ARG, "rows must be non-null and 16-byte aligned");
  if (stride < static_cast<int64_t>(heads) * d || stride % 8)
    return refuse(SINKATTN_INVALID_ARG,
                  "token strides must be multiples of 8 and at least heads * head_dim");
  return SINKATTN_OK;
}

int check_out(const void* x, const char* text) {
  return x && aligned(x, 16) ? SINKATTN_OK : refuse(SINKATTN_INVALID_ARG, text);
}

// Pairs of kHalf threads lie in whole groups of four; other sizes take kHalfOdd.
int layout_of(int32_t rotary_dim, int32_t interleaved) {
  return interleaved ? kInterleaved : rotary_dim % 8 == 0 ? kHalf : kHalfOdd;
}

template <int D, int KIND>
void (*pick_layout(int layout))(const RopeParams) {
  return layout == kHalf          ? rope_kernel<D, kHalf, KIND>
         : layout == kInterleaved ? rope_kernel<D, kInterleaved, KIND>
                                  : rope_kernel<D, kHalfOdd, KIND>;
}

template <int D, bool NORM>
void (*pick_backward(int layout))(const RopeParams) {
  return layout == kHalf          ? rope_backward_kernel<D, kHalf, NORM>
         : layout == kInterleaved ? rope_backward_kernel<D, kInterleaved, NORM>
                                  : rope_backward_kernel<D, kHalfOdd, NORM>;
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

int launch_forward(RopeParams& p, int d, int kind, int interleaved, cudaStream_t stream) {
  const int layout = layout_of(p.r, interleaved);
  const int64_t units = (static_cast<int64_t>(p.Hq) + 2 * p.Hkv) * (d / 8);   // threads of a token
  // tokens of a block: four, while that leaves every SM eight blocks
  p.per_block = 1;
  while (p.per_block < 4 && p.tokens / (2 * p.per_block) >= 8LL * sm_count()) p.per_block *= 2;
  // few tokens: their heads go to several blocks
  p.parts = 1;
  while (p.tokens * int64_t{p.parts} < sm_count() && units > int64_t{p.parts} * kThreads) p.parts *= 2;
  const int64_t blocks = (int64_t{p.tokens} + p.per_block - 1) / p.per_block * p.parts;
  if (blocks >= (int64_t{1} << 31)) return refuse(SINKATTN_UNSUPPORTED, "too many work items");
  void (*kern)(const RopeParams) =
      d == 64 ? (kind == kPack     ? pick_layout<64, kPack>(layout)
                 : kind == kAppend ? pick_layout<64, kAppend>(layout)
                                   : pick_layout<64, kAppendFp8>(layout))
              : (kind == kPack     ? pick_layout<128, kPack>(layout)
                 : kind == kAppend ? pick_layout<128, kAppend>(layout)
                                   : pick_layout<128, kAppendFp8>(layout));
  kern<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return launched("rope");
}

// (a fixed bound, so that neither the workspace nor the order of the sums goes by the device)
int backward_blocks(int32_t tokens) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((int64_t{tokens} + 1) / 2, 6 * 152)));
}

int append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
           int64_t v_stride, const int32_t* positions, const int32_t* slots, int32_t tokens,
           int32_t Hq, int32_t Hkv, int32_t d, const uint64_t* turns, int32_t rotary_dim,
           int32_t interleaved, float factor, const float* q_weight, const float* k_weight,
           float eps, const float* k_scale, const float* v_scale, bool fp8, void* q_out,
           void* k_pages, void* v_pages, int32_t num_pages, int32_t page_size, void* stream) {
  RopeParams p;
  int rc = rope_args(tokens, Hq, Hkv, d, turns, rotary_dim, interleaved, factor, q_weight,
                     k_weight, eps, &p);
  if (rc) return rc;
  if (!k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return refuse(SINKATTN_INVALID_ARG, "k_pages and v_pages must be non-null and 16-byte aligned");
  if (num_pages < 1) return refuse(SINKATTN_INVALID_ARG, "num_pages must be positive");
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return refuse(SINKATTN_UNSUPPORTED, "page_size is not a power of two in [16, 256]");
  if (static_cast<int64_t>(num_pages) * Hkv * page_size >= (int64_t{1} << 31))
    return refuse(SINKATTN_UNSUPPORTED, "page pools exceed 2^31 rows");
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return refuse(SINKATTN_INVALID_ARG, "k_scale and v_scale must be non-null and 4-byte aligned");
  if (tokens == 0) return SINKATTN_OK;
  if ((rc = check_rows(q, q_stride, Hq, d)) || (rc = check_rows(k, k_stride, Hkv, d)) ||
      (rc = check_rows(v, v_stride, Hkv, d)))
    return rc;
  if (!positions || !slots || !aligned(positions, 4) || !aligned(slots, 4))
    return refuse(SINKATTN_INVALID_ARG, "positions and slots must be non-null and 4-byte aligned");
  if ((rc = check_out(q_out, "q_out must be non-null and 16-byte aligned"))) return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slots;
  p.k_scale = k_scale, p.v_scale = v_scale;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  while ((1 << p.shift) < page_size) ++p.shift;
  p.n_slots = static_cast<long long>(num_pages) * page_size;
  return launch_forward(p, d, fp8 ? kAppendFp8 : kAppend, interleaved,
                        static_cast<cudaStream_t>(stream));
}

}  // namespace

int read_status_rope(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_rope, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_status_rope, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn

extern "C" {

using namespace sinkattn;

int sinkattn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                              int32_t original_len, double beta_fast, double beta_slow,
                              double* inv_freq, float* attention_factor) {
  set_error("%s", "");
  if (rotary_dim < 0 || rotary_dim % 2)
    return refuse(SINKATTN_INVALID_ARG, "rotary_dim must be even and non-negative");
  if (!inv_freq || !attention_factor)
    return refuse(SINKATTN_INVALID_ARG, "inv_freq and attention_factor must be non-null");
  if (scaling < SINKATTN_ROPE_PLAIN || scaling > SINKATTN_ROPE_YARN)
    return refuse(SINKATTN_INVALID_ARG, "no such scaling");
  if (!(base > 1.0) || !std::isfinite(base))
    return refuse(SINKATTN_INVALID_ARG, "base must be above 1 and finite");
  if (scaling != SINKATTN_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return refuse(SINKATTN_INVALID_ARG, "factor must be at least 1 and finite");
  if (scaling == SINKATTN_ROPE_YARN &&
      (original_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return refuse(SINKATTN_INVALID_ARG,
                  "YaRN needs original_len of at least 1 and 0 < beta_slow < beta_fast");
  const double r = rotary_dim;
  if (scaling == SINKATTN_ROPE_NTK && rotary_dim > 2) base *= std::pow(factor, r / (r - 2.0));
  // YaRN: pairs below `low` keep their frequency, pairs above `high` have it
  // divided by the factor, those between are blended
  double low = 0.0, high = 0.0;
  if (scaling == SINKATTN_ROPE_YARN) {
    const double pi2 = 6.283185307179586476925;
    low = std::max(0.0, r * std::log(original_len / (beta_fast * pi2)) / (2.0 * std::log(base)));
    high = std::min(r - 1.0, r * std::log(original_len / (beta_slow * pi2)) / (2.0 * std::log(base)));
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    inv_freq[i] = f;
    if (scaling == SINKATTN_ROPE_LINEAR) inv_freq[i] = f / factor;
    if (scaling == SINKATTN_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      inv_freq[i] = f / factor * ramp + f * (1.0 - ramp);
    }
  }
  *attention_factor =
      scaling == SINKATTN_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return SINKATTN_OK;
}

int sinkattn_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  set_error("%s", "");
  if (n < 0 || (n > 0 && (!inv_freq || !turns)))
    return refuse(SINKATTN_INVALID_ARG, "inv_freq and turns must be non-null, n non-negative");
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i]))
      return refuse(SINKATTN_INVALID_ARG, "inv_freq must be finite");
  for (int i = 0; i < n; ++i) {
    const double t = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    const double part = t - std::floor(t);
    turns[i] = part < 1.0 ? static_cast<uint64_t>(std::ldexp(part, 64)) : 0;
  }
  return SINKATTN_OK;
}

int sinkattn_rope_qkv(const void* q, const void* k, const void* v, int64_t q_stride,
                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                      const int32_t* positions, int32_t batch, int32_t tokens,
                      int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                      const uint64_t* turns, int32_t rotary_dim, int32_t interleaved,
                      float attention_factor, const float* q_weight, const float* k_weight,
                      float eps, void* q_out, void* k_out, void* v_out, void* stream) {
  RopeParams p;
  int rc = rope_args(tokens, num_qo_heads, num_kv_heads, head_dim, turns, rotary_dim, interleaved,
                     attention_factor, q_weight, k_weight, eps, &p);
  if (rc) return rc;
  if (batch < 0) return refuse(SINKATTN_INVALID_ARG, "batch must be non-negative");
  if (tokens == 0 || batch == 0) return SINKATTN_OK;
  if ((rc = check_rows(q, q_stride, num_qo_heads, head_dim)) ||
      (rc = check_rows(k, k_stride, num_kv_heads, head_dim)) ||
      (rc = check_rows(v, v_stride, num_kv_heads, head_dim)))
    return rc;
  if (!cu_seqlens || !aligned(cu_seqlens, 4) || !aligned(positions, 4))
    return refuse(SINKATTN_INVALID_ARG,
                  "cu_seqlens must be non-null, cu_seqlens and positions 4-byte aligned");
  if ((rc = check_out(q_out, "q_out must be non-null and 16-byte aligned")) ||
      (rc = check_out(k_out, "k_out must be non-null and 16-byte aligned")) ||
      (rc = check_out(v_out, "v_out must be non-null and 16-byte aligned")))
    return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.cu = cu_seqlens;
  p.batch = batch;
  p.positions = positions;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  return launch_forward(p, head_dim, kPack, interleaved, static_cast<cudaStream_t>(stream));
}

int sinkattn_rope_qkv_backward_workspace_bytes(int32_t tokens, int32_t head_dim, size_t* bytes) {
  set_error("%s", "");
  if (!bytes) return refuse(SINKATTN_INVALID_ARG, "bytes must be non-null");
  if (tokens < 0) return refuse(SINKATTN_INVALID_ARG, "tokens must be non-negative");
  if (head_dim != 64 && head_dim != 128)
    return refuse(SINKATTN_UNSUPPORTED, "head_dim is not 64 or 128");
  *bytes = static_cast<size_t>(backward_blocks(tokens)) * 2 * head_dim * sizeof(float);
  return SINKATTN_OK;
}

int sinkattn_rope_qkv_backward(const void* dq, const void* dk, const void* dv, const void* q,
                               const void* k, int64_t q_stride, int64_t k_stride,
                               const int32_t* cu_seqlens, const int32_t* positions, int32_t batch,
                               int32_t tokens, int32_t num_qo_heads, int32_t num_kv_heads,
                               int32_t head_dim, const uint64_t* turns, int32_t rotary_dim,
                               int32_t interleaved, float attention_factor, const float* q_weight,
                               const float* k_weight, float eps, void* dq_in, void* dk_in,
                               void* dv_in, int64_t dq_stride, int64_t dk_stride,
                               int64_t dv_stride, float* dq_weight, float* dk_weight,
                               void* workspace, size_t workspace_bytes, void* stream) {
  RopeParams p;
  int rc = rope_args(tokens, num_qo_heads, num_kv_heads, head_dim, turns, rotary_dim, interleaved,
                     attention_factor, q_weight, k_weight, eps, &p);
  if (rc) return rc;
  if (batch < 0) return refuse(SINKATTN_INVALID_ARG, "batch must be non-negative");
  if ((q_weight && (!dq_weight || !aligned(dq_weight, 4))) ||
      (k_weight && (!dk_weight || !aligned(dk_weight, 4))))
    return refuse(SINKATTN_INVALID_ARG,
                  "dq_weight and dk_weight must be non-null and 4-byte aligned where there is a norm");
  const bool norm = q_weight || k_weight;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0 || batch == 0) {
    // no token has a gradient: the weights' are zero
    for (float* w : {q_weight ? dq_weight : nullptr, k_weight ? dk_weight : nullptr})
      if (w && cudaMemsetAsync(w, 0, sizeof(float) * head_dim, s) != cudaSuccess)
        return refuse(SINKATTN_CUDA_ERROR, "cudaMemsetAsync failed");
    return SINKATTN_OK;
  }
  if ((rc = check_out(dq, "dq must be non-null and 16-byte aligned")) ||
      (rc = check_out(dk, "dk must be non-null and 16-byte aligned")) ||
      (rc = check_out(dv, "dv must be non-null and 16-byte aligned")) ||
      (q_weight && (rc = check_rows(q, q_stride, num_qo_heads, head_dim))) ||
      (k_weight && (rc = check_rows(k, k_stride, num_kv_heads, head_dim))) ||
      (rc = check_rows(dq_in, dq_stride, num_qo_heads, head_dim)) ||
      (rc = check_rows(dk_in, dk_stride, num_kv_heads, head_dim)) ||
      (rc = check_rows(dv_in, dv_stride, num_kv_heads, head_dim)))
    return rc;
  if (!cu_seqlens || !aligned(cu_seqlens, 4) || !aligned(positions, 4))
    return refuse(SINKATTN_INVALID_ARG,
                  "cu_seqlens must be non-null, cu_seqlens and positions 4-byte aligned");
  const int blocks = backward_blocks(tokens);
  if (norm) {
    if (!workspace || !aligned(workspace, 256))
      return refuse(SINKATTN_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
    if (workspace_bytes < static_cast<size_t>(blocks) * 2 * head_dim * sizeof(float))
      return refuse(SINKATTN_INVALID_ARG, "workspace is too small");
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_stride = q_stride, p.k_stride = k_stride;
  p.cu = cu_seqlens;
  p.batch = batch;
  p.positions = positions;
  p.dq = static_cast<const __nv_bfloat16*>(dq);
  p.dk = static_cast<const __nv_bfloat16*>(dk);
  p.dv = static_cast<const __nv_bfloat16*>(dv);
  p.dq_in = static_cast<__nv_bfloat16*>(dq_in);
  p.dk_in = static_cast<__nv_bfloat16*>(dk_in);
  p.dv_in = static_cast<__nv_bfloat16*>(dv_in);
  p.dq_stride = dq_stride, p.dk_stride = dk_stride, p.dv_stride = dv_stride;
  p.part = static_cast<float*>(workspace);
  p.per_block = tokens >= 8 * blocks ? 4 : 2;
  const int layout = layout_of(p.r, interleaved);
  void (*kern)(const RopeParams) =
      head_dim == 64 ? (norm ? pick_backward<64, true>(layout) : pick_backward<64, false>(layout))
                     : (norm ? pick_backward<128, true>(layout) : pick_backward<128, false>(layout));
  kern<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  if ((rc = launched("rope backward")) || !norm) return rc;
  rope_weights_kernel<<<static_cast<unsigned>(2 * head_dim / 32), 256, 0, s>>>(
      p.part, blocks, head_dim, q_weight ? dq_weight : nullptr, k_weight ? dk_weight : nullptr);
  return launched("rope weights");
}

int sinkattn_rope_append_paged(const void* q, const void* k, const void* v, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, const int32_t* positions,
                               const int32_t* slots, int32_t tokens, int32_t num_qo_heads,
                               int32_t num_kv_heads, int32_t head_dim, const uint64_t* turns,
                               int32_t rotary_dim, int32_t interleaved, float attention_factor,
                               const float* q_weight, const float* k_weight, float eps,
                               void* q_out, void* k_pages, void* v_pages, int32_t num_pages,
                               int32_t page_size, void* stream) {
  return append(q, k, v, q_stride, k_stride, v_stride, positions, slots, tokens, num_qo_heads,
                num_kv_heads, head_dim, turns, rotary_dim, interleaved, attention_factor, q_weight,
                k_weight, eps, nullptr, nullptr, false, q_out, k_pages, v_pages, num_pages,
                page_size, stream);
}

int sinkattn_rope_append_paged_fp8(const void* q, const void* k, const void* v, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, const int32_t* positions,
                                   const int32_t* slots, int32_t tokens, int32_t num_qo_heads,
                                   int32_t num_kv_heads, int32_t head_dim, const uint64_t* turns,
                                   int32_t rotary_dim, int32_t interleaved, float attention_factor,
                                   const float* q_weight, const float* k_weight, float eps,
                                   const float* k_scale, const float* v_scale, void* q_out,
                                   void* k_pages, void* v_pages, int32_t num_pages,
                                   int32_t page_size, void* stream) {
  return append(q, k, v, q_stride, k_stride, v_stride, positions, slots, tokens, num_qo_heads,
                num_kv_heads, head_dim, turns, rotary_dim, interleaved, attention_factor, q_weight,
                k_weight, eps, k_scale, v_scale, true, q_out, k_pages, v_pages, num_pages,
                page_size, stream);
}

}  // extern "C"
