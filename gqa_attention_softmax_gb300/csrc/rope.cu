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
// Angles. The frequencies come as turns per position in units of 2^-64, rounded
// to the nearest, so position * turns modulo 2^64 is the angle's fraction of a
// turn with an error of at most |position| 2^-65 turns, 2^-34 at the farthest; its upper
// 32 bits go to sincospif, which takes 24 of them (2^-26 turns). A 32-bit product
// of position and frequency would be off by up to 2^-24 |position| radians instead.
//
// A thread holds eight elements of one head, four whole pairs, so that the
// rotation needs no exchange; d / 8 threads hold a head, a warp takes two or
// four heads at a time and, where there are tokens enough, all heads of its
// token: cosines and weights stay in registers. Rows come through a ring in
// shared memory, three steps ahead of the arithmetic and the first ones before the
// token's sequence is known: in registers, four rows a thread, too little was on
// its way (82 us where the ring takes 71). The mean squares and all arithmetic between the
// loads and the stores are 32-bit; each output is rounded once. The weight is multiplied into
// cosine and sine once for all heads, and the inverse root comes last: a multiplication
// an element fewer, in another order than the formula's, which bf16 outputs do not show and which
// moves an e4m3 code now and then where the quotient lies next to the middle of two.
//
// All passes are bound by HBM. Measured, several calls in a graph, reads and writes together
// (copy: 6.78 TB/s): 12,000 tokens of 64 + 2 x 4 heads of 128 with norms, forward 71 to 77 us
// (by where the buffers lie; 6.2 to 5.8 TB/s), backward 120.6 us (5.4 TB/s, with the weights' sums),
// 21,800 of them into e4m3 pages 121 us (6.4 TB/s); 10,168 tokens of 64 + 2 x 8 heads of 64,
// backward without norms, 33.7 us (6.2 TB/s). Interleaved pairs and a rotation of half a head take
// the same. The half layout with a rotary_dim that is no multiple of 8 does not: a thread's four
// pairs then straddle words, so elements come from the ring and go to memory one by one. With 100
// of the 128 rotated: forward 138 us, backward 171, e4m3 pages 264; with 38 of 64, backward 71.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chain.cuh"
#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_rope;

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 4;  // of a warp's ring in shared memory: one step's rows each

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
  int parts;                                // warps that share the heads of a token
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

// Where a token's keys and values lie.
struct Token {
  long long row;   // pack, backward: ragged row of KV head 0 (-1: none); append: pool row of it
  int step;        // rows from one KV head's to the next's
  int pos;
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
    return *reinterpret_cast<const uint4*>(row + 8 * c);
  } else if constexpr (LAYOUT == kHalf) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + first_of<LAYOUT>(c, 0, r));
    const uint2 b = *reinterpret_cast<const uint2*>(row + second_of<LAYOUT>(c, 0, r));
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

// The four pairs' members, two pairs in one register pair.
template <int LAYOUT>
__device__ __forceinline__ void unpack(uint4 u, float2 (&a)[2], float2 (&b)[2]) {
  if constexpr (LAYOUT == kInterleaved) {
    a[0] = make_float2(lo_f(u.x), lo_f(u.y)), b[0] = make_float2(hi_f(u.x), hi_f(u.y));
    a[1] = make_float2(lo_f(u.z), lo_f(u.w)), b[1] = make_float2(hi_f(u.z), hi_f(u.w));
  } else {
    a[0] = make_float2(lo_f(u.x), hi_f(u.x)), a[1] = make_float2(lo_f(u.y), hi_f(u.y));
    b[0] = make_float2(lo_f(u.z), hi_f(u.z)), b[1] = make_float2(lo_f(u.w), hi_f(u.w));
  }
}

template <int LAYOUT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int c, int r, const float2 (&a)[2],
                                          const float2 (&b)[2]) {
  if constexpr (LAYOUT == kInterleaved) {
    *reinterpret_cast<uint4*>(row + 8 * c) =
        make_uint4(pack_bf16x2(a[0].x, b[0].x), pack_bf16x2(a[0].y, b[0].y),
                   pack_bf16x2(a[1].x, b[1].x), pack_bf16x2(a[1].y, b[1].y));
  } else if constexpr (LAYOUT == kHalf) {
    *reinterpret_cast<uint2*>(row + first_of<LAYOUT>(c, 0, r)) =
        make_uint2(pack_bf16x2(a[0].x, a[0].y), pack_bf16x2(a[1].x, a[1].y));
    *reinterpret_cast<uint2*>(row + second_of<LAYOUT>(c, 0, r)) =
        make_uint2(pack_bf16x2(b[0].x, b[0].y), pack_bf16x2(b[1].x, b[1].y));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      row[first_of<LAYOUT>(c, e, r)] = __float2bfloat16_rn(e & 1 ? a[e >> 1].y : a[e >> 1].x);
      row[second_of<LAYOUT>(c, e, r)] = __float2bfloat16_rn(e & 1 ? b[e >> 1].y : b[e >> 1].x);
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
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int r, const float2 (&a)[2],
                                            const float2 (&b)[2], float s) {
  if constexpr (LAYOUT == kInterleaved) {
    *reinterpret_cast<uint2*>(row + 8 * c) =
        make_uint2(codes2(a[0].x, b[0].x, s) | codes2(a[0].y, b[0].y, s) << 16,
                   codes2(a[1].x, b[1].x, s) | codes2(a[1].y, b[1].y, s) << 16);
  } else if constexpr (LAYOUT == kHalf) {
    *reinterpret_cast<uint32_t*>(row + first_of<LAYOUT>(c, 0, r)) =
        codes2(a[0].x, a[0].y, s) | codes2(a[1].x, a[1].y, s) << 16;
    *reinterpret_cast<uint32_t*>(row + second_of<LAYOUT>(c, 0, r)) =
        codes2(b[0].x, b[0].y, s) | codes2(b[1].x, b[1].y, s) << 16;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t two = codes2(e & 1 ? a[e >> 1].y : a[e >> 1].x, e & 1 ? b[e >> 1].y : b[e >> 1].x, s);
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

__device__ __forceinline__ float dot_pairs(const float2 (&a)[2], const float2 (&b)[2], const float2 (&x)[2],
                                           const float2 (&y)[2]) {
  const float2 s = __ffma2_rn(a[1], x[1], __ffma2_rn(b[0], y[0], __fmul2_rn(a[0], x[0])));
  const float2 t = __ffma2_rn(b[1], y[1], s);
  return t.x + t.y;
}

__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

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

// Records cu_seqlens that leave [0, tokens] or decrease, entry by entry (a bad one need
// not be where any token looks): thread `i` of `n`.
__device__ __forceinline__ void check_sequences(const RopeParams& p, long long i, long long n) {
  for (; i <= p.batch; i += n) {
    const int at = p.cu[i];
    if (at < 0 || at > p.tokens || (i > 0 && p.cu[i - 1] > at)) atomicExch(&g_status_rope, SINKATTN_BAD_LENGTHS);
  }
}

template <bool APPEND>
__device__ __forceinline__ Token token_of(const RopeParams& p, int t) {
  Token k{-1, 0, 0};
  if constexpr (APPEND) {
    k.pos = p.positions[t];
    const int slot = p.slots[t];
    if (slot >= 0 && slot < p.n_slots) {   // (a padding token writes no keys)
      k.row = ((static_cast<long long>(slot >> p.shift) * p.Hkv) << p.shift) + (slot & ((1 << p.shift) - 1));
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
        k.pos = p.positions ? p.positions[t] : t - start;
      }
    }
  }
  return k;
}

// Cosine and sine of thread c's four pairs at a position (1 and 0 past the rotated ones).
__device__ __forceinline__ void angles(const RopeParams& p, int pos, int c, float2 (&co)[2], float2 (&si)[2]) {
  float x[4], y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = 4 * c + e;
    x[e] = 1.f;
    y[e] = 0.f;
    if (i < p.r / 2) {
      const unsigned long long turn = p.turns[i] * static_cast<unsigned long long>(static_cast<long long>(pos));
      // the upper 32 bits as a signed fraction: half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &y[e], &x[e]);
      x[e] *= p.factor;
      y[e] *= p.factor;
    }
  }
  co[0] = make_float2(x[0], x[1]), co[1] = make_float2(x[2], x[3]);
  si[0] = make_float2(y[0], y[1]), si[1] = make_float2(y[2], y[3]);
}

// Thread c's pairs past the rotated ones as they were: by 1 and 0 an infinity would make its
// partner NaN. (Not under a norm, which lets no element stay as it is.)
__device__ __forceinline__ void keep_rest(int c, int r, const float2 (&a)[2], const float2 (&b)[2],
                                          float2 (&y)[2], float2 (&z)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (4 * c + 2 * e >= r / 2) y[e].x = a[e].x, z[e].x = b[e].x;
    if (4 * c + 2 * e + 1 >= r / 2) y[e].y = a[e].y, z[e].y = b[e].y;
  }
}

// Thread c's eight weights (1 without a norm).
template <int LAYOUT>
__device__ __forceinline__ void load_weights(const float* w, int c, int r, float2 (&a)[2], float2 (&b)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    a[e] = b[e] = make_float2(1.f, 1.f);
    if (w == nullptr) continue;
    a[e] = make_float2(w[first_of<LAYOUT>(c, 2 * e, r)], w[first_of<LAYOUT>(c, 2 * e + 1, r)]);
    b[e] = make_float2(w[second_of<LAYOUT>(c, 2 * e, r)], w[second_of<LAYOUT>(c, 2 * e + 1, r)]);
  }
}

// Share `part` of a token's work: passes of 32 / C heads, PER of them a step,
// first q's, then k's, then v's.
struct Share {
  int lo[3], hi[3];   // passes
};
__device__ __forceinline__ Share share_of(int Hq, int Hkv, int per_pass, int part, int parts) {
  const int nq = (Hq + per_pass - 1) / per_pass, nk = (Hkv + per_pass - 1) / per_pass;
  const int all = nq + 2 * nk;
  const int lo = all * part / parts, hi = all * (part + 1) / parts;
  return {{min(lo, nq), min(max(lo - nq, 0), nk), max(lo - nq - nk, 0)},
          {min(hi, nq), min(max(hi - nq, 0), nk), max(hi - nq - nk, 0)}};
}

// 16 bytes to shared memory; zeros, and nothing read, unless `ok`.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Norm and rotation of a step's rows, from the ring; h0 is this thread's head in the first pass.
// REST: rows without a norm of which a part is not rotated. (Kernels of their own: the choice among
// the elements took 3 % of every other pass, and as a path of the same kernel up to 2 %.)
template <int D, int LAYOUT, int PER, bool REST, typename Store>
__device__ __forceinline__ void rotate_step(const RopeParams& p, const __nv_bfloat16* slot, int h0, int left,
                                            int heads, bool normed, const float2 (&ca)[2], const float2 (&sb)[2],
                                            const float2 (&cb)[2], const float2 (&sa)[2], int c, int s,
                                            Store store) {
  constexpr int R = 32 / (D / 8);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int h = h0 + u * R;
    float2 a[2], b[2], y[2], z[2];
    unpack<LAYOUT>(load_row<LAYOUT>(slot + (u * R + s) * D, c, p.r), a, b);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      y[e] = __ffma2_rn(a[e], ca[e], __fmul2_rn(b[e], sb[e]));
      z[e] = __ffma2_rn(b[e], cb[e], __fmul2_rn(a[e], sa[e]));
    }
    if constexpr (REST) keep_rest(c, p.r, a, b, y, z);
    if (!REST && normed) {
      const float rs = rsqrtf(head_sum<D>(dot_pairs(a, b, a, b)) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        y[e] = __fmul2_rn(y[e], make_float2(rs, rs));
        z[e] = __fmul2_rn(z[e], make_float2(rs, rs));
      }
    }
    if (u < left && h < heads) store(h, y, z);
  }
}

template <int D, int LAYOUT, int KIND, bool REST>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeParams p) {
  constexpr int C = D / 8, R = 32 / C;   // threads of a head, heads of a pass
  constexpr int PER = 2;
  __shared__ alignas(16) __nv_bfloat16 ring[kThreads / 32][kSlots][PER * R * D];
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int t = static_cast<int>(unit / p.parts), part = static_cast<int>(unit % p.parts);
  if (t >= p.tokens) return;             // (whole warps)
  const int lane = threadIdx.x & 31, c = lane % C, s = lane / C;
  auto& mine = ring[threadIdx.x / 32];
  const Share sh = share_of(p.Hq, p.Hkv, R, part, p.parts);
  const int nq = (sh.hi[0] - sh.lo[0] + PER - 1) / PER, nk = (sh.hi[1] - sh.lo[1] + PER - 1) / PER;
  const int n = nq + nk + (sh.hi[2] - sh.lo[2] + PER - 1) / PER;   // steps
  const auto issue = [&](int st) {
    if (st < n) {
      const int seg = st < nq ? 0 : st < nq + nk ? 1 : 2;
      const int pass = (seg == 0 ? sh.lo[0] + PER * st
                                 : seg == 1 ? sh.lo[1] + PER * (st - nq) : sh.lo[2] + PER * (st - nq - nk));
      const int hi = seg == 0 ? sh.hi[0] : seg == 1 ? sh.hi[1] : sh.hi[2];
      const __nv_bfloat16* row = (seg == 0 ? p.q + t * p.q_stride
                                           : seg == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride) + 8 * c;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int h = (pass + u) * R + s;
        const bool ok = pass + u < hi && h < (seg == 0 ? p.Hq : p.Hkv);
        copy16(&mine[st % kSlots][u * R * D + lane * 8], row + (ok ? h * D : 0), ok);
      }
    }
    commit_copies();   // (an empty group keeps the count)
  };
  int st = 0;
  // the rows of step st are there, and those of the step before have been read by all lanes
  const auto next = [&]() {
    wait_copies<kSlots - 2>();
    __syncwarp();
    issue(st + kSlots - 1);
  };
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) issue(i);

  const Token at = token_of<KIND != kPack>(p, t);
  if constexpr (KIND == kPack) check_sequences(p, unit * 32 + lane, static_cast<long long>(p.tokens) * p.parts * 32);
  if (KIND == kPack && at.row < 0) {
    wait_copies<0>();
    return;
  }
  float2 co[2], si[2];
  angles(p, at.pos, c, co, si);
#pragma unroll 1
  for (int seg = 0; seg < 2; ++seg) {   // queries, keys
    const float* w = seg ? p.k_weight : p.q_weight;
    const int heads = seg ? p.Hkv : p.Hq, end = seg ? nq + nk : nq;
    if (seg && at.row < 0) break;
    if (st >= end) continue;
    // y_a = rs (x_a (w_a cos) - x_b (w_b sin)), y_b = rs (x_b (w_b cos) + x_a (w_a sin))
    float2 wa[2], wb[2], ca[2], sb[2], cb[2], sa[2];
    load_weights<LAYOUT>(w, c, p.r, wa, wb);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ca[e] = __fmul2_rn(wa[e], co[e]);
      sa[e] = __fmul2_rn(wa[e], si[e]);
      cb[e] = __fmul2_rn(wb[e], co[e]);
      sb[e] = neg2(__fmul2_rn(wb[e], si[e]));
    }
    const auto rows = [&](auto rest) {
      constexpr bool kRest = decltype(rest)::value;
      if (seg == 0) {
        __nv_bfloat16* q_out = p.q_out + static_cast<long long>(t) * p.Hq * D;
        for (int pass = sh.lo[0]; st < end; ++st, pass += PER) {
          next();
          rotate_step<D, LAYOUT, PER, kRest>(
              p, mine[st % kSlots], pass * R + s, sh.hi[0] - pass, heads, w != nullptr, ca, sb, cb, sa, c, s,
              [&](int h, const float2 (&a)[2], const float2 (&b)[2]) {
                store_row<LAYOUT>(q_out + h * D, c, p.r, a, b);
              });
        }
      } else {
        for (int pass = sh.lo[1]; st < end; ++st, pass += PER) {
          next();
          rotate_step<D, LAYOUT, PER, kRest>(
              p, mine[st % kSlots], pass * R + s, sh.hi[1] - pass, heads, w != nullptr, ca, sb, cb, sa, c, s,
              [&](int h, const float2 (&a)[2], const float2 (&b)[2]) {
                const long long row = at.row + static_cast<long long>(h) * at.step;
                if constexpr (KIND == kAppendFp8)
                  store_codes<LAYOUT>(p.k_pages + row * D, c, p.r, a, b, p.k_scale[h]);
                else
                  store_row<LAYOUT>(
                      (KIND == kPack ? p.k_out : reinterpret_cast<__nv_bfloat16*>(p.k_pages)) + row * D, c, p.r,
                      a, b);
              });
        }
      }
    };
    if (REST && w == nullptr) rows(std::bool_constant<REST>());
    else rows(std::false_type());
  }
  if (at.row >= 0) {
    for (int pass = sh.lo[2]; st < n; ++st, pass += PER) {
      next();
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int h = (pass + u) * R + s;
        if (pass + u >= sh.hi[2] || h >= p.Hkv) continue;
        const uint4 raw = load_row<kInterleaved>(mine[st % kSlots] + (u * R + s) * D, c, p.r);
        const long long row = at.row + static_cast<long long>(h) * at.step;
        if constexpr (KIND == kAppendFp8) {
          float2 a[2], b[2];
          unpack<kInterleaved>(raw, a, b);
          store_codes<kInterleaved>(p.v_pages + row * D, c, p.r, a, b, p.v_scale[h]);
        } else {
          __nv_bfloat16* out = KIND == kPack ? p.v_out : reinterpret_cast<__nv_bfloat16*>(p.v_pages);
          *reinterpret_cast<uint4*>(out + row * D + 8 * c) = raw;
        }
      }
    }
  }
  wait_copies<0>();
}

// Gradients of a step's rows: dy in the slot's first half, x, with a norm, in
// the second; this thread's share of the weights' gradients is added to `sum`.
template <int D, int LAYOUT, bool NORM, int PER, bool REST, typename Store>
__device__ __forceinline__ void rotate_step_back(const RopeParams& p, const __nv_bfloat16* slot, int h0, int left,
                                                 int heads, bool normed, const float2 (&wa)[2],
                                                 const float2 (&wb)[2], const float2 (&co)[2],
                                                 const float2 (&si)[2], int c, int s, float2 (&sum_a)[2],
                                                 float2 (&sum_b)[2], Store store) {
  constexpr int R = 32 / (D / 8);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int h = h0 + u * R;
    const bool real = u < left && h < heads;   // (rows past the last are zeros)
    float2 a[2], b[2], y[2], z[2];
    unpack<LAYOUT>(load_row<LAYOUT>(slot + (u * R + s) * D, c, p.r), a, b);
#pragma unroll
    for (int e = 0; e < 2; ++e) {   // g = R^T dy
      y[e] = __ffma2_rn(a[e], co[e], __fmul2_rn(b[e], si[e]));
      z[e] = __ffma2_rn(b[e], co[e], __fmul2_rn(neg2(a[e]), si[e]));
    }
    if constexpr (REST) keep_rest(c, p.r, a, b, y, z);
    if (NORM && !REST && normed) {
      float2 xa[2], xb[2], ua[2], ub[2];
      unpack<LAYOUT>(load_row<LAYOUT>(slot + (PER * R + u * R + s) * D, c, p.r), xa, xb);
      const float ms = head_sum<D>(dot_pairs(xa, xb, xa, xb)) * (1.f / D) + p.eps;
      const float rs = real ? rsqrtf(ms) : 0.f;   // (without eps that of zeros is infinite, and 0 x inf NaN)
      const float2 rs2 = make_float2(rs, rs);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        xa[e] = __fmul2_rn(xa[e], rs2);
        xb[e] = __fmul2_rn(xb[e], rs2);
        sum_a[e] = __ffma2_rn(y[e], xa[e], sum_a[e]);
        sum_b[e] = __ffma2_rn(z[e], xb[e], sum_b[e]);
        ua[e] = __fmul2_rn(y[e], wa[e]);
        ub[e] = __fmul2_rn(z[e], wb[e]);
      }
      const float dot = head_sum<D>(dot_pairs(ua, ub, xa, xb)) * (-1.f / D);
      const float2 dot2 = make_float2(dot, dot);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        y[e] = __fmul2_rn(rs2, __ffma2_rn(xa[e], dot2, ua[e]));
        z[e] = __fmul2_rn(rs2, __ffma2_rn(xb[e], dot2, ub[e]));
      }
    }
    if (real) store(h, y, z);
  }
}

// Gradients of the projection's rows; warps walk over the tokens (and shares
// of them) with the grid's stride and leave their block's sums of the weights'
// gradients in p.part.
// With norms, two rows of dy and of x a thread at once take 110 registers and 16 KB of ring a
// slot: two blocks an SM (120 us for 12,000 tokens of 64 + 2 x 4 heads of 128; one row each, three blocks: 146).
template <int D, bool NORM>
struct BackCfg {
  static constexpr int PER = 2;
  static constexpr int BLOCKS = NORM ? 2 : 3;               // of an SM
  static constexpr int SLOT = (NORM ? 4 : 2) * (32 / (D / 8)) * D;   // elements
  static constexpr int RING = kThreads / 32 * kSlots * SLOT * 2;     // bytes
  static constexpr int SMEM = RING + (NORM ? 16 * kThreads * 4 : 0);
};
template <int D, int LAYOUT, bool NORM, bool REST>
__global__ void __launch_bounds__(kThreads, BackCfg<D, NORM>::BLOCKS) rope_backward_kernel(const RopeParams p) {
  constexpr int C = D / 8, R = 32 / C;
  using C_ = BackCfg<D, NORM>;
  constexpr int PER = C_::PER;
  extern __shared__ __align__(16) uint8_t smem[];
  // q's, then k's; a column is its thread's own
  float (*sums)[kThreads] = reinterpret_cast<float(*)[kThreads]>(smem + C_::RING);
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, c = lane % C, s = lane / C;
  auto* mine = reinterpret_cast<__nv_bfloat16(*)[C_::SLOT]>(smem + threadIdx.x / 32 * (C_::RING / (kThreads / 32)));
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 16; ++e) sums[e][threadIdx.x] = 0.f;
  }
  const long long units = static_cast<long long>(p.tokens) * p.parts;
  for (long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; unit < units;
       unit += static_cast<long long>(gridDim.x) * (kThreads / 32)) {
    const int t = static_cast<int>(unit / p.parts), part = static_cast<int>(unit % p.parts);
    Token at{-1, 0, 0};
    const Share sh = share_of(p.Hq, p.Hkv, R, part, p.parts);
    const int nq = (sh.hi[0] - sh.lo[0] + PER - 1) / PER, nk = (sh.hi[1] - sh.lo[1] + PER - 1) / PER;
    const int n = nq + nk + (sh.hi[2] - sh.lo[2] + PER - 1) / PER;   // steps
    const auto issue = [&](int st) {
      if (st < n) {
        const int seg = st < nq ? 0 : st < nq + nk ? 1 : 2;
        const int pass = (seg == 0 ? sh.lo[0] + PER * st
                                   : seg == 1 ? sh.lo[1] + PER * (st - nq) : sh.lo[2] + PER * (st - nq - nk));
        const int hi = seg == 0 ? sh.hi[0] : seg == 1 ? sh.hi[1] : sh.hi[2];
        const __nv_bfloat16* g = (seg == 0 ? p.dq + static_cast<long long>(t) * p.Hq * D
                                           : (seg == 1 ? p.dk : p.dv) + at.row * D) + 8 * c;
        const long long step = seg == 0 ? D : static_cast<long long>(at.step) * D;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int h = (pass + u) * R + s;
          const bool ok = pass + u < hi && h < (seg == 0 ? p.Hq : p.Hkv);
          copy16(&mine[st % kSlots][u * R * D + lane * 8], g + (ok ? h * step : 0), ok);
          if (NORM && (seg == 0 ? p.q_weight : seg == 1 ? p.k_weight : nullptr) != nullptr) {
            const __nv_bfloat16* x = (seg == 0 ? p.q + t * p.q_stride : p.k + t * p.k_stride) + 8 * c;
            copy16(&mine[st % kSlots][(PER + u) * R * D + lane * 8], x + (ok ? h * D : 0), ok);
          }
        }
      }
      commit_copies();   // (an empty group keeps the count)
    };
    int st = 0;
    const auto next = [&]() {   // as in rope_kernel
      wait_copies<kSlots - 2>();
      __syncwarp();
      issue(st + kSlots - 1);
    };
    __syncwarp();   // the unit before has been read
    // (only the rows of k and v are where the sequence says)
    for (int i = 0; i < min(nq, kSlots - 1); ++i) issue(i);
    at = token_of<false>(p, t);
    if (at.row < 0) {
      wait_copies<0>();
      continue;
    }
    for (int i = min(nq, kSlots - 1); i < kSlots - 1; ++i) issue(i);
    float2 co[2], si[2];
    angles(p, at.pos, c, co, si);
#pragma unroll 1
    for (int seg = 0; seg < 2; ++seg) {   // queries, keys
      const int end = seg ? nq + nk : nq, hi = seg ? sh.hi[1] : sh.hi[0];
      if (st >= end) continue;
      const float* w = !NORM ? nullptr : seg ? p.k_weight : p.q_weight;
      __nv_bfloat16* out = seg ? p.dk_in + t * p.dk_stride : p.dq_in + t * p.dq_stride;
      float2 wa[2], wb[2], sum_a[2], sum_b[2];
      load_weights<LAYOUT>(w, c, p.r, wa, wb);
      sum_a[0] = sum_a[1] = sum_b[0] = sum_b[1] = make_float2(0.f, 0.f);
      const auto rows = [&](auto rest) {
        for (int pass = seg ? sh.lo[1] : sh.lo[0]; st < end; ++st, pass += PER) {
          next();
          rotate_step_back<D, LAYOUT, NORM, PER, decltype(rest)::value>(
              p, mine[st % kSlots], pass * R + s, hi - pass, seg ? p.Hkv : p.Hq, w != nullptr, wa, wb, co, si, c,
              s, sum_a, sum_b, [&](int h, const float2 (&a)[2], const float2 (&b)[2]) {
                store_row<LAYOUT>(out + h * D, c, p.r, a, b);
              });
        }
      };
      if (REST && w == nullptr) rows(std::bool_constant<REST>());   // (as in rope_kernel)
      else rows(std::false_type());
      if constexpr (NORM) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sums[8 * seg + 2 * e][threadIdx.x] += sum_a[e].x;
          sums[8 * seg + 2 * e + 1][threadIdx.x] += sum_a[e].y;
          sums[8 * seg + 4 + 2 * e][threadIdx.x] += sum_b[e].x;
          sums[8 * seg + 5 + 2 * e][threadIdx.x] += sum_b[e].y;
        }
      }
    }
    for (int pass = sh.lo[2]; st < n; ++st, pass += PER) {
      next();
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int h = (pass + u) * R + s;
        if (pass + u < sh.hi[2] && h < p.Hkv)
          *reinterpret_cast<uint4*>(p.dv_in + t * p.dv_stride + h * D + 8 * c) =
              load_row<kInterleaved>(mine[st % kSlots] + (u * R + s) * D, c, p.r);
      }
    }
  }
  wait_copies<0>();
  check_sequences(p, static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x,
                  static_cast<long long>(gridDim.x) * kThreads);
  if constexpr (NORM) {
    // the block's sums, over the threads that hold the same elements, in a fixed order
    __syncthreads();
    if (threadIdx.x < 2 * D) {
      const int which = threadIdx.x / D, cc = threadIdx.x % D / 8, e = threadIdx.x % 8;
      float x = 0.f;
      for (int j = 0; j < kThreads / C; ++j) x += sums[8 * which + e][j * C + cc];
      const int el = e < 4 ? first_of<LAYOUT>(cc, e, p.r) : second_of<LAYOUT>(cc, e - 4, p.r);
      p.part[(static_cast<long long>(blockIdx.x) * 2 + which) * D + el] = x;
    }
  }
}

// The weights' gradients: the blocks' sums added in a fixed order, 32 columns
// of the 2 d a block, 32 threads a column.
__global__ void __launch_bounds__(1024) rope_weights_kernel(const float* part, int blocks, int d,
                                                            float* dq_weight, float* dk_weight) {
  __shared__ float s[32][33];
  grid_dependency_wait();
  const int x = threadIdx.x % 32, slice = threadIdx.x / 32, col = blockIdx.x * 32 + x;
  float sum = 0.f;
#pragma unroll 8
  for (int b = slice; b < blocks; b += 32) sum += part[static_cast<long long>(b) * 2 * d + col];
  s[slice][x] = sum;
  __syncthreads();
  if (slice != 0) return;
  for (int j = 1; j < 32; ++j) sum += s[j][x];
  float* out = col < d ? dq_weight : dk_weight;
  if (out) out[col % d] = sum;
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

// Whether some rows are neither normed nor rotated as a whole.
bool has_rest(const RopeParams& p, int d) { return p.r < d && !(p.q_weight && p.k_weight); }

template <int D, int KIND, bool REST>
void (*pick_layout(int layout))(const RopeParams) {
  return layout == kHalf          ? rope_kernel<D, kHalf, KIND, REST>
         : layout == kInterleaved ? rope_kernel<D, kInterleaved, KIND, REST>
                                  : rope_kernel<D, kHalfOdd, KIND, REST>;
}
template <int D, int KIND>
void (*pick_forward(const RopeParams& p, int layout))(const RopeParams) {
  return has_rest(p, D) ? pick_layout<D, KIND, true>(layout) : pick_layout<D, KIND, false>(layout);
}

template <int D, bool NORM, bool REST>
void (*pick_back_layout(int layout))(const RopeParams) {
  return layout == kHalf          ? rope_backward_kernel<D, kHalf, NORM, REST>
         : layout == kInterleaved ? rope_backward_kernel<D, kInterleaved, NORM, REST>
                                  : rope_backward_kernel<D, kHalfOdd, NORM, REST>;
}
template <int D, bool NORM>
void (*pick_backward(const RopeParams& p, int layout))(const RopeParams) {
  return has_rest(p, D) ? pick_back_layout<D, NORM, true>(layout) : pick_back_layout<D, NORM, false>(layout);
}

int launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

// Warps that share a token's heads: one, while that leaves every SM 16 warps. (37 tokens of
// 64 + 2 x 8 heads of 64: 3.2 us.)
int shares(int32_t tokens, int32_t Hq, int32_t Hkv, int d) {
  const int R = 256 / d, passes = (Hq + R - 1) / R + 2 * ((Hkv + R - 1) / R);
  int parts = 1;
  while (int64_t{tokens} * parts < 16LL * 152 && 2 * parts <= passes) parts *= 2;
  return parts;
}

int launch_forward(RopeParams& p, int d, int kind, int interleaved, cudaStream_t stream) {
  const int layout = layout_of(p.r, interleaved);
  p.parts = shares(p.tokens, p.Hq, p.Hkv, d);
  const int64_t blocks = (int64_t{p.tokens} * p.parts + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks >= (int64_t{1} << 31)) return refuse(SINKATTN_UNSUPPORTED, "too many work items");
  void (*kern)(const RopeParams) =
      d == 64 ? (kind == kPack     ? pick_forward<64, kPack>(p, layout)
                 : kind == kAppend ? pick_forward<64, kAppend>(p, layout)
                                   : pick_forward<64, kAppendFp8>(p, layout))
              : (kind == kPack     ? pick_forward<128, kPack>(p, layout)
                 : kind == kAppend ? pick_forward<128, kAppend>(p, layout)
                                   : pick_forward<128, kAppendFp8>(p, layout));
  kern<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return launched("rope", cudaGetLastError());
}

// (a fixed bound, so that neither the workspace nor the order of the sums goes by the device)
int backward_blocks(int32_t tokens) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tokens, 2 * 152)));
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
  // YaRN: pairs below `low` keep their frequency, pairs above `high` (which may be below
  // the first) have it divided by the factor, those between are blended, linearly in the index
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
      const double ramp =
          i > high ? 1.0 : std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
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
    // f / (2 pi) as hi + lo: 1 / (2 pi) in two doubles, and the product's rounding (hi is an
    // fma, so that no compiler takes the product unrounded into the difference below)
    const double f = std::fabs(inv_freq[i]), c = 0x1.45f306dc9c883p-3, c_lo = -0x1.6b01ec5417056p-57;
    const double hi = std::fma(f, c, 0.0), lo = std::fma(f, c_lo, std::fma(f, c, -hi));
    // whole units of hi (its fraction is exact), then what is left of it and lo, rounded
    const double units = std::ldexp(hi - std::floor(hi), 64), whole = std::floor(units);
    const double rest = std::nearbyint(units - whole + std::ldexp(std::fmod(lo, 1.0), 64));
    const uint64_t far = std::fabs(rest) < 0x1p64 ? static_cast<uint64_t>(std::fabs(rest)) : 0;
    const uint64_t word = static_cast<uint64_t>(whole) + (rest < 0.0 ? uint64_t{0} - far : far);
    turns[i] = inv_freq[i] < 0.0 ? uint64_t{0} - word : word;
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
  p.parts = shares(tokens, num_qo_heads, num_kv_heads, head_dim);
  // without sums of weights' gradients there is no reason to hold a block longer
  const int64_t blocks = norm ? backward_blocks(tokens) : (int64_t{tokens} * p.parts + kThreads / 32 - 1) /
                                                              (kThreads / 32);
  if (blocks >= (int64_t{1} << 31)) return refuse(SINKATTN_UNSUPPORTED, "too many work items");
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
  const int layout = layout_of(p.r, interleaved);
  void (*kern)(const RopeParams) =
      head_dim == 64 ? (norm ? pick_backward<64, true>(p, layout) : pick_backward<64, false>(p, layout))
                     : (norm ? pick_backward<128, true>(p, layout) : pick_backward<128, false>(p, layout));
  const int smem = head_dim == 64 ? (norm ? BackCfg<64, true>::SMEM : BackCfg<64, false>::SMEM)
                                  : (norm ? BackCfg<128, true>::SMEM : BackCfg<128, false>::SMEM);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return refuse(SINKATTN_CUDA_ERROR, "cudaFuncSetAttribute failed");
  kern<<<static_cast<unsigned>(blocks), kThreads, smem, s>>>(p);
  if ((rc = launched("rope backward", cudaGetLastError())) || !norm) return rc;
  return launched("rope weights",
                  launch_chained(rope_weights_kernel, dim3(static_cast<unsigned>(2 * head_dim / 32)), 1024, 0, s,
                                 static_cast<const float*>(p.part), static_cast<int>(blocks), head_dim,
                                 q_weight ? dq_weight : nullptr, k_weight ? dk_weight : nullptr));
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
