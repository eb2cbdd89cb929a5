// Fold of one (row, query head)'s split-KV partials with the sink counted
// exactly once, by one warp ("GPT-OSS on Day 0", section "Kernels for
// GPT-OSS / Sink attention": the sink belongs to one block only when the
// sequence is split). With M the maximum of the sink and every chunk's m_s:
//   w_s = e^{m_s - M},  D = e^{s_h - M} + sum_s w_s d_s,
//   out = sum_s w_s acc_s / D,  lse = M + ln D
// (the sink term is absent without a sink; an empty chunk has m_s = -inf).
// Lane s computes w_s; every lane owns D/32 output columns and reads each
// chunk's accumulator slice with one vector load. Up to 16 chunks, all loads
// (the (m, d) pairs and every slice) are in flight at once, one memory round
// trip per row; beyond that, eight slices at a time after a pass over the
// maxima. Partials are read once, through L2 only (ld.global.cg).
#pragma once

#include "common.cuh"

namespace sinkattn {

template <int D>
__device__ __forceinline__ void merge_row(const float* md, const float* acc, float sink, int S,
                                          int lane, __nv_bfloat16* orow, float* lse_out) {
  constexpr int VEC = D / 32;   // 2 or 4 floats per lane
  constexpr float NEG_INF = kNegInf;
  float o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = 0.f;
  float M = sink, dpart = 0.f;
  if (S <= 16) {
    // one round trip: lane s's (m_s, d_s) and every chunk's accumulator
    // slice are loaded together; the weights follow from the maximum
    const float2 mdl = lane < S ? __ldcg(reinterpret_cast<const float2*>(md + 2 * lane))
                                : make_float2(NEG_INF, 0.f);
    float a[16][VEC];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      if (u < S) {
        const float* src = acc + u * D + lane * VEC;
        if constexpr (VEC == 4) {
          const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
          a[u][0] = t.x; a[u][1] = t.y; a[u][2] = t.z; a[u][3] = t.w;
        } else {
          const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
          a[u][0] = t.x; a[u][1] = t.y;
        }
      }
    }
    M = fmaxf(M, mdl.x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float w = 0.f;
    if (mdl.x != NEG_INF) {
      w = ex2((mdl.x - M) * kLog2e);
      dpart = mdl.y * w;
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const float wu = __shfl_sync(0xffffffffu, w, u);
      if (u < S) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(a[u][e], wu, o[e]);
      }
    }
  } else {
    for (int s = lane; s < S; s += 32) M = fmaxf(M, __ldcg(md + 2 * s));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int s0 = 0; s0 < S; s0 += 32) {
      float w = 0.f;
      if (s0 + lane < S) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(md + 2 * (s0 + lane)));
        if (v.x != NEG_INF) {
          w = ex2((v.x - M) * kLog2e);
          dpart = fmaf(v.y, w, dpart);
        }
      }
      const int cnt = min(32, S - s0);
      for (int i = 0; i < cnt; i += 8) {
        float a[8][VEC];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (i + u < cnt) {
            const float* src = acc + (s0 + i + u) * D + lane * VEC;
            if constexpr (VEC == 4) {
              const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
              a[u][0] = t.x; a[u][1] = t.y; a[u][2] = t.z; a[u][3] = t.w;
            } else {
              const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
              a[u][0] = t.x; a[u][1] = t.y;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w, (i + u) & 31);
          if (i + u < cnt) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = fmaf(a[u][e], wu, o[e]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dpart += __shfl_xor_sync(0xffffffffu, dpart, off);
  const float dsum = dpart + ((sink == NEG_INF) ? 0.f : ex2((sink - M) * kLog2e));
  const float inv = dsum > 0.f ? 1.f / dsum : 0.f;
  __nv_bfloat16* op = orow + lane * VEC;
  if constexpr (VEC == 4) {
    uint2 pk;
    pk.x = pack_bf16x2(o[0] * inv, o[1] * inv);
    pk.y = pack_bf16x2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(op) = pk;
  } else {
    *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(o[0] * inv, o[1] * inv);
  }
  if (lse_out != nullptr && lane == 0) *lse_out = dsum > 0.f ? M + lg2(dsum) * kLn2 : NEG_INF;
}

// The same fold for rows of which many slots are empty (d_s = 0; a NaN sum is
// a row's answer, and no empty slot): R rows per
// warp, 32 / R lanes each for the (m, d) pairs (S <= 32 / R), and then only the
// accumulators that have a weight. A row's loads depend on its weights, two
// memory round trips, so the rows of a warp take theirs together: eight
// accumulator loads are in flight. Slots are taken in order.
template <int D, int R>
__device__ __forceinline__ void merge_rows_sparse(const float* part_md, const float* part_acc,
                                                  const float* sinks, long long row0, int rows,
                                                  int Hq, int S, int lane, __nv_bfloat16* out,
                                                  float* lse) {
  constexpr int VEC = D / 32, W = 32 / R, U = 8 / R;
  const int r = lane / W, s = lane % W;   // the lane's row and slot
  const bool real = r < rows;
  const long long row = row0 + r;
  const float2 mine = real && s < S
                          ? __ldcg(reinterpret_cast<const float2*>(part_md + (row * S + s) * 2))
                          : make_float2(kNegInf, 0.f);
  const float sink = real && sinks ? sinks[static_cast<int>(row % Hq)] : kNegInf;
  const bool some = mine.y != 0.f;
  float M = fmaxf(sink, some ? mine.x : kNegInf);
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float w = some ? ex2((mine.x - M) * kLog2e) : 0.f;
  float total = w * mine.y;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (sink != kNegInf) total += sink == M ? 1.f : ex2((sink - M) * kLog2e);
  w *= total != 0.f ? 1.f / total : 0.f;
  if (lse != nullptr && real && s == 0) lse[row] = total != 0.f ? M + lg2(total) * kLn2 : kNegInf;
  const uint32_t vote = __ballot_sync(0xffffffffu, some);
  uint32_t left[R];
  float o[R][VEC];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    left[i] = R == 1 ? vote : (vote >> (i * W)) & ((1u << (W & 31)) - 1u);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[i][e] = 0.f;
  }
  for (uint32_t any = vote; any;) {   // warp-uniform
    float a[U][R][VEC], wu[U][R];
    any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int slot = left[i] ? __ffs(left[i]) - 1 : -1;
        left[i] &= left[i] - 1;   // (0 stays 0)
        const float t = __shfl_sync(0xffffffffu, w, i * W + max(slot, 0));
        wu[u][i] = slot >= 0 ? t : 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[u][i][e] = 0.f;
        if (slot >= 0) {
          const float* src = part_acc + ((row0 + i) * S + slot) * D + lane * VEC;
          if constexpr (VEC == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            a[u][i][0] = v.x; a[u][i][1] = v.y; a[u][i][2] = v.z; a[u][i][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            a[u][i][0] = v.x; a[u][i][1] = v.y;
          }
        }
        if (u == U - 1) any |= left[i];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[i][e] = fmaf(a[u][i][e], wu[u][i], o[i][e]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i >= rows) break;
    __nv_bfloat16* op = out + (row0 + i) * D + lane * VEC;
    if constexpr (VEC == 4) {
      uint2 pk;
      pk.x = pack_bf16x2(o[i][0], o[i][1]);
      pk.y = pack_bf16x2(o[i][2], o[i][3]);
      *reinterpret_cast<uint2*>(op) = pk;
    } else {
      *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(o[i][0], o[i][1]);
    }
  }
}

// One row of any number of slots, 32 at a time.
template <int D>
__device__ __forceinline__ void merge_row_sparse(const float* md, const float* acc, float sink,
                                                 int S, int lane, __nv_bfloat16* orow,
                                                 float* lse_out) {
  constexpr int VEC = D / 32;
  float o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = 0.f;
  float M = sink, total = (sink == kNegInf) ? 0.f : 1.f;   // relative to M
  for (int s0 = 0; s0 < S; s0 += 32) {
    const float2 mine = s0 + lane < S ? __ldcg(reinterpret_cast<const float2*>(md + 2 * (s0 + lane)))
                                      : make_float2(kNegInf, 0.f);
    const bool some = mine.y != 0.f;
    const uint32_t vote = __ballot_sync(0xffffffffu, some);
    if (vote == 0) continue;
    float top = some ? mine.x : kNegInf;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float m1 = fmaxf(M, top);
    const float keep = M == m1 ? 1.f : (M == kNegInf ? 0.f : ex2((M - m1) * kLog2e));
    M = m1;
    const float w = some ? ex2((mine.x - M) * kLog2e) : 0.f;
    float sum = w * mine.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    total = total * keep + sum;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] *= keep;
    for (uint32_t left = vote; left; left &= left - 1) {
      const int s = __ffs(left) - 1;
      const float wu = __shfl_sync(0xffffffffu, w, s);
      const float* src = acc + static_cast<size_t>(s0 + s) * D + lane * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = fmaf(__ldcg(src + e), wu, o[e]);
    }
  }
  const float inv = total != 0.f ? 1.f / total : 0.f;
  __nv_bfloat16* op = orow + lane * VEC;
#pragma unroll
  for (int e = 0; e < VEC; e += 2)
    *reinterpret_cast<uint32_t*>(op + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (lse_out != nullptr && lane == 0) *lse_out = total != 0.f ? M + lg2(total) * kLn2 : kNegInf;
}

}  // namespace sinkattn
