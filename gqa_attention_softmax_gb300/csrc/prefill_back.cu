// Backward pass of the varlen prefill with a per-head softmax sink (rules:
// sinkattn.h) on the 5th-generation tensor cores. With P = exp(l - lse) over
// the visible keys and delta = dout . out - dlse, dS = P (dout v^T - delta):
// dq = c dS k, dk = c dS^T q, dv = P^T dout, dsink = -sum exp(s - lse) delta.
//
// Three passes. back_delta_kernel: delta and the sinks' gradients, one read of
// dout and out. back_dkv_kernel: one CTA holds 128 keys of a KV head and walks
// over the query rows that see them; back_dq_kernel: one CTA holds 128 query
// rows (tokens x the heads of a group) and walks over the keys they see. P and
// dS are computed in both, seven products a tile pair instead of five: no sum
// crosses CTAs, so there are no atomics (whose order would change the results),
// no fp32 buffer of dq in memory, and the group's heads add up in the
// accumulators.
//
// Both kernels: warp 0 stages tiles by TMA, warp 1 issues every MMA, warps
// 2 .. 9 compute P and dS, one thread per TMEM lane and half of the 128 columns.
// P and dS are rounded to bf16 for the products that take them; P enters dS
// unrounded. Every wait is bounded; on a timeout the CTA records
// SINKATTN_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace sinkattn {

__device__ int g_status_prefill_back;

namespace {

struct BackParams {
  const __nv_bfloat16 *dout, *q, *k, *v, *out;
  const float *lse, *sinks, *dlse;
  const int32_t *cu_q, *cu_k;
  int batch, total_q, total_k, max_q, max_kv, Hq, Hkv, G;
  float sm_scale, scale_log2;
  int causal, window;
  __nv_bfloat16 *dq, *dk, *dv;
  float *dsinks, *delta, *sink_part;
  int per;       // tokens of a block of the delta pass
  int QB, nqb;   // query tokens of a tile of 128 rows, tiles of the longest sequence
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

// ---------------------------------------------------------------------------
constexpr int kBackThreads = 320;   // producer, MMA issuer, 8 warps of P and dS
constexpr int kSoftThreads = 256;
constexpr int kSub = 128 * 128;     // [128 rows][64 bf16], 128B-swizzled: 16 KB

// dK, dV. S^T = K Q^T and dP^T = V dO^T (M 128 keys, N 128 query rows, K d; all from shared
// memory), dV += P^T dO and dK += dS^T Q (M 128 keys, N d, K 128; P^T and dS^T
// from TMEM, where they replace S^T and dP^T). Keys in the TMEM lanes make
// P^T and dS^T the MMA's A operand as they are.
template <int D>
struct DkvCfg {
  static constexpr int NSUB = D / 64;
  static constexpr int TILE = NSUB * kSub;
  static constexpr int NST = D == 64 ? 4 : 2;       // stages of Q and dO
  static constexpr int STAGE = 2 * TILE;
  static constexpr int NSB = D == 64 ? 2 : 1;       // S^T buffers (TMEM holds no more at d 128)
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;            // stage s: Q, then dO
  static constexpr int OFF_ROW = OFF_Q + NST * STAGE;   // [2][2][128] -lse log2 e, -delta
  static constexpr int OFF_BAR = OFF_ROW + 2 * 2 * 128 * 4;
  static constexpr int N_BARS = 1 + 2 * NST + 2 * NSB + 5 + 2;
  static constexpr int SMEM = 1024 + OFF_BAR + N_BARS * 8 + 64;
  static constexpr uint32_t COL_S = 0;
  static constexpr uint32_t COL_DP = 128 * NSB;
  static constexpr uint32_t COL_DV = COL_DP + 128;
  static constexpr uint32_t COL_DK = COL_DV + D;
  static_assert(COL_DK + D <= 512, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Zeros rows [from, 128) of a tile in shared memory (threads 0 .. 255 of the softmax warps).
template <int NSUB>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int tid, int threads) {
  const int n = (128 - from) * 8;
  for (int u = tid; u < n * NSUB; u += threads)
    *reinterpret_cast<uint4*>(tile + (u / n) * kSub + from * 128 + (u % n) * 16) = make_uint4(0, 0, 0, 0);
}

// The A operand of a TS product: bf16 pairs that replaced 128 fp32 columns, each half's
// 64 elements in the first 32 columns of its half. K step kk covers elements 16 kk ...
__device__ __forceinline__ uint32_t half_packed(uint32_t base, int kk) {
  return base + static_cast<uint32_t>(8 * kk + (kk >= 4 ? 32 : 0));
}

template <int D>
__global__ void __launch_bounds__(kBackThreads, 1)
    back_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const BackParams p) {
  using C = DkvCfg<D>;
  constexpr int NST = C::NST, NSB = C::NSB, NSUB = C::NSUB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* q_full = kv_full + 1;      // [NST]
  uint64_t* q_empty = q_full + NST;    // [NST]
  uint64_t* s_full = q_empty + NST;    // [NSB] S^T(j) written
  uint64_t* p_full = s_full + NSB;     // [NSB] P^T(j) written (256 arrivals)
  uint64_t* dp_full = p_full + NSB;    // dP^T(j) written
  uint64_t* ds_full = dp_full + 1;     // dS^T(j) written (256 arrivals)
  uint64_t* dv_done = ds_full + 1;
  uint64_t* dk_done = dv_done + 1;
  uint64_t* row_full = dk_done + 1;    // [2] the rows' lse and delta staged (256 arrivals)
  uint64_t* drain = row_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefill_back;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // items: the first key tiles (which the most queries see) of all sequences and KV heads first
  const int per = p.Hkv * p.batch;
  const int kt = static_cast<int>(blockIdx.x) / per;
  const int kvh = static_cast<int>(blockIdx.x) % per % p.Hkv;
  const int b = static_cast<int>(blockIdx.x) % per / p.Hkv;
  const Seq s = load_seq(p, b);
  if (!s.ok) {
    if (threadIdx.x == 0) atomicExch(status, SINKATTN_BAD_LENGTHS);
    return;
  }
  const int k0 = kt * 128;
  if (k0 >= s.lk) return;   // uniform over the CTA, before any barrier or TMEM use
  const int nk = min(128, s.lk - k0);
  const int off = s.lk - s.lq;   // position of query 0
  // queries [i0, i1) see some key of the tile
  const int i0 = p.causal ? max(0, k0 - off) : 0;
  const int i1 = p.window > 0 ? max(0, min(s.lq, k0 + nk - 1 + p.window - off)) : s.lq;
  const int n = i1 > i0 ? (i1 - i0 + p.QB - 1) / p.QB : 0;
  const int G = p.G, rows = G * p.QB;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftThreads);
    }
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kSoftThreads);
    mbar_init(dv_done, 1);
    mbar_init(dk_done, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&row_full[i], kSoftThreads);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (rows < 128) {   // rows that no copy writes
    for (int i = 0; i < 2 * NST; ++i)
      zero_rows<NSUB>(smem + C::OFF_Q + i * C::TILE, rows, threadIdx.x, kBackThreads);
    tc::fence_proxy_async_smem();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;   // producer: stages whose copies were issued (or left out by the test hook)

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmDo);
      mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
      const int slab = p.Hkv * s.k0 + kvh * s.lk + k0;
#pragma unroll
      for (int sub = 0; sub < NSUB; ++sub) {
        tma_load_2d(smem + C::OFF_K + sub * kSub, &tmK, sub * 64, slab, kv_full);
        tma_load_2d(smem + C::OFF_V + sub * kSub, &tmV, sub * 64, slab, kv_full);
      }
      const int skip_tile = hook_skip_tile();
      const uint32_t bytes = static_cast<uint32_t>(2 * NSUB * 128 * rows);
      for (int j = 0; j < n; ++j) {
        const int st = j % NST;
        if (!mbar_wait(&q_empty[st], ((j / NST) & 1) ^ 1, abort_flag, status)) break;
        issued = j + 1;
        if (j == skip_tile) continue;   // test hook: the waits for this tile run out
        uint8_t* qt = smem + C::OFF_Q + st * C::STAGE;
        mbar_arrive_expect_tx(&q_full[st], bytes);
        const int tok = s.q0 + i0 + j * p.QB;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tc::tma_load_3d(qt + sub * kSub, &tmQ, sub * 64, kvh * G, tok, &q_full[st]);
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tc::tma_load_3d(qt + C::TILE + sub * kSub, &tmDo, sub * 64, kvh * G, tok, &q_full[st]);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = tc::elect_one();
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };
    constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, true);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t qt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), kSub, 1024);   // MN-major
    // D (+)= A B^T over d; both K-major
    auto ss = [&](uint32_t d_tm, uint64_t a, uint64_t bq, uint64_t* bar) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t at = static_cast<uint64_t>(kk >> 2) * (kSub >> 4) + (kk & 3) * 2;
          tc::mma_ss(d_tm, a + at, bq + at, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc::commit(bar);
      }
      __syncwarp();
    };
    auto ts = [&](uint32_t d_tm, uint32_t a, uint64_t bq, bool first) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_ts(d_tm, half_packed(a, kk), bq + static_cast<uint64_t>(kk) * 128u, idesc_o,
                     first && kk == 0 ? 0u : 1u);
      }
      __syncwarp();
    };
    auto stage = [&](int j) { return static_cast<uint64_t>(j % NST) * (C::STAGE >> 4); };
    auto issue_s = [&](int j) {
      ss(tmem + C::COL_S + 128 * (j % NSB), kd, qd + stage(j), &s_full[j % NSB]);
    };
    auto issue_dp = [&](int j) {
      ss(tmem + C::COL_DP, vd, qd + stage(j) + (C::TILE >> 4), dp_full);
    };
    bool ok = n > 0 && wwait(kv_full, 0) && wwait(&q_full[0], 0);
    if (ok) {
      tc::fence_after_sync();
      issue_s(0);
      issue_dp(0);
    }
    for (int j = 0; ok && j < n; ++j) {
      const bool more = j + 1 < n;
      // S^T(j + 1) overwrites the P^T that dV(j + 1 - NSB) reads
      if (NSB == 2 && more) {
        if (!wwait(&q_full[(j + 1) % NST], ((j + 1) / NST) & 1) || (j >= 1 && !wwait(dv_done, (j - 1) & 1))) break;
        tc::fence_after_sync();
        issue_s(j + 1);
      }
      if (!wwait(&p_full[j % NSB], (j / NSB) & 1)) break;
      tc::fence_after_sync();
      ts(tmem + C::COL_DV, tmem + C::COL_S + 128 * (j % NSB), qt + stage(j) + (C::TILE >> 4), j == 0);
      if (leader) tc::commit(dv_done);
      __syncwarp();
      if (NSB == 1 && more) {
        if (!wwait(&q_full[(j + 1) % NST], ((j + 1) / NST) & 1) || !wwait(dv_done, j & 1)) break;
        tc::fence_after_sync();
        issue_s(j + 1);
      }
      if (!wwait(ds_full, j & 1)) break;
      tc::fence_after_sync();
      ts(tmem + C::COL_DK, tmem + C::COL_DP, qt + stage(j), j == 0);
      if (leader) {
        tc::commit(dk_done);
        tc::commit(&q_empty[j % NST]);
      }
      __syncwarp();
      if (more) {
        // dP^T(j + 1) overwrites the dS^T that dK(j) reads
        if (!wwait(dk_done, j & 1)) break;
        tc::fence_after_sync();
        issue_dp(j + 1);
      }
    }
    // every MMA this warp issued has completed before the CTA frees TMEM
    if (leader) tc::commit(drain);
    __syncwarp();
    mbar_drain(drain, 0);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int tid = threadIdx.x - 64;
    const int half = (warp - 2) >> 2;
    const int quad = warp & 3;         // TMEM lane quadrant this warp may access
    const int key = quad * 32 + lane;  // key of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* row_s = reinterpret_cast<float*>(smem + C::OFF_ROW);   // [2][2][128]
    const float c2 = p.scale_log2;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };
    // thread tid stages -lse log2(e) (tid < 128) or -delta of row tid % 128;
    // a row outside the tile, and one that sees nothing, gets lse = +inf: P = 0
    const int r = tid & 127, rt = r / G;
    auto fetch = [&](int j) -> float {
      const int i = i0 + j * p.QB + rt;
      if (r >= rows || i >= i1) return tid < 128 ? kNegInf : 0.f;
      const long long at = static_cast<long long>(s.q0 + i) * p.Hq + kvh * G + (r - rt * G);
      if (tid >= 128) return -p.delta[at];
      const float l = p.lse[at];
      return l == kNegInf ? kNegInf : -l * kLog2e;
    };
    auto put = [&](int j, float v) {
      row_s[(j & 1) * 256 + tid] = v;
      mbar_arrive(&row_full[j & 1]);
    };
    bool ok = true;
    if (n > 0) put(0, fetch(0));
    for (int j = 0; j < n; ++j) {
      float next = 0.f;
      if (j + 1 < n) next = fetch(j + 1);
      const int t0 = i0 + j * p.QB;              // first query of the tile
      const int nt = min(p.QB, i1 - t0);
      const int pos0 = off + t0;
      // columns [clo, chi) of this key's row are visible
      int clo = 0, chi = nt * G;
      bool masked = nt * G < 128;
      if (p.causal) {
        masked = masked || k0 + 127 > pos0;
        clo = max(0, min(nt, k0 + key - pos0)) * G;
      }
      if (p.window > 0) {
        masked = masked || k0 + p.window < pos0 + p.QB;
        chi = max(0, min(nt, k0 + key + p.window - pos0)) * G;
      }
      if (!wwait(&row_full[j & 1], (j >> 1) & 1) || !wwait(&s_full[j % NSB], (j / NSB) & 1)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t s_addr = lane_base + C::COL_S + 128 * (j % NSB) + 64 * half;
      const uint32_t dp_addr = lane_base + C::COL_DP + 64 * half;
      const float4* lse4 = reinterpret_cast<const float4*>(row_s + (j & 1) * 256 + 64 * half);
      const float4* del4 = lse4 + 32;
      const int lo = clo - 64 * half, hi = chi - 64 * half;
      float v[2][32];
      tc::tmem_ld32(s_addr, v[0]);
      tc::tmem_ld32(s_addr + 32, v[1]);
      tc::tmem_wait_ld();
      const float2 cc = make_float2(c2, c2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = lse4[c * 8 + e / 4];
          const float2 x = __ffma2_rn(make_float2(v[c][e], v[c][e + 1]), cc, make_float2(l.x, l.y));
          const float2 y = __ffma2_rn(make_float2(v[c][e + 2], v[c][e + 3]), cc, make_float2(l.z, l.w));
          v[c][e] = ex2(x.x);
          v[c][e + 1] = ex2(x.y);
          v[c][e + 2] = ex2(y.x);
          v[c][e + 3] = ex2(y.y);
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) v[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(v[c][2 * e], v[c][2 * e + 1]);
        tc::tmem_st16(s_addr + 16 * c, pk);
      }
      if (nt * G < rows) {
        // The sequence ends inside the tile: the rows behind it are another
        // sequence's, whose NaN would pass through zero weights. Both products
        // that read the tile along d are done.
        if (!wwait(dp_full, j & 1)) { ok = false; break; }
        uint8_t* tile = smem + C::OFF_Q + (j % NST) * C::STAGE;
        zero_rows<NSUB>(tile, nt * G, tid, kSoftThreads);
        zero_rows<NSUB>(tile + C::TILE, nt * G, tid, kSoftThreads);
        tc::fence_proxy_async_smem();
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&p_full[j % NSB]);

      if (!wwait(dp_full, j & 1)) { ok = false; break; }
      tc::fence_after_sync();
      float w[2][32];
      tc::tmem_ld32(dp_addr, w[0]);
      tc::tmem_ld32(dp_addr + 32, w[1]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = del4[c * 8 + e / 4];
          const float2 x = __fmul2_rn(make_float2(v[c][e], v[c][e + 1]),
                                      __fadd2_rn(make_float2(w[c][e], w[c][e + 1]), make_float2(d.x, d.y)));
          const float2 y = __fmul2_rn(make_float2(v[c][e + 2], v[c][e + 3]),
                                      __fadd2_rn(make_float2(w[c][e + 2], w[c][e + 3]), make_float2(d.z, d.w)));
          w[c][e] = x.x;
          w[c][e + 1] = x.y;
          w[c][e + 2] = y.x;
          w[c][e + 3] = y.y;
        }
        if (masked) {   // (0 x NaN of another row is not 0)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) w[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(w[c][2 * e], w[c][2 * e + 1]);
        tc::tmem_st16(dp_addr + 16 * c, pk);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(ds_full);
      if (j + 1 < n) put(j + 1, next);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && n > 0) ok = wwait(dv_done, (n - 1) & 1) && wwait(dk_done, (n - 1) & 1);
    tc::fence_after_sync();
    // half 0 stores dV, half 1 dK
    const long long row = static_cast<long long>(p.Hkv) * s.k0 + static_cast<long long>(kvh) * s.lk + k0 + key;
    tc::store_o_rows<D>(lane_base + (half ? C::COL_DK : C::COL_DV), !(ok && n > 0),
                        half ? p.sm_scale : 1.f, (half ? p.dk : p.dv) + row * D, key < nk, lane);
  }

  // a warp that left its loop early may still have TMEM loads or stores in flight
  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // a wait gave up: let every issued copy land before the CTA's shared
    // memory goes away (a left-out tile's phase never completes: bounded)
    if (n > 0) mbar_drain(kv_full, 0);
    for (int i = max(0, issued - NST); i < issued; ++i) mbar_drain(&q_full[i % NST], (i / NST) & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// dQ. S = Q K^T and dP = dO V^T (M 128 query rows, N 128 keys, K d; from shared memory),
// dQ += dS K (dS from TMEM, where it replaces S). Two S buffers, so that
// S(j + 1) is on its way while dS(j) is computed.
template <int D>
struct DqCfg {
  static constexpr int NSUB = D / 64;
  static constexpr int TILE = NSUB * kSub;
  static constexpr int NK = D == 64 ? 4 : 3;   // stages of K
  static constexpr int NV = D == 64 ? 4 : 2;   // stages of V, read by the first of the products only
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = TILE;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_BAR = OFF_V + NV * TILE;
  static constexpr int N_BARS = 1 + 2 * NK + 2 * NV + 8;
  static constexpr int SMEM = 1024 + OFF_BAR + N_BARS * 8 + 64;
  static constexpr uint32_t COL_S = 0;
  static constexpr uint32_t COL_DP = 256;
  static constexpr uint32_t COL_DQ = 384;
  static_assert(COL_DQ + D <= 512, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kBackThreads, 1)
    back_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const BackParams p) {
  using C = DqCfg<D>;
  constexpr int NK = C::NK, NV = C::NV, NSUB = C::NSUB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;       // [NK]
  uint64_t* k_empty = k_full + NK;     // [NK]
  uint64_t* v_full = k_empty + NK;     // [NV]
  uint64_t* v_empty = v_full + NV;     // [NV]
  uint64_t* s_full = v_empty + NV;     // [2] S(j) written
  uint64_t* ds_full = s_full + 2;      // [2] dS(j) written (256 arrivals)
  uint64_t* dp_full = ds_full + 2;     // dP(j) written
  uint64_t* dp_free = dp_full + 1;     // dP(j) read (256 arrivals)
  uint64_t* dq_done = dp_free + 1;
  uint64_t* drain = dq_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefill_back;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // items: the last query blocks (which see the most keys) first
  const int per = p.Hkv * p.batch;
  const int qb = p.nqb - 1 - static_cast<int>(blockIdx.x) / per;
  const int kvh = static_cast<int>(blockIdx.x) % per % p.Hkv;
  const int b = static_cast<int>(blockIdx.x) % per / p.Hkv;
  const Seq s = load_seq(p, b);
  if (!s.ok) {
    if (threadIdx.x == 0) atomicExch(status, SINKATTN_BAD_LENGTHS);
    return;
  }
  const int t0 = qb * p.QB;
  if (t0 >= s.lq) return;   // uniform over the CTA, before any barrier or TMEM use
  const int nt = min(p.QB, s.lq - t0);
  const int pos0 = s.lk - s.lq + t0;
  const int k_hi = p.causal ? pos0 + nt : s.lk;                 // keys [k_lo, k_hi) are seen by some row
  const int k_lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
  const int n = (k_hi - k_lo + 127) / 128;                      // at least 1
  const int G = p.G;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], kSoftThreads);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_free, kSoftThreads);
    mbar_init(dq_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued_k = 0, issued_v = 0;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      // (rows that no copy writes are lanes whose results are not stored)
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(2 * NSUB * 128 * G * p.QB));
#pragma unroll
      for (int sub = 0; sub < NSUB; ++sub) {
        tc::tma_load_3d(smem + C::OFF_Q + sub * kSub, &tmQ, sub * 64, kvh * G, s.q0 + t0, q_full);
        tc::tma_load_3d(smem + C::OFF_DO + sub * kSub, &tmDo, sub * 64, kvh * G, s.q0 + t0, q_full);
      }
      const uint64_t policy = policy_evict_last();   // K and V are re-read by every query block
      const int slab = p.Hkv * s.k0 + kvh * s.lk + k_lo;
      const int skip_tile = hook_skip_tile();
      for (int j = 0; j < n; ++j) {
        const int sk = j % NK, sv = j % NV;
        if (!mbar_wait(&k_empty[sk], ((j / NK) & 1) ^ 1, abort_flag, status)) break;
        issued_k = j + 1;
        if (j != skip_tile) {   // test hook: the waits for this tile run out
          mbar_arrive_expect_tx(&k_full[sk], C::TILE);
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub)
            tma_load_2d_hint(smem + C::OFF_K + sk * C::TILE + sub * kSub, &tmK, sub * 64,
                             slab + j * 128, &k_full[sk], policy);
        }
        if (!mbar_wait(&v_empty[sv], ((j / NV) & 1) ^ 1, abort_flag, status)) break;
        issued_v = j + 1;
        if (j != skip_tile) {
          mbar_arrive_expect_tx(&v_full[sv], C::TILE);
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub)
            tma_load_2d_hint(smem + C::OFF_V + sv * C::TILE + sub * kSub, &tmV, sub * 64,
                             slab + j * 128, &v_full[sv], policy);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = tc::elect_one();
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };
    constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, true);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t dod = tc::smem_desc_sw128(smem_u32(smem + C::OFF_DO), 16, 1024);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    const uint64_t kt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), kSub, 1024);   // MN-major
    auto ss = [&](uint32_t d_tm, uint64_t a, uint64_t bq, uint64_t* bar, uint64_t* bar2) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t at = static_cast<uint64_t>(kk >> 2) * (kSub >> 4) + (kk & 3) * 2;
          tc::mma_ss(d_tm, a + at, bq + at, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc::commit(bar);
        if (bar2) tc::commit(bar2);
      }
      __syncwarp();
    };
    auto issue_s = [&](int j) {
      ss(tmem + C::COL_S + 128 * (j & 1), qd, kd + static_cast<uint64_t>(j % NK) * (C::TILE >> 4),
         &s_full[j & 1], nullptr);
    };
    auto issue_dp = [&](int j) {
      ss(tmem + C::COL_DP, dod, vd + static_cast<uint64_t>(j % NV) * (C::TILE >> 4), dp_full,
         &v_empty[j % NV]);
    };
    bool ok = wwait(q_full, 0) && wwait(&k_full[0], 0);
    if (ok) {
      tc::fence_after_sync();
      issue_s(0);
      ok = wwait(&v_full[0], 0);
    }
    if (ok) {
      tc::fence_after_sync();
      issue_dp(0);
      if (n > 1) ok = wwait(&k_full[1 % NK], 0);
    }
    if (ok && n > 1) {
      tc::fence_after_sync();
      issue_s(1);
    }
    for (int j = 0; ok && j < n; ++j) {
      if (j + 1 < n) {   // dP(j + 1) overwrites dP(j)
        if (!wwait(dp_free, j & 1) || !wwait(&v_full[(j + 1) % NV], ((j + 1) / NV) & 1)) break;
        tc::fence_after_sync();
        issue_dp(j + 1);
      }
      if (!wwait(&ds_full[j & 1], (j >> 1) & 1)) break;
      tc::fence_after_sync();
      if (leader) {
        const uint64_t bk = kt + static_cast<uint64_t>(j % NK) * (C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_ts(tmem + C::COL_DQ, half_packed(tmem + C::COL_S + 128 * (j & 1), kk),
                     bk + static_cast<uint64_t>(kk) * 128u, idesc_o, j == 0 && kk == 0 ? 0u : 1u);
        tc::commit(dq_done);
        tc::commit(&k_empty[j % NK]);
      }
      __syncwarp();
      if (j + 2 < n) {   // S(j + 2) overwrites dS(j)
        if (!wwait(&k_full[(j + 2) % NK], ((j + 2) / NK) & 1) || !wwait(dq_done, j & 1)) break;
        tc::fence_after_sync();
        issue_s(j + 2);
      }
    }
    if (leader) tc::commit(drain);
    __syncwarp();
    mbar_drain(drain, 0);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int tid = threadIdx.x - 64;
    const int half = (warp - 2) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int rt = row / G;
    const bool valid = rt < nt && row < G * p.QB;
    const int h = kvh * G + (row - rt * G);
    const long long at = static_cast<long long>(s.q0 + t0 + rt) * p.Hq + h;
    const int pos = pos0 + rt;
    // keys [lo_r, hi_r) are visible to the row
    const int hi_r = valid ? (p.causal ? pos + 1 : s.lk) : 0;
    const int lo_r = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float nlse = kNegInf, ndel = 0.f;
    if (valid) {
      const float l = p.lse[at];
      if (l != kNegInf) nlse = -l * kLog2e;   // (a row that sees nothing: P = 0)
      ndel = -p.delta[at];
    }
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    const float2 nl = make_float2(nlse, nlse), nd = make_float2(ndel, ndel);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int j0 = k_lo + j * 128;
      // (rows that are not stored need no mask)
      const bool masked = j0 + 128 > s.lk || (p.causal && j0 + 127 > pos0) ||
                          (p.window > 0 && j0 + p.window <= pos0 + nt - 1);
      const int lo = lo_r - j0 - 64 * half, hi = hi_r - j0 - 64 * half;
      if (!wwait(&s_full[j & 1], (j >> 1) & 1)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t s_addr = lane_base + C::COL_S + 128 * (j & 1) + 64 * half;
      const uint32_t dp_addr = lane_base + C::COL_DP + 64 * half;
      float v[2][32], w[2][32];
      tc::tmem_ld32(s_addr, v[0]);
      tc::tmem_ld32(s_addr + 32, v[1]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = __ffma2_rn(make_float2(v[c][e], v[c][e + 1]), cc, nl);
          v[c][e] = ex2(x.x);
          v[c][e + 1] = ex2(x.y);
        }
      if (j0 + 128 > s.lk) {
        // The keys end inside the tile: the rows behind them are another head's or sequence's,
        // whose NaN would pass through zero weights. (S(j), the other reader, is done.)
        zero_rows<NSUB>(smem + C::OFF_K + (j % NK) * C::TILE, s.lk - j0, tid, kSoftThreads);
        tc::fence_proxy_async_smem();
      }
      if (!wwait(dp_full, j & 1)) { ok = false; break; }
      tc::fence_after_sync();
      tc::tmem_ld32(dp_addr, w[0]);
      tc::tmem_ld32(dp_addr + 32, w[1]);
      tc::tmem_wait_ld();
      tc::fence_before_sync();
      mbar_arrive(dp_free);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = __fmul2_rn(make_float2(v[c][e], v[c][e + 1]),
                                      __fadd2_rn(make_float2(w[c][e], w[c][e + 1]), nd));
          w[c][e] = x.x;
          w[c][e + 1] = x.y;
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) w[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(w[c][2 * e], w[c][2 * e + 1]);
        tc::tmem_st16(s_addr + 16 * c, pk);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&ds_full[j & 1]);
    }
    // ------------------------------------------------------------ epilogue
    if (ok) ok = wwait(dq_done, (n - 1) & 1);
    tc::fence_after_sync();
    // half h stores the 64-column block h
    if (half < NSUB)
      tc::store_o_rows<64>(lane_base + C::COL_DQ + 64 * half, !ok, p.sm_scale,
                           p.dq + at * D + 64 * half, valid, lane);
  }

  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    mbar_drain(q_full, 0);
    for (int i = max(0, issued_k - NK); i < issued_k; ++i) mbar_drain(&k_full[i % NK], (i / NK) & 1);
    for (int i = max(0, issued_v - NV); i < issued_v; ++i) mbar_drain(&v_full[i % NV], (i / NV) & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

template <typename Kern>
int set_smem(Kern kern, int bytes) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

template <int D>
int launch_back(const BackParams& p, cudaStream_t stream) {
  // every size is checked, and every map made, before the first launch
  const int64_t per = static_cast<int64_t>(p.Hkv) * p.batch;
  const int64_t dkv_items = (static_cast<int64_t>(p.max_kv) + 127) / 128 * per;
  const int64_t dq_items = p.nqb * per;
  if (std::max(dkv_items, dq_items) >= (int64_t{1} << 31)) {
    set_error("too many work items");
    return SINKATTN_UNSUPPORTED;
  }
  CUtensorMap tmQ, tmDo, tmK, tmV;
  const uint64_t kv_rows = static_cast<uint64_t>(p.Hkv) * p.total_k;
  // (with no query rows nothing is copied through the maps of q and dout)
  const void* q = p.total_q > 0 ? static_cast<const void*>(p.q) : p.k;
  const void* dout = p.total_q > 0 ? static_cast<const void*>(p.dout) : p.k;
  int rc = make_q_tmap(&tmQ, q, static_cast<uint64_t>(p.total_q), p.Hq, D, p.G, p.QB);
  if (rc || (rc = make_q_tmap(&tmDo, dout, static_cast<uint64_t>(p.total_q), p.Hq, D, p.G, p.QB)) ||
      (rc = make_rows_tmap(&tmK, p.k, kv_rows, D, 128, 128)) ||
      (rc = make_rows_tmap(&tmV, p.v, kv_rows, D, 128, 128)) ||
      (rc = set_smem(back_dkv_kernel<D>, DkvCfg<D>::SMEM)) ||
      (rc = set_smem(back_dq_kernel<D>, DqCfg<D>::SMEM)))
    return rc;
  const int64_t blocks = back_blocks(p.total_q, p.Hq);
  if (p.total_q > 0) {
    back_delta_kernel<D><<<dim3(static_cast<unsigned>(blocks),
                                static_cast<unsigned>((p.Hq + kDeltaHeads - 1) / kDeltaHeads)),
                           256, 0, stream>>>(p);
    if ((rc = launched("delta"))) return rc;
  }
  if (dkv_items > 0) {
    back_dkv_kernel<D><<<static_cast<unsigned>(dkv_items), kBackThreads, DkvCfg<D>::SMEM, stream>>>(
        tmQ, tmDo, tmK, tmV, p);
    if ((rc = launched("dk, dv"))) return rc;
  }
  if (p.total_q > 0 && dq_items > 0) {
    back_dq_kernel<D><<<static_cast<unsigned>(dq_items), kBackThreads, DqCfg<D>::SMEM, stream>>>(
        tmQ, tmDo, tmK, tmV, p);
    if ((rc = launched("dq"))) return rc;
  }
  if (!p.dsinks) return SINKATTN_OK;
  back_sinks_kernel<<<(p.Hq + 31) / 32, 256, 0, stream>>>(p.sink_part, static_cast<int>(blocks), p.Hq,
                                                          p.dsinks);
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
  p.sm_scale = a.sm_scale; p.scale_log2 = a.sm_scale * kLog2e;
  p.causal = a.causal;
  p.window = a.window < std::min(a.max_kv, a.total_k) ? a.window : 0;   // (one of all keys cuts nothing)
  p.QB = 128 / p.G;
  p.nqb = (a.max_q + p.QB - 1) / p.QB;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.dsinks = a.dsinks; p.delta = a.delta; p.sink_part = a.sink_part;
  p.per = back_block_tokens(a.Hq);
  return a.d == 64 ? launch_back<64>(p, stream) : launch_back<128>(p, stream);
}

SINKATTN_DEFINE_SET_HOOKS(set_hooks_prefill_back)

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
