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
// Both kernels: warp 0 stages tiles by TMA and issues the products that take P
// and dS, warp 1 those that make S and dP, then a warpgroup per stream computes P and dS, one thread per TMEM lane. A tile's way
// is a chain (product, weights, product), so two streams of tiles share an SM:
// at d 64 two CTAs of one stream, whose starts and ends overlap too; at d 128,
// where the accumulators leave no room for a second CTA, one CTA of two streams that
// take alternate tiles and add to the same accumulators.
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
  int delta_blocks, sink_blocks;
  int QB, nqb;   // query tokens of a tile of 128 rows, tiles of the longest sequence
  int GT, chunks, QB2;   // heads and tokens of a tile of 64 rows, tiles of a token
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
  constexpr int kIlp = 4;   // rows of a thread in flight
  __shared__ float term[kDeltaRows];
  const int h0 = blockIdx.y * kDeltaHeads;
  const int nh = min(kDeltaHeads, p.Hq - h0);
  const int t0 = blockIdx.x * p.per;
  const int total = min(p.total_q, p.cu_q[p.batch]);   // rows behind it are not read
  const int nt = min(p.per, total - t0);
  const int rows = max(nt, 0) * nh;
  const int c = threadIdx.x % C;
  for (int base = 0; base < rows; base += kIlp * 256 / C) {
    float s[kIlp];
    long long at[kIlp];
    uint4 x[kIlp], y[kIlp];
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      const int r = base + i * (256 / C) + threadIdx.x / C;
      x[i] = y[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        at[i] = static_cast<long long>(t0 + r / nh) * p.Hq + h0 + r % nh;
        x[i] = __ldg(reinterpret_cast<const uint4*>(p.dout + at[i] * D) + c);
        y[i] = __ldcs(reinterpret_cast<const uint4*>(p.out + at[i] * D) + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
      const int r = base + i * (256 / C) + threadIdx.x / C;
      s[i] = dot8(x[i], y[i], 0.f);
#pragma unroll
      for (int m = 1; m < C; m <<= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
      if (r < rows && c == 0) {
        if (p.dlse) s[i] -= p.dlse[at[i]];
        p.delta[at[i]] = s[i];
        // a row with no visible key and no sink has lse -inf, but then there are no sinks
        if (p.sinks) term[r] = -expf(p.sinks[h0 + r % nh] - p.lse[at[i]]) * s[i];
      }
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

// dsinks of 32 heads: the blocks' sums added in a fixed order, by all threads
// of a block. These are the first blocks of the pass that computes dq.
template <int kThreads>
__device__ __forceinline__ void reduce_sinks(const BackParams& p, int chunk) {
  constexpr int kSlices = kThreads / 32;
  __shared__ float s[kSlices][32];
  const int h = chunk * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  float x = 0.f;
  if (h < p.Hq) {
#pragma unroll 8
    for (int b = slice; b < p.delta_blocks; b += kSlices)
      x += p.sink_part[static_cast<long long>(b) * p.Hq + h];
  }
  s[slice][threadIdx.x % 32] = x;
  __syncthreads();
  if (slice != 0 || h >= p.Hq) return;
  for (int j = 1; j < kSlices; ++j) x += s[j][threadIdx.x];
  p.dsinks[h] = x;
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
// A warp's bounded wait (mbar_wait by all lanes, as one uniform branch: the
// lanes leave together, so the warp-collective TMEM accesses that follow never
// run with some of them missing).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > g_wait_limit_cycles)) {
      *abort_flag = 1;
      atomicExch(status, SINKATTN_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Zeros rows [from, to) of a tile of NSUB swizzled sub-tiles in shared memory.
template <int NSUB>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int sub_bytes, int from, int to, int tid,
                                          int threads) {
  const int n = (to - from) * 8;
  for (int u = tid; u < n * NSUB; u += threads)
    *reinterpret_cast<uint4*>(tile + (u / n) * sub_bytes + from * 128 + (u % n) * 16) =
        make_uint4(0, 0, 0, 0);
}

// Two of P's elements: 2^(s c2 - lse log2 e).
__device__ __forceinline__ void weights2(float& a, float& b, float2 cc, float2 nl) {
  const float2 x = __ffma2_rn(make_float2(a, b), cc, nl);
  a = ex2(x.x);
  b = ex2(x.y);
}

// Two of dS's elements: p (dp - delta).
__device__ __forceinline__ void scores2(float& a, float& b, float p0, float p1, float2 nd) {
  const float2 x = __fmul2_rn(make_float2(p0, p1), __fadd2_rn(make_float2(a, b), nd));
  a = x.x;
  b = x.y;
}

// 32 fp32 columns as bf16 pairs into 16 columns.
__device__ __forceinline__ void store_packed(uint32_t addr, const float (&v)[32]) {
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  tc::tmem_st16(addr, pk);
}

// dK, dV. S^T = K Q^T and dP^T = V dO^T (M 128 keys, N 64 query rows, K d; all
// from shared memory), dV += P^T dO and dK += dS^T Q (M 128 keys, N d, K 64; P^T
// and dS^T from TMEM, where they replace S^T and dP^T). Keys in the TMEM lanes
// make P^T and dS^T the MMA's A operand as they are. 64 rows a tile are what TMEM
// holds of two streams beside the accumulators.
template <int D>
struct DkvCfg {
  static constexpr int NS = D / 64;                 // streams of a CTA
  static constexpr int CTAS = 2 / NS;               // CTAs of an SM
  static constexpr int THREADS = 64 + 128 * NS;
  static constexpr int NSUB = D / 64;
  static constexpr int QT = 64;                     // query rows of a tile
  static constexpr int KSUB = 128 * 128;            // [128 keys][64 bf16], 128B-swizzled
  static constexpr int QSUB = QT * 128;
  static constexpr int K_TILE = NSUB * KSUB;
  static constexpr int Q_TILE = NSUB * QSUB;
  static constexpr int NST = 4;                     // stages of Q and dO
  static constexpr int STAGE = 2 * Q_TILE;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = K_TILE;
  static constexpr int OFF_Q = 2 * K_TILE;          // stage s: Q, then dO
  static constexpr int OFF_ROW = OFF_Q + NST * STAGE;   // [NS][2][-lse log2 e, -delta][QT]
  static constexpr int OFF_BAR = OFF_ROW + NS * 2 * 2 * QT * 4;
  static constexpr int N_BARS = 1 + NST + 6 * NS + 7;
  static constexpr int SMEM = 1024 + OFF_BAR + N_BARS * 8 + 64;
  static constexpr uint32_t COLS = 512 / CTAS;
  __host__ __device__ static constexpr uint32_t col_s(int st) { return static_cast<uint32_t>(2 * QT * st); }
  __host__ __device__ static constexpr uint32_t col_dp(int st) { return col_s(st) + QT; }
  static constexpr uint32_t COL_DV = 2 * QT * NS;
  static constexpr uint32_t COL_DK = COL_DV + D;
  static_assert(COL_DK + D <= COLS, "TMEM budget");
  static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(DkvCfg<D>::THREADS, DkvCfg<D>::CTAS)
    back_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const BackParams p) {
  using C = DkvCfg<D>;
  constexpr int NST = C::NST, NS = C::NS, NSUB = C::NSUB, QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* q_full = kv_full + 1;      // [NST]
  uint64_t* s_full = q_full + NST;     // [NS] S^T written
  uint64_t* p_full = s_full + NS;      // [NS] P^T written (128 arrivals)
  uint64_t* dp_full = p_full + NS;     // [NS] dP^T written
  uint64_t* ds_full = dp_full + NS;    // [NS] dS^T written (128 arrivals)
  uint64_t* row_full = ds_full + NS;   // [NS][2] the rows' lse and delta staged (128 arrivals)
  uint64_t* dv_done = row_full + 2 * NS;
  uint64_t* dk_done = dv_done + 2;     // [2] (and dv_done[2]) of even and odd tiles: another warp waits
  uint64_t* all_done = dk_done + 2;    // every product
  uint64_t* drain = all_done + 1;      // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
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
  // a tile is QB2 tokens times GT heads; groups of more than 64 heads come in two chunks
  const int GT = p.GT, cs = p.chunks - 1, QB2 = p.QB2;
  const int n = i1 > i0 ? (i1 - i0 + QB2 - 1) / QB2 << cs : 0;
  const int rows = GT * QB2;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < NST; ++i) mbar_init(&q_full[i], 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&dp_full[i], 1);
      mbar_init(&ds_full[i], 128);
      mbar_init(&row_full[2 * i], 128);
      mbar_init(&row_full[2 * i + 1], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dv_done[i], 1);
      mbar_init(&dk_done[i], 1);
      mbar_init(&drain[i], 1);
    }
    mbar_init(all_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (rows < QT) {   // rows that no copy writes
    for (int i = 0; i < 2 * NST; ++i)
      zero_rows<NSUB>(smem + C::OFF_Q + i * C::Q_TILE, C::QSUB, rows, QT, threadIdx.x, C::THREADS);
    tc::fence_proxy_async_smem();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;   // tiles whose copies were issued (or left out by the test hook)
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, status);
  };
  const uint64_t qt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), C::QSUB, 1024);   // MN-major
  auto stage = [&](int j) { return static_cast<uint64_t>(j % NST) * (C::STAGE >> 4); };

  if (warp == 0) {
    // ------------------------------------------ copies; dV += P^T dO and dK += dS^T Q
    const bool leader = tc::elect_one();
    const int skip_tile = hook_skip_tile();
    auto load = [&](int j) {   // of a stage that is free
      issued = j + 1;
      if (j != skip_tile && leader) {   // test hook: the waits for this tile run out
        uint8_t* to = smem + C::OFF_Q + (j % NST) * C::STAGE;
        uint64_t* bar = &q_full[j % NST];
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(2 * NSUB * 128 * rows));
        const int tok = s.q0 + i0 + (j >> cs) * QB2;
        const int head = kvh * p.G + (j & cs) * GT;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tc::tma_load_3d(to + sub * C::QSUB, &tmQ, sub * 64, head, tok, bar);
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tc::tma_load_3d(to + C::Q_TILE + sub * C::QSUB, &tmDo, sub * 64, head, tok, bar);
      }
      __syncwarp();
    };
    if (n > 0) {
      if (leader) {
        mbar_arrive_expect_tx(kv_full, 2 * C::K_TILE);
        const int slab = p.Hkv * s.k0 + kvh * s.lk + k0;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub) {
          tma_load_2d(smem + C::OFF_K + sub * C::KSUB, &tmK, sub * 64, slab, kv_full);
          tma_load_2d(smem + C::OFF_V + sub * C::KSUB, &tmV, sub * 64, slab, kv_full);
        }
      }
      for (int j = 0; j < min(NST, n); ++j) load(j);
    }
    constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, true);
    // D += A B over the tile's rows; A in TMEM
    auto ts = [&](uint32_t d_tm, uint32_t a, uint64_t bq, bool first, uint64_t* bar) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < QT / 16; ++kk)
          tc::mma_ts(d_tm, a + 8 * kk, bq + static_cast<uint64_t>(kk) * 128u, idesc_o,
                     first && kk == 0 ? 0u : 1u);
        tc::commit(bar);
      }
      __syncwarp();
    };
    for (int j = 0; j < n; ++j) {
      const int st = j % NS;
      if (!wwait(&p_full[st], (j / NS) & 1)) break;
      tc::fence_after_sync();
      ts(tmem + C::COL_DV, tmem + C::col_s(st), qt + stage(j) + (C::Q_TILE >> 4), j == 0, &dv_done[j & 1]);
      if (!wwait(&ds_full[st], (j / NS) & 1)) break;
      tc::fence_after_sync();
      ts(tmem + C::COL_DK, tmem + C::col_dp(st), qt + stage(j), j == 0, &dk_done[j & 1]);
      if (j + 1 == n) {
        if (leader) tc::commit(all_done);
        __syncwarp();
      }
      // the stage of the tile before is free when its dK, the last of its four products, is done
      if (j >= 1 && j - 1 + NST < n) {
        if (!wwait(&dk_done[(j - 1) & 1], ((j - 1) >> 1) & 1)) break;
        load(j - 1 + NST);
      }
    }
    // every MMA this warp issued has completed before the CTA frees TMEM
    if (leader) tc::commit(&drain[0]);
    __syncwarp();
    mbar_drain(&drain[0], 0);
  } else if (warp == 1) {
    // ------------------------------------------ S^T = K Q^T and dP^T = V dO^T
    // (a warp of its own: an issuer that waits for the weights of one tile would
    // leave the tensor core without the next tile's scores)
    const bool leader = tc::elect_one();
    constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, QT, false);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    // D = A B^T over d; both K-major
    auto ss = [&](uint32_t d_tm, uint64_t a, uint64_t bq, uint64_t* bar) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(d_tm, a + static_cast<uint64_t>(kk >> 2) * (C::KSUB >> 4) + (kk & 3) * 2,
                     bq + static_cast<uint64_t>(kk >> 2) * (C::QSUB >> 4) + (kk & 3) * 2, idesc_s,
                     kk > 0 ? 1u : 0u);
        tc::commit(bar);
      }
      __syncwarp();
    };
    if (n > 0 && wwait(kv_full, 0)) {
      for (int j = 0; j < n; ++j) {
        const int st = j % NS;
        // S^T(j) overwrites the P^T that dV(j - NS) reads, dP^T(j) the dS^T that dK(j - NS) reads
        if (!wwait(&q_full[j % NST], (j / NST) & 1) || (j >= NS && !wwait(&dv_done[(j - NS) & 1], ((j - NS) >> 1) & 1))) break;
        tc::fence_after_sync();
        ss(tmem + C::col_s(st), kd, qd + stage(j), &s_full[st]);
        if (j >= NS && !wwait(&dk_done[(j - NS) & 1], ((j - NS) >> 1) & 1)) break;
        tc::fence_after_sync();
        ss(tmem + C::col_dp(st), vd, qd + stage(j) + (C::Q_TILE >> 4), &dp_full[st]);
      }
    }
    if (leader) tc::commit(&drain[1]);
    __syncwarp();
    mbar_drain(&drain[1], 0);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int st = (warp - 2) >> 2;            // stream
    const int tid = threadIdx.x - 64 - 128 * st;
    const int quad = warp & 3;                 // TMEM lane quadrant this warp may access
    const int key = quad * 32 + lane;          // key of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr = lane_base + C::col_s(0) + 2 * QT * st;
    const uint32_t dp_addr = s_addr + QT;
    float* row_s = reinterpret_cast<float*>(smem + C::OFF_ROW) + st * 4 * QT;   // [2][2][QT]
    uint64_t* rows_in = row_full + 2 * st;
    // thread tid stages -lse log2(e) (tid < QT) or -delta of row tid % QT; a row outside
    // the tile, and one that sees nothing, gets lse = +inf: P = 0
    const int r = tid % QT, rt = r / GT;
    auto fetch = [&](int j) -> float {
      const int i = i0 + (j >> cs) * QB2 + rt;
      const int hh = (j & cs) * GT + (r - rt * GT);
      if (r >= rows || i >= i1 || hh >= p.G) return tid < QT ? INFINITY : 0.f;
      const long long at = static_cast<long long>(s.q0 + i) * p.Hq + kvh * p.G + hh;
      return (tid < QT ? p.lse : p.delta)[at];
    };
    // (what was fetched is first looked at here, half a tile later)
    auto put = [&](int u, float x) {   // of the stream's u-th tile
      row_s[(u & 1) * 2 * QT + tid] = tid >= QT ? -x : x == kNegInf ? kNegInf : -x * kLog2e;
      mbar_arrive(&rows_in[u & 1]);
    };
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    if (st < n) put(0, fetch(st));
    for (int j = st, u = 0; j < n; j += NS, ++u) {
      float next = 0.f;
      if (j + NS < n) next = fetch(j + NS);
      const int t0 = i0 + (j >> cs) * QB2;      // first query of the tile
      const int nt = min(QB2, i1 - t0);
      const int pos0 = off + t0;
      // columns [lo, hi) of this key's row are visible
      int lo = 0, hi = nt * GT;
      bool masked = nt < QB2;   // (the rows past rows are zeros of weight 0)
      if (p.causal) {
        masked = masked || k0 + 127 > pos0;
        lo = max(0, min(nt, k0 + key - pos0)) * GT;
      }
      if (p.window > 0) {
        masked = masked || k0 + p.window < pos0 + QB2;
        hi = max(0, min(nt, k0 + key + p.window - pos0)) * GT;
      }
      if (!wwait(&rows_in[u & 1], (u >> 1) & 1) || !wwait(&s_full[st], u & 1)) { ok = false; break; }
      tc::fence_after_sync();
      const float4* lse4 = reinterpret_cast<const float4*>(row_s + (u & 1) * 2 * QT);
      const float4* del4 = lse4 + QT / 4;
      float v[2][32];
      tc::tmem_ld32(s_addr, v[0]);
      tc::tmem_ld32(s_addr + 32, v[1]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = lse4[c * 8 + e / 4];
          weights2(v[c][e], v[c][e + 1], cc, make_float2(l.x, l.y));
          weights2(v[c][e + 2], v[c][e + 3], cc, make_float2(l.z, l.w));
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) v[c][e] = 0.f;
        }
        store_packed(s_addr + 16 * c, v[c]);
      }
      if (nt < QB2) {
        // The visible rows end inside the tile: those behind them may be another
        // sequence's, whose NaN would pass through zero weights. Both products
        // that read the tile along d are done.
        if (!wwait(&dp_full[st], u & 1)) { ok = false; break; }
        uint8_t* tile = smem + C::OFF_Q + (j % NST) * C::STAGE;
        zero_rows<NSUB>(tile, C::QSUB, nt * GT, QT, tid, 128);
        zero_rows<NSUB>(tile + C::Q_TILE, C::QSUB, nt * GT, QT, tid, 128);
        tc::fence_proxy_async_smem();
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&p_full[st]);

      if (!wwait(&dp_full[st], u & 1)) { ok = false; break; }
      tc::fence_after_sync();
      float w[2][32];
      tc::tmem_ld32(dp_addr, w[0]);
      tc::tmem_ld32(dp_addr + 32, w[1]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = del4[c * 8 + e / 4];
          scores2(w[c][e], w[c][e + 1], v[c][e], v[c][e + 1], make_float2(d.x, d.y));
          scores2(w[c][e + 2], w[c][e + 3], v[c][e + 2], v[c][e + 3], make_float2(d.z, d.w));
        }
        if (masked) {   // (0 x NaN of another row is not 0)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) w[c][e] = 0.f;
        }
        store_packed(dp_addr + 16 * c, w[c]);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&ds_full[st]);
      if (j + NS < n) put(u + 1, next);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && n > 0) ok = wwait(all_done, 0);
    tc::fence_after_sync();
    const long long row = static_cast<long long>(p.Hkv) * s.k0 + static_cast<long long>(kvh) * s.lk + k0 + key;
    // two streams: the first stores dV, the second dK
    if (NS == 1 || st == 0)
      tc::store_o_rows<D>(lane_base + C::COL_DV, !(ok && n > 0), 1.f, p.dv + row * D, key < nk, lane);
    if (NS == 1 || st == 1)
      tc::store_o_rows<D>(lane_base + C::COL_DK, !(ok && n > 0), p.sm_scale, p.dk + row * D, key < nk, lane);
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
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// dQ. S = Q K^T and dP = dO V^T (M 128 query rows, N 96 keys, K d; from shared
// memory), dQ += dS K (N d, K 96; dS from TMEM, where it replaces S). 96 keys a
// tile fill what TMEM holds of two streams beside the accumulators.
template <int D>
struct DqCfg {
  static constexpr int NS = D / 64;                 // streams of a CTA
  static constexpr int CTAS = 2 / NS;               // CTAs of an SM
  static constexpr int THREADS = 64 + 128 * NS;
  static constexpr int NSUB = D / 64;
  static constexpr int KT = 96;                     // keys of a tile
  static constexpr int KSUB = KT * 128;
  static constexpr int QSUB = 128 * 128;
  static constexpr int K_TILE = NSUB * KSUB;
  static constexpr int Q_TILE = NSUB * QSUB;
  static constexpr int NST = 3;                     // stages of K, and of V
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = Q_TILE;
  static constexpr int OFF_K = 2 * Q_TILE;
  static constexpr int OFF_V = OFF_K + NST * K_TILE;
  static constexpr int OFF_BAR = OFF_V + NST * K_TILE;
  static constexpr int N_BARS = 1 + 2 * NST + 3 * NS + 5;
  static constexpr int SMEM = 1024 + OFF_BAR + N_BARS * 8 + 64;
  static constexpr uint32_t COLS = 512 / CTAS;
  __host__ __device__ static constexpr uint32_t col_s(int st) { return static_cast<uint32_t>(2 * KT * st); }
  __host__ __device__ static constexpr uint32_t col_dp(int st) { return col_s(st) + KT; }
  static constexpr uint32_t COL_DQ = 2 * KT * NS;
  static_assert(COL_DQ + D <= COLS, "TMEM budget");
  static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(DqCfg<D>::THREADS, DqCfg<D>::CTAS)
    back_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const BackParams p) {
  using C = DqCfg<D>;
  constexpr int NST = C::NST, NS = C::NS, NSUB = C::NSUB, KT = C::KT;
  if (static_cast<int>(blockIdx.x) < p.sink_blocks) {
    reduce_sinks<C::THREADS>(p, blockIdx.x);
    return;
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;       // [NST]
  uint64_t* v_full = k_full + NST;     // [NST]
  uint64_t* s_full = v_full + NST;     // [NS] S written
  uint64_t* dp_full = s_full + NS;     // [NS] dP written
  uint64_t* ds_full = dp_full + NS;    // [NS] dS written, dP read (128 arrivals)
  uint64_t* dq_done = ds_full + NS;    // [2] of even and odd tiles (two warps wait for it)
  uint64_t* all_done = dq_done + 2;    // every product
  uint64_t* drain = all_done + 1;      // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefill_back;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // items: the last query blocks (which see the most keys) first
  const int item = static_cast<int>(blockIdx.x) - p.sink_blocks;
  const int per = p.Hkv * p.batch;
  const int qb = p.nqb - 1 - item / per;
  const int kvh = item % per % p.Hkv;
  const int b = item % per / p.Hkv;
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
  const int n = (k_hi - k_lo + KT - 1) / KT;                    // at least 1
  const int G = p.G;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&dp_full[i], 1);
      mbar_init(&ds_full[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dq_done[i], 1);
      mbar_init(&drain[i], 1);
    }
    mbar_init(all_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued_k = 0, issued_v = 0;   // tiles whose copies were issued (or left out by the test hook)
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, status);
  };
  auto stage = [&](int j) { return static_cast<uint64_t>(j % NST) * (C::K_TILE >> 4); };

  if (warp == 0) {
    // ------------------------------------------ copies; dQ += dS K
    const bool leader = tc::elect_one();
    const uint64_t policy = policy_evict_last();   // K and V are re-read by every query block
    const int slab = p.Hkv * s.k0 + kvh * s.lk + k_lo;
    const int skip_tile = hook_skip_tile();
    auto load_k = [&](int j) {   // into a stage that is free
      issued_k = j + 1;
      if (j != skip_tile && leader) {   // test hook: the waits for this tile run out
        mbar_arrive_expect_tx(&k_full[j % NST], C::K_TILE);
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tma_load_2d_hint(smem + C::OFF_K + (j % NST) * C::K_TILE + sub * C::KSUB, &tmK, sub * 64,
                           slab + j * KT, &k_full[j % NST], policy);
      }
      __syncwarp();
    };
    auto load_v = [&](int j) {
      issued_v = j + 1;
      if (j != skip_tile && leader) {
        mbar_arrive_expect_tx(&v_full[j % NST], C::K_TILE);
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tma_load_2d_hint(smem + C::OFF_V + (j % NST) * C::K_TILE + sub * C::KSUB, &tmV, sub * 64,
                           slab + j * KT, &v_full[j % NST], policy);
      }
      __syncwarp();
    };
    if (leader) {
      // (rows that no copy writes are lanes whose results are not stored)
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(2 * NSUB * 128 * G * p.QB));
#pragma unroll
      for (int sub = 0; sub < NSUB; ++sub) {
        tc::tma_load_3d(smem + C::OFF_Q + sub * C::QSUB, &tmQ, sub * 64, kvh * G, s.q0 + t0, q_full);
        tc::tma_load_3d(smem + C::OFF_DO + sub * C::QSUB, &tmDo, sub * 64, kvh * G, s.q0 + t0, q_full);
      }
    }
    for (int j = 0; j < min(NST, n); ++j) {
      load_k(j);
      load_v(j);
    }
    constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, true);
    const uint64_t kt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), C::KSUB, 1024);   // MN-major
    for (int j = 0; j < n; ++j) {
      const int st = j % NS;
      if (!wwait(&ds_full[st], (j / NS) & 1)) break;
      tc::fence_after_sync();
      if (leader) {
        const uint64_t bk = kt + stage(j);
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          tc::mma_ts(tmem + C::COL_DQ, tmem + C::col_s(st) + 8 * kk,
                     bk + static_cast<uint64_t>(kk) * 128u, idesc_o, j == 0 && kk == 0 ? 0u : 1u);
        tc::commit(&dq_done[j & 1]);
        if (j + 1 == n) tc::commit(all_done);
      }
      __syncwarp();
      // dS(j) came after dP(j), the only product that reads V's tile j
      if (j + NST < n) load_v(j + NST);
      if (j >= 1 && j - 1 + NST < n) {
        if (!wwait(&dq_done[(j - 1) & 1], ((j - 1) >> 1) & 1)) break;
        load_k(j - 1 + NST);
      }
    }
    // every MMA this warp issued has completed before the CTA frees TMEM
    if (leader) tc::commit(&drain[0]);
    __syncwarp();
    mbar_drain(&drain[0], 0);
  } else if (warp == 1) {
    // ------------------------------------------ S = Q K^T and dP = dO V^T
    const bool leader = tc::elect_one();
    constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, KT, false);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t dod = tc::smem_desc_sw128(smem_u32(smem + C::OFF_DO), 16, 1024);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    auto ss = [&](uint32_t d_tm, uint64_t a, uint64_t bk, uint64_t* bar) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(d_tm, a + static_cast<uint64_t>(kk >> 2) * (C::QSUB >> 4) + (kk & 3) * 2,
                     bk + static_cast<uint64_t>(kk >> 2) * (C::KSUB >> 4) + (kk & 3) * 2, idesc_s,
                     kk > 0 ? 1u : 0u);
        tc::commit(bar);
      }
      __syncwarp();
    };
    if (wwait(q_full, 0)) {
      for (int j = 0; j < n; ++j) {
        const int st = j % NS;
        // dP(j) overwrites a dP that has been read when its dS is there, S(j)
        // the dS(j - NS) that dQ reads: dP runs while that ends
        if (!wwait(&v_full[j % NST], (j / NST) & 1) ||
            (j >= NS && !wwait(&ds_full[st], (j / NS - 1) & 1))) break;
        tc::fence_after_sync();
        ss(tmem + C::col_dp(st), dod, vd + stage(j), &dp_full[st]);
        if (!wwait(&k_full[j % NST], (j / NST) & 1) ||
            (j >= NS && !wwait(&dq_done[(j - NS) & 1], ((j - NS) >> 1) & 1))) break;
        tc::fence_after_sync();
        ss(tmem + C::col_s(st), qd, kd + stage(j), &s_full[st]);
      }
    }
    if (leader) tc::commit(&drain[1]);
    __syncwarp();
    mbar_drain(&drain[1], 0);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int st = (warp - 2) >> 2;            // stream
    const int tid = threadIdx.x - 64 - 128 * st;
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
    const uint32_t s_addr = lane_base + C::col_s(0) + 2 * KT * st;
    const uint32_t dp_addr = s_addr + KT;
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    const float2 nl = make_float2(nlse, nlse), nd = make_float2(ndel, ndel);
    bool ok = true;
    for (int j = st, u = 0; j < n; j += NS, ++u) {
      const int j0 = k_lo + j * KT;
      // (rows that are not stored need no mask)
      const bool masked = j0 + KT > s.lk || (p.causal && j0 + KT - 1 > pos0) ||
                          (p.window > 0 && j0 + p.window <= pos0 + nt - 1);
      const int lo = lo_r - j0, hi = hi_r - j0;
      if (!wwait(&s_full[st], u & 1)) { ok = false; break; }
      tc::fence_after_sync();
      float v[KT / 32][32];
#pragma unroll
      for (int c = 0; c < KT / 32; ++c) tc::tmem_ld32(s_addr + 32 * c, v[c]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < KT / 32; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) weights2(v[c][e], v[c][e + 1], cc, nl);
      if (j0 + KT > s.lk) {
        // The keys end inside the tile: the rows behind them are another head's or sequence's,
        // whose NaN would pass through zero weights. (S(j), the other reader, is done.)
        zero_rows<NSUB>(smem + C::OFF_K + (j % NST) * C::K_TILE, C::KSUB, s.lk - j0, KT, tid, 128);
        tc::fence_proxy_async_smem();
      }
      if (!wwait(&dp_full[st], u & 1)) { ok = false; break; }
      tc::fence_after_sync();
#pragma unroll
      for (int c = 0; c < KT / 32; ++c) {
        float w[32];
        tc::tmem_ld32(dp_addr + 32 * c, w);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2) scores2(w[e], w[e + 1], v[c][e], v[c][e + 1], nd);
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < lo || c * 32 + e >= hi) w[e] = 0.f;
        }
        store_packed(s_addr + 16 * c, w);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&ds_full[st]);
    }
    // ------------------------------------------------------------ epilogue
    if (ok) ok = wwait(all_done, 0);
    tc::fence_after_sync();
    // stream s stores the 64-column block s
    tc::store_o_rows<64>(lane_base + C::COL_DQ + 64 * st, !ok, p.sm_scale, p.dq + at * D + 64 * st,
                         valid, lane);
  }

  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    mbar_drain(q_full, 0);
    for (int i = max(0, issued_k - NST); i < issued_k; ++i) mbar_drain(&k_full[i % NST], (i / NST) & 1);
    for (int i = max(0, issued_v - NST); i < issued_v; ++i) mbar_drain(&v_full[i % NST], (i / NST) & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

int set_smem(cudaError_t e) {
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

template <int D>
int launch_back(BackParams& p, cudaStream_t stream) {
  using KV = DkvCfg<D>;
  using DQ = DqCfg<D>;
  // every size is checked, and every map made, before the first launch
  const int64_t per = static_cast<int64_t>(p.Hkv) * p.batch;
  const int64_t dkv_items = (static_cast<int64_t>(p.max_kv) + 127) / 128 * per;
  p.sink_blocks = p.dsinks ? (p.Hq + 31) / 32 : 0;
  const int64_t dq_items = p.nqb * per + p.sink_blocks;
  if (std::max(dkv_items, dq_items) >= (int64_t{1} << 31)) {
    set_error("too many work items");
    return SINKATTN_UNSUPPORTED;
  }
  CUtensorMap tmQ, tmDo, tmQ2, tmDo2, tmK, tmV, tmK2, tmV2;
  const uint64_t kv_rows = static_cast<uint64_t>(p.Hkv) * p.total_k;
  const uint64_t q_rows = static_cast<uint64_t>(p.total_q);
  // (with no query rows nothing is copied through the maps of q and dout)
  const void* q = p.total_q > 0 ? static_cast<const void*>(p.q) : p.k;
  const void* dout = p.total_q > 0 ? static_cast<const void*>(p.dout) : p.k;
  int rc;
  if ((rc = make_q_tmap(&tmQ, q, q_rows, p.Hq, D, p.G, p.QB)) ||
      (rc = make_q_tmap(&tmDo, dout, q_rows, p.Hq, D, p.G, p.QB)) ||
      (rc = make_q_tmap(&tmQ2, q, q_rows, p.Hq, D, p.GT, p.QB2)) ||
      (rc = make_q_tmap(&tmDo2, dout, q_rows, p.Hq, D, p.GT, p.QB2)) ||
      (rc = make_rows_tmap(&tmK, p.k, kv_rows, D, DQ::KT, 128)) ||
      (rc = make_rows_tmap(&tmV, p.v, kv_rows, D, DQ::KT, 128)) ||
      (rc = make_rows_tmap(&tmK2, p.k, kv_rows, D, 128, 128)) ||
      (rc = make_rows_tmap(&tmV2, p.v, kv_rows, D, 128, 128)) ||
      (rc = set_smem(set_chained_smem(back_dkv_kernel<D>, KV::SMEM))) ||
      (rc = set_smem(set_chained_smem(back_dq_kernel<D>, DQ::SMEM))))
    return rc;
  if (p.delta_blocks > 0) {
    back_delta_kernel<D><<<dim3(static_cast<unsigned>(p.delta_blocks),
                                static_cast<unsigned>((p.Hq + kDeltaHeads - 1) / kDeltaHeads)),
                           256, 0, stream>>>(p);
    if ((rc = launched("delta"))) return rc;
  }
  if (dkv_items > 0) {
    back_dkv_kernel<D><<<static_cast<unsigned>(dkv_items), KV::THREADS, KV::SMEM, stream>>>(
        tmQ2, tmDo2, tmK2, tmV2, p);
    if ((rc = launched("dk, dv"))) return rc;
  }
  if (dq_items > 0) {
    back_dq_kernel<D><<<static_cast<unsigned>(dq_items), DQ::THREADS, DQ::SMEM, stream>>>(
        tmQ, tmDo, tmK, tmV, p);
    return launched("dq");
  }
  return SINKATTN_OK;
}

}  // namespace

// Rows of a block: 1024 where that leaves every SM several blocks, else 256.
int back_block_tokens(int32_t total_q, int32_t Hq) {
  const bool many = static_cast<int64_t>(total_q) * Hq >= int64_t{4 * 152} * kDeltaRows;
  return std::max(1, (many ? kDeltaRows : kDeltaRows / 4) / std::min<int32_t>(Hq, kDeltaHeads));
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
  p.per = back_block_tokens(a.total_q, a.Hq);
  p.delta_blocks = static_cast<int>(back_blocks(a.total_q, a.Hq));
  p.chunks = p.G > 64 ? 2 : 1;
  p.GT = (p.G + p.chunks - 1) / p.chunks;
  p.QB2 = 64 / p.GT;
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
