// Backward pass of the varlen prefill with a per-head softmax sink (rules:
// sinkattn.h) on the 5th-generation tensor cores. With P = exp(l - lse) over
// the visible keys and delta = dout . out - dlse, dS = P (dout v^T - delta):
// dq = c dS k, dk = c dS^T q, dv = P^T dout, dsink = -sum exp(s - lse) delta.
//
// Two passes. back_dq_kernel: one CTA holds 128 query rows (tokens x the heads of a
// group), computes their delta and walks over the keys they see;
// back_dkv_kernel: one CTA holds 128 keys of a KV head and walks over the query
// rows that see them; its last blocks sum the sinks' gradients. P and
// dS are computed in both, seven products a tile pair instead of five: no sum
// crosses CTAs, so there are no atomics (whose order would change the results),
// no fp32 buffer of dq in memory, and the group's heads add up in the
// accumulators.
//
// Both kernels: warp 0 stages tiles by TMA, warp 1 issues the product that makes
// S, warp 2 that of dP, warp 3 those that take P and dS, and groups of eight or sixteen
// warps compute these, one thread per TMEM lane and 32 columns. A product is
// seen by those who wait for it about 500 cycles after the tensor core has
// done it, and a tile goes through three of them in turn. So tiles are small (64 or 128
// columns), and TMEM holds as many of them on their way as fit beside the
// accumulators; each kind of product has a warp of its own, because an issuing
// warp's waits, MMAs and commits take 100 to 250 cycles each, one after the other.
// P and dS are rounded to bf16 for the products that take them; P enters dS
// unrounded. Every wait is bounded; on a timeout the CTA records
// SINKATTN_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
//
// Measured (full causal): 10,168 tokens of 64/8 heads of 64 in four sequences 759 us (837
// TFLOP/s of the formulas' five products); 2 x 6000 tokens of 64/4 heads of 128 2.73 to 2.89 ms
// (1.02 to 1.08 PFLOP/s), as the power limit allows: calls in a graph, one behind the other.
// Each pass alone, under the profiler: dq 346 us and dk, dv 400 (71 and 64 % of the tensor core's
// time); 1133 and 1525 us (89 and 95 %). What bounds them: at d 128 the tensor core, where
// an MMA of 64 columns takes as long as one of 128 (a tile of 128 columns has no
// room for a second buffer); at d 64 the chain of a tile's products and of P and dS.
// dq in tiles of 128 keys, one CTA an SM, took 450 us at d 64 and 1240 at d 128
// (42 and 66 % of the tensor core's time).
#include <algorithm>
#include <type_traits>

#include "chain.cuh"
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
  float *dsinks, *nlse, *ndelta, *sink_part;   // (workspace: [total_q, Hq] -lse log2 e, -delta)
  int* sink_count;                   // (workspace) blocks that have left their sums
  int sink_tokens, sink_blocks;      // tokens of a block that sums the sinks' gradients, these blocks
  int dkv_items;
  int QB, nqb;   // query tokens of a tile of 128 rows, tiles of the longest sequence
  int run, nrun; // tiles of a CTA of the pass of dq, CTAs of the longest sequence
  int krun;      // tiles of a CTA of the pass of dk and dv
  int GT, chunks, QB2;   // heads and tokens of a tile of the dk, dv pass, tiles of a token
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

// dsinks_h = sum over the rows of e^{s_h - lse} (-delta), of p.sink_tokens tokens a block, by all threads
// of it (s: shared memory, 32 words a warp and one more). Each block leaves its
// sums in p.sink_part; the one that comes last, whichever it is, adds them up in their order.
template <int kThreads>
__device__ __forceinline__ void sum_sinks(const BackParams& p, int blk, float (*s)[32]) {
  constexpr int kSlices = kThreads / 32;
  const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
  int* last = reinterpret_cast<int*>(s + kSlices);
  // (rows outside the sequences have no gradient; where the bound says that there are no
  // queries, the pass of dq, which leaves their numbers, has not run)
  const int t0 = max(blk * p.sink_tokens, p.cu_q[0]);
  const int end = p.max_q > 0 ? max(0, min(p.total_q, p.cu_q[p.batch])) : 0;
  const int t1 = min(end - blk * p.sink_tokens, p.sink_tokens) + blk * p.sink_tokens;
  auto reduce = [&](int h, float x, float* to) {   // over the slices
    s[slice][lane] = x;
    __syncthreads();
    if (slice == 0 && h < p.Hq) {
      for (int j = 1; j < kSlices; ++j) x += s[j][lane];
      to[h] = x;
    }
    __syncthreads();
  };
  for (int h = lane; h < p.Hq + lane; h += 32) {
    float x = 0.f;
    if (h < p.Hq) {
      const float sink = p.sinks[h] * kLog2e;
#pragma unroll 4
      for (int t = t0 + slice; t < t1; t += kSlices) {
        const long long at = static_cast<long long>(t) * p.Hq + h;
        x = fmaf(exp2f(sink + __ldcg(&p.nlse[at])), __ldcg(&p.ndelta[at]), x);
      }
    }
    reduce(h, x, p.sink_blocks == 1 ? p.dsinks : p.sink_part + static_cast<long long>(blk) * p.Hq);
  }
  if (p.sink_blocks == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *last = atomicAdd(p.sink_count, 1) == p.sink_blocks - 1;
  __syncthreads();
  if (!*last) return;
  __threadfence();
  for (int h = lane; h < p.Hq + lane; h += 32) {
    float x = 0.f;
    if (h < p.Hq) {
#pragma unroll 8
      for (int b = slice; b < p.sink_blocks; b += kSlices)
        x += __ldcg(&p.sink_part[static_cast<long long>(b) * p.Hq + h]);
    }
    reduce(h, x, p.dsinks);
  }
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
// One try of a wait, suspended for up to `ns` while the phase is not complete.
__device__ __forceinline__ bool try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// Between two tries of a wait that began at `since` (0: now): -1 where it is to be
// given up, because another warp has, or because its time is over, else when it
// began. The time is for a part that has failed, so it does not begin while the
// launch before still runs: what dk and dv wait for in the end may be that. (Here it
// costs nothing when the first try succeeds; before the waits, in every warp, the
// smallest call took 11.3 us instead of 10.7.) Out of line: the loops of the issuing
// warps are short, and what they fetch of their instructions is what they cost.
__device__ __noinline__ long long give_up(long long since, volatile int* abort_flag, int* status) {
  if (*abort_flag) return -1;
  if (since == 0) {
    grid_dependency_wait();
    return clock64();
  }
  const long long now = clock64();
  if (now - since <= g_wait_limit_cycles) return since;
  *abort_flag = 1;
  atomicExch(status, SINKATTN_TIMEOUT);
  return -1;
}

// A warp's bounded wait, as one uniform branch: the lanes leave together, so the
// warp-collective TMEM accesses that follow never run with some of them missing.
// A try is suspended for up to 20 us, because a warp that polls takes issue slots
// from the ones that compute.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  long long since = 0;
  while (!__all_sync(0xffffffffu, try_wait_for(bar, parity, 20000u)))
    if (__any_sync(0xffffffffu, (since = give_up(since, abort_flag, status)) < 0)) return false;
  return true;
}
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           volatile int* abort_flag, int* status) {
  long long since = 0;
  while (true) {
    const bool ra = try_wait_for(a, pa, 20000u), rb = try_wait_for(b, pb, 20000u);
    if (__all_sync(0xffffffffu, ra && rb)) return true;
    if (__any_sync(0xffffffffu, (since = give_up(since, abort_flag, status)) < 0)) return false;
  }
}
__device__ __forceinline__ bool warp_wait3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           uint64_t* c, uint32_t pc, volatile int* abort_flag,
                                           int* status) {
  long long since = 0;
  while (true) {
    const bool ra = try_wait_for(a, pa, 20000u), rb = try_wait_for(b, pb, 20000u),
               rc = try_wait_for(c, pc, 20000u);
    if (__all_sync(0xffffffffu, ra && rb && rc)) return true;
    if (__any_sync(0xffffffffu, (since = give_up(since, abort_flag, status)) < 0)) return false;
  }
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

// Four bytes from global to shared memory, asynchronously; an arrival on a barrier
// when the thread's copies so far have landed; the end of all of them.
__device__ __forceinline__ void copy4_async(float* to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

// The A operand of a TS product: bf16 pairs that replaced fp32 columns, each 16
// elements in 8 of their 16 columns. K step kk covers elements 16 kk ...
__device__ __forceinline__ uint32_t packed_step(uint32_t base, int kk) {
  return base + static_cast<uint32_t>(16 * kk);
}

// The products, by one lane of a warp. ss: D = A B^T over d, both in shared memory
// and K-major, in 64-column sub-tiles of a_sub and b_sub bytes. ts: D += A B over
// STEPS steps of 16 rows of B; A in TMEM (packed_step), B MN-major.
template <int D, int N>
__device__ __forceinline__ void issue_ss(bool leader, uint32_t d_tm, uint64_t a, uint64_t b, int a_sub,
                                         int b_sub) {
  if (!leader) return;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    tc::mma_ss(d_tm, a + static_cast<uint64_t>(kk >> 2) * (a_sub >> 4) + (kk & 3) * 2,
               b + static_cast<uint64_t>(kk >> 2) * (b_sub >> 4) + (kk & 3) * 2,
               tc::idesc_bf16_f32(128, N, false), kk > 0 ? 1u : 0u);
}
template <int D, int STEPS>
__device__ __forceinline__ void issue_ts(bool leader, uint32_t d_tm, uint32_t a, uint64_t b, bool first) {
  if (!leader) return;
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk)
    tc::mma_ts(d_tm, packed_step(a, kk), b + static_cast<uint64_t>(kk) * 128u,
               tc::idesc_bf16_f32(128, D, true), first && kk == 0 ? 0u : 1u);
}

// 16 fp32 columns as bf16 pairs into 8 columns.
__device__ __forceinline__ void store_packed(uint32_t addr, const float (&v)[16]) {
  uint32_t pk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  tc::tmem_st8(addr, pk);
}

__device__ __forceinline__ void store_zeros(uint32_t addr) {   // 8 columns
  const uint32_t zero[8] = {};
  tc::tmem_st8(addr, zero);
}

// Of a warp's 32 x 32 square of a tile that the mask cuts, 0 of the columns before lo
// and from hi on are visible to a lane. The diagonals cut few of a tile's squares: the
// others take no comparisons, or no arithmetic at all.
enum Seen { kAll, kSome, kNone };
__device__ __forceinline__ Seen seen_by_warp(bool masked, int lo, int hi) {
  if (!masked) return kAll;   // (uniform over the warp)
  if (__all_sync(0xffffffffu, lo <= 0 && hi >= 32)) return kAll;
  return __any_sync(0xffffffffu, max(lo, 0) < min(hi, 32)) ? kSome : kNone;
}

// dK, dV. S^T = K Q^T and dP^T = V dO^T (M 128 keys, N QT query rows, K d; all from
// shared memory), dV += P^T dO and dK += dS^T Q (M 128 keys, N d, K QT; P^T and
// dS^T from TMEM, where both replace S^T). Keys in the TMEM lanes make P^T and
// dS^T the MMA's A operand as they are. dP^T is free as soon as it has been read.
// A tile is QB2 tokens times GT heads; groups of more heads than it has rows come
// in two chunks.
template <int D>
struct DkvCfg {
  static constexpr int SOFT0 = 4;                   // first warp of P and dS
  static constexpr int NG = D / 64;                 // groups of warps, which take alternate tiles
  static constexpr int QT = D == 64 ? 128 : 64;     // query rows of a tile
  static constexpr int GROUP = 128 * QT / 32;       // threads of a group
  static constexpr int THREADS = SOFT0 * 32 + NG * GROUP;
  static constexpr int NSUB = D / 64;
  static constexpr int KSUB = 128 * 128;            // [128 keys][64 bf16], 128B-swizzled
  static constexpr int QSUB = QT * 128;
  static constexpr int K_TILE = NSUB * KSUB;
  static constexpr int Q_TILE = NSUB * QSUB;
  static constexpr int NSB = D == 64 ? 2 : 3;       // S^T buffers
  static constexpr int NB = D == 64 ? 2 : 6;        // tiles after which buffer and group repeat
  static constexpr int NQ = D == 64 ? 5 : 6;        // stages of Q
  static constexpr int ND = 4;                      // stages of dO, which is held for a shorter time
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = K_TILE;
  static constexpr int OFF_Q = 2 * K_TILE;
  static constexpr int OFF_DO = OFF_Q + NQ * Q_TILE;
  static constexpr int NR = 4;                      // slots of the rows' lse and delta
  static constexpr int OFF_ROW = OFF_DO + ND * Q_TILE;   // [NR][-lse log2 e, -delta][QT]
  static constexpr int OFF_BAR = OFF_ROW + NR * 2 * QT * 4;
  static constexpr int N_BARS = 2 + 2 * NQ + 2 * ND + NB + NR + 2 * NSB + 2 + 1 + 2 + 3;
  static_assert(NR % NG == 0 && NR <= ND && ND <= NQ, "order of the copies");
  static constexpr int SMEM = OFF_BAR + N_BARS * 8 + 16;
  static constexpr uint32_t COL_S = 0;
  static constexpr uint32_t COL_DP = QT * NSB;
  static constexpr uint32_t COL_DV = COL_DP + QT;
  static constexpr uint32_t COL_DK = COL_DV + D;
  static_assert(COL_DK + D <= 512, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(DkvCfg<D>::THREADS, 1)
    back_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const BackParams p) {
  using C = DkvCfg<D>;
  constexpr int NQ = C::NQ, ND = C::ND, NSB = C::NSB, NG = C::NG, NB = C::NB, NR = C::NR, NSUB = C::NSUB,
                QT = C::QT;
  extern __shared__ __align__(1024) uint8_t smem[];   // (swizzled tiles start on 1024 bytes)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + 1;    // S^T and dP^T of the key tile done
  uint64_t* q_full = kv_empty + 1;     // [NQ]
  uint64_t* q_empty = q_full + NQ;     // [NQ] dK, the last that reads the stage, done
  uint64_t* do_full = q_empty + NQ;    // [ND]
  uint64_t* do_empty = do_full + ND;   // [ND] dP^T and dV done
  uint64_t* s_full = do_empty + ND;    // [NB] S^T written
  uint64_t* row_full = s_full + NB;    // [NR] the rows' lse and delta staged (64 arrivals)
  uint64_t* s_free = row_full + NR;    // [NSB] the P^T and dS^T in it read
  uint64_t* p_full = s_free + NSB;     // [NSB] P^T and dS^T written (the group's arrivals)
  uint64_t* dp_full = p_full + NSB;    // [2] of even and odd tiles: dP^T written
  uint64_t* dp_free = dp_full + 2;     // dP^T read (the group's arrivals)
  uint64_t* dkv_full = dp_free + 1;    // a key tile's dV and dK done
  uint64_t* dkv_free = dkv_full + 1;   // and read
  uint64_t* drain = dkv_free + 1;      // [3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefill_back;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (static_cast<int>(blockIdx.x) >= p.dkv_items) {   // (the last blocks: they fill the SMs that the others leave)
    grid_dependency_wait();
    sum_sinks<C::THREADS>(p, blockIdx.x - p.dkv_items, reinterpret_cast<float(*)[32]>(smem));
    return;
  }
  // A CTA's key tiles: m of them; the first ones (which the most queries see) of all
  // sequences and KV heads are those of the first CTAs.
  const int per = p.Hkv * p.batch;
  const int kt = static_cast<int>(blockIdx.x) / per * p.krun;
  const int kvh = static_cast<int>(blockIdx.x) % per % p.Hkv;
  const int b = static_cast<int>(blockIdx.x) % per / p.Hkv;
  const Seq s = load_seq(p, b);
  if (!s.ok && threadIdx.x == 0) atomicExch(status, SINKATTN_BAD_LENGTHS);
  const int m = s.ok ? min(p.krun, (s.lk - 128 * kt + 127) / 128) : 0;
  if (m <= 0) {   // uniform over the CTA, before any barrier or TMEM use
    grid_dependency_wait();    // (this launch ends after the one before)
    return;
  }
  const int off = s.lk - s.lq;   // position of query 0
  const int GT = p.GT, cs = p.chunks - 1, QB2 = p.QB2, rows = GT * QB2;
  struct Tile {
    int k0, nk;        // its keys
    int i0, i1, n;     // queries [i0, i1) see some of them, in n tiles (which may be 0)
  };
  auto tile = [&](int i) {
    Tile t;
    t.k0 = 128 * (kt + i);
    t.nk = min(128, s.lk - t.k0);
    t.i0 = p.causal ? max(0, t.k0 - off) : 0;
    t.i1 = p.window > 0 ? max(0, min(s.lq, t.k0 + t.nk - 1 + p.window - off)) : s.lq;
    t.n = t.i1 > t.i0 ? (t.i1 - t.i0 + QB2 - 1) / QB2 << cs : 0;
    return t;
  };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 2);
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < NR; ++i) mbar_init(&row_full[i], 64);
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&s_free[i], 1);
      mbar_init(&p_full[i], C::GROUP);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&dp_full[i], 1);
    mbar_init(dp_free, C::GROUP);
    mbar_init(dkv_full, 1);
    mbar_init(dkv_free, 2 * NSUB * 128);
    for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (rows < QT) {   // rows that no copy writes
    for (int i = 0; i < NQ + ND; ++i)
      zero_rows<NSUB>(smem + C::OFF_Q + i * C::Q_TILE, C::QSUB, rows, QT, threadIdx.x, C::THREADS);
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
  int issued_kv = 0, issued_q = 0, issued_do = 0;   // tiles whose copies were issued (or left out by the test hook)
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, status);
  };
  auto wwait2 = [&](uint64_t* x, uint32_t px, uint64_t* y, uint32_t py) -> bool {
    return warp_wait2(x, px, y, py, abort_flag, status);
  };
  const bool leader = tc::elect_one();
  // an issuing warp's end: every MMA of it has completed before the CTA frees TMEM
  auto finish = [&](uint64_t* bar) {
    if (leader) tc::commit(bar);
    __syncwarp();
    mbar_drain(bar, 0);
  };
  const uint32_t tile16 = C::Q_TILE >> 4;   // a stage, in descriptor units

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    const int skip_tile = hook_skip_tile();
    // Tile j of the CTA, tile x of its key tile t, into a free stage.
    auto load = [&](const CUtensorMap* map, const Tile& t, int j, int x, uint8_t* to, uint64_t* bar) {
      if (j != skip_tile && leader) {   // test hook: the waits for this tile run out
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(NSUB * 128 * rows));
        const int tok = s.q0 + t.i0 + (x >> cs) * QB2, head = kvh * p.G + (x & cs) * GT;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tc::tma_load_3d(to + sub * C::QSUB, map, sub * 64, head, tok, bar);
      }
      __syncwarp();
    };
    // -lse log2(e) and -delta of a tile's rows, QT / 32 a lane. A row outside the tile
    // gets lse = +inf: P = 0. Both kinds of writes arrive, the copies when they have landed.
    constexpr int kRows = QT / 32;
    int rt[kRows], rh[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      rt[e] = (lane + 32 * e) / GT;
      rh[e] = (lane + 32 * e) % GT;
    }
    auto load_rows = [&](const Tile& t, int j, int x) {
      float* to = reinterpret_cast<float*>(smem + C::OFF_ROW) + j % NR * 2 * QT + lane;
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int i = t.i0 + (x >> cs) * QB2 + rt[e], h = (x & cs) * GT + rh[e];
        if (lane + 32 * e < rows && i < t.i1 && h < p.G) {
          const long long at = static_cast<long long>(s.q0 + i) * p.Hq + kvh * p.G + h;
          copy4_async(to + 32 * e, p.nlse + at);
          copy4_async(to + QT + 32 * e, p.ndelta + at);
        } else {
          to[32 * e] = kNegInf;
          to[QT + 32 * e] = 0.f;
        }
      }
      mbar_arrive(&row_full[j % NR]);
      arrive_after_copies(&row_full[j % NR]);
    };
    // Q of a key tile's tile x, and the tiles whose dO and rows take the places of
    // the same tile x - NQ. The first tiles' copies need nothing of the launch before this one, the rows do.
    bool ok = true;
    for (int i = 0, g = 0; i < m && ok; ++i) {   // g: tiles before
      const Tile t = tile(i);
      if (t.n == 0) continue;
      if (issued_kv > 0 && !wwait(kv_empty, (issued_kv - 1) & 1)) break;
      ++issued_kv;
      if (leader) {
        mbar_arrive_expect_tx(kv_full, 2 * C::K_TILE);
        const int slab = p.Hkv * s.k0 + kvh * s.lk + t.k0;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub) {
          tma_load_2d(smem + C::OFF_K + sub * C::KSUB, &tmK, sub * 64, slab, kv_full);
          tma_load_2d(smem + C::OFF_V + sub * C::KSUB, &tmV, sub * 64, slab, kv_full);
        }
      }
      __syncwarp();
      for (int x = 0; x < t.n + NQ - NR; ++x) {
        const int j = g + x;
        if (j >= NQ && !(ok = wwait(&q_empty[j % NQ], (j / NQ - 1) & 1))) break;
        if (x < t.n) {
          issued_q = j + 1;
          load(&tmQ, t, j, x, smem + C::OFF_Q + j % NQ * C::Q_TILE, &q_full[j % NQ]);
        }
        const int y = x - (NQ - ND), z = x - (NQ - NR);
        if (y >= 0 && y < t.n) {
          const int jy = g + y;
          if (jy >= ND && !(ok = wwait(&do_empty[jy % ND], (jy / ND - 1) & 1))) break;
          issued_do = jy + 1;
          load(&tmDo, t, jy, y, smem + C::OFF_DO + jy % ND * C::Q_TILE, &do_full[jy % ND]);
        }
        if (z >= 0) {
          if (g + z == 0) grid_dependency_wait();
          load_rows(t, g + z, z);
        }
      }
      g += t.n;
    }
    grid_dependency_wait();   // (without rows too: this launch ends after the one before)
    wait_copies();   // (before the CTA's shared memory goes away)
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S^T = K Q^T
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    bool ok = true;
    for (int i = 0, j = 0, c = 0; i < m && ok; ++i) {   // c: key tiles with work before
      const int end_j = j + tile(i).n;
      if (j == end_j) continue;
      if (!wwait(kv_full, c & 1)) break;
      for (; j < end_j; ++j) {
        const int sb = j % NSB;
        ok = j < NSB ? wwait(&q_full[j % NQ], 0)
                     : wwait2(&s_free[sb], (j / NSB - 1) & 1, &q_full[j % NQ], j / NQ & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_ss<D, QT>(leader, tmem + C::COL_S + QT * sb, kd, qd + j % NQ * tile16, C::KSUB, C::QSUB);
        if (leader) tc::commit(&s_full[j % NB]);
        __syncwarp();
      }
      if (leader) tc::commit(kv_empty);
      __syncwarp();
      ++c;
    }
    finish(&drain[0]);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- dP^T = V dO^T
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    const uint64_t dod = tc::smem_desc_sw128(smem_u32(smem + C::OFF_DO), 16, 1024);
    bool ok = true;
    for (int i = 0, j = 0, c = 0; i < m && ok; ++i) {
      const int end_j = j + tile(i).n;
      if (j == end_j) continue;
      if (!wwait(kv_full, c & 1)) break;
      for (; j < end_j; ++j) {
        ok = j < 1 ? wwait(&do_full[0], 0) : wwait2(dp_free, (j - 1) & 1, &do_full[j % ND], j / ND & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_ss<D, QT>(leader, tmem + C::COL_DP, vd, dod + j % ND * tile16, C::KSUB, C::QSUB);
        if (leader) tc::commit(&dp_full[j & 1]);
        __syncwarp();
      }
      if (leader) tc::commit(kv_empty);
      __syncwarp();
      ++c;
    }
    finish(&drain[1]);
  } else if (warp == 3) {
    // ------------------------------------------ dV += P^T dO and dK += dS^T Q
    const uint64_t dot = tc::smem_desc_sw128(smem_u32(smem + C::OFF_DO), C::QSUB, 1024);   // MN-major
    const uint64_t qt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), C::QSUB, 1024);
    bool ok = true;
    for (int i = 0, j = 0, c = 0; i < m && ok; ++i) {
      const int first = j, end_j = j + tile(i).n;
      if (j == end_j) continue;
      if (c > 0 && !wwait(dkv_free, (c - 1) & 1)) break;
      for (; j < end_j; ++j) {
        const int sb = j % NSB;
        const uint32_t pt = tmem + C::COL_S + QT * sb;
        if (!(ok = wwait(&p_full[sb], j / NSB & 1))) break;
        tc::fence_after_sync();
        issue_ts<D, QT / 16>(leader, tmem + C::COL_DV, pt, dot + j % ND * tile16, j == first);
        if (leader) tc::commit(&do_empty[j % ND]);
        issue_ts<D, QT / 16>(leader, tmem + C::COL_DK, pt + 8, qt + j % NQ * tile16, j == first);
        if (leader) {
          tc::commit(&s_free[sb]);
          tc::commit(&q_empty[j % NQ]);
        }
        __syncwarp();
      }
      if (leader) tc::commit(dkv_full);
      __syncwarp();
      ++c;
    }
    finish(&drain[2]);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int grp = NG == 1 ? 0 : (threadIdx.x - 32 * C::SOFT0) / C::GROUP;   // tiles grp, grp + NG ...
    const int tid = threadIdx.x - 32 * C::SOFT0 - grp * C::GROUP;
    const int cols = 32 * (tid >> 7);          // first of this thread's columns
    const int quad = warp & 3;                 // TMEM lane quadrant this warp may access
    const int key = quad * 32 + lane;          // key of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float* row_s = reinterpret_cast<const float*>(smem + C::OFF_ROW) + cols;   // [NR][2][QT]
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int i = 0, g = 0, done = 0; i < m && ok; ++i) {   // tiles, key tiles with work before
      const Tile t = tile(i);
      // every key of the tile sees every row of tiles [j_lo, j_hi), whole blocks of tokens
      int j_lo = g, j_hi = (t.i1 - t.i0) / QB2;
      if (p.causal) j_lo += max(0, (t.k0 + 127 - off - t.i0 + QB2 - 1) / QB2) << cs;
      if (p.window > 0) j_hi = min(j_hi, (t.k0 + p.window - off - t.i0) / QB2);
      j_hi = g + (j_hi << cs);
      const int end_j = g + t.n;
      for (int j = NG == 1 ? g : g + ((grp ^ g) & (NG - 1)); j < end_j; j += NG) {
        const int sb = j % NSB;
        const bool masked = j < j_lo || j >= j_hi;
        int lo = -128, hi = 128, nt = QB2;         // this thread's visible columns
        if (masked) {
          const int t0 = t.i0 + ((j - g) >> cs) * QB2;   // first query of the tile
          const int pos0 = off + t0;
          nt = min(QB2, t.i1 - t0);
          lo = (p.causal ? max(0, min(nt, t.k0 + key - pos0)) * GT : 0) - cols;
          hi = (p.window > 0 ? max(0, min(nt, t.k0 + key + p.window - pos0)) : nt) * GT - cols;
        }
        const Seen seen = seen_by_warp(masked, lo, hi);
        const uint32_t s_addr = lane_base + C::COL_S + QT * sb + cols;
        const uint32_t dp_addr = lane_base + C::COL_DP + cols;
        const float4* lse4 = reinterpret_cast<const float4*>(row_s + j % NR * 2 * QT);
        const float4* del4 = lse4 + QT / 4;
        if (!warp_wait3(&row_full[j % NR], j / NR & 1, &s_full[j % NB], j / NB & 1, &dp_full[j & 1], j >> 1 & 1,
                        abort_flag, status)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        auto square = [&](auto cut) {   // P and dS of the warp's square
          float w[2][16];
          tc::tmem_ld16(dp_addr, w[0]);
          tc::tmem_ld16(dp_addr + 16, w[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v[16];
            tc::tmem_ld16(s_addr + 16 * c, v);
            tc::tmem_wait_ld();
            if (c == 0) {
              tc::fence_before_sync();
              mbar_arrive(dp_free);   // the next tile's dP^T may come
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 l = lse4[c * 4 + e / 4], d = del4[c * 4 + e / 4];
              weights2(v[e], v[e + 1], cc, make_float2(l.x, l.y));
              weights2(v[e + 2], v[e + 3], cc, make_float2(l.z, l.w));
              scores2(w[c][e], w[c][e + 1], v[e], v[e + 1], make_float2(d.x, d.y));
              scores2(w[c][e + 2], w[c][e + 3], v[e + 2], v[e + 3], make_float2(d.z, d.w));
            }
            if constexpr (decltype(cut)::value) {   // (0 x NaN of another row is not 0)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c * 16 + e < lo || c * 16 + e >= hi) v[e] = w[c][e] = 0.f;
            }
            store_packed(s_addr + 16 * c, v);
            store_packed(s_addr + 16 * c + 8, w[c]);
          }
        };
        if (seen == kAll) {
          square(std::false_type());
        } else if (seen == kSome) {
          square(std::true_type());
        } else {
          mbar_arrive(dp_free);
#pragma unroll
          for (int c = 0; c < 4; ++c) store_zeros(s_addr + 8 * c);
        }
        if (nt < QB2) {
          // The visible rows end inside the tile: those behind them may be another
          // sequence's, whose NaN would pass through zero weights. Both products
          // that read the tile along d are done.
          zero_rows<NSUB>(smem + C::OFF_Q + j % NQ * C::Q_TILE, C::QSUB, nt * GT, QT, tid, C::GROUP);
          zero_rows<NSUB>(smem + C::OFF_DO + j % ND * C::Q_TILE, C::QSUB, nt * GT, QT, tid, C::GROUP);
          tc::fence_proxy_async_smem();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&p_full[sb]);
      }
      // ------------------------------------------------------------ epilogue
      if (ok && t.n > 0) ok = wwait(dkv_full, done & 1);
      tc::fence_after_sync();
      const int k = 128 * (kt + i) + key;
      const long long row = static_cast<long long>(p.Hkv) * s.k0 + static_cast<long long>(kvh) * s.lk + k;
      // four warps store 64 columns: dV's, then dK's
      const int blk = (warp - C::SOFT0) >> 2;
      const bool is_dk = blk >= NSUB;
      if (blk < 2 * NSUB) {
        tc::store_o_rows<64>(lane_base + C::COL_DV + 64 * blk, !(ok && t.n > 0), is_dk ? p.sm_scale : 1.f,
                             (is_dk ? p.dk : p.dv) + row * D + 64 * (is_dk ? blk - NSUB : blk), k < s.lk,
                             lane);
        tc::fence_before_sync();
        if (t.n > 0) mbar_arrive(dkv_free);
      }
      g = end_j;
      done += t.n > 0;
    }
  }

  // a warp that left its loop early may still have TMEM loads or stores in flight
  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // a wait gave up: let every issued copy land before the CTA's shared
    // memory goes away (a left-out tile's phase never completes: bounded)
    if (issued_kv > 0) mbar_drain(kv_full, (issued_kv - 1) & 1);
    for (int i = max(0, issued_q - NQ); i < issued_q; ++i) mbar_drain(&q_full[i % NQ], i / NQ & 1);
    for (int i = max(0, issued_do - ND); i < issued_do; ++i) mbar_drain(&do_full[i % ND], i / ND & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// dQ. S = Q K^T and dP = dO V^T (M 128 query rows, N 64 keys, K d; from shared
// memory), dQ += dS K (N d, K 64; dS from TMEM, where it replaces S). At d 64 two
// CTAs of one group share an SM: one starts or ends while the other computes. At
// d 128, where shared memory holds one CTA, it has two groups, which take
// alternate tiles.
template <int D>
struct DqCfg {
  static constexpr int CTAS = D == 64 ? 2 : 1;      // CTAs of an SM
  static constexpr int NG = D / 64;                 // groups of a CTA
  static constexpr int KT = 64;                     // keys of a tile
  static constexpr int SOFT0 = 4;                   // first warp of dS
  static constexpr int GROUP = 256;                 // threads of a group: 32 columns of a row each
  static constexpr int THREADS = SOFT0 * 32 + NG * GROUP;
  static constexpr int NSUB = D / 64;
  static constexpr int KSUB = KT * 128;
  static constexpr int QSUB = 128 * 128;
  static constexpr int K_TILE = NSUB * KSUB;
  static constexpr int Q_TILE = NSUB * QSUB;
  static constexpr int NSB = 2 * NG;                // S buffers
  static constexpr int NDP = NG;                    // dP buffers
  static constexpr int NK = D == 64 ? 5 : 6;        // stages of K
  static constexpr int NV = 4;                      // stages of V, which one product reads
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = Q_TILE;
  static constexpr int OFF_K = 2 * Q_TILE;
  static constexpr int OFF_V = OFF_K + NK * K_TILE;
  static constexpr int OFF_BAR = OFF_V + NV * K_TILE;
  static constexpr int N_BARS = 2 + 2 * NK + 2 * NV + 3 * NSB + 2 + NDP + 2 + 2 + 3;
  static constexpr int OFF_ROW = OFF_BAR + N_BARS * 8 + 16;   // [2][128] (-lse log2 e, -delta)
  static constexpr int SMEM = OFF_ROW + 2 * 128 * 8;
  static constexpr uint32_t COLS = 512 / CTAS;
  static constexpr uint32_t COL_S = 0;
  static constexpr uint32_t COL_DP = NSB * KT;
  static constexpr uint32_t COL_DQ = COL_DP + NDP * KT;
  static_assert(COL_DQ + D <= COLS, "TMEM budget");
  static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory budget");
};

template <int D>
__device__ __forceinline__ void back_dq_block(const CUtensorMap& tmQ, const CUtensorMap& tmDo,
                                              const CUtensorMap& tmK, const CUtensorMap& tmV,
                                              const BackParams& p) {
  using C = DqCfg<D>;
  constexpr int NK = C::NK, NV = C::NV, NSB = C::NSB, NDP = C::NDP, NG = C::NG, NSUB = C::NSUB, KT = C::KT;
  extern __shared__ __align__(1024) uint8_t smem[];   // (swizzled tiles start on 1024 bytes)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + 1;      // S and dP of the query tile done
  uint64_t* k_full = q_empty + 1;      // [NK]
  uint64_t* k_empty = k_full + NK;     // [NK] dQ, the last that reads the stage, done
  uint64_t* v_full = k_empty + NK;     // [NV]
  uint64_t* v_empty = v_full + NV;     // [NV] dP done
  uint64_t* s_full = v_empty + NV;     // [NSB] S written
  uint64_t* s_free = s_full + NSB;     // [NSB] the dS in it read by dQ
  uint64_t* ds_full = s_free + NSB;    // [NSB] dS written (the group's arrivals)
  uint64_t* dp_full = ds_full + NSB;   // [2] of even and odd tiles: dP written
  uint64_t* dp_free = dp_full + 2;     // [NDP] dP read (the group's arrivals)
  uint64_t* dq_full = dp_free + NDP;   // a query tile's dQ done
  uint64_t* dq_free = dq_full + 1;     // and read
  uint64_t* row_full = dq_free + 1;    // [2] the rows' numbers there (all arrive)
  uint64_t* drain = row_full + 2;      // [3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefill_back;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // A CTA's query tiles: m of them, the highest first. Those of the first CTAs see the
  // most keys. The next one's rows and first products come while it ends the one before.
  const int per = p.Hkv * p.batch;
  const int run = p.nrun - 1 - static_cast<int>(blockIdx.x) / per;
  const int kvh = static_cast<int>(blockIdx.x) % per % p.Hkv;
  const int b = static_cast<int>(blockIdx.x) % per / p.Hkv;
  const Seq s = load_seq(p, b);
  if (!s.ok) {
    if (threadIdx.x == 0) atomicExch(status, SINKATTN_BAD_LENGTHS);
    return;
  }
  const int end = min((run + 1) * p.run, (s.lq + p.QB - 1) / p.QB);
  const int m = end - run * p.run;
  if (m <= 0) return;   // uniform over the CTA, before any barrier or TMEM use
  const int G = p.G;
  struct Tile {
    int t0, nt, pos0;   // its queries, the first one's position
    int k_lo, n;        // tiles of the keys [k_lo ...) that some row sees (at least 1)
  };
  auto tile = [&](int i) {
    Tile x;
    x.t0 = (end - 1 - i) * p.QB;
    x.nt = min(p.QB, s.lq - x.t0);
    x.pos0 = s.lk - s.lq + x.t0;
    x.k_lo = p.window > 0 ? max(0, x.pos0 - p.window + 1) : 0;
    x.n = ((p.causal ? x.pos0 + x.nt : s.lk) - x.k_lo + KT - 1) / KT;
    return x;
  };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 1);
      mbar_init(&ds_full[i], C::GROUP);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&dp_full[i], 1);
    for (int i = 0; i < NDP; ++i) mbar_init(&dp_free[i], C::GROUP);
    mbar_init(dq_full, 1);
    mbar_init(dq_free, NSUB * 128);
    for (int i = 0; i < 2; ++i) mbar_init(&row_full[i], NG * C::GROUP);
    for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
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
  int issued_q = 0, issued_k = 0, issued_v = 0;   // tiles whose copies were issued (or left out by the test hook)
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, status);
  };

  auto wwait2 = [&](uint64_t* x, uint32_t px, uint64_t* y, uint32_t py) -> bool {
    return warp_wait2(x, px, y, py, abort_flag, status);
  };
  const bool leader = tc::elect_one();
  // an issuing warp's end: every MMA of it has completed before the CTA frees TMEM
  auto finish = [&](uint64_t* bar) {
    if (leader) tc::commit(bar);
    __syncwarp();
    mbar_drain(bar, 0);
  };
  const uint32_t tile16 = C::K_TILE >> 4;   // a stage, in descriptor units

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    const uint64_t policy = policy_evict_last();   // K and V are re-read by every query block
    const int skip_tile = hook_skip_tile();
    auto load = [&](const CUtensorMap* map, int j, int row, uint8_t* to, uint64_t* bar) {   // into a free stage
      if (j != skip_tile && leader) {   // test hook: the waits for this tile run out
        mbar_arrive_expect_tx(bar, C::K_TILE);
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
          tma_load_2d_hint(to + sub * C::KSUB, map, sub * 64, row, bar, policy);
      }
      __syncwarp();
    };
    bool ok = true;
    for (int i = 0, g = 0; i < m && ok; ++i) {   // g: tiles of keys before
      const Tile t = tile(i);
      const int slab = p.Hkv * s.k0 + kvh * s.lk + t.k_lo;
      if (i > 0 && !wwait(q_empty, (i - 1) & 1)) break;
      issued_q = i + 1;
      if (leader) {
        // (rows that no copy writes are lanes whose results are not stored)
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(2 * NSUB * 128 * G * p.QB));
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub) {
          tc::tma_load_3d(smem + C::OFF_Q + sub * C::QSUB, &tmQ, sub * 64, kvh * G, s.q0 + t.t0, q_full);
          tc::tma_load_3d(smem + C::OFF_DO + sub * C::QSUB, &tmDo, sub * 64, kvh * G, s.q0 + t.t0, q_full);
        }
      }
      __syncwarp();
      for (int x = g; x < g + t.n + NK - NV; ++x) {
        if (x < g + t.n) {
          if (x >= NK && !(ok = wwait(&k_empty[x % NK], (x / NK - 1) & 1))) break;
          issued_k = x + 1;
          load(&tmK, x, slab + (x - g) * KT, smem + C::OFF_K + x % NK * C::K_TILE, &k_full[x % NK]);
        }
        const int y = x - (NK - NV);   // V lags by the stages that K has more
        if (y < g) continue;
        if (y >= NV && !(ok = wwait(&v_empty[y % NV], (y / NV - 1) & 1))) break;
        issued_v = y + 1;
        load(&tmV, y, slab + (y - g) * KT, smem + C::OFF_V + y % NV * C::K_TILE, &v_full[y % NV]);
      }
      g += t.n;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S = Q K^T
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    bool ok = true;
    for (int i = 0, j = 0; i < m && ok; ++i) {
      const int end_j = j + tile(i).n;
      if (!wwait(q_full, i & 1)) break;
      for (; j < end_j; ++j) {
        ok = j < NSB ? wwait(&k_full[j % NK], j / NK & 1)
                     : wwait2(&s_free[j % NSB], (j / NSB - 1) & 1, &k_full[j % NK], j / NK & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_ss<D, KT>(leader, tmem + C::COL_S + KT * (j % NSB), qd, kd + j % NK * tile16, C::QSUB, C::KSUB);
        if (leader) tc::commit(&s_full[j % NSB]);
        __syncwarp();
      }
      if (leader) tc::commit(q_empty);
      __syncwarp();
    }
    finish(&drain[0]);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- dP = dO V^T
    const uint64_t dod = tc::smem_desc_sw128(smem_u32(smem + C::OFF_DO), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
    bool ok = true;
    for (int i = 0, j = 0; i < m && ok; ++i) {
      const int end_j = j + tile(i).n;
      if (!wwait(q_full, i & 1)) break;
      for (; j < end_j; ++j) {
        ok = j < NDP ? wwait(&v_full[j % NV], 0)
                     : wwait2(&dp_free[j % NDP], (j / NDP - 1) & 1, &v_full[j % NV], j / NV & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_ss<D, KT>(leader, tmem + C::COL_DP + KT * (j % NDP), dod, vd + j % NV * tile16, C::QSUB, C::KSUB);
        if (leader) {
          tc::commit(&dp_full[j & 1]);
          tc::commit(&v_empty[j % NV]);
        }
        __syncwarp();
      }
      if (leader) tc::commit(q_empty);
      __syncwarp();
    }
    finish(&drain[1]);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- dQ += dS K
    const uint64_t kt = tc::smem_desc_sw128(smem_u32(smem + C::OFF_K), C::KSUB, 1024);   // MN-major
    bool ok = true;
    for (int i = 0, j = 0; i < m && ok; ++i) {
      const int first = j, end_j = j + tile(i).n;
      if (i > 0 && !wwait(dq_free, (i - 1) & 1)) break;
      for (; j < end_j; ++j) {
        if (!(ok = wwait(&ds_full[j % NSB], j / NSB & 1))) break;
        tc::fence_after_sync();
        issue_ts<D, KT / 16>(leader, tmem + C::COL_DQ, tmem + C::COL_S + KT * (j % NSB), kt + j % NK * tile16,
                             j == first);
        if (leader) {
          tc::commit(&s_free[j % NSB]);
          tc::commit(&k_empty[j % NK]);
        }
        __syncwarp();
      }
      if (leader) tc::commit(dq_full);
      __syncwarp();
    }
    finish(&drain[2]);
  } else {
    // ---------------------------------------------------------------- P and dS
    const int grp = NG == 1 ? 0 : (threadIdx.x - 32 * C::SOFT0) / C::GROUP;   // tiles grp, grp + NG ...
    const int tid = threadIdx.x - 32 * C::SOFT0 - grp * C::GROUP;
    const int cols = 32 * (tid >> 7);          // first of this thread's columns
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int rt = row / G;
    float2* const rows = reinterpret_cast<float2*>(smem + C::OFF_ROW);
    // -lse log2 e and -delta of tile i's rows, D / 8 threads a row, all of a thread's
    // loads at once: for this pass and, through the workspace, for that of dk and dv.
    auto row_numbers = [&](int i) {
      constexpr int DC = D / 8, R = 32 / DC, N = 128 / (NG * C::GROUP / 32 * R);
      const int c = lane % DC, r0 = (warp - C::SOFT0) * N * R + lane / DC;
      const Tile t = tile(i);
      uint4 x[N], y[N];
      float lse[N], dlse[N];
      long long where[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int r = r0 + e * R, tok = r / G;
        x[e] = y[e] = make_uint4(0, 0, 0, 0);
        lse[e] = dlse[e] = 0.f;
        where[e] = -1;
        if (tok >= t.nt || r >= G * p.QB) continue;
        where[e] = static_cast<long long>(s.q0 + t.t0 + tok) * p.Hq + kvh * G + (r - tok * G);
        x[e] = __ldg(reinterpret_cast<const uint4*>(p.dout + where[e] * D) + c);
        y[e] = __ldcs(reinterpret_cast<const uint4*>(p.out + where[e] * D) + c);
        if (c != 0) continue;
        lse[e] = p.lse[where[e]];
        if (p.dlse) dlse[e] = p.dlse[where[e]];
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float sum = dot8(x[e], y[e], 0.f);
#pragma unroll
        for (int k = 1; k < DC; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (c != 0) continue;
        // a row with lse -inf has no weights (P = 0, as for lse +inf, which exponentials give)
        const float nl = where[e] < 0 || lse[e] == kNegInf ? kNegInf : -lse[e] * kLog2e;
        const float nd = dlse[e] - sum;
        rows[(i & 1) * 128 + r0 + e * R] = make_float2(nl, nd);
        if (where[e] >= 0) {
          p.nlse[where[e]] = nl;
          p.ndelta[where[e]] = nd;
        }
      }
      mbar_arrive(&row_full[i & 1]);
    };
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t dp_addr = lane_base + C::COL_DP + KT * grp + cols;
    const float2 cc = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int i = 0, g = 0;; ++i) {   // g: tiles of keys before
      if (i < m && ok) row_numbers(i);
      if (i > 0) {
        // -------------------------------------------------------- epilogue of the tile before
        if (ok) ok = wwait(dq_full, (i - 1) & 1);
        tc::fence_after_sync();
        const int blk = (warp - C::SOFT0) >> 2;   // four warps store 64 columns
        if (blk < NSUB) {
          const Tile t = tile(i - 1);
          const long long at = static_cast<long long>(s.q0 + t.t0 + rt) * p.Hq + kvh * G + (row - rt * G);
          tc::store_o_rows<64>(lane_base + C::COL_DQ + 64 * blk, !ok, p.sm_scale, p.dq + at * D + 64 * blk,
                               rt < t.nt && row < G * p.QB, lane);
          tc::fence_before_sync();
          mbar_arrive(dq_free);
        }
      }
      if (i == m || !ok) break;
      const Tile t = tile(i);
      const bool valid = rt < t.nt && row < G * p.QB;
      const int pos = t.pos0 + rt;
      // keys [lo_r, hi_r) are visible to the row
      const int hi_r = valid ? (p.causal ? pos + 1 : s.lk) : 0;
      const int lo_r = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      // every row of the block sees every key of tiles [j_lo, j_hi) (rows that are not stored need no mask)
      int j_lo = g;
      const int j_hi = g + ((p.causal ? min(s.lk, t.pos0 + 1) : s.lk) - t.k_lo) / KT;
      if (p.window > 0) j_lo = g + max(0, (t.pos0 + t.nt - p.window - t.k_lo + KT - 1) / KT);
      ok = wwait(&row_full[i & 1], i >> 1 & 1);
      const float2 num = rows[(i & 1) * 128 + row];
      const float2 nl = make_float2(num.x, num.x), nd = make_float2(num.y, num.y);
      const int end_j = g + t.n;
      for (int j = NG == 1 ? g : g + ((grp ^ g) & (NG - 1)); j < end_j && ok; j += NG) {
        const bool masked = j < j_lo || j >= j_hi;
        const int j0 = t.k_lo + (j - g) * KT;
        const int lo = lo_r - j0 - cols, hi = hi_r - j0 - cols;
        const Seen seen = seen_by_warp(masked, lo, hi);
        const uint32_t s_addr = lane_base + C::COL_S + KT * (j % NSB) + cols;
        if (!(ok = wwait2(&s_full[j % NSB], j / NSB & 1, &dp_full[j & 1], j >> 1 & 1))) break;
        tc::fence_after_sync();
        if (j0 + KT > s.lk) {
          // The keys end inside the tile: the rows behind them are another head's or sequence's,
          // whose NaN would pass through zero weights. (S(j), the other reader, is done.)
          zero_rows<NSUB>(smem + C::OFF_K + j % NK * C::K_TILE, C::KSUB, s.lk - j0, KT, tid, C::GROUP);
          tc::fence_proxy_async_smem();
        }
        auto square = [&](auto cut) {   // dS of the warp's square
          float w[2][16];
          tc::tmem_ld16(dp_addr, w[0]);
          tc::tmem_ld16(dp_addr + 16, w[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v[16];
            tc::tmem_ld16(s_addr + 16 * c, v);
            tc::tmem_wait_ld();
            if (c == 0) {
              tc::fence_before_sync();
              mbar_arrive(&dp_free[grp]);   // a later tile's dP may come
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              weights2(v[e], v[e + 1], cc, nl);
              scores2(w[c][e], w[c][e + 1], v[e], v[e + 1], nd);
            }
            if constexpr (decltype(cut)::value) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c * 16 + e < lo || c * 16 + e >= hi) w[c][e] = 0.f;
            }
            store_packed(s_addr + 16 * c, w[c]);
          }
        };
        if (seen == kAll) {
          square(std::false_type());
        } else if (seen == kSome) {
          square(std::true_type());
        } else {
          mbar_arrive(&dp_free[grp]);
#pragma unroll
          for (int c = 0; c < 2; ++c) store_zeros(s_addr + 16 * c);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&ds_full[j % NSB]);
      }
      g = end_j;
    }
  }

  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    mbar_drain(q_full, (issued_q - 1) & 1);
    for (int i = max(0, issued_k - NK); i < issued_k; ++i) mbar_drain(&k_full[i % NK], i / NK & 1);
    for (int i = max(0, issued_v - NV); i < issued_v; ++i) mbar_drain(&v_full[i % NV], i / NV & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// The first launch of a call: the blocks of dk and dv may come as these leave
// their SMs, and wait for the rows' numbers where they need them.
template <int D>
__global__ void __launch_bounds__(DqCfg<D>::THREADS, DqCfg<D>::CTAS)
    back_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const BackParams p) {
  grid_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.sink_count = 0;
  back_dq_block<D>(tmQ, tmDo, tmK, tmV, p);
}

int launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s launch: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

int set_smem(cudaError_t e) {
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

// How many of `items` equal tiles a CTA goes through, `ctas` of them on an SM: the
// number for which the last wave ends first, if a tile takes `steps` steps and a CTA
// one more, to start and to end. 10,168 tokens of 64/8 heads of 64 in windows of
// 128: dq 114 us with the 17 that this gives (150 with one), dk and dv 101 with 5
// (113 with one).
int tiles_of_cta(int64_t items, int ctas, int64_t steps) {
  int best = 1;
  int64_t least = 0;
  for (int n = 1; n <= 32; ++n) {
    const int64_t waves = ((items + n - 1) / n + 152 * ctas - 1) / (152 * ctas);
    const int64_t time = waves * (n * steps + 1);
    if (n == 1 || time < least) best = n, least = time;
  }
  return best;
}

template <int D>
int launch_back(BackParams& p, cudaStream_t stream) {
  using KV = DkvCfg<D>;
  using DQ = DqCfg<D>;
  // every size is checked, and every map made, before the first launch
  const int64_t per = static_cast<int64_t>(p.Hkv) * p.batch;
  // Tiles of a CTA. In windows that are short for their sequences all tiles see about
  // as much. Else the longest come first, and the pass of dk and dv, whose tiles are long,
  // takes one each (2 x 6000 tokens of 64/4 heads of 128: 2.83 ms with one, 3.37 with
  // two), that of dq up to eight while they leave every place on an SM four runs (2.68 ms,
  // 24 x 512 tokens 456 us; with one 2.83 and 557. 3,000 tokens of 24/8 heads, which
  // leave too few: 64 us with one, 97 with eight). With equal shares in windows of a third
  // of the sequences the same 12,000 tokens took 1.90 ms, 1.73 with one each. (All of these in
  // short bursts, before the power limit.) At the border between the two rules, 10,168 tokens
  // of 64/8 heads of 64 in sequences of up to 4096: windows of 512 take 368 us with equal
  // shares, of 513 347 without; of 128, 212 and of 256, 264.
  const bool alike = p.window > 0 && p.window <= p.max_q / 8;
  const int64_t window = p.window;
  const int64_t q_tiles =
      p.Hkv * std::min<int64_t>(p.total_q / p.QB + p.batch, static_cast<int64_t>(p.nqb) * p.batch);
  const int64_t k_tiles =
      p.Hkv * std::min<int64_t>(p.total_k / 128 + p.batch, (int64_t{p.max_kv} + 127) / 128 * p.batch);
  p.run = alike ? tiles_of_cta(q_tiles, DQ::CTAS, (window + p.QB) / DQ::KT + 1)
                : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, q_tiles / (4 * 152 * DQ::CTAS))));
  p.krun = alike ? tiles_of_cta(k_tiles, 1, ((window + 127) / p.QB2 + 1) * p.chunks) : 1;
  p.nrun = (p.nqb + p.run - 1) / p.run;
  // (one tile where the bound says none: its CTAs see a sequence that has keys all the same)
  const int64_t longest = std::max<int64_t>(1, (static_cast<int64_t>(p.max_kv) + 127) / 128);
  const int64_t dkv_items = (longest + p.krun - 1) / p.krun * per;
  const int64_t dq_items = p.total_q > 0 ? p.nrun * per : 0;
  p.sink_blocks = p.dsinks ? (dq_items ? static_cast<int>(back_sink_blocks(p.total_q, p.Hq)) : 1) : 0;
  if (std::max(dkv_items + p.sink_blocks, dq_items) >= (int64_t{1} << 31)) {
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
  if (dq_items > 0) {
    back_dq_kernel<D><<<static_cast<unsigned>(dq_items), DQ::THREADS, DQ::SMEM, stream>>>(tmQ, tmDo, tmK, tmV, p);
    if ((rc = launched("dq", cudaGetLastError()))) return rc;
  }
  p.dkv_items = static_cast<int>(dkv_items);
  const dim3 grid(static_cast<unsigned>(dkv_items + p.sink_blocks));
  if (dq_items > 0)
    return launched("dk, dv", launch_chained(back_dkv_kernel<D>, grid, KV::THREADS, KV::SMEM, stream, tmQ2,
                                             tmDo2, tmK2, tmV2, p));
  // the first launch of the call reads its inputs at once
  back_dkv_kernel<D><<<grid, KV::THREADS, KV::SMEM, stream>>>(tmQ2, tmDo2, tmK2, tmV2, p);
  return launched("dk, dv", cudaGetLastError());
}

}  // namespace

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
  p.max_q = std::min(a.max_q, a.total_q);   // (a bound may be above what there is)
  p.max_kv = std::min(a.max_kv, a.total_k);
  p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv;
  p.sm_scale = a.sm_scale; p.scale_log2 = a.sm_scale * kLog2e;
  p.causal = a.causal;
  p.window = a.window < p.max_kv ? a.window : 0;   // (one of all keys cuts nothing)
  p.QB = 128 / p.G;
  p.nqb = static_cast<int>((int64_t{p.max_q} + p.QB - 1) / p.QB);
  const int rows = a.d == 64 ? DkvCfg<64>::QT : DkvCfg<128>::QT;
  p.chunks = p.G > rows ? 2 : 1;
  p.GT = (p.G + p.chunks - 1) / p.chunks;
  p.QB2 = rows / p.GT;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.dsinks = a.dsinks; p.nlse = a.nlse; p.ndelta = a.ndelta; p.sink_part = a.sink_part;
  p.sink_count = a.sink_count;
  p.sink_tokens = back_sink_tokens(a.Hq);
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
