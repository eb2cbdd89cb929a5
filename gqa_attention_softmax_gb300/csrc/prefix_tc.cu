// The shared prefix of shared-prefix decode on the 5th-generation tensor
// cores: all query rows of a group of sequences against the prefix's keys,
// which every row sees (but for a window), read once per block of rows.
//
// Rows are (query token, head in group) pairs of one KV head, 128 to a tile;
// a block has NT tiles that share each K/V tile in shared memory. A work item
// is (row block, KV head, run of its key tiles); it leaves the rows' partials
// (m, d, acc) WITHOUT the sink for the merge, like the split-KV kernels:
//
//   S_t = Q_t K^T     M 128 rows, N KT keys, K d   (operands in shared memory)
//   O_t += P_t V      M 128 rows, N d, K KT keys   (P_t from TMEM)
//
// With hundreds of rows per KV head the prefix is compute-bound (4 d
// operations per row and key against 4 d / rows bytes), so the kernel follows
// the persistent prefill: one block per SM, a TMA producer warp, MMA issuer
// warps, and per tile four softmax warps, one thread per row. Two tiles
// per block (three would not divide 512 rows, the gpt-oss-shaped batch of 64
// sequences, and TMEM holds no more at d 128); the tiles' chains S -> softmax
// -> P V interleave on the tensor core. A tile whose rows all lie behind the
// group's last token is left out.
//
// The work is cut into equal runs: a unit is one K/V tile of one (row block,
// KV head), block c takes the c-th run of units in a fixed order (their number
// is the plan's: with own keys to read beside the prefix, fewer blocks with
// longer runs leave SMs to those and partials out), and a row block's
// partial number is that of its block of units. So few row blocks, ragged
// groups and prefixes of any mix of lengths fill the SMs alike, and a row
// block has as many partials as thread blocks worked on it; the merge reads
// only those.
//
// e4m3 pools: the producer copies codes into a ring of their own, two
// converter warps (four at d 128) widen each tile to f16 in the layout the MMAs read (exact:
// f16 holds every e4m3 value) and turn Q to f16 once per item; each code is
// converted once per row block, not once per sequence. The key scale joins
// the logit scale, the value scale the written accumulator.
//
// Weights are taken relative to a reference maximum that lies at most 2^8
// below the true one; each is rounded by at most half a step of bf16 (f16) for
// P V, and the row sum l is kept in fp32 from the unrounded weights. Where one
// weight is most of a row's sum its rounding would reach the output whole, as
// it is no power of two when the reference lies behind it. So the largest
// weight of each step counts as rounded in a second sum l', the divisor:
//   l' = l + sum over steps (RN(w_max) - w_max),
// and the partial is (m + ln(l / l'), l', acc), whose log-sum-exp is still that
// of the unrounded weights. Rows of normal logits over 4032 keys, spread by
// 3, 6 and 12 times (float64 restatement): the mean over rows of the largest
// error goes from 1.5e-3, 1.1e-3, 7.6e-4 of the row's largest value to 1.3e-3,
// 7.3e-4, 3.8e-4, the same as with every weight's rounding in the divisor, which
// takes three more instructions per pair of weights. (f16 weights are within
// 2^-11, an eighth of the output's own rounding: their divisor is l.) Every
// wait is bounded.
//
// At d 64 (and with codes) each row tile has two S buffers and an issuer of
// its own, which sends the next S while the softmax of the present one runs.
// A step of 96 keys took 2.8k cycles with one buffer (softmax 1.4k, then P V,
// S and their latencies; what TMEM leaves at d 128), 2.25k with two and one
// issuer, 2.0k with two issuers.
//
// Measured: a unit (256 rows, 96 keys) at d 64 1.05 us, at d 128 (128 keys)
// 1.75 us, the softmax warps' chain; a block's first P comes 6 us after the plan's
// end, a run's end costs about 3 us at d 128. 512 rows of 8 KV heads behind 8192
// keys: 22 us; 12288 rows of 4 behind 4032: 89 us, 1.15 PFLOP/s (tensor pipe 48 %
// of the time, 57 % while blocks run).
#include <algorithm>

#include "chain.cuh"
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace sinkattn {

__device__ int g_status_prefix_tc;

namespace {

struct PxParams {
  const int32_t* grp_q;      // [groups + 1] first query token
  const int32_t* grp_k;      // [groups + 1] running sum of the prefixes' keys
  const int32_t* grp_pages;  // [groups + 1] first entry in page_indices
  const int32_t* grp_unit;   // [groups + 1] running sum of units
  const int32_t* quota;      // [1] units of one thread block
  const int32_t* row_pos;    // [tokens] position of each query token (windows)
  const int32_t* page_indices;
  int groups, Hq, Hkv, G, QB;
  int splits;                // partials a row block may have
  int window;
  float sm_scale, scale_log2;
  int page_size, box_rows;
  const float* k_scale;
  const float* v_scale;
  float* part_acc;
  float* part_md;
  int part_slots;
};

template <int D, bool FP8>
struct PxCfg {
  static constexpr int NT = 2;
  static constexpr int NSUB = D / 64;
  static constexpr int KT = D == 64 ? 96 : (FP8 ? 64 : 128);   // keys per tile
  static constexpr int NSB = D == 64 || FP8 ? 2 : 1;           // S buffers per row tile (TMEM)
  static constexpr int NST = D == 64 ? (FP8 ? 3 : 4) : (FP8 ? 3 : 2);   // K/V stages
  static constexpr int NSTF = FP8 ? 3 : 0;     // code stages
  static constexpr int NSTF_MOD = FP8 ? NSTF : 1;
  static constexpr int QSUB = 128 * 128;                       // [128 rows][64], 128-byte swizzle
  static constexpr int KVSUB = KT * 128;
  static constexpr int Q_TILE = NSUB * QSUB;
  static constexpr int KV_TILE = NSUB * KVSUB;
  static constexpr int STAGE = 2 * KV_TILE;
  static constexpr int CODE_STAGE = 2 * KT * D;
  static constexpr int OFF_KV = NT * Q_TILE;
  static constexpr int OFF_CODE = OFF_KV + NST * STAGE;
  static constexpr int GRP_CAP = 512;                          // groups staged in shared memory
  static constexpr int OFF_GRP = OFF_CODE + NSTF * CODE_STAGE;
  static constexpr int NIT = 4;                                // items in the ring
  static constexpr int OFF_ITEM = OFF_GRP + (4 * (GRP_CAP + 1) * 4 + 15) / 16 * 16;
  static constexpr int OFF_BAR = OFF_ITEM + NIT * 48;
  // MMA issuers: with two S buffers a step is bound by the issue of its MMAs,
  // about 1.0k cycles per row tile with their waits, so each tile has its own
  static constexpr int NI = NSB == 2 ? NT : 1;
  static constexpr int N_BARS = 3 + 2 * NST + 3 * NSB * NT + NI + 2 * NSTF + 2 * NIT;
  static constexpr int SMEM = 1024 + OFF_BAR + N_BARS * 8 + 64;
  static constexpr int W_MMA1 = 2 + 4 * NT;                    // the second tile's issuer
  static constexpr int N_CVT = D == 64 ? 2 : 4;
  static constexpr int W_CVT = W_MMA1 + NI - 1;                // first converter warp
  static constexpr int THREADS = (W_CVT + (FP8 ? N_CVT : 0)) * 32;
  // registers: 10 warps put 3 on two SM sub-partitions (168 a thread), 13
  // warps and more put 4 on one (128, bounded by a 512-thread launch)
  static constexpr int LB_THREADS = FP8 || D == 64 ? 512 : 320;
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t col_s(int t, int buf) {
    return static_cast<uint32_t>(KT * (NSB * t + buf));
  }
  __host__ __device__ static constexpr uint32_t col_o(int t) {
    return static_cast<uint32_t>(KT * NSB * NT + D * t);
  }
  static_assert(NT * (NSB * KT + D) <= 512, "TMEM budget");
  static_assert(KVSUB % 1024 == 0 && KT % 32 == 0, "tile shape");
  // one block per SM, so the 512-column TMEM allocation always succeeds
  static_assert(SMEM <= 232448 && 2 * (SMEM + 1024) > 233472, "one block per SM");
};

struct PxItem {
  int kvh, slot, tok0, nq, tiles, keys, first;
  int n;       // K/V tiles; -1: no more items
  int list0, pages;
  int last;    // the item ends its row block's keys
  int pad;
};

// The group with gu[g] <= u < gu[g + 1].
__device__ __forceinline__ int px_group(const int32_t* gu, int groups, int u) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (gu[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Walks a thread block's units item by item: (group, KV head, row block),
// neighbouring row blocks of the same keys finding them in L2. The producer
// warp walks and hands the items to the other warps through a ring in shared
// memory, which keeps the walk's registers out of theirs.
template <int KT, int NT>
struct PxCursor {
  const int32_t *gq, *gk, *gp, *gu;
  int u, end;                       // next unit, and the block's last but one
  int g, kvh, blk, t0, slot;        // where u is
  int T, blocks, keys, tok, toks;   // of group g

  __device__ __forceinline__ void group(const PxParams& p) {
    keys = gk[g + 1] - gk[g];
    T = (keys + KT - 1) / KT;
    tok = gq[g];
    toks = gq[g + 1] - tok;
    blocks = (toks + NT * p.QB - 1) / (NT * p.QB);
  }

  // This thread block's run of units. One partial per row: row blocks are not
  // cut, a run starts and ends at the next row block's first unit.
  __device__ __forceinline__ void start(const PxParams& p, const int32_t* gq_, const int32_t* gk_,
                                        const int32_t* gp_, const int32_t* gu_) {
    gq = gq_;
    gk = gk_;
    gp = gp_;
    gu = gu_;
    const int all = gu[p.groups];
    const int quota = *p.quota;
    const long long from = static_cast<long long>(blockIdx.x) * quota;
    u = static_cast<int>(min(from, static_cast<long long>(all)));
    end = static_cast<int>(min(from + quota, static_cast<long long>(all)));
    if (p.splits == 1) {
      u = whole(p, u, all);
      end = whole(p, end, all);
    }
    if (u >= end) return;
    g = px_group(gu, p.groups, u);
    group(p);
    const int pair = (u - gu[g]) / T;
    t0 = u - gu[g] - pair * T;
    kvh = pair / blocks;
    blk = pair - kvh * blocks;
    slot = p.splits > 1 ? static_cast<int>(blockIdx.x) - (u - t0) / quota : 0;
  }

  __device__ __forceinline__ int whole(const PxParams& p, int v, int all) const {
    if (v >= all) return all;
    const int h = px_group(gu, p.groups, v);
    const int n = (gk[h + 1] - gk[h] + KT - 1) / KT;
    return gu[h] + (v - gu[h] + n - 1) / n * n;
  }

  __device__ __forceinline__ bool more() const { return u < end; }

  // The item at u, and on to the next. Whole warp: with a window the keys
  // before the block's earliest visible one are left out, which takes a
  // minimum over its tokens.
  __device__ __forceinline__ PxItem next(const PxParams& p, int lane) {
    PxItem t;
    t.kvh = kvh;
    t.slot = slot;
    const int at = blk * NT * p.QB;
    t.tok0 = tok + at;
    t.nq = min(NT * p.QB, toks - at);
    t.tiles = t.nq > p.QB ? 2 : 1;
    t.keys = keys;
    t.list0 = gp[g];
    t.pages = gp[g + 1] - t.list0;
    int from = t0;
    const int to = min(T, t0 + end - u);
    t.last = to == T;
    u += to - t0;
    if (p.window > 0) {
      int pos = INT32_MAX;
      for (int i = lane; i < t.nq; i += 32) pos = min(pos, p.row_pos[t.tok0 + i]);
      pos = __reduce_min_sync(0xffffffffu, pos);
      from = min(max(from, max(0, pos - p.window + 1) / KT), to);
    }
    t.first = from * KT;
    t.n = to - from;
    t0 = 0;   // (only a block's last item ends inside a row block)
    slot = 0;
    if (++blk == blocks) {
      blk = 0;
      if (++kvh == p.Hkv) {
        kvh = 0;
        if (u < end) {
          do ++g;
          while (gu[g + 1] == gu[g]);
          group(p);
        }
      }
    }
    return t;
  }
};

// A tile row's accumulator from TMEM to its fp32 partial row, 32 columns at a
// time: the eight 16-byte pieces of a lane's row are transposed within groups
// of eight lanes, so that a store instruction writes four whole 128-byte rows.
// Warp-collective.
template <int D>
__device__ __forceinline__ void store_partial(uint32_t o_addr, float scale, float* row, bool valid,
                                              int lane) {
  const int i = lane & 7;
  const unsigned long long mine = valid ? reinterpret_cast<unsigned long long>(row) : 0ull;
  float* to[8];   // the rows of the lane's group of eight
#pragma unroll
  for (int e = 0; e < 8; ++e)
    to[e] = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, mine, (lane & ~7) + e));
#pragma unroll
  for (int blk = 0; blk < D / 32; ++blk) {
    float o[32];
    tc::tmem_ld32(o_addr + blk * 32, o);
    tc::tmem_wait_ld();
    float4 ch[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      ch[e] = make_float4(o[4 * e] * scale, o[4 * e + 1] * scale, o[4 * e + 2] * scale,
                          o[4 * e + 3] * scale);
    transpose8_chunks(ch, lane);   // ch[e] of lane i: piece i of the group's row e
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (to[e]) *reinterpret_cast<float4*>(to[e] + blk * 32 + i * 4) = ch[e];
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PxCfg<D, FP8>::LB_THREADS, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PxParams p) {
  using C = PxCfg<D, FP8>;
  constexpr int KT = C::KT, NST = C::NST, NT = C::NT, NSB = C::NSB;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);   // by item
  uint64_t* q_empty = q_full + 1;       // the item's last S has completed
  uint64_t* q_cvt = q_empty + 1;        // FP8: Q is f16
  uint64_t* kv_full = q_cvt + 1;        // [NST] by K/V tile
  uint64_t* kv_empty = kv_full + NST;
  uint64_t* s_full = kv_empty + NST;    // [NT][NSB] by the row tile's own steps
  uint64_t* p_full = s_full + NT * NSB; // [NT][NSB] P_t written and O_t rescaled (128 arrivals)
  uint64_t* pv_done = p_full + NT * NSB;   // [NT][NSB] by the step's buffer
  uint64_t* drain = pv_done + NT * NSB; // [NI]
  uint64_t* c_full = drain + C::NI;     // FP8: [NSTF] codes landed
  uint64_t* c_empty = c_full + C::NSTF;
  uint64_t* i_full = c_empty + C::NSTF; // [NIT] item written
  uint64_t* i_empty = i_full + C::NIT;  // [NIT] every other warp is done with it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(i_empty + C::NIT);
  PxItem* items = reinterpret_cast<PxItem*>(smem + C::OFF_ITEM);
  static_assert(sizeof(PxItem) == 48, "ring of items");
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* status = &g_status_prefix_tc;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, C::NI);
    mbar_init(q_cvt, C::N_CVT);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&kv_full[i], FP8 ? C::N_CVT : 1);
      mbar_init(&kv_empty[i], C::NI);
    }
    for (int t = 0; t < NT * NSB; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&pv_done[t], 1);
    }
    for (int i = 0; i < C::NI; ++i) mbar_init(&drain[i], 1);
    for (int i = 0; i < C::NSTF; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], C::N_CVT);
    }
    for (int i = 0; i < C::NIT; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], C::THREADS / 32 - 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  // all of the above overlaps the plan's launch; the next launch of the chain
  // may start as this one's blocks end
  grid_dependency_wait();
  grid_launch_dependents();
  // the groups' tables in shared memory: every role looks every item up
  int32_t* gs = reinterpret_cast<int32_t*>(smem + C::OFF_GRP);
  const bool staged = p.groups <= C::GRP_CAP;
  const int32_t *gq = p.grp_q, *gk = p.grp_k, *gp = p.grp_pages, *gu = p.grp_unit;
  if (staged) {
    for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) {
      gs[i] = gq[i];
      gs[C::GRP_CAP + 1 + i] = gk[i];
      gs[2 * (C::GRP_CAP + 1) + i] = gp[i];
      gs[3 * (C::GRP_CAP + 1) + i] = gu[i];
    }
    gq = gs;
    gk = gs + C::GRP_CAP + 1;
    gp = gs + 2 * (C::GRP_CAP + 1);
    gu = gs + 3 * (C::GRP_CAP + 1);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // A wait that gives up in any lane makes the whole warp leave its loop.
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
  };
  // P V of row tile t's step s has completed. One barrier per S buffer: whoever
  // waits for step s knows that step s - NSB has completed, which is what a
  // wait by parity needs to know.
  auto pv_wait = [&](int t, int s) -> bool {
    return wwait(&pv_done[t * NSB + s % NSB], (s / NSB) & 1);
  };
  // Item number k of the ring; its n is -1 behind the last one.
  auto item_wait = [&](int k) -> bool { return wwait(&i_full[k % C::NIT], (k / C::NIT) & 1); };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&i_empty[k % C::NIT]);
  };
  int g_prod = 0, qi_prod = 0;   // producer: K/V tiles and Q loads issued

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    const bool leader = (lane == 0);
    const uint64_t policy = policy_evict_last();   // the row blocks of a group re-read the keys
    const uint32_t q_bytes = static_cast<uint32_t>(C::NSUB * 128 * p.G * p.QB);
    const int nbox = KT / p.box_rows;
    const int skip_tile = hook_skip_tile();
    int g = 0, qi = 0;
    bool ok = true;
    PxCursor<KT, NT> cur;
    cur.start(p, gq, gk, gp, gu);
    for (int k = 0; ok; ++k) {
      PxItem t{};
      const bool more = cur.more();
      if (more) t = cur.next(p, lane);
      else t.n = -1;
      if (!wwait(&i_empty[k % C::NIT], ((k / C::NIT) & 1) ^ 1)) break;
      if (leader) {
        items[k % C::NIT] = t;
        mbar_arrive(&i_full[k % C::NIT]);
      }
      __syncwarp();
      if (!more) break;
      if (leader && t.keys > t.pages * p.page_size) atomicExch(status, SINKATTN_BAD_LENGTHS);
      if (t.n == 0) continue;
      PageCursor pc;   // (its loads are in flight while Q's turn comes)
      pc.start(p.page_indices + t.list0, t.pages, t.first / p.page_size, lane);
      if (qi > 0 && !wwait(q_empty, (qi - 1) & 1)) break;
      if (leader) {
        mbar_arrive_expect_tx(q_full, q_bytes * t.tiles);
        for (int tt = 0; tt < t.tiles; ++tt)
#pragma unroll
          for (int sub = 0; sub < C::NSUB; ++sub)
            tc::tma_load_3d(smem + tt * C::Q_TILE + sub * C::QSUB, &tmQ, sub * 64, t.kvh * p.G,
                            t.tok0 + tt * p.QB, q_full);
      }
      ++qi;
      for (int j = 0; j < t.n; ++j, ++g) {
        const int st = g % (FP8 ? C::NSTF_MOD : NST);
        uint64_t* full = FP8 ? &c_full[st] : &kv_full[st];
        if (!wwait(FP8 ? &c_empty[st] : &kv_empty[st],
                   ((g / (FP8 ? C::NSTF_MOD : NST)) & 1) ^ 1)) {
          ok = false;
          break;
        }
        if (g == skip_tile) continue;   // test hook: the waits for this tile run out
        if (leader) mbar_arrive_expect_tx(full, FP8 ? C::CODE_STAGE : C::STAGE);
        // one box per page segment, lane i issuing box i: rows (page, head, slot) of the pool
        const int j0 = t.first + j * KT;
        const int a = j0 + min(lane, nbox - 1) * p.box_rows;
        const int page = pc.get(j0 / p.page_size, a / p.page_size, lane);
        __syncwarp();   // (the expected bytes are announced before any lane's copy)
        if (lane < nbox) {
          // (boxes behind the prefix come as zeros, from a row before the pool: what lies
          // there is one sequence's own, and its infinities and NaN with it)
          const int row = a < t.keys ? (page * p.Hkv + t.kvh) * p.page_size + a % p.page_size
                                     : -p.box_rows;
          if constexpr (FP8) {
            uint8_t* codes = smem + C::OFF_CODE + st * C::CODE_STAGE + (a - j0) * D;
            tma_load_2d_hint(codes, &tmK, 0, row, full, policy);
            tma_load_2d_hint(codes + KT * D, &tmV, 0, row, full, policy);
          } else {
            uint8_t* kt = smem + C::OFF_KV + st * C::STAGE + (a - j0) * 128;
#pragma unroll
            for (int sub = 0; sub < C::NSUB; ++sub) {
              tma_load_2d_hint(kt + sub * C::KVSUB, &tmK, sub * 64, row, full, policy);
              tma_load_2d_hint(kt + C::KV_TILE + sub * C::KVSUB, &tmV, sub * 64, row, full, policy);
            }
          }
        }
      }
    }
    g_prod = g;
    qi_prod = qi;
  } else if (warp == 1 || (C::NI == 2 && warp == C::W_MMA1)) {
    // --------------------------------------------------------------- MMA issuers
    // The whole warp runs the schedule; one elected lane issues. Issuer i has
    // row tile i, or the one issuer both.
    const int me = warp == 1 ? 0 : 1;
    const bool leader = tc::elect_one();
    constexpr uint32_t idesc_s =
        FP8 ? tc::idesc_f16_f32(128, KT, false) : tc::idesc_bf16_f32(128, KT, false);
    constexpr uint32_t idesc_o =
        FP8 ? tc::idesc_f16_f32(128, D, true) : tc::idesc_bf16_f32(128, D, true);
    constexpr uint64_t STAGE16 = C::STAGE >> 4, QSUB16 = C::QSUB >> 4, KVSUB16 = C::KVSUB >> 4;
    const uint64_t qd0 = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t kd0 = tc::smem_desc_sw128(smem_u32(smem + C::OFF_KV), 16, 1024);
    const uint64_t vd0 = tc::smem_desc_sw128(smem_u32(smem + C::OFF_KV + C::KV_TILE),
                                             static_cast<uint32_t>(C::KVSUB), 1024);
    auto commit1 = [&](uint64_t* bar) {
      if (leader) tc::commit(bar);
      __syncwarp();
    };
    // S_t of K/V tile g into buffer b of the row tile
    auto issue_s = [&](int t, int b, int g) {
      const uint64_t kd = kd0 + static_cast<uint64_t>(g % NST) * STAGE16;
      const uint64_t qd = qd0 + static_cast<uint64_t>(t) * (C::Q_TILE >> 4);
      const uint32_t d_tm = tmem + C::col_s(0, 0) + static_cast<uint32_t>((t * NSB + b) * KT);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t s = static_cast<uint64_t>(kk & 3) * 2;
          tc::mma_ss(d_tm, qd + static_cast<uint64_t>(kk >> 2) * QSUB16 + s,
                     kd + static_cast<uint64_t>(kk >> 2) * KVSUB16 + s, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc::commit(&s_full[t * NSB + b]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int b, int g, bool first) {
      const uint64_t vd = vd0 + static_cast<uint64_t>(g % NST) * STAGE16;
      const uint32_t a_tm = tmem + C::col_s(0, 0) + static_cast<uint32_t>((t * NSB + b) * KT);
      const uint32_t d_tm = tmem + C::col_o(0) + static_cast<uint32_t>(t * D);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          tc::mma_ts(d_tm, a_tm + kk * 8, vd + static_cast<uint64_t>(kk) * 128u, idesc_o,
                     (!first || kk > 0) ? 1u : 0u);
        tc::commit(&pv_done[t * NSB + b]);
      }
      __syncwarp();
    };
    // all P V up to step s - 1 of the row tile have completed
    auto pv_before = [&](int t, int s) -> bool {
      return s <= 0 || pv_wait(t, s - 1);
    };
    auto kv_wait = [&](int g) -> bool { return wwait(&kv_full[g % NST], (g / NST) & 1); };
    int g = 0, qi = 0;
    bool ok = true;
    if constexpr (C::NI == 2) {
      // Two S buffers: S of the next K/V tile goes out before this step's P
      // is there, into the buffer where the step before left its P.
      int steps = 0;   // P V steps of the row tile so far: buffers and phases go by it
      for (int k = 0; ok && item_wait(k); ++k) {
        const int n = items[k % C::NIT].n, tiles = items[k % C::NIT].tiles;
        item_done(k);
        if (n < 0) break;
        if (n == 0) continue;
        ok = wwait(FP8 ? q_cvt : q_full, qi & 1);
        ++qi;
        if (me >= tiles) {
          // no rows: this issuer's share of the barriers, in step with the tiles
          if (ok && lane == 0) mbar_arrive(q_empty);
          __syncwarp();
          for (int j = 0; ok && j < n; ++j) {
            ok = kv_wait(g + j);
            if (ok && lane == 0) mbar_arrive(&kv_empty[(g + j) % NST]);
            __syncwarp();
          }
          g += n;
          continue;
        }
        if (!ok || !kv_wait(g) || !pv_before(me, steps)) { ok = false; break; }
        tc::fence_after_sync();
        issue_s(me, steps % NSB, g);
        if (n == 1) commit1(q_empty);
        for (int j = 0; j < n; ++j, ++g, ++steps) {
          if (j + 1 < n) {
            if (!kv_wait(g + 1) || !pv_before(me, steps)) { ok = false; break; }
            tc::fence_after_sync();
            issue_s(me, (steps + 1) % NSB, g + 1);
            if (j + 2 == n) commit1(q_empty);
          }
          if (!wwait(&p_full[me * NSB + steps % NSB], (steps / NSB) & 1)) { ok = false; break; }
          tc::fence_after_sync();
          issue_pv(me, steps % NSB, g, j == 0);
          commit1(&kv_empty[g % NST]);
        }
      }
    } else {
      // One S buffer: per K/V tile and row tile P V, then the next S into the
      // same buffer once that P V has completed (S overwrites P).
      int steps[NT];
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) steps[tt] = 0;
      for (int k = 0; ok && item_wait(k); ++k) {
        const int n = items[k % C::NIT].n, tiles = items[k % C::NIT].tiles;
        item_done(k);
        if (n < 0) break;
        if (n == 0) continue;
        ok = wwait(FP8 ? q_cvt : q_full, qi & 1) && kv_wait(g);
        ++qi;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
          if (!ok || tt >= tiles) break;
          if (!pv_before(tt, steps[tt])) { ok = false; break; }
          tc::fence_after_sync();
          issue_s(tt, 0, g);
        }
        if (!ok) break;
        if (n == 1) commit1(q_empty);
        for (int j = 0; ok && j < n; ++j) {
          const int gg = g + j;
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) {
            if (tt >= tiles) break;
            if (!wwait(&p_full[tt], steps[tt] & 1)) { ok = false; break; }
            tc::fence_after_sync();
            issue_pv(tt, 0, gg, j == 0);
            if (tt == tiles - 1) commit1(&kv_empty[gg % NST]);
            ++steps[tt];
            if (j + 1 < n) {
              if ((tt == 0 && !kv_wait(gg + 1)) || !pv_before(tt, steps[tt])) { ok = false; break; }
              tc::fence_after_sync();
              issue_s(tt, 0, gg + 1);
              if (j + 2 == n && tt == tiles - 1) commit1(q_empty);
            }
          }
        }
        g += n;
      }
    }
    // every MMA this warp issued has completed before the block frees TMEM
    commit1(&drain[me]);
    mbar_drain(&drain[me], 0);
  } else if (FP8 && warp >= C::W_CVT) {
    // ------------------------------------------------------------ converters
    // Per item Q in place, bf16 -> f16; per K/V tile 16-byte runs of codes ->
    // f16 in the tile ring. Generic-proxy writes that the tensor core reads:
    // fenced before each hand-over.
    constexpr int N = C::N_CVT * 32;
    constexpr int RUNS_ROW = D / 16, RUNS = 2 * KT * RUNS_ROW, PER = RUNS / N;
    static_assert(RUNS % N == 0, "whole runs per converter thread");
    const int ct = static_cast<int>(threadIdx.x) - C::W_CVT * 32;
    int g = 0, qi = 0;
    bool ok = true;
    for (int k = 0; ok && item_wait(k); ++k) {
      const int n = items[k % C::NIT].n, tiles = items[k % C::NIT].tiles;
      item_done(k);
      if (n < 0) break;
      if (n == 0) continue;
      if (!wwait(q_full, qi & 1)) break;
      for (int c = ct; c < tiles * C::Q_TILE / 16; c += N) {
        uint4 w = *reinterpret_cast<const uint4*>(smem + c * 16);
        w.x = pack_f16x2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        w.y = pack_f16x2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
        w.z = pack_f16x2(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u));
        w.w = pack_f16x2(__uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u));
        *reinterpret_cast<uint4*>(smem + c * 16) = w;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_cvt);
      ++qi;
      for (int j = 0; j < n; ++j, ++g) {
        const int sc = g % C::NSTF_MOD, st = g % NST;
        if (!wwait(&c_full[sc], (g / C::NSTF_MOD) & 1)) { ok = false; break; }
        const uint8_t* codes = smem + C::OFF_CODE + sc * C::CODE_STAGE;
        uint8_t* dst = smem + C::OFF_KV + st * C::STAGE;
        uint4 w[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
          w[i] = *reinterpret_cast<const uint4*>(codes + (ct + i * N) * 16);   // [K | V][KT][D]
        __syncwarp();
        if (lane == 0) mbar_arrive(&c_empty[sc]);
        if (!wwait(&kv_empty[st], ((g / NST) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int c = ct + i * N;
          const int tensor = c / (KT * RUNS_ROW);   // 0: K, 1: V
          const int rem = c - tensor * (KT * RUNS_ROW);
          const int row = rem / RUNS_ROW, cb = rem % RUNS_ROW;
          uint4 h0, h1;
          h0.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].x));
          h0.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].x >> 16));
          h0.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].y));
          h0.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].y >> 16));
          h1.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].z));
          h1.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].z >> 16));
          h1.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].w));
          h1.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].w >> 16));
          uint8_t* sub = dst + tensor * C::KV_TILE + (cb >> 2) * C::KVSUB;
          const int ch = (cb & 3) * 2;
          *reinterpret_cast<uint4*>(sub + sw128_offset(row, ch)) = h0;
          *reinterpret_cast<uint4*>(sub + sw128_offset(row, ch + 1)) = h1;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[st]);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int tt = (warp - 2) >> 2;  // row tile
    const int quad = warp & 3;       // TMEM lane quadrant this warp may access
    const int row = quad * 32 + lane;
    const int G = p.G;
    const int rg = row / G;          // token within the tile
    const int hig = row - rg * G;    // head within the group
    const int tl = tt * p.QB + rg;   // token within the block
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr0 = lane_base + C::col_s(tt, 0);
    const uint32_t o_addr = lane_base + C::col_o(tt);
    constexpr int NCH = KT / 32;     // 32-column pieces of a score row
    int steps = 0;
    bool ok = true;
    for (int k = 0; ok && item_wait(k); ++k) {
      const PxItem& t = items[k % C::NIT];   // (shared memory: read where needed)
      const int n = t.n;
      if (n < 0 || tt >= t.tiles) {
        item_done(k);
        if (n < 0) break;
        continue;
      }
      const bool valid = rg < p.QB && tl < t.nq;
      const float kscale = FP8 ? p.k_scale[t.kvh] : 1.f;
      const float c2 = p.scale_log2 * kscale;   // raw logits -> base-2 exponents
      int lo_r = 0;
      if (p.window > 0 && valid) lo_r = max(0, p.row_pos[t.tok0 + tl] - p.window + 1);
      // the row's first and last visible key, from the first column of the tile
      int clo = lo_r - t.first, chi = t.keys - 1 - t.first;
      float m_used = kNegInf, l = 0.f, lag = 0.f;   // lag: l' - l
      for (int j = 0; j < n; ++j, ++steps, clo -= KT, chi -= KT) {
        const int b = steps % NSB;
        if (!wwait(&s_full[tt * NSB + b], (steps / NSB) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t s_addr = s_addr0 + static_cast<uint32_t>(b * KT);
        float v[NCH][32];
#pragma unroll
        for (int c = 0; c < NCH; ++c) tc::tmem_ld32(s_addr + 32 * c, v[c]);
        tc::tmem_wait_ld();
        if (clo > 0 || chi < KT - 1) {
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const int lo_c = clo - c * 32, hi_c = chi - c * 32;
            if (lo_c <= 0 && hi_c >= 31) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e < lo_c || e > hi_c) v[c][e] = kNegInf;
          }
        }
        // row maximum: 2 NCH independent chains of three-input maxima
        float mxc[2 * NCH];
#pragma unroll
        for (int i = 0; i < 2 * NCH; ++i)
          mxc[i] = fmaxf(v[i >> 1][(i & 1) * 16], v[i >> 1][(i & 1) * 16 + 1]);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int e = 2; e < 16; e += 2) {
            mxc[2 * c] = fmax3(mxc[2 * c], v[c][e], v[c][e + 1]);
            mxc[2 * c + 1] = fmax3(mxc[2 * c + 1], v[c][16 + e], v[c][16 + e + 1]);
          }
        float mx = fmax3(mxc[0], mxc[1], mxc[2]);
#pragma unroll
        for (int i = 3; i < 2 * NCH; i += 2)
          mx = (i + 1 < 2 * NCH) ? fmax3(mx, mxc[i], mxc[i + 1]) : fmaxf(mx, mxc[i]);

        // the reference moves only when the maximum is past it by more than
        // 2^8, or O_t, which the tensor core holds, would be rescaled in
        // almost every step by one row or another of the warp
        float alpha = 1.f;
        bool rescale = false;
        if (m_used == kNegInf ? mx > m_used : (mx - m_used) * c2 > 8.f) {
          alpha = (m_used == kNegInf) ? 0.f : ex2((m_used - mx) * c2);
          m_used = mx;
          rescale = true;
        }
        const float mb = (m_used == kNegInf) ? 0.f : m_used * c2;
        if constexpr (!FP8) {   // the step's largest weight, by the arithmetic of P below
          const float top = ex2(fmaf(mx, c2, -mb));
          lag = lag * alpha + (__bfloat162float(__float2bfloat16_rn(top)) - top);
        }

        // P = 2^(s c2 - mb) into the first KT / 2 columns of this S buffer
        // (all scores are in registers); scale-subtract and the exact sum
        // run two lanes per instruction.
        const float2 c2x2 = make_float2(c2, c2), nmb2 = make_float2(-mb, -mb);
        float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int k = hh * 16 + e;
              const float2 x = __ffma2_rn(make_float2(v[c][k], v[c][k + 1]), c2x2, nmb2);
              const float2 a = make_float2(ex2(x.x), ex2(x.y));
              rs2[(e >> 1) & 3] = __fadd2_rn(rs2[(e >> 1) & 3], a);
              pk[e >> 1] = FP8 ? pack_f16x2(a.x, a.y) : pack_bf16x2(a.x, a.y);
            }
            tc::tmem_st8(s_addr + 16 * c + 8 * hh, pk);
          }
        const float2 rsa = __fadd2_rn(__fadd2_rn(rs2[0], rs2[1]), __fadd2_rn(rs2[2], rs2[3]));

        // Rescale O_t when some row of this warp moved its reference
        // (warp-uniform branch), once the previous step's PV_t has completed.
        if (j >= 1 && __any_sync(0xffffffffu, rescale)) {
          if (!pv_wait(tt, steps - 1)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::tmem_ld32(o_addr + c * 32, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tc::tmem_st32(o_addr + c * 32, o);
          }
        }
        tc::tmem_wait_st();
        l = l * alpha + (rsa.x + rsa.y);
        tc::fence_before_sync();
        mbar_arrive(&p_full[tt * NSB + b]);
      }
      if (!ok) break;
      // O_t is read out before this thread hands over P of the next item, so
      // the next item's first PV (which overwrites O_t) comes after it.
      if (n >= 1) {
        if (!pv_wait(tt, steps - 1)) { ok = false; break; }
        tc::fence_after_sync();
      }
      const bool some = l != 0.f;   // the row sees a key of the chunk (or a NaN)
      const float lr = l + lag;
      const size_t slot =
          (static_cast<size_t>(t.tok0 + tl) * p.Hq + t.kvh * G + hig) * p.part_slots + t.slot;
      if (n >= 1)
        store_partial<D>(o_addr, FP8 ? p.v_scale[t.kvh] : 1.f, p.part_acc + slot * D, valid, lane);
      tc::fence_before_sync();
      if (valid) {
        float2* md = reinterpret_cast<float2*>(p.part_md + slot * 2);
        const float shift = FP8 ? 0.f : (lg2(l) - lg2(lr)) * kLn2;
        *md = some ? make_float2(m_used * (p.sm_scale * kscale) + shift, lr)
                   : make_float2(kNegInf, 0.f);
        if (t.last)   // the partials that no block writes
          for (int s = t.slot + 1; s < p.splits; ++s) md[s - t.slot] = make_float2(kNegInf, 0.f);
      }
      item_done(k);
    }
    // rows of groups without a prefix: no block has units of theirs. All
    // warps share the rows of each group, or with many groups the groups.
    const int warps = static_cast<int>(gridDim.x) * NT * 4;
    const int me = static_cast<int>(blockIdx.x) * NT * 4 + (warp - 2);
    const bool many = p.groups > warps;
    const int width = (many ? 1 : warps) * 32;
    const int mine = (many ? 0 : me) * 32 + lane;
    for (int g = many ? me : 0; g < p.groups; g += many ? warps : 1) {
      if (gk[g + 1] > gk[g]) continue;
      const long long n = static_cast<long long>(gq[g + 1] - gq[g]) * p.Hq * p.splits;
      for (long long i = mine; i < n; i += width) {
        const long long r = static_cast<long long>(gq[g]) * p.Hq + i / p.splits;
        *reinterpret_cast<float2*>(p.part_md + (r * p.part_slots + i % p.splits) * 2) =
            make_float2(kNegInf, 0.f);
      }
    }
  }

  // a warp that left its loop early may still have TMEM loads or stores in flight
  tc::tmem_wait_ld();
  tc::tmem_wait_st();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // a wait gave up: let every issued copy land before the block's shared
    // memory goes away (a left-out tile's phase never completes: bounded)
    if (qi_prod > 0) mbar_drain(q_full, (qi_prod - 1) & 1);
    constexpr int R = FP8 ? C::NSTF_MOD : NST;
    for (int i = max(0, g_prod - R); i < g_prod; ++i)
      mbar_drain(FP8 ? &c_full[i % R] : &kv_full[i % R], (i / R) & 1);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool FP8>
int launch(const AttnArgs& a, const SharedPlan& plan, cudaStream_t stream) {
  using C = PxCfg<D, FP8>;
  const int G = a.Hq / a.Hkv, QB = 128 / G;
  CUtensorMap tmQ, tmK, tmV;
  int rc = make_q_tmap(&tmQ, a.q, static_cast<uint64_t>(a.total_q), a.Hq, D, G, QB);
  if (rc) return rc;
  const uint64_t rows = kv_map_rows(a);
  const int box = kv_box_rows(a, C::KT);
  rc = FP8 ? make_rows_tmap_u8(&tmK, a.k, rows, D, box) : make_rows_tmap(&tmK, a.k, rows, D, box, 128);
  if (rc) return rc;
  rc = FP8 ? make_rows_tmap_u8(&tmV, a.v, rows, D, box) : make_rows_tmap(&tmV, a.v, rows, D, box, 128);
  if (rc) return rc;
  PxParams p{};
  p.grp_q = plan.grp_q;
  p.grp_k = plan.grp_k;
  p.grp_pages = plan.grp_pages;
  p.grp_unit = plan.grp_unit;
  p.quota = plan.quota;
  p.row_pos = plan.row_pos;
  p.page_indices = a.page_indices;
  p.groups = a.batch;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = G;
  p.QB = QB;
  p.splits = a.num_splits;
  p.window = a.window;
  p.sm_scale = a.sm_scale;
  p.scale_log2 = a.sm_scale * kLog2e;
  p.page_size = a.page_size;
  p.box_rows = box;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.part_acc = a.part_acc;
  p.part_md = a.part_md;
  p.part_slots = part_slots(a);
  // row blocks: at most one per group more than its full ones (units below 2^31: the caller checks)
  const int64_t tiles = (a.max_kv + C::KT - 1) / C::KT;
  const int64_t units = (a.batch + a.total_q / (C::NT * QB)) * a.Hkv * tiles;
  auto kern = prefix_tc_kernel<D, FP8>;
  cudaError_t e = set_chained_smem(kern, C::SMEM);
  if (e == cudaSuccess) {
    e = launch_chained(kern, dim3(static_cast<unsigned>(std::min<int64_t>(units, sm_count()))),
                       C::THREADS, C::SMEM, stream, tmQ, tmK, tmV, p);
  }
  if (e != cudaSuccess) {
    set_error("shared-prefix kernel launch: %s", cudaGetErrorString(e));
    return SINKATTN_CUDA_ERROR;
  }
  return SINKATTN_OK;
}

}  // namespace

int prefix_block_tokens(int G) { return 2 * (128 / G); }
int prefix_tile_keys(int d, bool fp8) {
  if (d == 64) return PxCfg<64, false>::KT;
  return fp8 ? PxCfg<128, true>::KT : PxCfg<128, false>::KT;
}

int launch_prefix_tc(const AttnArgs& a, const SharedPlan& plan, cudaStream_t stream) {
  if (a.d == 64) return a.kv_fp8 ? launch<64, true>(a, plan, stream) : launch<64, false>(a, plan, stream);
  return a.kv_fp8 ? launch<128, true>(a, plan, stream) : launch<128, false>(a, plan, stream);
}

SINKATTN_DEFINE_SET_HOOKS(set_hooks_prefix_tc)

int read_status_prefix_tc(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_prefix_tc, sizeof(int), 0,
                                cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  if (cudaMemcpyToSymbolAsync(g_status_prefix_tc, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                              s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn
