// Page tables of a paged KV cache, and the copies of whole or partly filled
// pages that they ask for (layout and rules: sinkattn.h).
//
// The table's work is integer work on a few kilobytes to megabytes, so time
// is launch and memory latency, not bandwidth. Each call is one launch of one
// thread-block cluster: its phases (check, count, rank, commit) are separated
// by cluster barriers of a fraction of a microsecond, where separate launches
// would cost two microseconds each, and nothing has to be read back by the
// host, so every call can be captured into a graph. A call with up to
// kOneBlock entries runs as one block, larger ones as a cluster of kCluster.
// Before the first barrier a call checks and writes scratch; one that cannot
// be served as a whole ends there, with the table unchanged. (Reserve takes its
// pages off the free count there, by the thread that has the check's result.)
//
// No result depends on the order in which atomics arrive: they only count,
// or elect a page's first writer or first appearance by its position (a
// maximum), and ranks come from ordered scans.
//
// Page copies follow as a second launch over the whole GPU that reads the
// pairs the first one found (a programmatic dependent, so its start-up
// overlaps the first launch's end).
//
// Measured, calls back to back: a small reserve, fork or truncate 3 to 5 us;
// freeing 256 of 512 sequences of up to 8000 tokens (50000 counts) 20 us;
// packing a pool of four layers (1.6 GB of reads and writes) 260 us, the moves
// alone 6.4 TB/s.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_pages;

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 16;         // blocks of a large call (the hardware's limit)
// Entries that one block takes alone: 22000 new tokens took 36 us with one block
// (append and table copy included), 23 with the cluster, eight forks of 16 lists
// 31 and 21; 64 tokens 10.8 and 12.0, packing a small pool 7.8 and 10.1.
constexpr int kOneBlock = 4096;
constexpr int kHeader = 16;
constexpr int kRun = 8;              // list entries of a thread, whose loads are in flight together
constexpr int kKept = 1024;          // sequences of a call whose ranges stay in shared memory

// Header words besides the free count (scratch of one call).
enum { H_FREE = 0, H_OK = 1, H_COUNT = 2, H_PAIRS = 3 };

struct PageTab {
  int32_t* base;
  int N, P, S, M, shift;   // pages, page size (= 1 << shift), sequences, pages per sequence
  __device__ __forceinline__ int32_t* hdr() const { return base; }
  __device__ __forceinline__ int32_t* lens() const { return base + kHeader; }
  __device__ __forceinline__ int32_t* list() const { return lens() + S; }
  __device__ __forceinline__ int32_t* rc() const { return list() + static_cast<size_t>(S) * M; }
  __device__ __forceinline__ int32_t* free_list() const { return rc() + N; }
  __device__ __forceinline__ int32_t* aux(int k) const {   // k < 7: one word per sequence
    return free_list() + N + static_cast<size_t>(S) * k;
  }
  __device__ __forceinline__ int32_t* work(int k) const {  // k < 2: one word per page
    return aux(7) + static_cast<size_t>(N) * k;
  }
  __device__ __forceinline__ int pages(int tokens) const { return (tokens + P - 1) >> shift; }
  __device__ __forceinline__ bool seq_ok(int id) const {
    return static_cast<unsigned>(id) < static_cast<unsigned>(S);
  }
  __device__ __forceinline__ bool page_ok(int p) const {
    return static_cast<unsigned>(p) < static_cast<unsigned>(N);
  }
};

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// Exclusive sum over the block's threads; *total gets the sum. Every thread
// of the block calls it; `sums` is 32 words of shared memory.
__device__ __forceinline__ int block_scan(int v, int* total, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();   // the last call's sums have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int w = sums[lane];   // kThreads / 32 == 32 warps
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int upto = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? upto : 0) + x - v;
}

// Which sequences a call names: one bit each in dynamic shared memory.
extern __shared__ uint32_t seen_s[];

__device__ __forceinline__ void seen_clear(const PageTab& t) {
  for (int i = threadIdx.x; i < (t.S + 31) / 32; i += kThreads) seen_s[i] = 0u;
}
// Marks `id` (in range); true if it was marked before.
__device__ __forceinline__ bool seen_twice(int id) {
  const uint32_t bit = 1u << (id & 31);
  return atomicOr(&seen_s[id >> 5], bit) & bit;
}
__device__ __forceinline__ bool seen(int id) { return seen_s[id >> 5] >> (id & 31) & 1u; }

// Sum of *word (one per block of the cluster, written before the last cluster
// barrier) over all blocks and over those before this one. The words must
// stay until a later cluster barrier.
__device__ __forceinline__ int cluster_sum(const int* word, int rank, int nr, int* before) {
  int all = 0, low = 0;
  if (nr == 1) {
    *before = 0;
    __syncthreads();
    return *word;
  }
  for (int r = 0; r < nr; ++r) {
    const int x = __float_as_int(ld_dsmem(reinterpret_cast<const float*>(word), r));
    low += r < rank ? x : 0;
    all += x;
  }
  *before = low;
  return all;
}

// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) pages_init_kernel(const PageTab t) {
  const long long n = static_cast<long long>(t.S) * t.M;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t0 < kHeader) t.hdr()[t0] = t0 == H_FREE ? t.N : 0;
  for (long long i = t0; i < t.S; i += step) t.lens()[i] = 0;
  for (long long i = t0; i < n; i += step) t.list()[i] = -1;
  for (long long i = t0; i < t.N; i += step) {
    t.rc()[i] = 0;
    t.free_list()[i] = t.N - 1 - static_cast<int>(i);
  }
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
struct ReserveItem {
  int id, len, grow, tail, rc;   // tail: the shared page the new tokens start in, or -1
  bool ok;
};

__device__ __forceinline__ ReserveItem reserve_item(const PageTab& t, const int32_t* ids,
                                                    const int32_t* cu, int i) {
  ReserveItem r;
  r.id = ids[i];
  const int c0 = cu[i], c1 = cu[i + 1];
  r.ok = t.seq_ok(r.id) && c1 >= c0 && c0 >= 0;
  r.grow = r.ok ? c1 - c0 : 0;
  r.len = r.ok ? t.lens()[r.id] : 0;
  r.ok = r.ok && r.len >= 0 &&
         static_cast<long long>(r.len) + r.grow <= static_cast<long long>(t.M) * t.P;
  r.tail = -1;
  r.rc = 0;
  if (r.ok && r.grow > 0 && (r.len & (t.P - 1))) {
    const int p = t.list()[static_cast<size_t>(r.id) * t.M + (r.len >> t.shift)];
    r.ok = t.page_ok(p);
    if (r.ok) {
      r.rc = t.rc()[p];
      if (r.rc > 1) r.tail = p;
    }
  }
  return r;
}

// aux(0): rank of the item's first new page among the call's pages (its
// copied page, if any, is the one before); aux(1): its length before the
// call; aux(2): 1 if its tail page is copied; aux(3 .. 5): the copies'
// (source, destination, rows).
__global__ void __launch_bounds__(kThreads)
    pages_reserve_kernel(const PageTab t, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ cu, int n, int total_new,
                         int32_t* __restrict__ slots) {
  __shared__ int sums[32];
  __shared__ int kept_s[3][kKept];
  __shared__ int ok_s, count_s;
  const int tid = threadIdx.x;
  int32_t* hdr = t.hdr();
  // one block: what the second half reads of an item stays in shared memory
  const bool alone = cluster_size() == 1;
  int* first_of = alone && n <= kKept ? kept_s[0] : t.aux(0);
  int* len_of = alone && n <= kKept ? kept_s[1] : t.aux(1);
  int* copy_of = alone && n <= kKept ? kept_s[2] : t.aux(2);
  if (cluster_rank() == 0) {
    // the first item of each thread stays in registers
    ReserveItem mine{};
    if (tid < n) mine = reserve_item(t, ids, cu, tid);
    seen_clear(t);
    __syncthreads();
    bool bad = false, shared = false;
    for (int i = tid; i < n; i += kThreads) {
      const ReserveItem r = i == tid ? mine : reserve_item(t, ids, cu, i);
      if (!r.ok || seen_twice(r.id)) bad = true;
      if (r.tail >= 0) {
        shared = true;
        t.work(0)[r.tail] = t.work(1)[r.tail] = 0;
      }
    }
    if (__syncthreads_or(shared)) {
      for (int i = tid; i < n; i += kThreads) {
        const ReserveItem r = i == tid ? mine : reserve_item(t, ids, cu, i);
        if (r.tail >= 0) {
          atomicAdd(&t.work(0)[r.tail], 1);       // writers of the page in this call
          atomicMax(&t.work(1)[r.tail], n - i);   // the first of them
        }
      }
      __syncthreads();
    }
    long long need = 0;
    for (int base = 0; base < n; base += kThreads) {
      const int i = base + tid;
      int want = 0, copies = 0;
      if (i < n) {
        const ReserveItem r = base == 0 ? mine : reserve_item(t, ids, cu, i);
        if (r.ok) {
          copies = r.tail >= 0 && !(__ldcg(&t.work(0)[r.tail]) == r.rc &&
                                    __ldcg(&t.work(1)[r.tail]) == n - i);
          want = t.pages(r.len + r.grow) - t.pages(r.len) + copies;
          len_of[i] = r.len;
          copy_of[i] = copies;
        }
      }
      int total;
      const int before = block_scan(want, &total, sums);
      // (a call that needs 2^31 pages has failed long before: need is exact)
      if (i < n) first_of[i] = static_cast<int>(need) + before + copies;
      need += total;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      const int count = hdr[H_FREE];
      int status = SINKATTN_OK;
      if (cu[0] != 0 || cu[n] != total_new) status = SINKATTN_BAD_LENGTHS;
      else if (bad || count < 0 || count > t.N) status = SINKATTN_BAD_PAGES;
      else if (need > count) status = SINKATTN_OUT_OF_PAGES;
      if (status) atomicExch(&g_status_pages, status);
      ok_s = hdr[H_OK] = status == SINKATTN_OK;
      count_s = hdr[H_COUNT] = count;
      hdr[H_PAIRS] = 0;
      if (!status) hdr[H_FREE] = count - static_cast<int>(need);
    }
  }
  if (alone) __syncthreads();
  else cluster_sync_all();
  const int nt = cluster_size() * kThreads;
  const int t0 = cluster_rank() * kThreads + tid;
  if (!(alone ? ok_s : __ldcg(&hdr[H_OK]))) {
    for (int i = t0; i < total_new; i += nt) slots[i] = -1;
    return;
  }
  const int count = alone ? count_s : __ldcg(&hdr[H_COUNT]);
  int32_t* list = t.list();
  for (int i = t0; i < n; i += nt) {
    const int id = ids[i], len = len_of[i];
    t.lens()[id] = len + (cu[i + 1] - cu[i]);
    if (copy_of[i]) {
      int32_t* entry = &list[static_cast<size_t>(id) * t.M + (len >> t.shift)];
      const int src = *entry, dst = t.free_list()[count - first_of[i]];
      if (!t.page_ok(dst)) continue;   // (a table that was written over: nothing to copy to)
      *entry = dst;
      atomicSub(&t.rc()[src], 1);
      t.rc()[dst] = 1;
      const int k = atomicAdd(&hdr[H_PAIRS], 1);   // (the copies' order does not matter)
      t.aux(3)[k] = src;
      t.aux(4)[k] = dst;
      t.aux(5)[k] = len & (t.P - 1);
    }
  }
  for (int k = t0; k < total_new; k += nt) {
    int lo = 0, hi = n;   // the item with cu[item] <= k < cu[item + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= k) lo = mid;
      else hi = mid;
    }
    const int len = len_of[lo], first = first_of[lo];
    const int pos = len + (k - cu[lo]), e = pos >> t.shift, have = t.pages(len);
    int32_t* row = list + static_cast<size_t>(ids[lo]) * t.M;
    int page;
    if (e < have) {
      page = copy_of[lo] ? t.free_list()[count - first] : row[e];
    } else {
      page = t.free_list()[count - 1 - first - (e - have)];
      if ((pos & (t.P - 1)) == 0 && t.page_ok(page)) {   // a new page's first slot is a new token's
        row[e] = page;
        t.rc()[page] = 1;
      }
    }
    slots[k] = t.page_ok(page) ? page * t.P + (pos & (t.P - 1)) : -1;
  }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every block checks the whole request, so none has to wait for another.
__global__ void __launch_bounds__(kThreads)
    pages_fork_kernel(const PageTab t, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int n) {
  __shared__ int most_s;
  const int tid = threadIdx.x;
  if (tid == 0) most_s = 0;
  seen_clear(t);
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kThreads) {
    const int b = dst[i];
    if (!t.seq_ok(b) || seen_twice(b) || t.lens()[b] != 0) bad = true;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int a = src[i];
    if (!t.seq_ok(a) || seen(a)) {
      bad = true;
      continue;
    }
    const int len = t.lens()[a];
    if (len < 0 || t.pages(len) > t.M) bad = true;
    else atomicMax(&most_s, t.pages(len));
  }
  if (__syncthreads_or(bad)) {
    if (cluster_rank() == 0 && tid == 0) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
    return;   // every block of the cluster
  }
  cluster_sync_all();   // every block has seen the dst sequences empty
  const int most = most_s;
  const int nt = cluster_size() * kThreads;
  const int t0 = cluster_rank() * kThreads + tid;
  for (int i = t0; i < n; i += nt) t.lens()[dst[i]] = t.lens()[src[i]];   // (no src is a dst)
  // (item, entry) pairs over the rectangle n x (longest list)
  const int cells = n * most;   // < max_seqs * max_pages
  for (int c0 = t0; c0 < cells; c0 += kRun * nt) {
    int p[kRun];
    int32_t* to[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const int c = c0 + k * nt;
      to[k] = nullptr;
      if (c >= cells) continue;
      const int i = c / most, e = c - i * most;
      if (e >= t.pages(t.lens()[src[i]])) continue;
      p[k] = t.list()[static_cast<size_t>(src[i]) * t.M + e];
      to[k] = &t.list()[static_cast<size_t>(dst[i]) * t.M + e];
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (!to[k]) continue;
      *to[k] = p[k];
      if (t.page_ok(p[k])) atomicAdd(&t.rc()[p[k]], 1);
    }
  }
}

// ---------------------------------------------------------------------------
// truncate
// ---------------------------------------------------------------------------
// A dropped page that only this list held is free at once. One that other
// lists hold too is counted down, and if nothing is left its first appearance
// in the request (its position is elected in work(0)) gives it back. Scattered
// words are what a block can touch least often (a few per ten cycles), so
// pages of one holder cost one read and one write of their count, shared
// pages five.
//
// Every block checks the whole request and keeps what each item keeps and
// drops, in shared memory for calls of up to kKept sequences, else in aux(0)
// and aux(1), where all blocks write the same words. Cells (item, entry) of the
// rectangle n x (longest drop) are taken in request order: a block has a run
// of them, a warp kRun * 32 consecutive ones at a time, lane by lane, so list
// and free-list accesses are contiguous and ranks are ballots and one scan.
// Where one block's step holds all cells, block 0 goes on alone.
__global__ void __launch_bounds__(kThreads)
    pages_truncate_kernel(const PageTab t, const int32_t* __restrict__ ids,
                          const int32_t* __restrict__ new_lens, int n) {
  constexpr int kStep = kRun * kThreads;
  __shared__ int sums[32];
  __shared__ int most_s, found_s;
  __shared__ int keep_s[kKept], drop_s[kKept];
  const int tid = threadIdx.x, lane = tid & 31, rank = cluster_rank();
  int nr = cluster_size();
  int32_t* hdr = t.hdr();
  int* keep = n <= kKept ? keep_s : t.aux(0);
  int* drop = n <= kKept ? drop_s : t.aux(1);
  if (tid == 0) most_s = 0;
  seen_clear(t);
  const int count = __ldcg(&hdr[H_FREE]);
  __syncthreads();
  bool bad = count < 0 || count > t.N;   // (not a table)
  for (int i = tid; i < n; i += kThreads) {
    const int id = ids[i], to = new_lens ? new_lens[i] : 0;
    if (!t.seq_ok(id) || seen_twice(id)) {
      bad = true;
      continue;
    }
    const int len = __ldcg(&t.lens()[id]);
    if (to < 0 || to > len || t.pages(len) > t.M) {
      bad = true;
      continue;
    }
    const int k = t.pages(to), d = t.pages(len) - k;
    keep[i] = k;
    drop[i] = d;
    if (d > 0) atomicMax(&most_s, d);
  }
  if (__syncthreads_or(bad)) {
    if (rank == 0 && tid == 0) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
    return;   // every block of the cluster
  }
  const int most = most_s;
  const int cells = n * most;        // < max_seqs * max_pages
  const bool alone = cells <= kStep;
  if (nr > 1 && alone) {
    cluster_sync_all();              // every block has read the lengths
    if (rank > 0) return;
    nr = 1;
  }
  const int per = ((cells + nr - 1) / nr + kStep - 1) / kStep * kStep;
  const int c0 = static_cast<int>(min(static_cast<long long>(cells), static_cast<long long>(rank) * per));
  const int c1 = min(cells, c0 + per);
  // A block with one step keeps its cells in registers over the phases, one
  // with more loads them again and takes the shared way for every page.
  const bool single = c1 - c0 <= kStep;
  int at[kRun], page[kRun];   // the entry in words from the first list, its page; -1: none
  uint32_t shared = 0, back = 0;
  int found = 0, before = 0, all = 0, total;
#pragma unroll 1
  for (int phase = 0; phase < 4; ++phase) {
#pragma unroll 1
    for (int base = c0; base < c1; base += kStep) {
      // the thread's cells: its warp's run, lane by lane
      const int first = base + (tid >> 5) * (kRun * 32) + lane;
      if (phase == 0 || !single) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int c = first + k * 32;
          at[k] = -1;
          if (c >= c1) continue;
          const int i = c / most, e = c - i * most;
          if (e < drop[i]) at[k] = ids[i] * t.M + keep[i] + e;
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) page[k] = at[k] >= 0 ? t.list()[at[k]] : -1;
#pragma unroll
        for (int k = 0; k < kRun; ++k) page[k] = t.page_ok(page[k]) ? page[k] : -1;
      }
      if (phase == 0) {          // which pages other lists hold too, before any count changes
        shared = 0xffu;
        if (single) {
          int r[kRun];
#pragma unroll
          for (int k = 0; k < kRun; ++k) r[k] = page[k] >= 0 ? __ldcg(&t.rc()[page[k]]) : 1;
          shared = 0;
#pragma unroll
          for (int k = 0; k < kRun; ++k) shared |= r[k] != 1 ? 1u << k : 0u;
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k)
          if ((shared >> k & 1u) && page[k] >= 0) t.work(0)[page[k]] = 0;
      } else if (phase == 1) {   // count down, elect
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          if (page[k] < 0) continue;
          if (shared >> k & 1u) {
            atomicSub(&t.rc()[page[k]], 1);
            atomicMax(&t.work(0)[page[k]], INT32_MAX - (first + k * 32));
          } else {
            t.rc()[page[k]] = 0;
          }
        }
      } else {                   // who gives a page back (counted in phase 2, written in phase 3)
        if (phase == 2 || !single) {
          int r[kRun], w[kRun];
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            const bool look = page[k] >= 0 && (shared >> k & 1u);
            r[k] = look ? __ldcg(&t.rc()[page[k]]) : 1;
            w[k] = look ? __ldcg(&t.work(0)[page[k]]) : 0;
          }
          back = 0;
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            const bool yes = shared >> k & 1u ? r[k] == 0 && w[k] == INT32_MAX - (first + k * 32)
                                              : page[k] >= 0;
            if (yes) back |= 1u << k;
          }
        }
        // ranks: the warps' sums by a scan (lane 0 carries them), then by lanes within 32 cells
        uint32_t vote[kRun];
        int sum = 0;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          vote[k] = __ballot_sync(0xffffffffu, back >> k & 1u);
          sum += __popc(vote[k]);
        }
        int r = block_scan(lane == 0 ? sum : 0, &total, sums);
        if (phase == 2) {
          found += total;
        } else {
          r = before + __shfl_sync(0xffffffffu, r, 0);
          before += total;
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            if (at[k] >= 0) t.list()[at[k]] = -1;
            if ((back >> k & 1u) && count + all <= t.N)
              t.free_list()[count + all - 1 - r - __popc(vote[k] & ((1u << lane) - 1u))] = page[k];
            r += __popc(vote[k]);
          }
        }
      }
    }
    if (phase == 2 && tid == 0) found_s = found;
    if (phase < 3) {
      if (alone) __syncthreads();
      else cluster_sync_all();
    }
    if (phase == 0) {   // every block has read the lengths and the counts
      for (int i = rank * kThreads + tid; i < n; i += nr * kThreads)
        t.lens()[ids[i]] = new_lens ? new_lens[i] : 0;
      if (most == 0) return;   // uniform: no page leaves a list
    } else if (phase == 2) {
      all = cluster_sum(&found_s, rank, nr, &before);
      if (rank == 0 && tid == 0) hdr[H_FREE] = count + all;
    }
  }
  if (!alone) cluster_sync_all();   // the other blocks have read this one's sum
}

// ---------------------------------------------------------------------------
// compact: ranks of holes and movers, the page map, the counts
// ---------------------------------------------------------------------------
// work(0): the free pages below L in order; work(1): the live pages from L
// on, last first (a live page's rank from the end is L - 1 less the live
// pages before it, which needs no second count).
__global__ void __launch_bounds__(kThreads)
    pages_compact_kernel(const PageTab t, int32_t* __restrict__ page_map) {
  __shared__ int sums[32];
  __shared__ int live_s;
  const int tid = threadIdx.x, rank = cluster_rank(), nr = cluster_size();
  int32_t* hdr = t.hdr();
  const int per = ((t.N + nr - 1) / nr + kThreads - 1) / kThreads * kThreads;
  const int p0 = min(t.N, rank * per), p1 = min(t.N, p0 + per);
  int live = 0;
#pragma unroll 4
  for (int p = p0 + tid; p < p1; p += kThreads) live += t.rc()[p] > 0;
  int total, before;
  block_scan(live, &total, sums);
  if (tid == 0) live_s = total;
  cluster_sync_all();
  const int kept = cluster_sum(&live_s, rank, nr, &before);
  if (rank == 0 && tid == 0) {
    hdr[H_FREE] = t.N - kept;
    if (kept == t.N) hdr[H_PAIRS] = 0;
  }
  for (int base = p0; base < p1; base += kThreads) {
    const int p = base + tid;
    const bool is = p < p1 && t.rc()[p] > 0;
    const int at = before + block_scan(is, &total, sums);   // live pages before p
    before += total;
    if (p >= p1) continue;
    if (p == kept) hdr[H_PAIRS] = kept - at;
    page_map[p] = is && p < kept ? p : -1;
    if (!is && p < kept) t.work(0)[p - at] = p;
    if (is && p >= kept) t.work(1)[kept - 1 - at] = p;
  }
  cluster_sync_all();
  const int pairs = __ldcg(&hdr[H_PAIRS]);
  for (int k = rank * kThreads + tid; k < pairs; k += nr * kThreads) {
    const int dst = __ldcg(&t.work(0)[k]), src = __ldcg(&t.work(1)[pairs - 1 - k]);
    page_map[src] = dst;
    t.rc()[dst] = t.rc()[src];
    t.rc()[src] = 0;
  }
}

// ---------------------------------------------------------------------------
// page copies
// ---------------------------------------------------------------------------
struct Pools {
  uint8_t* k;
  uint8_t* v;
  int layers, Hkv, row_bytes;
  long long layer_stride;
};

// One warp copies `bytes` (a multiple of 16) from src to dst, four 16-byte
// loads per lane in flight.
__device__ __forceinline__ void warp_copy(uint8_t* dst, const uint8_t* src, int bytes, int lane) {
  for (int at = lane * 16; at < bytes; at += 4 * 32 * 16) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * 512 < bytes) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + at + u * 512));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * 512 < bytes) __stcs(reinterpret_cast<uint4*>(dst + at + u * 512), v[u]);
  }
}

// Copy on write: the rows in use of each (pair, layer, K or V, head).
__global__ void __launch_bounds__(256) pages_cow_kernel(const PageTab t, const Pools b) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const long long w0 = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int per = 2 * b.layers * b.Hkv;
  const long long items = static_cast<long long>(__ldcg(&t.hdr()[H_PAIRS])) * per;
  for (long long w = w0; w < items; w += warps) {
    const int k = static_cast<int>(w / per), r = static_cast<int>(w - static_cast<long long>(k) * per);
    const int h = r % b.Hkv, x = r / b.Hkv;
    uint8_t* pool = (x & 1 ? b.v : b.k) + (x >> 1) * b.layer_stride;
    const size_t run = static_cast<size_t>(t.P) * b.row_bytes;   // one head of one page
    const size_t s = (static_cast<size_t>(__ldcg(&t.aux(3)[k])) * b.Hkv + h) * run;
    const size_t d = (static_cast<size_t>(__ldcg(&t.aux(4)[k])) * b.Hkv + h) * run;
    warp_copy(pool + d, pool + s, __ldcg(&t.aux(5)[k]) * b.row_bytes, lane);
  }
}

// Compaction. Whole pages move through shared memory by bulk copies, one
// thread per block: a ring of kStages pieces of up to kPiece bytes, so that a
// block always has several reads and writes in flight and no registers hold
// data. Then the lists follow the map and the free list is written anew.
constexpr int kStages = 6, kPiece = 16384;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__global__ void __launch_bounds__(256)
    pages_move_kernel(const PageTab t, const Pools b, const int32_t* __restrict__ page_map) {
  extern __shared__ __align__(128) uint8_t ring[];   // [kStages][kPiece]
  __shared__ uint64_t full[kStages];
  __shared__ int abort_s;
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    abort_s = 0;
    fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) {
    const int pairs = __ldcg(&t.hdr()[H_PAIRS]);
    const long long page_bytes = static_cast<long long>(b.Hkv) * t.P * b.row_bytes;
    const int per_page = static_cast<int>((page_bytes + kPiece - 1) / kPiece);
    // pieces in the order pair, layer, K or V, part of the page; this block
    // takes every gridDim.x-th
    const int per = 2 * b.layers * per_page;
    const long long pieces = static_cast<long long>(pairs) * per;
    struct Piece {
      uint8_t *src, *dst;
      uint32_t bytes;
    };
    auto piece = [&](long long w) -> Piece {
      const int k = static_cast<int>(w / per), r = static_cast<int>(w - static_cast<long long>(k) * per);
      const int x = r / per_page, c = r - x * per_page;
      uint8_t* pool = (x & 1 ? b.v : b.k) + (x >> 1) * b.layer_stride + static_cast<long long>(c) * kPiece;
      return {pool + __ldcg(&t.work(1)[pairs - 1 - k]) * page_bytes,
              pool + __ldcg(&t.work(0)[k]) * page_bytes,
              static_cast<uint32_t>(min(static_cast<long long>(kPiece),
                                        page_bytes - static_cast<long long>(c) * kPiece))};
    };
    uint8_t* to[kStages];
    uint32_t size[kStages];
    long long w = blockIdx.x;
    int issued = 0, done = 0;
    bool ok = true;
    auto issue = [&](int st) {
      const Piece q = piece(w);
      to[st] = q.dst;
      size[st] = q.bytes;
      mbar_arrive_expect_tx(&full[st], q.bytes);
      bulk_load(ring + st * kPiece, q.src, q.bytes, &full[st]);
      ++issued;
      w += gridDim.x;
    };
    // loads run kStages - 1 ahead of the stores; a stage is loaded again once
    // all but the newest store have read theirs
    for (; ok && (done < issued || w < pieces);) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        if (done == 0 && st == 0)
          for (int i = 0; i < kStages - 1 && w < pieces; ++i) issue(i);
        if (!ok || done >= issued) break;
        if (!mbar_wait(&full[st], (done / kStages) & 1, &abort_s, &g_status_pages)) {
          ok = false;
          break;
        }
        bulk_store(to[st], ring + st * kPiece, size[st]);
        ++done;
        if (w < pieces) {
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          issue((st + kStages - 1) % kStages);
        }
      }
    }
    if (!ok)   // a wait gave up: the loads in flight land before the block's shared memory goes
      for (int i = done; i < issued; ++i) mbar_drain(&full[i % kStages], (i / kStages) & 1);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.x + tid;
  const long long cells = static_cast<long long>(t.S) * t.M;
  for (long long i = t0; i < cells; i += step) {
    const int p = t.list()[i];
    if (t.page_ok(p)) t.list()[i] = page_map[p];
  }
  const int spare = t.hdr()[H_FREE];
  for (long long i = t0; i < spare; i += step) t.free_list()[i] = t.N - 1 - static_cast<int>(i);
}

// ---------------------------------------------------------------------------
// lists: one block per sequence; each block sums the lengths before its own
// (n loads over 256 threads, from L2) rather than wait for a scan. That is n^2
// loads in all, so n is bounded (a table has at most 2^18 sequences).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    pages_lists_kernel(const PageTab t, const int32_t* __restrict__ ids, int n,
                       int32_t* __restrict__ kv_indptr, int32_t* __restrict__ page_indptr,
                       int32_t* __restrict__ page_indices, int capacity) {
  __shared__ long long part[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x;
  if (n == 0) {   // no sequences: the running sums are their first zeros
    if (tid == 0 && kv_indptr) kv_indptr[0] = 0;
    if (tid == 0 && page_indptr) page_indptr[0] = 0;
    return;
  }
  auto len_of = [&](int j) -> int {
    const int id = ids[j];
    if (!t.seq_ok(id)) return -1;
    const int len = t.lens()[id];
    return len >= 0 && t.pages(len) <= t.M ? len : -1;
  };
  long long tokens = 0, pages = 0;
  for (int j = tid; j < i; j += blockDim.x) {
    const int len = max(0, len_of(j));
    tokens += len;
    pages += t.pages(len);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    tokens += __shfl_xor_sync(0xffffffffu, tokens, off);
    pages += __shfl_xor_sync(0xffffffffu, pages, off);
  }
  if (lane == 0) {
    part[0][warp] = tokens;
    part[1][warp] = pages;
  }
  __syncthreads();
  tokens = pages = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    tokens += part[0][w];
    pages += part[1][w];
  }
  const int len = len_of(i), mine = t.pages(max(0, len));
  const bool fits = pages + mine <= capacity && tokens + max(0, len) <= INT32_MAX;
  if (tid == 0) {
    if (len < 0) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
    else if (!fits) atomicExch(&g_status_pages, SINKATTN_BAD_LENGTHS);
    if (i == 0) kv_indptr[0] = page_indptr[0] = 0;
    kv_indptr[i + 1] = static_cast<int>(min(tokens + max(0, len), static_cast<long long>(INT32_MAX)));
    page_indptr[i + 1] = static_cast<int>(min(pages + mine, static_cast<long long>(capacity)));
  }
  if (!fits || len < 0) return;
  const int32_t* row = t.list() + static_cast<size_t>(ids[i]) * t.M;
  for (int e = tid; e < mine; e += blockDim.x) page_indices[pages + e] = row[e];
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SINKATTN_OK;
  set_error("%s: %s", what, cudaGetErrorString(e));
  return SINKATTN_CUDA_ERROR;
}

template <typename... Params, typename... Args>
int launch_table(const char* what, long long entries, const PageTab& t, cudaStream_t stream,
                 void (*kern)(Params...), Args... args) {
  const unsigned blocks = entries <= kOneBlock ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>((t.S + 31) / 32) * 4;   // one bit per sequence
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (blocks > 1) {
    if (blocks > 8) {
      const int rc = launched(cudaFuncSetAttribute(
          kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), what);
      if (rc) return rc;
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return launched(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

// A launch that may start while the one before it ends (it waits for that
// one's results itself).
template <typename... Params, typename... Args>
int launch_after(const char* what, unsigned blocks, size_t smem, cudaStream_t stream,
                 void (*kern)(Params...), Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

int refuse(int status, const char* text) {
  set_error("%s", text);
  return status;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int check_sizes(int32_t num_pages, int32_t max_seqs, int32_t max_pages) {
  if (num_pages < 1 || max_seqs < 1 || max_pages < 1)
    return refuse(SINKATTN_INVALID_ARG, "num_pages, max_seqs and max_pages must be positive");
  if (static_cast<int64_t>(max_seqs) * max_pages >= (int64_t{1} << 30))
    return refuse(SINKATTN_UNSUPPORTED, "max_seqs * max_pages reaches 2^30");
  if (max_seqs > (1 << 18)) return refuse(SINKATTN_UNSUPPORTED, "max_seqs exceeds 2^18");
  return SINKATTN_OK;
}

int make_table(const int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
               int32_t max_pages, PageTab* t) {
  set_error("%s", "");
  int rc = check_sizes(num_pages, max_seqs, max_pages);
  if (rc) return rc;
  if (!table || !aligned(table, 16))
    return refuse(SINKATTN_INVALID_ARG, "table must be non-null and 16-byte aligned");
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return refuse(SINKATTN_UNSUPPORTED, "page_size is not a power of two in [16, 256]");
  if (static_cast<int64_t>(num_pages) * page_size >= (int64_t{1} << 31) ||
      static_cast<int64_t>(max_pages) * page_size >= (int64_t{1} << 31))
    return refuse(SINKATTN_UNSUPPORTED, "num_pages or max_pages times page_size reaches 2^31");
  t->base = const_cast<int32_t*>(table);
  t->N = num_pages;
  t->P = page_size;
  t->S = max_seqs;
  t->M = max_pages;
  t->shift = 0;
  while ((1 << t->shift) < page_size) ++t->shift;
  return SINKATTN_OK;
}

int make_pools(const PageTab& t, void* k, void* v, int32_t layers, int64_t stride, int32_t Hkv,
               int32_t row_bytes, Pools* b) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return refuse(SINKATTN_INVALID_ARG, "k_pages and v_pages must be non-null and 16-byte aligned");
  if (layers < 1 || Hkv < 1 || row_bytes < 16 || row_bytes % 16)
    return refuse(SINKATTN_INVALID_ARG,
                  "num_layers and num_kv_heads must be positive, row_bytes a multiple of 16");
  const int64_t rows = static_cast<int64_t>(t.N) * t.P * Hkv;
  if (rows >= (int64_t{1} << 31) || static_cast<int64_t>(layers) * Hkv >= (int64_t{1} << 28) ||
      static_cast<int64_t>(Hkv) * t.P * row_bytes >= (int64_t{1} << 31))
    return refuse(SINKATTN_UNSUPPORTED, "page pools exceed 2^31 rows, or a page 2^31 bytes");
  if (layers > 1 && (stride % 16 || stride < rows * row_bytes))
    return refuse(SINKATTN_INVALID_ARG,
                  "layer_stride must be a multiple of 16 and hold one layer's pages");
  b->k = static_cast<uint8_t*>(k);
  b->v = static_cast<uint8_t*>(v);
  b->layers = layers;
  b->Hkv = Hkv;
  b->row_bytes = row_bytes;
  b->layer_stride = stride;
  return SINKATTN_OK;
}

int check_ids(const PageTab& t, const int32_t* ids, int32_t n) {
  if (n < 0) return refuse(SINKATTN_INVALID_ARG, "n must be non-negative");
  if (n > t.S) return refuse(SINKATTN_INVALID_ARG, "more sequence ids than the table has sequences");
  if (n > 0 && (!ids || !aligned(ids, 4)))
    return refuse(SINKATTN_INVALID_ARG, "sequence ids must be non-null and 4-byte aligned");
  return SINKATTN_OK;
}

unsigned copy_blocks() { return static_cast<unsigned>(sm_count()) * 8u; }   // 64 warps per SM

}  // namespace

// (the move kernel has waits but no K/V tiles: the limit is all that counts here)
SINKATTN_DEFINE_SET_HOOKS(set_hooks_pages)

int read_status_pages(cudaStream_t s, int* status) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(status, g_status_pages, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                s) != cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  if (cudaMemcpyToSymbolAsync(g_status_pages, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
      cudaSuccess)
    return SINKATTN_CUDA_ERROR;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SINKATTN_CUDA_ERROR;
  return SINKATTN_OK;
}

}  // namespace sinkattn

using namespace sinkattn;

extern "C" {

int sinkattn_pages_table_ints(int32_t num_pages, int32_t max_seqs, int32_t max_pages,
                              int64_t* ints) {
  set_error("%s", "");
  if (!ints) return refuse(SINKATTN_INVALID_ARG, "ints must be non-null");
  const int rc = check_sizes(num_pages, max_seqs, max_pages);
  if (rc) return rc;
  *ints = kHeader + static_cast<int64_t>(max_seqs) * (8 + static_cast<int64_t>(max_pages)) +
          static_cast<int64_t>(num_pages) * 4;
  return SINKATTN_OK;
}

int sinkattn_pages_init(int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
                        int32_t max_pages, void* stream) {
  PageTab t;
  const int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (rc) return rc;
  const int64_t words = std::max<int64_t>(static_cast<int64_t>(max_seqs) * max_pages, num_pages);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((words + 255) / 256, copy_blocks()));
  pages_init_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(t);
  return launched(cudaGetLastError(), "page table init launch");
}

int sinkattn_pages_reserve(int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
                           int32_t max_pages, const int32_t* seq_ids, const int32_t* cu_new,
                           int32_t n, int32_t total_new, void* k_pages, void* v_pages,
                           int32_t num_layers, int64_t layer_stride, int32_t num_kv_heads,
                           int32_t row_bytes, int32_t* slots, void* stream) {
  PageTab t;
  Pools b;
  int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (!rc) rc = check_ids(t, seq_ids, n);
  if (!rc)
    rc = make_pools(t, k_pages, v_pages, num_layers, layer_stride, num_kv_heads, row_bytes, &b);
  if (rc) return rc;
  if (total_new < 0) return refuse(SINKATTN_INVALID_ARG, "total_new must be non-negative");
  if (total_new >= (1 << 30)) return refuse(SINKATTN_UNSUPPORTED, "total_new reaches 2^30");
  if (n == 0 && total_new > 0) return refuse(SINKATTN_INVALID_ARG, "new tokens without sequences");
  if (n == 0 || total_new == 0) return SINKATTN_OK;
  if (!cu_new || !slots || !aligned(cu_new, 4) || !aligned(slots, 4))
    return refuse(SINKATTN_INVALID_ARG, "cu_new and slots must be non-null and 4-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch_table("page reserve launch", std::max(n, total_new), t, s, pages_reserve_kernel, t,
                    seq_ids, cu_new, n, total_new, slots);
  if (rc) return rc;
  const int64_t warps = static_cast<int64_t>(n) * 2 * num_layers * num_kv_heads;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((warps + 7) / 8, copy_blocks()));
  return launch_after("page copy launch", blocks, 0, s, pages_cow_kernel, t, b);
}

int sinkattn_pages_fork(int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
                        int32_t max_pages, const int32_t* src_ids, const int32_t* dst_ids,
                        int32_t n, void* stream) {
  PageTab t;
  int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (!rc) rc = check_ids(t, src_ids, n);
  if (!rc) rc = check_ids(t, dst_ids, n);
  if (rc) return rc;
  if (n == 0) return SINKATTN_OK;
  return launch_table("page fork launch", static_cast<long long>(n) * max_pages, t,
                      static_cast<cudaStream_t>(stream), pages_fork_kernel, t, src_ids, dst_ids, n);
}

int sinkattn_pages_truncate(int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
                            int32_t max_pages, const int32_t* seq_ids, const int32_t* new_lens,
                            int32_t n, void* stream) {
  PageTab t;
  int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (!rc) rc = check_ids(t, seq_ids, n);
  if (rc) return rc;
  if (!aligned(new_lens, 4)) return refuse(SINKATTN_INVALID_ARG, "new_lens must be 4-byte aligned");
  if (n == 0) return SINKATTN_OK;
  return launch_table("page truncate launch", static_cast<long long>(n) * max_pages, t,
                      static_cast<cudaStream_t>(stream), pages_truncate_kernel, t, seq_ids,
                      new_lens, n);
}

int sinkattn_pages_compact(int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_seqs,
                           int32_t max_pages, void* k_pages, void* v_pages, int32_t num_layers,
                           int64_t layer_stride, int32_t num_kv_heads, int32_t row_bytes,
                           int32_t* page_map, void* stream) {
  PageTab t;
  Pools b;
  int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (!rc)
    rc = make_pools(t, k_pages, v_pages, num_layers, layer_stride, num_kv_heads, row_bytes, &b);
  if (rc) return rc;
  if (!page_map || !aligned(page_map, 4))
    return refuse(SINKATTN_INVALID_ARG, "page_map must be non-null and 4-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch_table("page compact launch", num_pages, t, s, pages_compact_kernel, t, page_map);
  if (rc) return rc;
  constexpr int smem = kStages * kPiece;   // two blocks per SM
  rc = launched(cudaFuncSetAttribute(pages_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     smem), "page move launch");
  if (rc) return rc;
  return launch_after("page move launch", static_cast<unsigned>(sm_count()) * 2u, smem, s,
                      pages_move_kernel, t, b, static_cast<const int32_t*>(page_map));
}

int sinkattn_pages_lists(const int32_t* table, int32_t num_pages, int32_t page_size,
                         int32_t max_seqs, int32_t max_pages, const int32_t* seq_ids, int32_t n,
                         int32_t* kv_indptr, int32_t* page_indptr, int32_t* page_indices,
                         int32_t capacity, void* stream) {
  PageTab t;
  int rc = make_table(table, num_pages, page_size, max_seqs, max_pages, &t);
  if (rc) return rc;
  if (n < 0 || capacity < 0)
    return refuse(SINKATTN_INVALID_ARG, "n and capacity must be non-negative");
  if (n > (1 << 18)) return refuse(SINKATTN_UNSUPPORTED, "n exceeds 2^18");
  if (n == 0 && !kv_indptr && !page_indptr) return SINKATTN_OK;
  if ((n > 0 && (!seq_ids || !kv_indptr || !page_indptr || (capacity > 0 && !page_indices))) ||
      !aligned(seq_ids, 4) || !aligned(kv_indptr, 4) || !aligned(page_indptr, 4) ||
      !aligned(page_indices, 4))
    return refuse(SINKATTN_INVALID_ARG,
                  "seq_ids, kv_indptr, page_indptr and page_indices must be non-null and 4-byte aligned");
  pages_lists_kernel<<<static_cast<unsigned>(std::max(n, 1)), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      t, seq_ids, n, kv_indptr, page_indptr, page_indices, capacity);
  return launched(cudaGetLastError(), "page lists launch");
}

}  // extern "C"
