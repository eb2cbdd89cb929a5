// Page tables of a paged KV cache, and the copies of whole or partly filled
// pages that they ask for (layout and rules: sinkattn.h).
//
// The table's work is integer work on a few kilobytes to megabytes, so time
// is launch and memory latency, not bandwidth. Each call is one launch of one
// thread-block cluster: its phases (check, count, rank, commit) are separated
// by cluster barriers of a fraction of a microsecond, where separate launches
// would cost two microseconds each, and nothing has to be read back by the
// host, so every call can be captured into a graph. A call with up to
// kOneBlock entries runs as a cluster of one block, larger ones as kCluster
// blocks. Phase 1 only checks and writes scratch; a call that cannot be
// served as a whole ends there, with the table unchanged.
//
// No result depends on the order in which atomics arrive: they only count,
// or elect a page's first writer or first appearance by its position (a
// maximum), and ranks come from ordered scans.
//
// Page copies follow as a second launch over the whole GPU that reads the
// pairs the first one found (a programmatic dependent, so its start-up
// overlaps the first launch's end). They move 16 bytes per lane, and each
// lane has four loads in flight.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sinkattn {

__device__ int g_status_pages;

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;          // blocks of a large call (the portable limit)
constexpr int kOneBlock = 4096;      // entries that one block takes alone
constexpr int kHeader = 16;

// Header words besides the free count (scratch of one call).
enum { H_FREE = 0, H_OK = 1, H_COUNT = 2, H_PAIRS = 3, H_MOST = 4, H_RANK = 8 };

struct PageTab {
  int32_t* base;
  int N, P, S, M, shift;   // pages, page size (= 1 << shift), sequences, pages per sequence
  __device__ __forceinline__ int32_t* hdr() const { return base; }
  __device__ __forceinline__ int32_t* lens() const { return base + kHeader; }
  __device__ __forceinline__ int32_t* list() const { return lens() + S; }
  __device__ __forceinline__ int32_t* rc() const { return list() + static_cast<size_t>(S) * M; }
  __device__ __forceinline__ int32_t* free_list() const { return rc() + N; }
  __device__ __forceinline__ int32_t* mark() const { return free_list() + N; }
  __device__ __forceinline__ int32_t* aux(int k) const {   // k < 6: one word per sequence
    return mark() + static_cast<size_t>(S) * (1 + k);
  }
  __device__ __forceinline__ int32_t* work(int k) const {  // k < 2: one word per page
    return mark() + static_cast<size_t>(S) * 7 + static_cast<size_t>(N) * k;
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
  const int tid = threadIdx.x;
  int32_t* hdr = t.hdr();
  if (cluster_rank() == 0) {
    // the first item of each thread stays in registers
    ReserveItem mine{};
    if (tid < n) mine = reserve_item(t, ids, cu, tid);
    for (int i = tid; i < n; i += kThreads) {
      const ReserveItem r = i == tid ? mine : reserve_item(t, ids, cu, i);
      if (t.seq_ok(r.id)) t.mark()[r.id] = 0;
      if (r.tail >= 0) t.work(0)[r.tail] = t.work(1)[r.tail] = 0;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const ReserveItem r = i == tid ? mine : reserve_item(t, ids, cu, i);
      if (t.seq_ok(r.id)) atomicAdd(&t.mark()[r.id], 1);
      if (r.tail >= 0) {
        atomicAdd(&t.work(0)[r.tail], 1);       // writers of the page in this call
        atomicMax(&t.work(1)[r.tail], n - i);   // the first of them
      }
    }
    __syncthreads();
    bool bad = false;
    long long need = 0;
    for (int base = 0; base < n; base += kThreads) {
      const int i = base + tid;
      int want = 0, copies = 0;
      if (i < n) {
        const ReserveItem r = base == 0 ? mine : reserve_item(t, ids, cu, i);
        if (!r.ok || __ldcg(&t.mark()[r.id]) != 1) {
          bad = true;
        } else {
          copies = r.tail >= 0 && !(__ldcg(&t.work(0)[r.tail]) == r.rc &&
                                    __ldcg(&t.work(1)[r.tail]) == n - i);
          want = t.pages(r.len + r.grow) - t.pages(r.len) + copies;
          t.aux(1)[i] = r.len;
          t.aux(2)[i] = copies;
        }
      }
      int total;
      const int before = block_scan(want, &total, sums);
      // (a call that needs 2^31 pages has failed long before: need is exact)
      if (i < n) t.aux(0)[i] = static_cast<int>(need) + before + copies;
      need += total;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      const int count = hdr[H_FREE];
      int status = SINKATTN_OK;
      if (cu[0] != 0 || cu[n] != total_new) status = SINKATTN_BAD_LENGTHS;
      else if (bad) status = SINKATTN_BAD_PAGES;
      else if (need > count) status = SINKATTN_OUT_OF_PAGES;
      if (status) atomicExch(&g_status_pages, status);
      hdr[H_OK] = status == SINKATTN_OK;
      hdr[H_COUNT] = count;
      hdr[H_PAIRS] = 0;
      if (!status) hdr[H_FREE] = count - static_cast<int>(need);
    }
  }
  cluster_sync_all();
  const int nt = cluster_size() * kThreads;
  const int t0 = cluster_rank() * kThreads + tid;
  if (!__ldcg(&hdr[H_OK])) {
    for (int i = t0; i < total_new; i += nt) slots[i] = -1;
    return;
  }
  const int count = __ldcg(&hdr[H_COUNT]);
  int32_t* list = t.list();
  for (int i = t0; i < n; i += nt) {
    const int id = ids[i], len = __ldcg(&t.aux(1)[i]);
    t.lens()[id] = len + (cu[i + 1] - cu[i]);
    if (__ldcg(&t.aux(2)[i])) {
      int32_t* entry = &list[static_cast<size_t>(id) * t.M + (len >> t.shift)];
      const int src = *entry, dst = t.free_list()[count - __ldcg(&t.aux(0)[i])];
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
    const int len = __ldcg(&t.aux(1)[lo]), first = __ldcg(&t.aux(0)[lo]);
    const int pos = len + (k - cu[lo]), e = pos >> t.shift, have = t.pages(len);
    int32_t* row = list + static_cast<size_t>(ids[lo]) * t.M;
    int page;
    if (e < have) {
      page = __ldcg(&t.aux(2)[lo]) ? t.free_list()[count - first] : row[e];
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
__global__ void __launch_bounds__(kThreads)
    pages_fork_kernel(const PageTab t, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int n) {
  __shared__ int most_s;
  const int tid = threadIdx.x;
  int32_t* hdr = t.hdr();
  if (cluster_rank() == 0) {
    if (tid == 0) most_s = 0;
    for (int i = tid; i < n; i += kThreads) {
      if (t.seq_ok(src[i])) t.mark()[src[i]] = 0;
      if (t.seq_ok(dst[i])) t.mark()[dst[i]] = 0;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (t.seq_ok(dst[i])) atomicAdd(&t.mark()[dst[i]], 1);
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) {
      const int a = src[i], b = dst[i];
      if (!t.seq_ok(a) || !t.seq_ok(b) || __ldcg(&t.mark()[b]) != 1 || __ldcg(&t.mark()[a]) != 0 ||
          t.lens()[b] != 0) {
        bad = true;
        continue;
      }
      const int len = t.lens()[a];
      if (len < 0 || t.pages(len) > t.M) bad = true;
      else atomicMax(&most_s, t.pages(len));
      t.aux(0)[i] = len;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      if (bad) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
      hdr[H_OK] = !bad;
      hdr[H_MOST] = most_s;
    }
  }
  cluster_sync_all();
  if (!__ldcg(&hdr[H_OK])) return;
  const int most = __ldcg(&hdr[H_MOST]);
  const int nt = cluster_size() * kThreads;
  const int t0 = cluster_rank() * kThreads + tid;
  for (int i = t0; i < n; i += nt) t.lens()[dst[i]] = __ldcg(&t.aux(0)[i]);
  // (item, entry) pairs over the rectangle n x (longest list)
  const int cells = n * most;   // < max_seqs * max_pages
  for (int c = t0; c < cells; c += nt) {
    const int i = c / most, e = c - i * most;
    if (e >= t.pages(__ldcg(&t.aux(0)[i]))) continue;
    const int p = t.list()[static_cast<size_t>(src[i]) * t.M + e];
    t.list()[static_cast<size_t>(dst[i]) * t.M + e] = p;
    if (t.page_ok(p)) atomicAdd(&t.rc()[p], 1);
  }
}

// ---------------------------------------------------------------------------
// truncate
// ---------------------------------------------------------------------------
// aux(0): entries the item keeps, aux(1): entries it drops. A dropped page is
// given back by its first appearance in the request (its position is elected
// in work(0)) if its count has come to zero.
__global__ void __launch_bounds__(kThreads)
    pages_truncate_kernel(const PageTab t, const int32_t* __restrict__ ids,
                          const int32_t* __restrict__ new_lens, int n) {
  __shared__ int sums[32];
  __shared__ int most_s;
  const int tid = threadIdx.x, rank = cluster_rank(), nr = cluster_size();
  int32_t* hdr = t.hdr();
  if (rank == 0) {
    if (tid == 0) most_s = 0;
    for (int i = tid; i < n; i += kThreads)
      if (t.seq_ok(ids[i])) t.mark()[ids[i]] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (t.seq_ok(ids[i])) atomicAdd(&t.mark()[ids[i]], 1);
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) {
      const int id = ids[i], to = new_lens ? new_lens[i] : 0;
      if (!t.seq_ok(id) || __ldcg(&t.mark()[id]) != 1) {
        bad = true;
        continue;
      }
      const int len = t.lens()[id];
      if (to < 0 || to > len || t.pages(len) > t.M) {
        bad = true;
        continue;
      }
      const int keep = t.pages(to), drop = t.pages(len) - keep;
      t.aux(0)[i] = keep;
      t.aux(1)[i] = drop;
      if (drop > 0) atomicMax(&most_s, drop);
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      if (bad) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
      hdr[H_OK] = !bad;
      hdr[H_COUNT] = hdr[H_FREE];
      hdr[H_MOST] = most_s;
    }
  }
  cluster_sync_all();
  if (!__ldcg(&hdr[H_OK])) return;   // uniform over the cluster
  const int most = __ldcg(&hdr[H_MOST]), count = __ldcg(&hdr[H_COUNT]);
  for (int i = rank * kThreads + tid; i < n; i += nr * kThreads)
    t.lens()[ids[i]] = new_lens ? new_lens[i] : 0;
  if (most == 0) return;             // uniform: no page leaves a list
  // cells (item, entry) in request order; each block takes a run of them
  const int cells = n * most;        // < max_seqs * max_pages
  const int per = ((cells + nr - 1) / nr + kThreads - 1) / kThreads * kThreads;
  const int c0 = min(cells, rank * per), c1 = min(cells, c0 + per);
  auto entry = [&](int c) -> int32_t* {
    const int i = c / most, e = c - i * most;
    if (e >= __ldcg(&t.aux(1)[i])) return nullptr;
    return &t.list()[static_cast<size_t>(ids[i]) * t.M + __ldcg(&t.aux(0)[i]) + e];
  };
  auto page_of = [&](int32_t* at) -> int { return at && t.page_ok(*at) ? *at : -1; };
  int32_t* mine = c0 + tid < c1 ? entry(c0 + tid) : nullptr;   // the thread's first cell
  const int page0 = page_of(mine);
  for (int c = c0 + tid; c < c1; c += kThreads) {
    const int p = c == c0 + tid ? page0 : page_of(entry(c));
    if (p >= 0) t.work(0)[p] = 0;
  }
  cluster_sync_all();
  for (int c = c0 + tid; c < c1; c += kThreads) {
    const int p = c == c0 + tid ? page0 : page_of(entry(c));
    if (p >= 0) {
      atomicSub(&t.rc()[p], 1);
      atomicMax(&t.work(0)[p], INT32_MAX - c);
    }
  }
  cluster_sync_all();
  auto gives_back = [&](int p, int c) -> bool {
    return p >= 0 && __ldcg(&t.rc()[p]) == 0 && __ldcg(&t.work(0)[p]) == INT32_MAX - c;
  };
  int found = 0;
  for (int c = c0 + tid; c < c1; c += kThreads) {
    const int p = c == c0 + tid ? page0 : page_of(entry(c));
    found += gives_back(p, c);
  }
  int total;
  block_scan(found, &total, sums);
  if (tid == 0) hdr[H_RANK + rank] = total;
  cluster_sync_all();
  int before = 0, all = 0;
  for (int r = 0; r < nr; ++r) {
    const int x = __ldcg(&hdr[H_RANK + r]);
    before += r < rank ? x : 0;
    all += x;
  }
  if (rank == 0 && tid == 0) hdr[H_FREE] = count + all;
  for (int base = c0; base < c1; base += kThreads) {
    const int c = base + tid;
    int32_t* at = c < c1 ? (base == c0 ? mine : entry(c)) : nullptr;
    const int p = base == c0 ? page0 : page_of(at);
    const bool back = c < c1 && gives_back(p, c);
    const int r = before + block_scan(back, &total, sums);
    if (back && count + all <= t.N) t.free_list()[count + all - 1 - r] = p;
    before += total;
    if (at) *at = -1;
  }
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
  const int tid = threadIdx.x, rank = cluster_rank(), nr = cluster_size();
  int32_t* hdr = t.hdr();
  const int per = ((t.N + nr - 1) / nr + kThreads - 1) / kThreads * kThreads;
  const int p0 = min(t.N, rank * per), p1 = min(t.N, p0 + per);
  int live = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) live += t.rc()[p] > 0;
  int total;
  block_scan(live, &total, sums);
  if (tid == 0) hdr[H_RANK + rank] = total;
  cluster_sync_all();
  int before = 0, kept = 0;
  for (int r = 0; r < nr; ++r) {
    const int x = __ldcg(&hdr[H_RANK + r]);
    before += r < rank ? x : 0;
    kept += x;
  }
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

// Compaction: whole pages, 2 KB per warp and step; then the lists follow the
// map and the free list is written anew.
__global__ void __launch_bounds__(256)
    pages_move_kernel(const PageTab t, const Pools b, const int32_t* __restrict__ page_map) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const long long w0 = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int pairs = __ldcg(&t.hdr()[H_PAIRS]);
  const long long page_bytes = static_cast<long long>(b.Hkv) * t.P * b.row_bytes;
  const int per_page = static_cast<int>((page_bytes + 2047) / 2048);
  const long long per = 2LL * b.layers * per_page;
  for (long long w = w0; w < pairs * per; w += warps) {
    const int k = static_cast<int>(w / per);
    const long long r = w - k * per;
    const int x = static_cast<int>(r / per_page), c = static_cast<int>(r - static_cast<long long>(x) * per_page);
    uint8_t* pool = (x & 1 ? b.v : b.k) + (x >> 1) * b.layer_stride + c * 2048LL;
    warp_copy(pool + __ldcg(&t.work(0)[k]) * page_bytes,
              pool + __ldcg(&t.work(1)[pairs - 1 - k]) * page_bytes,
              static_cast<int>(min(2048LL, page_bytes - c * 2048LL)), lane);
  }
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
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
// (n loads over 256 threads, from L2) rather than wait for a scan.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    pages_lists_kernel(const PageTab t, const int32_t* __restrict__ ids, int n,
                       int32_t* __restrict__ kv_indptr, int32_t* __restrict__ page_indptr,
                       int32_t* __restrict__ page_indices, int capacity) {
  __shared__ long long part[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x;
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
  const bool fits = pages + mine <= capacity;
  if (tid == 0) {
    if (len < 0) atomicExch(&g_status_pages, SINKATTN_BAD_PAGES);
    else if (!fits) atomicExch(&g_status_pages, SINKATTN_BAD_LENGTHS);
    if (i == 0) kv_indptr[0] = page_indptr[0] = 0;
    kv_indptr[i + 1] = static_cast<int>(tokens + max(0, len));
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
int launch_table(const char* what, long long entries, cudaStream_t stream,
                 void (*kern)(Params...), Args... args) {
  const unsigned blocks = entries <= kOneBlock ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

// A launch that may start while the one before it ends (it waits for that
// one's results itself).
template <typename... Params, typename... Args>
int launch_after(const char* what, unsigned blocks, cudaStream_t stream, void (*kern)(Params...),
                 Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
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
  if (static_cast<int64_t>(max_seqs) * max_pages >= (int64_t{1} << 31))
    return refuse(SINKATTN_UNSUPPORTED, "max_seqs * max_pages reaches 2^31");
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
  if (n == 0 && total_new > 0) return refuse(SINKATTN_INVALID_ARG, "new tokens without sequences");
  if (n == 0 || total_new == 0) return SINKATTN_OK;
  if (!cu_new || !slots || !aligned(cu_new, 4) || !aligned(slots, 4))
    return refuse(SINKATTN_INVALID_ARG, "cu_new and slots must be non-null and 4-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch_table("page reserve launch", std::max(n, total_new), s, pages_reserve_kernel, t,
                    seq_ids, cu_new, n, total_new, slots);
  if (rc) return rc;
  const int64_t warps = static_cast<int64_t>(n) * 2 * num_layers * num_kv_heads;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((warps + 7) / 8, copy_blocks()));
  return launch_after("page copy launch", blocks, s, pages_cow_kernel, t, b);
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
  return launch_table("page fork launch", static_cast<long long>(n) * max_pages,
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
  return launch_table("page truncate launch", static_cast<long long>(n) * max_pages,
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
  rc = launch_table("page compact launch", num_pages, s, pages_compact_kernel, t, page_map);
  if (rc) return rc;
  return launch_after("page move launch", copy_blocks(), s, pages_move_kernel, t, b,
                      static_cast<const int32_t*>(page_map));
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
  if (n == 0) return SINKATTN_OK;
  if (!seq_ids || !kv_indptr || !page_indptr || (capacity > 0 && !page_indices) ||
      !aligned(seq_ids, 4) || !aligned(kv_indptr, 4) || !aligned(page_indptr, 4) ||
      !aligned(page_indices, 4))
    return refuse(SINKATTN_INVALID_ARG,
                  "seq_ids, kv_indptr, page_indptr and page_indices must be non-null and 4-byte aligned");
  pages_lists_kernel<<<static_cast<unsigned>(n), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      t, seq_ids, n, kv_indptr, page_indptr, page_indices, capacity);
  return launched(cudaGetLastError(), "page lists launch");
}

}  // extern "C"
