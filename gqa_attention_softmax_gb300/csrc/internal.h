// Host-side interface between the C ABI (api.cu) and the kernel translation
// units. Not installed; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sinkattn {

// Everything the attention kernels need besides the K/V tensor maps.
struct AttnArgs {
  const void* q;            // bf16 [total_q, Hq, d]
  const void* k;            // bf16 ragged HND
  const void* v;            // bf16 ragged HND
  const int32_t* cu_q;      // [B+1] (prefill) or nullptr (decode: uniform q_len)
  const int32_t* cu_k;      // [B+1]
  int32_t batch, q_len, max_q, max_kv;
  int32_t total_q;          // rows of q (prefill)
  int32_t Hq, Hkv, d;
  float sm_scale;
  int32_t causal, window;
  int32_t num_splits;       // 1 for the single-pass (final) mode
  // final mode
  const float* sinks;
  void* out;
  float* lse;
  // split mode: chunk s of a row is slot part_first + s of the row's
  // part_slots partials (0: num_splits, this call writes all of them)
  float* part_acc;
  float* part_md;
  int32_t part_slots, part_first;
  // rows that are not the last queries of the keys they see (a shared prefix):
  // any number of rows per key, and with a window the position of each query
  // token counted from the first key (nullptr: no window)
  int32_t free_rows;
  const int32_t* row_pos;
  // an own pass: cu_k holds lengths, page_indptr first entries, both of
  // sequence seq[b] (nullptr: none of this)
  const int32_t* seq;
  // a prefix pass: running sum of the groups' row blocks [batch + 1], each of
  // attn_mma_block_tokens() query tokens (nullptr: blocks per sequence)
  const int32_t* blk;
  int32_t chain;            // kChain*: its place in a chain of dependent launches
  // paged KV (page_size > 0): k and v are page pools [num_pages, Hkv, page_size, d];
  // sequence b's keys [e * page_size, (e + 1) * page_size) live in page
  // page_indices[page_indptr[b] + e]; cu_k still gives the key counts
  int32_t page_size;
  int32_t num_pages;
  const int32_t* page_indptr;   // [B+1]
  const int32_t* page_indices;  // [page_indptr[B]]
  // FP8 KV (kv_fp8 != 0): k and v hold e4m3 codes (one byte per element, same
  // layout); KV head g's keys are code * k_scale[g], values code * v_scale[g]
  int32_t kv_fp8;
  const float* k_scale;         // [Hkv], device
  const float* v_scale;         // [Hkv], device
};

// Rows of the 2-D tensor map over K or V, and the box height: contiguous HND
// rows, or page-pool rows (page, head, slot) with boxes of min(page, tile) rows.
inline uint64_t kv_map_rows(const AttnArgs& a) {
  return a.page_size > 0 ? static_cast<uint64_t>(a.num_pages) * a.Hkv * a.page_size
                         : static_cast<uint64_t>(a.Hkv) * a.batch * a.max_kv;
}
// Paged KV: boxes of min(page_size, the largest power of two dividing the
// tile) rows, so a box starting on a multiple of its height never crosses a
// page; contiguous KV: one box per tile.
inline int kv_box_rows(const AttnArgs& a, int tile_keys) {
  if (a.page_size <= 0) return tile_keys;
  const int pow2 = tile_keys & -tile_keys;
  return a.page_size < pow2 ? a.page_size : pow2;
}

// A chain of launches, each a programmatic dependent of the one before: a
// launch may start while the one before it still runs. kChainWaitFirst: it
// waits for that one's results before it reads anything. kChainWaitLast: it
// needs none of them (the one before waited for what it does need, which this
// one loads around L1, chain_load), but its first block ends only after it, so
// that whoever waits for this launch has waited for both (one block, as a block
// that waits keeps its place on the SM). kChainFollow: the next launch may
// start as soon as this one has waited.
constexpr int32_t kChainWaitFirst = 1, kChainWaitLast = 2, kChainFollow = 4;

// Sets a kernel of a chain up: its dynamic shared memory, and the largest
// shared-memory share of the SM, without which the next launch's blocks could
// not start beside its own.
template <typename Kern>
inline cudaError_t set_chained_smem(Kern kern, int smem) {
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

// Launches `kern` as a programmatic dependent of the launch before it.
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kern)(Params...), dim3 grid, int threads, size_t smem,
                                  cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Partials of a row, this call's or shared with another call's.
inline int part_slots(const AttnArgs& a) { return a.part_slots > 0 ? a.part_slots : a.num_splits; }

// Encodes a 2-D tensor map over a [rows, d] bf16 buffer with [box_rows, 64]
// boxes and 128-byte swizzling. Returns 0 or a SINKATTN_* status.
int make_rows_tmap(CUtensorMap* map, const void* base, uint64_t rows, int d, int box_rows,
                   int swizzle_bytes);
// The same over a [rows, d] array of bytes (e4m3 codes), [box_rows, d] boxes,
// swizzled in 16-byte chunks over swizzle_bytes (64 or 128; 0: none; the
// row must be that wide).
int make_rows_tmap_u8(CUtensorMap* map, const void* base, uint64_t rows, int d, int box_rows,
                      int swizzle_bytes = 0);

// Encodes a 3-D tensor map over q [total_q, Hq, d] bf16 whose box is
// [QB tokens][G heads][64 columns] (128 rows of one GQA group), 128-byte swizzled.
int make_q_tmap(CUtensorMap* map, const void* q, uint64_t total_q, int Hq, int d, int G, int QB);

// Split-KV decode (per-chunk partial outputs) on the warp-level tensor-core
// path. Returns a SINKATTN_* status.
int launch_attn_mma(const AttnArgs& a, cudaStream_t stream);
// The same as a part of shared-prefix decode (a.part_slots, a.chain, ...).
int launch_attn_mma_shared(const AttnArgs& a, cudaStream_t stream);
int attn_mma_block_tokens(int G, int64_t tokens);   // of `tokens` query tokens in all

// Split-KV decode with the merge done on chip: the num_splits (<= 16) chunks
// of one (sequence, KV head) form a thread-block cluster that folds its
// partials through distributed shared memory. Writes out / lse directly.
int launch_attn_mma_fused(const AttnArgs& a, cudaStream_t stream);


// Split-KV decode on the tcgen05/TMEM path (head_dim 128; 16, 32, 48 or 64
// query rows per KV head and query block). Same partial layout as
// launch_attn_mma.
bool decode_tc_supported(const AttnArgs& a);
int launch_decode_tc(const AttnArgs& a, cudaStream_t stream);

// Single-pass prefill on the tcgen05/TMEM path. Returns a SINKATTN_* status.
int launch_prefill_tc(const AttnArgs& a, int kind, cudaStream_t stream);

// drop_partials: the partials are the library's scratch (sinkattn_decode's
// workspace): after folding a row, drop its accumulator lines from L2 without
// write-back. Never for caller-visible partials.
int launch_merge(const float* part_acc, const float* part_md, const float* sinks, int32_t rows,
                 int32_t Hq, int32_t d, int32_t num_splits, void* out, float* lse,
                 cudaStream_t stream, bool drop_partials);
// The same for partials of which many are empty (d = 0): those slots'
// accumulators are not read and need not have been written.
// `check` (nullptr: none): a few more blocks hold the caller's lengths and groups
// to the rules of shared-prefix decode, where no plan has.
struct SharedCheck {
  const int32_t *kv_indptr, *page_indptr, *group_indptr, *prefix_lens;
  int groups, page_size, batch, q_len, max_prefix, max_suffix;
  int blocks;   // (set by the launch)
};
int launch_merge_sparse(const float* part_acc, const float* part_md, const float* sinks,
                        int32_t rows, int32_t Hq, int32_t d, int32_t num_slots, void* out,
                        float* lse, const SharedCheck* check, cudaStream_t stream);

// Shared-prefix decode: what the prefix and the per-sequence passes read,
// derived on the device from the page lists and the groups. All int32.
struct SharedPlan {
  // the sequences, longest own keys first (to 64 classes of length): an own
  // pass whose blocks take them in this order ends with its short ones
  int32_t* own_seq;   // [batch] sequence
  int32_t* own_len;   // [batch] its own keys
  int32_t* own_page;  // [batch] first entry of its own pages in page_indices
  int32_t* grp_q;     // [groups + 1] first query token of each group
  int32_t* grp_k;     // [groups + 1] running sum of the prefixes' keys
  int32_t* grp_pages; // [groups + 1] first entry of the prefixes' pages
  int32_t* grp_unit;  // [groups + 1] running sum of the tcgen05 kernel's units of work, or
                      // (tile_keys 0) of the warp-level kernel's row blocks
  int32_t* quota;     // [1] units of one thread block
  int32_t* row_pos;   // [batch * q_len] position of each query token
};
inline size_t shared_plan_ints(int64_t batch, int64_t q_len, int64_t groups) {
  return static_cast<size_t>(3 * batch + 4 * (groups + 1) + 1 + batch * q_len);
}
// What the plan's choice of the quota goes by, in microseconds of one SM: a
// unit, an own key (of all its KV heads; 0: the own pass does not run beside
// the prefix's), and a row block's start and end.
struct SharedCost {
  float unit, own_key, ramp;
  int sms;
};
int launch_shared_plan(const int32_t* kv_indptr, const int32_t* page_indptr,
                       const int32_t* group_indptr, const int32_t* prefix_lens, int32_t groups,
                       int32_t page_size, int32_t batch, int32_t q_len, int32_t max_prefix,
                       int32_t max_suffix, int32_t block_tokens, int32_t tile_keys, int32_t Hkv,
                       int32_t window, int32_t splits, const SharedCost& cost, const SharedPlan& plan,
                       cudaStream_t stream);

// The groups' prefixes on the tcgen05/TMEM path: partials of every query row
// over its group's prefix (a.batch: groups, a.total_q: query tokens).
int launch_prefix_tc(const AttnArgs& a, const SharedPlan& plan, cudaStream_t stream);
int prefix_block_tokens(int G);            // query tokens of one row block
int prefix_tile_keys(int d, bool fp8);     // keys of one K/V tile

// Reads and clears the device status word of one translation unit.
int read_status_pages(cudaStream_t s, int* status);
int read_status_shared(cudaStream_t s, int* status);
int read_status_prefix_tc(cudaStream_t s, int* status);
int read_status_attn_mma(cudaStream_t s, int* status);
int read_status_merge(cudaStream_t s, int* status);
int read_status_prefill_tc(cudaStream_t s, int* status);
int read_status_decode_tc(cudaStream_t s, int* status);

// Failure-detection test hooks of one translation unit (wait limit in clock
// cycles, <= 0: the default; KV tile the first thread block's producer leaves
// out, -1: none). Host, synchronous.
int set_hooks_attn_mma(long long limit, int skip);
int set_hooks_prefill_tc(long long limit, int skip);
int set_hooks_decode_tc(long long limit, int skip);
int set_hooks_prefix_tc(long long limit, int skip);
int set_hooks_pages(long long limit, int skip);

// Thread-local error text used by the C ABI.
void set_error(const char* fmt, ...);

// Number of SMs on the current device (queried once).
int sm_count();

}  // namespace sinkattn
