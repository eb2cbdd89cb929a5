/*
 * sinkattn — grouped-query attention with a learned per-head softmax sink,
 * for NVIDIA GB300 (sm_103a).
 *
 * The operation ("GPT-OSS on Day 0", Perplexity, section "Kernels for GPT-OSS /
 * Sink attention"; "Attention: GQA with attention sinks"):
 *
 *     attn = softmax(q @ k^T * sm_scale + sink) * V
 *
 * where the sink s_h of query head h is one extra logit column whose value row
 * is zero:
 *
 *     out_i = sum_j e^{l_j - M} v_j / (e^{s_h - M} + sum_j e^{l_j - M}),
 *     l_j   = sm_scale * q_i . k_j,   M = max(s_h, max_j l_j),
 *     lse_i = M + ln(e^{s_h - M} + sum_j e^{l_j - M})      (natural log, sink included).
 *
 * Several query heads share one KV head (GQA): query head h reads KV head
 * floor(h / G), G = num_qo_heads / num_kv_heads. The online softmax seeds its
 * running max with the head's sink (m = s_h, d = 1), so the sink is counted
 * exactly once; when the keys are split into chunks (split-KV decode), the
 * chunks carry no sink and the merge seeds with it (same section: the sink
 * belongs to one block only).
 *
 * Layouts (all device memory, row-major, contiguous):
 *   q, out       bf16 [total_q, Hq, d]  (token-major). Decode: total_q = batch*q_len,
 *                token b*q_len + t is draft t of sequence b.
 *   k, v         bf16 ragged HND ("Hosting Qwen on Blackwell", section "Deployment on
 *                GB200 NVL72": heads leading, tokens contiguous): sequence b is the
 *                contiguous block [Hkv, Lk_b, d] starting at element Hkv*cu_k[b]*d.
 *   sinks        fp32 [Hq], natural-log units of the scaled logits; NULL = no sink.
 *   lse          fp32 [total_q, Hq]; NULL = not written.
 *   cu_seqlens_* int32 [batch+1], non-decreasing, cu[0] = 0 (device memory).
 *
 * Masking: query i of a sequence with Lq queries and Lk keys sits at position
 * p = Lk - Lq + i (queries are the last Lq positions). causal: key j visible
 * iff j <= p. window W > 0 (requires causal): additionally j > p - W, i.e. the
 * W keys p-W+1 .. p. A row with no visible key and no sink gets out = 0,
 * lse = -inf; with a sink and no key, out = 0, lse = s_h.
 *
 * Supported: head_dim 64 or 128; num_qo_heads % num_kv_heads == 0; sm_scale > 0.
 *
 * Ownership and streams: the caller allocates and owns every buffer,
 * including the decode workspace. The library never allocates, frees or
 * synchronises in these calls; it enqueues kernels on `stream` (a
 * cudaStream_t; NULL = legacy default stream) and returns. Inputs are read
 * only. q, k, v, out and the partial buffers must be 16-byte aligned.
 *
 * Errors: every call validates its arguments on the host before launching
 * anything and returns a status code; on error nothing is launched and
 * sinkattn_last_error() (thread-local) describes the problem. Faults inside a
 * kernel (for example a bounded wait that gave up, or device-side lengths
 * that contradict the host-side sizes) are recorded in a device status word
 * that sinkattn_debug_status() reads.
 */
#ifndef SINKATTN_H_
#define SINKATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SINKATTN_API __attribute__((visibility("default")))
#else
#define SINKATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

enum sinkattn_status {
  SINKATTN_OK = 0,
  SINKATTN_INVALID_ARG = 1,  /* null/misaligned pointer, negative size, bad workspace */
  SINKATTN_UNSUPPORTED = 2,  /* head_dim not 64/128, Hq % Hkv != 0, window without causal */
  SINKATTN_CUDA_ERROR = 3,   /* a CUDA runtime/driver call or launch failed */
  SINKATTN_TIMEOUT = 4,      /* device status: a bounded wait inside a kernel gave up */
  SINKATTN_BAD_LENGTHS = 5,  /* device status: cu_seqlens/kv_indptr contradict the host sizes */
  SINKATTN_OUT_OF_PAGES = 6, /* device status: a page table had fewer free pages than a call needs */
  SINKATTN_BAD_PAGES = 7     /* device status: sequence ids or lengths a page table cannot serve */
};

/*
 * Prefill / varlen attention with sink, single pass (no split), output
 * normalised. Steps: logits, mask, online softmax seeded with the sink,
 * P·V, finalize ("GPT-OSS on Day 0", "Kernels for GPT-OSS / Sink attention").
 *
 *   q [total_q, Hq, d], k/v ragged HND, sinks [Hq] or NULL,
 *   cu_seqlens_q / cu_seqlens_k [batch+1] (device),
 *   batch, total_q, max_seqlen_q, max_seqlen_k: host-side sizes for the grid
 *     (max_seqlen_* must bound every sequence; total_q = cu_seqlens_q[batch]),
 *   causal (0/1), window (<= 0: none; > 0 requires causal),
 *   out [total_q, Hq, d] bf16, lse [total_q, Hq] fp32 or NULL.
 * Each sequence needs Lq_b <= Lk_b.
 */
SINKATTN_API int sinkattn_prefill(const void* q, const void* k, const void* v, const float* sinks,
                     const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t batch,
                     int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                     int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                     float sm_scale, int32_t causal, int32_t window, void* out, float* lse,
                     void* stream);

/*
 * Split-KV decode / MTP, step 1: per-chunk partial state WITHOUT the sink
 * (heads and KV length both parallel: same section, "parallelise over heads
 * and KV sequence length").
 *
 *   q [batch*q_len, Hq, d] bf16; k/v ragged HND with kv_indptr [batch+1] (device);
 *   max_kv_len bounds every Lk_b (host); each sequence needs Lk_b >= q_len.
 *   Sequence b's keys are cut into num_splits chunks of
 *   c = 64 * ceil(Lk_b / (64 * num_splits)) keys (ceil(Lk_b / num_splits)
 *   rounded up to whole 64-key tiles); chunk s covers
 *   [s*c, min((s+1)*c, Lk_b)) and may be empty.
 *   part_md:  fp32 [batch*q_len, Hq, num_splits, 2]: (m_s, d_s), natural
 *             units, with m_s + ln d_s = ln sum_j e^{l_j}, the chunk's
 *             log-sum-exp over its visible keys;
 *   part_acc: fp32 [batch*q_len, Hq, num_splits, d]: d_s times the chunk's
 *             softmax-weighted mean of v_j, i.e. sum_j e^{l_j - m_s} v_j.
 *   The pair is defined up to the common rescale (m_s + c, d_s e^{-c},
 *   acc e^{-c}), which the merge is invariant to. The warp-level kernel
 *   writes m_s = the chunk's largest visible logit and d_s = the exact sum;
 *   the tcgen05 kernel writes d_s = the sum of the bf16-rounded weights its
 *   P.V product applied, with m_s adjusted so that m_s + ln d_s stays exact.
 *   An empty chunk gives (-inf, 0) and acc 0.
 */
SINKATTN_API int sinkattn_decode_split(const void* q, const void* k, const void* v,
                          const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                          int32_t max_kv_len, int32_t num_qo_heads, int32_t num_kv_heads,
                          int32_t head_dim, float sm_scale, int32_t causal, int32_t window,
                          int32_t num_splits, float* part_acc, float* part_md, void* stream);

/*
 * Split-KV decode / MTP, step 2: fold the num_splits partials of every
 * (row, head) with the sink counted exactly once: the running state starts at
 * m = s_h, d = 1 (m = -inf, d = 0 without a sink) and absorbs each chunk with
 * the rescale to the larger maximum; out = acc / d, lse = m + ln d ("GPT-OSS
 * on Day 0", section "Kernels for GPT-OSS / Sink attention": the running max
 * m and scale d of the online softmax, the max seeded with the sink and d
 * with 1, the sink in the first block only when the sequence is split).
 *   part_acc/part_md as produced by sinkattn_decode_split; rows = batch*q_len;
 *   out [rows, Hq, d] bf16; lse [rows, Hq] fp32 or NULL.
 */
SINKATTN_API int sinkattn_merge(const float* part_acc, const float* part_md, const float* sinks,
                   int32_t rows, int32_t num_qo_heads, int32_t head_dim, int32_t num_splits,
                   void* out, float* lse, void* stream);

/*
 * Split-KV decode / MTP in one call ("GPT-OSS on Day 0", section "Kernels for
 * GPT-OSS / Sink attention": parallel over heads and KV length, the sink
 * counted once; "Hosting Qwen on Blackwell", section "Decoders": MTP drafts,
 * q_len > 1, attend causally to the cache): sinkattn_decode_split then
 * sinkattn_merge on the same stream, with the partials in the caller's workspace (at least
 * sinkattn_decode_workspace_bytes() bytes, 256-byte aligned, device memory;
 * contents on entry do not matter). num_splits <= 0 selects
 * sinkattn_decode_default_splits(). When a KV head has more query rows than
 * one 128-row tile (G x q_len > 128, e.g. 16 drafts of 16 heads) and the
 * kernel choice is SINKATTN_DECODE_AUTO, the call runs the single-pass
 * prefill kernel instead (the drafts are its queries, bottom-right causal,
 * every KV tile read once); the workspace is then unused and num_splits has
 * no effect on the result.
 */
SINKATTN_API int sinkattn_decode(const void* q, const void* k, const void* v, const int32_t* kv_indptr,
                    int32_t batch, int32_t q_len, int32_t max_kv_len, int32_t num_qo_heads,
                    int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
                    int32_t window, int32_t num_splits, const float* sinks, void* workspace,
                    size_t workspace_bytes, void* out, float* lse, void* stream);

/*
 * Split-KV decode / MTP with the merge done on chip (no workspace): the
 * num_splits chunks of one (sequence, KV head) run as one thread-block
 * cluster; each chunk's partial (m, d, acc) stays in its CTA's shared memory
 * and the cluster folds them through distributed shared memory, seeding the
 * running state with the sink so it counts exactly once ("GPT-OSS on Day 0",
 * section "Kernels for GPT-OSS / Sink attention": parallel over heads and KV
 * length, the sink in one block only). Same chunking and results as
 * sinkattn_decode_split followed by sinkattn_merge.
 *   Arguments as sinkattn_decode without the workspace; num_splits <= 0
 *   selects sinkattn_decode_default_splits(); 1 <= num_splits <= 16 (a
 *   cluster of more than 16 CTAs is not launched: SINKATTN_UNSUPPORTED).
 *   out [batch*q_len, Hq, d] bf16; lse [batch*q_len, Hq] fp32 or NULL.
 */
SINKATTN_API int sinkattn_decode_fused(const void* q, const void* k, const void* v,
                                       const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                                       int32_t max_kv_len, int32_t num_qo_heads,
                                       int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                                       int32_t causal, int32_t window, int32_t num_splits,
                                       const float* sinks, void* out, float* lse, void* stream);

/*
 * sinkattn_decode for callers that cannot allocate device memory (for example
 * code inside another runtime whose memory manager owns all device memory and
 * gives plugins no allocator, or loops where a cudaMalloc, which may
 * synchronise the device, is not acceptable). The pages have no counterpart:
 * this is a deployment convenience, not part of the method.
 *
 * Same arguments and results as sinkattn_decode minus the workspace: the
 * partials live in a fixed 32 MiB array inside the library's own device
 * memory (every GPU that loads the library holds it until the process exits).
 * Calls whose partials need more than that (sinkattn_decode_workspace_bytes)
 * are rejected with SINKATTN_UNSUPPORTED before anything launches. The call
 * allocates nothing and frees nothing.
 *
 * Set-up: the first call in each CUDA context looks up the array's device
 * address (with that context current) and caches it under the context's
 * unique id; make that first call before any stream capture. A new context
 * (after cudaDeviceReset, or a non-primary context made current by another
 * runtime) gets its own lookup on its first call. `stream` must belong to the
 * current device (SINKATTN_INVALID_ARG otherwise, nothing launched): the
 * address is only valid on that device. Every call shares the one array:
 * calls whose kernels may overlap on the GPU (different streams, or several
 * host threads) race on it and must be serialised by the caller. Nothing
 * needs clearing between calls.
 */
SINKATTN_API int sinkattn_decode_noalloc(const void* q, const void* k, const void* v,
                                         const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                                         int32_t max_kv_len, int32_t num_qo_heads,
                                         int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                                         int32_t causal, int32_t window, int32_t num_splits,
                                         const float* sinks, void* out, float* lse, void* stream);

/* Workspace bytes sinkattn_decode needs for these sizes (host only, no CUDA call). */
SINKATTN_API int sinkattn_decode_workspace_bytes(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                    int32_t head_dim, int32_t num_splits, size_t* bytes);

/*
 * The split count sinkattn_decode and sinkattn_decode_fused use when given
 * num_splits <= 0: enough (sequence, KV head, chunk) work items to fill every
 * SM several times over, without chunks shorter than a few KV tiles; at most
 * 16. Host only; queries the current device's SM count once.
 */
SINKATTN_API int sinkattn_decode_default_splits(int32_t batch, int32_t q_len, int32_t num_qo_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t max_kv_len,
                                   int32_t* num_splits);

/*
 * Which kernel computes the split-KV partials (sinkattn_decode_split, and so
 * sinkattn_decode and sinkattn_decode_noalloc). Process-wide, host only.
 *   SINKATTN_DECODE_AUTO (0, default): the tcgen05 kernel at head_dim 128,
 *     the warp-level kernel at head_dim 64;
 *   SINKATTN_DECODE_WARP (1): the warp-level (mma.sync) kernel;
 *   SINKATTN_DECODE_TCGEN05 (2): the tcgen05/TMEM kernel (head_dim 128;
 *     the query tokens x heads of a GQA group fill up to 128 MMA rows, e.g.
 *     3 MTP tokens x 16 heads = 48); head_dim 64 then returns
 *     SINKATTN_UNSUPPORTED.
 * Both kernels produce the same partial layout and meaning. Returns
 * SINKATTN_INVALID_ARG for any other value.
 */
#define SINKATTN_DECODE_AUTO 0
#define SINKATTN_DECODE_WARP 1
#define SINKATTN_DECODE_TCGEN05 2
SINKATTN_API int sinkattn_set_decode_kernel(int kind);

/*
 * Process-wide choice of the prefill launch (both run the same tcgen05
 * kernel body and give the same results up to floating-point rounding order):
 *   SINKATTN_PREFILL_AUTO (0, default): persistent when the work items are
 *     short (a sliding window, or prompts of a few KV tiles) or when there
 *     are at least 16 items per SM; else one block per item;
 *   SINKATTN_PREFILL_ONE_BLOCK (1): one thread block per (query block, KV
 *     head, sequence), scheduled by the hardware;
 *   SINKATTN_PREFILL_PERSISTENT (2): one thread block per SM working through
 *     a fixed list of items, streaming K/V across item boundaries.
 * Returns SINKATTN_INVALID_ARG for any other value.
 */
#define SINKATTN_PREFILL_AUTO 0
#define SINKATTN_PREFILL_ONE_BLOCK 1
#define SINKATTN_PREFILL_PERSISTENT 2
SINKATTN_API int sinkattn_set_prefill_kernel(int kind);

/*
 * Paged KV cache (HND within a page: heads leading, tokens contiguous): the
 * same operations as sinkattn_prefill, sinkattn_decode_split and
 * sinkattn_decode, with K and V held in page pools
 *   k_pages, v_pages: bf16 [num_pages, Hkv, page_size, d] (device)
 * and sequence b's keys [e * page_size, (e + 1) * page_size) in page
 * page_indices[page_indptr[b] + e]:
 *   page_indptr  int32 [batch + 1] (device), page_indices int32
 *   [page_indptr[batch]] (device), each entry in [0, num_pages).
 * Key counts still come from cu_seqlens_k / kv_indptr (only their
 * differences are used); sequence b needs at least ceil(Lk_b / page_size)
 * pages -- fewer makes the kernel record SINKATTN_BAD_LENGTHS (see
 * sinkattn_debug_status). page_size is a power of two in [16, 256]
 * (SINKATTN_UNSUPPORTED otherwise); num_pages * Hkv * page_size < 2^31.
 * Slots of the last page past Lk_b are read and masked (weight 0): they must
 * hold finite values (a zero-initialised pool does). A page index outside
 * [0, num_pages) gives undefined values for its sequence but no read outside
 * the pools (the copy engine bounds every copy by the pool's extent).
 * Every other argument, layout, rule and result is that of the contiguous
 * entry point; in particular the partials and the merge are the same.
 */
SINKATTN_API int sinkattn_prefill_paged(const void* q, const void* k_pages, const void* v_pages,
                                        const float* sinks, const int32_t* cu_seqlens_q,
                                        const int32_t* cu_seqlens_k, const int32_t* page_indptr,
                                        const int32_t* page_indices, int32_t num_pages,
                                        int32_t page_size, int32_t batch, int32_t total_q,
                                        int32_t max_seqlen_q, int32_t max_seqlen_k,
                                        int32_t num_qo_heads, int32_t num_kv_heads,
                                        int32_t head_dim, float sm_scale, int32_t causal,
                                        int32_t window, void* out, float* lse, void* stream);
SINKATTN_API int sinkattn_decode_split_paged(const void* q, const void* k_pages,
                                             const void* v_pages, const int32_t* kv_indptr,
                                             const int32_t* page_indptr,
                                             const int32_t* page_indices, int32_t num_pages,
                                             int32_t page_size, int32_t batch, int32_t q_len,
                                             int32_t max_kv_len, int32_t num_qo_heads,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             float sm_scale, int32_t causal, int32_t window,
                                             int32_t num_splits, float* part_acc, float* part_md,
                                             void* stream);
SINKATTN_API int sinkattn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                       const int32_t* kv_indptr, const int32_t* page_indptr,
                                       const int32_t* page_indices, int32_t num_pages,
                                       int32_t page_size, int32_t batch, int32_t q_len,
                                       int32_t max_kv_len, int32_t num_qo_heads,
                                       int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                                       int32_t causal, int32_t window, int32_t num_splits,
                                       const float* sinks, void* workspace,
                                       size_t workspace_bytes, void* out, float* lse,
                                       void* stream);

/*
 * FP8 KV cache: sinkattn_decode_split and sinkattn_decode with K and V held
 * as e4m3 codes (the OCP 8-bit floating-point format E4M3, one byte per
 * element, in the same ragged HND layout) and per-KV-head fp32 scales:
 *   k, v:     uint8 codes [Hkv * total_k, d] (device);
 *   k_scale:  float [Hkv] (device): key j of KV head g is code * k_scale[g];
 *   v_scale:  float [Hkv] (device): value j of KV head g is code * v_scale[g].
 * Every other argument, layout, result, the partials and the merge are those
 * of the bf16 entry points ("GPT-OSS on Day 0", section "Kernels for GPT-OSS /
 * Sink attention", with the keys and values dequantised). The kernel widens
 * the codes to f16, which holds every e4m3 value exactly, and runs the
 * products in f16 with q converted to f16: |q| must stay below 65504, and
 * q elements below 2^-14 in magnitude lose relative precision. Kernel
 * choice (sinkattn_set_decode_kernel): at head_dim 128 with at most 64 query
 * heads per KV head the tcgen05 kernel runs (AUTO or TCGEN05), other shapes
 * take the warp-level kernel (TCGEN05 forced there: SINKATTN_UNSUPPORTED).
 * k_scale / v_scale null or misaligned: SINKATTN_INVALID_ARG.
 */
SINKATTN_API int sinkattn_decode_split_fp8(const void* q, const void* k, const void* v,
                                           const float* k_scale, const float* v_scale,
                                           const int32_t* kv_indptr, int32_t batch,
                                           int32_t q_len, int32_t max_kv_len,
                                           int32_t num_qo_heads, int32_t num_kv_heads,
                                           int32_t head_dim, float sm_scale, int32_t causal,
                                           int32_t window, int32_t num_splits, float* part_acc,
                                           float* part_md, void* stream);
SINKATTN_API int sinkattn_decode_fp8(const void* q, const void* k, const void* v,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* kv_indptr, int32_t batch, int32_t q_len,
                                     int32_t max_kv_len, int32_t num_qo_heads,
                                     int32_t num_kv_heads, int32_t head_dim, float sm_scale,
                                     int32_t causal, int32_t window, int32_t num_splits,
                                     const float* sinks, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     void* stream);

/*
 * Decode over a paged cache whose sequences share prefixes: the same result as
 * sinkattn_decode_paged over the same page lists, with the shared pages read
 * and multiplied once for all sequences that share them. The partials and
 * the merge are those of split-KV decode, so the sink counts once.
 *   The batch is cut into num_groups runs of consecutive sequences:
 *   group_indptr int32 [num_groups + 1] (device; group g holds sequences
 *   group_indptr[g] .. group_indptr[g+1] - 1, group_indptr[0] = 0,
 *   group_indptr[num_groups] = batch, non-decreasing), and
 *   prefix_lens int32 [num_groups] (device): the first prefix_lens[g] keys of
 *   every sequence of group g are the same, a multiple of page_size (0: the
 *   group shares nothing). They are read from the first sequence's page list;
 *   every list still holds all of its own sequence's pages.
 *   Each sequence needs Lk_b >= prefix_lens[g] + q_len (the drafts' own keys
 *   are not shared), so every query sees the whole prefix but for the window.
 *   max_prefix_len / max_suffix_len (host) bound prefix_lens[g] and
 *   Lk_b - prefix_lens[g]; lengths and groups that break one of these rules
 *   make the call record SINKATTN_BAD_LENGTHS (sinkattn_debug_status), and the
 *   results of the sequences concerned are not defined.
 *   sinkattn_set_decode_kernel decides for the prefixes too: AUTO takes the
 *   tcgen05 kernel where a group has more than 48 query rows per KV head on
 *   average. TCGEN05 takes it for both parts, which needs head_dim 128 and bf16
 *   pools (SINKATTN_UNSUPPORTED otherwise).
 *   prefix_splits / num_splits: KV chunks of a prefix and of a sequence's own
 *   keys; <= 0 selects sinkattn_decode_shared_default_splits(). Its
 *   prefix_splits is 0 for a call of so few keys that it is faster to let every
 *   sequence read all of its own (num_splits then cuts those).
 *   workspace: at least sinkattn_decode_shared_workspace_bytes() bytes for
 *   the split counts in use, 256-byte aligned, device memory; contents on
 *   entry do not matter. Two calls that may overlap need two workspaces.
 * A sequence whose own keys or values hold NaN gets NaN, in lse too where its
 * keys do; the other sequences of its group do not.
 * Every other argument and rule is that of sinkattn_decode_paged
 * (num_kv_heads groups of at most 64 query heads). The _fp8 form reads pools
 * of e4m3 codes, uint8 [num_pages, Hkv, page_size, d], with the scales and
 * rules of sinkattn_decode_fp8.
 */
SINKATTN_API int sinkattn_decode_shared_paged(
    const void* q, const void* k_pages, const void* v_pages, const int32_t* kv_indptr,
    const int32_t* page_indptr, const int32_t* page_indices, const int32_t* group_indptr,
    const int32_t* prefix_lens, int32_t num_groups, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t q_len, int32_t max_prefix_len, int32_t max_suffix_len,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t causal,
    int32_t window, int32_t prefix_splits, int32_t num_splits, const float* sinks,
    void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream);
SINKATTN_API int sinkattn_decode_shared_paged_fp8(
    const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
    const float* v_scale, const int32_t* kv_indptr, const int32_t* page_indptr,
    const int32_t* page_indices, const int32_t* group_indptr, const int32_t* prefix_lens,
    int32_t num_groups, int32_t num_pages, int32_t page_size, int32_t batch, int32_t q_len,
    int32_t max_prefix_len, int32_t max_suffix_len, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, float sm_scale, int32_t causal, int32_t window, int32_t prefix_splits,
    int32_t num_splits, const float* sinks, void* workspace, size_t workspace_bytes, void* out,
    float* lse, void* stream);

/* Workspace bytes of the shared-prefix decode for these sizes (host only, no CUDA call). */
SINKATTN_API int sinkattn_decode_shared_workspace_bytes(int32_t batch, int32_t q_len,
                                                        int32_t num_qo_heads, int32_t head_dim,
                                                        int32_t num_groups, int32_t prefix_splits,
                                                        int32_t num_splits, size_t* bytes);

/* The split counts the shared-prefix decode uses when given <= 0 (host only);
 * prefix_splits 0: every sequence reads its own keys. */
SINKATTN_API int sinkattn_decode_shared_default_splits(
    int32_t batch, int32_t q_len, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t num_groups, int32_t max_prefix_len, int32_t max_suffix_len, int32_t* prefix_splits,
    int32_t* num_splits);

/*
 * Writes new keys and values into page pools.
 *   k, v: bf16 [tokens, Hkv, d] (device), rows of one token contiguous, token
 *     i at element i * k_stride (v_stride): multiples of 8 and at least
 *     Hkv * d, so slices of a fused projection's output need no copy;
 *   slots: int32 [tokens] (device), slot = page * page_size + position in the
 *     page, as sinkattn_pages_reserve gives them; a token whose slot lies
 *     outside [0, num_pages * page_size) is left out (padding: -1);
 *   k_pages, v_pages: the pools, bf16 [num_pages, Hkv, page_size, d], or for
 *     the _fp8 form uint8 e4m3 codes of the same shape: the code is the e4m3
 *     value nearest to x / scale[head] (the fp32 quotient; ties to even; beyond
 *     +-448 the largest code of that sign; NaN the NaN code).
 * Two tokens with the same slot leave one of the two rows' elements.
 */
SINKATTN_API int sinkattn_append_paged(const void* k, const void* v, int64_t k_stride,
                                       int64_t v_stride, const int32_t* slots, int32_t tokens,
                                       void* k_pages, void* v_pages, int32_t num_pages,
                                       int32_t page_size, int32_t num_kv_heads, int32_t head_dim,
                                       void* stream);
SINKATTN_API int sinkattn_append_paged_fp8(const void* k, const void* v, int64_t k_stride,
                                           int64_t v_stride, const int32_t* slots, int32_t tokens,
                                           const float* k_scale, const float* v_scale,
                                           void* k_pages, void* v_pages, int32_t num_pages,
                                           int32_t page_size, int32_t num_kv_heads,
                                           int32_t head_dim, void* stream);

/*
 * Page tables: which pages each sequence holds, how many sequences hold each
 * page, and which pages are free. One table serves all layers of a cache
 * (page p is page p of every layer's pools).
 * A table is one int32 device buffer of sinkattn_pages_table_ints() words,
 * 16-byte aligned, owned by the caller:
 *   word 0                 number of free pages (words 1 .. 15: scratch)
 *   seq_lens  [max_seqs]             tokens of each sequence
 *   page_list [max_seqs][max_pages]  its pages in order; -1 past the last
 *   refcount  [num_pages]            lists that hold the page
 *   free_list [num_pages]            the free pages are its first word-0 entries
 *   scratch   [7 * max_seqs + 2 * num_pages]
 * The j-th page that a call takes is free_list[count - 1 - j]; the j-th of K
 * pages that it gives back goes to free_list[count + K - 1 - j]: results do
 * not depend on timing. sinkattn_pages_init makes every page free (the first
 * page taken is page 0) and every sequence empty.
 * A call that cannot be served as a whole changes nothing and records
 * SINKATTN_OUT_OF_PAGES, SINKATTN_BAD_PAGES (an id outside [0, max_seqs), an
 * id twice, a length the table cannot hold, a free count outside
 * [0, num_pages]) or SINKATTN_BAD_LENGTHS (cu_new contradicts total_new); see
 * sinkattn_debug_status. Calls on one table must
 * be ordered (one stream, or events); max_seqs <= 2^18, max_seqs * max_pages
 * < 2^30, total_new < 2^30, page_size as for the paged attention.
 * Where a call copies pages it takes the pools of all layers:
 *   k_pages, v_pages [num_layers][num_pages][Hkv][page_size] rows of
 *   row_bytes bytes (d * 2, or d for codes; a multiple of 16), one layer
 *   layer_stride bytes after the other (a multiple of 16, at least one
 *   layer's bytes unless num_layers is 1).
 */
SINKATTN_API int sinkattn_pages_table_ints(int32_t num_pages, int32_t max_seqs, int32_t max_pages,
                                           int64_t* ints);
SINKATTN_API int sinkattn_pages_init(int32_t* table, int32_t num_pages, int32_t page_size,
                                     int32_t max_seqs, int32_t max_pages, void* stream);

/*
 * Room for new tokens at the ends of n sequences: sequence seq_ids[i] grows by
 * cu_new[i+1] - cu_new[i] tokens (seq_ids int32 [n], cu_new int32 [n + 1],
 * device; total_new = cu_new[n], host), taking pages in the order of i, and
 * slots [total_new] (device) gets each new token's slot. A sequence that
 * starts inside a page that other sequences also hold first gets a page of
 * its own, with the rows in use copied in every layer (copy on write): all
 * writers do, except that when every holder writes in this call the first of
 * them keeps the page. A call that cannot be served fills slots with -1.
 * A page keeps what it held before: the attention reads and masks the slots
 * past a sequence's length, so rows that are written have to be finite.
 * With total_new 0 nothing is read or written.
 */
SINKATTN_API int sinkattn_pages_reserve(int32_t* table, int32_t num_pages, int32_t page_size,
                                        int32_t max_seqs, int32_t max_pages,
                                        const int32_t* seq_ids, const int32_t* cu_new, int32_t n,
                                        int32_t total_new, void* k_pages, void* v_pages,
                                        int32_t num_layers, int64_t layer_stride,
                                        int32_t num_kv_heads, int32_t row_bytes, int32_t* slots,
                                        void* stream);

/*
 * dst_ids[i] becomes a copy of src_ids[i] that shares all of its pages (the
 * partly filled last one too: the first append to it copies it). The dst
 * sequences must be empty, distinct and no src of the same call.
 */
SINKATTN_API int sinkattn_pages_fork(int32_t* table, int32_t num_pages, int32_t page_size,
                                     int32_t max_seqs, int32_t max_pages, const int32_t* src_ids,
                                     const int32_t* dst_ids, int32_t n, void* stream);

/*
 * Shortens seq_ids[i] to new_lens[i] tokens (0 <= new_lens[i] <= its length;
 * new_lens NULL: 0, which frees the sequence). Pages past the new end leave
 * its list; those that no list holds any more are free again, given back in
 * the order (i, position in the list) of their first appearance.
 */
SINKATTN_API int sinkattn_pages_truncate(int32_t* table, int32_t num_pages, int32_t page_size,
                                         int32_t max_seqs, int32_t max_pages,
                                         const int32_t* seq_ids, const int32_t* new_lens,
                                         int32_t n, void* stream);

/*
 * Packs the L pages in use into pages 0 .. L - 1: the live pages at or above L
 * move, in order, into the free ones below L, in every layer; lists and
 * reference counts follow, and the free list becomes num_pages - 1 .. L.
 * page_map int32 [num_pages] (device): the new index of each old page, -1
 * where it was free.
 */
SINKATTN_API int sinkattn_pages_compact(int32_t* table, int32_t num_pages, int32_t page_size,
                                        int32_t max_seqs, int32_t max_pages, void* k_pages,
                                        void* v_pages, int32_t num_layers, int64_t layer_stride,
                                        int32_t num_kv_heads, int32_t row_bytes,
                                        int32_t* page_map, void* stream);

/*
 * The paged attention's view of n <= 2^18 sequences of a table (an id may come
 * more than once): kv_indptr [n + 1] and page_indptr [n + 1] (running sums of
 * lengths and of page counts), and their page lists one after the other in
 * page_indices (capacity entries; what lies past the last list stays as it
 * was). Lists that do not fit, and lengths whose sum passes 2^31 - 1, record
 * SINKATTN_BAD_LENGTHS and are left out; an id outside the table counts as an
 * empty sequence and records SINKATTN_BAD_PAGES. With n 0 the first entries,
 * zero, are written where the pointers are given.
 */
SINKATTN_API int sinkattn_pages_lists(const int32_t* table, int32_t num_pages, int32_t page_size,
                                      int32_t max_seqs, int32_t max_pages,
                                      const int32_t* seq_ids, int32_t n, int32_t* kv_indptr,
                                      int32_t* page_indptr, int32_t* page_indices,
                                      int32_t capacity, void* stream);

/*
 * Gradients of sinkattn_prefill. With P_ij = e^{l_ij - lse_i} over the visible
 * keys, delta_i = dout_i . out_i - dlse_i and dS_ij = P_ij (dout_i . v_j - delta_i):
 *   dq_i = sm_scale sum_j dS_ij k_j        dk_j = sm_scale sum_i dS_ij q_i
 *   dv_j = sum_i P_ij dout_i               dsinks_h = -sum_i e^{s_h - lse_i} delta_i
 * with the sums over i also over the query heads of the KV head's group. The
 * derivation is that of the softmax with the sink as one more column whose
 * value row is zero; the pages hold no training.
 *   dout, out, q, dq: bf16 [total_q, Hq, d]; k, v, dk, dv: bf16 ragged HND,
 *     [Hkv * total_k, d]; lse fp32 [total_q, Hq]; sinks, dsinks fp32 [Hq] or
 *     NULL, both or neither; dlse fp32 [total_q, Hq] or NULL: the gradient of lse.
 *     out and lse are what sinkattn_prefill gave for these q, k, v and sinks.
 *   cu_seqlens_*, batch, max_seqlen_*, the masks: as there; total_q and total_k
 *     (host) are the tensors' tokens, cu_seqlens_q[batch] and cu_seqlens_k[batch]
 *     at least. max_seqlen_* bound the lengths; each tile within the bound is a
 *     thread block for every sequence and KV head, so a bound far above the lengths
 *     costs time (64 sequences of 256 tokens, 64/8 heads of 64: 0.29 ms with 256, 0.47
 *     with 4096, 1.05 with 2^31 - 1).
 *   workspace: sinkattn_prefill_backward_workspace_bytes() bytes, 256-byte
 *     aligned, device memory; contents on entry do not matter. Two calls that
 *     may overlap need two workspaces.
 * Every element of dq, dk, dv and dsinks up to the last sequence's end is
 * written (zeros where nothing is visible); rows behind it stay as they are.
 * Outputs must not overlap the inputs, which the second pass reads again, or one another.
 * Sums are fp32; P and dS are rounded to bf16 for the products. Results do not
 * depend on timing. A sequence whose inputs hold NaN or infinities gets NaN; the
 * other sequences do not. A row whose lse is -inf has no weights: it gives and gets
 * no gradient. Each sequence needs Lq_b <= Lk_b. Lengths that contradict the host sizes record
 * SINKATTN_BAD_LENGTHS and leave that sequence's gradients and dsinks undefined.
 * (A call of no keys, total_k = 0, or of no sequences reads nothing, cu_seqlens neither;
 * dsinks is zero.)
 */
SINKATTN_API int sinkattn_prefill_backward(
    const void* dout, const void* q, const void* k, const void* v, const void* out,
    const float* lse, const float* sinks, const float* dlse, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int32_t batch, int32_t total_q, int32_t total_k,
    int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, float sm_scale, int32_t causal, int32_t window, void* dq, void* dk, void* dv,
    float* dsinks, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of the backward pass for these sizes (host only, no CUDA call). */
SINKATTN_API int sinkattn_prefill_backward_workspace_bytes(int32_t total_q, int32_t num_qo_heads,
                                                           size_t* bytes);

/*
 * Rotary positions. A head's first rotary_dim elements are cut into pairs, in
 * the interleaved layout (2i, 2i + 1), else (i, i + rotary_dim / 2); pair i is
 * turned by the angle position * f_i and scaled by attention_factor; the other
 * elements stay as they are (without a norm bit for bit, infinities and zeros'
 * signs too). The frequencies are passed as
 *   turns: uint64 [rotary_dim / 2] (device), f_i / (2 pi) modulo 1 in units of 2^-64,
 * rounded to the nearest, so that position times turns is off by at most 2^-34
 * turns at any int32 position (sinkattn_rope_turns makes them from f_i in host
 * memory); cosine and sine are then fp32, of an angle rounded to 2^-26 turns.
 * sinkattn_rope_frequencies (host only) gives f_i = base^(-2i / rotary_dim) and
 * the factor of cosine and sine, scaled for contexts beyond the trained ones:
 *   SINKATTN_ROPE_PLAIN: as they are, attention_factor 1;
 *   SINKATTN_ROPE_LINEAR: f_i / factor;
 *   SINKATTN_ROPE_NTK: base times factor^(r / (r - 2)), r = rotary_dim, which divides the
 *     lowest frequency by factor;
 *   SINKATTN_ROPE_YARN (after "YaRN: Efficient Context Window Extension of Large
 *     Language Models", Peng et al., 2023): pairs that turn more than beta_fast
 *     times within original_len positions keep f_i, those that turn less than
 *     beta_slow times get f_i / factor; between, the share of f_i / factor grows
 *     linearly with the pair's index i, from the index at which a pair turns
 *     beta_fast times (0 at least) to that at which it turns beta_slow times
 *     (rotary_dim - 1 at most), neither of them rounded. attention_factor =
 *     0.1 ln(factor) + 1. This is the ramp of common model code, gpt-oss's among
 *     it; the paper's is linear in the number of turns instead, and other model
 *     code rounds the two indices outwards: for a model made with another rule
 *     compute its f_i and pass those to sinkattn_rope_turns.
 */
#define SINKATTN_ROPE_PLAIN 0
#define SINKATTN_ROPE_LINEAR 1
#define SINKATTN_ROPE_NTK 2
#define SINKATTN_ROPE_YARN 3
SINKATTN_API int sinkattn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling,
                                           double factor, int32_t original_len, double beta_fast,
                                           double beta_slow, double* inv_freq,
                                           float* attention_factor);
SINKATTN_API int sinkattn_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns);

/*
 * From a fused projection's rows to what sinkattn_prefill reads: per-head norm
 * and rotation of queries and keys, and the ragged HND layout, in one pass.
 *   q [tokens, Hq, d], k, v [tokens, Hkv, d] bf16 (device), the heads of a
 *     token contiguous, token i at element i * q_stride (k_stride, v_stride):
 *     multiples of 8, so slices of one projection's output need no copy;
 *   cu_seqlens int32 [batch + 1] (device), tokens = cu_seqlens[batch] (rows
 *     behind it have no effect, and none are written);
 *   positions int32 [tokens] (device), or NULL: the index in the sequence;
 *   q_weight, k_weight fp32 [d] (device) or NULL: y = w * x * rsqrt(mean x^2 +
 *     eps) over the head's d elements before the rotation; NULL: no norm;
 *   q_out bf16 [tokens, Hq, d]; k_out, v_out bf16 ragged HND [Hkv * tokens, d].
 * Arithmetic is fp32, each output is rounded once; the weight multiplies cosine
 * and sine first, the inverse root comes last. (Outputs of a row whose mean square
 * plus eps is 0, as one of zeros without eps, or leaves fp32's range are undefined.)
 * Outputs must not overlap the inputs or one another. cu_seqlens that leave
 * [0, tokens] or decrease record SINKATTN_BAD_LENGTHS; tokens of sequences that
 * leave [0, tokens] are left out, those of sequences that overlap are undefined.
 * (A call of no tokens or no sequences reads nothing, cu_seqlens neither.)
 */
SINKATTN_API int sinkattn_rope_qkv(const void* q, const void* k, const void* v, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                                   const int32_t* positions, int32_t batch, int32_t tokens,
                                   int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                   const uint64_t* turns, int32_t rotary_dim, int32_t interleaved,
                                   float attention_factor, const float* q_weight,
                                   const float* k_weight, float eps, void* q_out, void* k_out,
                                   void* v_out, void* stream);

/*
 * Gradients of sinkattn_rope_qkv. dq bf16 [tokens, Hq, d] and dk, dv bf16
 * ragged HND are those of its outputs; q and k its inputs, read only where there is
 * a norm (NULL otherwise). dq_in, dk_in, dv_in with their token strides get
 * the gradients of q, k, v (rows behind the last sequence stay as they are);
 * dq_weight, dk_weight fp32 [d] those of the weights, summed in an order that
 * does not depend on timing. workspace: sinkattn_rope_qkv_backward_workspace_bytes()
 * bytes, 256-byte aligned, needed where there is a norm. With no tokens the weights'
 * gradients are zero. cu_seqlens are checked as there.
 */
SINKATTN_API int sinkattn_rope_qkv_backward(
    const void* dq, const void* dk, const void* dv, const void* q, const void* k, int64_t q_stride,
    int64_t k_stride, const int32_t* cu_seqlens, const int32_t* positions, int32_t batch,
    int32_t tokens, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    const uint64_t* turns, int32_t rotary_dim, int32_t interleaved, float attention_factor,
    const float* q_weight, const float* k_weight, float eps, void* dq_in, void* dk_in, void* dv_in,
    int64_t dq_stride, int64_t dk_stride, int64_t dv_stride, float* dq_weight, float* dk_weight,
    void* workspace, size_t workspace_bytes, void* stream);
SINKATTN_API int sinkattn_rope_qkv_backward_workspace_bytes(int32_t tokens, int32_t head_dim,
                                                            size_t* bytes);

/*
 * sinkattn_append_paged with the norm and the rotation of sinkattn_rope_qkv on
 * the way: q goes to q_out [tokens, Hq, d], k and v to their slots in the
 * pools. positions int32 [tokens] (device) as the rotation takes them; slots,
 * pools, scales and padding (a slot outside the pool: k and v are left out, q
 * is written) as there. The _fp8 form rounds the fp32 quotient of the rotated
 * key, not rounded to bf16 before, and its scale; where that lies next to the middle
 * of two codes, its own fp32 roundings may decide. v gets the codes that
 * sinkattn_append_paged_fp8 gives.
 */
SINKATTN_API int sinkattn_rope_append_paged(
    const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const int32_t* positions, const int32_t* slots, int32_t tokens,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, const uint64_t* turns,
    int32_t rotary_dim, int32_t interleaved, float attention_factor, const float* q_weight,
    const float* k_weight, float eps, void* q_out, void* k_pages, void* v_pages, int32_t num_pages,
    int32_t page_size, void* stream);
SINKATTN_API int sinkattn_rope_append_paged_fp8(
    const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const int32_t* positions, const int32_t* slots, int32_t tokens,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, const uint64_t* turns,
    int32_t rotary_dim, int32_t interleaved, float attention_factor, const float* q_weight,
    const float* k_weight, float eps, const float* k_scale, const float* v_scale, void* q_out,
    void* k_pages, void* v_pages, int32_t num_pages, int32_t page_size, void* stream);

/* Human-readable name of a status code (static string). */
SINKATTN_API const char* sinkattn_status_string(int status);

/* Description of the last error returned on this thread ("" if none). */
SINKATTN_API const char* sinkattn_last_error(void);

/*
 * Diagnostic, not for the hot path: synchronises `stream`, then reads and
 * clears the device status word of every kernel in the library. *status gets
 * SINKATTN_OK, SINKATTN_TIMEOUT, SINKATTN_BAD_LENGTHS, SINKATTN_OUT_OF_PAGES
 * or SINKATTN_BAD_PAGES. Returns
 * SINKATTN_CUDA_ERROR if the synchronisation or the read failed.
 */
SINKATTN_API int sinkattn_debug_status(void* stream, int* status);

/*
 * Diagnostic, test only (failure detection without a GPU fault; the pages
 * have no counterpart): sets, for every kernel of the library, the number of
 * SM clock cycles a bounded wait allows before it gives up
 * (wait_limit_cycles <= 0 restores the default, about 1 s), and makes the
 * TMA producer of the first thread block of every later launch leave out the
 * copies of its KV tile number skip_tile (-1: none). A left-out tile's
 * waits run out: the kernel records SINKATTN_TIMEOUT (read by
 * sinkattn_debug_status), drains its copies and MMAs, frees its tensor
 * memory and exits; its outputs are then undefined. Host call, synchronous
 * with the device; make it while no kernel of the library is running.
 * skip_tile < -1: SINKATTN_INVALID_ARG.
 */
SINKATTN_API int sinkattn_debug_set_hooks(long long wait_limit_cycles, int skip_tile);

#ifdef __cplusplus
}
#endif

#endif /* SINKATTN_H_ */
