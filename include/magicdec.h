/*
 * magicdec.h -- C ABI of the GB300 (sm_103a) hot path for MagicDec-style
 * long-context self-speculative decoding.
 *
 * Method: "MagicDec: Breaking the Latency-Throughput Tradeoff for Long Context
 * Generation with Speculative Decoding" (arXiv 2408.11049v5).  A target model
 * drafts gamma tokens with attention over a sparse subset of its own KV cache
 * (StreamingLLM sinks + recent window, or SnapKV observation-window top-k,
 * section 4.4), then verifies them with attention of the gamma+1 speculated
 * queries over the full KV cache (section 3.1, T_V(B,S,gamma)), and keeps the
 * accepted prefix by speculative sampling (Leviathan et al., cited for Eq. 1)
 * or greedy matching (section 5.1).
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    allocates nothing and keeps no state between calls, apart from one
 *    device-side error word (see magicdec_device_error).
 *  - bf16 tensors are passed as uint16_t bit patterns.  Layouts are dense
 *    row-major with the shapes given beside each argument.
 *  - Every pointer that a kernel reads or writes in 16-byte vectors must be
 *    16-byte aligned (checked; MAGICDEC_ERR_ALIGN).
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *    validate their arguments on the host, enqueue kernels and return without
 *    synchronising.  A status other than MAGICDEC_OK means nothing was
 *    enqueued, except MAGICDEC_ERR_CUDA, which reports a launch error.
 *  - Per-sequence lengths live on the device and cannot be checked on the
 *    host: kernels clamp them to [0, capacity].
 *  - Inputs must be finite.
 *  - Workspaces are caller-owned device buffers of at least the size the
 *    matching *_workspace_size() returns.  They must be zero-filled once
 *    before first use; every call leaves them ready for the next call.  Calls
 *    that share one workspace must not overlap on the GPU.
 */
#ifndef MAGICDEC_H
#define MAGICDEC_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MAGICDEC_API __attribute__((visibility("default")))
#else
#define MAGICDEC_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MAGICDEC_OK = 0,
    MAGICDEC_ERR_NULL = -1,        /* a required pointer is NULL */
    MAGICDEC_ERR_SHAPE = -2,       /* a size is out of range or inconsistent */
    MAGICDEC_ERR_ALIGN = -3,       /* a pointer is not 16-byte aligned */
    MAGICDEC_ERR_WORKSPACE = -4,   /* workspace smaller than *_workspace_size() */
    MAGICDEC_ERR_UNSUPPORTED = -5, /* a valid shape the library has no kernel for */
    MAGICDEC_ERR_CUDA = -6         /* the CUDA runtime reported an error */
} magicdec_status;

/* Attention problem shape.  KV cache K/V: [B, L_cap, H_kv, d].  Query head hq
 * reads KV head hq / (H_q / H_kv) (grouped-query attention).  d is 64 or 128;
 * H_q must be a multiple of H_kv. */
typedef struct {
    int B;
    int H_q;
    int H_kv;
    int d;
    int L_cap;
} magicdec_kv_shape;

/* Human-readable name of a status code (static string). */
MAGICDEC_API const char *magicdec_status_string(int status);

/* Copies the device error word of the current device into *out and clears it
 * (synchronises the device).  Non-zero means a kernel gave up on a bounded
 * wait (value 1) or met an inconsistent internal state (value 2), and its
 * outputs are then undefined; or that magicdec_draft_cache_update skipped a
 * row whose slot was at or past the cache capacity (value 3; the calls on a
 * paged cache likewise), or that a call on a paged cache met a block-table
 * entry outside the pool (value 5).  In the
 * range-checking build (libmagicdec_debug.so, compiled with
 * MAGICDEC_DEBUG_CHECKS) value 4 means a kernel read a sequence length
 * outside [0, capacity] or a gather index outside [0, L_cap) other than the
 * -1 padding mark (in the calls on trees also a node count outside [0, n], a
 * parent that is not before its node, or a path entry or n_acc that names no
 * node); that build still clamps or skips the value as documented
 * for each call, so its outputs equal the release build's, which records
 * nothing for it.  The first error since the last read is kept.  Returns MAGICDEC_OK or
 * MAGICDEC_ERR_CUDA. */
MAGICDEC_API magicdec_status magicdec_device_error(int32_t *out);

/*
 * StreamingLLM draft-KV selection (paper section 4.4 and section 5.1:
 * attention sinks plus a recent window; budget n_sink + n_recent).
 *   seq_len [B] int32   current sequence lengths (clamped below at 0)
 *   idx     [B, H_kv, n_sink + n_recent] int32 out: for each sequence the
 *           positions [0, min(n_sink, len)) then [max(n_sink, len-n_recent),
 *           len), ascending, identical for every KV head; -1 after n_sel[b].
 *   n_sel   [B] int32 out: number of valid entries per sequence.
 * Errors: NULL pointers, B <= 0, H_kv <= 0, n_sink < 0, n_recent < 0,
 * n_sink + n_recent == 0 or above INT_MAX; MAGICDEC_ERR_UNSUPPORTED when B or H_kv exceeds
 * 65535 (the kernel's grid has one block row per KV head and sequence).
 */
MAGICDEC_API magicdec_status magicdec_streaming_select(const int32_t *seq_len, int B, int H_kv, int n_sink,
                                          int n_recent, int32_t *idx, int32_t *n_sel, void *stream);

/* Workspace bytes magicdec_snapkv_select needs for this shape and window. */
MAGICDEC_API size_t magicdec_snapkv_workspace_size(magicdec_kv_shape shape, int window);

/*
 * SnapKV draft-KV selection, run once after prefill (paper section 4.4: a
 * static method whose compact cache is built once; section 5.2: best budget
 * about 2048).  For each sequence of length L = seq_len[b] (clamped to
 * [0, L_cap]) and KV head h, the last `window` positions form the
 * observation window; window row r (position L-window+r) of query head hq has
 * query q_win[b, r, hq, :] and attends causally over positions 0..L-window+r.
 * The score of a prefix position j < L-window is the sum over window rows and
 * over the H_q/H_kv query heads of the group of the softmax probability at j.
 * Scores are max-pooled (kernel pool_kernel, stride 1, clipped at the ends),
 * the budget-window largest are kept (ties to the smaller position), sorted
 * ascending, and the window positions [L-window, L) are appended.  When
 * L <= budget all positions 0..L-1 are kept.
 *   q_win [B, window, H_q, d] bf16;  k [B, L_cap, H_kv, d] bf16
 *   idx   [B, H_kv, budget] int32 out (-1 after n_sel[b]);  n_sel [B] int32 out
 *   ws    workspace of magicdec_snapkv_workspace_size(shape, window) bytes
 * Errors: NULL pointers, bad shape, window <= 0, budget < window,
 * pool_kernel even or <= 0, alignment, workspace too small;
 * MAGICDEC_ERR_UNSUPPORTED when window * (H_q/H_kv) > 256 or pool_kernel > 9.
 */
MAGICDEC_API magicdec_status magicdec_snapkv_select(magicdec_kv_shape shape, const uint16_t *q_win, const uint16_t *k,
                                       const int32_t *seq_len, int window, int pool_kernel, int budget,
                                       int32_t *idx, int32_t *n_sel, void *ws, size_t ws_bytes, void *stream);

/*
 * SnapKV selection with a budget per sequence (heterogeneous batches; paper
 * section 4.3 discusses draft budgets per sequence length).  As
 * magicdec_snapkv_select, except that sequence b keeps budgets[b] positions
 * (device int32 [B], clamped to [window, max_budget]) and idx rows have
 * max_budget entries ([B, H_kv, max_budget], -1 after n_sel[b]); the gather
 * and the draft attention then take n_idx = cap = max_budget and
 * draft_len = n_sel.
 * Errors: as magicdec_snapkv_select, with max_budget in the role of budget.
 */
MAGICDEC_API magicdec_status magicdec_snapkv_select_budgets(magicdec_kv_shape shape, const uint16_t *q_win,
                                                            const uint16_t *k, const int32_t *seq_len, int window,
                                                            int pool_kernel, const int32_t *budgets, int max_budget,
                                                            int32_t *idx, int32_t *n_sel, void *ws, size_t ws_bytes,
                                                            void *stream);

/*
 * Gather of the selected rows into the compact draft cache (paper section
 * 4.4: the static selections copy their rows into a compact cache once).
 *   k, v   [B, L_cap, H_kv, d] bf16;  idx [B, H_kv, n_idx] int32
 *   kc, vc [B, H_kv, cap, d] bf16 out: row i < n_idx of head h is
 *          k[b, idx[b,h,i], h] (zero row when the index is outside [0, L_cap));
 *          rows n_idx..cap-1 are not touched (room for appended tokens).
 * Errors: NULL pointers, bad shape, n_idx < 0, n_idx > cap, alignment.
 */
MAGICDEC_API magicdec_status magicdec_gather_kv(magicdec_kv_shape shape, const uint16_t *k, const uint16_t *v,
                                   const int32_t *idx, int n_idx, int cap, uint16_t *kc, uint16_t *vc,
                                   void *stream);

/*
 * Draft-cache update: append, post-verification refresh and rollback of the
 * compact draft cache (paper section 4.4: the static drafts select once and
 * afterwards only take in new tokens; section 3.1: verification keeps the
 * accepted prefix, so rows the sparse draft wrote for rejected or
 * re-verified positions are replaced).  Layouts of kc, vc [B, H_kv, cap, d]:
 *   ring > 0 (StreamingLLM, sinks + recent window): position q < origin[b]
 *     at slot q; position q >= origin[b] at slot
 *     origin[b] + (q - origin[b]) mod ring.  The occupied slots hold exactly
 *     positions [0, min(len, origin)) and [max(origin, len - ring), len);
 *     from an empty cache, update(0, 0, L) builds the StreamingLLM selection
 *     for length L.  base is not read (may be NULL).
 *   ring == 0 (SnapKV): slots [0, base[b]) hold the rows kept at selection
 *     (magicdec_gather_kv); position q >= origin[b] (the length at selection)
 *     is appended at slot base[b] + q - origin[b].
 * Lengths (device int32 [B], clamped to [0, L_cap]; len_valid to at most
 * min(len_old, len_new)): rows of positions >= len_valid in the compact cache
 * are stale (drafted, or never written); len_old is the length the cache was
 * last brought to, len_new the new one.  The call copies from k, v
 * [B, L_cap, H_kv, d] every position of the new window at or past len_valid,
 * and (ring layout) restores every slot that a position in [len_new, len_old)
 * overwrote with the window position it displaced.  Typical use, per layer:
 * drafting appends position L+i as update(L+i, L+i, L+i+1); after
 * verification with n_acc accepted, update(L, L+gamma, L+n_acc+1).
 *   draft_len [B] int32 out: occupied slots (the draft attention's length),
 *   clamped to cap.
 * Errors: NULL pointers, bad shape, ring < 0, cap <= 0, base NULL when
 * ring == 0, ring > 0 with ring > cap, alignment.  A copy whose slot is at or
 * past cap is skipped and sets the device error word to 3.
 */
MAGICDEC_API magicdec_status magicdec_draft_cache_update(magicdec_kv_shape shape, const uint16_t *k, const uint16_t *v,
                                                         const int32_t *len_valid, const int32_t *len_old,
                                                         const int32_t *len_new, const int32_t *origin,
                                                         const int32_t *base, int ring, int cap, uint16_t *kc,
                                                         uint16_t *vc, int32_t *draft_len, void *stream);

/*
 * Lengths of one speculative step (paper section 3.1: gamma draft steps, one
 * verification of the gamma+1 block, then the sequence keeps its accepted
 * prefix and the emitted token; section 4.4: the static draft caches take in
 * each new position).  For every sequence b:
 *   len = len_in[b] + (n_acc ? n_acc[b] + 1 : 0), clamped to [0, L_cap];
 *   len_out[b] = len;  table[j * B + b] = min(len + j, L_cap), j = 0..gamma+1.
 * With len the number of cached positions at the start of a step, the step's
 * calls take: draft step g appends position len + g before attending,
 * magicdec_draft_cache_update(table[g], table[g], table[g+1]); verification
 * runs at seq_len = table[gamma+1] (the block's K/V at [len, len+gamma+1));
 * after acceptance a second call with n_acc gives the next length, and
 * magicdec_draft_cache_update(table[0], table[gamma], that length) refreshes
 * the verified rows and drops the rejected ones.
 *   len_in, n_acc (nullable: advance by 0), len_out [B] int32 device;
 *   table [(gamma+2) * B] int32 device.  len_out may alias len_in.
 * Errors: NULL pointers, B <= 0, gamma < 0 or > 1024, L_cap <= 0.
 */
MAGICDEC_API magicdec_status magicdec_step_lengths(int B, int gamma, int L_cap, const int32_t *len_in,
                                                   const int32_t *n_acc, int32_t *len_out, int32_t *table,
                                                   void *stream);

/* Workspace bytes magicdec_draft_attn / magicdec_verify_attn need for this
 * shape and query count (n_q = 1 for draft) on the current device. */
MAGICDEC_API size_t magicdec_attn_workspace_size(magicdec_kv_shape shape, int n_q);

/*
 * Draft attention (paper section 4.1, Eq. 3: decoding cost T_D(B,K) over the
 * K-row draft cache).  One query token per sequence attends to rows
 * 0..draft_len[b]-1 of its KV head in the compact cache (draft_len clamped to
 * [0, cap]; an empty cache gives a zero row).  Softmax scale 1/sqrt(d).
 *   shape.L_cap is the compact capacity `cap`.
 *   q  [B, 1, H_q, d] bf16;  kc, vc [B, H_kv, cap, d] bf16;  draft_len [B] int32
 *   out [B, 1, H_q, d] bf16
 * Errors: NULL pointers, bad shape, alignment, workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_draft_attn(magicdec_kv_shape shape, const uint16_t *q, const uint16_t *kc,
                                    const uint16_t *vc, const int32_t *draft_len, uint16_t *out, void *ws,
                                    size_t ws_bytes, void *stream);

/*
 * Verification attention (paper section 3.1, T_V(B,S,gamma); section 3.2:
 * verification loads the same KV as decoding).  The n_q = gamma+1 speculated
 * tokens already occupy cache positions [len-n_q, len), len = seq_len[b]
 * clamped to [0, L_cap]; query row i sees positions 0..len-n_q+i (causal
 * inside the speculated block; a row that sees nothing gives zeros).
 *   q [B, n_q, H_q, d] bf16;  k, v [B, L_cap, H_kv, d] bf16;  seq_len [B] int32
 *   out [B, n_q, H_q, d] bf16
 * Supported: (H_q/H_kv) * n_q <= 32 (MAGICDEC_ERR_UNSUPPORTED beyond).
 * Errors: NULL pointers, bad shape, alignment, workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_verify_attn(magicdec_kv_shape shape, int n_q, const uint16_t *q, const uint16_t *k,
                                     const uint16_t *v, const int32_t *seq_len, uint16_t *out, void *ws,
                                     size_t ws_bytes, void *stream);

/* Workspace bytes magicdec_topk_draft_attn needs: fp32 scores of every query
 * head over the whole cache, B * H_q * (L_cap rounded up to 4) * 4. */
MAGICDEC_API size_t magicdec_topk_attn_workspace_size(magicdec_kv_shape shape);

/*
 * Top-K attention draft (paper section 1 and Figure 1(c); section 4.4,
 * "Static vs Dynamic": the dynamic per-query selection whose acceptance rate
 * the static methods are compared against, and whose search over the whole
 * cache is its selection cost).  For query head h of sequence b, with
 * len = seq_len[b] clamped to [0, L_cap], the scores s_j = q . k_j / sqrt(d)
 * over j < len are ranked, the top_k largest are kept (equal scores: the
 * smaller position first; every position when len <= top_k), and
 *   out = sum_{j kept} softmax(s over the kept positions)_j v_j
 * (a zero row when len == 0).  Query head h reads KV head h / (H_q/H_kv).
 *   q [B, 1, H_q, d] bf16;  k, v [B, L_cap, H_kv, d] bf16;  seq_len [B] int32
 *   out [B, 1, H_q, d] bf16
 *   idx (nullable) [B, H_q, top_k] int32 out: the kept positions in ascending
 *       order, -1 after min(len, top_k)
 *   ws  workspace of magicdec_topk_attn_workspace_size(shape) bytes; no
 *       initial contents needed
 * Supported: H_q/H_kv <= 8 and top_k <= 8192 (MAGICDEC_ERR_UNSUPPORTED).
 * Errors: NULL pointers, bad shape, top_k <= 0, alignment (q, k, v, out, ws),
 * workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_topk_draft_attn(magicdec_kv_shape shape, const uint16_t *q, const uint16_t *k,
                                                      const uint16_t *v, const int32_t *seq_len, int top_k,
                                                      uint16_t *out, int32_t *idx, void *ws, size_t ws_bytes,
                                                      void *stream);

/*
 * PQCache-style dynamic selection (paper section 4.4 and Figure 5: a dynamic
 * KV selection that searches the cache per query through product-quantised
 * keys, with a search cost that grows with the batch).  Keys of each
 * (sequence, KV head) split into M = d/8 sub-vectors of 8 channels; subspace
 * m has C (1..256) centroids.
 *   codebook [B, H_kv, M, C, 8] fp32;  codes [B, H_kv, L_cap, M] uint8
 * A codebook is built at prefill by Lloyd iterations: encode, then update,
 * repeated, from initial centroids chosen by the caller.
 *
 * Encode: codes[b,h,j,m] = the centroid c of subspace m nearest to the key's
 * sub-vector (squared distance, evaluated as |c|^2 - 2 k.c in fp32; equal
 * values: the smaller c), for every position j < L_cap.
 * Errors: NULL pointers, bad shape, M != d/8, C outside [1, 256], alignment
 * (k, codebook); MAGICDEC_ERR_UNSUPPORTED when the codebook of one
 * (sequence, head) does not fit in shared memory.
 */
MAGICDEC_API magicdec_status magicdec_pq_encode(magicdec_kv_shape shape, const uint16_t *k, int M, int C,
                                                const float *codebook, uint8_t *codes, void *stream);

/*
 * Update (one Lloyd step after an encode): centroid c of subspace m becomes
 * the mean of the sub-vectors of positions j < seq_len[b] coded c (exact sum,
 * correctly rounded mean, rounded to fp32); a centroid without positions
 * keeps its value.  codebook is updated in place.
 * Errors as magicdec_pq_encode.
 */
MAGICDEC_API magicdec_status magicdec_pq_update(magicdec_kv_shape shape, const uint16_t *k, const int32_t *seq_len,
                                                int M, int C, const uint8_t *codes, float *codebook, void *stream);

/* Workspace bytes magicdec_pq_draft_attn needs: fp32 approximate scores,
 * B * H_q * (L_cap rounded up to 4) * 4. */
MAGICDEC_API size_t magicdec_pq_attn_workspace_size(magicdec_kv_shape shape);

/*
 * PQ draft attention.  For query head h of sequence b (KV head h/(H_q/H_kv)),
 * with len = seq_len[b] clamped to [0, L_cap]: LUT[m][c] = q_m . centroid(m,c)
 * / sqrt(d); approximate score a_j = sum_m LUT[m][codes[b,h,j,m]] for j < len;
 * the top_k positions by a_j are kept (equal: the smaller position; all when
 * len <= top_k) and
 *   out = sum_{j kept} softmax(q . k_j / sqrt(d) over the kept j) v_j
 * with the EXACT scores (a zero row when len == 0).
 *   q [B, 1, H_q, d] bf16;  k, v [B, L_cap, H_kv, d] bf16;  out [B, 1, H_q, d] bf16
 *   idx (nullable) [B, H_q, top_k] int32 out: kept positions, ascending, -1 padded
 *   ws  workspace of magicdec_pq_attn_workspace_size(shape) bytes
 * Supported: top_k <= 8192.  Errors: as magicdec_pq_encode, plus top_k <= 0,
 * alignment of q, v, out, ws, workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_pq_draft_attn(magicdec_kv_shape shape, const uint16_t *q, const uint16_t *k,
                                                    const uint16_t *v, const int32_t *seq_len, int M, int C,
                                                    const float *codebook, const uint8_t *codes, int top_k,
                                                    uint16_t *out, int32_t *idx, void *ws, size_t ws_bytes,
                                                    void *stream);

/*
 * Verification attention that allocates nothing (no counterpart in the paper;
 * an addition for callers that cannot allocate device memory, such as a
 * plug-in that receives only its input and output buffers from a host
 * runtime, an engine whose memory plan is fixed before it starts, or a
 * process whose device memory is owned by another allocator).  Same
 * arguments, layouts and results as magicdec_verify_attn, without `ws`: its
 * scratch is a 32 MiB array inside the library, which every GPU that loads
 * the library holds until the process exits.
 *  - The first call on a device, with that device current, looks up the
 *    array's device address (cudaGetSymbolAddress); make that first call
 *    before any stream capture.
 *  - Every call first clears the part of the array that must start at zero
 *    (the merge counters and scheduler words, 256 KB) with cudaMemsetAsync
 *    on `stream`, then launches on the same stream; so a call that gave up on
 *    a bounded wait (device error word 1) leaves nothing that a later call
 *    can trip over.
 *  - All calls on a device share the array, which keeps the last call's
 *    contents; calls that overlap on the GPU race, so order them (one
 *    stream).
 *  - Returns MAGICDEC_ERR_UNSUPPORTED, and enqueues nothing, when the
 *    kernel's scratch for the current device would not fit in the array.
 * Errors otherwise as magicdec_verify_attn.
 */
MAGICDEC_API magicdec_status magicdec_verify_attn_noalloc(magicdec_kv_shape shape, int n_q, const uint16_t *q,
                                                          const uint16_t *k, const uint16_t *v,
                                                          const int32_t *seq_len, uint16_t *out, void *stream);

/* Workspace bytes magicdec_spec_accept needs. */
MAGICDEC_API size_t magicdec_spec_accept_workspace_size(int B, int gamma, int V);

/*
 * Speculative-sampling accept / resample for one verification step
 * (Leviathan et al., as used for Eq. 1 in paper section 3.1), or greedy
 * verification (paper section 5.1).
 *   target [B, gamma+1, V] fp32 logits of the target at the gamma+1 positions
 *   draft  [B, gamma, V]   fp32 logits of the draft (may be NULL when greedy)
 *   draft_tok [B, gamma] int32; u_acc [B, gamma], u_res [B] uniforms in [0,1)
 * Sampling (greedy == 0), temperature 1, p = softmax(target_i),
 *   q = softmax(draft_i): draft token x is accepted iff u_acc < p(x)/q(x)
 *   (q(x) == 0 accepts iff p(x) > 0; x outside [0,V) is rejected).  At the
 *   first rejection the emitted token is the smallest t whose running sum of
 *   max(0, p - q) exceeds u_res times its total (of p if that total is 0).
 *   If all gamma drafts are accepted, a bonus token is drawn the same way from
 *   softmax(target_gamma).
 * Greedy (greedy != 0): accept while x equals argmax target_i (ties to the
 *   smaller token); emit that argmax at the first mismatch, else the argmax of
 *   target_gamma.
 * Outputs: n_acc [B] accepted count in [0, gamma]; out_tok [B, gamma+1]: the
 *   accepted tokens, then the emitted one, -1 after; n_ambiguous [B]
 *   (nullable): decisions taken near their boundary -- |u - p/q| < 1e-4, a
 *   top-2 logit gap below 1e-4, or u * total within 1e-7 of the total from a
 *   token edge of the inverse CDF.
 * Precision: per-logit exponentials in fp32; normalisers, p/q ratios and
 *   running sums in fp64 / double-float.
 * Errors: NULL pointers, B <= 0, gamma < 0, V <= 0, workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_spec_accept(int B, int gamma, int V, const float *target_logits,
                                     const float *draft_logits, const int32_t *draft_tok, const float *u_acc,
                                     const float *u_res, int greedy, int32_t *n_acc, int32_t *out_tok,
                                     int32_t *n_ambiguous, void *ws, size_t ws_bytes, void *stream);

/*
 * Paged KV cache, and the tree of drafted tokens over it.
 *
 * A cache is a pool of n_pages pages k_pages, v_pages [n_pages, page_size,
 * H_kv, d] bf16 and a table block_table [B, max_pages] int32: slot s of
 * sequence b is row s % page_size of page block_table[b, s / page_size].  Any
 * page_size >= 1.  A dense cache [B, L_cap, H_kv, d] is the pool with n_pages =
 * B, page_size = L_cap, max_pages = 1 and block_table[b, 0] = b.  The capacity of
 * a sequence is page_size * max_pages slots (at most INT_MAX - 255; B at most 4096,
 * H_q at most 65535; MAGICDEC_ERR_SHAPE beyond).  Only entries of the slots that a
 * call reads or writes are looked at; one outside [0, n_pages) sets the device error
 * word to 5, and nothing outside the pool is touched.
 *
 * A tree: len[b] positions of sequence b are committed.  Its node i (a drafted
 * token; node 0 is the last emitted one, whose K and V are not in the cache yet)
 * has slot len[b] + i.  parent[b, i] < i is the node before it; a negative entry
 * makes it a root, which follows the committed positions directly.  An entry >= i
 * counts as negative (and, in the range-checking build, sets error 4).  parent ==
 * NULL is the chain, parent i - 1.  n_nodes[b], clamped to [0, n], is the number
 * of nodes of sequence b (NULL: n for all).
 *
 * One step of tree speculation, per layer: magicdec_paged_append writes the
 * nodes' keys and values, magicdec_tree_attn attends; then, once,
 * magicdec_tree_accept walks down the tree and magicdec_tree_commit moves the
 * accepted rows to the slots [len, len + n_acc + 1), all layers in one call; and
 * magicdec_step_lengths gives the next len.
 */
typedef struct {
    int B;
    int H_q;
    int H_kv;
    int d;
    int page_size;
    int n_pages;
    int max_pages;
} magicdec_paged_shape;

/*
 * Append of n new tokens per sequence to a paged cache, with the rotary position
 * embedding applied on the way.  Token i of sequence b has slot len[b] + i and
 * position len[b] + i, or, with parent, len[b] + the number of nodes before node i
 * on its path.  K goes to its slot rotated, V unchanged; q, if given, is rotated
 * into q_out.  Rotation of channels [0, rot_dim) of every head: pair f, 0 <= f <
 * rot_dim / 2, turns by the angle position * inv_freq[f]; it is channels (f, f +
 * rot_dim / 2), or (2f, 2f + 1) if interleaved.  Other channels are copied.
 *   q, k, v  bf16; token i of sequence b starts at element (b * n + i) * stride,
 *            its heads dense ([H_q, d], [H_kv, d], [H_kv, d]); strides are multiples
 *            of 8 elements, so the three may be views of one projection's output
 *   q_out    [B, n, H_q, d] bf16; NULL together with q; may be q itself if that is
 *            dense (q_stride == H_q * d)
 *   n_new    (nullable) [B] int32: tokens i >= n_new[b], clamped to [0, n], are
 *            neither read nor written
 *   parent   (nullable) [B, n] int32, n <= 256
 *   inv_freq [rot_dim / 2] fp32 (NULL if rot_dim == 0)
 * A token whose slot is at or past the capacity is not stored (device error 3),
 * nor one whose page is outside the pool (error 5); its query is rotated all the same.
 * No two sequences may share a page that the call writes.
 * Errors: NULL pointers, bad shape, n <= 0, rot_dim < 0, odd or > d, a stride below
 * the row, alignment (pointers to 16 bytes, strides to 8 elements);
 * MAGICDEC_ERR_UNSUPPORTED when rot_dim is not a multiple of 16, or parent is given
 * and n > 256.
 */
MAGICDEC_API magicdec_status magicdec_paged_append(magicdec_paged_shape shape, int n, const uint16_t *q,
                                                   long long q_stride, const uint16_t *k, long long k_stride,
                                                   const uint16_t *v, long long v_stride, const int32_t *len,
                                                   const int32_t *n_new, const int32_t *parent, const float *inv_freq,
                                                   int rot_dim, int interleaved, const int32_t *block_table,
                                                   uint16_t *q_out, uint16_t *k_pages, uint16_t *v_pages,
                                                   void *stream);

/*
 * Append as magicdec_paged_append, for models that norm every query and key head before
 * the rotation, and for tokens whose positions have several axes (time, height and width
 * of images and video).  A query head x becomes x / sqrt(mean(x^2) + eps) * q_weight over
 * its d channels, a key head likewise with k_weight, then is rotated; norm and rotation
 * in fp32, with one rounding to bf16 at the end.
 *   q_weight, k_weight (nullable, each) [d] bf16: NULL leaves the query (key) heads as
 *            they are
 *   eps      finite and at least 2^-126, if there is a weight (squares below lose their last bits)
 *   pos      (nullable) [B, n, n_axes] int32: token i of sequence b has these positions
 *            instead of those counted from len; not with parent.  Slots go by len as before
 *   axis     (nullable if n_axes == 1) [rot_dim / 2] int32: pair f turns by the angle
 *            pos[b, i, axis[f]] * inv_freq[f]; an entry outside [0, n_axes) counts as 0 (and,
 *            in the range-checking build, sets error 4)
 * Everything else as there, the errors too; further ones: MAGICDEC_ERR_NULL for n_axes > 1
 * without axis, MAGICDEC_ERR_SHAPE for eps below 2^-126 or not finite beside a weight, pos
 * together with parent, n_axes <= 0 with pos, or axis without pos, MAGICDEC_ERR_ALIGN for
 * weights off a 16-byte boundary, MAGICDEC_ERR_UNSUPPORTED for n_axes > 64.
 */
MAGICDEC_API magicdec_status magicdec_norm_append(magicdec_paged_shape shape, int n, const uint16_t *q,
                                                  long long q_stride, const uint16_t *k, long long k_stride,
                                                  const uint16_t *v, long long v_stride, const uint16_t *q_weight,
                                                  const uint16_t *k_weight, float eps, const int32_t *len,
                                                  const int32_t *n_new, const int32_t *parent, const int32_t *pos,
                                                  int n_axes, const int32_t *axis, const float *inv_freq, int rot_dim,
                                                  int interleaved, const int32_t *block_table, uint16_t *q_out,
                                                  uint16_t *k_pages, uint16_t *v_pages, void *stream);

/* Workspace bytes magicdec_tree_attn needs for this shape and node count on the
 * current device (0 for a shape that it refuses). */
MAGICDEC_API size_t magicdec_tree_attn_workspace_size(magicdec_paged_shape shape, int n);

/*
 * Attention of the tree's nodes over a paged cache.  Node i of sequence b attends
 * to positions [0, len[b]) and to the slots of its ancestors and itself; softmax
 * scale 1/sqrt(d); query head hq reads KV head hq / (H_q/H_kv).  With n = 1 it is
 * the attention of a single new token, with parent NULL that of a causal block.
 *   q   [B, n, H_q, d] bf16;  out [B, n, H_q, d] bf16: rows of nodes i >=
 *       n_nodes[b] are zero, as is a row that sees nothing
 *   len [B] int32, clamped to [0, capacity]; slots at or past the capacity hold
 *       nothing (no node sees them)
 *   ws  workspace of magicdec_tree_attn_workspace_size(shape, n) bytes; no initial
 *       contents needed
 * Pool rows outside [0, len + n_nodes) may hold anything, NaN included; a node's
 * own rows reach it and its descendants only, whatever they hold.  A page outside
 * the pool counts as keys and values of zero (device error 5).
 * Supported: n <= 256, H_q/H_kv <= 128, below 4 rows a page fewer than INT_MAX rows
 * in the pool, and a capacity whose tiles of 128 keys, counted for every KV head and
 * every 128 H_kv / H_q nodes, fit 32 bits (MAGICDEC_ERR_UNSUPPORTED beyond).
 * Errors: NULL pointers, bad shape, n <= 0, alignment, workspace too small.
 */
MAGICDEC_API magicdec_status magicdec_tree_attn(magicdec_paged_shape shape, int n, const uint16_t *q,
                                                const uint16_t *k_pages, const uint16_t *v_pages,
                                                const int32_t *block_table, const int32_t *len,
                                                const int32_t *n_nodes, const int32_t *parent, uint16_t *out, void *ws,
                                                size_t ws_bytes, void *stream);

/* Workspace bytes magicdec_prefix_attn needs for this shape, number of prefixes and node
 * count on the current device (0 for a shape that it refuses). */
MAGICDEC_API size_t magicdec_prefix_attn_workspace_size(magicdec_paged_shape shape, int n_prefixes, int n);

/*
 * Attention as magicdec_tree_attn for a batch whose sequences share long prefixes (samples of
 * one prompt, a system prompt of all): a prefix's keys and values are read once for all
 * sequences behind it.  The sequences [first[g], first[g+1]) follow prefix g, which is the
 * prefix_len[g] positions of the pages prefix_table[g]; each one's own slots, counted from 0, are
 * those of block_table, and len, n_nodes and parent are as in magicdec_tree_attn.  Node i of
 * sequence b attends to its prefix, to its own positions [0, len[b]), and to the slots of its
 * ancestors and itself.  Keys are taken as they are: rotate them (magicdec_norm_append with pos,
 * magicdec_paged_append) by the position that counts the prefix in.
 *   prefix_table [n_prefixes, max_prefix_pages] int32, of the same pool;  prefix_len [n_prefixes]
 *            int32, clamped to [0, page_size * max_prefix_pages]
 *   first    [n_prefixes + 1] int32, ascending, clamped to [0, B]; sequences outside all groups
 *            have no prefix; NULL with n_prefixes == 1: all sequences follow the one prefix.  Of
 *            entries that do not ascend the rows come out unspecified
 *   q   [B, n, H_q, d] bf16;  out [B, n, H_q, d] bf16: rows of nodes i >= n_nodes[b] are zero, as
 *       is a row that sees nothing
 *   ws  workspace of magicdec_prefix_attn_workspace_size(shape, n_prefixes, n) bytes; no initial
 *       contents needed
 * Pool rows that no node sees may hold anything, and a node's own rows reach it and its descendants only;
 * a page outside the pool counts as keys and values of zero (device error 5).
 * Supported, errors: as magicdec_tree_attn, the prefixes' capacity and their tiles with those of all
 * B n nodes included; n_prefixes at most 4096, one unless first is given; MAGICDEC_ERR_SHAPE for
 * n_prefixes <= 0 or max_prefix_pages <= 0.
 */
MAGICDEC_API magicdec_status magicdec_prefix_attn(magicdec_paged_shape shape, int n_prefixes, int max_prefix_pages, int n,
                                                  const uint16_t *q, const uint16_t *k_pages, const uint16_t *v_pages,
                                                  const int32_t *prefix_table, const int32_t *prefix_len,
                                                  const int32_t *first, const int32_t *block_table,
                                                  const int32_t *len, const int32_t *n_nodes, const int32_t *parent,
                                                  uint16_t *out, void *ws, size_t ws_bytes, void *stream);

/*
 * Greedy acceptance down the tree.  From node u = 0: t = argmax target[b, u], ties
 * to the smaller token; the walk goes on to the lowest node whose parent is u and
 * whose token is t, and ends where there is none.
 *   target [B, n, V] fp32 logits of the target at every node; infinities are values
 *          like others, NaN counts as -inf, and of a row of nothing else token 0 is
 *          the argmax
 *   tok    [B, n] int32: the nodes' tokens (tok[b, 0] is not looked at)
 * Outputs: n_acc [B]: nodes accepted after node 0, -1 for a sequence without nodes
 *   (so that len + n_acc + 1 is its next length in every case); path [B, n]: node 0
 *   and the accepted nodes, then -1; out_tok [B, n]: the n_acc accepted tokens, then
 *   the emitted one (the argmax at the last node of the path), then -1.
 * Errors: NULL pointers, B <= 0, n <= 0, V <= 0, alignment (target);
 * MAGICDEC_ERR_UNSUPPORTED when n > 256 or B > 65536.
 */
MAGICDEC_API magicdec_status magicdec_tree_accept(int B, int n, int V, const float *target_logits, const int32_t *tok,
                                                  const int32_t *parent, const int32_t *n_nodes, int32_t *n_acc,
                                                  int32_t *path, int32_t *out_tok, void *stream);

/*
 * Commit of an accepted path: in every layer, slot len[b] + i takes the row of slot
 * len[b] + path[b, i], for i = 0 .. n_acc[b] (clamped to [-1, n - 1]).  path ascends
 * with path[b, i] >= i, as magicdec_tree_accept gives it; an entry outside [0, n) is
 * skipped, and other orders give unspecified rows of the same slots.
 *   k_pages, v_pages [layers, n_pages, page_size, H_kv, d] bf16, one block_table for
 *   all layers
 * A move from or to a slot at or past the capacity is skipped (device error 3), as is
 * one through a page outside the pool (error 5).
 * Errors: NULL pointers, bad shape, n <= 0, layers <= 0, alignment;
 * MAGICDEC_ERR_UNSUPPORTED when n > 256 or layers > 65535.
 */
MAGICDEC_API magicdec_status magicdec_tree_commit(magicdec_paged_shape shape, int n, int layers, const int32_t *len,
                                                  const int32_t *path, const int32_t *n_acc,
                                                  const int32_t *block_table, uint16_t *k_pages, uint16_t *v_pages,
                                                  void *stream);

/*
 * A draft cache that keeps its heavy hitters (no counterpart in the paper, which drafts over
 * static selections: the rows kept here follow what the attention finds heavy while it
 * drafts).  Rows of K and V lie in kc, vc [B, H_kv, cap, d] as in the compact draft cache,
 * draft_len[b] of them in use, in any order; beside each row its accumulated attention
 * weight, weight [B, H_kv, cap] fp32, and the position of its token, pos [B, H_kv, cap]
 * int32.  A step appends a token's rows behind the others (magicdec_draft_cache_update),
 * attends with magicdec_heavy_attn, and, when the rows have outgrown the budget, drops those
 * of least weight with magicdec_heavy_evict.
 *
 * A speculative step, from L positions and r rows (table as magicdec_step_lengths gives it):
 *   for each of the gamma drafted tokens magicdec_draft_cache_update(table[g], table[g],
 *   table[g+1]) with ring = 0, origin = L and base = r, then magicdec_heavy_attn with
 *   next_pos = table[g]; after verification magicdec_draft_cache_update(table[0],
 *   table[gamma], L + n_acc + 1), which puts the verified rows in place of the drafted ones and
 *   leaves out the rejected; then magicdec_heavy_evict with that length as seq_len.
 * weight and pos are set by magicdec_heavy_attn alone, so what it has not attended with is the
 * caller's to set: the rows that a cache begins with (magicdec_gather_kv), and row r + gamma,
 * position L + gamma, which the refresh brings in where all gamma tokens were accepted (weight 0
 * and that position, at any time between the step's last attention and its eviction; in other
 * sequences the row is not in use, and both may be set there as well).
 * Attention of tokens that are rejected afterwards stays in the weights of the rows that they saw.
 * The update and the gather read dense K and V; rows of a paged cache are the caller's to bring in.
 */

/*
 * Attention of n_q query tokens over the draft cache, whose last n_q rows are the tokens'
 * own; every row's weight grows by the attention that it got.  Token i sees rows
 * 0 .. len - n_q + i, len = draft_len[b] clamped to [0, cap]; softmax scale 1/sqrt(d); query
 * head hq reads KV head hq / (H_q/H_kv).  weight[b, h, j] += the probabilities of row j
 * summed over the tokens and the H_q/H_kv query heads of KV head h.
 *   q [B, n_q, H_q, d] bf16;  kc, vc [B, H_kv, cap, d] bf16;  shape.L_cap is cap
 *   out [B, n_q, H_q, d] bf16: zero rows for tokens that see nothing
 *   next_pos (nullable) [B] int32: the last n_q rows are new: what weight and pos hold there
 *            is replaced, pos by next_pos[b] + i, the weight by this call's alone.  NULL: pos is not
 *            looked at (and may be NULL), and all weights are added to
 * Rows at or past len may hold anything, NaN included, and are left as they are; a token's own
 * row reaches it and later tokens only, whatever it holds; a query row that meets a score of NaN or
 * plus infinity comes out as NaN, and so do the weights of the rows it sees.  Probabilities are summed
 * in fp32, in an order that is the same from run to run.
 * Supported: (H_q/H_kv) * n_q <= 32 and H_kv <= 65535 (MAGICDEC_ERR_UNSUPPORTED beyond).
 * Errors: NULL pointers, bad shape, n_q <= 0, alignment (q, kc, vc, out).
 */
MAGICDEC_API magicdec_status magicdec_heavy_attn(magicdec_kv_shape shape, int n_q, const uint16_t *q,
                                                 const uint16_t *kc, const uint16_t *vc, const int32_t *draft_len,
                                                 const int32_t *next_pos, float *weight, int32_t *pos, uint16_t *out,
                                                 void *stream);

/*
 * Eviction, all layers in one call: of every (layer, sequence, KV head) with more than
 * `budget` rows, `budget` stay: those whose position is below n_sink or at least
 * seq_len[b] - n_recent, and of the others the ones of largest weight (equal weights: the
 * smaller position, then the smaller row; protected rows count as of infinite weight).
 * Rows that stay and lie at or past the budget move, in ascending order, into the places below
 * it of rows that went, with their weight and position; all others stay where they are.
 *   kc, vc [layers, B, H_kv, cap, d] bf16, weight, pos [layers, B, H_kv, cap]; shape.L_cap is
 *   cap, shape.H_q is not looked at beyond being a multiple of H_kv
 *   draft_len [B] int32, for all layers;  seq_len [B] int32: positions of the sequence so far
 *   draft_len_out [B] int32 out: min(draft_len clamped to [0, cap], budget); not draft_len itself
 * What rows at or past the new length hold is left as it was.  No weight may be NaN.
 * Errors: NULL pointers, bad shape, layers <= 0, budget <= 0, n_sink or n_recent < 0, or their
 * sum above the budget, draft_len_out == draft_len, alignment (kc, vc);
 * MAGICDEC_ERR_UNSUPPORTED when layers > 65535 or cap > 1048576.
 */
MAGICDEC_API magicdec_status magicdec_heavy_evict(magicdec_kv_shape shape, int layers, const int32_t *draft_len,
                                                  const int32_t *seq_len, int budget, int n_sink, int n_recent,
                                                  uint16_t *kc, uint16_t *vc, float *weight, int32_t *pos,
                                                  int32_t *draft_len_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAGICDEC_H */
