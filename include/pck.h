/*
 * pck.h -- C ABI of libpck: attention of query rows over a resident shared-prefix KV cache
 * on one GB300 (sm_103a).
 *
 * The calls follow the problem statement of the ATTEND.PREFIX.* wire forms on the page
 * "ATTEND.* and ATTEND.PREFIX.*", section "Wire forms" (STORE / LOOKUP / QUERY /
 * QUERY_FUSED / QUERY_SPARSE_AUTO / QUERY_SPARSE_AUTO_FUSED), with explicit M, dtypes and
 * pointer ownership. The mlx4g32 tier follows "Shared KV Cache Serving -- Pion as LLM
 * Memory", section "Quantized tier -- mlx4g32".
 *
 * Conventions for every call:
 *  - Tensor pointers (Q, O, LSE, K, V, K_suf, V_suf, records, idx_out) are DEVICE pointers
 *    on the context's device, caller-owned, contiguous, and must stay valid until the stream
 *    reaches the call. O, K, V and Q must be 16-byte aligned, and K_suf / V_suf too when M > 1
 *    (PCK_EINVAL otherwise). head_map is a small HOST array (int32[H_q], entries in [0, H_kv));
 *    NULL means the grouped default h / (H_q / H_kv).
 *  - `stream` is a cudaStream_t passed as void*; NULL is the legacy default stream.
 *  - Calls are asynchronous on `stream`. Argument, shape and slot errors are detected on the
 *    host and returned before anything is launched. Asynchronous CUDA errors are reported as
 *    PCK_ECUDA by pck_sync or by a later call.
 *  - One context serialises its work: queries on one context must be issued on one stream
 *    (they share the context's split-K workspace). Use one context per stream otherwise.
 *  - Scores are tau * q.k with tau = 1/sqrt(D). LSE is in natural-log units of the scaled
 *    logits: LSE = ln(sum_t exp(tau q.k_t)). O is fp32 [H_q, M, D], LSE fp32 [H_q, M].
 *  - On a non-OK status, pck_last_error(ctx) holds a one-line reason.
 */
#ifndef PCK_H
#define PCK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. PCK_MISS matches the wire's +MISS / "-ERR session not found"; PCK_COLDMISS
 * matches STATUS_COLDMISS = 0x03 of the binary lane ("Shared KV Cache Serving", section
 * "Cold-tier state machine"): the slot was evicted by LRU and must be stored again. */
#define PCK_OK            0
#define PCK_MISS          1
#define PCK_COLDMISS      3
#define PCK_EINVAL       (-1)
#define PCK_EUNSUPPORTED (-2)
#define PCK_ENOMEM       (-3)
#define PCK_ECUDA        (-4)

/* Resident formats of a slot. */
#define PCK_FMT_FP16     0  /* fp16 K/V */
#define PCK_FMT_MLX4G32  1  /* int4, group 32, affine, fp16 scale + fp16 bias per group */

/* Element types of caller tensors. */
#define PCK_DT_F32       0
#define PCK_DT_F16       1
#define PCK_DT_BF16      2  /* the paged-tail calls only */

/* Head dimensions with kernels: fp16 slots 32, 64, 96, 128, 160, 192, 256 (M = 1 and M > 1) and
 * 512 (M = 1 only: M > 1 returns PCK_EUNSUPPORTED); mlx4g32 slots 64, 128, 192, 256 (M > 1: 64,
 * 128); QUERY_SPARSE_AUTO(_FUSED) 64, 128, 256; QUERY_SPARSE every fp16 slot. More than 8 q heads
 * per kv head (4 at D = 512) are split into work groups, each of which reads the kv head. */
#define PCK_MAX_BATCH    64   /* descriptors per pck_query_batch call */
#define PCK_MAX_HEADS    64   /* H_q and H_kv limit */

typedef struct pck_ctx pck_ctx;

typedef struct pck_info_t {
    int64_t slots_used;       /* resident (sid, layer) slots */
    int64_t slots_max;        /* capacity (LRU eviction beyond it) */
    int64_t cold_entries;     /* evicted keys remembered for PCK_COLDMISS */
    int64_t bytes_resident;   /* device bytes held by resident K/V (+ block means) */
    int64_t queries_served;   /* query calls that launched work */
    int64_t stores;           /* store calls that launched work */
    int64_t evictions;        /* LRU demotions */
} pck_info_t;

/* One M=1 query of a pck_query_batch call. */
typedef struct pck_query_desc {
    const char *sid;          /* session id (NUL-terminated) */
    int layer;
    const void *Q;            /* device [H_q, D], q_dtype of the batch */
    float *O;                 /* device [H_q, D] fp32 */
    float *LSE;               /* device [H_q] fp32, or NULL */
    const void *K_suf;        /* device fp16 [H_kv, S_suf, D], or NULL when S_suf == 0 */
    const void *V_suf;
} pck_query_desc;

/* One M=1 query of a pck_query_sparse_batch call. */
typedef struct pck_sparse_desc {
    const char *sid;          /* session id (NUL-terminated) */
    int layer;
    const void *Q;            /* device [H_q, D], q_dtype of the batch */
    float *O;                 /* device [H_q, D] fp32 */
    float *LSE;               /* device [H_q] fp32, or NULL */
    const void *K_suf;        /* device fp16 [H_kv, S_suf, D], or NULL when S_suf == 0 */
    const void *V_suf;
    int32_t *idx_out;         /* device [H_q, min(K_top, nb)] selected blocks (ascending), or NULL */
} pck_sparse_desc;

/* Create a context on CUDA device `device` with room for `max_slots` resident (sid, layer)
 * slots (<= 0 selects 256, the per-worker slot table size of the pages' session cache).
 * Allocates the split-K workspace. Returns PCK_OK and *out, or PCK_ECUDA / PCK_ENOMEM. */
int pck_create(pck_ctx **out, int device, int max_slots);

/* Free every resident slot and the workspace. Synchronises the device first. NULL is a no-op. */
void pck_destroy(pck_ctx *ctx);

/* One-line description of the last error on ctx ("" if none). Owned by ctx. */
const char *pck_last_error(const pck_ctx *ctx);

/* ATTEND.PREFIX.STORE <sid> <layer> <H> <N> <D> <K_blob> <V_blob>.
 * K, V: device [H_kv, N, D], src_dtype F16 or F32. fmt FP16 keeps fp16 K/V resident;
 * fmt MLX4G32 quantises both on the device (same arithmetic as pck_quantize_mlx4g32) and keeps
 * the codes/scales/biases resident. Replaces an existing slot with the same key. The library
 * copies K/V into its own memory: the caller may reuse K/V once the stream passes the call.
 * D: see above; H_kv <= 64, N >= 1. Errors: EINVAL, EUNSUPPORTED, ENOMEM. */
int pck_store(pck_ctx *ctx, const char *sid, int layer, int H_kv, int N, int D, int fmt,
              const void *K, const void *V, int src_dtype, void *stream);

/* Store pre-quantised mlx4g32 records (token-major [N, rec] with rec = H_kv*D/8*4 + 2*(H_kv*D/32)*2
 * bytes: codes words, then scales, then biases; see pck_quantize_mlx4g32) as a MLX4G32 slot. */
int pck_store_records(pck_ctx *ctx, const char *sid, int layer, int H_kv, int N, int D,
                      const void *K_rec, const void *V_rec, void *stream);

/* ATTEND.PREFIX.LOOKUP: PCK_OK if (sid, layer) is resident, PCK_COLDMISS if it was evicted,
 * PCK_MISS otherwise. */
int pck_lookup(pck_ctx *ctx, const char *sid, int layer);

/* Drop (sid, layer), or every layer of sid when layer < 0. Memory is released in stream order
 * on `stream` (queued work on that stream still sees valid K/V). Returns the number dropped. */
int pck_drop(pck_ctx *ctx, const char *sid, int layer, void *stream);

/* Precompute the block means of K (fp32, [H_kv, ceil(N/B), D]) used by the sparse selector, and
 * (at D in {64, 128, 256} with at most 1024 blocks) their fp16 hi + lo copy for the one-kernel form.
 * The sparse queries build them on first use per (slot, B); this lets a caller do it at store
 * time (e.g. before capturing a CUDA graph). Only fp16 slots. The means of all slots share
 * device memory the context sets aside in large chunks (packed together, the batched sparse
 * form reads them faster); a build that would allocate while `stream` is being captured
 * returns PCK_EINVAL, so a captured sparse call needs its slots' means built beforehand. */
int pck_build_block_means(pck_ctx *ctx, const char *sid, int layer, int B, void *stream);

/* ATTEND.PREFIX.QUERY <sid> <layer> <H> <D> <top_k> <Q_blob> [<fa_window>].
 * Q: device [H_q, M, D] of q_dtype. M == 1: split-K decode over the slot (fp16 or mlx4g32).
 * M > 1: tiled tensor-core kernel; needs q_dtype F16 (PCK_EUNSUPPORTED otherwise). Over an
 * mlx4g32 slot (D in {64, 128}) the call first dequantises the slot into a stream-ordered
 * temporary of H_kv * N * 8 * D bytes, each value as an fp16 hi + lo pair, and attends to it
 * with the same kernel at width 2D, so K and V keep ~22 bits.
 * top_k: 0 or >= N (dense); smaller values are PCK_EUNSUPPORTED.
 * fa_window (listed on every QUERY form of the pages, never defined there; this library's reading):
 * 0 = no window; W > 0 = a sliding attention window: query row i, at absolute position
 * p_i = N + S_suf - M + i (prefix positions 0 .. N-1, then the suffix), sees only positions
 * p_i - W + 1 .. p_i (and, with causal, no suffix key past its own). Built for every dense QUERY
 * form (M = 1 and M > 1, both formats, with or without a suffix); the sparse forms take W = 0
 * only (PCK_EUNSUPPORTED otherwise); W < 0 is PCK_EINVAL.
 * Writes O [H_q, M, D] and, if LSE != NULL, LSE [H_q, M]. */
int pck_query(pck_ctx *ctx, const char *sid, int layer, int H_q, int D, int M, int q_dtype,
              const void *Q, const int32_t *head_map, int top_k, int fa_window,
              float *O, float *LSE, void *stream);

/* ATTEND.PREFIX.QUERY_FUSED: prefix attention plus attention to a dense suffix
 * K_suf/V_suf (device fp16 [H_kv, S_suf, D]), merged by online softmax in the same launch.
 * causal != 0: query row i (of M) sees suffix keys j <= S_suf - M + i (bottom-right aligned);
 * causal == 0: every row sees the whole suffix. The merged LSE is written if LSE != NULL. */
int pck_query_fused(pck_ctx *ctx, const char *sid, int layer, int H_q, int D, int M, int S_suf,
                    int H_kv, int q_dtype, const void *Q, const void *K_suf, const void *V_suf,
                    const int32_t *head_map, int causal, int fa_window,
                    float *O, float *LSE, void *stream);

/* ATTEND.PREFIX.QUERY_SPARSE_AUTO: M=1. Scores the slot's B-token blocks by
 * tau * q_h . mean(K of the block), keeps the K_top best per q head (ties -> lower index,
 * K_top clamped to ceil(N/B)), and attends only to their tokens. idx_out (device
 * int32 [H_q, min(K_top, nblocks)], nullable) receives the selected blocks, sorted ascending.
 * fp16 slots only. */
int pck_query_sparse_auto(pck_ctx *ctx, const char *sid, int layer, int H_q, int D, int B,
                          int K_top, int H_kv, int q_dtype, const void *Q,
                          const int32_t *head_map, int fa_window,
                          float *O, float *LSE, int32_t *idx_out, void *stream);

/* ATTEND.PREFIX.QUERY_SPARSE_AUTO_FUSED: the sparse prefix plus a dense suffix (device fp16
 * [H_kv, S_suf, D]) merged by online softmax. */
int pck_query_sparse_auto_fused(pck_ctx *ctx, const char *sid, int layer, int H_q, int D, int B,
                                int K_top, int H_kv, int S_suf, int q_dtype, const void *Q,
                                const void *K_suf, const void *V_suf, const int32_t *head_map,
                                int fa_window, float *O, float *LSE, int32_t *idx_out,
                                void *stream);

/* ATTEND.PREFIX.QUERY_SPARSE <sid> <layer> <H> <D> <K_sparse_max> <Q> <indices> <counts>
 * ("ATTEND.* and ATTEND.PREFIX.*", command table: M=1 attention restricted to caller-supplied
 * per-head token indices, e.g. from a learned router). Q: device [H_q, D] of q_dtype; O: device
 * fp32 [H_q, D]; LSE: device fp32 [H_q] or NULL. indices: HOST int32 [H_q, K_sparse_max], row h
 * holding counts[h] prefix token positions (HOST int32 [H_q]) that q head h attends to, of kv
 * head head_map[h] (NULL head_map: h / (H_q / H_kv)). Checked on the host before anything is
 * launched: 1 <= counts[h] <= K_sparse_max, positions in [0, N) and strictly ascending (no
 * duplicates), else PCK_EINVAL. fp16 slots, H_q <= 64, fa_window 0. The index lists are copied
 * to the device with a pageable host-to-device copy (the host arrays may be reused once the call
 * returns; the call cannot be captured in a CUDA graph); the selected tokens are gathered into a
 * stream-ordered temporary and attended by the split-K decode. */
int pck_query_sparse(pck_ctx *ctx, const char *sid, int layer, int H_q, int D, int K_sparse_max, int q_dtype,
                     const void *Q, const int32_t *indices, const int32_t *counts, const int32_t *head_map,
                     int fa_window, float *O, float *LSE, void *stream);

/* Copy the slot's block means (fp32 [H_kv, ceil(N/B), D], built first when absent; see
 * pck_build_block_means) into the device buffer `out`. */
int pck_get_block_means(pck_ctx *ctx, const char *sid, int layer, int B, float *out, void *stream);

/* n independent M=1 queries of one shape (H_q, H_kv, D, S_suf, q_dtype, head_map) in ONE
 * launch: the whole batch is split evenly over the GPU. 1 <= n <= PCK_MAX_BATCH. All slots
 * must have the same format. */
int pck_query_batch(pck_ctx *ctx, int n, const pck_query_desc *descs, int H_q, int H_kv, int D,
                    int S_suf, int q_dtype, const int32_t *head_map, void *stream);

/* pck_query_batch over HOST buffers: descs[i].Q, K_suf, V_suf (inputs) and O, LSE (outputs) are
 * page-locked host pointers (cudaHostAlloc, cudaHostRegister or a pinned tensor), 16-byte
 * aligned; everything else is as pck_query_batch. The call moves the bytes itself, on `stream`:
 * a copy kernel reads the inputs over the host link into the context's staging memory (at most
 * PCK_HOST_STAGE_BYTES per call), the batch runs on the staged copies, and its merge kernel
 * writes O and LSE straight into the host buffers. The outputs are valid, and the inputs may be
 * reused, once `stream` has been synchronised. Errors: as pck_query_batch; PCK_EINVAL for a
 * pointer that is not page-locked host memory; PCK_EUNSUPPORTED above the staging size. */
#define PCK_HOST_STAGE_BYTES (16u << 20)
int pck_query_batch_host(pck_ctx *ctx, int n, const pck_query_desc *descs, int H_q, int H_kv, int D,
                         int S_suf, int q_dtype, const int32_t *head_map, void *stream);

/* n independent ATTEND.PREFIX.QUERY_SPARSE_AUTO(_FUSED) queries (page "ATTEND.* and
 * ATTEND.PREFIX.*", section "Wire forms"; batching them is this library's addition, as for
 * pck_query_batch) of one shape (H_q, H_kv, D, B, K_top, S_suf, q_dtype, head_map) over fp16
 * slots of the same N. A batch of at least 32 work items (query x group of up to 8 q heads of a
 * kv head, 4 at D = 256) over at most 1024 blocks per kv head, with 16-byte aligned suffixes,
 * runs as ONE kernel with a CTA per work item (scores, top-K, union, gather decode of the union
 * and the suffix, merge); otherwise the block scores of all queries run in one scoring launch,
 * their top-K selections in one selection launch, and their gathers (+ suffixes) in one split-K
 * decode and its merge (four launches). Each query is as pck_query_sparse_auto_fused
 * (S_suf > 0) or pck_query_sparse_auto (S_suf == 0) would compute it alone. The first sparse
 * call on a slot builds its block means (and their fp16 hi + lo copy, which the one-kernel form
 * scores from) with stream-ordered allocations: call pck_build_block_means, or make a first
 * call, before capturing the call in a CUDA graph.
 * 1 <= n <= PCK_MAX_BATCH. Errors: EINVAL, EUNSUPPORTED (slots of different N, B not a multiple
 * of 16, K_top > 64, fa_window), MISS / COLDMISS for an absent slot. */
int pck_query_sparse_batch(pck_ctx *ctx, int n, const pck_sparse_desc *descs, int H_q, int H_kv, int D,
                           int B, int K_top, int S_suf, int q_dtype, const int32_t *head_map,
                           void *stream);

/* mlx4g32 quantiser (store side). X: device [rows, kv_dim] of src_dtype (F16 or F32);
 * out_records: device [rows, rec] bytes, rec = kv_dim/2 + kv_dim/8. Per group of 32:
 * mn/mx as fp32, s32 = (mx - mn)/15 in fp32, scale = fp16(s32) (rounded BEFORE the codes are
 * chosen), bias = fp16(mn), code = clamp(rint((x - bias)/scale), 0, 15) in fp32, all codes 0 when
 * scale == 0; code j fills bits 4*(j%8) .. 4*(j%8)+3 of word j/8. kv_dim % 32 == 0. Inputs must be
 * finite and within the fp16 range. Needs no context. */
int pck_quantize_mlx4g32(const void *X, int src_dtype, int64_t rows, int kv_dim,
                         void *out_records, void *stream);

/* The KV.PREFIX.WARM / V.FETCH RANGE form of stored mlx4g32 records ("Shared KV Cache Serving
 * -- Pion as LLM Memory", sections "KV.PREFIX.WARM" and "Cold-tier state machine"; "V.* -- the
 * V-store", V.FETCH): records (device, token-major [N, rec] as in pck_store_records, 4-byte
 * aligned) -> out (device, [H_kv, N, D], 16-byte aligned), the dequantised x = scale * code +
 * bias rounded once to fp32 (out_dtype F32), or that fp32 value rounded to fp16 (F16): the
 * dequantise and the [N, H*D] -> [H, N, D] transpose in one pass. H_kv * D % 32 == 0,
 * D % 8 == 0. Needs no context. Errors: EINVAL, ECUDA. */
int pck_dequantize_mlx4g32(const void *records, int64_t N, int H_kv, int D, int out_dtype, void *out,
                           void *stream);

/* Attention of M=1 queries over mlx4g32 records the caller holds, allocating nothing.
 * The pages have no counterpart: it exists for callers that cannot allocate device memory at
 * call time (code running under another framework's allocator budget, a request path that must
 * not touch the allocator, or a process without a pck context). It runs the same kernels as
 * pck_store_records + pck_query_fused (M=1), with the same split of the work, but all scratch
 * lives in device arrays compiled into libpck (PCK_NOALLOC_SCRATCH_BYTES per GPU, held from
 * library load until process exit).
 * K_rec, V_rec: device token-major records [N, rec] as in pck_store_records. Q: device [H_q, D];
 * O: device fp32 [H_q, D]; LSE: device fp32 [H_q] or NULL; K_suf/V_suf: device fp16
 * [H_kv, S_suf, D] or NULL when S_suf == 0. Limits: H_kv * ceil(N/16) * 20*D bytes of resident
 * tiles <= 16 MiB, D in {64, 128, 192, 256}; larger inputs return PCK_EUNSUPPORTED before any
 * launch. The first call on a device (or the first pck_noalloc_status there) looks up the
 * scratch addresses and the kernels' occupancy: make it before any stream capture. All calls
 * share the scratch: calls that overlap on the GPU (other streams or host threads) race and
 * must be serialised by the caller. Returns PCK_OK, PCK_EINVAL, PCK_EUNSUPPORTED or PCK_ECUDA
 * (no context, so no pck_last_error text). A kernel-side failure (see pck_sync's codes) shows
 * only in pck_noalloc_status. */
#define PCK_NOALLOC_SCRATCH_BYTES ((16u << 20) + (16u << 20) + 64u * 4u)
int pck_attend_records_noalloc(int H_kv, int N, int D, const void *K_rec, const void *V_rec, int H_q,
                               int q_dtype, const void *Q, const int32_t *head_map, int S_suf,
                               const void *K_suf, const void *V_suf, float *O, float *LSE, void *stream);

/* Status of the pck_attend_records_noalloc calls made on the current device since the last
 * status call. Synchronises `stream`, reads the scratch's device error word and clears it.
 * PCK_OK: no kernel reported an error. PCK_ECUDA: a CUDA error, or some call's kernels set a
 * device error code (written to *code when code != NULL; the codes are pck_sync's): at least
 * one of those calls wrote invalid results. Callers that use the results should check it. */
int pck_noalloc_status(void *stream, int *code);

/* ---- The paged tail: what a session adds behind (or without) a resident prefix.
 *
 * The caller owns a cache of pages and says, per call, which pages each sequence uses. These calls
 * take the device's tables and lengths as they are when the stream reaches them, allocate nothing
 * and use no workspace of the context, so calls of several streams, and replays of several
 * captured graphs, may overlap when their own buffers do not; on the host, one context is still
 * called by one thread at a time. A value on the device that is out of range (a page number
 * outside [0, n_pages), a rotary position outside the table, a length beyond the table's width, more
 * rows than max_rows, cu_rows that descends or points outside [0, T]) is never followed: the call's results are then
 * invalid and pck_sync reports PCK_ECUDA with code 8, 9 or 10. The current device is left as it was. */

/* A cache: K and V hold [n_pages, H_kv, page_size, D] in any order of the first three dimensions
 * (strides in elements, D innermost and contiguous), fp16 or bf16. Both must be 16-byte aligned,
 * strides of dimensions larger than 1 positive multiples of 8. page_size: a multiple of 16. */
typedef struct pck_paged_cache {
    void *K, *V;              /* device */
    int dtype;                /* PCK_DT_F16 or PCK_DT_BF16 */
    int H_kv, D, page_size;
    int64_t n_pages;
    int64_t k_page, k_head, k_token;   /* strides of K */
    int64_t v_page, v_head, v_token;   /* strides of V */
} pck_paged_cache;

/* The sequences of a call. Sequence b's rows are cu_rows[b] .. cu_rows[b+1]-1 of T (cu_rows
 * ascending; rows in front of the first sequence's or behind the last's are neither read nor written, but that attention's
 * tiles may load Q rows behind the last, among the T, that they do not use); they are the
 * last ones of its kv_len[b] cached tokens: row i of its n rows stands at cache position
 * kv_len[b] - n + i, and token p of the cache lies in page table[b][p / page_size], slot
 * p % page_size. Table entries that no visible token needs are not read. cu_rows NULL: one row per
 * sequence (T == B). max_pages * page_size is at most 2^30. Rows with a negative
 * cache position (a padded sequence of length 0) see and store nothing: attention gives O = 0 and LSE = -inf (or the
 * prior's), an append Q = 0. */
typedef struct pck_paged_batch {
    int B, T;
    const int32_t *cu_rows;   /* device [B + 1], or NULL */
    const int32_t *kv_len;    /* device [B] */
    const int32_t *table;     /* device [B, max_pages] */
    int max_pages;
    int max_rows;             /* host bound on one sequence's rows, at least 1 (T will do) */
} pck_paged_batch;
#define PCK_PAGED_MAX_BATCH 2048

/* A rotation of the first R elements of each head (R a multiple of 16, at most D). cos_sin: device
 * fp32 [n_pos, R], R/2 cosines and then R/2 sines of each position's angles. Pair i is elements
 * (i, i + R/2), or (2i, 2i + 1) when interleaved: (a, b) -> (a cos - b sin, b cos + a sin).
 * positions: device int32 [T], or NULL (append only: the rows' cache positions). */
typedef struct pck_rotary {
    const float *cos_sin;
    int n_pos, R, interleaved;
    const int32_t *positions;
} pck_rotary;

/* Rows [T, H, D] in, and the same out (in place allowed): strides in elements, D contiguous,
 * 16-byte aligned, strides of dimensions larger than 1 multiples of 8 (4 for fp32). */
typedef struct pck_rows {
    const void *in;           /* device; NULL: none of this kind */
    void *out;
    int H;
    int64_t in_row, in_head, out_row, out_head;
    const void *weight;       /* norm weight [D] of the rows' type, or NULL (all ones) */
} pck_rows;

/* RMS norm of each head of Q and K, then the rotation, in one pass, held in fp32 and rounded once:
 * y = x / sqrt(mean(x^2) + eps) * weight. Q or K may have no rows (in NULL). norm 0: rotation only;
 * rope NULL: norm only. dtype: F32, F16 or BF16 (in, out and weights). D: a multiple of 16 up to
 * 512. The output strides fit Q for pck_query_fused ([H_q, M, D]) and K for its dense suffix as
 * they fit [T, H, D]. */
int pck_qk_norm_rope(pck_ctx *ctx, int dtype, int T, int D, const pck_rows *Q, const pck_rows *K, int norm,
                     float eps, const pck_rotary *rope, void *stream);

/* Append: stores K (normed and rotated as above, where asked) and V (as it is) of every row into
 * its cache slot, and in the same pass norms and rotates Q, out of or in place, when Q is not NULL.
 * K->out, V->out and their strides are not used. dtype: the cache's, or F32 (rounded once into the
 * cache; Q stays F32). D: a multiple of 16 up to 512. Two rows of one call must not name one slot. */
int pck_paged_append(pck_ctx *ctx, const pck_paged_cache *cache, const pck_paged_batch *batch, int dtype,
                     const pck_rows *Q, const pck_rows *K, const pck_rows *V, int norm, float eps,
                     const pck_rotary *rope, void *stream);

/* Attention of Q rows over the cached tokens of their sequences. Q: device [T, H_q, D] of the
 * cache's type (strides in elements, D contiguous, 16-byte aligned, multiples of 8), q head h on kv
 * head h / (H_q / H_kv). A row at cache position p sees tokens 0 .. p; with window > 0 only the
 * last `window` of these and the first `sinks` of the cache. O: device [T, H_q, D] of the
 * cache's type, contiguous; LSE: device fp32 [T, H_q] or NULL. A row that sees nothing gets O = 0
 * and LSE = -inf. Cached tokens that no row of the call sees are not used, whatever they hold.
 * O_prior (device fp32 [T, H_q, D]) and LSE_prior ([T, H_q]): attention of the same rows over other
 * keys, e.g. what pck_query_batch gave for a resident prefix: O and LSE are then those over both
 * (both NULL otherwise). pck_query at M > 1 gives [H_q, M, D] and [H_q, M]: the caller transposes these. `window`
 * and `sinks` count the tokens of this cache alone and a prior is taken whole, so a layer whose window, or whose first
 * tokens, lie in a resident prefix is not window + prior.
 * Scores, maxima, sums and O are held in fp32. The weights 2^(s - m) that multiply V are rounded: in the one-token
 * kernel to a pair of 16-bit values (22 bits in fp16, 16 in bf16; the output's own rounding is coarser), in the
 * row kernel once to the cache's type (11 bits, 8 in bf16; prompts of the kind measured then differ from 64 bits by
 * 1.3 times the output's own rounding in bf16, 1.4 times in fp16). fp16 weights below 2^-37 (rows: 2^-31) of the largest
 * one are lost.
 * One row per sequence (cu_rows NULL), or a few (min(max_rows, T) * H_q / H_kv at most 16, 8 at D > 128): split
 * over the cache's length and joined; D in {64, 128, 192, 256}. More rows: tiles of 256 rows (tokens x
 * heads of a kv head) on the tensor cores, D in {64, 128}, H_q / H_kv at most 128. Other head dimensions, which an
 * append fills a cache with, return PCK_EUNSUPPORTED. B <= PCK_PAGED_MAX_BATCH.
 * workspace: device, 16-byte aligned, pck_paged_workspace bytes (which may be 0), read and written
 * by this call only while it runs: calls that may overlap need one each. */
int pck_paged_attend(pck_ctx *ctx, const pck_paged_cache *cache, const pck_paged_batch *batch, int H_q,
                     const void *Q, int64_t q_row, int64_t q_head, int window, int sinks,
                     const float *O_prior, const float *LSE_prior, void *O, float *LSE,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of that call into *bytes (it depends on sizes only, not on device values). */
int pck_paged_workspace(pck_ctx *ctx, const pck_paged_cache *cache, const pck_paged_batch *batch, int H_q,
                        int window, int sinks, size_t *bytes);

/* ---- The same tail held in 8 bits.
 *
 * A quantised cache: codes K and V [n_pages, H_kv, page_size, D] in FP8 e4m3 (1-4-3 bits, largest value 448, NaN 0x7f,
 * no infinities) in any order of the first three dimensions (strides in elements, D contiguous; 16-byte aligned, strides of
 * dimensions larger than 1 positive multiples of 16), and one scale per token and kv head, K_scale and V_scale
 * [n_pages, H_kv, page_size], contiguous, 16-byte aligned: a power of two 2^(byte - 127) (E8M0; 255 is NaN). A value is
 * code * 2^(byte - 127). D + 1 bytes a head row where 16-bit pages have 2 D.
 * page_size, D, the batch, the rotary table, streams, workspaces and errors are as above. */
typedef struct pck_paged_cache_e4m3 {
    void *K, *V;                       /* device */
    uint8_t *K_scale, *V_scale;        /* device */
    int H_kv, D, page_size;
    int64_t n_pages;
    int64_t k_page, k_head, k_token;   /* strides of K */
    int64_t v_page, v_head, v_token;   /* strides of V */
} pck_paged_cache_e4m3;

/* pck_paged_append into a quantised cache. dtype: of Q, K and V, F32, F16 or BF16. A head row y (K normed and rotated in fp32, V as
 * it is) whose largest finite magnitude is a gets the least e with a 2^-e <= 448, held to -126 .. 120 (a row of zeros: -126), and
 * the codes y 2^-e rounded to nearest even: one rounding, of half a step 2^-4 of the value, or 2^-10 * 2^e where that is
 * more. Infinities and NaN become NaN. A row whose largest magnitude is 2^128 (1 - 2^-5) or more, the last 2^-5 below fp32's end,
 * has a code that stands for 2^128: an infinity in fp32 and bf16. */
int pck_paged_append_e4m3(pck_ctx *ctx, const pck_paged_cache_e4m3 *cache, const pck_paged_batch *batch, int dtype,
                          const pck_rows *Q, const pck_rows *K, const pck_rows *V, int norm, float eps,
                          const pck_rotary *rope, void *stream);

/* pck_paged_attend over the values of a quantised cache: rows, window, sinks, priors, outputs and limits as there. q_dtype: of
 * Q and O, F16 or BF16.
 * One row per sequence, or a few (as there): the codes are multiplied as they are, exactly, and the scales applied to the
 * scores and to the weights, in fp32. Weights times their V scale are held as fp16 pairs, to 22 bits and to 2^-37 of a head's
 * largest; where the token with the largest has a V scale of 2^(-40 - b), to 2^(-37 + b) of it (below 2^-77 nothing is left). A bf16 q
 * is held to 2^-39 of the row's largest element; a scale of 2^-127 (byte 0, which an append never writes) counts as 0.
 * More rows: what they see is first read back, as by pck_paged_read_e4m3, into 16-bit pages of q_dtype in the workspace: as many as
 * max_pages and B name (with a window only those that it reaches), at most as many as the cache has. Where these would
 * take more than 4 GiB and more than half of the codes' bytes, the call goes through its kv heads, and then its sequences, some at a
 * time, down to one sequence's pages of one kv head. So the peak is the codes and half of them again (or 4 GiB), and a table no
 * wider than its sequences need keeps the workspace small and the call whole. bf16 holds the values as far as
 * pck_paged_read_e4m3 says. fp16 does not reach as far as the cache's scales: values below 2^-14 are held to 2^-25, and one
 * above 65,536 that a row sees makes the call's results invalid (pck_sync reports PCK_ECUDA with code 16): such a cache
 * takes a bf16 q. */
int pck_paged_attend_e4m3(pck_ctx *ctx, const pck_paged_cache_e4m3 *cache, const pck_paged_batch *batch, int q_dtype, int H_q,
                          const void *Q, int64_t q_row, int64_t q_head, int window, int sinks,
                          const float *O_prior, const float *LSE_prior, void *O, float *LSE,
                          void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of that call into *bytes. */
int pck_paged_workspace_e4m3(pck_ctx *ctx, const pck_paged_cache_e4m3 *cache, const pck_paged_batch *batch, int q_dtype,
                             int H_q, int window, int sinks, size_t *bytes);

/* Rows of a quantised cache read back: each sequence's last cached tokens (its rows, as in pck_paged_batch; cu_rows from
 * kv_len takes whole caches), K->out and V->out [T, H_kv, D] of dtype F32, F16 or BF16 with the strides given (in and weight are
 * not used): [H_kv, N, D], as pck_store takes it, is a row stride of D. Values are rounded once. fp32 holds
 * them exactly, bf16 those of scales 2^-124 .. 2^119 (below, codes end under its smallest step, 2^-133); in both, a value of 2^128
 * and more, which codes of 256 and above have at 2^120, is an infinity. In fp16 what is beyond 65,504 is 65,504. Rows at a
 * negative cache position are 0. */
int pck_paged_read_e4m3(pck_ctx *ctx, const pck_paged_cache_e4m3 *cache, const pck_paged_batch *batch, int dtype,
                        const pck_rows *K, const pck_rows *V, void *stream);

/* Counters of ctx. */
int pck_info(pck_ctx *ctx, pck_info_t *out);

/* Synchronise `stream` and report any asynchronous CUDA error as PCK_ECUDA. Also PCK_ECUDA when
 * a kernel's bounded wait gave up since the last check (a TMA stage or pipeline barrier that
 * never completed). The kernel then skipped the rest of its work, so the affected results are
 * invalid. pck_last_error names the code: 1 decode ring stage, 2 prefill producer, 3 prefill
 * MMA warp, 4 prefill softmax, 5 prefill final O, 6 sparse scoring copy, 7 an fp32 Q element
 * of an M=1 query with |q| * log2(e) / sqrt(D) >= 65504 (or not finite): the M=1 kernels
 * carry q * log2(e) / sqrt(D) as an fp16 hi + lo pair, so |q| < 65504 * sqrt(D) / log2(e)
 * (e.g. 363,000 at D = 64) is the valid range; 8 a page number, 9 a rotary position, 10 a cache
 * length, row count or cu_rows out of range (the paged-tail calls); 11 a page tile of a one-row paged attention; 12 loads, 13
 * MMAs, 14 softmax, 15 final O of a ragged paged attention. The error word and the selector's counters
 * are then reset, so the context stays usable. */
int pck_sync(pck_ctx *ctx, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PCK_H */
