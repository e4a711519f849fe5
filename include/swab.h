/*
 * swab.h -- C ABI of the sliding-window (banded) attention library for one
 * NVIDIA GB300 (sm_103a).
 *
 * The operation (pages: "Developing a faster schedule for Longformer's
 * kernel", TVM forum, posts 1, 3, 5 and 6):
 *   Longformer attention is built from a banded ("diagonal") matrix product:
 *   of Q.K^T only the diagonals k in [-w, w_upper] are computed, with
 *   dilation d (key stride s = d + 1), so query row i meets key
 *       j = i + k*s,   k = t - w,   slot t in [0, D),   D = w + w_upper + 1.
 *   A slot whose key falls outside [0, n) holds the constant `padding`.
 *   Post 6 names three modes of one kernel: the forward product (dense x
 *   dense^T -> band, t3d3 = 2w+1) and two backward products (band x dense,
 *   transpose_t1 = 0, and band^T x dense, transpose_t1 = 1).  The author
 *   merged them into one function only because they could not put several
 *   kernels into one .so; here they are separate entry points.
 *
 * Global tokens ("[WIP] Improve LongformerAttention performance", ONNX
 * Runtime issue, item (1): one global index of length S shared by the batch):
 *   G sorted, unique positions shared by every (b, h).  A row i not in G
 *   attends to its band keys that are not in G plus all of G; a row in G
 *   attends to every key.  The extra dense pieces live in caller-owned
 *   companion tensors (swab_glob): `cols` [b,h,n,G] holds every row's value
 *   at the G global keys, `rows` [b,h,G,n] holds the dense rows of the G
 *   global queries.  Band slots whose key is in G, and the band rows and
 *   `cols` rows of global queries, are not used by attention.
 *
 * Conventions for every entry point:
 *   - Layouts are row-major and contiguous: dense tensors (Q, K, V, O, dO,
 *     dQ, dK, dV) [b,h,n,head_dim]; band tensors (S, P, dP, dS) [b,h,n,D];
 *     lse [b,h,n] fp32.  Element type = desc->dtype for all but lse.
 *   - All tensor pointers are DEVICE pointers owned by the caller, 16-byte
 *     aligned.  Band tensors must be readable up to the next 16-byte
 *     boundary past their last element (any cudaMalloc / PyTorch allocation
 *     is).  The library allocates, frees and synchronises nothing.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous on it; results are ready when the stream reaches them.
 *   - Arguments are validated on the host before anything is launched; a
 *     failed validation returns an error and launches nothing.
 *   - Invalid slots (key outside [0, n)) of an INPUT band tensor are ignored,
 *     whatever they hold; `padding` is written only by band_qk.
 *   - No entry point aborts or prints.  A launch failure returns
 *     SWAB_ERR_CUDA.  Device-side waits are bounded: a wait that gives up
 *     records SWAB_ERR_TIMEOUT in the library's device status word, read with
 *     swab_device_status().
 *   - Tensor-core paths: dtype f16/bf16 with head_dim 64.  dtype f32 runs an
 *     exact-fp32 FFMA path (head_dim 1..128).
 */
#ifndef SWAB_H
#define SWAB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(_WIN32)
#define SWAB_API __declspec(dllexport)
#else
#define SWAB_API __attribute__((visibility("default")))
#endif

#define SWAB_MAX_GLOBAL 256  /* most global tokens per call */
#define SWAB_MAX_DILATION 15 /* key stride at most 16 */
#define SWAB_NOALLOC_MAX_ROWS (1u << 22) /* b*h*n limit of band_attention_bwd_noalloc */

typedef enum swab_status {
    SWAB_OK = 0,
    SWAB_ERR_INVALID_ARG = 1, /* NULL pointer, negative size, bad global index */
    SWAB_ERR_UNSUPPORTED = 2, /* head_dim / dtype / size outside what is built */
    SWAB_ERR_MISALIGNED = 3,  /* a tensor pointer is not 16-byte aligned */
    SWAB_ERR_CUDA = 4,        /* a CUDA call or kernel launch failed */
    SWAB_ERR_TIMEOUT = 5,     /* a device wait gave up (see swab_device_status) */
    SWAB_ERR_BOUNDS = 6       /* bounds-checked build only: a kernel's global access
                                 fell outside the call's buffers (swab_bounds_report) */
} swab_status;

typedef enum swab_dtype { SWAB_F32 = 0, SWAB_F16 = 1, SWAB_BF16 = 2 } swab_dtype;

/* Problem description: the kernel parameters of the TVM forum thread, posts
 * 5-6 (b, n, h, w, w_upper, padding; the head dimension replaces m = 768
 * divided over h = 12 heads) plus the dilation of post 3 and the global
 * index of the ONNX Runtime issue. */
typedef struct swab_desc {
    int32_t b;                 /* batch */
    int32_t h;                 /* heads (merged with the batch: slices b*h) */
    int32_t n;                 /* sequence length, >= 1 */
    int32_t head_dim;          /* 64 for f16/bf16; 1..128 for f32 */
    int32_t w;                 /* keys on the left, >= 0 */
    int32_t w_upper;           /* keys on the right, >= 0 (0 = autoregressive) */
    int32_t dilation;          /* 0..SWAB_MAX_DILATION; key stride dilation+1 */
    float padding;             /* value band_qk writes where the key is outside [0,n) */
    int32_t dtype;             /* swab_dtype of every tensor except lse */
    int32_t n_global;          /* G, 0..SWAB_MAX_GLOBAL; 0 = no global tokens */
    const int32_t *global_idx; /* HOST array of G sorted unique positions in [0,n) */
    /* Optional key-padding bias (nvFuser issue "HuggingFace BertForMaskedLM -
     * Log Softmax Fusion...", fusion 1, adds (1 - mask) * -10000 per key to the
     * scaled scores): DEVICE array of b*n fp32, 4-byte aligned, row bb holding
     * the term added to the score of every query of batch bb with key j
     * before the softmax; NULL for none.  Read by band_softmax, band_attention
     * and band_attention_bwd (the other calls do not depend on it).  With
     * n_global > 0 the fused pair adds it to every key a row attends to: the
     * band keys and the global columns of a local row, every key of a global
     * row; band_softmax likewise adds it to the band slots, the global
     * columns (key global_idx[g]) and the dense global rows.
     * global_attention, global_attention_bwd and band_attention_bwd_noalloc
     * return SWAB_ERR_UNSUPPORTED when it is set. */
    const float *key_bias;
    /* Optional dropout of the attention probabilities (the nvFuser fusion 1
     * dropout, p with 1/(1-p) scaling), in band_attention and
     * band_attention_bwd (pass the same values to both): dropout_p in [0, 1) is
     * rounded to t = round(256 * dropout_p) (at most 255); an element is kept
     * with probability 1 - t/256 and then scaled by 256 / (256 - t).  Element
     * (slice bh, query i, key j) is kept iff byte (b mod 32), b = floor(j / s),
     * of the Philox4x64-10 block at counter (floor(b / 32), i, bh, 0) and key
     * (dropout_seed, 0) -- bytes little-endian from the four output words --
     * is >= t.  lse is that of the probabilities before dropout.  Read by
     * band_softmax_dropout, band_softmax_bwd, band_attention and
     * band_attention_bwd; with t > 0, band_softmax (use band_softmax_dropout),
     * global tokens and band_attention_bwd_noalloc return SWAB_ERR_UNSUPPORTED;
     * the other calls do not depend on it. */
    float dropout_p;
    uint64_t dropout_seed;
    /* Optional strided layout of the dense tensors in band_attention and
     * band_attention_bwd (ONNX Runtime issue "[WIP] Improve LongformerAttention
     * performance": the merged QKV projection leaves rows of [b, n, 3, h,
     * head_dim]).  0 = the contiguous [b, h, n, head_dim] layout.  Otherwise
     * the row stride in elements: element (batch bb, head hh, position i,
     * channel c) is at (bb * n + i) * stride + hh * head_dim + c, i.e. rows of
     * [b, n, stride] with the heads side by side; stride >= h * head_dim and a
     * multiple of 16 bytes (else SWAB_ERR_INVALID_ARG / SWAB_ERR_MISALIGNED).
     * qkv_row_stride applies to Q, K, V, dQ, dK, dV (3 h head_dim reads Q, K, V
     * straight from the merged projection: pass its base, base + h head_dim and
     * base + 2 h head_dim); out_row_stride to O and dO.  lse stays [b, h, n].
     * The other calls (materialised band products, band_attention_bwd_noalloc)
     * take the contiguous layout only (SWAB_ERR_UNSUPPORTED). */
    int64_t qkv_row_stride;
    int64_t out_row_stride;
    /* Optional keep-bit cache of the fused dropout (f16 / bf16 band_attention
     * and band_attention_bwd with dropout_p > 0): DEVICE buffer of
     * band_attention_dropout_mask_bytes(desc) bytes, 4-byte aligned; NULL for
     * none.  band_attention writes into it the keep bits it draws (32 keys of
     * a query row to a word); band_attention_bwd, given the buffer that
     * band_attention filled for the same description (sizes, window, dilation,
     * dropout_p, dropout_seed), reads them instead of drawing them again.  The
     * decisions are the same either way.  The other calls ignore it. */
    uint32_t *dropout_mask;
} swab_desc;

/* Companion of a band tensor when n_global > 0 (device pointers, dtype of the
 * band tensor).  Pass NULL when n_global == 0. */
typedef struct swab_glob {
    void *cols; /* [b,h,n,G]: value of row i at key global_idx[g] */
    void *rows; /* [b,h,G,n]: dense row of query global_idx[g] over all keys */
} swab_glob;

/* Forward product (TVM thread, post 6: dense x dense^T -> t3d3 = D diagonals):
 *   S[i,t] = alpha * sum_c A[i,c] * B[j,c]  with j = i + (t-w)*s in [0,n),
 *   S[i,t] = padding otherwise; accumulation in fp32, one round-to-nearest
 *   into the output dtype.
 * Forward scores: A = Q, B = K, alpha = 1/sqrt(head_dim).  Backward:
 * A = dO, B = V, alpha = 1 gives dP.  With globals, also writes
 * Sg->cols[i,g] = alpha*A[i].B[G[g]] and Sg->rows[g,j] = alpha*A[G[g]].B[j]. */
SWAB_API swab_status band_qk(const swab_desc *desc, float alpha, const void *A, const void *B,
                             void *S, const swab_glob *Sg, void *stream);

/* Masked row softmax over the band (nvFuser issue "HuggingFace
 * BertForMaskedLM - Log Softmax Fusion...", fusion 1: max, exp(x - max), sum,
 * divide, in fp32):
 *   P[i,t] = exp(S[i,t] - m_i) / Z_i on used slots, 0 on the others;
 *   lse[i] = m_i + log Z_i (lse may be NULL).
 * With globals the row also covers Sg->cols (written to Pg->cols); a global
 * query's row is the dense Sg->rows row (written to Pg->rows) and its band
 * row and cols row are written as zeros. */
SWAB_API swab_status band_softmax(const swab_desc *desc, const void *S, const swab_glob *Sg,
                                  void *P, const swab_glob *Pg, float *lse, void *stream);

/* Masked row softmax followed by dropout (nvFuser issue "HuggingFace
 * BertForMaskedLM - Log Softmax Fusion...", fusion 1, whose outputs include
 * both the probabilities and the dropped, rescaled probabilities):
 *   P[i,t]  as band_softmax (before dropout; P may be NULL if not needed);
 *   Pd[i,t] = f(i,t) * P[i,t], f = 256/(256-t) or 0 the keep-and-scale factor
 *             of the slot's key under the descriptor's dropout (f = 1 when
 *             dropout_p rounds to 0); 0 on unused slots;
 *   lse[i]  as band_softmax (before dropout; may be NULL).
 * The forward product is then O = band_pv(Pd, V); for the backward,
 * band_softmax_bwd with the same descriptor takes P and the gradient of Pd.
 * The keep decisions are recomputed from the descriptor, never stored.
 * No global tokens (SWAB_ERR_UNSUPPORTED); D <= 65536 (else
 * SWAB_ERR_UNSUPPORTED). */
SWAB_API swab_status band_softmax_dropout(const swab_desc *desc, const void *S, void *P, void *Pd,
                                          float *lse, void *stream);

/* AddBiasTranspose (ONNX Runtime issue "[WIP] Improve LongformerAttention
 * performance", item (2): the bias add and the transpose after the merged
 * projection in one kernel, with the widest vector loads, conclusion (g)):
 *   Y[m, bb, hh, i, c] = X[bb, i, m, hh, c] + bias[m, hh, c]
 * for M matrices side by side in each row of X (M = 3: Q, K, V), i.e.
 * X = rows of [b, n, M, h, head_dim] -> Y = M tensors [b, h, n, head_dim].
 * b, h, n, head_dim and dtype come from desc (head_dim * element size a
 * multiple of 16 bytes); the sum is rounded once to the dtype (correctly
 * rounded).  bias ([M, h, head_dim]) may be NULL: a pure transpose.  X, Y,
 * bias device pointers, 16-byte aligned; Y must not overlap X. */
SWAB_API swab_status add_bias_transpose(const swab_desc *desc, int32_t M, const void *X,
                                        const void *bias, void *Y, void *stream);

/* Global queries with their own projections (ONNX Runtime issue "[WIP]
 * Improve LongformerAttention performance", item (3) and its "compact
 * global_q"): the G = desc->n_global global queries, given compact as
 * Qg [b, h, G, 64] (the global_q projection of the global tokens only), attend
 * to every position through separate global key / value projections
 * Kg, Vg [b, h, n, 64]:
 *   Og[g] = sum_j p_gj Vg[j],  p_gj = softmax_j(scale * Qg[g].Kg[j]),
 *   lseg[g] = log sum_j exp(scale * Qg[g].Kg[j])   ([b, h, G] fp32, may be NULL).
 * Together with the band path this gives attention with separate global
 * projections: run the band calls with global_idx (local rows attend to their
 * band keys outside G plus G, with Q, K, V), then replace O's global rows
 * O[G[g]] by Og[g].  In the backward, give the band calls dO with its global
 * rows set to 0 and global_attention_bwd dOg[g] = dO[G[g]].
 * head_dim 64, contiguous layout, no key bias or dropout.  workspace:
 * global_attention_workspace(desc) bytes of device memory, 16-byte aligned,
 * shared by the forward and the backward (not concurrently). */
SWAB_API size_t global_attention_workspace(const swab_desc *desc);
SWAB_API swab_status global_attention(const swab_desc *desc, float scale, const void *Qg,
                                      const void *Kg, const void *Vg, void *Og, float *lseg,
                                      void *workspace, void *stream);
/* Backward of global_attention: with delta_g = dOg[g].Og[g] and
 * ds_gj = p_gj (dOg[g].Vg[j] - delta_g):
 *   dQg = scale ds Kg,  dKg = scale ds^T Qg,  dVg = p^T dOg.
 * lseg is the forward's (required).  dKg, dVg rows have one writer each;
 * dQg sums per-tile partials in a fixed order (bitwise repeatable). */
SWAB_API swab_status global_attention_bwd(const swab_desc *desc, float scale, const void *Qg,
                                          const void *Kg, const void *Vg, const void *Og,
                                          const void *dOg, const float *lseg, void *dQg,
                                          void *dKg, void *dVg, void *workspace, void *stream);

/* Band x dense product (TVM thread, post 6: transpose_t1 = 0, t1d3 = 2w+1):
 *   O[i,c] = alpha * sum over used slots t of P[i,t] * V[j(i,t), c]
 *            (+ alpha * sum_g Pg->cols[i,g] * V[G[g],c]);
 *   a global query's row is alpha * sum_j Pg->rows[g,j] * V[j,c].
 * Forward: O = P.V (alpha = 1).  Backward: dQ = band_pv(alpha, dS, K). */
SWAB_API swab_status band_pv(const swab_desc *desc, float alpha, const void *P,
                             const swab_glob *Pg, const void *V, void *O, void *stream);

/* Transposed band x dense product (TVM thread, post 6: transpose_t1 = 1):
 *   X[j,c] = alpha * sum over (i,t) with j(i,t) = j, t used, of Bd[i,t]*Y[i,c]
 *            (+ global terms of Bg->cols and Bg->rows).
 * band_qk_bwd_t gives dK = alpha * dS^T.Q; band_pv_bwd_t gives
 * dV = P^T.dO (alpha = 1).  The two names run the same kernel.
 * Deterministic: every output row has one writer, no atomics. */
SWAB_API swab_status band_qk_bwd_t(const swab_desc *desc, float alpha, const void *dS,
                                   const swab_glob *dSg, const void *Q, void *dK, void *stream);
SWAB_API swab_status band_pv_bwd_t(const swab_desc *desc, float alpha, const void *P,
                                   const swab_glob *Pg, const void *dO, void *dV, void *stream);

/* Softmax backward on the band (derivative of band_softmax):
 *   dS[i,t] = P[i,t] * (dP[i,t] - delta_i) on used slots, 0 elsewhere,
 *   delta_i = sum over used slots of P*dP (+ sum_g Pg*dPg);
 * global pieces likewise (dSg->cols, dSg->rows).  With the descriptor's
 * dropout (derivative of band_softmax_dropout's Pd): P is the probabilities
 * before dropout, dP the gradient of Pd, and
 *   dS[i,t] = P[i,t] * (f(i,t) dP[i,t] - delta_i), delta_i = sum P*f*dP
 * (D <= 65536, else SWAB_ERR_UNSUPPORTED). */
SWAB_API swab_status band_softmax_bwd(const swab_desc *desc, const void *P, const swab_glob *Pg,
                                      const void *dP, const swab_glob *dPg, void *dS,
                                      const swab_glob *dSg, void *stream);

/* Fused forward: the same O (and lse, may be NULL) as band_qk(scale) ->
 * band_softmax -> band_pv, with the scores kept on chip (never written to
 * memory).  With global tokens (f16 / bf16, contiguous layout, lse required,
 * n <= 188416): local rows attend to their band keys outside G plus G, global
 * rows to every key, as in the materialised calls; computed as the band part
 * (global keys masked), the global columns merged into the local rows by
 * log-sum-exp, and the global rows' dense attention.  fp32 or the strided
 * layout with global tokens: SWAB_ERR_UNSUPPORTED. */
SWAB_API swab_status band_attention(const swab_desc *desc, float scale, const void *Q,
                                    const void *K, const void *V, void *O, float *lse,
                                    void *stream);

/* Fused backward of band_attention: dQ, dK, dV of
 *   O = softmax_band(scale * Q.K^T) . V
 * recomputing the band probabilities on chip from lse (the forward's
 * log-sum-exp) and never writing a band tensor:
 *   P = exp(scale*Q.K^T - lse), dP = dO.V^T, delta_i = dO_i . O_i,
 *   dS = P*(dP - delta), dQ = scale*dS.K, dK = scale*dS^T.Q, dV = P^T.dO
 * on the used slots (the two backward products of the TVM thread, post 6,
 * with the textbook softmax derivative).
 * `workspace` is caller-owned device memory of band_attention_bwd_workspace()
 * bytes, 16-byte aligned; its contents on entry do not matter.  For fp16 /
 * bf16 it holds the per-row delta and an fp32 dQ accumulator: dK and dV have
 * one writer per row, while each key tile's contribution to dQ is added into
 * the accumulator by TMA reduce-add stores (cp.reduce.async.bulk.tensor, fp32
 * additions in the memory system) in an order that varies between runs, so
 * dQ may differ in its last bits from run to run (within the rounding of one
 * fp32 sum; band_attention_bwd_noalloc is bitwise repeatable).  For fp32 it holds the delta only and every output is
 * repeatable.
 * For fp16 / bf16 the call launches three kernels.  The last two are launched
 * as programmatic dependents: they may start while the one before runs and
 * wait inside for what it wrote.  For the caller the call stays ordered on
 * the stream like any kernel launch.
 * Global tokens (f16 / bf16, contiguous layout, no key bias or dropout,
 * n <= 98304; else SWAB_ERR_UNSUPPORTED): the gradients of the attention with
 * global tokens of band_attention -- local rows over their band keys outside G
 * plus G, global rows over every key.  The call then runs the band (global
 * keys and global queries left out), the global columns (every local row
 * against the G global keys, gathered into the workspace) and the global
 * rows (the global_attention_bwd computation with the shared Q, K, V as the
 * global projections), the dK, dV terms of all three added in fp32 before one
 * rounding; the workspace (band_attention_bwd_workspace) then also holds the
 * gathered rows and keys and the global rows' dK, dV terms. */
SWAB_API swab_status band_attention_bwd(const swab_desc *desc, float scale, const void *Q,
                                        const void *K, const void *V, const void *O,
                                        const void *dO, const float *lse, void *dQ, void *dK,
                                        void *dV, void *workspace, void *stream);

/* Bytes of the keep-bit cache (swab_desc.dropout_mask) for `desc`: b*h*n rows
 * of ceil((w + w_upper + 1) / 32) + 1 words (0 if desc is NULL). */
SWAB_API size_t band_attention_dropout_mask_bytes(const swab_desc *desc);

/* Bytes of workspace band_attention_bwd needs for `desc` (0 if desc is NULL):
 * fp16 / bf16: round_up(b*h*n*4, 256) + b*h*n*64*4, plus with global tokens
 * the sections of the gathered global rows, keys and values and the global
 * rows' dK, dV terms (about 2*b*h*n*64*2 bytes more);
 * fp32: round_up(b*h*n*4, 256). */
SWAB_API size_t band_attention_bwd_workspace(const swab_desc *desc);

/* band_attention_bwd for callers that cannot allocate device memory: the same
 * computation and arguments, minus the workspace.  It needs only the per-row
 * delta as scratch because it computes dQ in a kernel of its own (one writer
 * per row) instead of summing it in an fp32 accumulator, so its results agree
 * with band_attention_bwd within rounding and repeat bitwise.  Some callers have
 * no way to obtain a device buffer of their own -- code running under an
 * allocator or memory pool they do not control, plugins handed only input and
 * output pointers, or contexts where a cudaMalloc would synchronise or is
 * forbidden -- so this variant keeps its per-row scratch in a module-scope
 * device array of SWAB_NOALLOC_MAX_ROWS floats (16 MiB), which every GPU that
 * loads the library holds until the process exits.  Nothing is allocated or
 * freed by the call (no cudaMalloc, cudaFree or allocating library routine).
 *   - b*h*n must not exceed SWAB_NOALLOC_MAX_ROWS; larger problems return
 *     SWAB_ERR_UNSUPPORTED (use band_attention_bwd with a workspace).
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) and caches it; make that first call before any
 *     stream capture.  A first call made while `stream` is being captured
 *     returns SWAB_ERR_UNSUPPORTED and launches nothing.
 *   - The cached address belongs to the device's context at the first call:
 *     resetting the device (cudaDeviceReset) after that call is not
 *     supported, since later calls would use the old address.
 *   - All calls share the one array, which keeps the last call's contents
 *     (every call overwrites what it reads before reading it).  Calls whose
 *     executions overlap on the GPU -- on different streams, or from different
 *     threads without ordering -- race on it; serialise them.
 * The pages have no counterpart for this entry point: it only changes where
 * the library's own scratch lives. */
SWAB_API swab_status band_attention_bwd_noalloc(const swab_desc *desc, float scale, const void *Q,
                                                const void *K, const void *V, const void *O,
                                                const void *dO, const float *lse, void *dQ,
                                                void *dK, void *dV, void *stream);

/* ---------------------------------------------------------------------------
 * Answering with the banded attention: rotary positions, a paged key / value
 * cache and the attention of a few new tokens a request over it.  One step of
 * a running batch is
 *     cache_slots      lengths -> block table, slot of every new token
 *     rotary_append    Q, K rotated; K, V written to their slots
 *     band_decode      attention of the new tokens over the cache
 * and needs no value on the host, so the three can be captured in a CUDA graph
 * and replayed.  No counterpart on the pages; the key set of a query is theirs
 * (band on the left with dilation, leading global tokens), continued one
 * token at a time.
 *
 * Tokens of a step are flat: row t of the [tokens, heads, head_dim] tensors
 * belongs to request r when q_start[r] <= t < q_start[r + 1]; rows before
 * q_start[0] (cache_slots writes 0) and from q_start[batch] on belong to none.
 *
 * The cache holds K and V as two tensors [n_blocks, hk, page, head_dim].  A
 * request's positions j = 0, 1, ... lie in blocks of `page` positions; block
 * number j / page is found in column c of the request's row of the block table
 * [batch, cols] (int32 block ids), at row j mod page of the block:
 *     c = j / page                                        below cols,
 *     c = pinned + (j / page - pinned) mod (cols - pinned)  from there on when
 *         `ring` is set: the blocks behind the first `pinned` ones are recycled
 *         once a window has left them.
 * A slot is block * page + row.
 *
 * What lies in device memory is not seen by the host checks: a block id or
 * slot outside the cache is never addressed (its key counts as absent, its
 * token is not written) and raises SWAB_ERR_INVALID_ARG in the device status
 * word (swab_device_status).  Id -1 is an empty column: absent, no error.
 * ------------------------------------------------------------------------- */

/* Rotary positions over tokens [b, n] with h query heads and hk key heads. */
typedef struct swab_rotary_desc {
    int32_t b, n;          /* tokens, b * n >= 1 */
    int32_t h, hk;         /* heads of Q (>= 1) and of K (>= 0; 0: no K) */
    int32_t head_dim;      /* a multiple of 16 bytes, at most 512 */
    int32_t rot_dim;       /* leading channels that turn: even, 0..head_dim */
    int32_t interleaved;   /* 0: pairs (c, c + rot_dim / 2); 1: pairs (2c, 2c + 1) */
    int32_t dtype;         /* swab_dtype */
    float scale;           /* factor on cos and sin */
    int32_t pos0;          /* added to every position */
    /* Element strides over (b, n, head) of Q, K, their outputs, and V
     * (rotary_append), the channels adjacent; three zeros = contiguous
     * [b, n, heads, head_dim].  Multiples of 16 bytes; a tensor spans less than
     * 64 GB; the rows of an output must not overlap. */
    int64_t q_stride[3], k_stride[3], qo_stride[3], ko_stride[3], v_stride[3];
} swab_rotary_desc;

/* Ways of scaling the frequencies f_k = base^(-2k / rot_dim) to contexts longer
 * than the `original` one by `factor`: */
typedef enum swab_rotary_scaling {
    SWAB_ROTARY_NONE = 0,
    SWAB_ROTARY_LINEAR = 1, /* f_k / factor: positions interpolated */
    SWAB_ROTARY_NTK = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) */
    SWAB_ROTARY_YARN = 3,   /* Peng et al., "YaRN: Efficient Context Window Extension":
                               f_k / factor where pair k turns less than `low` times within
                               the original context, f_k where more than `high` times, a
                               linear ramp over the pair index between; cos and sin scaled by
                               0.1 ln(factor) + 1 */
    SWAB_ROTARY_BANDS = 4   /* the same limits with the blend linear in the turns */
} swab_rotary_scaling;

/* Fills the HOST array turns[rot_dim / 2] with the frequencies in turns a
 * position, as the fraction of one turn times 2^64 (rounded), and *scale with
 * the factor on cos and sin.  A position times such a number, modulo 2^64, is
 * the angle's fraction of a turn without loss, however far the position.
 * rot_dim even, >= 2; base > 1; factor >= 1; original > 0 and 0 < low < high for
 * YARN and BANDS (else SWAB_ERR_INVALID_ARG).  Needs no GPU. */
SWAB_API swab_status rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                        double original, double low, double high, uint64_t *turns,
                                        float *scale);

/* Rotary positions: with t = 2 pi * frac(p * turns[k] / 2^64) for the position
 * p = pos[bb, i] + pos0 (pos NULL: p = i + pos0) and pair k = (a, b) of a head,
 *     y_a = scale * (x_a cos t - x_b sin t),  y_b = scale * (x_b cos t + x_a sin t),
 * channels from rot_dim on copied; fp32, rounded once (the angle is off by at most
 * 2^-26 pi).  Q -> Qo and, with
 * hk > 0, K -> Ko.  turns: DEVICE array of rot_dim / 2 (NULL when rot_dim is
 * 0); pos: DEVICE int32 [b, n].  An output may be its own input (same pointer
 * and strides), no other overlap. */
SWAB_API swab_status rotary(const swab_rotary_desc *desc, const uint64_t *turns, const int32_t *pos,
                            const void *Q, const void *K, void *Qo, void *Ko, void *stream);
/* Gradient of rotary: the same with t -> -t, dQo -> dQ and dKo -> dK (q_stride,
 * k_stride are those of the inputs dQo, dKo; qo_stride, ko_stride of dQ, dK). */
SWAB_API swab_status rotary_bwd(const swab_rotary_desc *desc, const uint64_t *turns, const int32_t *pos,
                                const void *dQo, const void *dKo, void *dQ, void *dK, void *stream);

typedef struct swab_cache_desc {
    int32_t batch;     /* requests, 1..65535 */
    int32_t page;      /* positions a block: 16, 32, 64 or 128 */
    int32_t n_blocks;  /* blocks of the cache, >= 1; n_blocks * page < 2^31 - 255, and
                          n_blocks * page * hk < 2^32 - 1 */
    int32_t cols;      /* columns of the block table, >= 1 */
    int32_t ring;      /* 1: columns from `pinned` on are recycled */
    int32_t pinned;    /* 0..cols - 1; 0 without ring */
    int32_t max_new;   /* cache_slots: most new tokens of a request, and every token needs a
                          row of slots and pos; 0: no such limits */
} swab_cache_desc;

/* Block tables and slot maps from request lengths, for a step that adds
 * n_new[r] tokens to request r's lens[r] (negative values count as 0).
 *   q_start [batch + 1]: exclusive running sum of n_new (saturating).
 *   table [batch, cols]: the columns that become used, columns ceil(lens / page)
 *     to ceil((lens + n_new) / page) (at most cols), take the next blocks
 *     free_list[used[0]], free_list[used[0] + 1], ... in the order of the
 *     requests; the other columns stay.
 *   slots, pos [tokens]: slot and position + pos0 of every new token; rows past
 *     q_start[batch] get -1 and 0, tokens past `tokens` are not written.  Where
 *     a step adds more than a recycled table holds, tokens whose block the
 *     same step recycles get slot -1.
 *   lens_out [batch] = lens + n_new; used_out[0] = used[0] + blocks taken.
 * A request whose blocks are not all there -- the list (n_free long) runs out in
 * or before it, or, without ring, its length passes cols * page -- gets none:
 * its slots are -1 and lens_out[r] = lens[r]; used_out[1] counts the blocks
 * missing (0: every request was served).  The same holds, with max_new > 0, of a
 * request that adds more than max_new tokens or whose tokens do not all have
 * rows (q_start[r + 1] > tokens): it counts at least one in used_out[1] and raises
 * SWAB_ERR_INVALID_ARG in the status word.  An unserved request's rows of a
 * following band_decode are meaningless.
 * All arrays DEVICE int32, 4-byte aligned; lens_out may be lens and used_out
 * (2 elements) may be used, no other overlap. */
SWAB_API swab_status cache_slots(const swab_cache_desc *cache, int32_t tokens, int32_t pos0,
                                 const int32_t *lens, const int32_t *n_new, int32_t *table,
                                 const int32_t *free_list, int32_t n_free, const int32_t *used,
                                 int32_t *lens_out, int32_t *used_out, int32_t *q_start,
                                 int32_t *slots, int32_t *pos, void *stream);

/* rotary on Q and K fused with the cache write: Q -> Qo rotated; K rotated and V
 * as it is into row slots[t] of Kc, Vc [n_blocks, hk, page, head_dim].  b * n
 * tokens, slots and pos as written by cache_slots; a token with slot -1 is not
 * written (its Q still turns).  rot_dim 0: a plain append (turns, pos may be
 * NULL; Q and Qo both NULL leave Q out).  hk >= 1.  Slots other than -1 must
 * differ from each other.  cache->batch, cols, ring, pinned, max_new are not
 * used. */
SWAB_API swab_status rotary_append(const swab_rotary_desc *desc, const swab_cache_desc *cache,
                                   const uint64_t *turns, const int32_t *pos, const int32_t *slots,
                                   const void *Q, const void *K, const void *V, void *Qo, void *Kc,
                                   void *Vc, void *stream);

/* RMS norm of a head, before its rotary positions. */
typedef struct swab_norm_desc {
    float eps;             /* > 0 */
    float offset;          /* added to every weight (1 where a model stores w - 1) */
    int64_t q_stride[3], k_stride[3]; /* norm_rotary_bwd: element strides of Q and K, as those of swab_rotary_desc */
} swab_norm_desc;

/* Norms of queries and keys, a head at a time, and rotary positions in the same
 * pass: a row x of head_dim channels becomes the rotation (as `rotary`, by the
 * same desc, turns and pos) of
 *     x_c r (w_c + offset),   r = 1 / sqrt(mean_c x_c^2 + eps),
 * fp32, rounded once.  Q -> Qo with the weights wq and, with hk > 0, K -> Ko with
 * wk ([head_dim] of the tensors' dtype, 16-byte aligned; NULL: every weight and
 * the offset together count as 1).  An output may be its own input (same pointer
 * and strides), no other overlap.  The squares are summed in fp32: a row whose sum
 * passes its range gives 0, one with a NaN gives NaN. */
SWAB_API swab_status norm_rotary(const swab_rotary_desc *desc, const swab_norm_desc *norm, const uint64_t *turns,
                                 const int32_t *pos, const void *Q, const void *K, const void *wq,
                                 const void *wk, void *Qo, void *Ko, void *stream);

/* Bytes of workspace norm_rotary_bwd needs (0 if desc is bad). */
SWAB_API size_t norm_rotary_bwd_workspace(const swab_rotary_desc *desc);

/* Gradient of norm_rotary.  With g the gradient dQo turned back (rotary_bwd),
 *     dQ_c = r (g_c v_c - x_c r^2 mean_k(g_k v_k x_k)),   v = w + offset,
 *     dwq_c = sum over all rows of g_c x_c r,
 * the same for K.  Strides: q_stride, k_stride of desc are those of dQo, dKo,
 * qo_stride, ko_stride those of dQ, dK, and norm's those of Q, K.  dwq, dwk
 * [head_dim] fp32, 16-byte aligned; NULL leaves them out (they need wq, wk; dwk is 0
 * where hk is 0).  dQ may be dQo or Q (same pointer and strides), dK likewise, no
 * other overlap.  fp32, the sums over rows in a fixed order (results repeat bitwise
 * on one GPU).  A row of Q or K whose squares pass fp32's range (there norm_rotary
 * gives 0) has the gradient 0 and adds 0 to the weights'.
 * workspace: norm_rotary_bwd_workspace(desc) bytes, 16-byte aligned, needed where
 * dwq or dwk is given; its contents on entry do not matter, calls that may overlap on
 * the GPU need one each. */
SWAB_API swab_status norm_rotary_bwd(const swab_rotary_desc *desc, const swab_norm_desc *norm,
                                     const uint64_t *turns, const int32_t *pos, const void *dQo,
                                     const void *dKo, const void *Q, const void *K, const void *wq,
                                     const void *wk, void *dQ, void *dK, float *dwq, float *dwk,
                                     void *workspace, void *stream);

/* norm_rotary fused with the cache write: rotary_append with Q and K normed
 * first (V as it is). */
SWAB_API swab_status norm_rotary_append(const swab_rotary_desc *desc, const swab_norm_desc *norm,
                                        const swab_cache_desc *cache, const uint64_t *turns,
                                        const int32_t *pos, const int32_t *slots, const void *Q,
                                        const void *K, const void *V, const void *wq, const void *wk,
                                        void *Qo, void *Kc, void *Vc, void *stream);

/* ---------------------------------------------------------------------------
 * The cache in 4 bits.  K and V are two tensors of codes each with one of scales:
 *     codes  [n_blocks, hk, page, head_dim / 2] bytes, channel 2c in the low half
 *            of byte c, channel 2c + 1 in the high half,
 *     scales [n_blocks, hk, page, head_dim / 32] of the tensors' dtype;
 * blocks, slots and the block table as above, head_dim a multiple of 32, at most
 * 256.  Code c (0..15) of a channel stands for s (c - 8), s the scale of its 32
 * adjacent channels.  A group x is written as
 *     the values rounded to dtype (as the cache of that type would hold them),
 *     m = the value of largest magnitude (of two, the positive one),
 *     s = m / -8 rounded to 5 significant bits, but to a multiple of at least 2^-24
 *         (fp16) or 2^-120 (bf16, fp32), and at most 1.25 * 2^11 or 1.25 * 2^123,
 *     c = min(max(rint(x / s), -8), 7) + 8   (ties to even; 8 where s is 0),
 * so that s (c - 8) has at most 8 significant bits: fp16 and bf16 hold it as
 * it is.  With |m| from 2^-17 to 20480 (fp16) or 2^-113 to 1.25 * 2^126 (bf16, fp32)
 * m's own code is 0, its value within 1/32 of m; the others are off by at most
 * |s| / 2, or 1.25 |s| next to -m.  Beyond, values saturate: at 20480 (1.25 * 2^126) on
 * m's side of 0, at 7/8 of that on the other.  Below, m is off by at most 2^-22
 * (2^-118), and a group whose |m| is no more than that becomes zeros.  A group with a
 * NaN or infinity has a NaN scale, codes 8: all its values are NaN.  4.5 bits a value in
 * 16-bit types.
 * ------------------------------------------------------------------------- */

/* rotary_append into a cache in 4 bits (codes Kc, Vc; scales Ks, Vs): Q -> Qo
 * rotated; K rotated and V as it is, quantised, into row slots[t].  With norm Q
 * and K are normed first (norm_rotary); NULL: not (wq, wk are not used).  pos and
 * turns may be NULL with rot_dim 0; Q and Qo both NULL leave Q out.  Codes
 * 16-byte aligned, scales 16-byte aligned. */
SWAB_API swab_status rotary_append4(const swab_rotary_desc *desc, const swab_norm_desc *norm,
                                    const swab_cache_desc *cache, const uint64_t *turns,
                                    const int32_t *pos, const int32_t *slots, const void *Q,
                                    const void *K, const void *V, const void *wq, const void *wk,
                                    void *Qo, void *Kc, void *Ks, void *Vc, void *Vs, void *stream);

/* The values of rows slots[0..tokens) of a cache in 4 bits: K, V [tokens, hk,
 * head_dim] contiguous, of dtype (the scales' too).  Rows with slot -1 stay as they
 * are; other slots outside the cache likewise, recorded as SWAB_ERR_INVALID_ARG in the
 * status word.  tokens >= 1.  cache->batch, cols, ring, pinned, max_new are not used. */
SWAB_API swab_status cache_read4(const swab_cache_desc *cache, int32_t tokens, int32_t hk,
                                 int32_t head_dim, int32_t dtype, const int32_t *slots,
                                 const void *Kc, const void *Ks, const void *Vc, const void *Vs,
                                 void *K, void *V, void *stream);

typedef struct swab_decode_desc {
    swab_cache_desc cache;
    int32_t tokens;       /* rows of Q, O, lse, >= 1 */
    int32_t h, hk;        /* query heads, key heads (h a multiple of hk): query head q reads key
                             head q / (h / hk); h / hk at most 128 */
    int32_t head_dim;     /* a multiple of 16 bytes, at most 256 */
    int32_t w;            /* keys on the left, 0..2^30 (at least the longest context: all of them) */
    int32_t dilation;     /* 0..SWAB_MAX_DILATION; key stride dilation + 1 */
    int32_t n_sink;       /* leading positions every later query attends to, >= 0 */
    int32_t max_q;        /* most new tokens of a request, >= 1 */
    int32_t max_len;      /* longest context, >= 1 (divides the work; longer ones stay right) */
    int32_t prefix_len;   /* positions of the shared prefix, 0: none; at most n_blocks * page */
    int32_t dtype;        /* swab_dtype of Q, K, V, O */
    int64_t q_row_stride; /* elements between rows of Q, 0 = h * head_dim; multiple of 16 bytes */
    int64_t out_row_stride; /* the same of O */
} swab_decode_desc;

/* Bytes of workspace band_decode needs (0 if it needs none, or desc is bad). */
SWAB_API size_t band_decode_workspace(const swab_decode_desc *desc);

/* Banded attention of the new tokens over the cache.  Request r holds lens[r]
 * positions, its m = q_start[r + 1] - q_start[r] new tokens among them (the
 * last ones), so row q_start[r] + a is the query at position
 * i = lens[r] - m + a and attends to
 *     the positions j = i - k * (dilation + 1), 0 <= k <= w, j >= n_sink,
 *     the positions j < n_sink, j <= i,
 *     with prefix_len > 0 also every position of the shared prefix,
 * each once:  O = softmax(scale * q . K) . V,  lse = log of its sum of
 * exponentials ([tokens, h] fp32, may be NULL).  A query without a key (an
 * inconsistent length, absent blocks) gets O = 0 and lse = -inf, one with a NaN
 * score NaN in both; scores that are all -inf count as no key.  Without ring,
 * positions past the table (lens[r] > cols * page) count as absent and raise
 * SWAB_ERR_INVALID_ARG in the status word.  Rows of O
 * and lse that belong to no request are left as they were.
 * The shared prefix lies in the same cache: positions p of it in block
 * prefix_table[p / page] ([ceil(prefix_len / page)], DEVICE int32); it comes
 * before position 0 of every request.  For fp16 / bf16 with head_dim 64 or 128
 * it is read from memory once for all of them; with other types and head sizes
 * it is a part of every request's key list, read again for each request and
 * every four heads.  It stays visible whatever the window, like the global
 * tokens of the banded calls.
 * Scores, sums, lse and the parts of a cut list are fp32.  With fp16 / bf16 and
 * head_dim 64 or 128 the products run on the tensor cores: a weight, at most 2^8
 * relative to the running reference, is rounded to dtype before it multiplies
 * V (its sum is not); elsewhere weights are fp32.
 * With ring, the recycled columns must hold a step's window:
 * w * (dilation + 1) + max_q <= (cols - pinned - 1) * page + 1, and the pinned
 * ones the sinks: n_sink <= pinned * page (else SWAB_ERR_INVALID_ARG).
 * Every key and value that some query of the same request attends to has to
 * be finite; the others are never used, whatever they hold.
 * cache.max_new is not used.
 * workspace: band_decode_workspace(desc) bytes of device memory, 16-byte
 * aligned (NULL if 0); its contents on entry do not matter, and calls that may
 * overlap on the GPU need one each.  The call launches up to three kernels.
 * They, like those of the rotary and cache calls, are programmatic dependents:
 * set up while the kernel before them runs, they wait inside for what it
 * writes; for the caller a call stays ordered on the stream like any kernel
 * launch.  Results do not depend on timing (no atomics). */
SWAB_API swab_status band_decode(const swab_decode_desc *desc, float scale, const void *Q,
                                 const void *Kc, const void *Vc, const int32_t *table,
                                 const int32_t *lens, const int32_t *q_start,
                                 const int32_t *prefix_table, void *O, float *lse, void *workspace,
                                 void *stream);

/* Bytes of workspace band_decode4 needs (0 if it needs none, or desc is bad). */
SWAB_API size_t band_decode4_workspace(const swab_decode_desc *desc);

/* band_decode over a cache in 4 bits: the same key set, results, rows left alone,
 * handling of absent blocks, limits, workspace rules and launches, with K and V the
 * values of the codes Kc, Vc under the scales Ks, Vs.  head_dim a multiple of 32, at
 * most 256; no shared prefix (prefix_len must be 0), else SWAB_ERR_UNSUPPORTED.  The
 * values are exact in fp16 and bf16, so with head_dim 64, 128 or (without a dilation)
 * 96 the products run on the tensor cores as those of band_decode do (a weight, at
 * most 2^8 relative to the running reference, is rounded to dtype before it
 * multiplies V); elsewhere in fp32. */
SWAB_API swab_status band_decode4(const swab_decode_desc *desc, float scale, const void *Q,
                                  const void *Kc, const void *Ks, const void *Vc, const void *Vs,
                                  const int32_t *table, const int32_t *lens, const int32_t *q_start,
                                  void *O, float *lse, void *workspace, void *stream);

/* Human-readable name of a status code (static string). */
SWAB_API const char *swab_status_string(swab_status status);

/* Reads (and, if reset != 0, clears) the library's device status word on the
 * current device: bit k set means SWAB status k was raised by a kernel.
 * Synchronises the device.  Returns SWAB_ERR_CUDA if the read fails. */
SWAB_API swab_status swab_device_status(int32_t *flags, int32_t reset);

/* Failure-detection self-test: launches one warp that waits on an mbarrier no
 * thread ever arrives at, using the same bounded wait as every pipelined
 * kernel, with a limit of `limit_us` microseconds (1..1000000).  The wait gives
 * up, records SWAB_ERR_TIMEOUT in the device status word and the kernel
 * returns; nothing faults or hangs and the context stays usable.  Read the
 * result with swab_device_status().  No counterpart on the pages: it tests
 * the library's own error reporting. */
SWAB_API swab_status swab_selftest_wait_timeout(uint32_t limit_us, void *stream);

/* ---------------------------------------------------------------------------
 * Bounds-checked build.  The library also builds as libswab_bounds.so with
 * SWAB_BOUNDS_CHECK=1: the same kernels, in which every plain global load,
 * store and reduction first tests the bytes it touches against the extents of
 * the call's buffers.  The host derives those extents from the descriptor and
 * the documented shapes (dense [b, h, n, hd] or rows of [b, n, row_stride];
 * band [b*h, n, D]; companions, lse, key bias, keep-bit cache and workspace by
 * their sizes above), plus the library's own device arrays.  An access outside
 * all of them is not made (a store is dropped, a load reads a scratch line):
 * the kernel raises SWAB_ERR_BOUNDS in the device status word, records the
 * first such access (swab_bounds_report) and runs on.  TMA copies are clipped
 * by the hardware to their tensor map; the host checks each map's footprint
 * against the same extents before launching and returns SWAB_ERR_BOUNDS (no
 * launch) if one overhangs.  No counterpart on the pages: it stands in for a
 * memory checker where none can run.  The checked build is slower; its
 * results are the regular build's, bit for bit.
 * ------------------------------------------------------------------------- */

/* 1 in the bounds-checked build, 0 in the regular one. */
SWAB_API int32_t swab_bounds_checked(void);

/* First out-of-bounds access recorded on the current device since the last
 * reset: out[0] = source site (file id << 16 | line) + 1, 0 if none;
 * out[1] = its address; out[2] = its size in bytes.  Synchronises the device;
 * reset != 0 clears the record.  Always zero in the regular build. */
SWAB_API swab_status swab_bounds_report(uint64_t *out, int32_t reset);

/* Self-test of the bounds checks (checked build only, SWAB_ERR_UNSUPPORTED
 * otherwise): one warp stores through the check into a library-owned device
 * array of 128 floats with an extent table that covers only its first 64.
 * Lane l stores to element l (inside the extent) and to element 64 + l
 * (valid memory outside it).  Synchronises `stream`; returns SWAB_OK when the
 * stores inside landed and the ones outside did not (else SWAB_ERR_BOUNDS).
 * The refused stores also raise SWAB_ERR_BOUNDS in the device status word and
 * are recorded (swab_bounds_report).  Nothing outside the array is ever
 * addressed. */
SWAB_API swab_status swab_selftest_bounds(void *stream);

/* Library version, e.g. "0.1.0". */
SWAB_API const char *swab_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SWAB_H */
