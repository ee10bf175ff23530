/*
 * gdn.h - C ABI of the MI355X (gfx950) gated delta rule library, libgdn.so.
 *
 * What is computed. Per batch b and head h the library carries an fp32 state
 * h in R^{dk x dv} through the gated delta rule
 *
 *     alpha_t = exp(g_t * A),  A = -exp(A_log[h])
 *     h_t     = alpha_t (h_{t-1} - beta_t k_t (k_t^T h_{t-1})) + beta_t k_t v_t^T
 *     o_t     = h_t^T q_t
 *
 * The recurrence is the one of "GDN & MLA Mechanism Deep-Dive" (Intuition and
 * Math derivation, Step 4: per-head decay alpha_t = exp(g_t A) in (0,1), A kept
 * in log space as A_log, read o_t after the write) and of "HyMo-434M
 * documentation portal" (FIG. A0 probe and 01 GDN RECURRENCE: the delta rule
 * with gate beta_t), whose erase term is read with the key k_t. With
 * GDN_FLAG_ADDITIVE the erase term is off and the write/read pair of Step 4
 * remains: h_t = alpha_t h_{t-1} + beta_t k_t v_t^T. The forward runs the
 * chunked algorithm of Step 5 (chunk of 64 tokens solved in closed form with
 * 64 x 64 matrices, state carried serially between chunks); results equal the
 * serial definition above up to floating-point rounding.
 *
 * Layouts (all contiguous, row-major, no padding in memory):
 *   q, k, dq, dk        [B, T, H, dk]   dtype of the call (fp32 or bf16)
 *   v, o, do, dv        [B, T, H, dv]   dtype of the call
 *   g, beta, dg, dbeta  [B, T, H]       fp32; g and beta are the values the
 *                                       recurrence uses (post-sigmoid gate,
 *                                       no sigmoid is applied here)
 *   A_log, dA_log       [H]             fp32
 *   h0, hT, dhT, dh0    [B, H, dk, dv]  fp32 (row i = key index)
 *   decode (gdn_step):  q,k [N,H,dk], v,o [N,H,dv], g,beta [N,H],
 *                       states [N,H,dk,dv]; gdn_step_tokens: [N,S,H,*]
 *   D, dD               [H]             fp32 (skip term, optional)
 * bf16 outputs are rounded to nearest even. The library applies no scaling
 * to q; k is used as given unless GDN_FLAG_L2NORM_K asks for its per-token
 * normalisation.
 *
 * Layer edges. Two steps that sit on either side of the recurrence in the
 * GDN layer are fused into the kernels when asked for: the per-token L2
 * normalisation of the keys (GDN_FLAG_L2NORM_K) and the per-head skip term
 * o_t += D[h] v_t (a non-NULL D argument; "HyMo-434M documentation portal",
 * Architecture: the recurrence carries A_log, dt_bias and D). Both default
 * to off, which gives the recurrence above unchanged.
 *
 * Ownership. The caller allocates every buffer, including the workspaces
 * sized by the *_workspace_size queries; the library never allocates, frees
 * or synchronises. All device pointers are HIP device memory; `stream` is a
 * hipStream_t (NULL = the default stream). Work is enqueued on that stream and
 * the call returns without waiting for it.
 *
 * Errors. Argument checks run before anything is enqueued; a failing call
 * writes nothing and returns GDN_EINVAL / GDN_EUNSUPPORTED / GDN_EWORKSPACE.
 * A failed launch returns GDN_EHIP. Faults inside kernels surface at the
 * caller's next synchronisation. gdn_last_error_detail() gives a text for the
 * last non-OK status of the calling thread. NaN/Inf inputs propagate.
 * Results are bitwise reproducible for a given build, shape and device.
 *
 * Supported sizes: T >= 0 (a last chunk shorter than 64 is handled on chip),
 * 1 <= dk, dv <= 128 for bf16 and <= 64 for fp32, chunk 0 or 64, base
 * pointers 16-byte aligned, B*H < 2^31, tensors below 2^31 elements.
 *
 * Empty sequences (T = 0) run no step: gdn_fwd sets hT = h0 (zeros when h0
 * is NULL); gdn_bwd sets dh0 = dhT (zeros when dhT is NULL), dA_log = 0,
 * dD = 0 when given and, when asked, hT = h0. Pointers to arrays with a factor T in their extent may
 * then be NULL, and no workspace or context is used.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_EINVAL = 1,       /* bad argument (size, null pointer, alignment, aliasing) */
    GDN_EUNSUPPORTED = 2, /* valid request the library does not implement */
    GDN_EWORKSPACE = 3,   /* workspace pointer NULL or smaller than required */
    GDN_EHIP = 4          /* a HIP runtime call or kernel launch failed */
} gdn_status_t;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype_t;

/* Erase term off: h_t = alpha_t h_{t-1} + beta_t k_t v_t^T ("GDN & MLA
 * Mechanism Deep-Dive", Step 4 write line, write key b_t = beta_t k_t). */
#define GDN_FLAG_ADDITIVE 1u

/* g and beta are given as logits: the library applies the logistic sigmoid
 * on load (g = sigmoid(dt_proj(x)) in "GDN & MLA Mechanism Deep-Dive", Step 4;
 * the write gate beta likewise), and gdn_bwd returns dg and dbeta with
 * respect to the logits. dA_log is unchanged (it is taken through the gate
 * values). Without the flag g and beta are the gate values themselves. */
#define GDN_FLAG_GATE_LOGITS 2u

/* Keys are L2-normalised per token where the kernels load them: the
 * recurrence runs on k_hat = k / sqrt(sum_j k_j^2 + 1e-6), the unit-length
 * erase/write key of "GDN & MLA Mechanism Deep-Dive", Step 3 and Step 4 (the
 * epsilon under the root keeps a zero key finite). gdn_bwd then returns dk
 * with respect to the raw keys, dk = (dk_hat - k_hat (k_hat . dk_hat)) /
 * sqrt(sum_j k_j^2 + 1e-6). The raw keys are what the caller passes and
 * keeps; nothing normalised is written back. */
#define GDN_FLAG_L2NORM_K 4u

typedef struct {
    int32_t B, T, H; /* batch, tokens, heads */
    int32_t dk, dv;  /* key and value head dimensions */
    int32_t dtype;   /* gdn_dtype_t of q, k, v, o, do, dq, dk, dv */
    int32_t chunk;   /* 0 or 64 */
    uint32_t flags;  /* GDN_FLAG_ADDITIVE | GDN_FLAG_GATE_LOGITS | GDN_FLAG_L2NORM_K, or 0 */
} gdn_shape_t;

/* Bytes of device workspace gdn_fwd / gdn_bwd need for this shape. Return 0
 * for an invalid shape; the call itself then reports the error. */
size_t gdn_fwd_workspace_size(const gdn_shape_t *s);
size_t gdn_bwd_workspace_size(const gdn_shape_t *s);

/* Bytes of the optional forward context: what gdn_fwd can save for gdn_bwd
 * so that the backward skips recomputing the forward. It holds, in the
 * call's dtype, the state at the start of every 64-token chunk and the
 * chunk's -Tm diag(beta e^gam) K, Tm diag(beta) V and Tm = (I + L)^{-1}
 * blocks. Its layout is private to the library. */
size_t gdn_fwd_context_size(const gdn_shape_t *s);

/* Forward pass over a whole sequence ("GDN & MLA Mechanism Deep-Dive",
 * Step 4 and Step 5).
 *   q, k, v, g, beta, A_log  inputs (layouts above)
 *   D             [H] skip weights (o_t += D[h] v_t) or NULL (no skip term)
 *   h0            initial state or NULL (zero state)
 *   o             output [B,T,H,dv], or NULL: a state-only pass (e.g. the
 *                 prefill of a decode state), which writes hT and/or ctx
 *                 and skips the outputs
 *   hT            final state or NULL (not written)
 *   ctx           NULL, or gdn_fwd_context_size() bytes (256-byte aligned)
 *                 that receive the forward context for gdn_bwd
 *   ws, ws_bytes  workspace of gdn_fwd_workspace_size() bytes, 256-byte
 *                 aligned; its contents are scratch */
gdn_status_t gdn_fwd(const gdn_shape_t *s, const void *q, const void *k, const void *v,
                     const float *g, const float *beta, const float *A_log, const float *D,
                     const float *h0, void *o, float *hT, void *ctx, void *ws, size_t ws_bytes,
                     void *stream);

/* Bytes of the static device scratch gdn_fwd_noalloc uses as its workspace
 * (64 MiB per GPU, held until the process ends). */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)

/* gdn_fwd without a workspace argument and without any device allocation,
 * for callers that cannot allocate (code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation). Same computation,
 * arguments and results as gdn_fwd (bit for bit), with every launch on
 * `stream`. The workspace is a static device array of
 * GDN_NOALLOC_SCRATCH_BYTES in the library, one per GPU, shared by every
 * call on that GPU: calls that overlap in time on one GPU race and must be
 * ordered by the caller (e.g. issued on one stream). Shapes whose
 * gdn_fwd_workspace_size() exceeds GDN_NOALLOC_SCRATCH_BYTES are rejected
 * with GDN_EWORKSPACE before anything is enqueued (at d = 56 in bf16 the
 * scratch holds about 290,000 token-heads, e.g. B*T = 18,000 at H = 16). */
gdn_status_t gdn_fwd_noalloc(const gdn_shape_t *s, const void *q, const void *k, const void *v,
                             const float *g, const float *beta, const float *A_log, const float *D,
                             const float *h0, void *o, float *hT, void *ctx, void *stream);

/* Backward pass: gradients of sum(do * o) + sum(dhT * hT) with respect to q,
 * k, v, g, beta, A_log, D and h0, by the reverse-chunk derivative of the
 * chunked forward. Inputs are those of the gdn_fwd call (same flags, same D);
 * do is the upstream gradient of o, dhT that of the final state (NULL = zero).
 *   ctx           NULL (the forward is recomputed in the workspace) or the
 *                 context gdn_fwd saved for the same inputs
 *   dq, dk, dv    [B,T,H,*] in the call's dtype
 *   dg, dbeta     [B,T,H] fp32
 *   dA_log        [H] fp32, overwritten (sum over the batch)
 *   dD            [H] fp32 or NULL: overwritten with the sum over batch,
 *                 tokens and value columns of do * v, the gradient of the
 *                 skip weights (also when D is NULL: the gradient at D = 0)
 *   dh0           [B,H,dk,dv] fp32 or NULL
 *   hT            NULL, or receives the recomputed final state; only allowed
 *                 when ctx is NULL
 *   ws, ws_bytes  workspace of gdn_bwd_workspace_size() bytes, 256-byte
 *                 aligned
 * Supported head dimensions: those of gdn_fwd (bf16 up to 128, fp32 up to
 * 64). The local gradients of heads wider than 64 (bf16) or 16 (fp32) run in
 * a kernel that keeps its intermediates in the workspace; the workspace size
 * query includes that scratch. */
gdn_status_t gdn_bwd(const gdn_shape_t *s, const void *q, const void *k, const void *v,
                     const float *g, const float *beta, const float *A_log, const float *D,
                     const float *h0, const void *ctx, const void *dout, const float *dhT,
                     void *dq, void *dk, void *dv, float *dg, float *dbeta, float *dA_log,
                     float *dD, float *dh0, float *hT, void *ws, size_t ws_bytes, void *stream);

/* One decode token for each of N independent sequences: one step of the
 * recurrence from a carried state (the O(1)-state read/write of "GDN & MLA
 * Mechanism Deep-Dive", Intuition). h_in may be NULL (zero state) and may
 * equal h_out (in-place update); no other aliasing is allowed. `dtype` is the
 * gdn_dtype_t of q, k, v and o; `flags` is any of GDN_FLAG_ADDITIVE,
 * GDN_FLAG_GATE_LOGITS and GDN_FLAG_L2NORM_K, or 0; D is the [H] skip
 * weights or NULL, as in gdn_fwd. */
gdn_status_t gdn_step(int32_t N, int32_t H, int32_t dk, int32_t dv, int32_t dtype, uint32_t flags,
                      const void *q, const void *k, const void *v, const float *g,
                      const float *beta, const float *A_log, const float *D, const float *h_in,
                      float *h_out, void *o, void *stream);

/* S consecutive decode tokens for each of N independent sequences from a
 * carried state: the recurrence applied token after token (the serial
 * definition of "GDN & MLA Mechanism Deep-Dive", Step 4), as when the draft
 * tokens of a multi-token prediction are verified ("HyMo-434M documentation
 * portal", 04 MTP SPECULATION: a depth-2 draft, three tokens accepted per
 * step). q, k are
 * [N,S,H,dk], v, o [N,S,H,dv], g, beta [N,S,H] (the forward's layouts with
 * B = N, T = S); the states are [N,H,dk,dv]. The state is read once and
 * written once per call (heads up to 64 wide keep it on chip between the
 * tokens). For draft verification, call out of place: h_in then stays the
 * state to roll back to, and if only the first j tokens are accepted, a call
 * over those j tokens from h_in gives the state to keep.
 * h_in may be NULL (zero state) or equal h_out. S = 0 carries the
 * state over unchanged (h_out = h_in, zeros when h_in is NULL; the token
 * arrays may be NULL); N = 0 does nothing. gdn_step is this call with S = 1
 * and the [N,H,*] layouts. */
gdn_status_t gdn_step_tokens(int32_t N, int32_t S, int32_t H, int32_t dk, int32_t dv, int32_t dtype,
                             uint32_t flags, const void *q, const void *k, const void *v,
                             const float *g, const float *beta, const float *A_log, const float *D,
                             const float *h_in, float *h_out, void *o, void *stream);

/* ---------------------------------------------------------------------------
 * Latent attention and its paged cache: the softmax-attention layers that sit
 * between GDN layers in the hybrid stack ("HyMo-434M documentation portal",
 * MLA: one latent and one rotary key a token, shared by the heads). The
 * projections are the caller's. Two forms:
 *
 *   expanded (gdn_mla_fwd, gdn_mla_bwd; training and prompts): every head has
 *   keys k and values v made from the latent, and a rotary key k_rope that
 *   heads share;
 *   absorbed (gdn_mla_step; new tokens): the key and value maps are folded
 *   into q and the output projection, so every head attends to the cached
 *   rows [latent | rotary key] themselves.
 *
 * The rules at the top of this file hold (ownership, streams, errors, no
 * allocation, bitwise reproducible results). Tensors are contiguous; q, k, v,
 * o, c, x, cache and their gradients are fp32 or bf16 as the call's dtype
 * says, sums and softmax statistics fp32. fp32 calls round nothing below that.
 * bf16 calls round, besides their outputs, what the next matrix product takes:
 * the probabilities (for o and dv) and dS = P (dP - delta) (for dq, dk and
 * dk_rope), to nearest even; and delta = dout . o uses the bf16 o it is given,
 * except in rows that see at most 256 keys, where it is formed anew in fp32.
 * A caller who needs less rounding calls with fp32 tensors. Rows at or past a
 * length, and cache rows no table entry in use names, are not read. NaN/Inf in
 * rows that take part propagate, and as 0 * NaN within a tile also to masked
 * neighbours: from a key or value row to o and dq of queries up to 160
 * positions before it, from a row of q or dout to dk, dk_rope and dv of keys up
 * to 160 positions after it, from a cache row to all S tokens of a
 * gdn_mla_step.
 */

/* q [B,Tq,H,dn+dr], k [B,Tk,Hk,dn], k_rope [B,Tk,Hr,dr], v [B,Tk,Hk,dv],
 * o [B,Tq,H,dv], lse [B,Tq,H] fp32. Head h uses key head h / (H / Hk) and
 * rotary head h / (H / Hr); Hk divides H and Hr divides Hk. dr = 0: no rotary
 * part (k_rope may be NULL, Hr is not read). dn, dv: multiples of 8 up to
 * 128; dr: one up to 64 (GDN_EUNSUPPORTED else). scale > 0. Tk >= Tq: the
 * queries are the last Tq of the Tk positions (a chunk after cached ones).
 * Every tensor has fewer than 2^31 elements. */
typedef struct {
    int32_t B, Tq, Tk, H, Hk, Hr, dn, dr, dv, dtype;
    float scale;
} gdn_mla_shape_t;

/* Causal attention, forward: query i of sequence b sees the keys
 * j <= i + Tk - Tq with j < lens[b] (lens NULL: Tk; values outside [0, Tk]
 * are clamped).
 *   z_ij = scale (q_i[:dn] . k_j + q_i[dn:] . k_rope_j)
 *   o_i = sum_j softmax(z_i)_j v_j,  lse_i = log sum_j exp z_ij
 * A query at a position >= lens[b] (padding) gets o = 0 and lse = -inf.
 * lse may be NULL; gdn_mla_bwd needs it. Tq = 0 does nothing. */
gdn_status_t gdn_mla_fwd(const gdn_mla_shape_t *s, const void *q, const void *k, const void *k_rope, const void *v,
                         const int32_t *lens, void *o, float *lse, void *stream);

/* Its backward: the gradients of sum(do * o) with respect to q, k, k_rope and
 * v, summed over the heads that share a row; zero for padding. o and lse are
 * the forward's. ws: gdn_mla_bwd_workspace_size() bytes, 256-byte aligned. */
size_t gdn_mla_bwd_workspace_size(const gdn_mla_shape_t *s);
gdn_status_t gdn_mla_bwd(const gdn_mla_shape_t *s, const void *q, const void *k, const void *k_rope, const void *v,
                         const int32_t *lens, const void *o, const float *lse, const void *dout, void *dq, void *dk,
                         void *dk_rope, void *dv, void *ws, size_t ws_bytes, void *stream);

/* q [N,S,H,dl+dr], cache [pages,page_size,dl+dr], block_table [N,max_pages]
 * int32 (page of each page_size tokens of a sequence), lens [N] int32 (cached
 * tokens, the S new ones included), o [N,S,H,dl], lse [N,S,H] fp32. dl: a
 * multiple of 16 up to 512; dr: one of 8 up to 64. pages * page_size and
 * N * max_pages stay below 2^31, max_pages * page_size is at most 2^31 - 2048
 * (the cache itself may be larger than 2^32 bytes). */
typedef struct {
    int32_t N, S, H, dl, dr, dtype, pages, page_size, max_pages;
    float scale;
} gdn_mla_step_shape_t;

/* S new tokens for each of N sequences against their cached rows (which hold
 * the new tokens' rows already, see gdn_mla_write): token s sees the rows
 * j <= lens[n] - S + s.
 *   z_j = scale q . row_j,  o = sum_j softmax(z)_j row_j[:dl],  lse = log sum_j exp z_j
 * A token that sees no row gets o = 0 and lse = -inf. lens is clamped to
 * [0, max_pages * page_size]; a table entry outside [0, pages) masks its
 * rows. lse may be NULL. N = 0 or S = 0 does nothing. ws:
 * gdn_mla_step_workspace_size() bytes, 256-byte aligned (it depends on the
 * shape alone, not on the lengths). */
size_t gdn_mla_step_workspace_size(const gdn_mla_step_shape_t *s);
gdn_status_t gdn_mla_step(const gdn_mla_step_shape_t *s, const void *q, const void *cache, const int32_t *block_table,
                          const int32_t *lens, void *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/* Flags of gdn_norm_rope, gdn_norm_rope_bwd and gdn_mla_write. */
#define GDN_ROPE_NORM 1u        /* RMS norm of every row (times w, when given) */
#define GDN_ROPE_INTERLEAVED 2u /* pairs (2i, 2i + 1) instead of (i, i + r/2) */

/* Norm and position rotation of every head's row in one pass, x, y [M,H,d]:
 *   z = x / sqrt(mean(x^2) + eps) * w  (GDN_ROPE_NORM; w [d] fp32 or NULL = 1)
 *   y = z with its last r columns turned pairwise, (a, b) ->
 *       (a cos t - b sin t, b cos t + a sin t), t = positions[m] * freqs[i]
 * positions [M] int32, freqs [r/2] fp64 (the angle is formed in fp64); both
 * may be NULL with r = 0. 1 <= d <= 512, r even, 0 <= r <= d. y may be x. */
gdn_status_t gdn_norm_rope(int64_t M, int32_t H, int32_t d, int32_t r, int32_t dtype, uint32_t flags, float eps,
                           const void *x, const float *w, const int32_t *positions, const double *freqs, void *y,
                           void *stream);

/* Its backward: dx, and dw [d] fp32 (NULL: not wanted; overwritten). x may be
 * NULL without GDN_ROPE_NORM. ws: gdn_norm_rope_bwd_workspace_size() bytes,
 * 256-byte aligned, needed with dw. */
size_t gdn_norm_rope_bwd_workspace_size(int64_t M, int32_t H, int32_t d);
gdn_status_t gdn_norm_rope_bwd(int64_t M, int32_t H, int32_t d, int32_t r, int32_t dtype, uint32_t flags, float eps,
                               const void *dy, const void *x, const float *w, const int32_t *positions,
                               const double *freqs, void *dx, float *dw, void *ws, size_t ws_bytes, void *stream);

/* Rows of n new tokens into the paged cache [n_slots,dl+dr]: row slots[i] =
 * [norm(c_i) | turned k_rope_i], norm as above with GDN_ROPE_NORM (w [dl] fp32
 * or NULL), the turn by positions[i] * freqs (freqs NULL: k_rope as it is).
 * c [n,dl], k_rope [n,dr]. Slots outside [0, n_slots) are skipped; slots have
 * to differ from each other (a row named twice holds a mixture). Rows no slot
 * names stay as they are. dl: a multiple of 8 up to 512; dr: one up to 64. */
gdn_status_t gdn_mla_write(int64_t n, int32_t dl, int32_t dr, int32_t dtype, uint32_t flags, float eps, const void *c,
                           const void *k_rope, const float *w, const int32_t *positions, const double *freqs,
                           const int32_t *slots, void *cache, int64_t n_slots, void *stream);

/* Pages, slots and positions of the next step's tokens, on the GPU. Each of N
 * sequences holds lens[i] cached tokens in the pages of its block_table row
 * and asks for new_lens[i] more; new_lens[i] < 0 ends it: its pages go back on
 * the stack of free pages (free_pages [n_pages], n_free of them, the last one
 * on top) before any are taken, and its length becomes 0.
 * In order, a sequence is granted what it asks for when its table row has
 * room, the tokens asked for so far (by sequences with room) are at most
 * max_tokens, and the pages asked for so far are at most those free (or it
 * needs no new page); else it is granted nothing and stays as it is. New pages
 * are popped from the stack's top into the sequence's row.
 *   granted [N]        new tokens granted
 *   starts [N+1]       their prefix sums: where a sequence's new tokens begin
 *   slots [max_tokens] page * page_size + offset of every new token; -1 past
 *                      the last one
 *   positions [max_tokens]  its position in its sequence; 0 past the last one
 *   lens_out [N]       lengths afterwards (may be lens)
 *   n_free_out [1]     free pages afterwards (may be n_free)
 * block_table and free_pages are updated in place; with separate lens_out and
 * n_free_out the same call again gives the same result. All int32;
 * N * max_pages is at most 2^31 - 2048. */
gdn_status_t gdn_page_plan(int32_t N, int32_t max_pages, int32_t n_pages, int32_t page_size, int32_t max_tokens,
                           const int32_t *lens, const int32_t *new_lens, int32_t *block_table, int32_t *free_pages,
                           const int32_t *n_free, int32_t *lens_out, int32_t *n_free_out, int32_t *granted,
                           int32_t *starts, int32_t *slots, int32_t *positions, void *stream);

/* Timing aid for benchmarks (no effect on results). While `events` is
 * non-NULL, every kernel the library launches from this thread is bracketed
 * by hipEventRecord calls on the launch's stream: events[2i] before launch i
 * and events[2i+1] after it, for the first n/2 launches counted from this
 * call (later launches are not bracketed). `events` points to n hipEvent_t
 * handles owned by the caller; NULL switches the aid off. Returns the number
 * of launches bracketed since the previous call. */
int32_t gdn_time_launches(void *const *events, int32_t n);

/* Which kernel the i-th bracketed launch of the current (or, once switched
 * off, the last) bracketing period was: 0 forward prep, 1 forward serial
 * pass, 2 backward serial pass, 3 backward local gradients, 4 dA_log (or
 * dD) reduction, 5 decode step, 6 forward scan over chunk ranges, 7 backward
 * scan, 8 attention forward, 9 and 10 attention backward (query gradients;
 * key and value gradients), 11 sum of the shared rotary key's gradient, 12
 * attention against the paged cache, 13 join of its parts, 14 norm and
 * rotation, 15 their backward, 16 sum of the norm weight's gradient, 17 cache
 * write, 18 page plan, 19 slots of a page plan; -1 when i is out of range. A
 * forward call may launch its two kernels several times each, over
 * consecutive chunk ranges (prep of the next range runs on a second stream
 * while the serial pass works on the current one), and a serial pass run as a
 * parallel scan launches twice (the ranges' maps, then every range from its
 * start). */
int32_t gdn_launch_kind(int32_t i);

const char *gdn_status_string(gdn_status_t st);
const char *gdn_last_error_detail(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
