/*
 * gdn.h -- C ABI of the gated delta-rule layer on AMD Instinct MI355X (gfx950).
 *
 * The layer (gated-deltanet card, "Method"; per-key-channel decay as in GDN-2,
 * Marin note "Background") keeps a state S [Dk x Dv] per (batch, head) and,
 * for each token t, applies
 *     S <- diag(exp(g_t)) S;  m = S^T k_t;  d = beta_t (v_t - m);
 *     S <- S + k_t d^T;       o_t = scale * S^T q_t.
 * g_t is one log-decay per key channel (GDN_DECAY_PER_CHANNEL) or one scalar
 * per head broadcast over the channels (GDN_DECAY_PER_HEAD).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers are DEVICE pointers (hipMalloc'd or from a torch tensor), dense,
 * row-major, 16-byte aligned.  The caller owns every buffer; the library keeps
 * no allocation between calls and allocates nothing itself.  All work is
 * enqueued on `stream` (a hipStream_t; NULL = the null stream) with no host
 * synchronisation, so asynchronous faults surface at the caller's next sync.
 *
 * Tensor layouts (element types in brackets):
 *   q, k      [B, T, H, Dk]         (dtype: float32 or bf16)
 *   v, o, dO  [B, T, H, Dv]         (dtype)
 *   g         [B, T, H, Dk] per channel, or [B, T, H] per head   (float32)
 *   beta      [B, T, H]                                          (float32)
 *   states    h0, hT, dhT, dh0, decode state: [B, H, Dk, Dv]     (float32)
 *   dq, dk    [B, T, H, Dk] (dtype);  dv [B, T, H, Dv] (dtype)
 *   dg        like g (float32);  dbeta [B, T, H] (float32)
 * Grouped-query repetition of q/k heads is the caller's (gated-deltanet card,
 * "Requirements and limits").  q and k are used as given unless the shape's
 * qk_l2norm is set (the card's use_qk_l2norm, "Usage"): then every q and k row
 * (the Dk values of one token and head) is replaced inside the call by
 * x / sqrt(sum(x^2) + GDN_L2NORM_EPS) before the recurrence, and dq, dk are the
 * gradients with respect to the raw, unnormalised rows,
 * dx = r (dx_hat - x_hat (x_hat . dx_hat)) with r = 1 / sqrt(sum(x^2) + eps).
 * The card names the option but not its guard; 1e-6 inside the root is the
 * reading taken here.
 *
 * Errors: every call returns a status.  Bad shapes, NULL required pointers,
 * misaligned pointers and a too-small workspace are rejected before anything
 * is launched.  An unsupported (chunk, Dk, Dv) combination returns
 * GDN_ERR_UNSUPPORTED; there is no fallback path.  A failed launch returns
 * GDN_ERR_HIP.  Results are deterministic: repeated calls with the same inputs
 * are bitwise identical (gated-deltanet card, "Correctness").
 *
 * Supported sizes: chunked calls Dk = Dv in {64, 128} with chunk 64 (the
 * default) and Dk = Dv = 16 with chunk 16; decode Dk = Dv in {16, 32, 64, 128};
 * any T >= 0 (a ragged last chunk is processed as if padded with tokens that
 * have g = 0 and beta = 0, which leave the state exactly unchanged; their
 * outputs are not written); B, H >= 1, and for chunked calls
 * H * max(Dk, Dv) * chunk <= 2^28 (H <= 32768 at 128 x 128) and
 * B * H * ceil(T / chunk) * chunk < 2^27 (the token-heads of one call, the last
 * chunk counted whole; the largest launch has 32 work-items per token-head).
 * Anything else: GDN_ERR_UNSUPPORTED, before any launch.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,
    GDN_ERR_UNSUPPORTED = 2,
    GDN_ERR_ALIGNMENT = 3,
    GDN_ERR_WORKSPACE = 4,
    GDN_ERR_HIP = 5
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;
typedef enum { GDN_DECAY_PER_HEAD = 0, GDN_DECAY_PER_CHANNEL = 1 } gdn_decay;

#define GDN_L2NORM_EPS 1e-6f

/* Stage boundaries of the chunked forward that the numerical-safety options act
 * on (atomic_ops card, "Features": chunk scores -> WY block solve -> recompute
 * -> inter-chunk scan): the scores P (unscaled) and A (with beta), the solve's
 * T, the recompute's U and W, the outputs o and the final state hT. */
enum {
    GDN_DIAG_P = 0,
    GDN_DIAG_A = 1,
    GDN_DIAG_T = 2,
    GDN_DIAG_U = 3,
    GDN_DIAG_W = 4,
    GDN_DIAG_O = 5,
    GDN_DIAG_HT = 6,
    GDN_DIAG_STAGES = 7
};
/* counters: word 2*stage counts non-finite values, word 2*stage+1 finite
 * values with |x| > 1e6 */
#define GDN_DIAG_WORDS (2 * GDN_DIAG_STAGES)

typedef struct {
    int B, T, H, Dk, Dv;
    int dtype;     /* gdn_dtype of q, k, v, o, dO, dq, dk, dv */
    int decay;     /* gdn_decay */
    float scale;   /* output scale; 0 means Dk^-0.5 (the atomic_ops card passes d^-0.5) */
    int chunk;     /* chunk length C of the chunked form: 16 or 64; 0 means 64 */
    int qk_l2norm; /* 1: L2-normalise q and k rows inside the call (see above); 0: as given.
                      A training pair (gdn_forward_train, gdn_backward_train) must pass the
                      same value to both calls. */
    /* Numerical-safety options of the chunked calls (atomic_ops card, "Features"
     * and "Debugging"); all zero = off.  Not supported by gdn_decode_step.  A
     * training pair must pass the same values to both calls. */
    float wy_eps;  /* >= 0: the WY block solve inverts (1 + wy_eps) I + A instead of
                      I + A (damping on the diagonal); results then depend on the chunk */
    float clip;    /* >= 0; > 0: at each stage boundary (GDN_DIAG_*) values are made
                      finite (NaN -> 0, +-inf -> +-clip) and clamped to [-clip, clip],
                      and so are dq, dk, dv, dg, dbeta, dh0; gradients take the clipping
                      as the identity */
    int diag;      /* 1: the forward counts, per stage boundary and before clipping,
                      non-finite values and finite values with |x| > 1e6 into counters
                      in the workspace (read with gdn_diag_read); never changes values */
} gdn_shape;

/*
 * gdn_new_state -- zero-fill a caller-allocated state buffer [B,H,Dk,Dv] float32.
 * The gated-deltanet card's new_state(batch, heads, key_dim, value_dim) gives a
 * fresh state for a sequence ("Usage"); zero is the state before any token.
 * Errors: GDN_ERR_INVALID_ARG for NULL state or non-positive sizes.
 */
gdn_status gdn_new_state(float *state, int B, int H, int Dk, int Dv, void *stream);

/*
 * gdn_workspace_bytes -- device scratch size that gdn_forward
 * (for_backward = 0) or gdn_backward (for_backward = 1) needs for `shape`.
 * Returns 0 for an invalid or unsupported shape.  The workspace is caller
 * memory, 256-byte aligned, contents on entry irrelevant.
 */
size_t gdn_workspace_bytes(const gdn_shape *shape, int for_backward);

/*
 * gdn_forward -- the whole layer over T tokens in chunked form.
 *
 * Within each chunk of C tokens the per-channel cumulative decay is formed
 * (Marin note, "Background"); query-key and key-key scores that span the two
 * halves of a block are computed with the decay split at the last token of
 * the earlier half, so the spanning scores are one dense matrix product per
 * block pair (Marin note, "Approach"); the split is repeated inside every
 * half down to single tokens, so every score comes from such a product; the
 * unit-lower-triangular delta system of the chunk is solved in WY form; and
 * the state is carried across chunks
 * (atomic_ops card, "Features": chunk scores, WY block solve, recompute,
 * inter-chunk scan).  The result equals the token recurrence above up to
 * floating-point rounding.
 *
 * h0 may be NULL (zero initial state).  hT may be NULL (not written) and may
 * alias h0 (the state carries in place across calls, as in the gated-deltanet
 * card's "Usage").  o must not alias any input.  ws must hold
 * gdn_workspace_bytes(shape, 0) bytes (GDN_ERR_WORKSPACE otherwise).
 */
gdn_status gdn_forward(const gdn_shape *shape, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const float *h0, void *o, float *hT,
                       void *ws, size_t ws_bytes, void *stream);

/*
 * gdn_forward_noalloc -- gdn_forward for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): the same computation and results (bitwise), with the
 * workspace taken from a static device array of GDN_NOALLOC_SCRATCH_BYTES that
 * every device holds from the library's first use on it until the process
 * ends.  The call allocates nothing.  Every call on one device shares that
 * device's array, so calls that overlap on one device (concurrent streams or
 * host threads) race and must be serialised by the caller; consecutive calls on
 * one stream are safe.  The shape must have diag = 0 (the stage counters would
 * sit in the shared array, out of the caller's reach).
 * Errors: as gdn_forward; GDN_ERR_WORKSPACE when gdn_workspace_bytes(shape, 0)
 * exceeds GDN_NOALLOC_SCRATCH_BYTES (64 MiB: at 128 x 128 with chunk 64 about
 * 450 chunk-heads, e.g. B = 1, H = 6, T = 4096); GDN_ERR_UNSUPPORTED for diag = 1;
 * GDN_ERR_HIP if the array's device address cannot be obtained.
 */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)
gdn_status gdn_forward_noalloc(const gdn_shape *shape, const void *q, const void *k,
                               const void *v, const float *g, const float *beta, const float *h0,
                               void *o, float *hT, void *stream);

/*
 * gdn_backward -- gradients of the chunked forward with respect to q, k, v, g,
 * beta and h0, given dO = dL/do and dhT = dL/dhT (NULL = zero).  The forward
 * intermediates are recomputed from the inputs (nothing is kept between
 * calls); the backward runs a reverse scan over chunks followed by a
 * chunk-parallel gradient stage (atomic_ops card, "Features": fused backward).
 * dh0 may be NULL (not written).  Every other output is required.
 * ws must hold gdn_workspace_bytes(shape, 1) bytes.
 */
gdn_status gdn_backward(const gdn_shape *shape, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const float *h0, const void *dO,
                        const float *dhT, void *dq, void *dk, void *dv, float *dg, float *dbeta,
                        float *dh0, void *ws, size_t ws_bytes, void *stream);

/*
 * gdn_forward_train / gdn_backward_train -- the same forward and backward for
 * training, where the backward reuses what the forward computed instead of
 * recomputing it (atomic_ops card, "Features": the backward reuses forward
 * residuals).  gdn_forward_train writes o and hT exactly as gdn_forward and
 * also leaves its chunk intermediates and the state at the start of every
 * chunk in `ws`, which must hold gdn_workspace_bytes(shape, 1) bytes.
 * gdn_backward_train then reads them from the same `ws`: it must be called
 * with the same shape, the same q, k, v, g, beta contents and the workspace
 * untouched in between (the library cannot check this; a mismatch gives
 * wrong gradients, not an error).  Results equal gdn_backward's bitwise.
 * Errors as gdn_forward / gdn_backward.
 */
gdn_status gdn_forward_train(const gdn_shape *shape, const void *q, const void *k, const void *v,
                             const float *g, const float *beta, const float *h0, void *o,
                             float *hT, void *ws, size_t ws_bytes, void *stream);
gdn_status gdn_backward_train(const gdn_shape *shape, const void *q, const void *k,
                              const void *v, const float *g, const float *beta, const void *dO,
                              const float *dhT, void *dq, void *dk, void *dv, float *dg,
                              float *dbeta, float *dh0, void *ws, size_t ws_bytes, void *stream);

/*
 * gdn_decode_step -- one token of the recurrence for every (batch, head), with
 * the state updated in place: each state is read once and written once
 * (gated-deltanet card, "Method": the state is the whole cost).  shape->T must
 * be 1; q, k [B,1,H,Dk]; v, o [B,1,H,Dv]; g [B,1,H,Dk] or [B,1,H];
 * beta [B,1,H]; state [B,H,Dk,Dv] float32 (read and overwritten).
 * Decoding token by token equals the chunked forward up to rounding.
 */
gdn_status gdn_decode_step(const gdn_shape *shape, const void *q, const void *k, const void *v,
                           const float *g, const float *beta, float *state, void *o,
                           void *stream);

/*
 * Decode with a checkpoint and a buffer of recent tokens (the ReplaySSM idea:
 * news digest "Gated DeltaNet", the blurb on state traffic in SSM decoding).
 * The state of each (batch, head) is a checkpoint `ckpt` [B,H,Dk,Dv] fp32 plus
 * up to `depth` (1..16) buffered tokens (their key, accumulated log-decay and
 * delta).  gdn_replay_step reads the checkpoint, computes the token's output
 * and delta directly (no state write), and appends to the buffer; when the
 * buffer fills it folds it into the checkpoint.  Outputs and, after
 * gdn_replay_fold, the state are those of gdn_decode_step (same recurrence,
 * reassociated; equal up to fp32 rounding).  Shapes as gdn_decode_step
 * (T == 1, no numerical-safety options); `buf` is caller-owned device memory of
 * gdn_replay_buffer_bytes(shape, depth) bytes, emptied by gdn_replay_reset
 * before first use.  Every call must pass the same depth and decay kind.
 * Errors: GDN_ERR_INVALID_ARG for a bad shape or depth or a NULL pointer,
 * GDN_ERR_ALIGNMENT, GDN_ERR_UNSUPPORTED for sizes gdn_decode_step refuses.
 */
size_t gdn_replay_buffer_bytes(const gdn_shape *shape, int depth);
gdn_status gdn_replay_reset(const gdn_shape *shape, void *buf, int depth, void *stream);
gdn_status gdn_replay_step(const gdn_shape *shape, const void *q, const void *k, const void *v,
                           const float *g, const float *beta, float *ckpt, void *buf, int depth,
                           void *o, void *stream);
/* gdn_replay_fold -- fold the buffer into the checkpoint (ckpt becomes the
 * current state) and empty it; q, k, v, g, beta are not read. */
gdn_status gdn_replay_fold(const gdn_shape *shape, float *ckpt, void *buf, int depth,
                           void *stream);

/*
 * gdn_diag_read -- copy the stage counters of the last chunked forward pass run
 * in `ws` (gdn_forward, gdn_forward_train, or the recompute inside gdn_backward,
 * which has no o / hT stage) to host memory: counts[GDN_DIAG_WORDS].  The
 * shape must have diag = 1 and match the call that ran.  Synchronises `stream`
 * (atomic_ops card, "Debugging": per-stage reports of non-finite or > 1e6
 * values; diagnostic only).
 * Errors: GDN_ERR_INVALID_ARG for a bad shape, diag = 0, NULL ws or counts;
 * GDN_ERR_HIP if the copy fails.
 */
gdn_status gdn_diag_read(const gdn_shape *shape, const void *ws, unsigned int *counts,
                         void *stream);

/*
 * ---------------------------------------------------------------------------
 * Around the layer: what a stack of gated delta-rule layers and softmax
 * attention layers needs next to the recurrence.  The conventions above hold:
 * device pointers that the caller owns, 16-byte alignment (4-byte for the int
 * arrays and for rstd and lse), the caller's stream, no allocation, no host
 * synchronisation, deterministic results, statuses before any launch.
 * Everything is computed in float32 and rounded to the stored type once; the
 * operands of the matrix products after a softmax take the inputs' type.
 * ---------------------------------------------------------------------------
 *
 * Norms before and after a block.
 *
 * gdn_norm_block: h = x + res_scale o y, n = h o weight / sqrt(mean(h^2) + eps)
 * over rows of `width` values: the residual stream x takes the last block's
 * output y, scaled per channel (y NULL: h = x; res_scale NULL: 1), and the
 * next block gets n.  x, y, h, n [tokens, width] (dtype); res_scale, weight
 * [width], rstd [tokens] float32 (1 / sqrt(...), for the backward).  h and
 * rstd may be NULL (not written); h may be x or y themselves.  n is computed
 * from the unrounded h.  width: a multiple of 8 (bf16, at most 16384) or of 4
 * (float32, at most 8192).
 *
 * gdn_norm_block_backward: with dn, and dh the gradient that arrives at h from
 * behind (NULL = zero), dx = dL/dx, dy = res_scale o dx, dweight, dres_scale.
 * It reads x and y, not h.  With y but no res_scale dL/dy is dx itself; dy
 * and dres_scale are written only with res_scale.
 *
 * gdn_norm_gate: y = o weight / sqrt(mean(o^2) + eps) * gate / (1 + exp(-gate))
 * per head row of `width` = Dv values in {16, 32, 64, 128}: the layer's output
 * before its projection.  o, y [tokens, heads, width] dense, gate the same with
 * gate_stride elements between tokens (0: dense; a slice of a wider projection
 * otherwise), weight [width], rstd [tokens, heads] float32 (may be NULL).
 * gdn_norm_gate_backward: do, dgate (both dense), dweight.
 *
 * The backward's workspace holds gdn_norm_workspace_bytes(shape, gate) bytes
 * (gate: 0 for the block norm, 1 for the gated norm; 0 bytes: invalid shape).
 * tokens * heads <= 2^29.  With tokens = 0 the backward writes zero weights'
 * gradients.
 */
typedef struct {
    int tokens, heads, width; /* heads = 1 for the block norm */
    int dtype;                /* gdn_dtype */
    float eps;                /* in (0, 1] */
    long long gate_stride;    /* gated norm: elements between the gate's tokens, 0 = heads * width */
} gdn_norm_shape;

size_t gdn_norm_workspace_bytes(const gdn_norm_shape *shape, int gate);
gdn_status gdn_norm_block(const gdn_norm_shape *shape, const void *x, const void *y,
                          const float *res_scale, const float *weight, void *h, void *n,
                          float *rstd, void *stream);
gdn_status gdn_norm_block_backward(const gdn_norm_shape *shape, const void *dn, const void *dh,
                                   const void *x, const void *y, const float *res_scale,
                                   const float *weight, const float *rstd, void *dx, void *dy,
                                   float *dweight, float *dres_scale, void *ws, size_t ws_bytes,
                                   void *stream);
gdn_status gdn_norm_gate(const gdn_norm_shape *shape, const void *o, const void *gate,
                         const float *weight, void *y, float *rstd, void *stream);
gdn_status gdn_norm_gate_backward(const gdn_norm_shape *shape, const void *dy, const void *o,
                                  const void *gate, const float *weight, const float *rstd,
                                  void *dO, void *dgate, float *dweight, void *ws,
                                  size_t ws_bytes, void *stream);

/*
 * Causal softmax attention with grouped heads over packed sequences.
 *
 * Query head h uses key head h / (Hq / Hkv).  The T token rows of q, k, v, o
 * belong to B sequences: sequence b has rows cu_seqlens[b] .. cu_seqlens[b+1]-1
 * (device memory, B + 1 entries, non-decreasing, from 0 to at most T; entries
 * outside are clamped, never followed out of the buffers).  Rows of no
 * sequence are not used and not written: outputs there stay as they were.
 *   q [T, Hq, D], k, v [T, Hkv, D] (dtype): dense within a token, with
 *   q_stride, k_stride, v_stride elements between tokens (0 = dense; slices of
 *   one projection's output otherwise); o, dO, dq [T, Hq, D], dk, dv
 *   [T, Hkv, D] dense; lse [T, Hq] float32.
 * scale 0 means D^-0.5.  D in {64, 128}; Hq a multiple of Hkv, at most 1024;
 * T * Hq < 2^27.
 *
 * A value that is not finite reaches the results that depend on it and no
 * others: not those of other sequences, nor of earlier tokens (gradients: of
 * later keys).
 *
 * gdn_attn_forward: token i of a sequence attends to its tokens 0 .. i.
 * lse = log sum exp(scale q.k) over them (may be NULL; the backward needs it).
 * gdn_attn_backward: dq, dk, dv from dO; ws holds
 * gdn_attn_workspace_bytes(shape, GDN_ATTN_BACKWARD) bytes.  A key head's
 * gradient is the sum over its query heads.  In float32 T * Hq (at D = 128) is at most
 * 2^27 - 8, and the blocks of 128 keys and of 128 query rows, (T / 128 + B) Hkv
 * and (T (Hq / Hkv) / 128 + B) Hkv, are together below 2^24.
 *
 * The paged cache: k_cache, v_cache [num_pages, page_size, Hkv, D] (dtype),
 * page_size a power of two from 16 to 1024; position p of sequence b lies in
 * slot p % page_size of page page_table[b][p / page_size] (device memory,
 * [B, max_pages]; -1, or any value outside [0, num_pages), means that there is
 * no such page).  kv_len[b] (device memory) counts the sequence's positions
 * with its new tokens, so that the new token i of n stands at position
 * kv_len[b] - n + i.
 *
 * gdn_attn_append writes every new token's k and v to its position, k rotated:
 * for i < rot_dim / 2, with c, s = cos, sin[position][i],
 *   x'[i] = x[i] c - x[i + rot_dim/2] s,  x'[i + rot_dim/2] = x[i + rot_dim/2] c + x[i] s,
 * the rest of a head as it is; q rotated the same way into q_out [T, Hq, D]
 * (q and q_out both NULL: not done; q_out may be q where q is dense).
 * cos, sin [max_pos, rot_dim / 2] float32, rot_dim a multiple of 16 up to D (0:
 * no rotation, cos, sin not read).  A token whose position is negative, not
 * below max_pos or behind the table is left out, q_out included; one whose page
 * does not exist writes no cache row.  Positions that two sequences of one call
 * both write (pages they share) end with either's values.  At most 2^25 - 2
 * tokens a call.
 *
 * gdn_attn_paged: new token i attends to positions 0 .. kv_len[b] - n + i of
 * its sequence, i.e. the cache after gdn_attn_append; q already rotated.
 * Positions without a page are absent; a token that sees nothing gets zeros.
 * One new token a sequence is decoding.  ws holds
 * gdn_attn_workspace_bytes(shape, GDN_ATTN_PAGED) bytes.  k_stride and
 * v_stride are not used.  Cache slots that no position below kv_len[b] names are
 * not used, whatever they hold.  Calls that overlap must not share a workspace.
 */
typedef struct {
    int B, T, Hq, Hkv, D;
    int dtype;   /* gdn_dtype */
    float scale; /* 0 means D^-0.5 */
    long long q_stride, k_stride, v_stride; /* elements between tokens, 0 = dense */
    int num_pages, page_size, max_pages;    /* paged cache */
    int rot_dim, max_pos;                   /* gdn_attn_append */
} gdn_attn_shape;

enum { GDN_ATTN_PAGED = 0, GDN_ATTN_BACKWARD = 1 };

size_t gdn_attn_workspace_bytes(const gdn_attn_shape *shape, int call);
gdn_status gdn_attn_forward(const gdn_attn_shape *shape, const void *q, const void *k,
                            const void *v, const int *cu_seqlens, void *o, float *lse,
                            void *stream);
gdn_status gdn_attn_backward(const gdn_attn_shape *shape, const void *q, const void *k,
                             const void *v, const int *cu_seqlens, const void *o,
                             const float *lse, const void *dO, void *dq, void *dk, void *dv,
                             void *ws, size_t ws_bytes, void *stream);
gdn_status gdn_attn_append(const gdn_attn_shape *shape, const void *q, const void *k,
                           const void *v, const float *cos, const float *sin,
                           const int *cu_seqlens, const int *kv_len, const int *page_table,
                           void *k_cache, void *v_cache, void *q_out, void *stream);
gdn_status gdn_attn_paged(const gdn_attn_shape *shape, const void *q, const void *k_cache,
                          const void *v_cache, const int *page_table, const int *cu_seqlens,
                          const int *kv_len, void *o, void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * A state-space layer's operators, and the page step that feeds all layers.  The
 * conventions of the part above hold: sequences are packed, cu_seqlens and every
 * other int array are device data, clamped or checked where they are used, and
 * rows of no sequence are neither used nor written.  Weights, steps and states of
 * the scan are float32 (4-byte aligned where they are per head).  Outputs may not
 * overlap inputs or one another, but where a call says that one may be the other.
 * ---------------------------------------------------------------------------
 *
 * Short causal convolution along the tokens, every channel by itself: with e the
 * W - 1 rows of a sequence's state (NULL: zeros) followed by its rows of x,
 *   z_t = bias + sum_j weight[.][j] e_{t+j},   y = z / (1 + exp(-z)) (silu) or z,
 * and the new state is the last W - 1 rows of e, as they are.
 *   x [T, C] (dtype) with x_stride elements between tokens (0 = dense), y, dy, dx
 *   [T, C] dense; weight, dweight [C, W], bias, dbias [C] float32 (bias may be
 *   NULL); states [B, W - 1, C] (dtype), oldest row first.
 * W is 2, 3 or 4; C a multiple of 8 (bf16) or 4 (float32), at most 2^20; T at most
 * 2^28, B at most 65536, or 2^25 for single tokens.  Of bounds that decrease, one
 * below an earlier one counts as that one.  y may not be x, nor dx x or dy, dstate dstate_out, dweight
 * weight or dbias bias.
 *
 * gdn_conv_forward: state_out (NULL: not written) may be state.  A sequence
 * without rows keeps its state.
 * gdn_conv_backward: dx, dweight, dbias (may be NULL) and dstate (may be NULL) from
 * dy and dstate_out, the gradient that arrives at the new state (NULL = zero).  ws
 * holds gdn_conv_workspace_bytes(shape) bytes.
 * gdn_conv_step: one row a sequence (T = B, row b is sequence b's); state is
 * updated in place.
 */
typedef struct {
    int B, T, C, W;
    int dtype;          /* gdn_dtype */
    int silu;           /* 1: y = z / (1 + exp(-z)); 0: y = z */
    long long x_stride; /* elements between tokens of x, 0 = C */
} gdn_conv_shape;

size_t gdn_conv_workspace_bytes(const gdn_conv_shape *shape);
gdn_status gdn_conv_forward(const gdn_conv_shape *shape, const void *x, const float *weight,
                            const float *bias, const int *cu_seqlens, const void *state, void *y,
                            void *state_out, void *stream);
gdn_status gdn_conv_backward(const gdn_conv_shape *shape, const void *x, const float *weight,
                             const float *bias, const int *cu_seqlens, const void *state,
                             const void *dy, const void *dstate_out, void *dx, float *dweight,
                             float *dbias, void *dstate, void *ws, size_t ws_bytes, void *stream);
gdn_status gdn_conv_step(const gdn_conv_shape *shape, const void *x, const float *weight,
                         const float *bias, void *state, void *y, void *stream);

/*
 * Selective state space scan.  Head h of H, in group h / (H / G) of G, keeps a
 * state S [N x P] and for each token applies
 *   delta = log(1 + exp(dt + dt_bias)) (softplus) or dt + dt_bias,
 *   S <- exp(delta A) S + delta B x^T,   y = S^T C + D x.
 *   x, y, dy, dx [T, H, P], B, C, dB, dC [T, G, N] (dtype): x, B and C dense within
 *   a token, with x_stride, b_stride, c_stride elements between tokens (0 = dense;
 *   slices of a convolution's output otherwise), the others dense; dt, ddt [T, H],
 *   A, D, dt_bias and their gradients [H], states [B, H, N, P] float32.
 * D, dt_bias and h0 (zero state) may be NULL; A is meant to be negative, but is
 * not tested.  N and P in {64, 128}; H a multiple of G, at most 1024; T * H < 2^27,
 * B * H < 2^23, B at most 65536 but for single tokens; strides at most 2^24.  Of bounds
 * that decrease, one below an earlier one counts as that one.
 * A value that is not finite reaches the results that depend on it and no others; a
 * step (dt) that is not may reach all gradients of its head in its sequence, and of
 * the group's B and C there.
 *
 * gdn_ssm_forward: y, and hT the state behind each sequence (NULL: not written; may
 * be h0; a sequence without rows keeps its state).
 * gdn_ssm_backward: gradients of sum(y dy) + sum(hT dhT) (dhT NULL = zero); dD,
 * ddt_bias and dh0 may be NULL.  The states are formed
 * again; nothing is kept between the calls.  Float32 results, and hT, are as exact
 * for bf16 inputs as for the same values in float32.
 * Both: ws holds gdn_ssm_workspace_bytes(shape, GDN_SSM_...) bytes; calls that
 * overlap must not share one.
 * gdn_ssm_step: one token a sequence (T = B, row b is sequence b's), the state
 * updated in place.
 */
typedef struct {
    int B, T, H, G, N, P;
    int dtype;    /* gdn_dtype */
    int softplus; /* 1: delta = softplus(dt + dt_bias); 0: dt + dt_bias */
    long long x_stride, b_stride, c_stride; /* elements between tokens, 0 = dense */
} gdn_ssm_shape;

enum { GDN_SSM_FORWARD = 0, GDN_SSM_BACKWARD = 1 };

size_t gdn_ssm_workspace_bytes(const gdn_ssm_shape *shape, int call);
gdn_status gdn_ssm_forward(const gdn_ssm_shape *shape, const void *x, const float *dt,
                           const float *A, const void *B, const void *C, const float *D,
                           const float *dt_bias, const int *cu_seqlens, const float *h0, void *y,
                           float *hT, void *ws, size_t ws_bytes, void *stream);
gdn_status gdn_ssm_backward(const gdn_ssm_shape *shape, const void *x, const float *dt,
                            const float *A, const void *B, const void *C, const float *D,
                            const float *dt_bias, const int *cu_seqlens, const float *h0,
                            const void *dy, const float *dhT, void *dx, float *ddt, float *dA,
                            void *dB, void *dC, float *dD, float *ddt_bias, float *dh0, void *ws,
                            size_t ws_bytes, void *stream);
gdn_status gdn_ssm_step(const gdn_ssm_shape *shape, const void *x, const float *dt, const float *A,
                        const void *B, const void *C, const float *D, const float *dt_bias,
                        float *state, void *y, void *stream);

/*
 * The page step of continuous batching, for the paged cache above.  A pool of
 * num_pages pages; the free ones are free_pages[0 .. free_count[0] - 1], a stack
 * whose top is its end.  kv_len [B] counts the positions that each sequence has;
 * its pages are the first ceil(kv_len / page_size) entries of its row of page_table
 * [B, max_pages].  All arrays int32 device memory, but for slots (int64).
 * Entries of the table and of the stack are the caller's names of pages and are
 * trusted: num_pages is the room of the stack, not a limit on the names, which
 * gdn_attn_append and gdn_attn_paged test against their cache.  Only a name below 0
 * is known as no page (slot -1).  So a length that claims pages which its row does
 * not have (-1) puts -1 on the stack when they are released, and the tokens of a
 * sequence that takes it get slots of -1.
 *
 * gdn_pages_release: the pages of every sequence with done[b] != 0 go on the stack,
 * in the order of the sequences and of their tables, and its length becomes 0 (the
 * table keeps its entries, which no position names any more).
 *
 * gdn_pages_take: sequence b asks for want[b] new tokens (below 0: none) and gets
 * all of them or none.  It gets them if its pages fit its row of the table; if the
 * stack holds the pages that it and those before it whose rows fit need (or it
 * needs none); and if `rows` holds the tokens of it and of those before it that
 * pass the first two tests.  Its new pages come from the top of the stack, one
 * after the other, and are entered in the table.  kv_out = kv_len + the tokens it
 * gets; cu_seqlens [B + 1] their running sum, from 0; and for the tokens, packed in
 * that order, positions [rows] (in the sequence) and slots [rows] (page *
 * page_size + place in the page, -1 without a page), either of which may be NULL;
 * rows behind the last token stay as they were.  kv_out, cu_seqlens and page_table
 * are what gdn_attn_append and gdn_attn_paged take.
 *
 * kv_out and count_out may be kv_len and free_count: then both are updated in
 * place, by a launch of its own.  B at most 8192, page_size and max_pages as above.
 * A free_count outside 0 .. num_pages is taken as the nearest of them, a length
 * below 0 as 0.
 */
typedef struct {
    int B, num_pages, page_size, max_pages;
    int rows; /* gdn_pages_take: the most tokens */
} gdn_pages_shape;

gdn_status gdn_pages_release(const gdn_pages_shape *shape, const int *done, const int *kv_len,
                             const int *page_table, int *free_pages, const int *free_count,
                             int *kv_out, int *count_out, void *stream);
gdn_status gdn_pages_take(const gdn_pages_shape *shape, const int *want, const int *kv_len,
                          int *page_table, const int *free_pages, const int *free_count,
                          int *kv_out, int *count_out, int *cu_seqlens, int *positions,
                          long long *slots, void *stream);

/* gdn_status_string -- static, human-readable name of a status code. */
const char *gdn_status_string(gdn_status status);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */
