/*
 * attn_core.h -- C ABI of the GB300 (sm_103a) attention-core library.
 *
 * The attention core is QK^T, softmax, softmax dropout and attention over V:
 * the part of a transformer layer that selective activation recomputation
 * does not store, because its activations are large and its FLOPs few, and
 * recomputes in the backward pass instead ("Reducing Activation
 * Recomputation in Large Transformer Models", dmarx anthology LIT-736, Key
 * takeaways, fourth bullet; "Recomputing Activations", curionode Plate 2,
 * second paragraph and "Memory for compute, selectively").
 *
 * attn_core_fwd stores only O and one fp32 log-sum-exp per query row; with
 * Q, K, V and the Philox seed/offset that is everything the backward pass
 * needs.  attn_core_bwd_recompute rebuilds the scores, probabilities and
 * dropout mask on chip and never writes them to global memory, so the
 * 5 a s^2 b byte term of the per-layer activation formula sbh(34 + 5as/h)
 * is never held in device memory.  attn_core_stored_bytes reports that
 * accounting exactly.
 *
 * Tensors (all device pointers, 16-byte aligned, contiguous, row-major):
 *   Q, O, dO, dQ : bf16 [b, h_q,  s,    d]
 *   K, V, dK, dV : bf16 [b, h_kv, s_kv, d]   (s_kv = s unless set)
 *   LSE          : fp32 [b, h_q, s]   natural-log log-sum-exp of each row
 * Query head h uses KV head h / (h_q / h_kv) (grouped-query attention).
 * Causal masking is top-left aligned: query i sees keys 0..i; it needs
 * s_kv == s.  Without it, s queries attend to all s_kv keys
 * (cross-attention when s_kv != s).
 *
 * Readings the pages leave open (the CPU oracle in the tests follows the
 * same ones):
 *   - scale: scale <= 0 selects 1/sqrtf(d), computed in fp32.
 *   - LSE is in natural-log units.
 *   - dropout acts on the normalised probabilities, before the product with V.
 *   - dropout mask: Philox-4x32-10 (Salmon et al., SC'11) with key
 *     (seed & 0xffffffff, seed >> 32) and counter (j / 16, i, b*h_q + h,
 *     offset) for query i, key j of query head h in batch b; the call's four
 *     output words give sixteen 8-bit draws, key j taking byte j % 4 (bits
 *     8 (j % 4) .. 8 (j % 4) + 7) of word (j % 16) / 4.  With
 *     thr = round(p * 256) (at most 255) an element is dropped iff its draw <
 *     thr, and kept elements are scaled by 1 / (1 - thr / 256): the effective
 *     rate is p rounded to a multiple of 1/256 (p = 0.1 drops 26/256 =
 *     0.1015625 of the elements; p < 1/512 drops none).  p == 0 draws nothing.
 *
 * Every call is asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 * default stream).  The library allocates no device memory: the caller owns
 * every buffer, including the backward workspace.
 */
#ifndef ATTN_CORE_H
#define ATTN_CORE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes.  On any non-zero code no kernel has been launched and no
 * output has been written, except ATTN_CORE_ERR_CUDA from a launch, which
 * reports the CUDA error of that launch. */
#define ATTN_CORE_OK 0
#define ATTN_CORE_ERR_INVALID_ARG 1         /* null pointer, bad shape, p outside [0,1), offset >= 2^32 */
#define ATTN_CORE_ERR_UNSUPPORTED 2         /* head dimension or device not supported */
#define ATTN_CORE_ERR_MISALIGNED 3          /* a pointer is not 16-byte aligned (workspace: 256) */
#define ATTN_CORE_ERR_WORKSPACE_TOO_SMALL 4 /* bwd workspace smaller than attn_core_bwd_workspace_bytes */
#define ATTN_CORE_ERR_CUDA 5                /* a CUDA runtime or driver call failed */
#define ATTN_CORE_ERR_DEVICE_TIMEOUT 6      /* a kernel wait ran past its limit (reported via dev_status) */
#define ATTN_CORE_ERR_DEVICE_TABLE 7        /* a device table held an entry out of range (reported via dev_status) */

/* flags */
#define ATTN_CORE_FLAG_REDRAW_MASK 0x1         /* backward: the dK/dV kernel draws the dropout mask again
                                                  instead of reading keep bits the dQ kernel wrote to the
                                                  workspace; the workspace then holds only the row
                                                  statistics (smaller, see attn_core_bwd_workspace_bytes)
                                                  at the cost of a second Philox pass */
#define ATTN_CORE_FLAG_TEST_WAIT_TIMEOUT 0x100 /* test hook: every kernel waits on a barrier that nothing
                                                  completes; it gives up after wait_timeout_ms, writes
                                                  ATTN_CORE_ERR_DEVICE_TIMEOUT to dev_status and exits */

typedef struct {
    int32_t b, h_q, h_kv, s, d; /* s queries per head; h_q % h_kv == 0; d in {64, 96, 128, 160} */
    int32_t causal;             /* 0 or 1 */
    float p_drop;               /* softmax-dropout probability in [0, 1) */
    float scale;                /* score scale; <= 0 selects 1/sqrtf(d) */
    uint64_t seed;              /* Philox key */
    uint64_t offset;            /* Philox counter word 3; must be < 2^32 */
    /* Optional caller-owned device int32, zero before the call.  A kernel
     * whose wait runs out writes (ATTN_CORE_ERR_DEVICE_TIMEOUT | site << 8)
     * there (first error wins); read it after synchronising.  May be NULL. */
    int32_t* dev_status;
    int32_t flags;              /* ATTN_CORE_FLAG_* */
    uint32_t wait_timeout_ms;   /* limit of each in-kernel wait; 0 selects 2000 ms */
    /* Optional profiling hook: an array of cudaEvent_t handles, two per
     * kernel the call launches (fwd: 1 kernel; bwd: 2 kernels, in order
     * dQ, dK/dV), recorded on `stream` immediately before and
     * after each launch.  May be NULL. */
    void** timing_events;
    /* Keys (and value rows) per KV head; 0 selects s.  With s_kv != s the
     * causal mask is aligned top-left: query i sees keys 0 .. min(i, s_kv - 1)
     * (with more keys than queries, keys s .. s_kv - 1 are seen by no query
     * and get zero dK and dV).  The dropout mask of (query i, key j) does not
     * depend on s or s_kv. */
    int32_t s_kv;
} attn_core_params;

typedef struct {
    /* Per-layer activation bytes of one rank's shard, hidden h = h_q * d:
     * the activation-checkpointing page's per-token forms 34d + 5HT,
     * 34d and 2d ("Recomputing Activations", Workshop) times s * b. */
    int64_t layer_none;           /* 34 s b h + 5 h_q s^2 b : nothing recomputed */
    int64_t layer_selective;      /* 34 s b h               : attention core recomputed */
    int64_t layer_full;           /* 2 s b h                : only the layer input kept */
    int64_t core_scores_avoided;  /* 5 h_q s s_kv b         : what this library never stores */
    int64_t core_kept;            /* 2 d b (2 h_q s + 2 h_kv s_kv): Q, K, V, O in bf16 */
    int64_t core_recompute_state; /* 4 b h_q s + 16         : LSE and seed/offset */
} attn_core_bytes;

/* Forward: O and LSE from Q, K, V (the core's forward in the takeaways'
 * order: QK^T, softmax, softmax dropout, attention over V).  Launches one
 * kernel.  Writes O and LSE only. */
int attn_core_fwd(const attn_core_params* p, const void* q, const void* k, const void* v, void* o,
                  float* lse, void* stream);

/* Bytes of device workspace attn_core_bwd_recompute needs, 0 if p is invalid:
 *   8 * b * h_q * ceil(s / 128) * 128   two fp32 row statistics per padded
 *                                       query row, and, when p_drop > 0 and
 *                                       d <= 128,
 *   2048 * b * h_q * N                  the dropout keep bits, one bit per
 *                                       (query, key) of each 128 x 128 block,
 * with N = n (n + 1) / 2 blocks per head if causal with s_kv == s
 * (n = ceil(s / 128)), ceil(s / 128) * ceil(s_kv / 128) if not causal, and no
 * keep bits for causal with s_kv != s (the second kernel draws the mask again).  The keep bits are transient (written and
 * read within one backward call) but scale with s^2: 6.7 MB for b = 2,
 * h_q = 12, s = 2048, and 272 MB for h_q = 64, s = 8192.  Callers short of
 * memory set ATTN_CORE_FLAG_REDRAW_MASK to leave them out. */
size_t attn_core_bwd_workspace_bytes(const attn_core_params* p);

/* Backward with recomputation: dQ, dK, dV from Q, K, V, O, LSE and dO.  The
 * scores, probabilities and dropout mask are rebuilt on chip from Q, K, LSE
 * and (seed, offset); the mask is bit-identical to the forward's.  For
 * d <= 128 it is drawn once, by the first kernel, which hands it to the
 * second as bits in the workspace (nothing of it outlives the call); for
 * d = 160 each kernel draws it.  The
 * softmax row statistic sum_j P_ij dP_ij is formed exactly from the
 * recomputed P and dP (a first estimate from the stored bf16 O is corrected
 * in fp32), not rounded through the stored output.  Launches two kernels
 * (dQ with the row statistics, then dK/dV).  `workspace` is caller-owned
 * device memory of at least attn_core_bwd_workspace_bytes(p) bytes, 256-byte
 * aligned; its contents on entry do not matter.  dQ, dK, dV are written
 * whole (no accumulation into existing contents). */
int attn_core_bwd_recompute(const attn_core_params* p, const void* q, const void* k, const void* v,
                            const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Backward with recomputation for callers that cannot allocate device
 * memory.  Some callers have no allocator to call: code running inside
 * another framework that owns every byte of device memory through its own
 * pool, code invoked from a library that forbids allocation in its callbacks,
 * or services whose memory is planned once at start-up.  They cannot provide
 * the workspace attn_core_bwd_recompute asks for, so this variant uses a
 * fixed scratch array inside the library instead and allocates nothing
 * (no cudaMalloc, no cudaFree, no allocating library routine).  The paper
 * has no counterpart to this entry point.
 *
 * Same arguments and results as attn_core_bwd_recompute without the
 * workspace.  The array holds the row statistics only, so here the second
 * kernel draws the dropout mask again from Philox (the same bits).  Limit: b * h_q * ceil(s / 128) * 128 <= 1048576 padded query
 * rows (the array holds 8 MiB on every GPU that loads the library, until the
 * process exits); larger shapes return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL
 * without launching anything.  Every call looks up the array's device
 * address for the current device (cudaGetSymbolAddress, which allocates
 * nothing); the first call on a device may make the runtime load this
 * library's device code there, so make that first call before any stream
 * capture.  All calls on a device
 * share the one array and it keeps the last call's contents (nothing in it
 * needs to start at zero), so calls whose kernels overlap on the GPU --
 * concurrent streams, or several host threads -- race on it: order them. */
int attn_core_bwd_recompute_noalloc(const attn_core_params* p, const void* q, const void* k, const void* v,
                                    const void* o, const float* lse, const void* dout, void* dq, void* dk,
                                    void* dv, void* stream);

/* ------------------------------------------------------------------------
 * Variable-length (packed) batches.  n_seq sequences of different lengths in
 * one token-major tensor; the tokens of sequence i are rows cu_seqlens_q[i]
 * .. cu_seqlens_q[i + 1] - 1 (keys: cu_seqlens_k, NULL for the same table):
 *   Q, O, dO, dQ : bf16 [total_q, h_q, d]     total_q = cu_seqlens_q[n_seq]
 *   K, V, dK, dV : bf16 [total_k, h_kv, d]
 *   LSE          : fp32 [h_q, total_q]
 * Each sequence attends only within itself, as batch element i of the
 * padded layout would: the same causal rule (top-left aligned when a
 * sequence's query and key counts differ), and the same dropout mask
 * (Philox counter word 2 = i * h_q + head).  The sequence tables are arrays
 * of n_seq + 1 int32 starting at 0 and nondecreasing, given twice: in host
 * memory (cu_seqlens_q / _k: checked, and used to size the launch) and as a
 * device copy with the same values (cu_seqlens_q_dev / _k_dev, read by the
 * kernels; _k_dev may be NULL only when cu_seqlens_k is).  An empty sequence
 * is skipped, one with queries but no keys is invalid; one with keys but no
 * queries gets zero dK and dV rows.  `base` supplies h_q, h_kv, d, causal,
 * p_drop, scale, seed, offset, dev_status, flags and wait_timeout_ms; its b,
 * s and s_kv are ignored and its timing_events must be NULL.  The whole
 * batch is one launch per kernel (the same kernels as the padded entry
 * points): they take the batch as n_seq elements of the longest sequence's
 * length, skip the work past each sequence's end, and store the rows of a
 * sequence's last, partial block one by one so that nothing lands in the next
 * sequence.  Both tables must stay unchanged until the calls' kernels have
 * run. */
typedef struct {
    attn_core_params base;
    int32_t n_seq;
    const int32_t* cu_seqlens_q;       /* host, n_seq + 1 */
    const int32_t* cu_seqlens_k;       /* host, n_seq + 1, or NULL: as cu_seqlens_q */
    const int32_t* cu_seqlens_q_dev;   /* device copy of cu_seqlens_q */
    const int32_t* cu_seqlens_k_dev;   /* device copy of cu_seqlens_k, or NULL with it */
} attn_core_varlen_params;

int attn_core_fwd_varlen(const attn_core_varlen_params* p, const void* q, const void* k, const void* v, void* o,
                         float* lse, void* stream);

/* Workspace of attn_core_bwd_varlen, 0 if p is invalid: the two fp32 row
 * statistics of every query row, each sequence's rows padded to whole
 * 128-row blocks and aligned to 16 bytes:
 * 8 * h_q * (round_up(total_q, 4) + 132 * n_seq) bytes, rounded up to 256.
 * (The dropout mask is drawn twice in a packed batch; there are no keep bits.) */
size_t attn_core_bwd_varlen_workspace_bytes(const attn_core_varlen_params* p);

int attn_core_bwd_varlen(const attn_core_varlen_params* p, const void* q, const void* k, const void* v,
                         const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Activation-byte accounting (pure host, integer, exact).  Worked example of
 * the activation-checkpointing page: Llama 3 70B, s = 8192, b = 1, h_q = 64,
 * d = 128, 80 layers -> 1.9 TB none, 182.5 GB selective, 10.7 GB full. */
int attn_core_stored_bytes(const attn_core_params* p, attn_core_bytes* out);

/* Static description of a return code. */
const char* attn_core_strerror(int code);

/* ------------------------------------------------------------------------
 * Dropout + residual add + layer norm at a residual sub-layer boundary, on
 * either side of the attention core.  These are the layer norms and the
 * dropouts after the attention block and the MLP that tensor parallelism
 * leaves replicated and that act on each sequence position independently
 * ("Reducing Activation Recomputation in Large Transformer Models", dmarx
 * anthology LIT-736, Key takeaways, first and second bullets).  Reading of
 * the block (the pages give no formula), per row (token) of `hidden` values:
 *     z = residual + dropout(x)                            stored, bf16
 *     y = gamma * (z - mean) * rstd + beta                 bf16
 *     rstd = 1 / sqrt(var + eps), var the biased variance of the stored z.
 * Dropout mask: Philox-4x32-10 with the core's key, counter (col / 8, row,
 * 0xFFFFFFFF, offset) (word 2 is a value no attention head index takes) and
 * eight 16-bit draws per call, column col taking the low (col even) or high
 * (col odd) half of word (col % 8) / 2; dropped iff the draw <
 * round(p * 65536) (at most 65535), kept values scaled by
 * 1 / (1 - thr / 65536).  This block is bound by memory traffic, not by the
 * generator, so it keeps the finer 16-bit draws.  As
 * in the core, the backward redraws the mask from (seed, offset); the block
 * keeps z, mean and rstd only.
 *
 * Tensors (device pointers, 16-byte aligned, contiguous, row-major):
 *   x, residual, z, y, dy, dz_next, dx, d_residual : bf16 [n_rows, hidden]
 *   gamma, beta, dgamma, dbeta                      : fp32 [hidden]
 *   mean, rstd                                      : fp32 [n_rows]
 * Asynchronous on `stream`; nothing is allocated.  Return codes as above. */
typedef struct {
    int32_t n_rows;   /* tokens, >= 1 */
    int32_t hidden;   /* multiple of 8, 8 .. 28672 */
    float p_drop;     /* [0, 1) */
    float eps;        /* layer-norm epsilon, > 0 */
    uint64_t seed;    /* Philox key */
    uint64_t offset;  /* Philox counter word 3; must be < 2^32 */
    /* Optional caller-owned device int32, zero before the call: a forward
     * wait that runs out writes ATTN_CORE_ERR_DEVICE_TIMEOUT | 1 << 8 there.
     * May be NULL. */
    int32_t* dev_status;
    uint32_t wait_timeout_ms;   /* limit of each in-kernel wait; 0 selects 2000 ms */
} attn_core_dal_params;

/* Forward: writes z, y, mean and rstd.  Launches one kernel. */
int attn_core_dropout_add_ln_fwd(const attn_core_dal_params* p, const void* x, const void* residual,
                                 const float* gamma, const float* beta, void* z, void* y, float* mean,
                                 float* rstd, void* stream);

/* Bytes of device workspace the backward needs: 8 * hidden * min(n_rows, 320)
 * (per-CTA column sums for dgamma and dbeta), 0 if p is invalid. */
size_t attn_core_dropout_add_ln_bwd_workspace_bytes(const attn_core_dal_params* p);

/* Backward from dy (gradient of y) and, optionally, dz_next (the gradient
 * reaching z through the residual path; NULL for none):
 *     dz = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dz_next,
 *          g = dy * gamma, xhat = (z - mean) * rstd,
 *     d_residual = dz,  dx = dz * keep / (1 - p_eff),
 *     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy.
 * Needs z, mean and rstd from the forward, not x or residual.  dgamma and
 * dbeta are summed in a fixed order (bit-reproducible).  Launches two
 * kernels; `workspace` is caller-owned device memory of at least
 * attn_core_dropout_add_ln_bwd_workspace_bytes(p) bytes, 16-byte aligned. */
int attn_core_dropout_add_ln_bwd(const attn_core_dal_params* p, const void* dy, const void* dz_next,
                                 const void* z, const float* mean, const float* rstd, const float* gamma,
                                 void* dx, void* d_residual, float* dgamma, float* dbeta, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * GeLU of the layer's MLP, for the layer-level measurement of selective
 * recomputation (the anthology page's Key takeaways, fourth bullet: recompute
 * the whole layer, or only the attention core).  Tanh form:
 *     y = x / 2 * (1 + tanh(sqrt(2 / pi) * (x + 0.044715 x^3))),
 * elementwise on n bf16 values (n a multiple of 8, pointers 16-byte aligned),
 * fp32 arithmetic.  The backward writes dx = dy * dy/dx at x.  One kernel
 * each, asynchronous on `stream`. */
int attn_core_gelu_fwd(int64_t n, const void* x, void* y, void* stream);
int attn_core_gelu_bwd(int64_t n, const void* x, const void* dy, void* dx, void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions.  Pair i of a head's first rot_dim values, (x_a, x_b), is
 * turned by the angle w = position * f_i:
 *     y_a = m (x_a cos w - x_b sin w),   y_b = m (x_b cos w + x_a sin w),
 * with (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved.  The
 * values from rot_dim on are copied.  A score of two rotated heads depends on
 * the difference of their positions only.  f_i = base^(-2i / rot_dim) radians
 * per position, then scaled for contexts longer than the trained one:
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   BANDS   with n = original_len f_i / 2 pi (turns over the trained length)
 *           and k = clamp((n - low_freq) / (high_freq - low_freq), 0, 1):
 *           k f_i + (1 - k) f_i / factor
 *   YARN    ("YaRN: Efficient Context Window Extension", Peng et al. 2023)
 *           with c(n) = rot_dim ln(original_len / 2 pi n) / (2 ln base), the
 *           pair that turns n times over the trained length,
 *           lo = max(floor(c(beta_fast)), 0),
 *           hi = min(ceil(c(beta_slow)), rot_dim - 1) and
 *           k = clamp((i - lo) / max(hi - lo, 0.001), 0, 1):
 *           (1 - k) f_i + k f_i / factor, and m = 0.1 ln(factor) + 1
 * m = 1 unless YARN or `mscale` sets it. */
#define ATTN_CORE_ROPE_NONE 0
#define ATTN_CORE_ROPE_LINEAR 1
#define ATTN_CORE_ROPE_BANDS 2
#define ATTN_CORE_ROPE_YARN 3

typedef struct {
    int32_t d;            /* head dimension, multiple of 8, 8 .. 512 */
    int32_t rot_dim;      /* rotated leading part, multiple of 8, at most min(d, 256); 0 selects that */
    int32_t interleaved;  /* 0 or 1 */
    int32_t scaling;      /* ATTN_CORE_ROPE_* */
    double base;          /* > 1; 0 selects 10000 */
    double factor;        /* > 0; 0 selects 1 */
    double original_len;  /* trained context length, > 0 for BANDS and YARN */
    double low_freq, high_freq;     /* BANDS, low < high; both 0 select 1 and 4 */
    double beta_fast, beta_slow;    /* YARN, slow < fast; both 0 select 32 and 1 */
    double mscale;        /* m, > 0; 0 selects 1 (YARN: 0.1 ln(factor) + 1, at least 1) */
} attn_core_rope_config;

/* The frequencies as the kernels take them, filled by attn_core_rope_init and
 * passed by value to each launch: turns[i] is f_i / 2 pi turns per position
 * as a 64-bit fraction, so that position * turns[i] modulo 2^64 is the angle
 * reduced exactly, at any position. */
typedef struct {
    int32_t d, rot_dim, interleaved;
    float mscale;
    uint64_t turns[128];
} attn_core_rope_table;

int attn_core_rope_init(const attn_core_rope_config* c, attn_core_rope_table* out);   /* pure host */

/* Rotation of Q and K in one launch, over any layout whose heads are
 * contiguous in d: element (batch, head, token, c) of a tensor is at
 * batch * stride[0] + head * stride[1] + token * stride[2] + c.  Strides are
 * in elements, non-negative multiples of 8; an input's may be 0 (a broadcast
 * tensor), an output's must keep its rows apart.  [b, h, s, d] is
 * {h s d, s d, d}; a packed [tokens, h, d] is b = 1, {0, d, h d}.  Pointers are
 * 16-byte aligned.  An output may be its own input (same pointer and strides);
 * otherwise no output overlaps an input or the other output.  h_q or h_kv may be
 * 0 (its pointers are then ignored), their sum is at most 65535; s = 0 does
 * nothing. */
typedef struct {
    int32_t b, s, h_q, h_kv;
    int64_t q_stride[3], k_stride[3];     /* inputs: batch, head, token */
    int64_t yq_stride[3], yk_stride[3];   /* outputs */
    int32_t pos0;                         /* position of token 0 where `positions` is NULL */
    const int32_t* positions;             /* device int32 [b, s] (negative ones turn back), or NULL: pos0 + token */
} attn_core_rope_params;

int attn_core_rope_fwd(const attn_core_rope_params* p, const attn_core_rope_table* t, const void* q, const void* k,
                       void* yq, void* yk, void* stream);

/* Backward: dq, dk from the gradients of the rotated tensors.  The rotation is
 * orthogonal up to m, so this is the turn by -w, times m. */
int attn_core_rope_bwd(const attn_core_rope_params* p, const attn_core_rope_table* t, const void* dyq,
                       const void* dyk, void* dq, void* dk, void* stream);

/* ------------------------------------------------------------------------
 * A key/value cache in pages, and attention of new tokens over it (serving).
 *   k_pages, v_pages : bf16 [n_pages, h_kv, page_size, d]
 *   q, o             : bf16 [n_tokens, h_q, d]    packed new tokens
 *   lse              : fp32 [h_q, n_tokens]
 * Sequence i owns the new tokens cu_seqlens_q[i] .. cu_seqlens_q[i + 1] - 1 (n
 * of them) and kv_lens[i] keys, the new tokens' own among them; key j is row
 * j % page_size of page page_table[i * max_pages + j / page_size].  New token
 * t has position kv_lens[i] - n + t and, under the causal mask (aligned
 * bottom-right), sees the keys up to that position; without it, all of them.
 * A row that sees no key (kv_lens[i] < n, or no keys at all) gets O = 0 and
 * LSE = -inf.  Tokens from cu_seqlens_q[n_seq] on belong to no sequence: their
 * rows are left as they were.  What pages hold past a sequence's end is never
 * used, NaN included, nor are page_table entries past its last page.  (Within
 * a sequence a probability of 0 still meets its value in the product: an
 * infinite or NaN value of one key reaches rows of the same sequence that the
 * mask keeps from seeing it; rows that do see it are infinite or NaN.  A NaN
 * score makes its row's O and LSE NaN.)
 *
 * Probabilities are rounded to bf16 for their product with the values, in
 * batches of at most 32 rows (new tokens times group) a sequence on average to
 * two bf16 terms; and where a sequence's keys are cut into the parts that are
 * joined goes by the lengths of the whole batch.  So the last bits of a
 * sequence's O depend on the sizes and lengths of its batch, but never on the
 * other sequences' values, nor on what ran before.
 *
 * The three tables are in device memory and read by the kernels only, so a
 * captured graph follows them: one capture serves every step as long as the
 * sizes in this struct stay.  Each kernel checks the entries that it uses: one
 * out of range (a page outside the cache, lengths that are negative or exceed
 * max_pages * page_size, starts that are negative, decrease or exceed n_tokens)
 * writes ATTN_CORE_ERR_DEVICE_TABLE to dev_status, touches nothing outside the
 * tensors, and leaves that sequence's results undefined.  Starts that decrease
 * leave every sequence's results undefined; the append then writes nothing.
 *
 * One limit on sizes: ceil(n_tokens / floor(128 / group)) * ceil(max_pages *
 * page_size / 128) < 2^31, group = h_q / h_kv (ATTN_CORE_ERR_UNSUPPORTED). */
typedef struct {
    int32_t n_seq;          /* >= 1 */
    int32_t n_tokens;       /* rows of q and o; 0: nothing to do */
    int32_t h_q, h_kv, d;   /* h_q % h_kv == 0, h_q / h_kv <= 128, h_q + 2 h_kv <= 65535,
                               d in {64, 96, 128, 160} */
    int32_t page_size;      /* 16, 32, 64, 128 or 256 */
    int32_t n_pages;        /* pages in the cache */
    int32_t max_pages;      /* entries per sequence in page_table */
    int32_t causal;         /* 0 or 1 */
    float scale;            /* score scale; <= 0 selects 1/sqrtf(d) */
    const int32_t* cu_seqlens_q;   /* device [n_seq + 1], from 0, nondecreasing */
    const int32_t* kv_lens;        /* device [n_seq] */
    const int32_t* page_table;     /* device [n_seq, max_pages] */
    int32_t* dev_status;           /* as attn_core_params; may be NULL */
    int32_t flags;                 /* 0 or ATTN_CORE_FLAG_TEST_WAIT_TIMEOUT */
    uint32_t wait_timeout_ms;      /* limit of each in-kernel wait; 0 selects 2000 ms */
} attn_core_paged_params;

/* Adds the new tokens to the cache, rotating Q and K on the way (`t`; NULL for
 * no rotation, its d must equal p's): writes q_out [n_tokens, h_q, d] and the
 * new tokens' rows of the pages, nothing else.  strides (host; NULL for packed
 * tensors): elements from one token to the next of q, k and v, multiples of 8
 * -- slices of a fused [tokens, (h_q + 2 h_kv) d] projection qualify.  q and
 * q_out may both be NULL (only the cache is written), and q_out may be q if q
 * is packed.  No two new tokens may share a cache row (a page that two
 * sequences share is copied before either appends to it).  kv_lens[i] counts
 * the new tokens: where it is smaller than their number (which the attention
 * takes, for rows that see no key), the tokens before position 0 have no place
 * in the cache and are a table error.  One kernel. */
int attn_core_paged_append(const attn_core_paged_params* p, const attn_core_rope_table* t, const void* q,
                           const void* k, const void* v, const int64_t* strides, void* q_out, void* k_pages,
                           void* v_pages, void* stream);

/* Attention of the new tokens over the cache (which already holds their own
 * keys and values): O and LSE, which overlap no input.  `workspace`:
 * caller-owned device memory of at least attn_core_paged_workspace_bytes(p)
 * bytes (it depends on d alone: 21 MB at d = 128), 256-byte aligned, for the
 * partial results of rows whose keys are shared out among thread blocks.  Its
 * contents on entry do not matter; calls (or graph replays) that may overlap on
 * the GPU need one each.  One kernel, where tiles may be cut a second one that
 * joins their parts, and where they may be handed out whole a 4-byte memset
 * before.  Nothing is summed in an order that depends on timing:
 * the same inputs give the same bits on the same device. */
size_t attn_core_paged_workspace_bytes(const attn_core_paged_params* p);
int attn_core_paged_fwd(const attn_core_paged_params* p, const void* q, const void* k_pages, const void* v_pages,
                        void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* attn_core_paged_fwd where sequences share their first pages (forks of one
 * prompt): group g is the sequences group_starts[g] .. group_starts[g + 1] - 1,
 * whose page_table rows name the same pages in their first prefix_pages[g]
 * columns (only one row's entries are read there).  The shared keys are
 * visited once for all rows of the group instead of once for each sequence;
 * O and LSE are those of attn_core_paged_fwd up to rounding (with at least as
 * many terms of P; the last bits of a row depend on its group's other rows too,
 * whose maxima move together).  Both tables are
 * in device memory (group_starts [n_groups + 1], prefix_pages [n_groups]) and
 * followed by captured graphs; groups may be empty, and sequences outside all
 * groups share nothing.  Of a group's pages those count that all its sequences
 * (which have new tokens) hold before their first new token, so a count beyond
 * their lengths does no harm, nor does one that is smaller than what they
 * share, 0 among them.  A count beyond the columns in which the rows really
 * agree is not noticed: the sequences then attend to another one's keys there.
 * So counts are lowered, under a captured graph too, whenever a row's page is
 * replaced (copied before a write, or moved by an eviction).  Groups that are
 * out of order or range write ATTN_CORE_ERR_DEVICE_TABLE to dev_status and
 * share nothing.  1 <= n_groups <= n_seq.  The workspace holds the rows of
 * shared and own keys in fp32 until they are joined, and the parts of sequences
 * of few rows: about 8 n_tokens h_q (d + 3) + 123000 d bytes more than
 * attn_core_paged_fwd's (16 MB more at d = 128 for a few tokens).  Two to four
 * kernels; the same inputs give the same bits. */
size_t attn_core_paged_prefix_workspace_bytes(const attn_core_paged_params* p, int32_t n_groups);
int attn_core_paged_prefix_fwd(const attn_core_paged_params* p, int32_t n_groups, const int32_t* group_starts,
                               const int32_t* prefix_pages, const void* q, const void* k_pages, const void* v_pages,
                               void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The attention weight that each key has gathered, by which keys are evicted:
 *   weights_out[i, g, j] = (j < kv_lens[i] - n ? decay weights[i, g, j] : 0)
 *       + sum over the n new tokens t of sequence i that see key j and the
 *         query heads h of KV head g: exp(scale q[t, h] . k[j] - lse[h, t]),
 * j < kv_lens[i], with the lse that attn_core_paged_fwd (or _prefix_fwd) of the
 * same p, q and cache returned.  fp32 [n_seq, h_kv, max_pages * page_size],
 * each sequence its own row also where sequences share pages; weights_out may
 * be weights, but must not overlap it otherwise.  The new tokens' own keys
 * start at 0 whatever weights holds there.  Entries from kv_lens[i] on, and
 * sequences without new tokens, are left as they were.  A row whose lse is
 * -inf adds nothing; one whose lse is NaN makes the weights of all keys that
 * it sees NaN.  decay is finite and not negative.  One kernel, where items of
 * keys may be cut a second one that adds their parts; the same inputs give
 * the same bits.  The workspace (256-byte aligned) is 0.3 MB: that of
 * attn_core_paged_fwd serves. */
size_t attn_core_paged_weights_workspace_bytes(const attn_core_paged_params* p);
int attn_core_paged_weights(const attn_core_paged_params* p, const void* q, const void* k_pages, const float* lse,
                            float decay, const float* weights, float* weights_out, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Eviction by gathered weight.  Of the kv_lens[i] keys of sequence i, m =
 * min(keep[i], kv_lens[i]) stay, for each KV head its own: the last r =
 * min(recent, m), the first f = min(first, m - r), and of those between the
 * m - r - f of largest weight (ties to the lower index; NaN is below all).
 * They keep their order and become the keys 0 .. m - 1: key j's row of K and V
 * moves to page out_table[i * max_pages + j / page_size] (device; NULL: the
 * page table itself), its weight to weights_out[i, g, j], and kept[i, g, j] (int32,
 * like the weights) is the key it was.  Entries from m on are left as they
 * were, and so are K and V elsewhere.  kv_lens is the caller's to set to m, for
 * the calls that follow, and a rotation's positions are not the keys' places
 * any more: new tokens are rotated at their own (attn_core_rope_fwd) and
 * appended without a table.
 *
 * Each page that out_table names (in the places of the m keys) is one that no
 * page table of the call names, or the one that the sequence's own names in
 * the same place and no other sequence's does; no two places name one page.
 * So sequences that share pages move to others (PagePool.shrink).  weights_out may be weights.  keep is in device memory
 * and may exceed the length (all keys stay); negative entries, and lengths or
 * pages out of range, are table errors.  p's n_tokens, h_q and cu_seqlens_q are
 * not used (but checked as ever).  Two kernels; the result is exact.  Limits
 * (ATTN_CORE_ERR_UNSUPPORTED): max_pages * page_size <= 2^30, and n_seq h_kv
 * (max_pages page_size / 64 + 2) < 2^30.  The workspace (256-byte aligned) is
 * about n_seq h_kv max_pages page_size / 8 bytes. */
size_t attn_core_paged_evict_workspace_bytes(const attn_core_paged_params* p);
int attn_core_paged_evict(const attn_core_paged_params* p, const int32_t* keep, int32_t first, int32_t recent,
                          const int32_t* out_table, void* k_pages, void* v_pages, const float* weights,
                          float* weights_out, int32_t* kept, void* workspace, size_t workspace_bytes, void* stream);

/* Copies pages inside a cache: page pairs[2i + 1] <- page pairs[2i], in every
 * plane (one per layer and per K or V; a plane holds n_pages pages of
 * page_bytes and starts plane_stride bytes after the one before).  Forking a
 * sequence copies its last, partly filled page; compaction moves pages to the
 * free places of lower number.  `pairs` is a host array, consumed by the call
 * (a captured graph keeps the copies it was captured with).  The copies run in
 * no order, so each target is named once and is no copy's source: anything
 * else is refused.  page_bytes and plane_stride are multiples of 16. */
int attn_core_page_copy(void* pages, int64_t n_planes, int64_t plane_stride, int64_t n_pages, int64_t page_bytes,
                        const int32_t* pairs, int64_t n_pairs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_CORE_H */
