/*
 * gdn.h -- C ABI of libgdn.so: the chunked gated delta rule (Gated DeltaNet) on
 * AMD Instinct MI355X (gfx950).
 *
 * The operation.  Per sequence and head, with a d_k x d_v state S (initial
 * value S0, or zero) and for every token t in order:
 *
 *     S <- exp(g_t) * S                         forget
 *     e  = beta_t * (v_t - S^T k_t)             error of what is stored under k_t
 *     S <- S + k_t e^T                          write
 *     o_t = scale * S^T q_t                     read with the query, after the write
 *
 * This is the update of "Research Sprint Day 1 - Verifying the
 * flash-linear-attention Gated DeltaNet kernel on GB10", section "The GDN update",
 * with alpha = exp(g) kept in log space as on "Research Sprint Day 2 - Rooflines",
 * section "Building some intuition" (gates, step 5).  Its closed form on the
 * Day-2 page is S'_t = S'_{t-1} alpha_t (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 * with S' = S^T.  `scale` is the query scale that the cuLA issue #126 page
 * ("Minimal public reproduction") passes to its kernels as a separate argument.
 *
 * gdn_chunk_fwd / gdn_chunk_bwd evaluate this in chunks of 64 tokens (the
 * "chunk_gated_delta_rule" of the Day-1 page, "Conclusion"; intermediates of the
 * fla issue #1550 page, "Intermediate rounding diagnosis").  gdn_recurrent_ref
 * runs the token loop itself in IEEE fp32 (the "fused recurrent operator" of the
 * fla issue #1550 page, "Reproduction and evidence").
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - Tensors are dense, row-major, last dimension contiguous, on the device:
 *      q, k              [B, T, H, Dk]     io dtype
 *      v, o, dO, dv      [B, T, H, Dv]     io dtype
 *      dq, dk            [B, T, H, Dk]     io dtype
 *      g, beta, dg, dbeta[B, T, H]         fp32
 *      S0, S_final, dS_final, dS0
 *                        [N, H, Dk, Dv]    fp32  (N = number of sequences)
 *  - Packed variable-length sequences (fla issue #1550 page: sequence lengths
 *    [5120, 5120] in one row): B must be 1 and sequence n is tokens
 *    [cu[n], cu[n+1]) of the row.  Chunks restart at every sequence start; each
 *    sequence has its own S0 / S_final.  The caller passes the offsets twice:
 *    on the host (validated before any launch) and as a device copy holding the
 *    same values (read by the kernels).  Dense input: both NULL, N = B.
 *  - The value domain is documented, not checked: g <= 0 (alpha = exp(g) in
 *    (0, 1]), beta in (0, 2) (Day-2 page: beta = 2 sigmoid(.) under
 *    allow_neg_eigval), k rows L2-normalised.  NaN and Inf propagate.
 *  - Ownership: the caller allocates every buffer, including the workspace
 *    sized by gdn_workspace_size.  The library allocates nothing, keeps no state
 *    between calls and never synchronises the host -- except
 *    gdn_chunk_fwd_noalloc, whose workspace is a fixed device array the library
 *    holds (see there).
 *  - Execution: asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream).  Outputs are always overwritten, never accumulated.
 *  - Errors: every shape, pointer, dtype, support and workspace check happens on
 *    the host before the first launch, so an error leaves every output untouched.
 *    GDN_ERR_HIP reports a failed launch (hipGetLastError).  There is no silent
 *    fallback: an unsupported case is an error.
 *  - Precision (explicit, never switched by environment variables):
 *      io dtype GDN_FP32: every product in IEEE fp32 (fp32 MFMA), fp32 state.
 *      io dtype GDN_BF16: bf16 MFMA operands with fp32 accumulation; the state,
 *        the decay factors, the triangular solve and all gradients' reductions
 *        are fp32; outputs are rounded to bf16 (round to nearest even) once.
 *  - Supported: Dk in {64, 128};
 *    Dv a multiple of 16 with 16 <= Dv <= 256; chunk == 64; num_segments in
 *    {1, 2, 4, 8, 16}; N <= 65535.  The recurrent backward needs
 *    2 * Dk * (Dv + 1) * 4 bytes of LDS and so Dk * Dv <= 128 * 128.
 *  - All entry points are thread-safe.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The operators of the layer (gdn_step and all that follows it below) are additions within
 * version 6: the number does not tell whether a library has them, their symbols do. */
#define GDN_ABI_VERSION 6

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_NULL = 1,        /* a required pointer is NULL                               */
  GDN_ERR_SHAPE = 2,       /* a size is out of range or inconsistent                   */
  GDN_ERR_DTYPE = 3,       /* io_dtype is not a gdn_dtype                              */
  GDN_ERR_UNSUPPORTED = 4, /* valid but not built: Dk, Dv, chunk or num_segments       */
  GDN_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than gdn_workspace_size        */
  GDN_ERR_ALIAS = 6,       /* an output overlaps an input or another output            */
  GDN_ERR_HIP = 7,         /* a HIP launch failed                                      */
  GDN_ERR_SEQLENS = 8,     /* cu_seqlens not 0 = cu[0] <= cu[1] <= ... <= cu[N] = T     */
  GDN_ERR_ALIGN = 9,       /* q, k, v, o, dO, dq, dk, dv not 16-byte aligned, or an fp32
                              tensor not 4-byte aligned                                 */
  GDN_ERR_SCRATCH = 10     /* gdn_chunk_fwd_noalloc: the problem needs more workspace than
                              GDN_NOALLOC_SCRATCH_BYTES                                 */
} gdn_status;

typedef enum gdn_dtype { GDN_FP32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* Precision policy of the chunked products (the fla issue #1550 page, "Proposed
 * scope", asks for a policy for the score and WY intermediates that keeps the
 * public dtypes, chosen on measured latency and memory):
 *   GDN_PRECISION_IO   the io dtype decides: bf16 io -> bf16 MFMA operands (the
 *                      inverse T diag(beta), the score P, R, E and the state
 *                      operand rounded to bf16) with fp32 accumulation, state and
 *                      decays; fp32 io -> every product in IEEE fp32.
 *   GDN_PRECISION_FP32 every product in IEEE fp32 (fp32 MFMA) whatever the io
 *                      dtype: bf16 inputs are widened exactly, o is rounded to
 *                      bf16 once, the per-chunk workspace records are fp32.
 *                      gdn_chunk_fwd only (gdn_chunk_bwd, gdn_kda_chunk_fwd and
 *                      gdn_kda_chunk_bwd with bf16 io return GDN_ERR_UNSUPPORTED
 *                      for it). */
typedef enum gdn_precision { GDN_PRECISION_IO = 0, GDN_PRECISION_FP32 = 1 } gdn_precision;

typedef enum gdn_pass {
  GDN_PASS_CHUNK_FWD = 0,
  GDN_PASS_CHUNK_BWD = 1,
  GDN_PASS_RECURRENT_FWD = 2,
  GDN_PASS_RECURRENT_BWD = 3,
  GDN_PASS_KDA_FWD = 4,
  GDN_PASS_CHUNK_SAVED = 5, /* the buffer of gdn_chunk_fwd_save / gdn_chunk_bwd_saved */
  GDN_PASS_KDA_BWD = 6,
  GDN_PASS_KDA_SAVED = 7    /* the buffer of gdn_kda_chunk_fwd_save / gdn_kda_chunk_bwd_saved */
} gdn_pass;

typedef struct gdn_problem {
  int32_t B, T, H, Dk, Dv;         /* sizes; T may be 0                                     */
  int32_t num_seqs;                /* N: == B for dense input, else len(cu_seqlens) - 1     */
  const int32_t* cu_seqlens_host;  /* host, N + 1 offsets, or NULL (dense)                  */
  const int32_t* cu_seqlens_dev;   /* device copy of the same N + 1 values, or NULL         */
  int32_t io_dtype;                /* gdn_dtype of q, k, v, o, dO, dq, dk, dv               */
  float scale;                     /* output scale: o_t = scale * S_t^T q_t                 */
  int32_t chunk;                   /* tokens per chunk; must be 64                          */
  int32_t num_segments;            /* 1: serial over chunks; G > 1: segment split (fwd)     */
  int32_t precision;               /* gdn_precision of the chunked products                 */
} gdn_problem;

/* Version of this ABI (GDN_ABI_VERSION). */
int32_t gdn_abi_version(void);

/* Static string naming a status code; never NULL. */
const char* gdn_status_str(int32_t status);

/* Bytes of device workspace that `pass` needs for `problem` (0 is possible; the
 * workspace pointer may then be NULL).  Validates the problem like the entry
 * point it sizes for. */
gdn_status gdn_workspace_size(const gdn_problem* problem, int32_t pass, size_t* bytes);

/* Forward pass of the chunked gated delta rule.
 *   in : q, k, v, g, beta; S0 (NULL = zero initial state)
 *   out: o; S_final (NULL = not wanted)
 * Chunk algebra per (sequence, head), chunk of n <= 64 tokens, state S_c before it:
 *   gamma = cumsum(g) within the chunk; D_ij = exp(gamma_i - gamma_j) (j <= i)
 *   A = strict_lower(diag(beta) (K K^T) o D); T = (I + A)^-1 (unit lower triangular)
 *   E = T diag(beta) (V - diag(exp(gamma)) K S_c)      (the errors e_t of the chunk)
 *   O = scale (diag(exp(gamma)) Q S_c + lower_incl(Q K^T o D) E)
 *   S_{c+1} = exp(gamma_n) S_c + (diag(exp(gamma_n - gamma)) K)^T E
 * num_segments = G > 1 splits every sequence of nch chunks into G runs of whole
 * chunks (segment s covers chunks [s L, min((s + 1) L, nch)), L = ceil(nch / G))
 * that run in parallel: each segment's state map S -> M S + b is taken by the
 * same chunk pass (b from a zero start, M from the identity with V = 0), the
 * start states are composed in fp32 in segment order, and the segments are run
 * again from them with their outputs (cuLA issue #126 page, "Summary" and
 * "Hypothesis": segment affine transforms and carries).  G = 2 gives results
 * bit-identical to G = 1; G > 2 agrees to the bf16 rounding of M's operands.
 * Workspace: gdn_workspace_size(..., GDN_PASS_CHUNK_FWD, ...): per chunk and
 * head, T diag(beta) (its 16x16 blocks on and below the diagonal), the causal
 * score and the chunk's decays, plus for G > 1 fp32 buffers of
 * 2 G N H Dk Dv + G N H Dk Dk floats. */
gdn_status gdn_chunk_fwd(const gdn_problem* problem, const void* q, const void* k,
                         const void* v, const float* g, const float* beta, const float* S0,
                         void* o, float* S_final, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Size of the device array that gdn_chunk_fwd_noalloc uses as its workspace
 * (64 MiB: the bf16 forward of 4 x 4096 tokens x 8 heads at Dk = Dv = 128 needs
 * about 30 MiB). */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* gdn_chunk_fwd without a caller-provided workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, serving loops or
 * harnesses that forbid allocation).  Same arguments, results and kernels as
 * gdn_chunk_fwd; the workspace is a file-scope device array of
 * GDN_NOALLOC_SCRATCH_BYTES that the library holds on every device it runs on
 * until the process ends.  The call allocates nothing: the array's device
 * address is looked up once per device (on the first call with that device
 * current; the current device must be the one `stream` belongs to).
 *   Errors: as gdn_chunk_fwd, plus GDN_ERR_SCRATCH (before any launch) when
 *   gdn_workspace_size(problem, GDN_PASS_CHUNK_FWD) exceeds the array, and
 *   GDN_ERR_HIP if the address lookup fails.
 *   Concurrency: every call on one device shares that device's array, which
 *   keeps the last call's contents (nothing in it has to start at zero).  Calls
 *   whose executions overlap on one device -- different streams, or different
 *   host threads -- race on the array and give undefined results; serialise
 *   them (one stream, or events). */
gdn_status gdn_chunk_fwd_noalloc(const gdn_problem* problem, const void* q, const void* k,
                                 const void* v, const float* g, const float* beta, const float* S0,
                                 void* o, float* S_final, void* stream);

/* Backward pass of the chunked gated delta rule: gradients of
 *   L = <o, dO> + <S_final, dS_final>
 * with respect to q, k, v, g, beta and S0 (the six gradients of the Day-1 page's
 * "Results" tables plus the initial-state gradient).
 *   in : q, k, v, g, beta, S0 (NULL = zero), dO, dS_final (NULL = zero)
 *   out: dq, dk, dv (io dtype), dg, dbeta (fp32), dS0 (fp32; NULL = not wanted)
 * num_segments must be 1.  Workspace: GDN_PASS_CHUNK_BWD (T, T diag(beta), the
 * decays and the causal score P of every chunk, and the state before and its
 * gradient after every chunk, held in the products' operand type: bf16 for bf16
 * io, fp32 for fp32 io, the type in which the gradient products consume them). */
gdn_status gdn_chunk_bwd(const gdn_problem* problem, const void* q, const void* k,
                         const void* v, const float* g, const float* beta, const float* S0,
                         const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                         float* dg, float* dbeta, float* dS0, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Training with retained states: the forward keeps what the backward needs, so
 * the backward does not run the forward's state pass again (the fla issue #1550
 * page, "Proposed scope", asks for retained or recomputed states as a measured
 * choice; gdn_chunk_bwd is the recomputing one).
 *
 * gdn_chunk_fwd_save computes exactly what gdn_chunk_fwd computes (o, S_final;
 * the same arithmetic, so bit-identical results) and also fills `saved` with
 * T, T diag(beta), the decays and the causal score P of every chunk and the state
 * before every chunk (in the operand type, as for gdn_chunk_bwd).  gdn_chunk_bwd_saved then runs only the reverse
 * passes of gdn_chunk_bwd and gives bit-identical gradients, provided q, k, v, g,
 * beta, S0 and the problem are the same as in the gdn_chunk_fwd_save call and
 * `saved` was not modified in between (neither is checked: other contents give
 * undefined gradients, not an error).  gdn_chunk_bwd_saved writes the state
 * gradients into `saved` as well; `saved` may be reused for the next step.
 *   saved: caller-allocated device buffer of gdn_workspace_size(problem,
 *          GDN_PASS_CHUNK_SAVED) bytes (the backward workspace plus P in the
 *          forward's operand order), 16-byte aligned.
 *   Supported and errors: as gdn_chunk_bwd (num_segments 1, precision IO).
 *   S0 is not an argument of gdn_chunk_bwd_saved (the saved states carry it);
 *   dS0 is still produced. */
gdn_status gdn_chunk_fwd_save(const gdn_problem* problem, const void* q, const void* k,
                              const void* v, const float* g, const float* beta, const float* S0,
                              void* o, float* S_final, void* saved, size_t saved_bytes,
                              void* stream);
gdn_status gdn_chunk_bwd_saved(const gdn_problem* problem, const void* q, const void* k,
                               const void* v, const float* g, const float* beta, const void* dO,
                               const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                               float* dbeta, float* dS0, void* saved, size_t saved_bytes,
                               void* stream);

/* Token-by-token recurrence in IEEE fp32 on the GPU: the full-length second
 * reference (not the fast path).  Forward always (o, S_final as gdn_chunk_fwd).
 * If dO is non-NULL it also runs the token-level reverse mode and writes dq, dk,
 * dv, dg, dbeta (all required then) and dS0 (optional), like gdn_chunk_bwd.
 * num_segments is ignored.  Workspace: GDN_PASS_RECURRENT_FWD when dO == NULL,
 * else GDN_PASS_RECURRENT_BWD. */
gdn_status gdn_recurrent_ref(const gdn_problem* problem, const void* q, const void* k,
                             const void* v, const float* g, const float* beta,
                             const float* S0, void* o, float* S_final, const void* dO,
                             const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                             float* dbeta, float* dS0, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Chunked forward pass with one log-decay per key channel: the gate layout of
 * the cuLA issue #126 page ("Minimal public reproduction", where g has the shape
 * of q and is handed to the KDA kernels).  Per token, with a = exp(g_t) a vector
 * of Dk factors:  S <- diag(a) S,  e = beta (v - S^T k),  S <- S + k e^T,
 * o = scale S^T q  (the update of "Research Sprint Day 1", "The GDN update",
 * with a diagonal forget factor; with equal factors on every channel it is
 * gdn_chunk_fwd's recurrence).
 *   in : q, k [B,T,H,Dk] and v [B,T,H,Dv] (io dtype); g [B,T,H,Dk] fp32, finite
 *        and <= 0; beta [B,T,H] fp32; S0 [N,H,Dk,Dv] fp32 or NULL (zero)
 *   out: o [B,T,H,Dv] (io dtype), S_final [N,H,Dk,Dv] fp32 or NULL
 * Packed sequences through cu_seqlens as for gdn_chunk_fwd.  Dk 64 or 128 and
 * Dv a multiple of 16 up to 256, for both io dtypes.  num_segments in {1, 2, 4,
 * 8, 16}: the segment split of gdn_chunk_fwd (segment maps S -> M S + b, M a
 * Dk x Dk matrix, composed in fp32; G = 2 and the first two segments are
 * bit-identical to G = 1) -- the intra-card split whose error the cuLA issue
 * #126 page measures ("Summary").
 * Precision: decays, A, the inverse and the state are fp32; the products take
 * bf16 operands with fp32 accumulation for bf16 io and are IEEE fp32 for fp32 io.
 * Workspace: gdn_workspace_size(..., GDN_PASS_KDA_FWD, ...): one record per chunk
 * and head (T diag(beta), the causal score, K and Q scaled by the decays, the
 * decayed keys of the state update, in the io element type; the chunk's decay),
 * then for G > 1 fp32 buffers of 2 G N H Dk Dv + G N H Dk Dk floats.  Errors as gdn_chunk_fwd: every check
 * runs before the first launch. */
gdn_status gdn_kda_chunk_fwd(const gdn_problem* problem, const void* q, const void* k,
                             const void* v, const float* g, const float* beta, const float* S0,
                             void* o, float* S_final, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Reverse mode of gdn_kda_chunk_fwd: the gradients of
 *   L = <o, dO> + <S_final, dS_final>
 * with respect to q, k, v, the per-channel log-decays g, beta and S0, for the
 * recurrence of gdn_kda_chunk_fwd (per token, a = exp(g_t) of length Dk:
 * S <- diag(a) S, e = beta (v - S^T k), S <- S + k e^T, o = scale S^T q; the
 * update of "Research Sprint Day 1", "The GDN update", with the diagonal forget
 * factor of the cuLA issue #126 page's gate layout).
 *   in : q, k, v, g, beta, S0 (NULL = zero) as gdn_kda_chunk_fwd; dO [B,T,H,Dv]
 *        (io dtype); dS_final [N,H,Dk,Dv] fp32 or NULL (zero)
 *   out: dq, dk [B,T,H,Dk] and dv [B,T,H,Dv] (io dtype); dg [B,T,H,Dk] fp32 (one
 *        gradient per key channel); dbeta [B,T,H] fp32; dS0 [N,H,Dk,Dv] fp32
 *        (NULL = not wanted)
 * The forward's chunk preparation and state pass run again (no o is written);
 * then a reverse pass over the chunks forms the state gradient after every
 * chunk, and one workgroup per chunk forms its gradients.  Packed sequences as
 * for gdn_kda_chunk_fwd; Dk 64 or 128, Dv a multiple of 16 up to 256, both io
 * dtypes; num_segments must be 1 and precision GDN_PRECISION_IO.
 * Precision: decays, the inverse, the state and its gradient are fp32; the
 * products take bf16 operands with fp32 accumulation for bf16 io (the records,
 * the per-chunk states and state gradients, and the intermediate tiles rounded to
 * bf16) and are IEEE fp32 for fp32 io; the pair sums through the per-channel
 * decays are fp32 for both.
 * Workspace: gdn_workspace_size(..., GDN_PASS_KDA_BWD, ...): the forward's records,
 * then per chunk and head 12288 floats (T, Ab, P in fp32) and the state before and
 * its gradient after the chunk, Dk Dv values each in the io element type.  Errors
 * as gdn_kda_chunk_fwd. */
gdn_status gdn_kda_chunk_bwd(const gdn_problem* problem, const void* q, const void* k,
                             const void* v, const float* g, const float* beta, const float* S0,
                             const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                             float* dg, float* dbeta, float* dS0, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Training with retained states for the per-channel decay, as gdn_chunk_fwd_save /
 * gdn_chunk_bwd_saved for the scalar gate (the fla issue #1550 page, "Proposed
 * scope": retained or recomputed states).  gdn_kda_chunk_fwd_save computes exactly
 * what gdn_kda_chunk_fwd computes with num_segments = 1 (o, S_final; bit-identical)
 * and also fills `saved` with the chunk records, fp32 T, Ab and P, and the state
 * before every chunk; gdn_kda_chunk_bwd_saved then runs only the reverse passes of
 * gdn_kda_chunk_bwd and gives bit-identical gradients, provided q, k, v, g, beta, S0
 * and the problem are those of the save call and `saved` was not modified in
 * between (neither is checked: other contents give undefined gradients, not an
 * error).  It writes the state gradients into `saved` as well.
 *   saved: caller-allocated device buffer of gdn_workspace_size(problem,
 *          GDN_PASS_KDA_SAVED) bytes (the gdn_kda_chunk_bwd workspace), 16-byte
 *          aligned.
 *   Supported and errors: as gdn_kda_chunk_bwd.  S0 is not an argument of
 *   gdn_kda_chunk_bwd_saved (the saved states carry it); dS0 is still produced. */
gdn_status gdn_kda_chunk_fwd_save(const gdn_problem* problem, const void* q, const void* k,
                                  const void* v, const float* g, const float* beta, const float* S0,
                                  void* o, float* S_final, void* saved, size_t saved_bytes,
                                  void* stream);
gdn_status gdn_kda_chunk_bwd_saved(const gdn_problem* problem, const void* q, const void* k,
                                   const void* v, const float* g, const float* beta, const void* dO,
                                   const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                                   float* dbeta, float* dS0, void* saved, size_t saved_bytes,
                                   void* stream);

/* Gate forms of gdn_prologue. */
typedef enum {
  GDN_GATE_GDN = 0,         /* g = -exp(A_log[h]) * softplus(a + dt_bias[h])            */
  GDN_GATE_BOUNDED5 = 1,    /* g = -5 * sigmoid(a), in (-5, 0)                          */
  GDN_GATE_GDN_CHANNEL = 2  /* g[..., c] = -exp(A_log[h]) * softplus(a[..., c] + dt_bias[h, c]) */
} gdn_gate_kind;

/* Fused input prologue: the elementwise step that produces the operator's inputs
 * from the raw projections, in one pass over HBM.
 *   q_out = q / max(||q||_2, 1e-30), k_out = k / max(||k||_2, 1e-30): norms over
 *           the last dimension in fp32 from the io-dtype inputs, then rounded to
 *           the io dtype (round to nearest even).  The fla issue #1550 page
 *           ("Proposed scope") asks for exactly this order: normalise in FP32,
 *           then cast.
 *   beta  = sigmoid(b), or 2 sigmoid(b) when allow_neg_eigval != 0 (the range
 *           (0, 2) of the Day-2 page, "Building some intuition", gates).
 *   g     = -exp(A_log[h]) softplus(a + dt_bias[h])   (GDN_GATE_GDN: the gate
 *           formula of the Day-2 page, "Building some intuition", steps 4-5), or
 *           -5 sigmoid(a)                              (GDN_GATE_BOUNDED5: the
 *           bounded gates of the fla issue #1550 workload), or the first form
 *           channel by channel, one log-decay per key channel for
 *           gdn_kda_chunk_fwd (GDN_GATE_GDN_CHANNEL: the gate layout of the cuLA
 *           issue #126 page, "Minimal public reproduction", dt_bias per head and
 *           channel).
 * Shapes: q, k, q_out, k_out [B, T, H, Dk] io dtype; b, beta [B, T, H] fp32; a, g
 * [B, T, H] fp32, or [B, T, H, Dk] for GDN_GATE_GDN_CHANNEL; A_log [H] fp32 and
 * dt_bias [H] fp32, or [H, Dk] for GDN_GATE_GDN_CHANNEL (both required for the
 * two GDN forms, ignored for GDN_GATE_BOUNDED5).
 * `problem` is the problem of the chunked call the outputs feed (only B, T, H,
 * Dk and io_dtype are used; it is validated as for gdn_recurrent_ref).  Outputs
 * must not overlap inputs (GDN_ERR_ALIAS).  No workspace.  In fp32 the results
 * are the correctly computed fp32 expressions up to a few units of the last
 * place (the exponentials and the division). */
gdn_status gdn_prologue(const gdn_problem* problem, const void* q, const void* k, const float* a,
                        const float* b, const float* A_log, const float* dt_bias, int32_t gate_kind,
                        int32_t allow_neg_eigval, void* q_out, void* k_out, float* g, float* beta,
                        void* stream);

/* Output epilogue: the gated, normalised output the operator's result feeds,
 * in one pass over HBM ("Research Sprint Day 2", "Building some intuition",
 * step 7: normalise per head, then gate):
 *   y = o / sqrt(mean_j(o_j^2) + eps) * weight * silu(z),  silu(z) = z sigmoid(z)
 * per (token, head) over the Dv values, in fp32, rounded once to the io dtype.
 * Shapes: o, z, y [B, T, H, Dv] io dtype; weight [Dv] fp32, 16-byte aligned (NULL =
 * all ones).
 * eps >= 0 is documented, not checked.  `problem` is that of the chunked call
 * that produced o (B, T, H, Dv and io_dtype are used; validated as for
 * gdn_recurrent_ref); Dv must be a power of two (16 .. 256), else
 * GDN_ERR_UNSUPPORTED.  y must not overlap o or z (GDN_ERR_ALIAS).  No workspace. */
gdn_status gdn_epilogue(const gdn_problem* problem, const void* o, const void* z, const float* weight,
                        float eps, void* y, void* stream);

/* Measurement helper, not part of the operator: copies `bytes` bytes of device
 * memory from src to dst (16-byte vectors, non-temporal, grid-strided), the copy
 * that calibrates the HBM roofline the chunked kernels are measured against
 * ("Research Sprint Day 2 - Rooflines", section "Rooflines": the bandwidth of a
 * large copy, bytes read plus bytes written).  dst, src and bytes must be
 * multiples of 16 (GDN_ERR_ALIGN), the ranges must not overlap (GDN_ERR_ALIAS);
 * asynchronous on `stream`. */
gdn_status gdn_device_copy(void* dst, const void* src, size_t bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The operators around and beside the chunked delta rule in a layer: its
 * single-token step, the short causal convolution in front of it, and the
 * selective state space scan.  The conventions above hold (ownership, streams,
 * errors, packed sequences); what differs is said at each entry point.
 * ------------------------------------------------------------------------- */

/* One token of the gated delta rule for every sequence of a batch (decoding):
 *     S <- exp(g) S;  e = beta (v - S^T k);  S <- S + k e^T;  o = scale S^T q
 * with the state updated in place.  `problem` is dense with T == 1 (num_seqs ==
 * B; GDN_ERR_SHAPE otherwise); chunk, num_segments and precision are checked as
 * for gdn_recurrent_ref and not used.
 *   in    : q, k [B,1,H,Dk], v [B,1,H,Dv] (io dtype); g, beta [B,1,H] fp32
 *   in/out: S [B,H,Dk,Dv] fp32, 16-byte aligned
 *   out   : o [B,1,H,Dv] (io dtype)
 * All arithmetic is fp32 whatever the io dtype; o is rounded once.  B H ceil(Dv / 32)
 * < 2^24 (else GDN_ERR_UNSUPPORTED).  No output may
 * overlap another tensor (GDN_ERR_ALIAS).  No workspace. */
gdn_status gdn_step(const gdn_problem* problem, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, float* S, void* o, void* stream);

/* gdn_step with one log-decay per key channel (the recurrence of
 * gdn_kda_chunk_fwd): g [B,1,H,Dk] fp32, 4-byte aligned. */
gdn_status gdn_kda_step(const gdn_problem* problem, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, float* S, void* o, void* stream);

typedef enum gdn_activation { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

/* Short causal depthwise convolution over the tokens of every sequence:
 *     p_t[c] = bias[c] + sum_{j=0}^{W-1} weight[c][j] x_{t-(W-1)+j}[c]
 *     y_t = p_t (GDN_ACT_NONE)  or  p_t sigmoid(p_t) (GDN_ACT_SILU)
 * where the W - 1 rows before a sequence are its state (zero without one).
 * Tensors: x, y, dy, dx [B,T,C]; state0, state_final, state, dstate_final, dstate0
 * [N,W-1,C], oldest row first (io dtype; state rows are input rows, kept exactly);
 * weight, dweight [C,W] and bias, dbias [C] fp32.  All of them 16-byte aligned.
 * Supported: C a multiple of 8 up to 2^20, W in {2, 3, 4}, N <= 65535, B T < 2^31, and
 * B T C / 32 + N (W - 1) C / V <= 2^32 - 2^23 (the threads of a launch; V = 8 for bf16, 4
 * for fp32), else GDN_ERR_UNSUPPORTED.  Sums are fp32; io outputs are rounded once. */
typedef struct gdn_conv_problem {
  int32_t B, T, C, W;
  int32_t num_seqs;                /* N: == B for dense input, else len(cu_seqlens) - 1     */
  const int32_t* cu_seqlens_host;  /* host, N + 1 offsets, or NULL (dense)                  */
  const int32_t* cu_seqlens_dev;   /* device copy of the same N + 1 values, or NULL         */
  int32_t io_dtype;                /* gdn_dtype                                             */
  int32_t activation;              /* gdn_activation; another value: GDN_ERR_UNSUPPORTED    */
} gdn_conv_problem;

/* Forward.  in: x, weight, bias (NULL: none), state0 (NULL: zero);
 * out: y, state_final (NULL: not wanted; the last W - 1 rows of state0 followed by
 * the sequence, so a sequence of no tokens keeps state0).  No workspace. */
gdn_status gdn_conv_fwd(const gdn_conv_problem* problem, const void* x, const float* weight,
                        const float* bias, const void* state0, void* y, void* state_final,
                        void* stream);

/* Bytes of workspace gdn_conv_bwd needs (partial sums of dweight and dbias). */
gdn_status gdn_conv_workspace_size(const gdn_conv_problem* problem, size_t* bytes);

/* Backward: gradients of L = <y, dy> + <state_final, dstate_final>.
 *   in : x, weight, bias, state0 as gdn_conv_fwd; dy; dstate_final (NULL: zero)
 *   out: dx, dweight; dbias and dstate0 (NULL: not wanted)
 * The pre-activation is formed again from x.  dweight and dbias are summed in a
 * fixed order (bit-identical from call to call). */
gdn_status gdn_conv_bwd(const gdn_conv_problem* problem, const void* x, const float* weight,
                        const float* bias, const void* state0, const void* dy,
                        const void* dstate_final, void* dx, float* dweight, float* dbias,
                        void* dstate0, void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (decoding; dense with T == 1): y from the state's
 * rows and x, then the state shifted by one row in place.  y and state must not
 * overlap another tensor.  No workspace. */
gdn_status gdn_conv_step(const gdn_conv_problem* problem, const void* x, const float* weight,
                         const float* bias, void* state, void* y, void* stream);

/* Selective state space scan: per sequence, channel d and state n, with a state
 * h[d][n] (initially h0, or zero) and for every token t in order
 *     delta = softplus(dt_t[d] + dt_bias[d])   (dt_softplus; else dt_t[d] + dt_bias[d])
 *     h[d][n] <- exp(delta A[d][n]) h[d][n] + delta u_t[d] Bm_t[grp(d)][n]
 *     s = sum_n Cm_t[grp(d)][n] h[d][n] + Dskip[d] u_t[d]
 *     y_t[d] = s   or, with z,   s z_t[d] sigmoid(z_t[d])
 * where grp(d) = d / (D / G).  Tensors: u, dt, z, y [B,T,D], Bm, Cm [B,T,G,N] (io
 * dtype); A [D,N], Dskip, dt_bias [D], h0, h_final [num_seqs,D,N] fp32.  All of them
 * 16-byte aligned.  Supported: N in {8, 16, 32, 64}, D / G a multiple of 8, D up to
 * 2^20, B T < 2^31, B T G N < 2^32, up to 65535 sequences, else GDN_ERR_UNSUPPORTED.
 * Finite A <= 0 and delta >= 0 are documented, not checked.  All arithmetic is fp32; io outputs are rounded once.
 * NaN and Inf reach what the definition makes of them and nothing that it leaves finite.  Where it
 * gives an infinity NaN may stand instead: a state that is infinite while the decays over 16
 * tokens or more underflow to zero, and dA where dh_final is infinite and the sequence's length is no
 * multiple of 16. */
typedef struct gdn_scan_problem {
  int32_t B, T, D, N, G;
  int32_t num_seqs;                /* == B for dense input, else len(cu_seqlens) - 1        */
  const int32_t* cu_seqlens_host;  /* host, num_seqs + 1 offsets, or NULL (dense)           */
  const int32_t* cu_seqlens_dev;   /* device copy of the same values, or NULL               */
  int32_t io_dtype;                /* gdn_dtype                                             */
  int32_t dt_softplus;             /* nonzero: delta = softplus(dt + dt_bias)               */
} gdn_scan_problem;

typedef enum gdn_scan_pass {
  GDN_SCAN_FWD = 0,   /* workspace of gdn_scan_fwd and gdn_scan_fwd_save */
  GDN_SCAN_SAVED = 1, /* the `saved` buffer                              */
  GDN_SCAN_BWD = 2    /* workspace of gdn_scan_bwd_saved                 */
} gdn_scan_pass;

/* Bytes of the device buffer `pass` needs (0 is possible; the pointer may then be
 * NULL); GDN_ERR_UNSUPPORTED for another pass.  The sizes depend on the problem's
 * sizes and offsets alone. */
gdn_status gdn_scan_workspace_size(const gdn_scan_problem* problem, int32_t pass, size_t* bytes);

/* Forward.  in: u, dt, A, Bm, Cm; Dskip, z, dt_bias, h0 (each may be NULL: no
 * skip, no gate, no bias, zero); out: y, h_final (NULL: not wanted; a sequence of
 * no tokens keeps h0).  Long sequences with few channels are split over the time
 * axis: segment end states from a zero start are composed in fp32, so results are
 * those of the serial order up to fp32 rounding. */
gdn_status gdn_scan_fwd(const gdn_scan_problem* problem, const void* u, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* Dskip, const void* z,
                        const float* dt_bias, const float* h0, void* y, float* h_final,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Training: gdn_scan_fwd_save computes what gdn_scan_fwd computes (bit-identical)
 * and keeps the state at regular tokens in `saved` (GDN_SCAN_SAVED bytes, 16-byte
 * aligned); gdn_scan_bwd_saved forms from it the gradients of
 *     L = <y, dy> + <h_final, dh_final>.
 * The problem and the inputs must be those of the save call and `saved` unmodified
 * (not checked).  `saved` is only read by the backward.
 *   in : u, dt, A, Bm, Cm, Dskip, z, dt_bias as gdn_scan_fwd; dy; dh_final (NULL: zero)
 *   out: du, ddt, dBm, dCm (io dtype), dA (fp32); dDskip, dz, ddt_bias, dh0 (NULL:
 *        not wanted; dDskip may be asked for without Dskip and ddt_bias without dt_bias;
 *        dz needs z, GDN_ERR_NULL otherwise)
 * Sums over tokens and channels are fp32 in a fixed order (bit-identical from call
 * to call). */
gdn_status gdn_scan_fwd_save(const gdn_scan_problem* problem, const void* u, const void* dt, const float* A,
                             const void* Bm, const void* Cm, const float* Dskip, const void* z,
                             const float* dt_bias, const float* h0, void* y, float* h_final,
                             void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                             void* stream);
gdn_status gdn_scan_bwd_saved(const gdn_scan_problem* problem, const void* u, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const void* dy, const float* dh_final,
                              const void* saved, size_t saved_bytes, void* du, void* ddt, float* dA,
                              void* dBm, void* dCm, float* dDskip, void* dz, float* ddt_bias, float* dh0,
                              void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (decoding; dense with T == 1): y, and the state h
 * [B,D,N] fp32 updated in place.  y and h must not overlap another tensor.  No
 * workspace. */
gdn_status gdn_scan_step(const gdn_scan_problem* problem, const void* u, const void* dt, const float* A,
                         const void* Bm, const void* Cm, const float* Dskip, const void* z,
                         const float* dt_bias, float* h, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * The operators that hybrid models put next to the delta rule: the gated linear
 * recurrence, the norm and rotation of queries and keys, and attention over a
 * sliding window.  The conventions above hold; what differs is said at each entry
 * point.
 * ------------------------------------------------------------------------- */

/* Gated linear recurrence: per sequence and channel, with a state h (initially h0, or
 * zero) and for every token t in order
 *     la = -c softplus(lam) sigmoid(r_t);  a = exp(la)
 *     h <- a h + sqrt(1 - a^2) sigmoid(i_t) x_t
 *     y_t = h   or, with z,   h z_t sigmoid(z_t)
 * Tensors: x, r, i, z, y and their gradients [B,T,C] (io dtype); lam, dlam [C], h0,
 * h_final, dh_final, dh0, h [num_seqs,C] fp32.  All of them 16-byte aligned.  Supported: C a
 * multiple of 8 up to 2^20, B T < 2^31, up to 65535 sequences, c >= 0 and finite, and
 * (B T / 64 + sequences) ceil(C / 64) < 2^24, else GDN_ERR_UNSUPPORTED.  Finite lam is documented,
 * not checked.  All arithmetic is fp32; io outputs are rounded once.  NaN and Inf reach what
 * the definition makes of them and nothing that it leaves finite; where it gives an infinity
 * NaN may stand instead (a state that is infinite while the decays over several tokens
 * underflow to zero). */
typedef struct gdn_glr_problem {
  int32_t B, T, C;
  int32_t num_seqs;                /* == B for dense input, else len(cu_seqlens) - 1        */
  const int32_t* cu_seqlens_host;  /* host, num_seqs + 1 offsets, or NULL (dense)           */
  const int32_t* cu_seqlens_dev;   /* device copy of the same values, or NULL               */
  int32_t io_dtype;                /* gdn_dtype                                             */
  float c;                         /* factor of the log-decay                               */
} gdn_glr_problem;

typedef enum gdn_glr_pass {
  GDN_GLR_FWD = 0,   /* workspace of gdn_glr_fwd and gdn_glr_fwd_save */
  GDN_GLR_SAVED = 1, /* the `saved` buffer                            */
  GDN_GLR_BWD = 2    /* workspace of gdn_glr_bwd_saved                */
} gdn_glr_pass;

/* Bytes of the device buffer `pass` needs (0 is possible; the pointer may then be
 * NULL); GDN_ERR_UNSUPPORTED for another pass.  The sizes depend on the problem's
 * sizes and offsets alone. */
gdn_status gdn_glr_workspace_size(const gdn_glr_problem* problem, int32_t pass, size_t* bytes);

/* Forward.  in: x, r, i, lam; z, h0 (each may be NULL: no gate, zero); out: y, h_final
 * (NULL: not wanted; a sequence of no tokens keeps h0).  The time axis is composed of runs
 * and segments: results are those of the serial order up to fp32 rounding, bit-identical from
 * call to call.  The segments of a call pass their states on in the workspace: calls that may
 * overlap in time must not share one.  If they do, their outputs are wrong (NaN, a mixture, or
 * left as they were) and they end late, since every wait for a word is bounded (by a second or
 * so) but may run out once for each segment; nothing outside their outputs and workspace is
 * written. */
gdn_status gdn_glr_fwd(const gdn_glr_problem* problem, const void* x, const void* r, const void* i,
                       const float* lam, const void* z, const float* h0, void* y, float* h_final,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Training: gdn_glr_fwd_save computes what gdn_glr_fwd computes (bit-identical) and keeps
 * the state every few tokens in `saved` (GDN_GLR_SAVED bytes, 16-byte aligned);
 * gdn_glr_bwd_saved forms from it the gradients of L = <y, dy> + <h_final, dh_final>.
 * The problem and the inputs must be those of the save call and `saved` unmodified (not
 * checked).  `saved` is only read by the backward.
 *   in : x, r, i, lam, z as gdn_glr_fwd; dy; dh_final (NULL: zero)
 *   out: dx, dr, di (io dtype), dlam (fp32); dz, dh0 (NULL: not wanted; dz needs z,
 *        GDN_ERR_NULL otherwise)
 * dlam is summed in a fixed order (bit-identical from call to call). */
gdn_status gdn_glr_fwd_save(const gdn_glr_problem* problem, const void* x, const void* r, const void* i,
                            const float* lam, const void* z, const float* h0, void* y, float* h_final,
                            void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                            void* stream);
gdn_status gdn_glr_bwd_saved(const gdn_glr_problem* problem, const void* x, const void* r, const void* i,
                             const float* lam, const void* z, const void* dy, const float* dh_final,
                             const void* saved, size_t saved_bytes, void* dx, void* dr, void* di,
                             float* dlam, void* dz, float* dh0, void* workspace, size_t workspace_bytes,
                             void* stream);

/* One token of every sequence (decoding; dense with T == 1): y, and the state h [B,C] fp32
 * updated in place.  y and h must not overlap another tensor.  No workspace. */
gdn_status gdn_glr_step(const gdn_glr_problem* problem, const void* x, const void* r, const void* i,
                        const float* lam, const void* z, float* h, void* y, void* stream);

typedef enum gdn_rope_norm {
  GDN_ROPE_NONE = 0, /* n = x                                           */
  GDN_ROPE_RMS = 1,  /* n = x / sqrt(mean(x^2) + eps) w                 */
  GDN_ROPE_L2 = 2    /* n = x / max(||x||_2, 1e-30), as gdn_prologue    */
} gdn_rope_norm;

/* Norm of queries and keys per head (over its D values) with the rotation by position in
 * the same pass.  The first R values of a head are R / 2 pairs (j, j'), with j' = j + R / 2,
 * or, interleaved, (2 j, 2 j + 1); pair j is turned by the angle position inv_freq[j]
 * (radians):
 *     out_j = n_j cos - n_j' sin;  out_j' = n_j' cos + n_j sin
 * and the values behind the first R are n.
 *   in : q [B,T,Hq,D], k [B,T,Hk,D] (io dtype): a token's heads and values contiguous,
 *        tokens q_stride and k_stride values apart (0: Hq D and Hk D), so that both may be
 *        views of one projection's rows; inv_freq [R / 2] fp32 (NULL with R == 0);
 *        positions [B,T] int32 (NULL: 0 .. T - 1 in every row); wq, wk [D] fp32 (each NULL:
 *        ones; only with GDN_ROPE_RMS, else GDN_ERR_UNSUPPORTED)
 *   out: q_out, k_out, contiguous
 * 16-byte aligned but for inv_freq and positions (4 bytes); strides (with T == 1 those from
 * sequence to sequence) of whole 16 bytes
 * (GDN_ERR_ALIGN), at least Hq D and Hk D (GDN_ERR_SHAPE), up to 2^21.  Supported: D in {64, 128, 256},
 * R a multiple of 16 up to D, Hq and Hk up to 4096, B T (Hq + Hk) < 2^31, else
 * GDN_ERR_UNSUPPORTED.  Angles are reduced in fp64 (2^-52 of the angle); all else is fp32,
 * squares included, and outputs are rounded once.  A NaN in a row makes the row NaN (with
 * GDN_ROPE_NONE its pair) and no other.  eps >= 0 and finite frequencies are documented, not
 * checked. */
typedef struct gdn_rope_problem {
  int32_t B, T, Hq, Hk, D, R;
  int32_t norm;             /* gdn_rope_norm; another value: GDN_ERR_UNSUPPORTED */
  int32_t interleaved;      /* nonzero: pairs (2 j, 2 j + 1)                     */
  int32_t io_dtype;         /* gdn_dtype                                         */
  float eps;                /* GDN_ROPE_RMS                                      */
  int64_t q_stride, k_stride;
} gdn_rope_problem;

gdn_status gdn_rope_fwd(const gdn_rope_problem* problem, const void* q, const void* k,
                        const float* inv_freq, const int32_t* positions, const float* wq,
                        const float* wk, void* q_out, void* k_out, void* stream);

/* Bytes of workspace gdn_rope_bwd needs where dwq or dwk is wanted (their partial sums). */
gdn_status gdn_rope_workspace_size(const gdn_rope_problem* problem, size_t* bytes);

/* Backward: gradients of <q_out, dq_out> + <k_out, dk_out>.
 *   in : as gdn_rope_fwd; dq_out [B,T,Hq,D], dk_out [B,T,Hk,D] (io dtype), contiguous
 *   out: dq, dk (io dtype), contiguous; dwq, dwk [D] fp32 (each NULL: not wanted; only with
 *        GDN_ROPE_RMS, else GDN_ERR_UNSUPPORTED; without a weight it is that of ones)
 * A row whose norm the L2 form cuts off at 1e-30 has the gradient of the product that is
 * left.  Weights' gradients are summed in a fixed order (bit-identical from call to call). */
gdn_status gdn_rope_bwd(const gdn_rope_problem* problem, const void* q, const void* k,
                        const float* inv_freq, const int32_t* positions, const float* wq,
                        const float* wk, const void* dq_out, const void* dk_out, void* dq, void* dk,
                        float* dwq, float* dwk, void* workspace, size_t workspace_bytes, void* stream);

/* Causal attention over a sliding window whose first tokens stay visible: query i of a
 * sequence sees key j <= i where j > i - window or j < sinks, and
 *     o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i . k_j - lse_i),
 *     lse_i = log sum_j exp(scale q_i . k_j)       over the keys it sees
 * (at least its own).  Query head h attends to key head h / (Hq / Hk).
 * Tensors: q, o, dout, dq [B,T,Hq,D], k, v, dk, dv [B,T,Hk,D] (io dtype), lse [B,T,Hq] fp32.
 * q, k and v may have their tokens q_stride, k_stride, v_stride values apart as in
 * gdn_rope_problem (0: contiguous; up to 2^21); all else is contiguous.  16-byte aligned,
 * lse and lens 4-byte.  Supported: D in {64, 128}, Hq a multiple of Hk up to 4096, window >= 1 (as long as
 * wanted), sinks up to 1024, a finite scale, B T up to 2^30, up to 65535 sequences, and (but for
 * gdn_swa_fill) fewer than 2^24 workgroups in a launch, else GDN_ERR_UNSUPPORTED: counted as one for every
 * query head and every 32 tokens of a sequence, or part of them; and, where windows leave first tokens
 * behind, one for every sequence, key head and first token, and one for every key head, 16 first
 * tokens and 64 tokens of a sequence, or part of them.
 * Scores, sums and statistics of the softmax are fp32; with bf16 io the probabilities and
 * the scores' gradients are rounded to bf16 as operands of the products that sum over them
 * (gdn_swa_step keeps the probabilities' next 8 bits in a second product).
 * Outputs are rounded once.  Sums run in a fixed order (bit-identical from call to call).
 * NaN and Inf reach what sees them and nothing else, in a result as the definition makes of
 * them or, where it gives an infinity, NaN; a key whose probability is zero because its score
 * is minus infinity may give its queries' dq NaN or nothing. */
typedef struct gdn_swa_problem {
  int32_t B, T, Hq, Hk, D;
  int32_t window, sinks;
  int32_t num_seqs;                /* == B for dense input, else len(cu_seqlens) - 1        */
  const int32_t* cu_seqlens_host;  /* host, num_seqs + 1 offsets, or NULL (dense)           */
  const int32_t* cu_seqlens_dev;   /* device copy of the same values, or NULL               */
  int32_t io_dtype;                /* gdn_dtype                                             */
  float scale;
  int64_t q_stride, k_stride, v_stride;
} gdn_swa_problem;

typedef enum gdn_swa_pass {
  GDN_SWA_BWD = 0, /* workspace of gdn_swa_bwd  */
  GDN_SWA_STEP = 1 /* workspace of gdn_swa_step */
} gdn_swa_pass;

/* Bytes of the device buffer `pass` needs (0 is possible; the pointer may then be NULL);
 * GDN_ERR_UNSUPPORTED for another pass.  The sizes depend on the problem alone. */
gdn_status gdn_swa_workspace_size(const gdn_swa_problem* problem, int32_t pass, size_t* bytes);

/* Forward.  out: o; lse (NULL: not wanted).  No workspace. */
gdn_status gdn_swa_fwd(const gdn_swa_problem* problem, const void* q, const void* k, const void* v,
                       void* o, float* lse, void* stream);

/* Backward: gradients of <o, dout>, from the forward's o and lse (of the same problem and
 * inputs, not checked). */
gdn_status gdn_swa_bwd(const gdn_swa_problem* problem, const void* q, const void* k, const void* v,
                       const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                       void* workspace, size_t workspace_bytes, void* stream);

/* The cache of a sequence: sinks + window slots of Hk D values for keys and as many for
 * values, [num_seqs, sinks + window, Hk, D] (io dtype).  Token j < sinks stands in slot j,
 * any other in slot sinks + (j - sinks) mod window: the slots that n tokens have left hold
 * exactly what token n - 1 sees.
 *
 * gdn_swa_fill writes the slots of prompts of their own (dense or packed): for every
 * sequence its first tokens and the last of the others; slots that it does not reach are
 * left as they were. */
gdn_status gdn_swa_fill(const gdn_swa_problem* problem, const void* k, const void* v, void* kcache,
                        void* vcache, void* stream);

/* One token of every sequence (decoding; dense with T == 1): its key and value are written
 * to their slot, and o is what the token sees.  lens [B] int32 on the device holds the
 * tokens that each sequence had before (the caller adds one behind its last layer); a
 * negative one marks an idle place of the batch: its cache is left alone, its o is zero.
 * Slots that have not been written are not read.  The caches and o must not overlap another
 * tensor. */
gdn_status gdn_swa_step(const gdn_swa_problem* problem, const void* q, const void* k, const void* v,
                        void* kcache, void* vcache, const int32_t* lens, void* o, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */
