/*
 * dr.h -- C ABI of libdr.so: chunkwise-parallel forward and backward of the
 * delta-rule recurrent memory (DeltaNet, Gated DeltaNet, Kimi Delta Attention)
 * on one GB300 GPU (sm_103a).
 *
 * The operation (page "Linear Attention Architectures: Mechanisms, Trade-offs,
 * and Cross-Layer Routing", section "Metodologia y Marco de Trabajo", item 1,
 * the unified recurrent-memory notation and its three variant bullets): per
 * (sequence, head) a memory matrix W (d_v x d_k) is, token by token,
 *   decayed   Wd_t = W_{t-1} diag(a_t)       a_t = 1 (DeltaNet), exp(g_t) * 1 (Gated
 *                                            DeltaNet, one scalar gate), exp(g_t) per
 *                                            key channel (Kimi Delta Attention)
 *   corrected r_t  = v_t - Wd_t k_t          (the delta-rule residual r = v - vbar)
 *   written   W_t  = Wd_t + beta_t r_t k_t^T
 *   read      o_t  = scale * W_t q_t
 * The gate enters as its logarithm g = log(alpha) <= 0.  beta_t, the read after
 * the write and `scale` are the standard delta-rule reading of that notation.
 * Also here: the recurrent step for inference (dr_decode), the emitted write
 * u = beta r with its gradient (dr_fwd_u / dr_bwd_u), input preparation inside the
 * library (DR_FLAG_PREPARE_INPUTS), and Gated DeltaNet-2, the fourth variant of the
 * same section (dr_gdn2_*, separate erase and write gates; its equations are a
 * reading, stated at its entry points).
 *
 * Memory: the caller allocates every buffer (device memory unless stated) and
 * the workspace; the library never allocates, frees or synchronises inside
 * dr_fwd / dr_bwd.  All work is enqueued on `stream` (a cudaStream_t passed as
 * void*, NULL = legacy default stream) in stream order.  Calls are re-entrant;
 * two calls that run concurrently must not share a workspace.
 *
 * Layouts (row-major, contiguous, every pointer 16-byte aligned):
 *   q, k, dq, dk   [B, T, H, d_k]       io dtype (grad dtype for dq, dk)
 *   v, dO, dv      [B, T, H, d_v]       io dtype (grad dtype for dv)
 *   o              [B, T, H, d_v]       out dtype
 *   beta, dbeta    [B, T, H]            fp32, beta in [0, 1]
 *   g, dg          Gated DeltaNet [B, T, H]; KDA [B, T, H, d_k]; fp32; NULL for DeltaNet
 *   h0, hT, dhT, dh0  [N, H, d_k, d_v]  fp32, the state S = W^T (d_v contiguous)
 * N = B for dense batches.  For packed ragged sequences B == 1, T is the total
 * length and cu_seqlens (N + 1 offsets) splits the T axis; every sequence
 * starts from its own h0[n] (zero when h0 is NULL) and ends in hT[n].
 *
 * Errors: every entry point returns a dr_status_code.  When the host detects
 * an error nothing is launched and no output is touched.  A launch failure is
 * DR_ERR_CUDA.  Device-side waits are bounded: a wait that runs out records
 * DR_ERR_TIMEOUT in the workspace, which dr_check_status reports.
 */
#ifndef DR_H
#define DR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum dr_status_code {
    DR_OK = 0,
    DR_ERR_INVALID_ARG = 1,   /* null pointer, negative size, bad enum, bad cu_seqlens */
    DR_ERR_UNSUPPORTED = 2,   /* valid but outside the supported set (below)         */
    DR_ERR_WORKSPACE = 3,     /* workspace NULL or smaller than dr_workspace_bytes   */
    DR_ERR_ALIGNMENT = 4,     /* a pointer is not 16-byte aligned                    */
    DR_ERR_CUDA = 5,          /* a CUDA call or launch failed                        */
    DR_ERR_TIMEOUT = 6,       /* a bounded device-side wait ran out                  */
    DR_ERR_SCRATCH_LIMIT = 7, /* dr_fwd_noalloc: problem larger than its static scratch */
    DR_ERR_INDEX = 8          /* a kernel met a page number or length outside its range  */
};

enum dr_variant { DR_DELTANET = 0, DR_GDN = 1, DR_KDA = 2, DR_GDN2 = 3 /* dr_gdn2_* only */ };
enum dr_dtype { DR_BF16 = 0, DR_F32 = 1 };

/* dr_desc.flags */
#define DR_FLAG_REUSE_FWD 1  /* dr_bwd: the workspace still holds the residuals
                                written by dr_fwd for the same desc and inputs;
                                skip their recomputation */
/*
 * DR_FLAG_PREPARE_INPUTS: q, k, beta and g arrive as the projections produce them,
 * and the library applies the input maps of these layers itself.  The pages give
 * the recurrence on prepared inputs only (q, k unit-norm keys, beta in [0, 1],
 * g = log alpha <= 0); the maps below are the standard ones the workloads use to
 * produce them (q, k L2-normalised per head, beta through a sigmoid, log alpha
 * through -softplus), with eps = 1e-6 guarding the zero vector:
 *   q_hat = q * rsqrt(sum_c q_c^2 + 1e-6)   per (token, head); the same for k
 *   beta  = sigmoid(b)                       b: the beta argument, a logit
 *   g     = -softplus(x) = -log(1 + e^x)     x: the g argument (GDN, KDA)
 * dr_bwd / dr_bwd_u take the same raw tensors and return gradients with respect to
 * them (dq, dk, dbeta, dg chained through the three maps).  On the bf16 tensor-core
 * path the kernels apply the maps on the fly, in fp32, to the raw tiles they load
 * (forward and backward alike; the prepared values are never stored, only the two
 * inverse row norms per token and head, 8 bytes, which dr_workspace_bytes counts and
 * the backward reads back) and chain the gradients before writing them.  On the fp32 CUDA-core path dr_fwd / dr_fwd_u write
 * q_hat, k_hat (io_dtype), beta and g (fp32) into the workspace (dr_workspace_bytes
 * counts them) and run on those; with DR_FLAG_REUSE_FWD the backward reuses them (the
 * same raw inputs must be passed).  dr_decode applies the maps in its own kernel.
 * dr_fwd_noalloc does not take the flag (DR_ERR_UNSUPPORTED).
 */
#define DR_FLAG_PREPARE_INPUTS 2

/*
 * Problem descriptor.  Supported set:
 *   io bf16: d_k = d_v in {64, 128}, chunk = 64  (tensor-core path)
 *   io fp32: d_k, d_v in {16, 32, 64, 128}, chunk in {16, 32, 64}  (fp32 CUDA-core path)
 *   any T >= 0 (a partial last chunk is fine), B >= 0, H >= 1.
 */
typedef struct dr_desc {
    int B, T, H;
    int d_k, d_v;
    int chunk;                    /* tokens per chunk of the chunkwise form            */
    int variant;                  /* enum dr_variant                                   */
    int io_dtype;                 /* q, k, v, dO                                       */
    int out_dtype;                /* o                                                 */
    int grad_dtype;               /* dq, dk, dv                                        */
    float scale;                  /* read scale (1.0 = the plain read o = W q)         */
    int flags;                    /* DR_FLAG_*                                          */
    int num_seqs;                 /* N: B for dense batches, or the packed count       */
    const int32_t* cu_seqlens;    /* device [N+1] or NULL (dense)                      */
    const int32_t* chunk_table;   /* device [num_chunks][2] = (sequence, first token),
                                     from dr_plan_varlen; NULL for dense batches      */
    const int32_t* chunk_offsets; /* device [N+1]: first chunk of each sequence        */
    int num_chunks;               /* total chunks (packed layout only)                 */
} dr_desc;

/* Bytes of workspace dr_fwd and dr_bwd need for `desc` (the same for both).
   Returns 0 when desc is invalid or unsupported. */
size_t dr_workspace_bytes(const dr_desc* desc);

/*
 * Host-side chunk plan of packed ragged sequences (no GPU work).
 * cu_seqlens_host: N + 1 non-decreasing offsets starting at 0.  Writes, for
 * every chunk of every sequence in order, (sequence, first token) into
 * chunk_table_host[2*i], [2*i+1] (chunks never straddle a sequence boundary;
 * the last chunk of a sequence may be short; an empty sequence has none), and
 * the index of each sequence's first chunk into chunk_offsets_host[0..N]
 * (chunk_offsets_host[N] = total).  *num_chunks receives the total; when it
 * exceeds max_chunks nothing is written and DR_ERR_INVALID_ARG is returned.
 * chunk_table_host / chunk_offsets_host may be NULL to query the count only.
 */
int dr_plan_varlen(const int32_t* cu_seqlens_host, int num_seqs, int chunk,
                   int32_t* chunk_table_host, int32_t* chunk_offsets_host, int max_chunks,
                   int* num_chunks);

/*
 * Forward: o (and hT when non-NULL) from q, k, v, beta, g, h0 (h0 NULL = zero
 * state).  Also leaves in the workspace the residuals dr_bwd can reuse
 * (DR_FLAG_REUSE_FWD).
 */
int dr_fwd(const dr_desc* desc, const void* q, const void* k, const void* v,
           const float* beta, const float* g, const float* h0, void* o, float* hT,
           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward: gradients of L = sum(dO * o) + sum(dhT * hT) with respect to q, k,
 * v, beta, g (the log-gate) and h0.  dhT NULL means a zero final-state
 * gradient; dh0 may be NULL when not needed; dg must be NULL for DeltaNet and
 * non-NULL otherwise.  Gradients are with respect to the tensors as passed
 * (q, k already normalised, beta after its sigmoid, g = log alpha; with
 * DR_FLAG_PREPARE_INPUTS the raw tensors before those maps).
 */
int dr_bwd(const dr_desc* desc, const void* q, const void* k, const void* v,
           const float* beta, const float* g, const float* h0, const void* dO,
           const float* dhT, void* dq, void* dk, void* dv, float* dbeta, float* dg,
           float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The write of every token, for routing it to another layer ("Linear Attention
 * Architectures: Mechanisms, Trade-offs, and Cross-Layer Routing", section
 * "Metodologia y Marco de Trabajo", item 3, CLER: the delta-rule write error of a
 * layer is forwarded to the next one).
 * dr_fwd_u is dr_fwd that also writes u_t = beta_t r_t, r_t = v_t - (decayed W) k_t
 * (the write the recurrence adds to the memory), to u: [B][T][H][d_v] in out_dtype
 * (packed layout as o), or nothing when u is NULL.
 * dr_bwd_u is dr_bwd for L = sum(dO * o) + sum(dhT * hT) + sum(dU * u): dU has the
 * layout of u in io_dtype; NULL means zero (dr_bwd).  With DR_FLAG_REUSE_FWD the
 * workspace may come from dr_fwd or dr_fwd_u.
 * Same supported set, ownership and errors as dr_fwd / dr_bwd (u and dU 16-byte
 * aligned).
 */
int dr_fwd_u(const dr_desc* desc, const void* q, const void* k, const void* v,
             const float* beta, const float* g, const float* h0, void* o, float* hT,
             void* u, void* workspace, size_t workspace_bytes, void* stream);
int dr_bwd_u(const dr_desc* desc, const void* q, const void* k, const void* v,
             const float* beta, const float* g, const float* h0, const void* dO,
             const float* dhT, const void* dU, void* dq, void* dk, void* dv, float* dbeta,
             float* dg, float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Forward for callers that cannot allocate device memory.  The paper has no
 * counterpart; this is an interface convenience of the library.
 *
 * Some callers cannot call cudaMalloc where they run this layer (a plugin
 * handed only its input and output buffers by its host framework, or code
 * that must not trigger an allocation and the device synchronisation it may
 * bring).  dr_fwd_noalloc computes the same o and hT as dr_fwd, with the
 * fp32 CUDA-core kernel (io fp32 only; the supported set of dr_fwd for fp32
 * inputs), but takes no workspace: its scratch is a 16 MiB array that the
 * library keeps in the global memory of every GPU that loads it, for the life
 * of the process.  It allocates nothing itself.
 *   - Size limit: N * H (sequences times heads) must not exceed 46 when d_k,
 *     d_v and chunk are at most 64, or 11 when d_k or d_v is 128; larger
 *     problems return DR_ERR_SCRATCH_LIMIT and launch nothing.
 *   - The first call on each device looks up the array's device address with
 *     that device current (a runtime symbol query); make that first call
 *     before any stream capture on the device.  The address is cached per
 *     device ordinal for the rest of the process: it belongs to the device's
 *     primary context (the one the CUDA runtime uses), is not valid after a
 *     cudaDeviceReset of that device, and must not be used from another
 *     context made current on it.
 *   - Every call shares the one array: calls whose kernels can overlap on the
 *     GPU (other streams, other host threads) race on it and must be
 *     serialised by the caller.  Contents left by an earlier call are never
 *     read before being overwritten.
 *   - It writes no workspace, so dr_bwd cannot reuse its residuals.
 * Errors as dr_fwd, plus DR_ERR_UNSUPPORTED for bf16 inputs.
 */
int dr_fwd_noalloc(const dr_desc* desc, const void* q, const void* k, const void* v,
                   const float* beta, const float* g, const float* h0, void* o, float* hT,
                   void* stream);

/*
 * Recurrent step for inference (decode): the delta-rule recurrence applied
 * token by token, without chunks, to a state that the caller keeps between
 * calls ("The Delta Rule and its gated forms", the per-token update with the
 * decay applied before the residual and the read after the write).
 *   For every sequence n < desc->B, head h and token t < desc->T in order:
 *     S~ = D_t S;  r = v_t - S~^T k_t;  S = S~ + beta_t k_t r^T;  o_t = scale S^T q_t
 *   with S = W^T and D_t = I (DeltaNet), e^{g_t} I (GDN) or diag(e^{g_t}) (KDA).
 * state: [B][H][d_k][d_v] fp32 (the layout of h0 / hT), read at entry and
 *   overwritten with the state after the last token; device memory owned by
 *   the caller, never NULL.
 * q, k: [B][T][H][d_k]; v, o: [B][T][H][d_v] in io_dtype / out_dtype;
 *   beta [B][T][H] fp32; g as for dr_fwd (NULL for DeltaNet).  Dense batches
 *   only (cu_seqlens NULL); desc->chunk is ignored (any value >= 1).
 * desc->flags: DR_FLAG_PREPARE_INPUTS (q, k normalised, beta and g mapped inside
 *   the kernel, as for dr_fwd); DR_FLAG_REUSE_FWD is ignored.
 * Supported: d_k, d_v in {16, 32, 64, 128}, io bf16 or fp32.  No workspace,
 *   nothing allocated, no device synchronisation; stream-ordered on `stream`.
 * Errors: DR_ERR_INVALID_ARG (bad desc, NULL state or input, packed layout),
 *   DR_ERR_UNSUPPORTED (sizes), DR_ERR_ALIGNMENT (pointers not 16-byte
 *   aligned), DR_ERR_CUDA (launch failure).  Nothing is launched on error.
 */
int dr_decode(const dr_desc* desc, const void* q, const void* k, const void* v,
              const float* beta, const float* g, float* state, void* o, void* stream);

/*
 * Gated DeltaNet-2: separate per-channel erase and write gates ("Linear Attention
 * Architectures: Mechanisms, Trade-offs, and Cross-Layer Routing", section "Metodologia
 * y Marco de Trabajo", item 1, the Gated DeltaNet-2 bullet, which describes it in words
 * only).  The library reads it as Gated DeltaNet's scalar decay followed by an erase
 * along the gated key channels and a write of the gated value channels:
 *   Wd_t = alpha_t W_{t-1};  p_t = Wd_t k_t;
 *   W_t  = Wd_t - p_t (erase_t . k_t)^T + (write_t . v_t) k_t^T;  o_t = scale W_t q_t
 * ("." elementwise), which is Gated DeltaNet when erase_t = write_t = beta_t.
 * desc->variant must be DR_GDN2.  Inputs as dr_fwd / dr_bwd with beta replaced by
 *   erase [B, T, H, d_k] fp32 (gate per key channel, normally in [0, 1]) and
 *   write [B, T, H, d_v] fp32 (gate per value channel, normally in [0, 1]);
 *   g [B, T, H] fp32 = log alpha, never NULL.
 * dr_gdn2_bwd returns dq, dk, dv (grad dtype), derase, dwrite, dg (fp32) and dh0
 * (optional) for L = sum(dO * o) + sum(dhT * hT).
 * Supported: d_k, d_v, chunk in {16, 32, 64}; io bf16 or fp32 (fp32 arithmetic on the
 * CUDA cores for both); dense or packed layout as dr_fwd.  dr_workspace_bytes sizes the
 * workspace (same value for both calls); dr_gdn2_fwd leaves the chunk-start states in
 * it, and dr_gdn2_bwd with DR_FLAG_REUSE_FWD reads them instead of recomputing them
 * (the same desc, inputs and workspace as the forward).  DR_FLAG_PREPARE_INPUTS is
 * DR_ERR_UNSUPPORTED.  Errors as dr_fwd / dr_bwd; dr_fwd and
 * dr_bwd refuse DR_GDN2 with DR_ERR_INVALID_ARG.
 */
int dr_gdn2_fwd(const dr_desc* desc, const void* q, const void* k, const void* v,
                const float* erase, const float* write, const float* g, const float* h0,
                void* o, float* hT, void* workspace, size_t workspace_bytes, void* stream);
int dr_gdn2_bwd(const dr_desc* desc, const void* q, const void* k, const void* v,
                const float* erase, const float* write, const float* g, const float* h0,
                const void* dO, const float* dhT, void* dq, void* dk, void* dv, float* derase,
                float* dwrite, float* dg, float* dh0, void* workspace, size_t workspace_bytes,
                void* stream);

/*
 * Recurrent step of Gated DeltaNet-2 (the update of dr_gdn2_fwd token by token, as
 * dr_decode for the other variants): for every sequence, head and token in order,
 *   S~ = e^{g_t} S;  p = S~^T k_t;  S = S~ - (erase_t . k_t) p^T + k_t (write_t . v_t)^T;
 *   o_t = scale S^T q_t
 * on the caller's fp32 state [B][H][d_k][d_v], updated in place.  desc->variant must be
 * DR_GDN2; erase [B][T][H][d_k], write [B][T][H][d_v], g [B][T][H] fp32, none NULL when
 * there are tokens.  Sizes, dtypes, layout and errors as dr_decode;
 * DR_FLAG_PREPARE_INPUTS is DR_ERR_UNSUPPORTED.
 */
int dr_gdn2_decode(const dr_desc* desc, const void* q, const void* k, const void* v,
                   const float* erase, const float* write, const float* g, float* state,
                   void* o, void* stream);

/*
 * The softmax-attention layer of a hybrid stack (page "Un Analisis Sistematico de la
 * Atencion Lineal Hibrida": a few softmax-attention layers among the delta-rule ones):
 * the norm and position rotation of its queries and keys, the paged 8-bit cache of its
 * keys and values, and the attention over that cache.  The pages name the layer only; the
 * equations are the standard ones, stated at each entry point.
 *
 * Norm of queries and keys for each head, with the position rotation in the same pass.
 * For every token (b, t), head and channel c < d:
 *   r = 1 / sqrt(mean_c x_c^2 + eps);  n_c = x_c r w_c   (w NULL: all ones)
 *   y = n with every pair (n_i, n_j) of its first `rot` channels turned by the angle of the
 *   token's position p:  y_i = n_i cos - n_j sin,  y_j = n_j cos + n_i sin,  angle index a:
 *   DR_ROPE_HALVES (i, j) = (a, a + rot/2);  DR_ROPE_PAIRS (i, j) = (2a, 2a + 1);  a < rot/2.
 *   p = (positions ? positions[b*T + t] : t) + (start ? start[b] : 0);  cos_table[p][a],
 *   sin_table[p][a]: [table_rows][rot/2] fp32.  A token whose position lies outside the
 *   table gets NaN outputs (and NaN gradients); nothing outside the table is read.
 * The norm runs whether or not channels are rotated (rot = 0: cos_table, sin_table NULL).
 * q: [B*T] rows of Hq*d values, ld_q elements from one row to the next (>= Hq*d: q and k
 *   may be column ranges of one packed projection), k: the same with Hk heads (Hk = 0: no
 *   keys); io dtype.  yq, yk: rows ld_oq, ld_ok elements apart, out dtype.  A y may be its x.
 * dr_norm_rope_bwd: with dyq, dyk (contiguous [B, T, H, d], io dtype) the gradients
 *   dq, dk (grad dtype, rows ld_oq, ld_ok apart) and dwq, dwk ([d] fp32, summed over all
 *   tokens and heads in a fixed order; NULL where the weight is NULL or not wanted).
 *   Workspace: dr_norm_rope_workspace_bytes (0 when desc is invalid).
 * Supported: d a multiple of 8 up to 256; rot a multiple of 16 up to d; io bf16 or fp32;
 *   any B, T >= 0.  Row distances are multiples of 16 bytes.  fp32 arithmetic, one rounding
 *   at the output.  Errors as dr_fwd.
 */
enum dr_rope_style { DR_ROPE_HALVES = 0, DR_ROPE_PAIRS = 1 };

typedef struct dr_rope_desc {
    int B, T, Hq, Hk, d;
    int rot;                      /* rotated channels, 0 .. d                          */
    int style;                    /* enum dr_rope_style                                */
    int io_dtype, out_dtype, grad_dtype;
    int table_rows;               /* rows of cos_table and sin_table                   */
    float eps;
    long long ld_q, ld_k;         /* elements between token rows of q, k               */
    long long ld_oq, ld_ok;       /* of yq, yk (forward), dq, dk (backward)            */
} dr_rope_desc;

int dr_norm_rope_fwd(const dr_rope_desc* desc, const void* q, const void* k, const float* wq,
                     const float* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, const int32_t* start, void* yq, void* yk,
                     void* stream);
size_t dr_norm_rope_workspace_bytes(const dr_rope_desc* desc);
int dr_norm_rope_bwd(const dr_rope_desc* desc, const void* q, const void* k, const float* wq,
                     const float* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, const int32_t* start, const void* dyq,
                     const void* dyk, void* dq, void* dk, float* dwq, float* dwk,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * A paged cache of keys and values in 8 bits with one fp32 scale for each page and head.
 * A page holds `page` consecutive positions of one sequence; value = code * scale.
 *   codes  k, v:              [num_pages][H][page][d], one byte each
 *   scales k_scale, v_scale:  [num_pages][H], >= 0 (NaN: the page holds a value that was not
 *                             finite, and reads as NaN)
 *   DR_CODE_I8: two's complement, -127 .. 127 (Q = 127); DR_CODE_E4M3: 8-bit floating point,
 *   4 exponent and 3 fraction bits, no infinities (Q = 448).
 *   status: one device int32 the caller sets to zero, or NULL.  A kernel that meets a page
 *   number outside 0 .. num_pages-1, a negative length, a count outside 0 .. T or a position
 *   past the table's row records it there (dr_check_status: DR_ERR_INDEX; it stays until the
 *   caller clears it) and touches nothing through it.
 * dr_cache_seqs names the positions of one call: position p of sequence b is row p % page of
 *   page page_table[b * table_stride + p / page]; the call's tokens t < n_b of sequence b
 *   (n_b = counts ? counts[b] : T, at most T) are the positions lens[b] + t.  Only table
 *   entries of pages that hold such positions (attention: or earlier, visible ones) are read.
 * Supported: d 64 or 128; page 16, 32, 64 or 128; any H >= 1, B, T >= 0.  Every array begins at a
 *   multiple of 16 bytes, page_table, lens and counts too (DR_ERR_ALIGNMENT).
 *
 * dr_cache_write appends the tokens k, v ([B*T] rows of H*d, ld_k / ld_v elements apart, io
 * dtype).  For each page and head it touches, with s_old the page's scale if the page holds
 * earlier positions of the sequence and 0 otherwise (what a page held before is forgotten
 * when its first position is written):
 *   s = max(s_old, max |x| * fl(1/Q)) over the new values;  NaN when one is not finite
 *   new codes: x / s, rounded to the nearest code, ties to even (0 where s = 0 or NaN)
 *   where s > s_old > 0: the earlier codes c become c s_old / s, rounded the same way
 * (fp32 arithmetic throughout).  A page that is written must belong to one sequence.
 * dr_cache_read writes the values at the call's tokens to k, v ([B, T, H, d] contiguous, out
 * dtype, each rounded once; either may be NULL), zeros for t >= n_b, NaN where an index is
 * out of range.
 */
enum dr_code { DR_CODE_I8 = 0, DR_CODE_E4M3 = 1 };

typedef struct dr_cache {
    int num_pages, H, d, page;
    int code;                     /* enum dr_code */
    void *k, *v;
    float *k_scale, *v_scale;
    int32_t* status;
} dr_cache;

typedef struct dr_cache_seqs {
    int B, T;
    const int32_t* page_table;    /* device [B][table_stride]                          */
    int table_stride;             /* pages that a sequence can have                    */
    const int32_t* lens;          /* device [B]: positions before the call's tokens    */
    const int32_t* counts;        /* device [B]: the call's tokens, or NULL (T each)   */
} dr_cache_seqs;

int dr_cache_write(const dr_cache* cache, const dr_cache_seqs* seqs, const void* k, long long ld_k,
                   const void* v, long long ld_v, int io_dtype, void* stream);
int dr_cache_read(const dr_cache* cache, const dr_cache_seqs* seqs, void* k, void* v, int out_dtype,
                  void* stream);

/*
 * Attention of the call's tokens over the cache (which already holds them): token t < n_b of
 * sequence b is the query at position p = lens[b] + t and sees the positions j <= p, and
 * with window > 0 only j > p - window.  Query head h reads cache head h / (Hq / H).
 *   s_j = scale * sum_c q_c k_jc;  o = sum_j e^{s_j} v_j / sum_j e^{s_j};
 *   lse = ln sum_j e^{s_j}
 * Tokens t >= n_b: o = 0, lse = -inf.  Where a sequence's length, count or a page number that
 * a token needs is out of range, its o and lse are NaN.  A query that is not finite makes its
 * own o NaN (also where all its scores are -inf, then with lse = -inf).
 * q: [B*T] rows of Hq*d, ld_q elements apart (io dtype); o [B, T, Hq, d] (out dtype); lse
 *   [B, T, Hq] fp32 or NULL.
 * Arithmetic: 16-bit floating-point operands that hold the codes and bf16 queries exactly and
 *   the weights (softmax weight times value scale) to 11 bits, or to 2^-37 of the row's
 *   largest weight where that is more (22 bits for queries and weights when io or out is fp32);
 *   fp32 accumulation, fp32 softmax statistics.
 * Workspace: dr_cache_attn_workspace_bytes, the same for every length (0 when desc is invalid
 *   or unsupported; needs the device current that will run the call).  Results of one call do
 *   not depend on what it held.  Hq must be a multiple of the cache's H.  Errors as dr_fwd.
 */
typedef struct dr_attn_desc {
    int Hq;
    int io_dtype, out_dtype;
    int window;                   /* 0: none                                           */
    float scale;
    long long ld_q;
} dr_attn_desc;

size_t dr_cache_attn_workspace_bytes(const dr_cache* cache, const dr_attn_desc* desc, int B, int T);
int dr_cache_attn(const dr_cache* cache, const dr_cache_seqs* seqs, const dr_attn_desc* desc,
                  const void* q, void* o, float* lse, void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * The two other token mixers of a hybrid stack, over whole prompts and for training (the same page:
 * its stacks set softmax attention and linear attention with a decay beside the delta rule; it
 * names them only, the equations are the standard ones, stated here).
 *
 * Sequences, for both: dense, cu_seqlens NULL, num_seqs == B sequences of T tokens; or packed,
 * B == 1, T rows, sequence s in the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (device
 * [num_seqs + 1], read when the kernels run: a captured call takes new lengths), num_seqs at most
 * 2^20 (every tile is looked up by a walk over the offsets: the time of many short sequences grows
 * with the square of their number).  Lengths may be zero.  Rows of no sequence are left as they
 * were.  An offset outside 0 .. T counts as the nearest of them and a sequence that would end
 * before it starts as empty: nothing else is touched (where sequences then overlap, their results
 * are undefined).
 * Tensors are rows of heads: q [B*T] rows of Hq*d values (or H*d_k), ld_q elements from one row to
 * the next, and k, v, dq, dk, dv likewise with their own distances (column ranges of one packed
 * projection, or of its gradient, will do); o, dO contiguous.  Everything is of io dtype except
 * statistics, decays and states, which are fp32.
 * Arithmetic: fp32 for fp32 tensors.  For bf16 the products take bf16 operands and accumulate in
 * fp32; softmax weights and their gradients, decayed scores and the state that queries read are rounded
 * to bf16 as operands, what is carried from chunk to chunk (the states) is not: states that come back
 * are good to 2^-16 of their terms.  The gradient takes dO.o from o as it was rounded.
 * Gradients of shared key heads are summed in a fixed order: the same inputs give the same bits.
 * Outputs do not overlap inputs.
 * A token that is not finite leaves other sequences alone; in its own it may also reach the results
 * of tokens that do not see it (a weight of zero times it).
 * Errors as dr_fwd.  status: one device int32 the caller sets to zero, or NULL; a kernel whose bounded
 * wait ran out records it there (dr_check_status: DR_ERR_TIMEOUT).
 *
 * Causal softmax attention: query i of a sequence sees its keys j <= i, and with window > 0 only
 * j > i - window; query head h reads key head h / (Hq / H).
 *   s_ij = scale q_i.k_j;  lse_i = ln sum_j e^{s_ij};  o_i = sum_j e^{s_ij - lse_i} v_j
 * Forward: o [B, T, Hq, d], lse [B, T, Hq] (or NULL).  Backward: dq, dk, dv of L = sum(dO * o), from
 * the forward's inputs, o and lse.  Workspace (backward): dr_prompt_attn_workspace_bytes (0 when desc
 * is invalid or unsupported); results do not depend on what it held.
 * Supported: d 64 or 128, H dividing Hq, any B, T >= 0, B*T < 2^30.
 */
typedef struct dr_prompt_desc {
    int B, T, Hq, H, d;
    int num_seqs;
    int io_dtype;
    int window;                   /* 0: none                                           */
    float scale;
    long long ld_q, ld_k, ld_v;
    long long ld_dq, ld_dk, ld_dv; /* backward                                          */
    int32_t* status;
} dr_prompt_desc;

int dr_prompt_attn_fwd(const dr_prompt_desc* desc, const void* q, const void* k, const void* v,
                       const int32_t* cu_seqlens, void* o, float* lse, void* stream);
size_t dr_prompt_attn_workspace_bytes(const dr_prompt_desc* desc);
int dr_prompt_attn_bwd(const dr_prompt_desc* desc, const void* q, const void* k, const void* v,
                       const void* o, const float* lse, const void* dO, const int32_t* cu_seqlens,
                       void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Linear attention with a decay for each head (sequences, tensors and arithmetic as above):
 *   S_t = e^{g_h} S_{t-1} + k_t v_t^T;  o_t = scale S_t^T q_t
 * g: [H] fp32, the log-decay of a step, <= 0, a constant of the layer (no gradient).  States
 * h0, hT, dhT, dh0 [num_seqs, H, d_k, d_v] fp32, NULL: zero (h0, dhT) or not wanted (hT, dh0).  A
 * sequence without tokens hands its state on (hT = h0, dh0 = dhT).
 * dr_linear_attn_fwd: o [B, T, H, d_v] and hT.  dr_linear_attn_bwd: dq, dk, dv and dh0 of
 * L = sum(dO * o) + sum(dhT * hT).  Workspace for both: dr_linear_attn_workspace_bytes (0 when desc
 * is invalid or unsupported; ld_dq, ld_dk, ld_dv are not looked at); results do not depend on what
 * it held.
 * dr_linear_attn_step: the recurrence token by token for T tokens of every sequence, on the caller's
 * state [B, H, d_k, d_v] fp32, updated in place (fp32 arithmetic for both types; dense only; ld_dq,
 * ld_dk, ld_dv are not looked at).
 * Supported: bf16 d_k, d_v in {64, 128} (step: also 16, 32); fp32 d_k, d_v in {16, 32, 64, 128};
 * any B, T >= 0, B*T < 2^30.
 */
typedef struct dr_linear_desc {
    int B, T, H, d_k, d_v;
    int num_seqs;
    int io_dtype;
    float scale;
    long long ld_q, ld_k, ld_v;
    long long ld_dq, ld_dk, ld_dv; /* backward                                          */
    int32_t* status;
} dr_linear_desc;

size_t dr_linear_attn_workspace_bytes(const dr_linear_desc* desc);
int dr_linear_attn_fwd(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* h0, const int32_t* cu_seqlens, void* o, float* hT,
                       void* workspace, size_t workspace_bytes, void* stream);
int dr_linear_attn_bwd(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* h0, const void* dO, const float* dhT,
                       const int32_t* cu_seqlens, void* dq, void* dk, void* dv, float* dh0,
                       void* workspace, size_t workspace_bytes, void* stream);
int dr_linear_attn_step(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                        const float* g, float* state, void* o, void* stream);

/*
 * Self-test of the device failure path (no counterpart on the pages).  Launches one
 * warp that waits, with the bounded wait every tensor-core kernel uses, on an mbarrier
 * phase that only completes when `arrive` is non-zero (the warp completes it itself);
 * a wait that runs out after limit_ns records DR_ERR_TIMEOUT in the workspace error
 * word, as the kernels do.  The workspace needs only its first 16 bytes (16-byte
 * aligned, device memory).  limit_ns in [0, 1e8].  Read the outcome with
 * dr_check_status: DR_ERR_TIMEOUT without `arrive`, DR_OK with it.  Nothing is copied
 * and no tensor memory is held, so the expired wait leaves nothing in flight.
 * Errors: DR_ERR_INVALID_ARG (NULL or misaligned workspace, limit out of range),
 * DR_ERR_CUDA (launch).
 */
int dr_selftest_wait(void* workspace, int arrive, long long limit_ns, void* stream);

/* Synchronise `stream` and report any device-side error recorded in the
   workspace by the last call that used it (DR_OK or DR_ERR_TIMEOUT), or
   DR_ERR_CUDA when the stream itself failed.  The same call reads the status word of a
   dr_cache (pass its address): DR_OK, DR_ERR_INDEX or DR_ERR_TIMEOUT. */
int dr_check_status(const void* workspace, void* stream);

/*
 * Kernel-level timing.  dr_trace_enable(n) (n > 0) creates n pairs of CUDA
 * events; while enabled, each of the next n kernel launches made by dr_fwd /
 * dr_bwd is bracketed by an event pair recorded on the call's stream.
 * dr_trace_enable(0) disables tracing and destroys the events;
 * dr_trace_reset() reuses them from the first slot.  dr_trace_get(i, ...)
 * waits for launch i to finish and returns its kernel name and device
 * duration in milliseconds.  Host-global state: not for concurrent callers.
 */
int dr_trace_enable(int max_launches);
int dr_trace_count(void);
void dr_trace_reset(void);
int dr_trace_get(int index, const char** kernel_name, float* milliseconds);

/* Human-readable name of a dr_status_code. */
const char* dr_error_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* DR_H */
