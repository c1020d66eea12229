/*
 * libpdscan -- hard-selection PD-SSM forward pass for AMD Instinct MI355X
 * (gfx950).  C ABI: plain pointers and sizes, no C++ or framework types.
 *
 * What is computed (per batch element b, head h, step t):
 *   scores  s_t[k] = sum_c W_sel[h,k,c] u_t[c]                 (k < K)
 *   select  k*_t   = lowest k with s_t[k] = max_j s_t[j]
 *   diag    D_t[n] = 1 / (1 + exp(-(sum_c W_d[h,n,c] u_t[c] + b_d[h,n])))
 *   step    h_t[i] = Bu_t[i] + sum_{j : dict[h,k*_t,j] = i} D_t[j] h_{t-1}[j]
 *   output  y_t    = sum_i C[h,i] h_t[i]
 * with h_{-1} = h0 and h_L the state after the last step.
 *
 * Sources: "Flash PD-SSM: Memory-Optimized Structured Sparse State-Space
 * Models" (gist.science explainer), technical summary -- methodology item 1
 * (scores from a linear map of u_t, argmax over a precomputed dictionary of K
 * sparse matrices, the chosen matrix a one-hot column selector, O(LN) memory)
 * and item 3 (three-phase chunked kernel: per-chunk sequential recurrences,
 * an inter-chunk prefix scan of carry states, a carry correction).  Readings
 * where the pages are silent: column j of the selected matrix carries its one
 * in row dict[h,k*,j]; the transition is that selector times diag(D_t); D_t
 * is the logistic of a second linear map; Bu is supplied by the caller; C has
 * one output per head.
 *
 * Conventions shared by every entry point
 *   - Every tensor argument is a caller-owned DEVICE pointer, row-major and
 *     contiguous, 16-byte aligned.  Shapes are given below in brackets.
 *   - u, W_sel and W_d are fp32 (dims.in_dtype = PDSSM_F32) or bf16
 *     (PDSSM_BF16, stored as raw 16-bit words).  Everything else is fp32
 *     (int32 for indices).
 *   - u is [B,H,L,d_in] when dims.u_shared = 0, or [B,L,d_in] shared by all
 *     heads when dims.u_shared = 1.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *     stream).  PDSSM_OK means "enqueued".  Faults surface at the caller's
 *     next synchronisation.
 *   - The library allocates nothing, never synchronises the device and holds
 *     no global mutable state: scratch memory comes from the caller's
 *     workspace.  Two calls that share one workspace must be ordered on one
 *     stream.
 *   - Workspace header.  Every call that takes a workspace clears it first;
 *     its 32-bit word at byte offset 4 is then nonzero when a look-back wait
 *     of that call (the inter-chunk carry, phase B) gave up after about 4M
 *     window reads.  The affected chunks then continued from the zero carry
 *     (h0 in the forward scans), so y, h_L and every gradient or sensitivity
 *     output of that call are wrong.  A wait ends only when the preceding
 *     chunks have published, which every launch order the runtime uses
 *     guarantees; the word guards against a stalled device.  Read it with
 *     pdssm_workspace_status after the call, on the same stream.
 *     (Test hook: with PDSSM_TEST_LOOKBACK_GIVEUP=1 in the environment every
 *     wait ignores the carries it finds and gives up after two reads, so a
 *     test can set the word on purpose.  Never set it in normal use.)
 *   - Tuning hook: PDSSM_XCD_HEAD_GROUPS = 0, 1, 2, 4 or 8 in the environment
 *     overrides how the general fused kernel groups its (b, h) sequences
 *     over the eight dies (0: no grouping).  Results do not depend on it.
 *   - Arguments are validated on the host before any HIP call.  On failure
 *     nothing is enqueued and a negative pdssm_status is returned; the
 *     calling thread's pdssm_last_error() then describes the problem.
 *   - Preconditions NOT checked on the device: dict values lie in [0, N);
 *     inputs are finite.
 *   - Shape limits (else PDSSM_EUNSUPPORTED): 1 <= N <= 64, 1 <= K <= 64,
 *     K + N <= 128, d_in % 8 == 0, d_in <= 8192, and the per-chunk on-chip
 *     footprint (about chunk * (N + 2) * 4 bytes) within 64 KiB (the folded
 *     and multi-output calls on the general kernel: within 160 KiB, see
 *     pdssm_fwd_wb).
 */
#ifndef PDSCAN_H
#define PDSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PDSSM_ABI_VERSION 1

typedef enum {
  PDSSM_OK = 0,
  PDSSM_EINVAL = -1,        /* bad argument: NULL, size <= 0, misaligned, aliasing */
  PDSSM_EUNSUPPORTED = -2,  /* valid but outside the shape limits above           */
  PDSSM_EWORKSPACE = -3,    /* workspace smaller than the matching *_workspace_bytes */
  PDSSM_EHIP = -4           /* a HIP launch or runtime call failed                */
} pdssm_status;

typedef enum { PDSSM_F32 = 0, PDSSM_BF16 = 1 } pdssm_dtype;

typedef struct {
  int32_t B, H, L, N, K, d_in;
  int32_t u_shared; /* 0: u is [B,H,L,d_in]; 1: u is [B,L,d_in], read by every head */
  int32_t in_dtype; /* pdssm_dtype of u, W_sel and W_d                               */
} pdssm_dims;

/* Selection: scores, argmax and the logistic diagonal for every (b,h,t)
 * ("Flash PD-SSM" summary, Methodology 1: fp32 scores over the K dictionary
 * entries, the argmax with ties to the lowest index, D = sigmoid(W_d u + b_d)).
 *   u [B,H,L,d] | [B,L,d]; W_sel [H,K,d]; W_d [H,N,d]; b_d [H,N]
 *   k_star [B,H,L] int32 (out, required); D [B,H,L,N] fp32 (out, required)
 *   dict_idx [H,K,N] int32 and P_idx [B,H,L,N] int32: optional pair.  When
 *   P_idx is non-NULL it receives dict_idx[h, k*_t, :] (the selected matrix as
 *   its N row indices) and dict_idx must be non-NULL; otherwise both may be
 *   NULL.
 * Score GEMMs run as fp32 MFMA for fp32 inputs and for bf16 inputs with
 * d_in < 128 (bf16 products are exact in fp32), and as bf16 MFMA with fp32
 * accumulation for bf16 inputs with d_in >= 128.  With u shared by the heads
 * in bf16 (K <= 32, N <= 64 a multiple of 4, d_in a multiple of 64, B*L below
 * 2^31) the selection runs as one bf16 GEMM over all tokens and heads (the
 * heads of each 256-token tile on one die, so the tile is read from HBM once). */
int pdssm_select(const pdssm_dims* dims, const void* u, const void* W_sel,
                 const int32_t* dict_idx, const void* W_d, const float* b_d,
                 int32_t* k_star, float* D, int32_t* P_idx, void* stream);

/* Bytes of workspace pdssm_scan_fwd needs for these dims and chunk length. */
int pdssm_scan_workspace_bytes(const pdssm_dims* dims, int32_t chunk, size_t* bytes);

/* Chunked scan given selections: phases A, B and C.
 *   k_star [B,H,L] int32; dict_idx [H,K,N] int32; D [B,H,L,N]; Bu [B,H,L,N];
 *   C [H,N]; h0 [B,H,N] or NULL (zero state)
 *   y [B,H,L] (out); h_L [B,H,N] (out)
 *   chunk >= 1: steps per chunk (the last chunk may be shorter).  Results do
 *   not depend on chunk beyond floating-point rounding.
 *   workspace: device scratch of at least pdssm_scan_workspace_bytes bytes;
 *   its contents on entry do not matter. */
int pdssm_scan_fwd(const pdssm_dims* dims, int32_t chunk, const int32_t* k_star,
                   const int32_t* dict_idx, const float* D, const float* Bu,
                   const float* C, const float* h0, float* y, float* h_L,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace pdssm_fwd needs for these dims and chunk length.  For
 * the shapes pdssm_fwd runs as two passes (below) this includes room for k*
 * and D: B*H*L*(N+1)*4 bytes beyond the look-back words. */
int pdssm_fwd_workspace_bytes(const pdssm_dims* dims, int32_t chunk, size_t* bytes);

/* Selection + chunked scan.  Arguments as in pdssm_select and
 * pdssm_scan_fwd; k_star [B,H,L] and D [B,H,L,N] are optional outputs (NULL:
 * not written).
 * Passes.  One fused kernel reads u and Bu once, except for u shared by the
 * heads with N > 32 and the shapes of pdssm_select's all-heads GEMM: there
 * the GEMM writes k* and D (into the caller's outputs, or the workspace) and
 * the chunked scan of pdssm_scan_fwd reads them, on the same stream.  Results
 * agree to the tolerances of both paths (k* identical; y and h_L differ by
 * rounding order only).
 * Score precision.  fp32 inputs on the step-major kernel (per-head u, N <= 16,
 * K <= 16, d_in in {32, 64}) form every product on the bf16 matrix cores from
 * an exact three-piece split of each fp32 operand (x = x0 + x1 + x2, each
 * piece the next eight significant bits), keeping the six piece products
 * whose weight is at least 2^-16 of |x w| and accumulating in fp32: the
 * dropped terms are below 2^-23 |x w|, so the scores carry fp32 accuracy.
 * Other fp32 shapes use fp32 MFMA; bf16 inputs use bf16 MFMA (d_in >= 128)
 * or exact fp32 MFMA products (d_in < 128). */
int pdssm_fwd(const pdssm_dims* dims, int32_t chunk, const void* u, const void* W_sel,
              const int32_t* dict_idx, const void* W_d, const float* b_d,
              const float* Bu, const float* C, const float* h0,
              int32_t* k_star, float* D, float* y, float* h_L,
              void* workspace, size_t workspace_bytes, void* stream);

/* Look-back scratch the allocation-free call below holds on each device. */
#define PDSSM_NOALLOC_SCRATCH_BYTES (16u << 20)

/* pdssm_fwd without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation).  Arguments and outputs as in pdssm_fwd, always on the
 * single fused kernel (never the two-pass route, whose k* and D would need
 * room); its look-back scratch lives in a 16 MiB device array that the
 * library holds on each GPU it runs on, until the process ends.
 *   status: optional (NULL: not written); one uint32 in device memory or
 *     pinned host memory, 4-byte aligned.  The call ORs its look-back error
 *     word into status[0] (nonzero = a wait gave up; see "Workspace header").
 * Every call on a GPU uses that GPU's one array (the array of the device
 * current at the call): two calls that may overlap on one GPU (different
 * streams, or host threads without ordering) race and give wrong results;
 * order them on one stream.  Each call clears the part of the array it uses
 * first, so nothing carries over from the previous call.  The array is found
 * on the first call on each device; calls allocate nothing.
 * Returns PDSSM_EUNSUPPORTED when the call needs more scratch than
 * PDSSM_NOALLOC_SCRATCH_BYTES (the fused kernel's look-back words above 16
 * MiB), with the other statuses as pdssm_fwd. */
int pdssm_fwd_noalloc(const pdssm_dims* dims, int32_t chunk, const void* u, const void* W_sel,
                      const int32_t* dict_idx, const void* W_d, const float* b_d,
                      const float* Bu, const float* C, const float* h0,
                      int32_t* k_star, float* D, float* y, float* h_L,
                      uint32_t* status, void* stream);

/* pdssm_fwd with the drive term computed in the same pass: Bu_t = W_b u_t
 * (the input map B of the state-space recurrence, "Flash PD-SSM" summary,
 * problem statement and methodology item 1) is a third set of columns of the
 * selection GEMM, so Bu is never read from or written to memory.
 *   W_b [H,N,d_in] (in, u's dtype): row n holds the weights of state row n.
 *   All other arguments, the workspace (pdssm_fwd_workspace_bytes) and the
 *   outputs as in pdssm_fwd (u per head or shared by the heads).  The
 *   products are formed like the scores (fp32 for fp32 inputs, bf16 x bf16
 *   with fp32 accumulation for bf16 inputs with d_in >= 128).
 * Shapes: the step-major kernel (per-head u, N <= 16, K <= 16, chunk <= 512,
 * fp32 d_in in {16, 32, 64} or bf16 d_in = 128: W_b is a third MFMA tile) and
 * the general kernel (every other shape: the drive terms of a chunk go to an
 * on-chip [N][chunk] buffer) when its selection GEMM holds the columns:
 * K + 2N <= 128, or for bf16 inputs with d_in >= 256 (a multiple of 32)
 * ceil(K/16) + 2 ceil(N/16) <= 10 tiles (N = 64 with K <= 32).  On the
 * general kernel the chunk's on-chip footprint (about chunk * (2N + 2) * 4
 * bytes plus the dictionary tables) may take up to the 160 KiB LDS of one
 * compute unit.  Anything else returns PDSSM_EUNSUPPORTED.
 * Exception: u shared by the heads in bf16 with N > 32 (the shapes of
 * pdssm_fwd's two passes) runs the all-heads selection GEMM, a second GEMM of
 * the same tiles that writes Bu = W_b u into the workspace, then the chunked
 * scan (pdssm_scan_fwd_multi with n_out rows): Bu passes through memory
 * there, and the on-chip limit above does not apply. */
int pdssm_fwd_wb(const pdssm_dims* dims, int32_t chunk, const void* u, const void* W_sel,
                 const int32_t* dict_idx, const void* W_d, const float* b_d,
                 const void* W_b, const float* C, const float* h0,
                 int32_t* k_star, float* D, float* y, float* h_L,
                 void* workspace, size_t workspace_bytes, void* stream);

/* Chunked scan that also writes the state after every step.
 *   Arguments as in pdssm_scan_fwd (same workspace size), plus
 *   H_all [B,H,L,N] (out): h_t for t = 0..L-1, the states the gradient pass
 *   below reads.  Each lane group replays its sub-chunk from its true entering
 *   state, so y here is the sequential recurrence itself. */
int pdssm_scan_states(const pdssm_dims* dims, int32_t chunk, const int32_t* k_star,
                      const int32_t* dict_idx, const float* D, const float* Bu, const float* C,
                      const float* h0, float* y, float* h_L, float* H_all, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Bytes of workspace pdssm_scan_bwd needs for these dims and chunk length
 * (PDSSM_EUNSUPPORTED when its on-chip layout, about chunk * N * 4 bytes
 * plus the dictionary, exceeds 64 KiB). */
int pdssm_scan_bwd_workspace_bytes(const pdssm_dims* dims, int32_t chunk, size_t* bytes);

/* Gradient of a scalar loss through the scan for fixed selections
 * ("Flash PD-SSM" summary, methodology item 2 covers the selection's own
 * surrogate gradient, which is not computed here: k* carries no gradient).
 * Given dLoss/dy and dLoss/dh_L, the adjoint recurrence
 *   lam_{L-1} = C g_y[L-1] + g_hL,  lam_t = C g_y[t] + A_{t+1}^T lam_{t+1}
 * gives
 *   g_Bu [B,H,L,N] = lam_t                              (out, required)
 *   g_D  [B,H,L,N] = lam_t[dict[h,k*_t,j]] h_{t-1}[j]   (out, required)
 *   g_h0 [B,H,N]   = A_0^T lam_0                        (out, optional)
 *   g_C  [H,N]     = sum over b and t of g_y h_t        (out, required)
 * Inputs: k_star, dict_idx, D, C and h0 (NULL = zero) as in the forward
 * call; H_all [B,H,L,N] the forward states (pdssm_scan_states); g_y [B,H,L];
 * g_hL [B,H,N] or NULL (zero).  chunk: as in the forward scan.  g_C is summed
 * in a fixed order, so results are bit-identical from run to run. */
int pdssm_scan_bwd(const pdssm_dims* dims, int32_t chunk, const int32_t* k_star,
                   const int32_t* dict_idx, const float* D, const float* C, const float* h0,
                   const float* H_all, const float* g_y, const float* g_hL, float* g_Bu,
                   float* g_D, float* g_h0, float* g_C, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Several outputs per head: y_t = C h_t ("Flash PD-SSM" summary, methodology
 * item 1) with C holding n_out rows per head, the output channels of a layer
 * that reads u and writes y.  The pass of pdssm_fwd_wb with
 *   n_out  1 <= n_out <= 4 (else PDSSM_EINVAL);
 *   C      [H,n_out,N] fp32 (in): row o of head h is C[h,o,:];
 *   y      [B,H,L,n_out] fp32 (out): y[b,h,t,o] = C[h,o,:] . h_t.
 * Everything else, the workspace (pdssm_fwd_workspace_bytes) and the shape
 * limits as in pdssm_fwd_wb.  The on-chip output weights grow with n_out
 * (n_out * N * chunk * 4 bytes), so the longest chunk shrinks with it
 * (step-major kernel, N = 16: n_out = 2 up to chunk 256, n_out = 3 or 4 up to
 * 128; general kernel within 160 KiB, e.g. N = 64 with d_in = 768 and the
 * drive folded: n_out = 2 up to chunk 128); a chunk that does not fit returns
 * PDSSM_EUNSUPPORTED. */
int pdssm_fwd_wb_multi(const pdssm_dims* dims, int32_t chunk, int32_t n_out, const void* u,
                       const void* W_sel, const int32_t* dict_idx, const void* W_d, const float* b_d,
                       const void* W_b, const float* C, const float* h0, int32_t* k_star, float* D,
                       float* y, float* h_L, void* workspace, size_t workspace_bytes, void* stream);

/* pdssm_scan_fwd with several outputs per head: C [H,n_out,N] and
 * y [B,H,L,n_out] as in pdssm_fwd_wb_multi; 1 <= n_out <= 4.  The step-major
 * scan (N <= 16, K <= 16, chunk <= 512) or the general one; a chunk whose
 * per-output on-chip rows do not fit returns PDSSM_EUNSUPPORTED.  Workspace
 * as pdssm_scan_workspace_bytes. */
int pdssm_scan_fwd_multi(const pdssm_dims* dims, int32_t chunk, int32_t n_out, const int32_t* k_star,
                         const int32_t* dict_idx, const float* D, const float* Bu, const float* C,
                         const float* h0, float* y, float* h_L, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Bytes of workspace pdssm_impulse_sens needs for these dims and chunk length
 * (256 + nC * B * H * 4 * N * 8 bytes: per chunk, its composed PD map and the
 * inclusive map entering the next chunk, 2 N tagged words each; no tangent
 * state crosses a chunk). */
int pdssm_impulse_sens_workspace_bytes(const pdssm_dims* dims, int32_t chunk, size_t* bytes);

/* Sensitivity of every output to the first input, dY[b,h,t,:] = dy_t / du_0,
 * for fixed selections ("Breaking the Memory Wall: Exact Analytical
 * Differentiation via Tiled Operator-Space Evolution" summary: exact
 * derivatives over long sequences without storing the graph; here the
 * 128k-step impulse-response derivative of this layer).  u_0 enters step 0
 * through D_0 = sigmoid(W_d u_0 + b_d) and the drive W_b u_0, so the state
 * tangent after step 0 is J = W_b + P_0 diag(D_0 (1 - D_0) h0) W_d, and
 * dY_t = C A_t ... A_1 J (k*_0 carries no derivative).
 *   k_star [B,H,L], dict_idx [H,K,N], D [B,H,L,N] (in): the selections of a
 *     forward pass (pdssm_select, or pdssm_fwd's optional outputs).
 *   W_d, W_b [H,N,d_in] (in, dtype in_dtype); C [H,N]; h0 [B,H,N] or NULL.
 *   dY [B,H,L,d_in] fp32 (out).
 * Shapes: per-head layout, N <= 16, d_in a multiple of 16 and at most 128,
 * on-chip layout within 64 KiB (chunk <= 512); else PDSSM_EUNSUPPORTED. */
int pdssm_impulse_sens(const pdssm_dims* dims, int32_t chunk, const int32_t* k_star,
                       const int32_t* dict_idx, const float* D, const void* W_d, const void* W_b,
                       const float* C, const float* h0, float* dY, void* workspace,
                       size_t workspace_bytes, void* stream);

/* The scan of pdssm_scan_fwd on per-step column maps instead of a
 * dictionary and selections: P_idx [B,H,L,N] (in) holds, for every step, the
 * row of column j's one (as pdssm_soft_select or pdssm_select's P_idx write
 * it; values in [0, N)).  dims->K is ignored.  Workspace as
 * pdssm_scan_workspace_bytes.  With N <= 16 and chunk <= 512 the maps stream
 * through registers; otherwise an on-chip table holds one map per step of a
 * chunk (chunk * (N + 1) * 8 bytes), and a chunk whose table does not fit
 * (N = 16: above 512; N = 20: above 548) returns PDSSM_EUNSUPPORTED. */
int pdssm_scan_fwd_pidx(const pdssm_dims* dims, int32_t chunk, const int32_t* P_idx, const float* D,
                        const float* Bu, const float* C, const float* h0, float* y, float* h_L,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Selection of the original (soft-selection) PD-SSM, kept as a comparison
 * path ("Flash PD-SSM" summary, background: the original model mixes dense
 * dictionary matrices and sparsifies the mixture column by column, at
 * O(L N^2) memory).  Per step t of sequence (b, h):
 *   alpha_t = softmax(W_sel u_t), M_t = sum_k alpha_t[k] M[h,k]  (written to M_t),
 *   P_idx_t[j] = lowest row i with M_t[i, j] maximal (column hardmax),
 *   D_t = sigmoid(W_d u_t + b_d).
 *   u, W_sel, W_d, b_d as in pdssm_select (fp32 or bf16); M [H,K,N,N] fp32,
 *   M[h,k,i,j] = row i, column j.  Outputs: M_t [B,H,L,N,N], P_idx [B,H,L,N],
 *   D [B,H,L,N] (all required).  fp32 arithmetic.
 * Shapes: N <= 16, K <= 16, d_in in {16, 32, 64, 128}; else PDSSM_EUNSUPPORTED. */
int pdssm_soft_select(const pdssm_dims* dims, const void* u, const void* W_sel, const float* M,
                      const void* W_d, const float* b_d, float* M_t, int32_t* P_idx, float* D,
                      void* stream);

/* The sparse dictionary of the hard-selection path from dense parameters:
 * dict_idx[h,k,j] = lowest row i with M[h,k,i,j] maximal (column hardmax of
 * every dictionary matrix; "Flash PD-SSM" summary, methodology item 1).
 *   M [H,K,N,N] fp32 (in); dict_idx [H,K,N] int32 (out). */
int pdssm_dict_hardmax(int32_t H, int32_t K, int32_t N, const float* M, int32_t* dict_idx, void* stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head: the state-space recurrence of
 * the calls above with the transition a_t I in place of P D and an outer
 * product as the drive, the layer that hybrids mix with PD-SSM layers.  Per
 * sequence b and value head h (its query / key head is h / (H / Hk)):
 *   S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T       S [dk, dv], S_{-1} = h0
 *   o_t = scale * S_t^T q_t                          h_L = the last S
 *
 * Conventions of the linattn calls where they differ from those above:
 *   - q, k, v, o, log_decay and their gradients are pdssm_views: a device
 *     pointer and element strides of the batch, head and step axes; the last
 *     axis is contiguous.  [B,H,L,d], [B,L,H,d] and slices of a wider row all
 *     pass as they are.  The pointer and every stride are multiples of 16
 *     bytes (log_decay: 4); strides are >= 0, and an input's may be 0
 *     (broadcast).  The stride of an axis of one element is not looked at.
 *   - q, k, v, o and their gradients have one type, in_dtype.  log_decay, the
 *     states and their gradients are fp32, states contiguous [B,H,dk,dv].
 *   - log_decay <= 0, finite or minus infinity (the state starts anew: its
 *     exponential is zero).  Not checked on the device.
 *   - q, k, v, g_o and the states are finite (as everywhere in this library:
 *     not checked).  A token that is not finite can spoil every output of
 *     its chunk of 64 tokens, and of the rest of its sequence; in a gradient
 *     also g_log_decay over its segment of up to 512 steps.
 *   - packed = 1: one step axis of L rows holds B sequences end to end;
 *     sequence b has the rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (device,
 *     int32 [B+1], not decreasing, within [0, L]; lengths of 0 pass h0 on).
 *     Rows outside every sequence are neither read nor written.  Offsets out
 *     of [0, L] or out of order are cut to it: nothing outside the tensors is
 *     touched, the results of the sequences concerned are unspecified.
 *   - Outputs must not overlap inputs, one another or themselves.
 *   - Results are the same from run to run, bit for bit.
 *   - The workspace header's error word stays zero: no call here waits for
 *     another workgroup.
 *   - Shape limits (else PDSSM_EUNSUPPORTED): dk and dv multiples of 8, at
 *     most 256; step strides at most 2^23 elements, and H * dk likewise where
 *     the gradient sums over shared heads; H times the sequences (or the
 *     segments, of 64 steps and more, that few long ones are cut into) at most
 *     (2^31 - 1) / 6.  The workspace queries apply the last of these too.
 * Precision: decay sums are held in 64 bits, states, weights and sums in
 * fp32.  On the matrix cores bf16 inputs are exact; what is computed enters
 * as two bf16 pieces where a bf16 output comes of it (2^-18 of a term) and as
 * three (24 bits) where an fp32 one does; fp32 inputs are three pieces, of
 * whose nine products the six largest are formed (2^-26 of a term is left).
 * Values under about 1e-30 in size lose digits there.  The decay over a chunk
 * is rounded to fp32; a constant decay is off to the same side in every chunk:
 * 1e-6 of a state that remembers 8192 steps. */
typedef struct {
  int32_t B;               /* sequences */
  int32_t H, Hk;           /* value heads; query / key heads (Hk divides H) */
  int32_t L;               /* steps per sequence; packed: rows of the step axis */
  int32_t dk, dv;
  int32_t in_dtype;        /* pdssm_dtype of q, k, v, o and their gradients */
  int32_t packed;          /* 1: cu_seqlens holds the sequences' bounds */
  int32_t decay_per_head;  /* 0: log_decay [B,H,L]; 1: [H], contiguous, one constant a head */
  float scale;
} pdssm_linattn_dims;

typedef struct {
  void* data;
  int64_t stride_b, stride_h, stride_t;   /* elements */
} pdssm_view;

/* Bytes of workspace pdssm_linattn_fwd / pdssm_linattn_bwd need.  With few
 * sequences and heads a long step axis is cut into segments that run side by
 * side, and their states live there. */
int pdssm_linattn_workspace_bytes(const pdssm_linattn_dims* dims, size_t* bytes);
int pdssm_linattn_bwd_workspace_bytes(const pdssm_linattn_dims* dims, size_t* bytes);

/* Prompts.
 *   q, k [B,Hk,L,dk]; v, o [B,H,L,dv]; log_decay [B,H,L] or [H] (views)
 *   cu_seqlens: packed = 1 only (NULL otherwise); h0 [B,H,dk,dv] or NULL (zero)
 *   h_L [B,H,dk,dv] (out, required) */
int pdssm_linattn_fwd(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k,
                      const pdssm_view* v, const pdssm_view* log_decay, const int32_t* cu_seqlens,
                      const float* h0, const pdssm_view* o, float* h_L, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Gradient of a scalar loss, given g_o [B,H,L,dv] and g_hL [B,H,dk,dv] (NULL:
 * zero).  Nothing of the forward pass is kept: the states are formed again.
 *   g_q, g_k [B,Hk,L,dk] (summed over the value heads that share them),
 *   g_v [B,H,L,dv], g_log_decay [B,H,L] or [H] (summed over b and t)
 *   (out, required); g_h0 [B,H,dk,dv] (out, optional)
 * g_log_decay is a difference of sums over the rest of t's segment (512 steps
 * at most) of q . g_q and k . g_k, each without the token's own key and query,
 * and of a product of states; what the sums miss at the segment's other end is
 * taken out along it (at a sequence's start: where h0 is NULL or g_h0 is asked
 * for).  Its error is theirs: 2^-23 of the root of the sum of their squares,
 * 2e-7 to 9e-7 of the gradient's norm.  An element that is small beside its
 * neighbours (a strong decay between weak ones) has fewer digits: at decays
 * around e^-0.02 the median element is good to 4e-7 of itself and one in a
 * hundred to 3e-5 or worse, around e^-3 the median to 6e-6, and what is below
 * 1e-7 of the neighbours has none.  Exactly zero where the decay is zero, and
 * for a first token without a state before it. */
int pdssm_linattn_bwd(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k,
                      const pdssm_view* v, const pdssm_view* log_decay, const int32_t* cu_seqlens,
                      const float* h0, const pdssm_view* g_o, const float* g_hL,
                      const pdssm_view* g_q, const pdssm_view* g_k, const pdssm_view* g_v,
                      const pdssm_view* g_log_decay, float* g_h0, void* workspace,
                      size_t workspace_bytes, void* stream);

/* One token of every row, on a pool of states that is updated in place.
 *   dims: L = 1, packed = 0, B rows.  q, k [B,Hk,dk]; v, o [B,H,dv];
 *   log_decay [B,H] or [H] (views; the step stride is not looked at)
 *   state [n_slots,H,dk,dv] fp32 (in and out)
 *   state_idx [B] int32 on the device: row b's slot; NULL: slot b (B <= n_slots)
 * A negative slot marks an empty row: its o is zero and no state is touched.
 * A slot >= n_slots, or one that an earlier row of the call has, gives NaN in
 * that row's o and touches no state.  The search for an earlier row reads B / 2
 * indices a row and head on average: for batches up to some ten thousand rows. */
int pdssm_linattn_step(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k,
                       const pdssm_view* v, const pdssm_view* log_decay, const int32_t* state_idx,
                       int32_t n_slots, float* state, const pdssm_view* o, void* stream);

/* ------------------------------------------------------------------------
 * Selective state-space layer: a short causal convolution of every channel, a
 * scan whose decay depends on the input, the channel and the state, and the
 * norm around a block.  Where PD-SSM selects a permutation and linear attention has
 * one decay a head, this scan's transition is a diagonal of its own at every
 * step; the layer is mixed with both.
 *
 * Conventions of these calls: those of the linattn calls above, with
 *   - channels as the last, contiguous axis of a view, a multiple of 8 of them; a view
 *     without heads (x, dt, z, y [B,L,D] and their gradients) does not look at stride_h;
 *   - inputs and outputs of one type, in_dtype; weights, scan states and
 *     the gradients of both fp32 and contiguous; a convolution's states hold
 *     inputs as they are, in in_dtype;
 *   - packed = 1, cu_seqlens, rows outside the sequences, offsets out of order:
 *     as there.  L, and B L, at most 2^31 - 256;
 *   - everything is finite (not checked).  What is not spoils its own channel, from its
 *     token on, and in a scan and its gradients what its tile of 32 tokens and
 *     its segment share. */
typedef struct {
  int32_t B;               /* sequences */
  int32_t L;               /* steps per sequence; packed: rows of the step axis */
  int32_t D;               /* channels */
  int32_t W;               /* taps, 2 to 4 */
  int32_t in_dtype;        /* pdssm_dtype of x, y, the states and their gradients */
  int32_t packed;          /* 1: cu_seqlens holds the sequences' bounds */
  int32_t silu;            /* 1: y = v / (1 + e^-v) of the sum v; 0: y = v */
} pdssm_conv_dims;

/* Short causal convolution: y_t = act(bias + sum_j w[:,j] x_{t-W+1+j}).
 *   x, y [B,L,D] (views); w [D,W], bias [D] or NULL (fp32)
 *   x0 [B,W-1,D] or NULL (zero): the rows before each sequence, the oldest first
 *   x_L [B,W-1,D] (out, required): its last rows, those of x0 among them where it
 *     is shorter: x0 of what follows */
int pdssm_conv_fwd(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                   const int32_t* cu_seqlens, const void* x0, const pdssm_view* y, void* x_L, void* stream);

/* Its gradient, given g_y [B,L,D] and g_xL [B,W-1,D] (NULL: zero).
 *   g_x [B,L,D], g_w [D,W], g_bias [D] (out, required); g_x0 [B,W-1,D] (out, optional) */
int pdssm_conv_bwd_workspace_bytes(const pdssm_conv_dims* dims, size_t* bytes);
int pdssm_conv_bwd(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                   const int32_t* cu_seqlens, const void* x0, const pdssm_view* g_y, const void* g_xL,
                   const pdssm_view* g_x, float* g_w, float* g_bias, void* g_x0, void* workspace,
                   size_t workspace_bytes, void* stream);

/* One token of every row on a pool of states, updated in place.
 *   dims: L = 1, packed = 0.  x, y [B,D] (views; the step stride is not looked at)
 *   state [n_slots,W-1,D] (in and out); state_idx [B] or NULL, as in pdssm_linattn_step:
 *   a negative slot gives zeros, one past the pool or of an earlier row NaN. */
int pdssm_conv_step(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                    const int32_t* state_idx, int32_t n_slots, void* state, const pdssm_view* y, void* stream);

typedef struct {
  int32_t B, L, D;         /* as above */
  int32_t N;               /* state values of a channel: a multiple of 8, at most 64 */
  int32_t G;               /* groups of channels that share B and C: D / G is a multiple of 8 */
  int32_t in_dtype, packed;
  int32_t softplus;        /* 1: steps d = log(1 + e^(dt + bias)); 0: d = dt + bias */
} pdssm_selscan_dims;

/* Selective scan, per sequence, channel d (of group d / (D / G)) and state n:
 *   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = (C_t . h_t + skip x_t) silu(z_t),   h_{-1} = h0
 *   x, dt, z, y [B,L,D], Bm, Cm [B,G,L,N] (views; z NULL: no gate)
 *   A [D,N]; skip, dt_bias [D] or NULL (zero); h0 [B,D,N] or NULL (zero)
 *   h_L [B,D,N] (out, required)
 * Steps d_t >= 0 and A <= 0 (not checked; exp(d A) past fp32 overflows).
 * With softplus any dt is a step: the type's lowest value, and minus infinity, are
 * steps of zero, which leave the state as it is.
 * Precision: fp32 throughout, sums of steps over more than a tile formed in 64
 * bits.  A decay is 2^(d (A log2 e)), both products rounded: 2.3 |d A| half steps of
 * fp32 and the exponential's two, so that its error counts where it is not small itself.
 * Decays below 2^-126 are zero.  The e^-|x| of softplus and of fp32 gates is good to two
 * steps whatever x; gates of bf16 calls take a shorter way (1.3 |z| half steps).
 * Where the query answers 0 (enough sequences and channels to run each
 * sequence in one) workspace may be NULL. */
int pdssm_selscan_workspace_bytes(const pdssm_selscan_dims* dims, size_t* bytes);
int pdssm_selscan_fwd(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                      const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                      const float* dt_bias, const int32_t* cu_seqlens, const float* h0, const pdssm_view* y,
                      float* h_L, void* workspace, size_t workspace_bytes, void* stream);

/* Its gradient, given g_y [B,L,D] and g_hL [B,D,N] (NULL: zero).  Nothing of
 * the forward pass is kept: the states are formed again, from states at every 32nd step
 * that the workspace holds (D N / 8 bytes a row, and 8 N a row and workgroup of channels for sums over them).
 *   g_x, g_dt, g_z [B,L,D] (g_z NULL with z), g_B, g_C [B,G,L,N] (views)
 *   g_A [D,N], g_skip [D], g_bias [D] (out, required); g_h0 [B,D,N] (out, optional) */
int pdssm_selscan_bwd_workspace_bytes(const pdssm_selscan_dims* dims, size_t* bytes);
int pdssm_selscan_bwd(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                      const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                      const float* dt_bias, const int32_t* cu_seqlens, const float* h0, const pdssm_view* g_y,
                      const float* g_hL, const pdssm_view* g_x, const pdssm_view* g_dt, float* g_A,
                      const pdssm_view* g_B, const pdssm_view* g_C, float* g_skip, const pdssm_view* g_z,
                      float* g_bias, float* g_h0, void* workspace, size_t workspace_bytes, void* stream);

/* One token of every row on a pool of states, updated in place.
 *   dims: L = 1, packed = 0.  x, dt, z, y [B,D], Bm, Cm [B,G,N] (views; the step stride is not looked at)
 *   state [n_slots,D,N] (in and out); state_idx [B] or NULL, as in pdssm_linattn_step. */
int pdssm_selscan_step(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                       const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                       const float* dt_bias, const int32_t* state_idx, int32_t n_slots, float* state,
                       const pdssm_view* y, void* stream);

typedef enum { PDSSM_GATE_NONE = 0, PDSSM_GATE_BEFORE = 1, PDSSM_GATE_AFTER = 2 } pdssm_gate;

typedef struct {
  int32_t B, H, L;         /* rows */
  int32_t d;               /* elements of a row: a multiple of 8, at most 8192 */
  int32_t in_dtype;        /* pdssm_dtype of x, z, the residual, y and their gradients */
  int32_t gate;            /* pdssm_gate: where silu(z) is multiplied in */
  int32_t per_head;        /* 0: w and res_scale [d]; 1: [H,d] */
  float eps;               /* > 0, a normal number */
} pdssm_norm_dims;

/* Norm before or behind a block, over the last axis of every row:
 *   y = residual + res_scale (w u / sqrt(mean(u^2) + eps)) [silu(z) with PDSSM_GATE_AFTER]
 *   u = x, or x silu(z) with PDSSM_GATE_BEFORE
 *   x, z, residual, y [B,H,L,d] (views; z NULL without a gate; residual NULL: zero)
 *   w, res_scale [H,d] or [d] (res_scale NULL: one)
 * A row's sum of squares has to be within fp32 (elements up to 2e17): a row
 * past it has a norm of zero.
 * B L at most 2^30 - 128, H at most 2^23 - 1, H d with per_head below 2^29. */
int pdssm_norm_fwd(const pdssm_norm_dims* dims, const pdssm_view* x, const float* w, const pdssm_view* z,
                   const pdssm_view* residual, const float* res_scale, const pdssm_view* y, void* stream);

/* Its gradient, given g_y [B,H,L,d]; the residual's is g_y itself.
 *   g_x, g_z [B,H,L,d] (views; g_z NULL without a gate), g_w and g_res_scale
 *   [H,d] or [d] (summed over the heads then; g_res_scale NULL with res_scale) */
int pdssm_norm_bwd_workspace_bytes(const pdssm_norm_dims* dims, size_t* bytes);
int pdssm_norm_bwd(const pdssm_norm_dims* dims, const pdssm_view* x, const float* w, const pdssm_view* z,
                   const float* res_scale, const pdssm_view* g_y, const pdssm_view* g_x, float* g_w,
                   const pdssm_view* g_z, float* g_res_scale, void* workspace, size_t workspace_bytes, void* stream);

/* Static text for a status code. */
const char* pdssm_status_str(int status);

/* Description of the calling thread's most recent failure ("" if none). */
const char* pdssm_last_error(void);

/* PDSSM_ABI_VERSION of the loaded library. */
int pdssm_abi_version(void);

/* Look-back status of the most recent call on `workspace` (any of the calls
 * above that take a workspace): enqueues on `stream` a one-lane kernel that
 * ORs the workspace error word (see "Workspace header" above; nonzero = some
 * look-back wait of that call gave up and its outputs are wrong) into
 * status[0].  Order it after the call on the same stream and read status
 * after synchronising; zero status[0] first, or keep ORing the words of
 * several calls into it to check them all at once.
 *   workspace: the call's workspace (16-byte aligned, at least 256 bytes).
 *   status: one uint32 in device memory or in pinned host memory visible to
 *     the device (4-byte aligned); owned by the caller.
 * Returns PDSSM_EINVAL for NULL or misaligned pointers, PDSSM_EWORKSPACE for
 * fewer than 256 bytes. */
int pdssm_workspace_status(const void* workspace, size_t workspace_bytes, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PDSCAN_H */
