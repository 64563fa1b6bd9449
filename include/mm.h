/*
 * mm.h — C ABI of the GB300 (sm_103a) SwiGLU FFN and top-k MoE forward.
 *
 * The operations follow the MiniMind pages on the FFN / MoE sub-layer:
 *   [L13] MiniMind course, lesson 13 "FFN 与 MoE" (course/13_ffn_and_moe.md),
 *         §0 / §1.2 (SwiGLU equations), §1.5 (router, softmax, top-k, alpha),
 *         §1.6 (load-balancing aux loss), §3 steps 3-6 (module forward).
 *   [CH4] minimind3.com, chapter 4 "前馈网络 MLP & MoE", §4.2 (SwiGLU),
 *         §4.3 (MoE routing, renormalisation, dispatch), §4.4 (aux loss).
 *
 * Conventions shared by every entry point:
 *   - All tensors are dense, row-major, in DEVICE memory owned by the caller,
 *     and 16-byte aligned.  Weights use the nn.Linear layout [out, in]:
 *       Wg, Wu: [I, H]   Wd: [H, I]   Wr: [E, H]   x, y: [T, H].
 *   - dtype selects the element type of x, the weights and y:
 *       MM_DTYPE_BF16 — bf16 storage, fp32 accumulation (tcgen05 tensor
 *                       cores; for T <= 128 (dense FFN) or T <= 64 (MoE)
 *                       one weight-streaming kernel that reads every
 *                       needed weight row once);
 *       MM_DTYPE_F32  — fp32 storage and fp32 SIMT arithmetic (no TF32).
 *     Router logits, probabilities, alpha and the aux loss are always fp32.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call only enqueues work on that stream and returns; none synchronises
 *     the host except mm_check_status().  No call allocates device memory:
 *     scratch lives in the caller's `workspace`, whose size the matching
 *     *_workspace_bytes() function returns.  The one exception is a fixed
 *     array of MM_NOALLOC_SCRATCH_BYTES that the library's module reserves
 *     on every GPU where it is loaded (used only by mm_swiglu_ffn_noalloc).
 *     Calls that share a workspace must be ordered on one stream.  The first 256 bytes of a
 *     workspace hold device-side state (the watchdog word and the counter of
 *     the streaming kernel's grid barrier): zero them once before the
 *     workspace's first use (cudaMemset).  Every call leaves them consistent,
 *     and mm_check_status() zeroes them again after it reports a timeout.
 *   - Argument errors are reported synchronously as a non-zero mm_status
 *     with nothing enqueued.  Device-side watchdog failures (a pipeline wait
 *     that exceeded its time limit) are recorded in the workspace and
 *     reported by mm_check_status().
 *   - The library keeps only a host-side cache of TMA tensor maps keyed by
 *     (device pointer, shape); it is safe to call from one host thread at a
 *     time per process.
 */
#ifndef MM_H_
#define MM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MM_OK = 0,
  MM_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, k > E, ... */
  MM_ERR_UNSUPPORTED = 2,   /* valid but outside this build's limits          */
  MM_ERR_WORKSPACE = 3,     /* workspace null or smaller than required        */
  MM_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed              */
  MM_ERR_TIMEOUT = 5,       /* a device pipeline wait hit its time limit      */
  MM_ERR_RANGE = 6          /* bf16 tensor-core paths: a value of h, or of Wd
                               (forward), or of dh = dy Wd (backward), is
                               beyond the fp16 range (|v| >= 65520) of its
                               intermediate copy; the results may hold
                               inf/NaN.  Recorded on the device, reported by
                               mm_check_status()                              */
} mm_status;

typedef enum { MM_DTYPE_F32 = 0, MM_DTYPE_BF16 = 1 } mm_dtype;

/* Which kernels carry the FFN part of a call (the *_ex entry points). */
typedef enum {
  MM_PATH_AUTO = 0,    /* bf16: streaming up to 128 (dense) / 64 (MoE) tokens, tensor-core GEMMs beyond; f32: SIMT */
  MM_PATH_TENSOR = 1,  /* bf16 only: grouped tcgen05/TMEM GEMMs fed by TMA          */
  MM_PATH_STREAM = 2,  /* bf16 only, T <= 16: weight streaming on the CUDA cores       */
  MM_PATH_SIMT = 3,    /* any dtype: plain fp32-FMA CUDA-core kernels                */
  MM_PATH_STREAM_TC = 4, /* bf16 only, T <= 128 dense / 64 MoE: weight streaming on the tensor cores */
  MM_PATH_TENSOR_GATHER = 5 /* bf16 MoE only: as MM_PATH_TENSOR, but the gate/up GEMM gathers x
                               rows by token index (TMA gather4) and no permuted copy of x
                               is made (a dense FFN call takes MM_PATH_TENSOR) */
} mm_path;

/* Limits of this build. */
#define MM_MAX_EXPERTS 64
#define MM_MAX_TOPK 8

/* Human-readable name of an mm_status value (static string). */
const char* mm_status_string(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
int mm_version(void);

/* Text of the last CUDA failure reported as MM_ERR_CUDA on this host thread
 * (static thread-local storage; empty if none). */
const char* mm_last_error(void);

/* ------------------------------------------------------------------------
 * Dense SwiGLU FFN   ([L13] §0 / §1.2; [CH4] §4.2)
 *
 *   u = Wu x,  g = Wg x,  h = SiLU(g) ⊙ u,  y = Wd h,  SiLU(z) = z·sigmoid(z)
 *
 * x [T,H], Wg/Wu [I,H], Wd [H,I] in; y [T,H] out (overwritten).  g and u
 * never reach memory; h ([T,I]) lives in the workspace, in fp16 on the bf16
 * tensor-core path (with Wd converted to fp16) and fp32 for fp32 inputs.  A
 * value of h or Wd at or beyond the fp16 range (|v| >= 65520) is recorded
 * on the device and reported by mm_check_status() as MM_ERR_RANGE (the
 * weight-streaming paths keep h in fp32 or as a bf16 pair and need no check).
 * Limits: T >= 0 (T = 0 enqueues nothing); H, I >= 1; bf16 tensor and
 * streaming paths need H and I to be multiples of 64.
 * ---------------------------------------------------------------------- */
size_t mm_swiglu_ffn_workspace_bytes(int64_t T, int H, int I, int dtype);

int mm_swiglu_ffn(const void* x, const void* Wg, const void* Wu, const void* Wd,
                  void* y, int64_t T, int H, int I, int dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

int mm_swiglu_ffn_ex(const void* x, const void* Wg, const void* Wu, const void* Wd,
                     void* y, int64_t T, int H, int I, int dtype,
                     void* workspace, size_t workspace_bytes, void* stream, int path);

/* Dense FFN in its MiniMind block ([L13] §3 step 2):
 *   y = x + FFN(RMSNorm(x)),  RMSNorm(x) = x / sqrt(mean_h x_h^2 + norm_eps) * w
 * norm_w [H] in x's dtype.  The normalised rows are written once (x's dtype)
 * for the GEMMs; the residual is added in the down GEMM's epilogue before y's
 * one rounding.  bf16: tensor cores; fp32: CUDA cores.  y must not alias x. */
size_t mm_swiglu_ffn_block_workspace_bytes(int64_t T, int H, int I, int dtype);

int mm_swiglu_ffn_block(const void* x, const void* norm_w, float norm_eps,
                        const void* Wg, const void* Wu, const void* Wd,
                        void* y, int64_t T, int H, int I, int dtype,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Prepared down weights
 *
 * The pages have no counterpart: the bf16 tensor-core prefill path keeps h
 * in fp16 (precision, see the dense FFN above), so it multiplies h by an fp16
 * copy of Wd, which both forwards otherwise make inside every call.  A caller
 * whose weights change less often than it runs the layer converts once:
 *   Wd16 [H, I] fp16 = Wd [H, I] bf16, exact for |w| >= 2^-14 (smaller
 *   magnitudes become fp16 subnormals, absolute error <= 2^-25).
 * A value at or beyond the fp16 range (|w| >= 65520) is recorded as
 * MM_ERR_RANGE in `status_ws` (a workspace of >= 256 bytes read by
 * mm_check_status; nullable: no report).  Asynchronous on `stream`.
 * H * I must be a multiple of 8; pointers 16-byte aligned.
 * ---------------------------------------------------------------------- */
int mm_prepare_down_weights(const void* Wd, void* Wd16, int H, int I, void* status_ws,
                            void* stream);

/* mm_swiglu_ffn_ex with prepared down weights: Wd16 (nullable) is used by the
 * tensor-core path in place of the in-call fp16 copy of Wd. */
int mm_swiglu_ffn_prepared(const void* x, const void* Wg, const void* Wu, const void* Wd,
                           const void* Wd16, void* y, int64_t T, int H, int I, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream, int path);

/* ------------------------------------------------------------------------
 * Dense SwiGLU FFN without caller-provided scratch
 *
 * The pages describe no counterpart of this entry point; it exists for
 * callers that cannot allocate device memory when they run the FFN: code
 * that enqueues work while a CUDA graph is being captured in a mode that
 * forbids cudaMalloc, plug-ins of inference runtimes whose enqueue step
 * must not allocate, and real-time loops that cannot afford the implicit
 * device synchronisation of cudaMalloc / cudaFree.
 *
 * Same arguments and result as mm_swiglu_ffn, minus the workspace: its
 * scratch is a fixed array of MM_NOALLOC_SCRATCH_BYTES bytes of device
 * memory that belongs to this library.  The CUDA runtime reserves it on
 * every GPU where the library is loaded and keeps it until the process
 * exits.  The call allocates nothing.
 *
 *   - Size limit: the call needs mm_swiglu_ffn_workspace_bytes(T, H, I,
 *     dtype) <= MM_NOALLOC_SCRATCH_BYTES.  Anything larger returns
 *     MM_ERR_UNSUPPORTED with nothing enqueued.  For example, with H = 768,
 *     I = 2432 and bf16 this means T <= 2681.
 *   - The first call on each device looks up the array's device address,
 *     with that device current.  Make that first call before any stream
 *     capture starts.
 *   - All calls share the one array, and it keeps the last call's contents.
 *     Calls that overlap on the GPU therefore race: order them on one
 *     stream, or finish one before starting the next.
 *   - Each call first zeroes the array's 256-byte state header on `stream`
 *     (grid-barrier counters and the watchdog word), so a call whose
 *     pipeline wait gave up leaves no state behind for the next one.  That
 *     watchdog word is not readable through mm_check_status: a timed-out
 *     call is not reported.  Stream errors are still reported by the CUDA
 *     runtime.
 * ---------------------------------------------------------------------- */
#define MM_NOALLOC_SCRATCH_BYTES (16u << 20)

int mm_swiglu_ffn_noalloc(const void* x, const void* Wg, const void* Wu, const void* Wd,
                          void* y, int64_t T, int H, int I, int dtype, void* stream);

/* ------------------------------------------------------------------------
 * Top-k MoE forward   ([L13] §1.5, §1.6, §3 steps 4-6; [CH4] §4.3, §4.4)
 *
 *   r = Wr x (+ logit_bias);  p = softmax(r)            (fp32)
 *   S = TopK(p, k): descending p, equal p -> lower expert index first
 *   alpha_e = p_e / (sum_{j in S} p_j + 1e-20)
 *   y = sum_{e in S} alpha_e · SwiGLU_e(x)   — the k terms are added in fp32
 *       and rounded once to y's dtype, in a fixed order per path (results are
 *       deterministic; the pages' index_add_ into y rounds every term, which
 *       costs accuracy)
 *   count_e = #{(t,s): S_t[s] = e},  P_e = sum_t p_{t,e}
 *   aux_loss = E · coef · sum_e (count_e / T) · (P_e / T)
 *
 * Arguments:
 *   x [T,H], Wr [E,H]                 device, dtype
 *   Wg, Wu, Wd                        HOST arrays of E device pointers, one
 *                                     [I,H] / [I,H] / [H,I] matrix per expert
 *   logit_bias                        device fp32 [E], or NULL (no bias: the
 *                                     pages' router exactly)
 *   y [T,H]                           device, dtype, overwritten
 *   topk_idx [T,k]                    device int32, slots in descending p
 *   topk_w [T,k]                      device fp32, alpha of each slot
 *   aux_loss                          device fp32 scalar (coef = 0 gives 0)
 * Limits: T >= 1; 1 <= E <= MM_MAX_EXPERTS; 1 <= k <= min(E, MM_MAX_TOPK);
 * H a multiple of 8 and (E*H + k*E)*4 <= 200 KiB.
 * ---------------------------------------------------------------------- */
size_t mm_moe_workspace_bytes(int64_t T, int H, int I, int E, int k, int dtype);
/* The workspace one path needs (0: the path does not take the shape); the
 * gathering path (MM_PATH_TENSOR_GATHER) needs no T*k*H permuted copy of x. */
size_t mm_moe_workspace_bytes_for_path(int64_t T, int H, int I, int E, int k, int dtype,
                                       int path);

int mm_moe_forward(const void* x, const void* Wr,
                   const void* const* Wg, const void* const* Wu, const void* const* Wd,
                   int64_t T, int H, int I, int E, int k, float coef, int dtype,
                   const float* logit_bias,
                   void* y, int32_t* topk_idx, float* topk_w, float* aux_loss,
                   void* workspace, size_t workspace_bytes, void* stream);

int mm_moe_forward_ex(const void* x, const void* Wr,
                      const void* const* Wg, const void* const* Wu, const void* const* Wd,
                      int64_t T, int H, int I, int E, int k, float coef, int dtype,
                      const float* logit_bias,
                      void* y, int32_t* topk_idx, float* topk_w, float* aux_loss,
                      void* workspace, size_t workspace_bytes, void* stream, int path);

/* ------------------------------------------------------------------------
 * Router variants and saved router statistics   (p-chao.com "MiniMind 学习笔记
 * 08：FeedForward 与 MoE" §10, table of large-scale MoE mechanisms: "router
 * noise" and "z-loss"; §7: the router gradient flows through topk_weight)
 *
 * The table names the two mechanisms without formulas; this build reads
 * them as:
 *   router noise:  r_{t,e} = W_router x_t + logit_bias_e + noise_{t,e}, with
 *                  the caller's draws noise [T, E] (scale included); the
 *                  noisy logits feed softmax, top-k, alpha and aux;
 *   z-loss:        z_loss = z_coef * (1/T) * sum_t lse_t^2,
 *                  lse_t = log sum_e exp(r_{t,e}).
 * router_probs / router_lse return p [T, E] and lse [T] as computed, the
 * statistics a backward pass needs.
 *
 * Every pointer is nullable (NULL: off / not written); an options struct of
 * zeros is the plain mm_moe_forward_ex with path AUTO.  Every path (tensor,
 * streaming, SIMT) takes every option.  Pointers must be 4-byte aligned.
 * ---------------------------------------------------------------------- */
typedef struct {
  int path;                   /* mm_path of the FFN part (MM_PATH_AUTO = 0)        */
  const float* logit_noise;   /* device fp32 [T, E]: router noise, or NULL         */
  float z_coef;               /* z-loss coefficient                                */
  float* z_loss;              /* device fp32 scalar out, or NULL (not computed)    */
  float* router_probs;        /* device fp32 [T, E] out: softmax p, or NULL        */
  float* router_lse;          /* device fp32 [T] out: logsumexp of the logits, or NULL */
  /* MiniMind block ([L13] §3 step 2: hidden + mlp(post_attention_layernorm(hidden))):
   * with norm_weight, the layer's input is x_n = x / sqrt(mean_h x_h^2 + norm_eps) * w
   * (RMSNorm; the router takes it at full precision, the experts rounded to x's
   * dtype); with residual != 0, y = x + MoE(...).  Either one runs the call on the
   * tensor-core (bf16) or CUDA-core GEMMs; the streaming paths return
   * MM_ERR_UNSUPPORTED.  y must not alias x. */
  const void* norm_weight;    /* device [H], x's dtype, or NULL                    */
  float norm_eps;
  int residual;
  /* Prepared down weights (mm_prepare_down_weights): a HOST array of E device
   * pointers to fp16 [H, I] copies of Wd[e], or NULL.  The bf16 tensor-core
   * path then multiplies by them instead of making the fp16 copy inside the
   * call; the other paths read Wd. */
  const void* const* wd_f16;
  /* Router and permute (prefill tensor-core path): 0 runs them as one kernel
   * where all of its blocks fit on the GPU at once (bf16, H <= 768, E <= 16
   * (8 with norm_weight), k <= 4, T <= 128 x the SMs), so that x is read once;
   * its blocks wait for one another at one grid-wide barrier (bounded: after
   * 1 s the call fails with MM_ERR_TIMEOUT), so it assumes no kernel of
   * another stream holds SMs meanwhile.  1 always runs the router and the
   * permute as two kernels with no grid-wide wait.  The results are the same
   * bit for bit. */
  int separate_routing;
} mm_moe_options;

int mm_moe_forward_opts(const void* x, const void* Wr,
                        const void* const* Wg, const void* const* Wu, const void* const* Wd,
                        int64_t T, int H, int I, int E, int k, float coef, int dtype,
                        const float* logit_bias,
                        void* y, int32_t* topk_idx, float* topk_w, float* aux_loss,
                        void* workspace, size_t workspace_bytes, void* stream,
                        const mm_moe_options* opts);

/* Router half of the MoE forward only (logits, softmax, top-k, alpha, aux):
 * same arguments and meaning as mm_moe_forward without the experts and y.
 * expert_counts (device int32 [E], nullable) receives count_e. */
size_t mm_moe_route_workspace_bytes(int64_t T, int E, int k);

int mm_moe_route(const void* x, const void* Wr, int64_t T, int H, int E, int k,
                 float coef, int dtype, const float* logit_bias,
                 int32_t* topk_idx, float* topk_w, float* aux_loss,
                 int32_t* expert_counts,
                 void* workspace, size_t workspace_bytes, void* stream);

/* The same with router variants (opts->path is ignored). */
int mm_moe_route_opts(const void* x, const void* Wr, int64_t T, int H, int E, int k,
                      float coef, int dtype, const float* logit_bias,
                      int32_t* topk_idx, float* topk_w, float* aux_loss,
                      int32_t* expert_counts,
                      void* workspace, size_t workspace_bytes, void* stream,
                      const mm_moe_options* opts);

/* ------------------------------------------------------------------------
 * Backward pass   (training objective L_train = L_lm + L_aux, [L13] step 8;
 * the router's gradient flows only through the selected weights alpha,
 * p-chao.com "MiniMind 学习笔记 08" §7; in aux only P_e carries gradient,
 * [CH4] §4.4)
 *
 * bf16 only, on the tensor cores; H and I multiples of 64.  Inputs and
 * outputs are device memory; every gradient is OVERWRITTEN (not added to).
 * The intermediate dh = dy Wd is kept in the workspace in fp16 (11
 * significant bits); a value beyond the fp16 range is reported by
 * mm_check_status() as MM_ERR_RANGE.
 *
 * Dense FFN: for dy = dL/dy [T, H] (bf16),
 *   dx [T, H] (bf16) and dWg, dWu [I, H], dWd [H, I] (fp32) with
 *   dWd = dy^T h, dh = dy Wd, dU = dh SiLU(g), dG = dh u SiLU'(g),
 *   dx = dG Wg + dU Wu, dWg = dG^T x, dWu = dU^T x  (g and u recomputed).
 * T = 0 zeroes the weight gradients.
 * ---------------------------------------------------------------------- */
size_t mm_swiglu_ffn_backward_workspace_bytes(int64_t T, int H, int I, int dtype);

int mm_swiglu_ffn_backward(const void* x, const void* Wg, const void* Wu, const void* Wd,
                           const void* dy, int64_t T, int H, int I, int dtype,
                           void* dx, float* dWg, float* dWu, float* dWd,
                           void* workspace, size_t workspace_bytes, void* stream);

/* MoE layer: gradients of L = <dy, y> + d_aux * aux_loss + d_z * z_loss
 * (d_aux = d_z = 1 for L_lm + L_aux + L_z), given the forward's saved routing:
 * topk_idx, topk_w (alpha) and router_probs [T, E] from mm_moe_forward_opts
 * (router_lse [T] too when z_coef and d_z are non-zero, else nullable).
 * The router noise and logit bias of the forward are already inside those
 * probabilities.  Outputs:
 *   dx [T, H] (bf16), dWr [E, H] (fp32), dWg[e], dWu[e] [I, H] and dWd[e]
 *   [H, I] (HOST arrays of E device fp32 pointers; an expert no token chose
 *   gets zeros), d_bias [E] (fp32, nullable): the gradient of the logit bias
 *   as a parameter (= sum_t dL/dlogits).
 * Deterministic: every sum runs in a fixed order.
 * ---------------------------------------------------------------------- */
size_t mm_moe_backward_workspace_bytes(int64_t T, int H, int I, int E, int k, int dtype);

int mm_moe_backward(const void* x, const void* Wr,
                    const void* const* Wg, const void* const* Wu, const void* const* Wd,
                    int64_t T, int H, int I, int E, int k, float coef, int dtype,
                    const int32_t* topk_idx, const float* topk_w,
                    const float* router_probs, const float* router_lse,
                    const void* dy, float d_aux, float z_coef, float d_z,
                    void* dx, float* dWr, float* const* dWg, float* const* dWu,
                    float* const* dWd, float* d_bias,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Around the experts' products   (the pages' block of [L13] §3 step 2 and its
 * dispatch of steps 4-5, as separate operators with gradients, for a program
 * that runs the products itself: adapters, a share of the experts, its own
 * grouped GEMM)
 *
 * MM_DTYPE_BF16 and MM_DTYPE_F32; every sum and statistic in fp32, in a fixed
 * order (deterministic), one rounding per output element.  Any width: rows
 * whose byte length is a multiple of 16 move in 16-byte vectors.  None of
 * these calls waits on the device (no watchdog), and none reads or writes the
 * 256-byte header of a workspace.  Outputs overlap neither inputs nor each
 * other, but where a declaration says so.  Workspace sizes are those of the
 * current device; where a size is 0, no workspace is needed (NULL will do).
 * ---------------------------------------------------------------------- */

/* Norms before and after a block, its gate and its residual scale, in one
 * pass over the rows:
 *   p = f * rho_f * post_w,  rho_f = 1 / sqrt(mean_h f^2 + eps)    (post_w NULL: p = f)
 *   r = residual_scale * x + gate * p                              (gate NULL: 1)
 *   n = r * rho_r * pre_w,   rho_r = 1 / sqrt(mean_h r^2 + eps)    (pre_w NULL: no n)
 * x, f, r, n [T, H]; post_w, pre_w [H]; gate [H], or [T, H] with
 * gate_per_token != 0; all of dtype.  n is the norm of r as stored (rounded),
 * which is what the next sub-layer and the backward pass see.  rstd_post /
 * rstd_pre [T] fp32 (nullable) receive rho_f / rho_r for the backward.
 * f NULL: a plain norm, r = x is not written (r, post_w, gate NULL,
 * residual_scale 1, pre_w given).
 * r may be x and n may be f (the same address: an update in place); no other
 * output may overlap an input.  T = 0 enqueues nothing.
 * Limits: 1 <= H <= MM_NORM_MAX_H; eps finite and > 0; residual_scale finite. */
#define MM_NORM_MAX_H 16384

int mm_block_norm(const void* x, const void* f, const void* post_w, const void* gate,
                  int gate_per_token, const void* pre_w, float residual_scale, float eps,
                  int64_t T, int H, int dtype, void* r, void* n, float* rstd_post, float* rstd_pre,
                  void* stream);

/* Its gradient for dn = dL/dn and dr = dL/dr (the residual path's; NULL: zero),
 * given r, f and the forward's rstd:
 *   D  = dr + rho_r pre_w dn - r rho_r^3 mean_h(r pre_w dn)
 *   dx = residual_scale D;  q = gate D
 *   df = rho_f post_w q - f rho_f^3 mean_h(f post_w q)             (post_w NULL: q)
 *   d_post_w = sum_t q f rho_f,  d_pre_w = sum_t dn r rho_r        (fp32 [H])
 *   d_gate = D p: summed over the tokens (fp32 [H]), or per token (dtype [T, H])
 * dn, r, rstd_pre, d_pre_w go with pre_w; rstd_post, d_post_w with post_w; f
 * is needed with post_w or gate and not read without; df NULL: the plain norm
 * (f NULL above).  The fp32 sums need 4-byte alignment only.  Every gradient
 * is overwritten; no output may overlap an input.  T = 0 zeroes the sums.
 * Without pre_w, post_w and a channel gate there are no sums, and no workspace
 * is needed whatever its size. */
size_t mm_block_norm_backward_workspace_bytes(int64_t T, int H, int dtype);

int mm_block_norm_backward(const void* dn, const void* dr, const void* r, const void* f,
                           const void* post_w, const void* gate, int gate_per_token,
                           const void* pre_w, const float* rstd_post, const float* rstd_pre,
                           float residual_scale, int64_t T, int H, int dtype, void* dx, void* df,
                           float* d_post_w, void* d_gate, float* d_pre_w, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Tokens sorted by expert: the assignments (t, s) in the order expert, token,
 * slot; each expert's group starts on a multiple of `align` rows.
 *   offsets [E+1]  first row of each group (offsets[E]: the end of the last)
 *   counts  [E]    assignments per expert
 *   pos     [T, k] row of each assignment; -1 where topk_idx is outside
 *                  [0, E) (dropped: another rank's expert, or over capacity)
 *   perm    [rows] assignment t*k + s of each row; -1 in padding and behind
 *   xs      [rows, H]  xs[pos[t,s]] = x[t]; zeros in a group's padding; rows
 *                  from offsets[E] on are left as they were
 * rows = mm_moe_permuted_rows(T, E, k, align) (-1: outside the limits), the
 * most that any routing can need.  An expert may appear twice in a token.
 * Limits: E <= MM_MAX_EXPERTS, k <= MM_MAX_TOPK (k > E is allowed), align <=
 * MM_PERMUTE_MAX_ALIGN, H <= MM_PERMUTE_MAX_H, T*k <= 2^30.  T = 0 zeroes offsets and counts. */
#define MM_PERMUTE_MAX_ALIGN 1024
#define MM_PERMUTE_MAX_H (1 << 24)

int64_t mm_moe_permuted_rows(int64_t T, int E, int k, int align);
size_t mm_moe_permute_workspace_bytes(int64_t T, int E, int k);

int mm_moe_permute(const void* x, const int32_t* topk_idx, int64_t T, int H, int E, int k,
                   int align, int dtype, void* xs, int32_t* offsets, int32_t* counts,
                   int32_t* perm, int32_t* pos, void* workspace, size_t workspace_bytes,
                   void* stream);

/* And back: y[t] = sum_s topk_w[t,s] ys[pos[t,s]] (fp32, slot order, rounded
 * once; topk_w NULL: weights of 1, which is the gradient of the permute).  A
 * pos outside [0, rows) adds nothing; a token with none gets zeros. */
int mm_moe_unpermute(const void* ys, const int32_t* pos, const float* topk_w, int64_t T, int H,
                     int k, int64_t rows, int dtype, void* y, void* stream);

/* Gradient of the weighted combine:
 *   dys[pos[t,s]] = topk_w[t,s] dy[t],  dw[t,s] = <dy[t], ys[pos[t,s]]>
 * dys: zeros in a group's padding, rows from offsets[E] on left as they were;
 * dw (fp32 [T, k], nullable; needs ys and topk_w): 0 for a dropped assignment.
 * topk_w NULL: dys[pos[t,s]] = dy[t] (the permute of dy by a known order). */
int mm_moe_unpermute_backward(const void* dy, const void* ys, const int32_t* pos,
                              const float* topk_w, const int32_t* offsets, const int32_t* counts,
                              int64_t T, int H, int E, int k, int64_t rows, int dtype, void* dys,
                              float* dw, void* stream);

/* Activations kept in 8 bits.  A row of C values is cut into groups of 32
 * columns (the last one may be short); with amax over the group's finite
 * values, e is the least integer >= -126 with amax <= 448 * 2^e, and
 *   codes [R, C]            e4m3 of x * 2^-e, round to nearest even
 *   exps  [R, ceil(C/32)]   e + 127 (one byte; 2^(exps - 127) is the scale)
 * so that a value of a group is off by at most max(2^-4 |x|, 2^-10 * 2^e).
 * An infinity or a NaN becomes a NaN code and leaves its group's scale alone.
 * Unpacking multiplies back: exact in fp32 and, above its subnormals, in bf16,
 * but for |x| > 1.9375 * 2^127, whose code stands for 2^128: an infinity there.
 * exps are taken as packing writes them (1 .. 247).
 * Limits: C <= MM_CHECKPOINT_MAX_COLS, R*C <= 2^40.  R = 0 enqueues nothing. */
#define MM_CHECKPOINT_MAX_COLS (1 << 20)

int mm_checkpoint_pack(const void* x, int64_t R, int64_t C, int dtype, void* codes, uint8_t* exps,
                       void* stream);
int mm_checkpoint_unpack(const void* codes, const uint8_t* exps, int64_t R, int64_t C, int dtype,
                         void* x, void* stream);

/* The SwiGLU activation of rows gu [R, 2I] (g in columns [0, I), u in
 * [I, 2I)): h = SiLU(g) u in dtype, and (codes / exps, both or neither) its
 * checkpoint: g and u packed as above, each half with its own groups (codes
 * [R, 2I], exps [R, 2 ceil(I/32)]).  n_rows (device int32, nullable): rows
 * from *n_rows on are left alone (the offsets[E] of a permute).  2I <=
 * MM_CHECKPOINT_MAX_COLS.  Here and in the backward exp(-|g|) is good to
 * 2^-20.5 relative for bf16 rows, and to fp32's expf for fp32 rows. */
int mm_swiglu_act(const void* gu, int64_t R, int I, int dtype, const int32_t* n_rows, void* h,
                  void* codes, uint8_t* exps, void* stream);

/* Its backward from the checkpoint's values g, u: with sg = sigmoid(g),
 *   dgu [R, 2I] = [ dh u sg (1 + g (1 - sg)) | dh g sg ],  h [R, I] = g sg u
 * (h nullable: the operand of the down weights' gradient). */
int mm_swiglu_act_backward(const void* codes, const uint8_t* exps, const void* dh, int64_t R, int I,
                           int dtype, const int32_t* n_rows, void* dgu, void* h, void* stream);

/* ------------------------------------------------------------------------
 * Experts' products   (the pages' expert loop of [L13] §3 step 5, for rows
 * sorted by mm_moe_permute or any tables of its form)
 *
 * Group e is rows [offsets[e], offsets[e+1]) of the sorted tensors; its first
 * counts[e] rows hold an assignment, the rest is padding.  offsets (int32
 * [E+1], ascending) and counts (int32 [E]) are device memory; both NULL: all
 * rows are one group (E = 1).  The tables may start at any row; entries
 * outside [0, rows] are taken as the nearest inside.
 * In results that have rows (ys, dxs) a group's padding rows become zeros and
 * rows from offsets[E] on (and before offsets[0]) are left as they were; what
 * stands in padding rows and behind in inputs (NaN too) has no effect.
 * Sums in fp32 in a fixed order (deterministic), one rounding per element.
 * fp32 operands are multiplied on the tensor cores as three bf16 parts each,
 * which hold all 24 bits of every number (six of the nine products; the others
 * are below 2^-25).  Where operands hold an infinity, a NaN or a magnitude of
 * 2^103 or more in a row that counts, the call is made on the CUDA cores
 * instead, and so is each of its results ys, dxs or dw of which a sum reaches
 * 2^80 (of few rows in either case: the results that are touched); with fp32's
 * accuracy, in four to nine times the time.
 * Outputs overlap neither inputs nor each other.  A device wait that exceeded
 * its time limit is recorded in the header of `status_ws` (nullable; a zeroed
 * workspace of >= 256 bytes) or, without one, of `workspace`, for
 * mm_check_status(); with neither there is no report.  Nothing else in a
 * workspace's header is read or written, so that other calls may share the
 * workspace; what it holds behind the header before the call does not matter,
 * and it may be NULL where the size is 0.  Sizes are those of the current
 * device.
 * Limits: E <= MM_MAX_EXPERTS; K, N <= MM_GROUPED_MAX_DIM; rows <=
 * MM_GROUPED_MAX_ROWS.  rows = 0 enqueues nothing, but that dw is zeroed.
 * ---------------------------------------------------------------------- */
#define MM_GROUPED_MAX_DIM (1 << 20)
#define MM_GROUPED_MAX_ROWS ((1 << 30) + (1 << 17))

/* ys[r] = w[e] xs[r]:  xs [rows, K], w [E, N, K], ys [rows, N], all of dtype. */
size_t mm_grouped_matmul_workspace_bytes(int64_t rows, int K, int N, int E, int dtype);

int mm_grouped_matmul(const void* xs, const void* w, const int32_t* offsets, const int32_t* counts,
                      int64_t rows, int K, int N, int E, int dtype, void* ys, void* workspace,
                      size_t workspace_bytes, void* status_ws, void* stream);

/* Its gradients for dys = dL/dys [rows, N]:
 *   dxs[r] = w[e]^T dys[r]  [rows, K] in dtype       (nullable; needs w)
 *   dw[e] = sum over the group's counts[e] rows of dys[r] xs[r]^T, fp32
 *           [E, N, K], overwritten; zeros for an empty group (nullable; needs xs) */
size_t mm_grouped_matmul_backward_workspace_bytes(int64_t rows, int K, int N, int E, int dtype);

int mm_grouped_matmul_backward(const void* dys, const void* xs, const void* w,
                               const int32_t* offsets, const int32_t* counts, int64_t rows, int K,
                               int N, int E, int dtype, void* dxs, float* dw, void* workspace,
                               size_t workspace_bytes, void* status_ws, void* stream);

/* Microscaled 4-bit floating point (OCP MX: e2m1 elements, a power of two per
 * 32 columns).  With amax over a group's magnitudes, e is the least integer
 * >= -126 with amax <= 6 * 2^e, and
 *   codes [R, 16 G]     G = ceil(C/32): e2m1 of x * 2^-e, to nearest, ties to
 *                       the even code, two to a byte (the even column in the
 *                       low half); the last group is filled up with zeros
 *   exps  [ceil(G/4), R, 4]  e + 127 of four neighbouring groups of a row next
 *                       to each other; 127 where there is no group
 * so that a value of a group is off by at most a quarter of itself or, below
 * 2^e, by 2^-2 * 2^e.  A group that holds an infinity or a NaN gets the byte
 * 255 and stands for NaN in all its columns.
 * Dequantising multiplies back: exact in fp32 and bf16, but for |x| above
 * 1.25 * 2^127, whose code can stand for 2^128: an infinity there.
 * Matrices of E experts are quantised as E * N rows.  n_rows (device int32,
 * nullable): rows from *n_rows on are left alone.
 * Limits: C <= MM_GROUPED_MAX_DIM, R <= 2^31 - 1.  R = 0 enqueues nothing. */
int mm_mx4_quantize(const void* x, int64_t R, int64_t C, int dtype, const int32_t* n_rows,
                    void* codes, uint8_t* exps, void* stream);
int mm_mx4_dequantize(const void* codes, const uint8_t* exps, int64_t R, int64_t C, int dtype,
                      const int32_t* n_rows, void* x, void* stream);

/* mm_grouped_matmul with w in 4 bits (codes [E * N, 16 G], exps), for xs in
 * 4 bits (x: codes, x_exps) or in bf16 (x_exps NULL); ys is bf16:
 *   ys[r, n] = sum_k v(xs[r, k]) v(w[e, n, k]),  v() the values stood for
 * (with xs in bf16 those that mm_mx4_dequantize gives in bf16: a weight of 2^128
 * is an infinity there). */
size_t mm_mx4_matmul_workspace_bytes(int64_t rows, int K, int N, int E, int x_in_4_bits);

int mm_mx4_matmul(const void* x, const uint8_t* x_exps, const void* w_codes, const uint8_t* w_exps,
                  const int32_t* offsets, const int32_t* counts, int64_t rows, int K, int N, int E,
                  void* ys, void* workspace, size_t workspace_bytes, void* status_ws, void* stream);

/* ------------------------------------------------------------------------
 * Status
 * ---------------------------------------------------------------------- */
/* Synchronises `stream`, reads and clears the device status word kept at
 * the start of `workspace` (any workspace used by the calls above), and
 * returns MM_ERR_TIMEOUT if a kernel gave up on a pipeline wait since the
 * last check, MM_ERR_RANGE if an fp16 intermediate overflowed (the first
 * failure recorded wins), MM_ERR_CUDA if the stream reported an error, else
 * MM_OK. */
int mm_check_status(void* workspace, void* stream);

/* Self-test of the watchdog: launches one block that waits on a barrier no
 * one arrives on, with the given limit in microseconds (1 .. 10,000,000).
 * The wait gives up, records MM_ERR_TIMEOUT in `workspace` (>= 256 bytes)
 * and the kernel returns normally; mm_check_status() then reports it. */
int mm_watchdog_selftest(void* workspace, size_t workspace_bytes,
                         uint32_t limit_us, void* stream);

/* ------------------------------------------------------------------------
 * Measurement hooks (host-side only; they add no work to the kernels)
 * ---------------------------------------------------------------------- */
typedef enum {
  MM_KERNEL_ROUTER = 1,     /* logits/softmax/top-k/alpha/aux partials      */
  MM_KERNEL_DISPATCH = 3,   /* aux finalisation, group offsets, token permute */
  MM_KERNEL_GATEUP = 4,     /* gate/up GEMM with the SwiGLU epilogue        */
  MM_KERNEL_DOWN = 5,       /* down GEMM with the alpha-scaled combine      */
  MM_KERNEL_DECODE = 7,     /* decode-sized weight-streaming kernel (whole call) */
  MM_KERNEL_BWD_DGRAD = 8,  /* backward: dh = dy Wd and dx = dG Wg + dU Wu GEMMs */
  MM_KERNEL_BWD_SWIGLU = 9, /* backward: gate/up recomputed, SwiGLU derivative */
  MM_KERNEL_BWD_WGRAD = 10, /* backward: weight-gradient GEMMs                */
  MM_KERNEL_BWD_ROUTER = 11, /* backward: dispatch, router gradient, dx combine */
  MM_KERNEL_NORM = 12,      /* block norm, forward and backward             */
  MM_KERNEL_PERMUTE = 13,   /* tokens sorted by expert and back             */
  MM_KERNEL_CHECKPOINT = 14, /* 8-bit checkpoints and the SwiGLU activation */
  MM_KERNEL_GROUPED = 15,   /* experts' products, forward and backward      */
  MM_KERNEL_MX4 = 16        /* 4-bit microscaled quantisation               */
} mm_kernel_id;

/* Number of kernels this library has enqueued since it was loaded. */
uint64_t mm_launch_count(void);

/* Start timing every launch of one kernel (mm_kernel_id) with a pair of CUDA
 * events recorded on the launching stream around it, for at most
 * max_launches launches (1 .. 100000).  The events are created by the
 * library.  Returns MM_ERR_INVALID_ARG for a bad id or count. */
int mm_profile_start(int kernel_id, int max_launches);

/* Stop timing: waits for the last recorded event, returns the summed
 * duration in milliseconds and the number of launches timed. */
int mm_profile_stop(double* total_ms, int* launches);

#ifdef __cplusplus
}
#endif

#endif /* MM_H_ */
