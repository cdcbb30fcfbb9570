/*
 * falcon.h -- C ABI of libfalcon, the forward pass of the Falcon fast-weight
 * memory on NVIDIA B200 (sm_100a).
 *
 * The method ("Fast Weight Attention for Continual Learning", authors'
 * abstract): every head keeps a state S of d_v x d_k numbers. At step t the
 * state is written with the prefix-aligned pair (x_t, y_t) = (phi(k_{t-1}), v_t)
 * by a gated, normalised first-order update, and it is read after the write:
 * o_t = S_t q_t. phi is the identity here.
 *
 *   Falcon-1  (scalar NLMS, squared-error regression):
 *       Sbar = alpha_t S_{t-1};  beta_t = eta_t / (||x_t||^2 + eps)
 *       S_t  = Sbar - beta_t (Sbar x_t - y_t) x_t^T
 *   Falcon-3  (sliding-window mini-batch over the last w pairs, one step):
 *       beta_t = eta_t / (sum_{j in W_t} ||x_j||^2 + eps)
 *       S_t  = Sbar - beta_t sum_{j in W_t} (Sbar x_j - y_j) x_j^T
 *   Falcon-1A / Falcon-3A (negative inner-product objective):
 *       S_t  = Sbar + beta_t sum_{j in W_t} y_j x_j^T
 *   Falcon-2 / Falcon-2A (the per-column extension; a reading of the pages, which
 *   name it without equations): column c of S keeps the running energy of its key
 *   coordinate, n_{t,c} = alpha_t n_{t-1,c} + x_{t,c}^2, and the step is the NLMS
 *   step in the metric D = diag(1 / (n_c + eps)):
 *       z_t = eta_t D x_t / (x_t^T D x_t + eps)
 *       Falcon-2:  S_t = Sbar - (Sbar x_t - y_t) z_t^T     Falcon-2A: S_t = Sbar + y_t z_t^T
 * The step size is the Kaczmarz/NLMS one (Kaczmarz Linear Attention abstract,
 * thelatestinai.com page "Fast Weight Attention for Continual Learning").
 * W_t = {max(1, t-w+1) .. t} (1-based). x_1 = k_prev when a cache is given,
 * else 0 (no write at the first step). A pair whose denominator
 * ||x||^2 + eps is 0 writes nothing (beta = 0). alpha in (0, 1] and eta >= 0
 * are preconditions; they are not checked per element.
 *
 * Conventions shared by every entry point:
 *  - All tensors are dense, row-major, contiguous, in DEVICE memory owned by
 *    the caller. The library never allocates, frees or synchronises (except
 *    falcon_check_device_errors, which synchronises the given stream).
 *  - q, k: (B,H,T,d_k); v, o: (B,H,T,d_v); alpha, eta: (B,H,T) fp32;
 *    S0, S_out: (B,H,d_v,d_k) fp32 with S[i][c] the weight from key
 *    coordinate c to value coordinate i; k_prev, k_last: (B,H,d_k).
 *    q, k, v, o, k_prev and k_last share io_dtype (fp32 or bf16).
 *  - Every pointer must be 16-byte aligned except alpha and eta (4 bytes).
 *  - Calls are asynchronous on `stream` (0 = the legacy default stream).
 *    Shape, pointer, alignment and dtype checks run on the host before any
 *    launch; a failed check launches nothing and returns
 *    FALCON_ERR_INVALID_ARG or FALCON_ERR_UNSUPPORTED.
 *  - A launch failure returns FALCON_ERR_CUDA (the CUDA error is left for
 *    cudaGetLastError to report).
 *  - No exception crosses this boundary.
 */
#ifndef FALCON_H_
#define FALCON_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define FALCON_API __attribute__((visibility("default")))
#else
#define FALCON_API
#endif

/* Same underlying type as cudaStream_t. */
typedef struct CUstream_st *falcon_stream_t;

typedef enum {
    FALCON_OK = 0,
    FALCON_ERR_INVALID_ARG = 1, /* null/misaligned pointer, negative size, bad enum   */
    FALCON_ERR_UNSUPPORTED = 2, /* valid but outside what the kernels implement      */
    FALCON_ERR_WORKSPACE = 3,   /* workspace smaller than falcon_workspace_size()    */
    FALCON_ERR_CUDA = 4,        /* a CUDA launch or runtime call failed              */
    FALCON_ERR_TIMEOUT = 5      /* a bounded device-side wait gave up                */
} falcon_status_t;

typedef enum {
    FALCON_RULE_1 = 1,  /* Falcon-1: scalar NLMS                                  */
    FALCON_RULE_1A = 2, /* Falcon-1A: normalised additive (inner-product) write   */
    FALCON_RULE_3 = 3,  /* Falcon-3: sliding-window mini-batch (window w)         */
    FALCON_RULE_3A = 4, /* Falcon-3A: windowed inner-product write (window w)     */
    FALCON_RULE_2 = 5,  /* Falcon-2: per-column normalised NLMS (see below)       */
    FALCON_RULE_2A = 6  /* Falcon-2A: its inner-product counterpart               */
} falcon_rule_t;

/*
 * Flag OR-ed into a rule value (the `rule` field, or the `rule` argument of
 * falcon_decode_step): write the same-step pair (k_t, v_t) at step t, the
 * association of Kaczmarz Linear Attention (thelatestinai.com page of "Fast Weight
 * Attention for Continual Learning", KLA abstract), instead of the prefix-aligned
 * pair (k_{t-1}, v_t) of the authors' abstract. k_prev is then not used as a key
 * (k_last is still the last key, and the decode step still stores k into k_prev).
 */
#define FALCON_SAME_STEP 0x100

typedef enum { FALCON_F32 = 0, FALCON_BF16 = 1 } falcon_dtype_t;

/* Arguments of the two sequence entry points. Integer fields hold the enums
 * above. */
typedef struct {
    int rule;           /* falcon_rule_t, optionally | FALCON_SAME_STEP               */
    int io_dtype;       /* falcon_dtype_t of q, k, v, k_prev, k_last and o            */
    int B, H, T;        /* batch, heads, tokens (T >= 0)                              */
    int dk, dv;         /* key/query and value widths                                 */
    const void *q;      /* (B,H,T,dk)                                                 */
    const void *k;      /* (B,H,T,dk)                                                 */
    const void *v;      /* (B,H,T,dv)                                                 */
    const float *alpha; /* (B,H,T) decay gate, preconditions 0 < alpha <= 1           */
    const float *eta;   /* (B,H,T) step gate, precondition eta >= 0                   */
    float eps;          /* >= 0, added to the (window) squared key norm                */
    int window;         /* Falcon-3/3A window w >= 1; ignored by Falcon-1/1A           */
    int chunk;          /* chunk-parallel block: 16, 32 or 64 pseudo-value rows        */
    const float *S0;    /* (B,H,dv,dk) initial state, or NULL for zero                 */
    const void *k_prev; /* (B,H,dk) key cached before this segment, or NULL (x_1 = 0);
                           not read with FALCON_SAME_STEP                              */
    void *o;            /* (B,H,T,dv) output, written                                  */
    float *S_out;       /* (B,H,dv,dk) final state, or NULL                            */
    void *k_last;       /* (B,H,dk) last key (the cache for a continuation), or NULL   */
    const float *n0;    /* Falcon-2/2A: (B,H,dk) running column energies to start from,
                           or NULL for zero; ignored by the other rules                */
    float *n_out;       /* Falcon-2/2A: (B,H,dk) running column energies after the
                           sequence (part of the continuation cache), or NULL          */
} falcon_args_t;

/*
 * Bytes of device workspace falcon_fwd_chunk uses for these arguments on the
 * current device (0 when it uses none). Returns 0 for invalid arguments as
 * well; the call itself reports those. Nonzero in two cases, both described at
 * falcon_fwd_chunk:
 *   - the sequence split of the inner-product rules, which needs it: about
 *     (B*H*T/piece + B*H*nseg) * dv*dk*4 bytes, a few tens of MB for 16 heads of
 *     32768 tokens;
 *   - the two-pass path of the regression rules (Falcon-1, and Falcon-3 at
 *     window 1, 2 or 4, on the dk = dv = 128 bf16 kernel), which is optional:
 *     16 KB per block of 64 / window tokens per head, B*H*ceil(T*window/64)*16384
 *     bytes (134 MB for 128 heads of 4096 tokens at window 1); given less, or
 *     NULL, those rules run in one kernel instead.
 * The caller allocates it (16-byte aligned) and owns it; the call only uses it
 * while its kernels run on `stream`.
 */
FALCON_API size_t falcon_workspace_size(const falcon_args_t *args);

/*
 * falcon_fwd_chunk -- chunk-parallel forward pass with positive-decay
 * renormalisation (authors' abstract of "Fast Weight Attention for Continual
 * Learning"; ai.info overview, section Methodology in Plain English, which
 * describes the blocked form).
 *
 * Per block of pseudo-value rows the kernel forms the decay-weighted key Gram
 * and query-key tiles, solves the unit lower-triangular system of the block
 * (Falcon-1/3), applies it to the residuals against the state carried in from
 * the previous block, writes the block's outputs and passes the fp32 state on.
 * Decay factors are only ever formed as exp(g_i - g_j) with i >= j on a
 * block-local cumulative log decay, so each lies in (0, 1].
 *
 * Supported: Falcon-1/1A/3/3A (Falcon-2/2A return UNSUPPORTED here: they run on
 * falcon_fwd_recurrent); io_dtype FALCON_BF16 only; dk, dv in {32, 64, 128}; chunk in
 * {16, 32, 64}; Falcon-3/3A need 1 <= window <= chunk and process
 * floor(chunk / window) tokens per block. Tensor-core products take the bf16
 * inputs as operands with fp32 accumulation and an fp32 state. FALCON_F32
 * inputs return FALCON_ERR_UNSUPPORTED: bf16 operands could not hold them to an
 * fp32 error bound, so fp32-accurate work goes through falcon_fwd_recurrent.
 *
 * Sequence split (inner-product write, window 1, dk = dv = 128, bf16, chunk 64,
 * T a multiple of 64, and room for nseg >= 2 segments of at least 8 blocks each
 * with B*H*nseg <= the SM count; the largest such nseg dividing T/64 is taken):
 * the additive write has a scalar
 * state transition, so each head is cut into nseg segments of whole blocks;
 * one parallel pass forms every piece's state increment
 * sum_t 2^(G_end - G_t) beta_t y_t x_t^T and its decay, a scan gives the state
 * at each segment start, and the segments then run as heads of their own.
 * The result is the same up to rounding; falcon_workspace_size() says when
 * this path is taken and how much workspace it needs.
 *
 * Two-pass path (regression write, window 1, 2 or 4, dk = dv = 128, bf16, chunk
 * 64, when the workspace holds falcon_workspace_size() bytes): the chunk-local step
 * of a block (its Gram matrix, step sizes, L and T = (I + L)^-1) depends only on
 * the block's keys and gates, so a first launch solves every block of every
 * head at once and leaves its two bf16 T tiles in the workspace; the second
 * launch runs the state recurrence over the blocks and reads them. Both paths
 * do the same arithmetic; with less workspace, or NULL, the single kernel runs.
 *
 * `workspace` may be NULL when falcon_workspace_size() is 0.
 * Errors: INVALID_ARG (also a workspace not 16-byte aligned), UNSUPPORTED,
 * WORKSPACE (NULL or smaller than falcon_workspace_size() where the sequence
 * split needs it), CUDA.
 */
FALCON_API falcon_status_t falcon_fwd_chunk(const falcon_args_t *args, void *workspace,
                                 size_t workspace_bytes, falcon_stream_t stream);

/* Size of the fixed scratch array behind falcon_fwd_chunk_noalloc: 32 MiB. */
#define FALCON_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * falcon_fwd_chunk_noalloc -- falcon_fwd_chunk without a caller-provided
 * workspace, for callers that cannot allocate device memory where they run
 * the forward pass: a plugin that receives raw device pointers from a host
 * runtime with no allocator to offer, a serving loop in which a cudaMalloc
 * (which may synchronise the device) is not acceptable, or a process whose
 * device memory is owned by a pool it does not control. The paper has no
 * counterpart; this is a deployment convenience of this library.
 *
 * Arguments, results and errors are those of falcon_fwd_chunk. Where that call
 * uses workspace (falcon_workspace_size() > 0), this one uses a fixed array of
 * FALCON_NOALLOC_SCRATCH_BYTES in the library's device image instead; every
 * GPU that uses the library holds that array until the process exits. A
 * sequence split that needs more is rejected before anything runs with
 * FALCON_ERR_WORKSPACE (use falcon_fwd_chunk with your own workspace then);
 * the regression rules' two-pass path runs when its tiles fit in the array and
 * their single-kernel path otherwise. The call allocates and frees nothing.
 *
 * The array is reserved on a device no later than the first call there (with
 * lazy module loading, the CUDA default, that first call loads it; with eager
 * loading it is reserved when the library loads). The first call on each device
 * resolves the array's device address (with that device current) and keeps it;
 * make that first call before any stream capture. The kept address does not
 * survive cudaDeviceReset: do not use this entry point on a device after
 * resetting it in the same process. All calls share the one array per device: calls whose kernels can
 * overlap on the GPU (different streams without an ordering between them,
 * several host threads) race on it and give wrong results, so order them, for
 * example on one stream. Nothing in the array needs clearing between calls:
 * each call writes every byte it later reads.
 */
FALCON_API falcon_status_t falcon_fwd_chunk_noalloc(const falcon_args_t *args, falcon_stream_t stream);

/*
 * falcon_fwd_recurrent -- recurrent form (authors' abstract; ai.info overview,
 * section Methodology in Plain English): the literal per-token recurrence
 * with an fp32 state and fp32 arithmetic. One CTA per (b, h) walks t = 1..T.
 * Supported: 1 <= dk, dv <= 128; window <= 64 for Falcon-3/3A; `chunk` is
 * ignored. This is the entry point for Falcon-2/2A (with n0 / n_out).
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
FALCON_API falcon_status_t falcon_fwd_recurrent(const falcon_args_t *args, falcon_stream_t stream);

/*
 * falcon_bwd_recurrent -- gradients of the recurrent form for a loss L, given the
 * upstream gradients of the outputs and of the final state. The pages define the
 * forward rules only (authors' abstract); these are their derivatives, taken step by
 * step backwards through the same per-token recurrence (reverse mode):
 *   U = dL/dS_t (U = dS_T after the last step), then for t = T..1:
 *   U += dO_t q_t^T;  dq_t = S_t^T dO_t;
 *   Falcon-1/3 (r_j = Sbar x_j - y_j):  dbeta = -sum_j r_j^T U x_j;
 *     dy_j = beta U x_j;  dx_j = -beta U^T r_j - beta Sbar^T U x_j;  dSbar = U - beta sum_j U x_j x_j^T
 *   Falcon-1A/3A:  dbeta = sum_j y_j^T U x_j;  dy_j = beta U x_j;  dx_j = beta U^T y_j;  dSbar = U
 *   deta_t = dbeta / (N_t + eps);  dx_j += -2 dbeta beta / (N_t + eps) x_j  (N_t the pairs' squared norms;
 *   nothing flows through beta when N_t + eps = 0);  dalpha_t = <dSbar, S_{t-1}>;  U <- alpha_t dSbar.
 * dx of pair j goes to the key row it was read from (k_{j-1}; k_prev for the first pair, or k_j with
 * FALCON_SAME_STEP), dy to v_j, and dS0 is the final U.
 *
 * `args` is the forward call's (q, k, v, alpha, eta, eps, window, S0, k_prev, rule with the
 * flag); its outputs o, S_out, k_last and chunk are ignored. `grads` (every array fp32, dense,
 * device memory; 4-byte alignment):
 *   dO (B,H,T,dv) required; dS_T (B,H,dv,dk) or NULL (zero);
 *   dq, dk (B,H,T,dk), dv (B,H,T,dv), dalpha, deta (B,H,T) written;
 *   dS0 (B,H,dv,dk) written when not NULL; dk_prev (B,H,dk) written when not NULL and
 *   args->k_prev is given.
 * Workspace: falcon_bwd_workspace_size(args) bytes, 16-byte aligned (the states at the
 * start of every segment of about sqrt(T) steps and one segment of recomputed states,
 * fp32, per slice of 8 value rows of a head). fp32 state and arithmetic; one CTA of 128
 * threads per slice of 8 value rows of a (b, h): the rows of S evolve independently, and the
 * slices add their parts of dq, dk, dalpha, deta and dk_prev to the outputs with atomic adds
 * (so those sums are taken in no fixed order, and their last bits can differ between runs);
 * dv and dS0 rows are each written by one slice.
 * Supported: Falcon-1, 1A, 3, 3A (with or without FALCON_SAME_STEP); 1 <= dk, dv <= 128;
 * windows of up to 8 pairs. Falcon-2/2A return
 * UNSUPPORTED.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 */
typedef struct {
    const float *dO;
    const float *dS_T;
    float *dq, *dk, *dv;
    float *dalpha, *deta;
    float *dS0;
    float *dk_prev;
} falcon_grads_t;

FALCON_API size_t falcon_bwd_workspace_size(const falcon_args_t *args);
FALCON_API falcon_status_t falcon_bwd_recurrent(const falcon_args_t *args, const falcon_grads_t *grads,
                                                void *workspace, size_t workspace_bytes,
                                                falcon_stream_t stream);

/*
 * falcon_decode_step -- one token of the recurrence for N independent
 * sequences x H heads, in place: the recurrent form applied to a single step,
 * the incremental state update that the ai.info overview of "Fast Weight
 * Attention for Continual Learning" lists for streaming inference (section
 * Why This Matters).
 *
 *   x = k_prev (x = k with FALCON_SAME_STEP); beta = eta / (||x||^2 + eps); Sbar = alpha S
 *   Falcon-1:  S <- Sbar - beta (Sbar x - v) x^T     Falcon-1A: S <- Sbar + beta v x^T
 *   o = S q;   k_prev <- k
 *
 * S (N,H,dv,dk) fp32 and k_prev (N,H,dk) io_dtype are read and written in
 * place; q, k (N,H,dk), v (N,H,dv) io_dtype; alpha, eta (N,H) fp32;
 * o (N,H,dv) io_dtype is written. The buffers of one call must not overlap.
 * Supported: rule Falcon-1 or Falcon-1A (Falcon-3/3A need a window of past
 * pairs and Falcon-2/2A their column energies: both return UNSUPPORTED); dk in
 * {32, 64, 128}; 1 <= dv <= 256.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
FALCON_API falcon_status_t falcon_decode_step(int rule, int io_dtype, int N, int H, int dk, int dv,
                                   float *S, void *k_prev, const void *q, const void *k,
                                   const void *v, const float *alpha, const float *eta,
                                   float eps, void *o, falcon_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Operators around the memory: the short causal convolution that its q, k and v pass through,
 * the norm of queries and keys with the position rotation, and the selective scan, a recurrence
 * with a decay of its own for every entry of the state.
 *
 * Conventions of these entry points, besides the ones above:
 *  - Sequence tensors are views: element (b, h, t, i) of a tensor is p[b*sb + h*sh + t*st + i],
 *    strides in elements, the innermost axis contiguous. A slice of a fused projection
 *    (token-major rows) goes in as it lies, and an output can be written head-major for
 *    falcon_fwd_chunk. Strides are >= 0 (0 repeats an input along that axis; the elements of
 *    an output or gradient must not overlap). Pointers of views need the alignment of their
 *    element only; when pointers and strides are 16-byte multiples, wider accesses are used.
 *  - Outputs and gradients must not overlap inputs or each other, except where an entry point
 *    says so. A sequence, state or gradient that starts where another one of the call does is refused
 *    (INVALID_ARG); other overlaps are not looked for.
 *  - Parameters (weights, biases, A, D, frequencies) and all gradients are fp32, whatever
 *    io_dtype is; gradients are views too where the tensor they belong to is one.
 *  - `lengths`: NULL, or B int32 on the device. Sequence b then has lengths[b] tokens (clamped to
 *    [0, T]); what lies at t >= lengths[b] is not read, rows of forward outputs there are left as
 *    they were, rows of gradients there are written 0, and final states are those after the last
 *    token of the sequence.
 *  - Sizes: T <= 2^30; B H and H d below 2^31 (also H dk and H dv); B H T d <= 2^50. Calls that would take more than
 *    2^31 - 1 blocks are UNSUPPORTED, and write nothing.
 *  - fp32 arithmetic takes subnormal values for 0, exponentials and reciprocals are good to 2^-21.
 *  - Sums over tokens are taken in a fixed order: repeated calls give the same bits.
 *  - A workspace is used only while the call's kernels run on `stream`; calls that can overlap on the GPU (other
 *    streams, graphs replayed side by side) need workspaces of their own. The first call of the library on a device
 *    looks up its properties: make it before any stream capture.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
    void *p;              /* device memory, or NULL where the tensor is optional */
    long long sb, sh, st; /* strides of batch, head and token, in elements        */
} falcon_view_t;

typedef enum { FALCON_ACT_NONE = 0, FALCON_ACT_SILU = 1 } falcon_act_t;

/*
 * falcon_conv_fwd -- causal depthwise convolution over the last K tokens:
 *   p_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = act(p_t)
 * for every channel of every head. x_{-1} .. x_{-(K-1)} come from `state` (the last K-1 inputs
 * before this segment, oldest first) or are 0. `state_out` gets the last K-1 inputs of the
 * extended sequence; it may be the same memory as `state`.
 * Supported: 1 <= K <= 8; any d >= 1; fp32 or bf16. Sums in fp32, one rounding at the end.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
typedef struct {
    int io_dtype;         /* falcon_dtype_t of x, y, state and state_out            */
    int B, H, T, d;       /* batch, heads, tokens (T >= 0), channels of a head       */
    int K;                /* taps                                                    */
    int act;              /* falcon_act_t                                            */
    falcon_view_t x;      /* (B,H,T,d)                                               */
    falcon_view_t y;      /* (B,H,T,d) output                                        */
    const float *w;       /* (H,d,K); w[..., K-1] multiplies the current token       */
    const float *bias;    /* (H,d) or NULL                                           */
    const int *lengths;   /* (B) or NULL                                             */
    const void *state;    /* (B,H,K-1,d) or NULL for zeros                           */
    void *state_out;      /* (B,H,K-1,d) or NULL                                     */
} falcon_conv_args_t;

FALCON_API falcon_status_t falcon_conv_fwd(const falcon_conv_args_t *args, falcon_stream_t stream);

/*
 * falcon_conv_step -- one token for B sequences: falcon_conv_fwd with T = 1, as one small kernel.
 * `state` and `state_out` are both required for K > 1 (the same memory updates the cache in place);
 * `lengths` must be NULL. Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
FALCON_API falcon_status_t falcon_conv_step(const falcon_conv_args_t *args, falcon_stream_t stream);

/*
 * falcon_conv_bwd -- gradients of falcon_conv_fwd. With dp_t = dy_t act'(p_t):
 *   dx_t = sum_j w_j dp_{t+K-1-j};  dw_j = sum_{b,t} dp_t x_{t-K+1+j};  dbias = sum_{b,t} dp_t;
 *   dstate is dx at the cached tokens; dstate_out adds to the tokens that state_out copied.
 * args->y and args->state_out are ignored. dbias is written when not NULL (args->bias may be
 * NULL), dstate when not NULL (args->state may be NULL).
 * Workspace: falcon_conv_bwd_workspace_size(args) bytes, 16-byte aligned.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 */
typedef struct {
    falcon_view_t dy;         /* (B,H,T,d) fp32                       */
    const float *dstate_out;  /* (B,H,K-1,d) or NULL (zero)           */
    falcon_view_t dx;         /* (B,H,T,d) fp32, written              */
    float *dw;                /* (H,d,K), written                     */
    float *dbias;             /* (H,d) or NULL                        */
    float *dstate;            /* (B,H,K-1,d) or NULL                  */
} falcon_conv_grads_t;

FALCON_API size_t falcon_conv_bwd_workspace_size(const falcon_conv_args_t *args);
FALCON_API falcon_status_t falcon_conv_bwd(const falcon_conv_args_t *args, const falcon_conv_grads_t *grads,
                                           void *workspace, size_t workspace_bytes, falcon_stream_t stream);

/*
 * falcon_scan_fwd -- selective scan: per head a d_v x d_k state whose entry (i, c) decays at a
 * rate of its own, over steps that the input chooses:
 *   dt_t[i]   = softplus(delta_t[i] + delta_bias[i])   (FALCON_SCAN_SOFTPLUS; else delta_t[i] + delta_bias[i])
 *   S_t[i,c]  = exp(dt_t[i] A[i,c]) S_{t-1}[i,c] + dt_t[i] v_t[i] k_t[c]
 *   o_t[i]    = (sum_c S_t[i,c] q_t[c] + D[i] v_t[i]) silu(z_t[i])
 * (the terms of D, delta_bias and z only where those are given). dt A <= 0 is a precondition: the
 * decays lie in [0, 1]; it is not checked per element. An A beyond 3.4e38 / log2(e) in size, infinities among them,
 * counts as that value of its sign: its decay is 0 for every step above 2^-120, and 1 for a step of 0 (as for any
 * other A).
 * The state, the decays and all sums are fp32.
 * Supported: 1 <= dk <= 128; 1 <= dv <= 2^31 - 512; token strides up to 2^28 elements; fp32 or bf16.
 * Workspace: with few channels the sequence is split into segments that run at once, in two
 * launches (each segment from a zero state; then each from the joined states before it).
 * falcon_scan_workspace_size(args) bytes, 16-byte aligned, are needed for that, 0 where it does not
 * pay; with less, or NULL, the sequence is not split. Results differ by rounding only.
 * S_out may be the same memory as S0. Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
#define FALCON_SCAN_SOFTPLUS 1

typedef struct {
    int io_dtype;            /* falcon_dtype_t of q, k, v, delta, z and o            */
    int B, H, T;             /* batch, heads, tokens (T >= 0)                        */
    int dk, dv;              /* columns and rows (channels) of a head's state        */
    int flags;               /* FALCON_SCAN_SOFTPLUS or 0                            */
    falcon_view_t q, k;      /* (B,H,T,dk)                                           */
    falcon_view_t v, delta;  /* (B,H,T,dv)                                           */
    falcon_view_t z;         /* (B,H,T,dv) or p = NULL                               */
    falcon_view_t o;         /* (B,H,T,dv) output                                    */
    const float *A;          /* (H,dv,dk)                                            */
    const float *D;          /* (H,dv) or NULL                                       */
    const float *delta_bias; /* (H,dv) or NULL                                       */
    const int *lengths;      /* (B) or NULL                                          */
    const float *S0;         /* (B,H,dv,dk) initial state, or NULL for zero          */
    float *S_out;            /* (B,H,dv,dk) final state, or NULL                     */
} falcon_scan_args_t;

FALCON_API size_t falcon_scan_workspace_size(const falcon_scan_args_t *args);
FALCON_API falcon_status_t falcon_scan_fwd(const falcon_scan_args_t *args, void *workspace,
                                           size_t workspace_bytes, falcon_stream_t stream);

/*
 * falcon_scan_step -- one token for B sequences: falcon_scan_fwd with T = 1 as one kernel, bound by
 * reading and writing the state. S0 and S_out are both required (the same memory updates the
 * state in place); `lengths` must be NULL. Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
FALCON_API falcon_status_t falcon_scan_step(const falcon_scan_args_t *args, falcon_stream_t stream);

/*
 * falcon_scan_bwd -- gradients of falcon_scan_fwd. With a_t = exp(dt_t A), dy_t = dO_t silu(z_t) and
 * G_t = dy_t q_t^T + a_{t+1} G_{t+1} (G behind the last token: dS_T):
 *   dq_t[c] = sum_i dy_t[i] S_t[i,c];            dk_t[c] = sum_i G_t[i,c] dt_t[i] v_t[i];
 *   dv_t[i] = dt_t[i] sum_c G_t[i,c] k_t[c] + D[i] dy_t[i];
 *   ddt_t[i] = sum_c G_t[i,c] (A[i,c] a_t[i,c] S_{t-1}[i,c] + v_t[i] k_t[c]), times the softplus' slope;
 *   dA = sum_{b,t} G_t dt_t a_t S_{t-1};  dD = sum_{b,t} dy_t v_t;  dS0 = a_1 G_1;
 *   dz_t[i] = dO_t[i] (sum_c S_t q_t + D v_t) silu'(z_t).
 * args->o and args->S_out are ignored. Optional gradients are written when not NULL; dz only with z.
 * q and k shared by heads (stride 0) get a gradient for each head, which the caller adds up.
 * Workspace: falcon_scan_bwd_workspace_size(args) bytes, 16-byte aligned (states and their gradients
 * between segments of a fixed length, and partial sums).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 */
typedef struct {
    falcon_view_t dO;      /* (B,H,T,dv) fp32                      */
    const float *dS_T;     /* (B,H,dv,dk) or NULL (zero)           */
    falcon_view_t dq, dk;  /* (B,H,T,dk) fp32, written             */
    falcon_view_t dv;      /* (B,H,T,dv) fp32, written             */
    falcon_view_t ddelta;  /* (B,H,T,dv) fp32, written             */
    falcon_view_t dz;      /* (B,H,T,dv) fp32, or p = NULL         */
    float *dA;             /* (H,dv,dk), written                   */
    float *dD;             /* (H,dv) or NULL                       */
    float *ddelta_bias;    /* (H,dv) or NULL                       */
    float *dS0;            /* (B,H,dv,dk) or NULL                  */
} falcon_scan_grads_t;

FALCON_API size_t falcon_scan_bwd_workspace_size(const falcon_scan_args_t *args);
FALCON_API falcon_status_t falcon_scan_bwd(const falcon_scan_args_t *args, const falcon_scan_grads_t *grads,
                                           void *workspace, size_t workspace_bytes, falcon_stream_t stream);

/*
 * falcon_qknorm_fwd -- norm of each head's query and key rows, with the rotation by position in
 * the same pass (what falcon_fwd_* expects of q and k is up to the layer; these are the usual ones):
 *   FALCON_NORM_RMS: n = x w / sqrt(mean(x^2) + eps);  FALCON_NORM_L2: n = x w / sqrt(sum(x^2) + eps);
 *   FALCON_NORM_NONE: n = x w   (w only where given; a row whose root is 0 gives 0)
 * then the first `rot` channels of n turn in pairs by the angle positions[b,t] freq[j]:
 *   pair j is (j, j + rot/2) for FALCON_ROT_HALF, (2j, 2j+1) for FALCON_ROT_PAIRS;
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
 * Angles are reduced in fp64, so far positions keep their accuracy; everything else is fp32: a row whose sum of
 * squares is below 2^-126 (entries near 1e-19) counts as one of 0, above 2^128 (near 1e19) as infinite.
 * positions NULL: t. rot = 0: no rotation. Hk (or Hq) = 0 leaves out that tensor. q_out may be the
 * same memory as q with the same strides (likewise k). One token per sequence is T = 1.
 * Supported: 1 <= d <= 256; Hq, Hk <= 65536; rot even, 0 <= rot <= d; fp32 or bf16.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
typedef enum { FALCON_NORM_NONE = 0, FALCON_NORM_RMS = 1, FALCON_NORM_L2 = 2 } falcon_norm_t;
typedef enum { FALCON_ROT_HALF = 0, FALCON_ROT_PAIRS = 1 } falcon_rot_t;

typedef struct {
    int io_dtype;               /* falcon_dtype_t of q, k, q_out and k_out                */
    int B, Hq, Hk, T, d;        /* batch, heads of q and of k, tokens, width              */
    int norm;                   /* falcon_norm_t                                          */
    int rot, rot_layout;        /* rotated channels, falcon_rot_t                         */
    falcon_view_t q, k;         /* (B,Hq,T,d), (B,Hk,T,d)                                 */
    falcon_view_t q_out, k_out; /* outputs of the same shapes                             */
    const float *wq, *wk;       /* (d) or NULL                                            */
    float eps;                  /* >= 0                                                   */
    const float *freq;          /* (rot/2) angle per position, or NULL when rot = 0       */
    const int *positions;       /* (B,T) int32 or NULL                                    */
    const int *lengths;         /* (B) or NULL                                            */
} falcon_qknorm_args_t;

FALCON_API falcon_status_t falcon_qknorm_fwd(const falcon_qknorm_args_t *args, falcon_stream_t stream);

/*
 * falcon_qknorm_bwd -- gradients of falcon_qknorm_fwd: with g the upstream row turned back by its
 * angles and xr = x / root:  dw = sum g xr;  u = g w;  dx = (u - xr mean(u xr)) / root (the sum in place
 * of the mean for FALCON_NORM_L2; dx = u for FALCON_NORM_NONE). args->q_out and k_out are ignored.
 * dq may be the same memory as dq_out with the same strides (likewise dk).
 * Workspace: falcon_qknorm_bwd_workspace_size(args) bytes, 16-byte aligned; none is needed when dwq and dwk are
 * both NULL (which the size, that of the forward arguments, does not know).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 */
typedef struct {
    falcon_view_t dq_out, dk_out; /* (B,Hq,T,d), (B,Hk,T,d) fp32          */
    falcon_view_t dq, dk;         /* the same shapes, fp32, written        */
    float *dwq, *dwk;             /* (d) or NULL                           */
} falcon_qknorm_grads_t;

FALCON_API size_t falcon_qknorm_bwd_workspace_size(const falcon_qknorm_args_t *args);
FALCON_API falcon_status_t falcon_qknorm_bwd(const falcon_qknorm_args_t *args, const falcon_qknorm_grads_t *grads,
                                             void *workspace, size_t workspace_bytes, falcon_stream_t stream);

/* Static, NUL-terminated description of a status code (never NULL). */
FALCON_API const char *falcon_status_string(falcon_status_t status);

/*
 * Synchronises `stream`, then reads and clears the library's device error
 * word (set by a kernel that detected an inconsistent launch, or by a bounded
 * wait that gave up). Returns FALCON_OK, FALCON_ERR_TIMEOUT, FALCON_ERR_CUDA
 * (a CUDA error surfaced while synchronising) or FALCON_ERR_INVALID_ARG
 * (a kernel rejected its launch geometry).
 */
FALCON_API falcon_status_t falcon_check_device_errors(falcon_stream_t stream);

/*
 * falcon_debug_stall_next_call -- test hook for the failure path; not for production use.
 * Arms a one-shot stall for the next falcon_fwd_chunk (or falcon_fwd_chunk_noalloc) call
 * made from this host thread: the TMA producer of every tensor-core kernel of that call
 * stops loading at block `block` (0-based 64-row block of each head or segment), and every
 * bounded device-side wait of the call gives up after `wait_budget_cycles` SM clocks
 * instead of about 2^31. A consumer's wait then runs out: the kernel records
 * FALCON_ERR_TIMEOUT in the device error word, waits for its own loads in flight (no load
 * is left pending, none was started for the stalled block), frees its tensor memory and
 * returns, so the context stays usable; falcon_check_device_errors() reports the timeout,
 * the call's outputs are undefined, and the following call runs normally. Calls that run
 * no tensor-core kernel, or that have fewer blocks than `block`, ignore the stall (it is
 * consumed all the same). The kernels' waits are bounded whether or not the hook is used;
 * the hook only lets a test reach that code without faulting or hanging a GPU (the pages
 * have no counterpart).
 * Errors: INVALID_ARG for block < 0 or a budget outside [10^4, 2^31].
 */
FALCON_API falcon_status_t falcon_debug_stall_next_call(int block, long long wait_budget_cycles);

/* Library version, major * 10000 + minor * 100 + patch. */
FALCON_API int falcon_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FALCON_H_ */
