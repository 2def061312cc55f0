/*
 * moe.h — C ABI of the MI355X (gfx950) sparse Mixture-of-Experts layer forward.
 *
 * The layer (pages cited by title):
 *   - router: s = x W_g (+ b), g = softmax(s), TopK(g), y = sum_{i in TopK} g_i E_i(x)
 *     ("MoE" primer on qiita, section "ゲート / ルーターって何者？", the four router
 *     equations; bias as in "机器学习基础系列——混合专家模型", GatingNetwork);
 *     the selected weights renormalised to sum to 1 as in
 *     "Mixture of Experts（MoE）の理論と実装", MoELayer.route, and
 *     "Sparse Mixture of Experts(MoE) 아키텍처 심층 분석", TopKGating;
 *   - experts: E_i(x) = (silu(x W_gate) * (x W_up)) W_down, silu(z) = z / (1 + e^-z)
 *     ("Mixture of Experts（MoE）の理論と実装", Expert.forward; the Korean page's
 *     SwiGLUExpert);
 *   - load-balancing statistics f_i, p_i and loss = E * sum_i (f_i / k) p_i
 *     ("Mixture of Experts（MoE）の理論と実装", load_balancing_loss; the Korean page's
 *     compute_load_balancing_loss);
 *   - router z-loss z = mean_t (log sum_e exp(s_te))^2 over the router logits s (the
 *     Korean page's router_z_loss);
 *   - noisy top-k gating for training: s + softplus(x W_noise) * eps before the softmax
 *     (the Korean page's TopKGating, training branch), or s + eps (the fixed-scale noise
 *     of "机器学习基础系列——混合专家模型", MoELayer, with eps scaled by the caller);
 *   - expert-choice routing with capacity C = floor(T * cf / E): each expert takes the
 *     C tokens of largest softmax-over-tokens score (the Korean page's
 *     ExpertChoiceGating);
 *   - token choice with an expert capacity C = int((T / E) * cf * k): top-k routing as
 *     above, after which each expert keeps its first C assignments in token order and
 *     drops the rest; a token that lost a slot has its kept weights divided by their
 *     sum ("机器学习基础系列——混合专家模型", expert_capacity_routing).
 *
 * Conventions for every entry point:
 *   - All tensors are row-major and live in device memory (HBM) unless stated; the
 *     caller allocates every buffer, including the workspace. The library never
 *     allocates, frees, synchronises or keeps a pointer after it returns.
 *   - Work is enqueued on `stream` in order; results are valid once the caller
 *     synchronises that stream.
 *   - Activations and weights have the type `shape->dtype` (fp32 or bf16). Router
 *     logits, probabilities, gate weights, the output y and the statistics are fp32.
 *     bf16 products accumulate in fp32.
 *   - Every argument is checked on the host before any HIP call; a failed check
 *     returns a status and enqueues nothing. MOE_ERR_HIP reports a launch failure.
 *   - Token-choice slots list experts by descending probability, lower index first on
 *     ties. Expert-choice lists each expert's tokens in ascending token order; ties at
 *     the capacity boundary go to the lower token index.
 *   - Results are deterministic: the same inputs give bitwise the same outputs.
 *   - Entry points are reentrant; calls on different streams may overlap if their
 *     workspaces differ.
 *
 * Limits: 1 <= E <= 64; token choice 1 <= k <= min(E, 8); d_model and d_ff at most 2^20;
 * 0 <= T and T * max(k, 1) < 2^31; expert choice needs 1 <= C <= T and E * C < 2^31
 * (outside these: MOE_ERR_BAD_SHAPE). Limits of this implementation, not of the method,
 * return MOE_ERR_UNSUPPORTED: E > 64, k > 8, d_model or d_ff not a multiple of 64 (the
 * kernels run whole 64-column tiles), and fp32 layers with more than 64 * (65535 - E)
 * routed rows (T * k, or E * C). x, weights, y and the workspace must be 16-byte aligned.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_NULL_ARG = 1,            /* a required pointer is NULL */
  MOE_ERR_BAD_SHAPE = 2,           /* sizes out of range or inconsistent */
  MOE_ERR_UNSUPPORTED = 3,         /* valid request this library does not provide */
  MOE_ERR_WORKSPACE_TOO_SMALL = 4, /* ws_bytes < moe_workspace_size() */
  MOE_ERR_MISALIGNED = 5,          /* a pointer is not 16-byte aligned */
  MOE_ERR_HIP = 6                  /* a HIP launch failed */
} moe_status;

typedef enum moe_dtype { MOE_FP32 = 0, MOE_BF16 = 1 } moe_dtype;

/* MOE_TOKEN_CHOICE_CAPACITY is token choice (every "token choice" rule below applies)
 * with an expert capacity: see moe_capacity and moe_route. */
typedef enum moe_mode {
  MOE_TOKEN_CHOICE = 0,
  MOE_EXPERT_CHOICE = 1,
  MOE_TOKEN_CHOICE_CAPACITY = 2
} moe_mode;

/* Shape of one layer call. */
typedef struct moe_shape {
  int64_t T;             /* tokens (rows of x) */
  int64_t d_model;       /* width of x and y */
  int64_t d_ff;          /* hidden width of each expert */
  int32_t E;             /* experts */
  int32_t k;             /* token choice: experts per token; ignored in expert choice */
  int32_t mode;          /* moe_mode */
  int32_t dtype;         /* moe_dtype of x, W_g, W_gate, W_up, W_down */
  int32_t renormalize;   /* token choice: 1 = selected weights divided by their sum
                            (Mixture of Experts（MoE）の理論と実装, MoELayer.route);
                            0 = raw probabilities (the qiita router equations) */
  double capacity_factor; /* expert choice: C = floor(T * capacity_factor / E);
                             token choice with capacity: C = int((T / E) * capacity_factor
                             * k); both in double, > 0 and finite; ignored in plain token
                             choice */
} moe_shape;

/* Training noise of noisy top-k gating, token choice only (both token-choice modes).
 *   W_noise [d_model, E] dtype, layout of W_g; or NULL for additive noise
 *   eps     [T, E] fp32, the normal draw (one per token and expert); or NULL to have the
 *           router kernel draw it: eps[t, e] = scale * n(t, e) below
 *   seed, offset, scale   the in-kernel draw (ignored when eps is given); a non-finite
 *           scale returns MOE_ERR_BAD_SHAPE
 * The router's logits become s + softplus(x W_noise) * eps (softplus(z) = log(1 + e^z)),
 * or s + eps without W_noise, with s = x W_g (+ b_g): the Korean page's TopKGating
 * (training branch) and 机器学习基础系列——混合专家模型's MoELayer. Everything downstream —
 * softmax, top-k, weights, probs, counts, f, p, loss, z_loss — sees the noisy logits.
 * The in-kernel draw is counter-based, so that n(t, e) depends on (seed, offset, t, e)
 * only, not on the launch:
 *   (r0, r1, r2, r3) = Philox4x32-10 with counter (t, floor(e / 4), offset mod 2^32,
 *                      floor(offset / 2^32)) and key (seed mod 2^32, floor(seed / 2^32))
 *                      (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
 *                      as 1, 2, 3", SC 2011)
 *   u_i = (floor(r_i / 2^8) + 1/2) / 2^24, strictly inside (0, 1)
 *   n(t, 4q + 2h + c) = sqrt(-2 ln u_{2h}) * (c = 0 ? cos : sin)(2 pi u_{2h+1})
 *                      (the Box-Muller transform, Box and Muller 1958)
 * evaluated in fp32 (the uniforms exactly; log, sqrt, cos and sin to about an ulp). A new
 * draw per training step takes a new offset (or seed). */
typedef struct moe_noise {
  const void* W_noise;
  const float* eps;
  uint64_t seed;
  uint64_t offset;
  float scale;
} moe_noise;

/* Human-readable name of a status code. Never NULL; the string is static. */
const char* moe_status_string(int32_t status);

/* Capacity C. Expert choice: floor(T * cf / E) (the Korean page's ExpertChoiceGating,
 * expert_capacity); MOE_ERR_BAD_SHAPE unless 1 <= C <= T. Token choice with capacity:
 * floor((T / E) * cf * k) evaluated in double in that order ("机器学习基础系列——混合专家
 * 模型", expert_capacity_routing); C = 0 is valid and drops every assignment. Host
 * only. Plain token choice returns MOE_ERR_BAD_SHAPE. */
moe_status moe_capacity(const moe_shape* shape, int64_t* capacity);

/* Bytes of device workspace moe_route / moe_forward / moe_aux_loss need for `shape`.
 * Host only; the same size serves all three entry points. */
moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes);

/* Byte offset, inside the workspace, of an intermediate buffer of moe_forward, for
 * tests and debugging. After a moe_forward call has completed on the stream the
 * buffer holds that call's values until the workspace is used again. Host only.
 *   MOE_WS_OFFSETS [E+1] int32   first row of each expert's group; [E] = R
 *   MOE_WS_POS     [T, k] int32  token choice: row of each (token, slot), -1 when the
 *                                expert capacity dropped the slot
 *   MOE_WS_SRC     [R] int32     token of each row
 *   MOE_WS_XPERM   [R, d_model]  dtype, x rows in expert-contiguous order; only where rows are
 *                                copied: fp32, or T * d_model >= 2^31 (otherwise the gate/up
 *                                GEMM reads the rows of x through MOE_WS_SRC and this returns
 *                                MOE_ERR_UNSUPPORTED)
 *   MOE_WS_H       [R, d_ff]     dtype, silu(x W_gate) * (x W_up) per row
 *   MOE_WS_O       [R, d_model]  fp32, expert output per row (before weighting)
 * Expert choice in bf16 carries h's bf16 rounding residual: the MOE_WS_H region then holds
 * 2R rows (h, then the residual), and MOE_WS_O row r is the down projection of row r plus
 * that of row R + r.
 * R = T*k (token choice) or E*C (expert choice). With an expert capacity only rows
 * [0, offsets[E]) hold kept slots, offsets[E] = sum_e min(counts_e, C). MOE_WS_POS is
 * MOE_ERR_UNSUPPORTED in expert choice. */
enum {
  MOE_WS_OFFSETS = 0,
  MOE_WS_POS = 1,
  MOE_WS_SRC = 2,
  MOE_WS_XPERM = 3,
  MOE_WS_H = 4,
  MOE_WS_O = 5
};
moe_status moe_workspace_offset(const moe_shape* shape, int32_t which, size_t* offset);

/* Router (the qiita router equations; Mixture of Experts（MoE）の理論と実装,
 * MoELayer.route; the Korean page's TopKGating and ExpertChoiceGating).
 *   x      [T, d_model]   dtype
 *   W_g    [d_model, E]   dtype (the x @ W layout of MoELayer.__init__)
 *   b_g    [E] fp32 router bias added to the logits, or NULL for none
 *   noise  training noise (moe_noise), or NULL for none; MOE_ERR_UNSUPPORTED in expert
 *          choice
 * Token choice outputs:
 *   idx    [T, k] int32   selected experts, descending probability
 *   w      [T, k] fp32    gate weights of the selected experts
 * Expert choice outputs (C = moe_capacity):
 *   idx    [E, C] int32   tokens chosen by each expert, ascending token index
 *   w      [E, C] fp32    their scores (column-softmax values)
 * Optional outputs (NULL to skip):
 *   probs  [T, E] fp32    softmax probabilities (expert choice: over tokens, per column)
 *   counts [E] int32      assignments per expert (expert choice: C each)
 *   z_loss [1] fp32       router z-loss: mean over tokens of (log sum_e exp(s_te))^2, s the
 *                         logits with the bias (every mode; 0 when T = 0). Computed in the
 *                         router's pass over x: one fp32 log-partition per token, fixed-order
 *                         fp32 sums per 64 tokens, then an fp64 sum over those.
 * Token choice with capacity: idx and counts are those of plain token choice (counts
 * before any drop); w holds the weights after the capacity: 0 for a dropped slot, and
 * for a token that lost a slot its kept weights divided by their sum when renormalize
 * = 1 (a token that lost every slot gets zeros), unchanged when renormalize = 0. An
 * expert keeps the assignments of lowest token index; a token's slots go to distinct
 * experts, so the order of slots within a token decides nothing.
 * idx and w are required when T > 0 (with T = 0 there is nothing to write). */
moe_status moe_route(const moe_shape* shape, const void* x, const void* W_g, const float* b_g,
                     const moe_noise* noise, int32_t* idx, float* w, float* probs,
                     int32_t* counts, float* z_loss, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/* Whole layer forward ("Mixture of Experts（MoE）の理論と実装", MoELayer.forward: route,
 * run each expert on its tokens, add the weighted expert outputs; the Korean page's
 * MoELayerWithAuxLoss, which also returns the load-balancing loss): router, dispatch
 * (histogram, prefix sum, stable permutation of token rows into expert-contiguous order),
 * grouped SwiGLU gate/up GEMM, grouped down GEMM, weighted combine, and (token choice) the
 * load-balancing statistics.
 *   x, W_g, b_g, noise   as in moe_route
 *   W_gate, W_up  [E, d_model, d_ff] dtype, expert e's matrix at offset e*d_model*d_ff
 *   W_down        [E, d_ff, d_model] dtype
 *   y             [T, d_model] fp32   y_t = sum over the token's experts of
 *                 weight * E_e(x_t); in expert choice a token no expert takes gets 0
 * Optional outputs (NULL to skip): idx, w, probs, counts, z_loss as in moe_route, and,
 * token choice only (with capacity: computed from the assignments before any drop):
 *   f     [E] fp32   counts / T (sums to k)
 *   p     [E] fp32   mean over tokens of probs
 *   loss  [1] fp32   E * sum_e (f_e / k) * p_e (1 under uniform routing)
 * Passing f, p or loss in expert-choice mode returns MOE_ERR_UNSUPPORTED: the pages
 * define these statistics for token choice only.
 * Precision (bf16): the hidden activation h = silu(x W_gate) * (x W_up) is formed in fp32
 * and rounded to bf16 for the down projection. In expert choice the bf16 rounding
 * residual of h is carried as a second bf16 term (h ~ h_hi + h_lo): expert-choice scores
 * span a wide range across tokens, and a single rounding of h would cost about 2.5% of
 * the output RMS on the 16-expert workload; the pair doubles the down projection's
 * multiply work (each tile takes 128 tokens' rows and their residual rows, and sums the
 * two products before storing o). */
moe_status moe_forward(const moe_shape* shape, const void* x, const void* W_g, const float* b_g,
                       const moe_noise* noise, const void* W_gate, const void* W_up,
                       const void* W_down, float* y,
                       int32_t* idx, float* w, float* probs, int32_t* counts, float* f, float* p,
                       float* loss, float* z_loss, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): moe_forward with the same arguments
 * and results, minus the workspace. The workspace is a file-scope device array of
 * MOE_NOALLOC_SCRATCH_BYTES (256 MiB) inside the library, one per GPU, held until the
 * process ends; its address is looked up (hipGetSymbolAddress) on the first call on each
 * device. The call allocates nothing (no hipMalloc, no library allocation).
 *   - Shapes whose moe_workspace_size exceeds MOE_NOALLOC_SCRATCH_BYTES return
 *     MOE_ERR_WORKSPACE_TOO_SMALL before any HIP call (every other check is moe_forward's).
 *   - Every call on one GPU shares that GPU's array, which keeps the last call's
 *     intermediates: calls that overlap on one GPU (different streams, or threads) race and
 *     must be ordered by the caller. Nothing in the array needs to start at zero.
 *   - MOE_ERR_HIP also reports a failed lookup of the array's address. */
#define MOE_NOALLOC_SCRATCH_BYTES (256u << 20)
moe_status moe_forward_noalloc(const moe_shape* shape, const void* x, const void* W_g,
                               const float* b_g, const moe_noise* noise, const void* W_gate,
                               const void* W_up, const void* W_down, float* y, int32_t* idx,
                               float* w, float* probs, int32_t* counts, float* f, float* p,
                               float* loss, float* z_loss, hipStream_t stream);

/* Load-balancing statistics from router outputs (Mixture of Experts（MoE）の理論と実装,
 * load_balancing_loss; the Korean page's compute_load_balancing_loss), token choice:
 *   probs [T, E] fp32, idx [T, k] int32 (values in [0, E)) ->
 *   f [E] = counts / T, p [E] = mean_t probs, loss [1] = E * sum (f / k) p,
 *   counts [E] int32 (optional, NULL to skip).
 * Expert-choice shapes return MOE_ERR_UNSUPPORTED. With T = 0, f, p, loss and counts
 * are zero. */
moe_status moe_aux_loss(const moe_shape* shape, const float* probs, const int32_t* idx, float* f,
                        float* p, float* loss, int32_t* counts, void* ws, size_t ws_bytes,
                        hipStream_t stream);

/* Stage timing. While enabled, every moe_route / moe_forward / moe_aux_loss call
 * records a hipEvent pair around each stage's kernel launch on the caller's stream.
 * moe_profile_read waits for the recorded events, returns per-stage totals
 * (milliseconds, and the number of timed launches) for stages 0..n-1 and clears them.
 * Not thread-safe: one profiling caller per process. */
enum {
  MOE_STAGE_ROUTER = 0,
  MOE_STAGE_SCAN = 1,
  MOE_STAGE_PERMUTE = 2,
  MOE_STAGE_GEMM_GATE_UP = 3,
  MOE_STAGE_GEMM_DOWN = 4,
  MOE_STAGE_COMBINE = 5,
  MOE_STAGE_AUX = 6,
  MOE_STAGE_EC_SELECT = 7,
  MOE_NUM_STAGES = 8
};
moe_status moe_profile_enable(int32_t on);
moe_status moe_profile_read(double* total_ms, int64_t* launches, int32_t n);
const char* moe_stage_name(int32_t stage);

/* ---- Training: the products, gradients and norms around the forward ------------------
 * The entry points below follow the conventions above (device memory, the caller's buffers
 * and stream, host checks before any HIP call, deterministic results) with these limits:
 * 1 <= E <= 64, row counts below 2^31. Index values read on the device (offsets, gathers,
 * idx, pos) that lie outside their range never move an access out of a buffer: each
 * function says what such a value is taken for. No output may overlap an input or another
 * output unless it says so. They record no stage timing. */

/* Products of rows grouped by expert: group e is rows [offsets[e], offsets[e+1]).
 *   MOE_MATMUL_NN  out[r] = a[r] b_e      a [R, K], b [E, K, N] -> out [R, N]
 *   MOE_MATMUL_NT  out[r] = a[r] b_e^T    a [R, K], b [E, N, K] -> out [R, N]
 *   MOE_MATMUL_TN  out_e = sum over the group's rows r of a[r]^T b[r]
 *                                         a [R, K], b [R, N]    -> out [E, K, N]
 * With a forward product y = x W (NN), NT with W is the gradient of x and TN of W. */
typedef enum moe_matmul_form {
  MOE_MATMUL_NN = 0,
  MOE_MATMUL_NT = 1,
  MOE_MATMUL_TN = 2
} moe_matmul_form;

typedef struct moe_matmul_shape {
  int64_t R;          /* rows of the grouped problem (at most 2^31 - 2^16); groups end at or
                         before R */
  int64_t rows_a;     /* rows of a: R without gather_a */
  int64_t rows_b;     /* TN: rows of b, R without gather_b; ignored otherwise */
  int64_t K;          /* width of a */
  int64_t N;          /* width of out */
  int32_t E;          /* groups */
  int32_t form;       /* moe_matmul_form */
  int32_t dtype;      /* moe_dtype of a and b */
  int32_t out_dtype;  /* moe_dtype of out: fp32, or bf16 where dtype is bf16 */
  int32_t accumulate; /* 1: the product is added to out's values (fp32 out only); 0: stored */
} moe_matmul_shape;

/*   offsets   [E+1] int32 on the device, ascending (offsets of moe_forward's workspace,
 *             MOE_WS_OFFSETS, as they are; a slice of them, with those experts' matrices, is a
 *             table of their groups alone). A bound is taken for the largest of itself, the
 *             bounds before it and 0, and at most R.
 *   gather_a  [R] int32 or NULL: row r of the problem is row gather_a[r] of a (the same row
 *             any number of times); values are clamped into [0, rows_a)
 *   gather_b  TN only: the same for b
 * Sums are fp32 (bf16 products are exact in it); bf16 outputs are rounded once. NN and NT
 * leave the rows of out in no group, before offsets[0] and at and past offsets[E], as they
 * are; a TN group without rows gives zeros (accumulate: leaves its matrix as it is). K and N
 * at most 2^20 and multiples of 8 (bf16) or 4 (fp32): rows are read in 16-byte pieces
 * (otherwise MOE_ERR_UNSUPPORTED). a, b and out must be 16-byte aligned, the workspace too.
 * gather_b in NN or NT, a bf16 out of fp32 inputs and accumulate into a bf16 out return
 * MOE_ERR_UNSUPPORTED. */
moe_status moe_grouped_matmul(const moe_matmul_shape* shape, const void* a, const void* b,
                              const int32_t* offsets, const int32_t* gather_a,
                              const int32_t* gather_b, void* out, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* Bytes of workspace moe_grouped_matmul needs for `shape`: partial sums where few output tiles
 * share a long sum, or a TN group may have most of the rows; some 64 MiB at most. 0 (and a NULL
 * workspace) elsewhere. Host only. */
moe_status moe_grouped_matmul_workspace_size(const moe_matmul_shape* shape, size_t* bytes);

/* Gradient of the experts' activation h = silu(g) * u and of the row's gate weight, for
 * y = sum over rows of w_r (h_r W_down): with dh = dy W_down^T (unweighted) and
 * s = 1 / (1 + e^-g), element by element,
 *   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  hw = w g s u,  dw_r = sum_f dh g s u
 * (hw^T dy is then the gradient of W_down). All rows' values are computed in fp32.
 *   g, u, dh     [R, f] dtype      dg, du, hw  [R, f] dtype (each may be the input of its
 *                                  place: dg = g, du = u, hw = dh), NULL to skip
 *   w            the gate weights, NULL for 1: [R] by row when pos is NULL; otherwise by
 *                slot, [T, k]: row r belongs to token src[r] and to the slot j of that token
 *                with pos[src[r], j] = r (MOE_WS_SRC, MOE_WS_POS), and a row that no slot of
 *                its token names has weight 0
 *   dw           [R] fp32 by row, NULL to skip
 *   offsets      NULL, or the [E+1] bounds, taken as in moe_grouped_matmul: rows in no group,
 *                before offsets[0] and at and past offsets[E], are neither read nor written
 * f at most 2^20 and a multiple of 8 (bf16) or 4 (fp32), else MOE_ERR_UNSUPPORTED. Tensors
 * of R rows must be 16-byte aligned. */
typedef struct moe_swiglu_shape {
  int64_t R;      /* rows */
  int64_t f;      /* width */
  int64_t T;      /* tokens (rows of pos), with pos */
  int32_t k;      /* slots per token, with pos: 1 .. 8 */
  int32_t E;      /* groups, with offsets */
  int32_t dtype;  /* moe_dtype */
} moe_swiglu_shape;
moe_status moe_swiglu_backward(const moe_swiglu_shape* shape, const void* g, const void* u,
                               const void* dh, const float* w, const int32_t* src,
                               const int32_t* pos, const int32_t* offsets, void* dg, void* du,
                               void* hw, float* dw, hipStream_t stream);

/* Gradient of the token-choice router (both token-choice modes, without training noise):
 * of its weights w, the load-balancing loss and the z-loss, with respect to x, W_g and b_g.
 * Per token, over the slots the forward kept (w != 0; the others' dw is not looked at),
 * S = sum of their probabilities:
 *   dp_e  = (dw_j - sum_i dw_i w_i) / S for e = idx_j (renormalize = 1), dw_j (= 0),
 *           plus loss_grad * E f_e / (k T) for every e
 *   ds_e  = p_e (dp_e - sum_c p_c dp_c) + z_loss_grad * 2 lse p_e / T
 *   db_g = sum_t ds,  dW_g = x^T ds,  dx = ds W_g^T (+ sum_j rows[pos[t, j]])
 * lse, the token's log sum_e exp(s_e), is s - log p at its most probable expert, from one
 * dot product in fp32 (z_loss_grad != 0 only); the counts behind f carry no gradient. */
typedef struct moe_route_upstream {
  const float* dw;        /* gradient of w, NULL for none: [T, k], or [R] by row (dw_by_row) */
  int32_t dw_by_row;      /* 1: dw of slot (t, j) is dw[pos[t, j]] */
  float loss_grad;        /* gradient of the load-balancing loss */
  float z_loss_grad;      /* gradient of the z-loss */
  const float* f;         /* [E] the forward's f; required when loss_grad != 0 */
  const void* rows;       /* [R, d_model] dtype, NULL for none: gradients of the routed rows */
  const int32_t* pos;     /* [T, k] row of each slot (MOE_WS_POS); values outside [0, R) add
                             nothing. Required with rows or dw_by_row */
  int64_t R;              /* rows of rows / by-row dw */
} moe_route_upstream;

/* Bytes of workspace moe_route_backward needs. Host only. */
moe_status moe_route_backward_workspace_size(const moe_shape* shape, size_t* bytes);

/*   x, W_g, b_g     as in moe_route
 *   probs, idx, w   moe_route's or moe_forward's outputs for them (an idx outside [0, E) is
 *                   taken for the nearest end)
 *   dx      [T, d_model] dtype, dW_g [d_model, E] dtype, db_g [E] fp32: NULL to skip
 *   dlogits [T, E] fp32, the ds above: always written
 * d_ff is ignored. Expert-choice shapes return MOE_ERR_UNSUPPORTED. x, W_g, rows, dx, dW_g
 * and the workspace must be 16-byte aligned. With T = 0 dW_g and db_g are zero. */
moe_status moe_route_backward(const moe_shape* shape, const void* x, const void* W_g,
                              const float* b_g, const float* probs, const int32_t* idx,
                              const float* w, const moe_route_upstream* up, void* dx, void* dW_g,
                              float* db_g, float* dlogits, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* RMS norms after a block and before the next one, with the block's gate and the residual
 * scale, in one pass. With rms(v) = sqrt(mean v^2 + eps) over the row:
 *   after   (y given)      out = residual_scale * x + gate * (y / rms(y) * gamma_post)
 *                          (out = x without y)
 *   before  (gamma given)  u = out / rms(out) * gamma
 * One or both parts run. `out` is rounded to dtype and `u` is computed from the rounded
 * values, so that both parts in one call give the bits of two calls. */
enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 };
typedef struct moe_norm_shape {
  int64_t T;             /* rows */
  int64_t d;             /* width: at most 16384 (a row is held in registers) and a multiple of 8 */
  int32_t dtype;         /* moe_dtype of x, out, u and their gradients, and of dy */
  int32_t gate;          /* gate: none (1), [d] per channel, or [T] per token */
  float eps;             /* > 0, finite */
  float residual_scale;  /* finite; only with y */
} moe_norm_shape;

/*   x [T, d] dtype, y [T, d] fp32 (moe_forward's output) or NULL, gamma_post [d] fp32 and
 *   gate fp32 (with y), gamma [d] fp32 or NULL
 *   out [T, d] dtype (with y; may be x), u [T, d] dtype (with gamma)
 *   rstd_post, rstd [T] fp32 = 1 / rms(y), 1 / rms(out): for the gradient, NULL to skip
 * Neither y nor gamma: MOE_ERR_NULL_ARG. All tensors but the [T] ones 16-byte aligned. */
moe_status moe_block_norm(const moe_norm_shape* shape, const void* x, const float* y,
                          const float* gamma_post, const float* gate, const float* gamma,
                          void* out, void* u, float* rstd_post, float* rstd, hipStream_t stream);

/* Bytes of workspace moe_block_norm_backward needs. Host only. */
moe_status moe_block_norm_backward_workspace_size(const moe_norm_shape* shape, size_t* bytes);

/* Its gradient. d_out, d_u [T, d] dtype: gradients of out and u; either may be NULL (the part
 * before runs with d_u, the part after with y).
 *   D  = d_out + r (dz - z mean(dz z)),  dz = d_u gamma, z = out r, r = rstd
 *   dx = residual_scale D (with y, else D),  dgamma = sum_t d_u z
 *   n = y q, q = rstd_post, dn = gate D gamma_post:  dy = q (dn - n mean(dn n)),
 *   dgamma_post = sum_t gate D n,  dgate = sum of D n gamma_post over t (per channel) or
 *   over the row (per token)
 *   out, rstd, gamma: with d_u (out: the forward's rounded sum; x where y was NULL)
 *   y, rstd_post, gamma_post, gate: with y
 *   dx, dy [T, d] dtype; dgamma, dgamma_post [d], dgate [d] or [T] fp32: NULL to skip. dx may
 *   be d_out or d_u. */
moe_status moe_block_norm_backward(const moe_norm_shape* shape, const void* d_out,
                                   const void* d_u, const void* out, const float* rstd,
                                   const float* gamma, const float* y, const float* rstd_post,
                                   const float* gamma_post, const float* gate, void* dx, void* dy,
                                   float* dgamma, float* dgamma_post, float* dgate, void* ws,
                                   size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
