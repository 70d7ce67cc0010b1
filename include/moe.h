/*
 * moe.h: C ABI of a single Mixture-of-Experts layer on one MI355X (gfx950) GPU.
 *
 * The layer computes y = sum_k g_k E_k(x): an fp32 router picks k experts per
 * token and renormalised gates g; token copies are dispatched into an
 * expert-contiguous ring buffer; every expert applies a SwiGLU FFN
 * E(x) = W_down (silu(W_gate x) * (W_up x)); the results are combined with the
 * gates in a fixed order.  Sources of each step:
 *
 *   routing of tokens to experts ........ dzen.guru page, section "Что именно тормозило
 *                                          обучение MoE-моделей?"
 *   fixed ring buffer, no dropped tokens,
 *   reverse traversal in the backward ... dzen.guru page, ring-buffer paragraph of
 *                                          "Три решения, которые дали результат"
 *   one deterministic result; BF16 and
 *   MXFP8 ................................ dzen.guru page, megakernel paragraph of the same
 *                                          section; @cursor_ai tweet on the khabar-ai page
 *   no CPU in the loop .................. @rohanpaul_ai tweet on the khabar-ai page
 *   output-parallel two-kernel decode ... toolnavs.com warp-decode page, sections "Cursor a
 *                                          réécrit le décodage de MoE" and "1.84x plus de
 *                                          vitesse…"
 * The pages give no formulas; the router (softmax over all experts, top-k,
 * renormalise), the SwiGLU expert and the MXFP8 encoding (E4M3 elements, one
 * E8M0 scale per 32 elements along the reduction dimension, RNE) are those of
 * the layer's workload definition.
 *
 * Conventions for every call
 *   - Every tensor pointer is a DEVICE pointer; `shape` is a HOST pointer.
 *   - Row-major, nn.Linear layout: W_gate, W_up [E, f, d]; W_down [E, d, f];
 *     W_r [E, d] fp32; b_r [E] fp32 (may be NULL).
 *   - "act" tensors are fp32 when shape->dtype == MOE_F32, otherwise bf16
 *     (raw 16-bit patterns).  With MOE_MXFP8 the router and the tokens x stay
 *     bf16; ring_x, H and the expert weights are E4M3 codes (uint8) with one
 *     E8M0 scale byte per 32 elements along the reduction dimension.  Every MX
 *     scale tensor of a matrix [rows, cols] is laid out [cols/128][rows][4]: for each
 *     group of 128 columns one 32-bit word per row holding that row's 4 block scales
 *     in column order (cols % 128 == 0), so that the scales a GEMM stage needs for
 *     consecutive rows are consecutive words.
 *   - With MOE_FP8 the router and the tokens x stay bf16 too; ring_x, H and the expert
 *     weights are E4M3 codes with fp32 scales, value = code * scale: a row matrix
 *     [rows, cols] (tokens, H) has one scale per row and 128 columns, laid out
 *     [cols/128][rows]; a weight matrix [rows, cols] one per 128 x 128 block, laid out
 *     [rows/128][cols/128] (an expert stack: [E][rows/128][cols/128]).  d and f are
 *     multiples of 128.  Scale arguments typed uint8_t* take the address of these floats.
 *     moe_route, moe_dispatch, moe_expert_ffn and moe_combine take MOE_FP8; so do the
 *     calls below that say so.
 *   - The caller owns every buffer.  The library allocates nothing, keeps no
 *     pointer after return, and only enqueues work on `stream`: there is no
 *     host synchronisation and no device-to-host copy inside any call.
 *   - Outputs are fully overwritten; read-only inputs are never written.  With
 *     tokens = 0 the per-expert outputs are zeros (expert_count, expert_offset,
 *     every weight gradient) and per-token outputs are empty; per-token arrays
 *     (x, dy, y, dx, topk_idx, topk_gate, copy_slot) may then be NULL.
 *   - Results are bitwise reproducible run to run (fixed reduction orders,
 *     no floating-point atomics).
 *   - Errors: arguments are validated on the host from `shape` before any
 *     launch.  A launch failure returns MOE_ERR_HIP.  No exception crosses
 *     the ABI.  Calls that share a workspace must not overlap in time.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum moe_status {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,       /* a required pointer is NULL */
  MOE_ERR_SHAPE = 2,      /* non-positive size, k > E, a length outside the kernels'
                             domain (see each call), a ring array of 4 GiB or more, ... */
  MOE_ERR_CAPACITY = 3,   /* ring capacity below tokens * top_k: tokens would be dropped */
  MOE_ERR_WORKSPACE = 4,  /* workspace smaller than moe_workspace_bytes() */
  MOE_ERR_HIP = 5,        /* a HIP launch or runtime call failed */
  MOE_ERR_DTYPE = 6,      /* unknown dtype, or a dtype the call does not support */
  MOE_ERR_SCRATCH = 7,    /* shape needs more than the static scratch of moe_decode_noalloc */
  MOE_ERR_ALIGN = 8       /* a tensor is not aligned to 16 bytes (calls that say so) */
};

enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1, MOE_MXFP8 = 2, MOE_FP8 = 3 };

enum moe_op {
  MOE_OP_ROUTE = 0, MOE_OP_DISPATCH = 1, MOE_OP_EXPERT_FFN = 2,
  MOE_OP_COMBINE = 3, MOE_OP_DECODE = 4, MOE_OP_BACKWARD = 5, MOE_OP_FORWARD = 6,
  MOE_OP_NORM_BACKWARD = 7, MOE_OP_ROUTE_BACKWARD = 8
};

/* Shape of one layer call (host struct). */
typedef struct moe_shape {
  int64_t tokens;      /* T: tokens of this call (decode: batch B) */
  int64_t capacity;    /* C: ring rows; must be >= tokens * top_k */
  int32_t hidden;      /* d */
  int32_t experts;     /* E */
  int32_t top_k;       /* k, 1 <= k <= E */
  int32_t ffn;         /* f: expert intermediate size */
  int32_t shared_ffn;  /* fs: always-on shared expert width (decode only), 0 = none */
  int32_t dtype;       /* enum moe_dtype */
} moe_shape;

/*
 * moe_route: the router (dzen.guru, "Что именно тормозило…": each layer routes
 * tokens to experts).  In fp32, with x widened exactly from bf16:
 *   l[t,e] = sum_i x[t,i] W_r[e,i] (+ b_r[e]);  p = softmax_e(l);
 *   S_t = the k largest l (ties to the lower id);  g[t,j] = p[S_tj] / sum_S p.
 * In:  x [T,d] act (bf16 for MOE_MXFP8), w_router [E,d] f32, b_router [E] f32 or NULL.
 * Out: topk_idx [T,k] int32, ascending expert id per token; topk_gate [T,k] f32;
 *      expert_count [E] int32 = copies routed to each expert.
 * workspace: moe_workspace_bytes(shape, MOE_OP_ROUTE) bytes, a size that serves moe_route_scored too;
 * moe_route refuses one only where its own planes of router logits do not fit.
 */
int moe_route(const moe_shape* shape, const void* x, const float* w_router,
              const float* b_router, int32_t* topk_idx, float* topk_gate,
              int32_t* expert_count, void* workspace, size_t workspace_bytes,
              hipStream_t stream);

/*
 * moe_dispatch: deterministic counting sort of the T*k token copies into the
 * fixed ring buffer (dzen.guru, ring-buffer paragraph: fixed size, nothing
 * dropped, no size computed on the CPU).  Copy c = t*k + j goes to
 *   slot = (ring_head + rank(c)) mod C,
 * where rank orders copies by (expert, token): segments are expert-contiguous
 * and hold their tokens in ascending order.
 * In:  x [T,d] act (bf16 for MOE_MXFP8 and MOE_FP8), topk_idx [T,k], ring_head in [0, C).
 * Out: ring_x [C,d] act (MOE_MXFP8, MOE_FP8: E4M3 codes, each row quantised along d)
 *        — only the T*k used slots are written;
 *      ring_x_scale [d/128][C][4] E8M0 bytes (MOE_MXFP8), [d/128][C] f32 (MOE_FP8: codes and
 *      scales of moe_quantize_fp8 with row_block 1), else NULL;
 *      expert_offset [E+1] int32, segment starts relative to the head (offset[E] = T*k);
 *      copy_slot [T,k] int32 absolute slot of each copy;
 *      slot_copy [C] int32 copy id t*k+j held by each used slot (other slots untouched).
 * workspace: moe_workspace_bytes(shape, MOE_OP_DISPATCH) bytes.  MOE_FP8: x and ring_x are aligned to
 * 16 bytes, ring_x_scale to 4 (MOE_ERR_ALIGN); fewer than 2^24 tokens (MOE_ERR_SHAPE).
 */
int moe_dispatch(const moe_shape* shape, const void* x, const int32_t* topk_idx,
                 int64_t ring_head, void* ring_x, uint8_t* ring_x_scale,
                 int32_t* expert_offset, int32_t* copy_slot, int32_t* slot_copy,
                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * moe_expert_ffn: every expert's SwiGLU FFN over its own ring segment, as two
 * grouped GEMMs (the expert-centric scheme the warp-decode page contrasts with;
 * MXFP8 expert kernels per the @rohanpaul_ai tweet on the khabar-ai page):
 *   [A|U] = X_e [W_gate[e]; W_up[e]]^T,  H = silu(A) * U,  Y_e = H W_down[e]^T.
 * H is bf16 (fp32 for MOE_F32; 8-bit along f for MOE_MXFP8 and MOE_FP8) and lives in the workspace.
 * MOE_FP8: a block of 128's sum comes from the 8-bit matrix instruction, to 2^-13 of the largest of every eight products
 * (few rows: the gate and up products have fp32 sums); code = RNE_E4M3(h / scale) as in moe_quantize_fp8.
 * In:  ring_x (+ ring_x_scale), expert_offset, ring_head; w_gate, w_up [E,f,d] and
 *      w_down [E,d,f] act, or E4M3 codes with w_gate_scale/w_up_scale [d/128][E*f][4]
 *      and w_down_scale [f/128][E*d][4] for MOE_MXFP8, as moe_quantize_mx writes them for
 *      the [E*f, d] and [E*d, f] matrices, or one fp32 scale per 128 x 128 for MOE_FP8 (above),
 *      as moe_quantize_fp8 writes them for the same matrices (NULL otherwise).
 * Out: ring_y [C,d] (bf16; fp32 for MOE_F32) at the segment slots;
 *      saved_au [C,2f] bf16 (A then U per slot) when not NULL — the backward's input
 *      (MOE_BF16, MOE_MXFP8 and MOE_FP8: the gate/up fp32 accumulations rounded to bf16; NULL
 *      for MOE_F32).
 * workspace: moe_workspace_bytes(shape, MOE_OP_EXPERT_FFN) bytes.  MOE_FP8: tensors and workspace
 * are aligned to 16 bytes, scales and offsets to 4 (MOE_ERR_ALIGN).
 */
int moe_expert_ffn(const moe_shape* shape, const void* ring_x, const uint8_t* ring_x_scale,
                   const int32_t* expert_offset, int64_t ring_head,
                   const void* w_gate, const void* w_up, const void* w_down,
                   const uint8_t* w_gate_scale, const uint8_t* w_up_scale,
                   const uint8_t* w_down_scale, void* ring_y, void* saved_au,
                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * moe_expert_ffn_timed: moe_expert_ffn for measurement.  When `events` is not
 * NULL, events[0] is recorded on `stream` before GEMM-1, events[1] between GEMM-1
 * and GEMM-2, events[2] after GEMM-2 (caller-created hipEvent_t handles).  No
 * host synchronisation; results identical to moe_expert_ffn.
 */
int moe_expert_ffn_timed(const moe_shape* shape, const void* ring_x, const uint8_t* ring_x_scale,
                         const int32_t* expert_offset, int64_t ring_head,
                         const void* w_gate, const void* w_up, const void* w_down,
                         const uint8_t* w_gate_scale, const uint8_t* w_up_scale,
                         const uint8_t* w_down_scale, void* ring_y, void* saved_au,
                         void* workspace, size_t workspace_bytes, hipEvent_t* events,
                         hipStream_t stream);

/*
 * moe_combine: y[t] = sum_j g[t,j] ring_y[copy_slot[t,j]], j in ascending expert
 * order, fp32 accumulation, one final rounding (deterministic gather; dzen.guru,
 * megakernel paragraph).
 * In: ring_y [C,d], copy_slot [T,k], topk_gate [T,k].  Out: y [T,d] (bf16; f32 for MOE_F32).
 */
int moe_combine(const moe_shape* shape, const void* ring_y, const int32_t* copy_slot,
                const float* topk_gate, void* y, hipStream_t stream);

/*
 * moe_forward: the whole forward (moe_route, moe_dispatch, moe_expert_ffn, moe_combine)
 * in ONE kernel launch, persistent and deterministic (dzen.guru page, megakernel
 * paragraph of "Три решения…": one GPU call moves and computes, with one deterministic
 * result; @cursor_ai tweet on the khabar-ai page: a single, fully deterministic kernel).
 * Same arguments and outputs as the four calls chained (the router's workspace, the
 * dispatch's and the FFN's live inside this call's workspace); every output is bitwise
 * the chained calls' where those run the 128-row GEMM tile (fewer than 256 copies per
 * expert on average), and equal up to fp32 rounding order otherwise.
 * In:  x [T,d] bf16, w_router [E,d] f32, b_router [E] f32 or NULL, w_gate/w_up [E,f,d] and
 *      w_down [E,d,f] bf16, ring_head in [0, C).
 * Out: topk_idx, topk_gate, expert_count (as moe_route); ring_x, expert_offset, copy_slot,
 *      slot_copy (as moe_dispatch); ring_y [C,d] bf16 and saved_au [C,2f] bf16 or NULL
 *      (as moe_expert_ffn); y [T,d] bf16 (as moe_combine).
 * The kernel is launched cooperatively, one workgroup per CU (a multiple of 8), and its
 * phases meet at grid barriers kept in the first 256 bytes of the workspace: those bytes
 * must be zero before the first call on a workspace and are kept consistent by every
 * call (the rest of the workspace needs no initial contents).  A barrier wait gives up
 * after spin_limit polls (0: 4,194,304, far beyond any normal wait) and then sets bit 0
 * of the 32-bit status word at byte offset 8 of the workspace; the results of that call
 * are then undefined, the bit stays set until the caller clears it, and the first 256
 * bytes must be zeroed before the next call.  Calls sharing a workspace must not overlap.
 * workspace: moe_workspace_bytes(shape, MOE_OP_FORWARD) bytes.  MOE_BF16 only.
 */
int moe_forward(const moe_shape* shape, const void* x, const float* w_router,
                const float* b_router, const void* w_gate, const void* w_up, const void* w_down,
                int64_t ring_head, int32_t* topk_idx, float* topk_gate, int32_t* expert_count,
                void* ring_x, int32_t* expert_offset, int32_t* copy_slot, int32_t* slot_copy,
                void* ring_y, void* saved_au, void* y, uint32_t spin_limit, void* workspace,
                size_t workspace_bytes, hipStream_t stream);

/*
 * moe_decode: small-batch decode parallelised over outputs, in two kernels and
 * with no permuted buffer (toolnavs.com warp-decode page, "1.84x plus de vitesse…"),
 * after a router kernel that writes the fp32 logits.  Kernel 1: the routing (rebuilt
 * in every workgroup), then each wavefront streams rows of W_gate/W_up of the shared
 * expert and of the experts the batch selected and
 * writes h = silu(a) * u in fp32, token-major.  Kernel 2: each wavefront owns a
 * group of output rows, streams W_down rows of every selected expert and of the
 * shared expert, and writes y = sum_j g_j (W_down h_j) + W_s_down h_s in bf16.
 * In:  x [B,d] bf16 (B = shape->tokens, 1..8; top_k <= 16), w_router, b_router (or NULL),
 *      w_gate/w_up/w_down bf16, shared ws_gate/ws_up [fs,d], ws_down [d,fs] bf16
 *      or NULL when shape->shared_ffn == 0.
 * Out: y [B,d] bf16, topk_idx [B,k], topk_gate [B,k].
 * workspace: moe_workspace_bytes(shape, MOE_OP_DECODE) bytes (no initial contents needed).
 * MOE_BF16 only; d a multiple of 512 up to 8192, f a multiple of 512 up to 4096,
 * shared_ffn 0 or equal to f (MOE_ERR_SHAPE otherwise).
 */
int moe_decode(const moe_shape* shape, const void* x, const float* w_router,
               const float* b_router, const void* w_gate, const void* w_up,
               const void* w_down, const void* ws_gate, const void* ws_up,
               const void* ws_down, void* y, int32_t* topk_idx, float* topk_gate,
               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * moe_decode_noalloc: moe_decode for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same kernels and results, bitwise, but the workspace is the library's own static
 * device array of 1 MiB (one per GPU, held until the process ends), so the caller passes
 * inputs and outputs only.  Shapes whose decode workspace
 * (moe_workspace_bytes(shape, MOE_OP_DECODE)) exceeds 1 MiB return MOE_ERR_SCRATCH
 * before any launch: B = 8, k = 8, f = fs = 2048, E = 256 needs 0.6 MiB, while
 * B = 8, k = 16, f = 4096 (2.3 MiB) is rejected.
 * No allocation of any kind happens inside the call.  Every call on one GPU shares that
 * GPU's array: calls that overlap in time on one GPU (two streams, or two threads) race
 * and must not be issued.  The array needs no initial contents (every word a call reads
 * it first writes in the same call).
 */
int moe_decode_noalloc(const moe_shape* shape, const void* x, const float* w_router,
                       const float* b_router, const void* w_gate, const void* w_up,
                       const void* w_down, const void* ws_gate, const void* ws_up,
                       const void* ws_down, void* y, int32_t* topk_idx, float* topk_gate,
                       hipStream_t stream);

/*
 * moe_backward: gradients of L = sum_t <dy_t, y_t> with the routing S held
 * fixed; the ring is traversed in reverse (dzen.guru, ring-buffer paragraph):
 * experts E-1 -> 0, and every weight gradient sums its segment's rows from the
 * last slot to the first.  Per copy (t,j) of expert e with gate g:
 *   dh = W_down[e]^T dy_t,  dg = <dh, h>,  da = g dh u s (1 + a (1 - s)),
 *   du = g dh a s  (s = sigmoid(a)),   dx_t += W_gate[e]^T da + W_up[e]^T du,
 *   dW_down[e] += g dy_t h^T,  dW_gate[e] += da x_t^T,  dW_up[e] += du x_t^T;
 *   router: dl_j = g_j (dg_j - sum_i g_i dg_i),  dW_r[e_j] += dl_j x_t,  dx_t += dl_j W_r[e_j].
 * The router part is that of gates renormalised from a softmax, unscaled (moe_route's): gates of
 * another moe_router rule take moe_backward_experts and moe_route_scored_backward.
 * In:  dy [T,d] bf16; x [T,d] bf16; w_router [E,d]; topk_idx, topk_gate; ring_x,
 *      expert_offset, copy_slot, slot_copy, ring_head from moe_dispatch; saved_au from
 *      moe_expert_ffn; w_gate, w_up, w_down bf16.
 * Out: dx [T,d] bf16; dw_gate, dw_up [E,f,d] bf16; dw_down [E,d,f] bf16 (zero for
 *      experts with no rows); dw_router [E,d] f32.
 * workspace: moe_workspace_bytes(shape, MOE_OP_BACKWARD) bytes.  MOE_BF16 only (the MXFP8
 * layer's backward is moe_backward_mx); d and f must be multiples of 128 (MOE_ERR_SHAPE
 * otherwise).
 */
int moe_backward(const moe_shape* shape, const void* dy, const void* x,
                 const float* w_router, const int32_t* topk_idx, const float* topk_gate,
                 const void* ring_x, const int32_t* expert_offset, const int32_t* copy_slot,
                 const int32_t* slot_copy, int64_t ring_head, const void* saved_au,
                 const void* w_gate, const void* w_up, const void* w_down,
                 void* dx, void* dw_gate, void* dw_up, void* dw_down, float* dw_router,
                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Validation of `shape` alone, as every call performs it first (MOE_OK or the status
 * a call would return; includes: every ring array the MFMA GEMMs address, C * d and
 * C * f elements of bf16 or E4M3, must stay below 4 GiB).  Host only, no GPU call. */
int moe_check_shape(const moe_shape* shape);

/*
 * moe_backward_mx: the MXFP8 layer's backward (the MXFP8 backward of the dzen.guru page,
 * "Что показали замеры?").  The gradients of moe_backward, with every backward GEMM's two
 * operands MX-quantised (E4M3, one E8M0 scale per 32) along that GEMM's reduction
 * dimension and fp32 accumulation; the forward's quantisation counts as the identity:
 *   dh = Q_d(W_down)^T Q_d(dy_t)        (W_down quantised along d, i.e. transposed)
 *   dx_t += Q_f(W_gate)^T Q_f(da) + Q_f(W_up)^T Q_f(du)   (weights along f)
 *   dW_down[e] = Q_t(dY_e)^T Q_t(g H_e),  dW_gate[e] = Q_t(dA_e)^T Q_t(X_e),
 *   dW_up[e] = Q_t(dU_e)^T Q_t(X_e)
 * The router part is moe_backward's, for moe_route's gates: a layer in MXFP8 that routes by
 * another moe_router rule has no backward.
 * Q_t: along the token axis, each expert's copies in ring-segment order in blocks of 32
 * aligned to the segment's last slot (the first block partial).  dg, da, du, the router
 * gradient and dx's router term as in moe_backward; saved_au from the MXFP8 forward's
 * moe_expert_ffn.
 * In:  dy, x [T,d] bf16; w_router; topk_idx, topk_gate; expert_offset, copy_slot,
 *      slot_copy, ring_head from moe_dispatch; saved_au [C,2f] bf16;
 *      w_gu_t [E,d,2f] E4M3 = [W_gate^T | W_up^T] of every expert quantised along f, scales
 *      w_gu_t_scale [2f/128][E*d][4]; w_down_t [E,f,d] = W_down^T quantised along d,
 *      scales w_down_t_scale [d/128][E*f][4] (both as moe_quantize_mx_t writes them).
 * Out: dx [T,d] bf16; dw_gate, dw_up [E,f,d] and dw_down [E,d,f] bf16; dw_router [E,d] f32.
 * workspace: moe_workspace_bytes(shape with dtype MOE_MXFP8, MOE_OP_BACKWARD) bytes.
 * MOE_MXFP8 only; d and f multiples of 128, f at most 13568 (the SwiGLU backward keeps
 * three f-wide rows of column maxima in LDS); MOE_ERR_SHAPE otherwise.
 */
int moe_backward_mx(const moe_shape* shape, const void* dy, const void* x,
                    const float* w_router, const int32_t* topk_idx, const float* topk_gate,
                    const int32_t* expert_offset, const int32_t* copy_slot,
                    const int32_t* slot_copy, int64_t ring_head, const void* saved_au,
                    const uint8_t* w_gu_t, const uint8_t* w_gu_t_scale, const uint8_t* w_down_t,
                    const uint8_t* w_down_t_scale, void* dx, void* dw_gate, void* dw_up,
                    void* dw_down, float* dw_router, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* Bytes of workspace `op` needs for `shape` (0 if none).  Host only, no GPU call. */
size_t moe_workspace_bytes(const moe_shape* shape, int op);

/* Static description of a status code. */
const char* moe_status_string(int status);

/*
 * moe_quantize_mx: MX-quantise a bf16 matrix [rows, cols] along cols (cols % 128 == 0):
 * per block of 32, X = floor(log2 amax) - 8 clamped to [-127, 127] (-127 for a zero
 * block), code = RNE_E4M3(clamp(v / 2^X, +-448)), scale = X + 127.
 * Out: codes [rows, cols] uint8, scales [cols/128][rows][4] uint8 (the MX scale
 * layout above).  Used for the weights.
 */
int moe_quantize_mx(const void* src_bf16, int64_t rows, int64_t cols, uint8_t* codes,
                    uint8_t* scales, hipStream_t stream);

/*
 * moe_quantize_mx_t: MX-quantise `batch` bf16 matrices [rows, cols] (src [batch, rows, cols])
 * along their rows and write them transposed: source column c of matrix b becomes row
 * b*cols + c of a code matrix with rows of ld bytes, its values in columns col0 .. col0 +
 * rows - 1; scales in that code matrix's layout [ld/128][batch*cols][4].  The MXFP8
 * backward's weights: W_down [E,d,f] -> (E, d, f, ld = d, col0 = 0); W_gate and W_up [E,f,d]
 * -> (E, f, d, ld = 2f, col0 = 0 and f).  rows % 32 == 0, ld % 128 == 0, col0 % 32 == 0.
 */
int moe_quantize_mx_t(const void* src_bf16, int64_t batch, int64_t rows, int64_t cols,
                      uint8_t* codes, int64_t ld, int64_t col0, uint8_t* scales,
                      hipStream_t stream);

/*
 * moe_quantize_mx_both: both MX layouts of `batch` bf16 matrices in one pass, for an MXFP8
 * training step that re-quantises its weights for the forward and for moe_backward_mx.
 * Writes exactly what moe_quantize_mx(src, batch*rows, cols, codes, scales) and
 * moe_quantize_mx_t(src, batch, rows, cols, codes_t, ld, col0, scales_t) write, bit for
 * bit, reading each bf16 value once.  rows, cols, ld and col0 multiples of 128, col0 +
 * rows <= ld (MOE_ERR_SHAPE otherwise); NULL pointers: MOE_ERR_NULL.  Both code matrices
 * and scale arrays are the caller's, as for the two calls it replaces.
 */
int moe_quantize_mx_both(const void* src_bf16, int64_t batch, int64_t rows, int64_t cols,
                         uint8_t* codes, uint8_t* scales, uint8_t* codes_t, int64_t ld,
                         int64_t col0, uint8_t* scales_t, hipStream_t stream);

/* ------------------------------------------------------------------ residual RMS norm
 * moe_add_rmsnorm: the norm in front of the layer, per token row:
 *   h = round(x + residual) (x itself when residual is NULL), rounded to the act type;
 *   rstd = 1 / sqrt(mean_i h_i^2 + eps);   y = h rstd weight,
 * everything after h's rounding in fp32.  h is the new residual stream.
 * In:  x [T,d] act, residual [T,d] act or NULL, weight [d] f32, eps >= 0 (finite).
 * Out: h [T,d] act or NULL (may be x or residual itself: each element is read before it is
 *      written); y [T,d] act or NULL; y8 [T,d] E4M3 codes of the unrounded y with y8_scale,
 *      or both NULL: MOE_FP8: scale = max(amax, 2^-100) / 448 per row and 128 columns, f32
 *      [d/128][T], code = RNE_E4M3(y / scale); MOE_MXFP8: codes and E8M0 bytes as
 *      moe_quantize_mx writes them, [d/128][T][4].  A block that holds an infinity or a NaN
 *      gets the scale NaN (E8M0 byte 255).  y or y8 must be given.  rstd [T] f32 or NULL
 *      (moe_add_rmsnorm_backward needs it).
 * Apart from h no output may overlap an input or another output.  y8 needs MOE_MXFP8 or
 * MOE_FP8 (MOE_ERR_DTYPE).  Tensors are aligned to 16 bytes (MOE_ERR_ALIGN); rstd and
 * y8_scale to 4.  eps that is negative, NaN or infinite, or more than 2^23 tokens: MOE_ERR_SHAPE.
 * A row whose sum of squares is above fp32's range has rstd 0; a row of zeros with eps 0 has
 * rstd infinite and y NaN.
 */
int moe_add_rmsnorm(const moe_shape* shape, const void* x, const void* residual,
                    const float* weight, float eps, void* h, void* y, uint8_t* y8,
                    void* y8_scale, float* rstd, hipStream_t stream);

/*
 * moe_add_rmsnorm_backward: with xh = h rstd and q = weight dy (the 8-bit rounding counts
 * as the identity):
 *   dx = dh + rstd (q - xh mean_i(q_i xh_i)),   dweight = sum_t dy xh,
 * dx being the gradient of x and of residual alike.
 * In:  dy [T,d] act; dh [T,d] act, the gradient that reaches h from elsewhere, or NULL;
 *      h, weight, rstd of the forward.
 * Out: dx [T,d] act (may be dy or dh itself); dweight [d] f32 or NULL.
 * Apart from dx no output may overlap an input or another output.
 * workspace: moe_workspace_bytes(shape, MOE_OP_NORM_BACKWARD) bytes.  Alignment as above.
 */
int moe_add_rmsnorm_backward(const moe_shape* shape, const void* dy, const void* dh,
                             const void* h, const float* weight, const float* rstd, void* dx,
                             float* dweight, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* ------------------------------------------------------------------ scored routing */
enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };

/* The rule of moe_route_scored (host struct). */
typedef struct moe_router {
  int32_t score;        /* enum moe_score */
  int32_t groups;       /* G equal groups of consecutive experts (G divides E, G <= 64); 1: none */
  int32_t top_groups;   /* groups a token may choose from, 1 <= top_groups <= G */
  int32_t group_top;    /* 1 or 2 (<= E / G): a group's score is the sum of its group_top best c */
  int32_t renormalise;  /* 0, or 1: the k gates are divided by their sum */
  float scale;          /* finite: every gate is multiplied by it */
} moe_router;

/*
 * moe_route_scored: moe_route with a choice of scores, a balance bias and groups.  In fp32:
 *   l = x W_r^T (+ b_r);   s = softmax_e(l) or 1 / (1 + exp(-l));   c = s (+ balance);
 *   the top_groups groups with the largest scores are kept; S = the k largest c among
 *   their experts (ties, of groups and of experts, to the lower id);
 *   g_j = scale s_j, or with renormalise scale s_j / sum_S s.
 * balance decides the choice only: gates and gradients are those of s.  Without balance the
 * experts of a token are ordered by l (the order of s).  An expert whose logit is -inf has
 * the score and the gate 0; a row whose scores are all 0 has the gates 0.  A NaN ranks
 * below every number; a row with a NaN or a +inf logit has valid expert ids, and gates that
 * may be NaN.
 * In:  x [T,d] act (bf16 for MOE_MXFP8 and MOE_FP8), w_router [E,d] f32, b_router [E] f32 or
 *      NULL, balance [E] f32 or NULL.  top_k <= top_groups * E / G.
 * Out: topk_idx, topk_gate, expert_count as moe_route; logits [T,E] f32 (l, with b_r) or
 *      NULL (moe_route_scored_backward needs them).
 * No output may overlap an input or another output.
 * workspace: moe_workspace_bytes(shape, MOE_OP_ROUTE) bytes.  A rule outside the limits
 * above, or MOE_F32 with more than 2^21 tokens: MOE_ERR_SHAPE.  x and w_router are aligned to 16 bytes (MOE_ERR_ALIGN).
 */
int moe_route_scored(const moe_shape* shape, const moe_router* router, const void* x,
                     const float* w_router, const float* b_router, const float* balance,
                     int32_t* topk_idx, float* topk_gate, int32_t* expert_count, float* logits,
                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * moe_route_scored_backward: gradients of the gates, the choice S held fixed.
 *   renormalised softmax: dl_j = g_j (dg_j - sum_S g_i dg_i / scale), softmax: dl_e =
 *   s_e (scale dg_e - sum_S scale s_i dg_i) for every e (dg_e = 0 outside S); renormalised
 *   sigmoid: dl_j = g_j (1 - s_j) (dg_j - sum_S g_i dg_i / scale), sigmoid: dl_j =
 *   scale dg_j s_j (1 - s_j);   then dl += dlogits,
 *   dx_t = dx_in_t + dl_t W_r,   dW_r = dl^T x,   db_r = sum_t dl_t.
 * In:  dgate [T,k] f32; dlogits [T,E] f32, a further gradient of the logits (a balance
 *      or z loss), or NULL; x, w_router, logits, topk_idx of the forward; dx_in [T,d] act or
 *      NULL (the experts' part of dx, moe_backward_experts).
 * Out: dx [T,d] act (may be dx_in itself); dw_router [E,d] f32; db_router [E] f32 or NULL.
 * Apart from dx no output may overlap an input or another output.
 * An id in topk_idx outside [0, E) is left out of the sums.  bf16 tokens: d times 4 E (E rounded up to
 * 64) below 2^32; MOE_F32: at most 2^21 tokens (MOE_ERR_SHAPE).
 * workspace: moe_workspace_bytes(shape, MOE_OP_ROUTE_BACKWARD) bytes.  x, w_router, dx_in, dx
 * and dw_router are aligned to 16 bytes (MOE_ERR_ALIGN).
 */
int moe_route_scored_backward(const moe_shape* shape, const moe_router* router,
                              const float* dgate, const float* dlogits, const void* x,
                              const float* w_router, const float* logits,
                              const int32_t* topk_idx, const void* dx_in, void* dx,
                              float* dw_router, float* db_router, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * moe_backward_experts: moe_backward without its router part, for a layer routed by
 * moe_route_scored: dgate [T,k] f32 (dg of each copy) is written instead of dw_router, and
 * dx holds the experts' part alone, rounded to bf16 once (moe_route_scored_backward takes
 * both and rounds dx a second time).  Arguments, limits and workspace otherwise as
 * moe_backward.
 */
int moe_backward_experts(const moe_shape* shape, const void* dy, const int32_t* topk_idx,
                         const float* topk_gate, const void* ring_x,
                         const int32_t* expert_offset, const int32_t* copy_slot,
                         const int32_t* slot_copy, int64_t ring_head, const void* saved_au,
                         const void* w_gate, const void* w_up, const void* w_down, void* dx,
                         void* dw_gate, void* dw_up, void* dw_down, float* dgate,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ FP8, scales per 128
 * moe_dispatch_q: moe_dispatch of rows that are 8-bit already (moe_add_rmsnorm's y8): x8 [T,d]
 * codes and x8_scale [d/128][T] (MOE_FP8: f32; MOE_MXFP8: 4 bytes each) are copied into the
 * ring; every other argument as moe_dispatch.  MOE_MXFP8 and MOE_FP8 only (MOE_ERR_DTYPE).
 * x8 and ring_x are aligned to 16 bytes (MOE_ERR_ALIGN); fewer than 2^24 tokens (MOE_ERR_SHAPE).
 */
int moe_dispatch_q(const moe_shape* shape, const uint8_t* x8, const uint8_t* x8_scale,
                   const int32_t* topk_idx, int64_t ring_head, void* ring_x,
                   uint8_t* ring_x_scale, int32_t* expert_offset, int32_t* copy_slot,
                   int32_t* slot_copy, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/*
 * moe_quantize_fp8: a bf16 matrix [rows, cols] (cols % 128 == 0) to E4M3 codes and fp32
 * scales, scale = max(amax, 2^-100) / 448 per block, code = RNE_E4M3(v / scale) (a block that
 * holds an infinity or a NaN: scale NaN).  row_block 1: one block per row and 128
 * columns, scales [cols/128][rows]; row_block 128: one per 128 x 128, the last block of
 * rows may be short, scales [ceil(rows/128)][cols/128].  At most 2^37 elements, and
 * with row_block 128 fewer than 2^24 blocks (MOE_ERR_SHAPE).  src and codes are aligned to 16
 * bytes (MOE_ERR_ALIGN).
 */
int moe_quantize_fp8(const void* src_bf16, int64_t rows, int64_t cols, int row_block,
                     uint8_t* codes, float* scales, hipStream_t stream);

/*
 * moe_matmul_fp8: out = A W^T of two E4M3 matrices in nn.Linear layout,
 *   out[m,n] = sum_b a_scale[b][m] w_scale[n/128][b] sum_{i in block b} a[m,i] w[n,i],
 * b running over the K/128 blocks of 128; fp32 products and sums, one rounding (a_scale w_scale is
 * formed first; a bf16 out takes a block's sum from the 8-bit matrix instruction, to 2^-13 of
 * the largest of every eight products).  out may not overlap an input.
 * In:  a [M,K], a_scale [K/128][M]; w [N,K], w_scale [ceil(N/128)][K/128] (moe_quantize_fp8
 *      with row_block 1 and 128).  K % 128 == 0; M K and N K < 2^32, M N < 2^38.
 * Out: out [M,N]: out_dtype MOE_BF16 or MOE_F32 (MOE_ERR_DTYPE otherwise).
 * M = 0 or N = 0: nothing is written.
 * workspace: moe_matmul_fp8_workspace_bytes(M, N, K) bytes (NULL if that is 0).  a and w are
 * aligned to 16 bytes, out to its element, a_scale, w_scale to 4 (MOE_ERR_ALIGN).
 */
int moe_matmul_fp8(const uint8_t* a, const float* a_scale, const uint8_t* w,
                   const float* w_scale, int64_t M, int64_t N, int64_t K, int out_dtype,
                   void* out, void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t moe_matmul_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H_ */
