/*
 * moe_backward.h -- the backward pass of the expert layer in libmoe.so: the
 * gradients of moe_combine, of the grouped products and of moe_permute, and
 * the global norm of many gradients with their clipping.
 *
 * A training step behind the forward pass of moe.h, on one stream:
 *   moe_combine_backward          d_out -> dY, d_topk_w
 *   moe_grouped_gemm (twice)      gate and up before SwiGLU, computed again
 *                                 from x_perm (the forward pass keeps only h)
 *   moe_grouped_gemm_dgrad_swiglu dY -> d_gate, d_up
 *   moe_grouped_gemm_wgrad        dY, h -> w_down's gradient
 *   moe_grouped_gemm_dgrad        d_gate, d_up -> dx_perm
 *   moe_grouped_gemm_wgrad        d_gate (d_up), x_perm -> w_gate's (w_up's)
 *   moe_permute_backward          dx_perm -> dx
 *   moe_route_backward            d_topk_w -> d_logits (moe_balance.h)
 *   moe_grad_norm, moe_grad_clip  over all of the step's gradients
 *
 * Conventions as in moe.h: device pointers to dense row-major arrays, 16-byte
 * aligned unless stated, sizes checked on the host before anything is
 * launched, work only enqueued on `stream`, nothing allocated, bit-identical
 * results for the same inputs on the same device.  Sums are held in fp32 or
 * more and rounded once, when they are stored.  An output may be an operand
 * only where its entry says so; one that overlaps an operand, another output
 * or the workspace otherwise, be it in part, is MOE_ERR_INVALID (arrays are
 * counted with all their rows, those of no group too).
 */
#ifndef MOE_BACKWARD_H
#define MOE_BACKWARD_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gradient of moe_combine ("DeepGEMM walkthrough" §2.1, y = E_shared(x) +
 * sum_i p_i E_i(x), differentiated by E_i(x) and p_i).  With row(t, j) =
 * flat_to_row[t k + j]:
 *   dY[row(t, j)][c]                    = topk_w[t][j] * d_out[t][c]
 *   dY[flat_to_row[T k + s T + t]][c]   = d_out[t][c]       (shared experts)
 *   d_topk_w[t][j] = sum_c d_out[t][c] * Y[row(t, j)][c]
 * An entry < 0 (a dropped one) writes no row of dY and gets d_topk_w 0; so
 * does one that is not below T k + n_shared T.  Rows of dY that no entry
 * names are left as they were.  No two entries may name the same row.
 *
 * d_out [T][d] and dY [T k + n_shared T][d] of type dt (MOE_F32 or MOE_BF16),
 * Y of type y_dt (either) as moe_combine read it; topk_w, d_topk_w [T][k]
 * fp32.  dY may be NULL, or d_topk_w with Y (a frozen router): that part is
 * then not computed; not both.  d_topk_w may be topk_w.
 * Requires d % 8 == 0, 1 <= k <= MOE_MAX_TOPK, n_shared <= 8, T < 2^24.
 */
moe_status_t moe_combine_backward(const void *d_out, moe_dtype_t dt, const void *Y,
                                  moe_dtype_t y_dt, const int32_t *flat_to_row,
                                  const float *topk_w, int T, int k, int d, int n_shared,
                                  void *dY, float *d_topk_w, moe_stream_t stream);

/*
 * Gradient of moe_permute's row copies (every token's row was copied to its
 * k experts and to the shared ones):
 *   dx[t][c] = sum_j dx_perm[flat_to_row[t k + j]][c]
 *            + sum_s dx_perm[flat_to_row[T k + s T + t]][c] + addend[t][c]
 * in fp32, in that order; entries < 0 or out of range add nothing.
 * dx_perm [T k + n_shared T][d] of type p_dt, dx [T][d] of type dt and
 * addend [T][d] of type dt or NULL (what reached x by another path: the
 * router's part, or a residual's); addend may be dx.
 * Requires d % 8 == 0, 1 <= k <= MOE_MAX_TOPK, n_shared <= 8, T < 2^24.
 */
moe_status_t moe_permute_backward(const void *dx_perm, moe_dtype_t p_dt,
                                  const int32_t *flat_to_row, int T, int k, int d, int n_shared,
                                  const void *addend, void *dx, moe_dtype_t dt,
                                  moe_stream_t stream);

/*
 * Gradient of a grouped product's input.  moe_grouped_gemm computed C[r][n] =
 * sum_k A[r][k] B[g][n][k]; with dC the gradient of C, for the rows r of
 * group g (offsets [G+1] as in moe_grouped_gemm):
 *   dA[r][k] = sum_n dC[r][n] B[g][n][k] + sum_n dC2[r][n] B2[g][n][k]
 * The second product (dC2, B2) is for two products of one input, as gate and
 * up; NULL, NULL without it.  The weights are read as the forward pass stores
 * them.  Rows of dA outside every group are left as they were; rows of dC
 * outside every group are not used.
 *
 * dC, dC2 [rows][N] and B, B2 [G][N][ldb] of type dt (ldb: row pitch of the
 * weights as in moe_grouped_gemm, 0 means K), dA [rows][K] of type a_dt: dt
 * or MOE_F32.  ws (device, 16-byte aligned) must
 * hold moe_grouped_gemm_dgrad_workspace_size bytes (else MOE_ERR_WORKSPACE;
 * NULL with ws_bytes 0 where that is 0); calls that share it must be ordered.
 * Few tiles with long sums are cut along N; the slices' fp32 sums lie in ws and
 * are added in a fixed order.
 * Requires N % 8 == 0, K % 8 == 0, N and ldb < MOE_MAX_GRAD_WIDTH,
 * 1 <= G <= MOE_MAX_GROUPS, G N ldb < 2^40, and fewer than 2^24 tiles of 64 x
 * 64 outputs ((rows / 64 + G) K / 64, and for the weights, of both calls, G N
 * K / 4096, each side in whole tiles).
 */
#define MOE_MAX_GRAD_WIDTH (1 << 23)
moe_status_t moe_grouped_gemm_dgrad(const void *dC, const void *B, const void *dC2,
                                    const void *B2, moe_dtype_t dt, void *dA, moe_dtype_t a_dt,
                                    const int32_t *offsets, int G, int rows, int N, int K,
                                    int ldb, void *ws, size_t ws_bytes, moe_stream_t stream);

/*
 * The same for an input that was SwiGLU's output, A = silu(gate) * up, with
 * SwiGLU's gradient behind the product.  With a = sum_n dC[r][n] B[g][n][k]
 * held in fp32 and s = 1 / (1 + e^-gate):
 *   d_gate[r][k] = a * up * s * (1 + gate * (1 - s))
 *   d_up[r][k]   = a * gate * s
 *   h[r][k]      = gate * s * up          (only if h is given)
 * gate, up, d_gate, d_up and h [rows][K] are of type dt.  d_gate may be gate,
 * and d_up may be up.
 * Everything else as moe_grouped_gemm_dgrad.
 */
moe_status_t moe_grouped_gemm_dgrad_swiglu(const void *dC, const void *B, moe_dtype_t dt,
                                           const void *gate, const void *up, void *d_gate,
                                           void *d_up, void *h, const int32_t *offsets, int G,
                                           int rows, int N, int K, int ldb, void *ws,
                                           size_t ws_bytes, moe_stream_t stream);

/* Workspace bytes of both (on the current device); 0 for invalid arguments. */
size_t moe_grouped_gemm_dgrad_workspace_size(int G, int rows, int N, int K, moe_dtype_t dt);

/*
 * Gradient of a grouped product's weights:
 *   dB[g][n][k] = sum_{r in group g} dC[r][n] A[r][k]   (+ dB, if accumulate)
 * A group without rows gets zeros (or keeps dB).  Rows outside every group
 * are not used and may hold anything.  dC [rows][N], A [rows][K] of type dt,
 * dB [G][N][K] dense, of type b_dt: dt or MOE_F32.  With accumulate != 0 the
 * sum is added in fp32 to what dB holds and rounded once.  ws as for
 * moe_grouped_gemm_dgrad (the sums are cut along a group's rows), of
 * moe_grouped_gemm_wgrad_workspace_size bytes.  Sizes as there.
 */
moe_status_t moe_grouped_gemm_wgrad(const void *dC, const void *A, moe_dtype_t dt, void *dB,
                                    moe_dtype_t b_dt, const int32_t *offsets, int G, int rows,
                                    int N, int K, int accumulate, void *ws, size_t ws_bytes,
                                    moe_stream_t stream);

size_t moe_grouped_gemm_wgrad_workspace_size(int G, int rows, int N, int K, moe_dtype_t dt);

/*
 * Global 2-norm of n gradients:
 *   *norm = sqrt(sum_i sum_e grads[i][e]^2)
 * grads, sizes and dts are HOST arrays of n device pointers, element counts
 * and types (MOE_F32 or MOE_BF16, mixed as they come); a pointer need only be
 * aligned to its type (a view into a bucket), and a size of 0 with any
 * pointer is skipped.  The squares are summed in 64 bits, in an order that
 * depends on sizes and alignments alone; NaN and infinity come through.  norm
 * [1] fp32 on the device.  ws (device, 8-byte aligned) must hold
 * moe_grad_norm_workspace_size(n) bytes (else MOE_ERR_WORKSPACE); calls that
 * share it must be ordered.  The host arrays are read before the call
 * returns.  Requires 0 <= n <= MOE_MAX_GRADS, sizes < 2^40.
 */
#define MOE_MAX_GRADS 65536
moe_status_t moe_grad_norm(const void *const *grads, const int64_t *sizes,
                           const moe_dtype_t *dts, int n, float *norm, void *ws, size_t ws_bytes,
                           moe_stream_t stream);

size_t moe_grad_norm_workspace_size(int n);

/*
 * Clipping by a norm that is on the device (moe_grad_norm's, or one that was
 * summed over several GPUs):
 *   out[i][e] = grads[i][e] * min(1, max_norm / (*norm + 1e-6))
 * in fp32, rounded once; out[i] of grads[i]'s size and type.  out == NULL
 * scales in place; out[i] may also be grads[i].  MOE_ERR_INVALID where an
 * output overlaps the norm, another gradient or output (the same tensor twice)
 * or its own gradient in part.  Where the factor is 1, what is in place is left
 * alone (bit for bit) and the rest copied.  A norm of NaN makes every value NaN, an infinite norm every finite one 0.
 * Arrays as in moe_grad_norm.
 * Requires max_norm >= 0 and finite.
 */
moe_status_t moe_grad_clip(const void *const *grads, const int64_t *sizes,
                           const moe_dtype_t *dts, int n, const float *norm, float max_norm,
                           void *const *out, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BACKWARD_H */
