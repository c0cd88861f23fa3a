/*
 * moe_lora.h -- low-rank adapters of many requests beside a shared
 * projection in libmoe.so, forward and backward.
 *
 * Every row of a batch belongs to a request, and every request may have an
 * adapter of its own: row t's is adapter[t], and a value outside [0, n) is
 * no adapter.  Rows may come in any order; runs of rows with the same
 * adapter (a prompt) are the fastest.  With a = adapter[t]:
 *   v[t] = scale[a] * A[a] x[t]                  [r]   (0 without an adapter)
 *   y[t] = W x[t] + sum_j v[t][j] B[a][j]        [N]
 *
 * Conventions as in moe.h: device pointers to dense row-major arrays, 16-byte
 * aligned (the shared weights may have a row pitch ldw >= K), sizes checked on
 * the host before anything is launched, work only enqueued on `stream`,
 * nothing allocated, bit-identical results for the same inputs.
 *
 * Both factors are stored rank-major, A [n][r][K] and B [n][r][N] (B[a][j] is
 * the column j of the usual [N][r] matrix): the forward and the backward pass
 * then read each of them along rows only.  An adapter of a lower rank than r
 * has zero rows behind it.  x, W, A and B are of one type dt, MOE_BF16 or
 * MOE_F32; products accumulate in fp32, and v and u are fp32.  Where a bf16 y
 * or dx is computed, v (u) may enter the product with its upper 16 bits only,
 * 2^-16 of each term; everywhere else with all 24.
 * An infinity or NaN in a row of x or in an adapter stays in the rows that
 * use it and changes no bit of the others; in those rows it gives an infinity
 * or a NaN, which of them is not specified.  Outputs must not overlap inputs.
 * Requires K % 8 == 0, r % 8 == 0, 8 <= r <= MOE_LORA_MAX_RANK,
 * 1 <= n <= MOE_LORA_MAX_ADAPTERS, T <= 2^24, N and K <= 2^20 and
 * T max(N, K) <= 2^34.
 */
#ifndef MOE_LORA_H
#define MOE_LORA_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LORA_MAX_RANK 128
#define MOE_LORA_MAX_ADAPTERS 1024

/*
 * The projection.  x [T][K], W [N][K] (row pitch ldw, 0 meaning K; ldw times
 * the element size a multiple of 16 bytes), A [n][r][K], B [n][r][N], scale
 * [n] fp32, adapter [T] int32.  y [T][N] of type y_dt (dt MOE_BF16: MOE_BF16
 * or MOE_F32; dt MOE_F32: MOE_F32) and v [T][r] fp32 are written; v is what
 * the backward pass needs.  W == NULL adds the adapters' part to y in place:
 * y then holds the shared projection, computed elsewhere (from quantised
 * weights, say), and ldw must be 0.  N may be any number >= 1.
 * T == 0 is a no-op.  ws (16-byte aligned) must hold
 * moe_lora_linear_workspace_size bytes (else MOE_ERR_WORKSPACE); 0 bytes: may
 * be NULL.  Calls that share it must be ordered.
 */
moe_status_t moe_lora_linear(const void *x, const void *W, int ldw, const void *A,
                             const void *B, moe_dtype_t dt, const float *scale,
                             const int32_t *adapter, int T, int N, int K, int r, int n, void *y,
                             moe_dtype_t y_dt, float *v, void *ws, size_t ws_bytes,
                             moe_stream_t stream);

/* Bytes of device workspace moe_lora_linear needs for these sizes. */
size_t moe_lora_linear_workspace_size(int T, int N, int K, int r, int n, moe_dtype_t dt);

/*
 * Its gradients, for a frozen W.  With a = adapter[t]:
 *   u[t]     = scale[a] * B[a] dy[t]                       [r] (0 without an adapter)
 *   dx[t]    = W^T dy[t] + sum_j u[t][j] A[a][j]           [K]
 *   dA[a][j] = sum over the rows t of a of u[t][j] x[t]    [K]
 *   dB[a][j] = sum over the rows t of a of v[t][j] dy[t]   [N]
 * dy [T][N], x [T][K] and v [T][r] as in the forward pass; W_t [K][N] is W
 * transposed (row pitch ldw, 0 meaning N), all but v of type dt (so dy is too
 * where y was fp32 beside bf16 factors: the caller rounds it).  dx [T][K] of type
 * dt or NULL; W_t == NULL adds the adapters' part to dx in place.  dA [n][r][K]
 * and dB [n][r][N], both fp32, are both written or both NULL; an adapter
 * without rows gets zeros (all of them for T == 0).  u [T][r] fp32 is written.  Requires N % 8 == 0
 * too.  The sums over rows run in a fixed order.
 * ws (16-byte aligned) must hold moe_lora_backward_workspace_size bytes
 * (else MOE_ERR_WORKSPACE); calls that share it must be ordered.
 */
moe_status_t moe_lora_linear_backward(const void *dy, const void *x, const void *W_t, int ldw,
                                      const void *A, const void *B, moe_dtype_t dt,
                                      const float *scale, const int32_t *adapter,
                                      const float *v, int T, int N, int K, int r, int n,
                                      float *u, void *dx, float *dA, float *dB, void *ws,
                                      size_t ws_bytes, moe_stream_t stream);

/* Bytes of device workspace moe_lora_linear_backward needs for these sizes. */
size_t moe_lora_backward_workspace_size(int T, int N, int K, int r, int n, moe_dtype_t dt);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LORA_H */
