// lora_internal.h -- what the translation units of the low-rank adapters
// share.
#pragma once

#include "moe_internal.h"
#include "../../include/moe_lora.h"

namespace moe {

// rows up to which the shrink runs one wave per (row, rank)
constexpr int kShrinkRowMax = 128;

// Piece p of a row of np pieces, zero behind the row's end.  The load itself is
// unconditional: under a condition, each load of a batch gets its own branch
// and wait.
__device__ __forceinline__ u32x4 load_piece(const u32x4 *row, int p, int np) {
  const u32x4 q = row[min(p, np - 1)];
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = p < np ? q[i] : 0u;
  return r;
}

// fp32 -> the bf16 terms of a sum that holds it: f = t[0] + t[1] (+ t[2]),
// each the rounded rest of the one before.  Two terms keep 16 bits of f,
// three all 24.
template <int TERMS>
__device__ __forceinline__ void split_bf16(const float (&f)[8], bf16x8 (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = f[i];
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      t[k][i] = (__bf16)rest;  // round to nearest even
      rest -= (float)t[k][i];
    }
  }
}

}  // namespace moe

hipError_t launch_lora_shrink(const void *x, const void *F, int dt, const float *scale,
                              const int32_t *adapter, int T, int K, int r, int n, float *v,
                              hipStream_t s);

// y (+)= x W^T + v F: W null adds to y
hipError_t launch_lora_expand(const void *x, const void *W, int ldw, const void *F, int dt,
                              const float *v, const int32_t *adapter, int T, int N, int K, int r,
                              int n, void *y, int y_dt, int cus, hipStream_t s);

size_t lora_wgrad_ws_bytes(int T, int N, int K, int r, int n);
hipError_t launch_lora_wgrad(const void *dy, const void *x, int dt, const float *u, const float *v,
                             const int32_t *adapter, int T, int N, int K, int r, int n, float *dA,
                             float *dB, void *ws, hipStream_t s);
