// backward_internal.h -- host launchers of the backward pass, the global norm
// and the clipping (include/moe_backward.h).  Arguments are validated by the
// C-ABI layer before these are called.
#pragma once

#include "../../include/moe_backward.h"
#include "moe_internal.h"

hipError_t launch_combine_backward(const void *d_out, int dt, const void *Y, int y_dt,
                                   const int32_t *flat_to_row, const float *topk_w, int T, int k,
                                   int d, int n_shared, void *dY, float *d_topk_w, hipStream_t s);
hipError_t launch_permute_backward(const void *dx_perm, int p_dt, const int32_t *flat_to_row, int T,
                                   int k, int d, int n_shared, const void *addend, void *dx, int dt,
                                   hipStream_t s);

// What the products' gradients work on.  dgrad: out [rows][K] = dC B (+ dC2
// B2); with gate: SwiGLU's gradient, out = d_gate, out2 = d_up, h or null.
// wgrad: out [G][N][K] (+)= dC^T A per group.  slices > 1: the sums are cut
// along their terms (dgrad: N, wgrad: a group's rows), slice i's fp32 sums go
// to part + i times the output's size, and a second launch adds them in order.
struct GradArgs {
  const void *dC = nullptr, *dC2 = nullptr, *B = nullptr, *B2 = nullptr, *A = nullptr;
  const void *gate = nullptr, *up = nullptr;
  void *out = nullptr, *out2 = nullptr, *h = nullptr;
  const int32_t *offsets = nullptr;
  int G = 0, rows = 0, N = 0, K = 0, ldb = 0;
  int dt = 0, out_dt = 0;
  int accumulate = 0;
  float *part = nullptr;
  int slices = 1;
};

namespace moe {

// Rows [*r0, *r1) of group g: group g begins at the largest of
// clamp(offsets[h], 0, rows) over h <= g, as in the tile scheduler.  Every wave
// looks for itself (no barrier); must be called by whole waves.
__device__ __forceinline__ void group_rows(const int32_t *__restrict__ offsets, int rows, int g,
                                           int *r0, int *r1) {
  int first = 0;
  for (int h = lane_id(); h <= g; h += kWave) first = max(first, min(offsets[h], rows));
  const int next = min(offsets[g + 1], rows);
  *r0 = __builtin_amdgcn_readlane(wave_inclusive_max(first), kWave - 1);
  *r1 = max(*r0, next);
}

// The rows of slice i of n: runs of a multiple of 32 rows.
__device__ __forceinline__ void slice_rows(int *r0, int *r1, int i, int n) {
  const int per = ((*r1 - *r0 + n - 1) / n + 31) / 32 * 32;
  const int first = min(*r1, *r0 + i * per);
  *r1 = min(*r1, first + per);
  *r0 = first;
}

}  // namespace moe

hipError_t launch_dgrad_f32(const GradArgs &a, hipStream_t s);
hipError_t launch_wgrad_f32(const GradArgs &a, hipStream_t s);
hipError_t launch_dgrad_bf16(const GradArgs &a, hipStream_t s);
hipError_t launch_wgrad_bf16(const GradArgs &a, hipStream_t s);
// the slices' sums added in slice order and stored as the launch without slices
// would (dgrad: the rows of all groups)
hipError_t launch_dgrad_reduce(const GradArgs &a, hipStream_t s);
hipError_t launch_wgrad_reduce(const GradArgs &a, hipStream_t s);

// The arguments of a launch that writes slices: plain fp32 sums.
inline GradArgs to_slices(GradArgs a) {
  if (a.slices > 1) {
    a.out = a.part;
    a.out_dt = MOE_F32;
    a.gate = nullptr;
    a.accumulate = 0;
  }
  return a;
}

// Row tiles of BM rows that groups can have: at most one partly filled tile for
// each group with a row.
inline int row_tiles(int rows, int G, int BM) { return rows / BM + (G < rows ? G : rows); }

// Slices of the sums, so that few tiles with long sums fill the chip.  A slice
// is worth its share of a second launch (4 us) from about eight stages or
// chunks on; it keeps at least four.
int dgrad_slices(int G, int rows, int N, int K, int dt, int cus);
int wgrad_slices(int G, int rows, int N, int K, int dt, int cus);

size_t grad_norm_ws_bytes(int n);
hipError_t launch_grad_norm(const void *const *grads, const int64_t *sizes, const int *dts, int n,
                            float *norm, void *ws, hipStream_t s);
hipError_t launch_grad_clip(const void *const *grads, const int64_t *sizes, const int *dts, int n,
                            const float *norm, float max_norm, void *const *out, hipStream_t s);
