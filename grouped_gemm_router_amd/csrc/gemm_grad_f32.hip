// gemm_grad_f32.hip -- the gradients of the grouped products of fp32 operands,
// for any sizes, on the fp32 matrix cores:
//   dgrad  dA[r][k] = sum_n dC[r][n] B[g][n][k] (+ dC2 B2), r in group g,
//          with SwiGLU's gradient behind it or not
//   wgrad  dB[g][n][k] (+)= sum_{r in group g} dC[r][n] A[r][k]
//
// One workgroup per 64 x 64 outputs, 4 waves of 32 x 32 on
// v_mfma_f32_32x32x2_f32, 32 terms of the sum at a time: both operands go
// through registers into LDS as [term][column], where a fragment (32 columns
// of two terms) is read without conflicts.  Every kFold steps the running sums
// are added to a second set, so no chain of fp32 additions is longer than 128
// instructions plus the number of folds (8192 random terms in one chain would
// err by about 2e-6 of their norm).
// The small layer's shapes (512 rows of 8 groups, 128 x 256) take 9 us, bound by
// the latency of the tile's lookup and of each step's loads; 532 rows of 1768 x
// 1128 with SwiGLU 54 us, 39 TFLOP/s of the 135 that a 4096^3 library product
// reaches: short of tiles and of loads in flight.
#include "backward_internal.h"

namespace {

using namespace moe;

constexpr int BT = 64;       // outputs a side
constexpr int KC = 32;       // terms of the sum a step
constexpr int LDT = BT + 32; // LDS row: its upper half wave reads other banks
constexpr int kFold = 8;     // steps between two folds

__device__ __forceinline__ void load8(const void *base, size_t elem, float v[8]) {
  const f32x4 *const p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem);
  *reinterpret_cast<f32x4 *>(v) = p[0];
  *reinterpret_cast<f32x4 *>(v + 4) = p[1];
}

struct Shared {
  float a[KC][LDT], b[KC][LDT];
};

// The 64 x 64 sums over `terms` terms.  fetch(term, x, y) loads this thread's
// 8 values of each operand for the step that begins at `term`; A_ROWS: its a
// values are 8 terms of one output row (else 8 output rows of one term).
template <bool A_ROWS, class Fetch>
__device__ __forceinline__ f32x16 product(Shared &s, int terms, Fetch fetch) {
  const int t = threadIdx.x, lane = lane_id(), wave = t / kWave;
  const int wm = wave / 2, wn = wave % 2;
  f32x16 acc{}, total{};
  float x[8], y[8];
  if (terms > 0) fetch(0, x, y);
  int steps = 0;
  for (int k0 = 0; k0 < terms; k0 += KC) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (A_ROWS) s.a[(t % 4) * 8 + i][t / 4] = x[i];
      else s.a[t / 8][(t % 8) * 8 + i] = x[i];
      s.b[t / 8][(t % 8) * 8 + i] = y[i];
    }
    __syncthreads();
    if (k0 + KC < terms) fetch(k0 + KC, x, y);
#pragma unroll
    for (int k = 0; k < KC; k += 2) {
      const float a = s.a[k + lane / 32][wm * 32 + lane % 32];
      const float b = s.b[k + lane / 32][wn * 32 + lane % 32];
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc, 0, 0, 0);
    }
    if (++steps == kFold) {
      total += acc;
      acc = f32x16{};
      steps = 0;
    }
  }
  return total + acc;
}

// calls f(row, column, value) for this thread's 16 of the 64 x 64 outputs
template <class F>
__device__ __forceinline__ void each_output(const f32x16 &acc, F f) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int wm = wave / 2, wn = wave % 2;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    f(wm * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4, wn * 32 + lane % 32, acc[r]);
}

template <bool SWIGLU>
__global__ __launch_bounds__(256) void dgrad_f32_kernel(const GradArgs a, int nt) {
  __shared__ Shared s;
  __shared__ int s_x[8];
  const int w = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const Sched sc = sched_lookup(a.offsets, a.G, a.rows, BT, nt, kTileChunk, false, s_x,
                                [w](int total) { return tile_of_workgroup(w, total); });
  if (sc.L < 0) return;
  const Tile tile = sc.tile;
  const int t = threadIdx.x;
  const int row = tile.m0 + t / 4, col = tile.nt * BT + (t % 8) * 8;
  // the second product's terms follow the first's, from a whole step on
  const int span = (a.N + KC - 1) / KC * KC;
  const int terms = a.dC2 ? 2 * span : span;
  const int per = (terms / KC + a.slices - 1) / a.slices * KC, first = slice * per;
  const f32x16 acc = product<true>(s, min(per, terms - first), [&](int k0, float *x, float *y) {
    k0 += first;
    const bool second = k0 >= span;
    const int n0 = second ? k0 - span : k0;
    const int na = n0 + (t % 4) * 8, nb = n0 + t / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (row < tile.mend && na < a.N)
      load8(second ? a.dC2 : a.dC, (size_t)row * a.N + na, x);
    if (nb < a.N && col < a.K)
      load8(second ? a.B2 : a.B, ((size_t)tile.g * a.N + nb) * a.ldb + col, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int m = tile.m0 + r, k = tile.nt * BT + c;
    if (m >= tile.mend || k >= a.K) return;
    const size_t at = ((size_t)slice * a.rows + m) * a.K + k;
    float *const out = static_cast<float *>(a.out);
    if constexpr (SWIGLU) {
      const float g = static_cast<const float *>(a.gate)[at], u = static_cast<const float *>(a.up)[at];
      const float sig = 1.f / (1.f + expf(-g));
      out[at] = v * u * sig * (1.f + g * (1.f - sig));
      static_cast<float *>(a.out2)[at] = v * g * sig;
      if (a.h) static_cast<float *>(a.h)[at] = g * sig * u;
    } else {
      out[at] = v;
    }
  });
}

__global__ __launch_bounds__(256) void wgrad_f32_kernel(const GradArgs a, int nt, int kt) {
  __shared__ Shared s;
  int w = blockIdx.x;
  const int k0 = w % kt * BT;
  w /= kt;
  const int n0 = w % nt * BT;
  w /= nt;
  const int g = w % a.G, slice = w / a.G;
  int r0, r1;
  group_rows(a.offsets, a.rows, g, &r0, &r1);
  if (a.slices > 1) slice_rows(&r0, &r1, slice, a.slices);
  const int t = threadIdx.x;
  const int ca = n0 + (t % 8) * 8, cb = k0 + (t % 8) * 8;
  const f32x16 acc = product<false>(s, r1 - r0, [&](int k, float *x, float *y) {
    const int r = r0 + k + t / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (r < r1 && ca < a.N) load8(a.dC, (size_t)r * a.N + ca, x);
    if (r < r1 && cb < a.K) load8(a.A, (size_t)r * a.K + cb, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int n = n0 + r, k = k0 + c;
    if (n >= a.N || k >= a.K) return;
    const size_t at = (((size_t)slice * a.G + g) * a.N + n) * a.K + k;
    float *const out = static_cast<float *>(a.out) + at;
    *out = a.accumulate ? v + *out : v;
  });
}

}  // namespace

hipError_t launch_dgrad_f32(const GradArgs &args, hipStream_t s) {
  const GradArgs a = to_slices(args);
  const int nt = (a.K + BT - 1) / BT;
  const dim3 grid((unsigned)(row_tiles(a.rows, a.G, BT) * (long long)nt * a.slices)), block(256);
  if (a.gate) hipLaunchKernelGGL(dgrad_f32_kernel<true>, grid, block, 0, s, a, nt);
  else hipLaunchKernelGGL(dgrad_f32_kernel<false>, grid, block, 0, s, a, nt);
  return hipGetLastError();
}

hipError_t launch_wgrad_f32(const GradArgs &args, hipStream_t s) {
  const GradArgs a = to_slices(args);
  const int nt = (a.N + BT - 1) / BT, kt = (a.K + BT - 1) / BT;
  const dim3 grid((unsigned)((long long)a.slices * a.G * nt * kt)), block(256);
  hipLaunchKernelGGL(wgrad_f32_kernel, grid, block, 0, s, a, nt, kt);
  return hipGetLastError();
}
