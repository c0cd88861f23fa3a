// gemm_grad_simple.hip -- the gradients of the grouped products on the fp32
// matrix cores, for any sizes: fp32 operands as they are, bf16 ones widened.
//
//   dgrad  dA[r][k] = sum_n dC[r][n] B[g][n][k] (+ dC2 B2), r in group g,
//          with SwiGLU's gradient behind it or not
//   wgrad  dB[g][n][k] (+)= sum_{r in group g} dC[r][n] A[r][k]
//
// One workgroup per 64 x 64 outputs, 4 waves of 32 x 32 on
// v_mfma_f32_32x32x2_f32, 32 terms of the sum at a time: both operands go
// through registers into LDS as [term][column], where a fragment (32 columns
// of two terms) is read without conflicts.  Every kFold terms the running sums
// are added to a second set, so no chain of fp32 additions is longer than that
// plus the number of folds.
#include "backward_internal.h"

namespace {

using namespace moe;

constexpr int BT = 64;       // outputs a side
constexpr int KC = 32;       // terms of the sum a step
constexpr int LDT = BT + 32; // LDS row: its upper half wave reads other banks
constexpr int kFold = 8;     // steps between two folds

template <int ES>
__device__ __forceinline__ void load8(const void *base, size_t elem, float v[8]) {
  if constexpr (ES == 2) {
    const u32x4 raw = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32(raw[i] & 0xffffu);
      v[2 * i + 1] = bf16_bits_to_f32(raw[i] >> 16);
    }
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <int ES>
__device__ __forceinline__ float get(const void *p, size_t e) {
  if constexpr (ES == 2) return bf16_bits_to_f32(static_cast<const uint16_t *>(p)[e]);
  else return static_cast<const float *>(p)[e];
}

template <int ES>
__device__ __forceinline__ void put(void *p, size_t e, float v) {
  if constexpr (ES == 2) static_cast<uint16_t *>(p)[e] = f32_to_bf16_bits(v);
  else static_cast<float *>(p)[e] = v;
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

template <int ES, int OS, bool SWIGLU>
__global__ __launch_bounds__(256) void dgrad_simple_kernel(const GradArgs a, int nt) {
  __shared__ Shared s;
  __shared__ int s_x[8];
  const Sched sc = sched_lookup(a.offsets, a.G, a.rows, BT, nt, kTileChunk, false, s_x,
                                [](int total) { return tile_of_workgroup(blockIdx.x, total); });
  if (sc.L < 0) return;
  const Tile tile = sc.tile;
  const int t = threadIdx.x;
  const int row = tile.m0 + t / 4, col = tile.nt * BT + (t % 8) * 8;
  // the second product's terms follow the first's, from a whole step on
  const int span = (a.N + KC - 1) / KC * KC;
  const f32x16 acc = product<true>(s, a.dC2 ? 2 * span : span, [&](int k0, float *x, float *y) {
    const bool second = k0 >= span;
    const int n0 = second ? k0 - span : k0;
    const int na = n0 + (t % 4) * 8, nb = n0 + t / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (row < tile.mend && na < a.N)
      load8<ES>(second ? a.dC2 : a.dC, (size_t)row * a.N + na, x);
    if (nb < a.N && col < a.K)
      load8<ES>(second ? a.B2 : a.B, ((size_t)tile.g * a.N + nb) * a.ldb + col, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int m = tile.m0 + r, k = tile.nt * BT + c;
    if (m >= tile.mend || k >= a.K) return;
    const size_t at = (size_t)m * a.K + k;
    if constexpr (SWIGLU) {
      const float g = get<ES>(a.gate, at), u = get<ES>(a.up, at);
      const float sig = 1.f / (1.f + expf(-g));
      put<OS>(a.out, at, v * u * sig * (1.f + g * (1.f - sig)));
      put<OS>(a.out2, at, v * g * sig);
      if (a.h) put<OS>(a.h, at, g * sig * u);
    } else {
      put<OS>(a.out, at, v);
    }
  });
}

template <int ES, int OS>
__global__ __launch_bounds__(256) void wgrad_simple_kernel(const GradArgs a, int nt, int kt) {
  __shared__ Shared s;
  __shared__ int s_rows[2];
  int w = blockIdx.x;
  const int k0 = w % kt * BT;
  w /= kt;
  const int n0 = w % nt * BT;
  w /= nt;
  const int g = w % a.G, slice = w / a.G;
  group_rows(a.offsets, a.rows, g, s_rows);
  int r0 = s_rows[0], r1 = s_rows[1];
  if (a.part) slice_rows(&r0, &r1, slice, a.slices);
  const int t = threadIdx.x;
  const int ca = n0 + (t % 8) * 8, cb = k0 + (t % 8) * 8;
  const f32x16 acc = product<false>(s, r1 - r0, [&](int k, float *x, float *y) {
    const int r = r0 + k + t / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (r < r1 && ca < a.N) load8<ES>(a.dC, (size_t)r * a.N + ca, x);
    if (r < r1 && cb < a.K) load8<ES>(a.A, (size_t)r * a.K + cb, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int n = n0 + r, k = k0 + c;
    if (n >= a.N || k >= a.K) return;
    const size_t at = ((size_t)g * a.N + n) * a.K + k;
    if (a.part) a.part[(size_t)slice * a.G * a.N * a.K + at] = v;
    else put<OS>(a.out, at, a.accumulate ? v + get<OS>(a.out, at) : v);
  });
}

// out (+)= the sum of the slices' partial sums, in slice order; 8 outputs a
// thread and step
template <int OS>
__global__ __launch_bounds__(256) void wgrad_reduce_kernel(const GradArgs a) {
  const size_t all = (size_t)a.G * a.N * a.K;
  for (size_t e = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; e < all;
       e += (size_t)gridDim.x * 256 * 8) {
    float sum[8], v[8];
    load8<4>(a.part, e, sum);
    for (int i = 1; i < a.slices; ++i) {
      load8<4>(a.part, (size_t)i * all + e, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += v[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      put<OS>(a.out, e + q, a.accumulate ? sum[q] + get<OS>(a.out, e + q) : sum[q]);
  }
}

}  // namespace

hipError_t launch_dgrad_simple(const GradArgs &a, hipStream_t s) {
  const int nt = (a.K + BT - 1) / BT;
  const dim3 grid((unsigned)(host_row_tile_bound(a.rows, a.G, BT) * (long long)nt)), block(256);
#define MOE_LAUNCH(ES, OS, SW) \
  hipLaunchKernelGGL((dgrad_simple_kernel<ES, OS, SW>), grid, block, 0, s, a, nt)
  if (a.gate) {
    if (a.dt == MOE_BF16) MOE_LAUNCH(2, 2, true); else MOE_LAUNCH(4, 4, true);
  } else if (a.dt == MOE_BF16) {
    if (a.out_dt == MOE_BF16) MOE_LAUNCH(2, 2, false); else MOE_LAUNCH(2, 4, false);
  } else {
    MOE_LAUNCH(4, 4, false);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_wgrad_simple(const GradArgs &a, hipStream_t s) {
  const int nt = (a.N + BT - 1) / BT, kt = (a.K + BT - 1) / BT;
  const dim3 grid((unsigned)((long long)a.slices * a.G * nt * kt)), block(256);
#define MOE_LAUNCH(ES, OS) \
  hipLaunchKernelGGL((wgrad_simple_kernel<ES, OS>), grid, block, 0, s, a, nt, kt)
  if (a.dt == MOE_F32) MOE_LAUNCH(4, 4);
  else if (a.out_dt == MOE_F32) MOE_LAUNCH(2, 4);
  else MOE_LAUNCH(2, 2);
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_wgrad_reduce(const GradArgs &a, hipStream_t s) {
  const size_t groups = ((size_t)a.G * a.N * a.K / 8 + 255) / 256;
  const dim3 grid((unsigned)(groups < 4096 ? groups : 4096)), block(256);
  if (a.out_dt == MOE_BF16) hipLaunchKernelGGL(wgrad_reduce_kernel<2>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(wgrad_reduce_kernel<4>, grid, block, 0, s, a);
  return hipGetLastError();
}
