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
      load8<ES>(second ? a.dC2 : a.dC, (size_t)row * a.N + na, x);
    if (nb < a.N && col < a.K)
      load8<ES>(second ? a.B2 : a.B, ((size_t)tile.g * a.N + nb) * a.ldb + col, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int m = tile.m0 + r, k = tile.nt * BT + c;
    if (m >= tile.mend || k >= a.K) return;
    const size_t at = ((size_t)slice * a.rows + m) * a.K + k;
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
    if (r < r1 && ca < a.N) load8<ES>(a.dC, (size_t)r * a.N + ca, x);
    if (r < r1 && cb < a.K) load8<ES>(a.A, (size_t)r * a.K + cb, y);
  });
  each_output(acc, [&](int r, int c, float v) {
    const int n = n0 + r, k = k0 + c;
    if (n >= a.N || k >= a.K) return;
    const size_t at = (((size_t)slice * a.G + g) * a.N + n) * a.K + k;
    put<OS>(a.out, at, a.accumulate ? v + get<OS>(a.out, at) : v);
  });
}

// the slices' sums of 8 outputs from e on, in slice order
__device__ __forceinline__ void sum8(const GradArgs &a, size_t all, size_t e, float sum[8]) {
  load8<4>(a.part, e, sum);
  float v[8];
  for (int i = 1; i < a.slices; ++i) {
    load8<4>(a.part, (size_t)i * all + e, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] += v[q];
  }
}

template <int OS>
__device__ __forceinline__ void store8(void *p, size_t e, const float v[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) put<OS>(p, e + q, v[q]);
}

template <int OS>
__global__ __launch_bounds__(256) void wgrad_reduce_kernel(const GradArgs a) {
  const size_t all = (size_t)a.G * a.N * a.K;
  for (size_t e = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; e < all;
       e += (size_t)gridDim.x * 256 * 8) {
    float sum[8], v[8];
    sum8(a, all, e, sum);
    if (a.accumulate) {
      load8<OS>(a.out, e, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += v[q];
    }
    store8<OS>(a.out, e, sum);
  }
}

// ES: element size of the operands; rows outside every group are left alone
template <int ES, int OS, bool SWIGLU>
__global__ __launch_bounds__(256) void dgrad_reduce_kernel(const GradArgs a) {
  int first, last, r;
  group_rows(a.offsets, a.rows, 0, &first, &r);
  group_rows(a.offsets, a.rows, a.G - 1, &r, &last);
  const size_t all = (size_t)a.rows * a.K;
  const size_t begin = (size_t)first * a.K, end = (size_t)last * a.K;
  for (size_t e = begin + ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; e < end;
       e += (size_t)gridDim.x * 256 * 8) {
    float v[8];
    sum8(a, all, e, v);
    if constexpr (SWIGLU) {
      float g[8], u[8], dg[8], du[8], h[8];
      load8<ES>(a.gate, e, g);
      load8<ES>(a.up, e, u);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float s = 1.f / (1.f + expf(-g[q]));
        dg[q] = v[q] * u[q] * s * (1.f + g[q] * (1.f - s));
        du[q] = v[q] * g[q] * s;
        h[q] = g[q] * s * u[q];
      }
      store8<OS>(a.out, e, dg);
      store8<OS>(a.out2, e, du);
      if (a.h) store8<OS>(a.h, e, h);
    } else {
      store8<OS>(a.out, e, v);
    }
  }
}

// the arguments of the launch that writes slices: plain fp32 sums
GradArgs sliced(const GradArgs &args) {
  GradArgs a = args;
  if (a.slices > 1) {
    a.out = a.part;
    a.out_dt = MOE_F32;
    a.gate = nullptr;
    a.accumulate = 0;
  }
  return a;
}

}  // namespace

hipError_t launch_dgrad_simple(const GradArgs &args, hipStream_t s) {
  const GradArgs a = sliced(args);
  const int nt = (a.K + BT - 1) / BT;
  const dim3 grid((unsigned)(row_tiles(a.rows, a.G, BT) * (long long)nt * a.slices)), block(256);
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

hipError_t launch_wgrad_simple(const GradArgs &args, hipStream_t s) {
  const GradArgs a = sliced(args);
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

namespace {

// 8 outputs a thread, at most 4096 workgroups
dim3 reduce_grid(size_t outputs) {
  const size_t groups = (outputs / 8 + 255) / 256;
  return dim3((unsigned)(groups < 4096 ? groups : 4096));
}

}  // namespace

hipError_t launch_wgrad_reduce(const GradArgs &a, hipStream_t s) {
  const dim3 grid = reduce_grid((size_t)a.G * a.N * a.K), block(256);
  if (a.out_dt == MOE_BF16) hipLaunchKernelGGL(wgrad_reduce_kernel<2>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(wgrad_reduce_kernel<4>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dgrad_reduce(const GradArgs &a, hipStream_t s) {
  const dim3 grid = reduce_grid((size_t)a.rows * a.K), block(256);
#define MOE_LAUNCH(ES, OS, SW) \
  hipLaunchKernelGGL((dgrad_reduce_kernel<ES, OS, SW>), grid, block, 0, s, a)
  if (a.gate) {
    if (a.dt == MOE_BF16) MOE_LAUNCH(2, 2, true); else MOE_LAUNCH(4, 4, true);
  } else if (a.out_dt == MOE_BF16) {
    MOE_LAUNCH(2, 2, false);
  } else {
    MOE_LAUNCH(4, 4, false);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}

int dgrad_slices(int G, int rows, int N, int K, int dt, int cus) {
  // the bf16 kernel's tiles are 256 x 256 outputs with stages of 64 terms, one
  // workgroup a CU; this file's 64 x 64 with steps of 32 terms, four a CU
  const bool bf16 = dt == MOE_BF16;
  const int side = bf16 ? 256 : BT, steps = (N + (bf16 ? 64 : KC) - 1) / (bf16 ? 64 : KC);
  const long long tiles = (long long)row_tiles(rows, G, side) * ((K + side - 1) / side);
  const long long room = (long long)cus * (bf16 ? 1 : 4);
  if (tiles == 0 || 2 * tiles > room || steps < 8) return 1;
  int n = (int)(room / tiles < steps / 4 ? room / tiles : steps / 4);
  const int per = (steps + n - 1) / n;
  return (steps + per - 1) / per;  // (none of them empty)
}

int wgrad_slices(int G, int rows, int N, int K, int dt, int cus) {
  // bf16: tiles of 128 x 256 weights with stages of 32 rows, two workgroups a CU
  const bool bf16 = dt == MOE_BF16;
  const long long tn = bf16 ? 128 : BT, tk = bf16 ? 256 : BT;
  const long long tiles = (N + tn - 1) / tn * ((K + tk - 1) / tk) * G;
  const long long room = (long long)cus * (bf16 ? 2 : 4);
  const int steps = rows / G / 32;  // of an average group
  // (two or three slices gain less than their sums cost: 36 groups of 847 rows,
  // 40 x 1560 weights in two slices 32 -> 40 us)
  if (4 * tiles > room || steps < 8) return 1;
  return (int)(room / tiles < steps / 4 ? room / tiles : steps / 4);
}
