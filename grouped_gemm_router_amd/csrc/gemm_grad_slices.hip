// gemm_grad_slices.hip -- products' gradients whose few, long sums are cut into
// slices: how many, and the launch that adds them.
//
// A tile's sum is one workgroup's work, whatever its length, so few tiles with
// long sums leave the chip idle (237 x 152 outputs with sums of 4984: 12 tiles
// of fp32, 193 us; in 39 slices 28).  The slices' fp32 sums lie one behind the
// other and are added in order; what the tiles do with their sums (SwiGLU's
// gradient, rounding, adding to what is there) is done here instead.
#include "backward_internal.h"

namespace {

using namespace moe;

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
    const f32x4 *const p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem);
    *reinterpret_cast<f32x4 *>(v) = p[0];
    *reinterpret_cast<f32x4 *>(v + 4) = p[1];
  }
}

template <int ES>
__device__ __forceinline__ void store8(void *base, size_t elem, const float v[8]) {
  if constexpr (ES == 2) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + elem) = o;
  } else {
    f32x4 *const p = reinterpret_cast<f32x4 *>(static_cast<float *>(base) + elem);
    p[0] = *reinterpret_cast<const f32x4 *>(v);
    p[1] = *reinterpret_cast<const f32x4 *>(v + 4);
  }
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
  // workgroup a CU; the fp32 kernel's 64 x 64 with steps of 32 terms, four a CU
  const bool bf16 = dt == MOE_BF16;
  const int side = bf16 ? 256 : 64, steps = (N + (bf16 ? 64 : 32) - 1) / (bf16 ? 64 : 32);
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
  const long long tn = bf16 ? 128 : 64, tk = bf16 ? 256 : 64;
  const long long tiles = (N + tn - 1) / tn * ((K + tk - 1) / tk) * G;
  const long long room = (long long)cus * (bf16 ? 2 : 4);
  const int steps = rows / G / 32;  // of an average group
  // (two or three slices gain less than their sums cost: 36 groups of 847 rows,
  // 40 x 1560 weights in two slices 32 -> 40 us)
  if (4 * tiles > room || steps < 8) return 1;
  return (int)(room / tiles < steps / 4 ? room / tiles : steps / 4);
}
