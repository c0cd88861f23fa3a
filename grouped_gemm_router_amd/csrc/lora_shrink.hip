// lora_shrink.hip -- v[t] = scale[a] A[a] x[t], a = adapter[t]: each row's
// product with the first factor of its own adapter.
//
// Both operands run along K, the axis of the sum, so the matrix cores'
// fragments are 16-byte pieces of rows straight from memory; nothing is
// shared between waves but the sum over K.
//
//   * few rows: one wave per (row, rank), whole rows read with 16-byte loads;
//     the factors are read once per row that uses them, which is what a
//     decode batch of different adapters has to read anyway;
//   * many rows: 16 rows per workgroup, eight waves cutting K, every adapter
//     among the 16 rows in turn (one or two of them where rows of a request
//     follow each other); partial sums meet in LDS in wave order.
#include "lora_internal.h"

namespace {

using namespace moe;

template <int ES>
__device__ __forceinline__ float dot_piece(u32x4 a, u32x4 b, float acc) {
  if constexpr (ES == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = fmaf(bf16_bits_to_f32(a[i] & 0xffffu), bf16_bits_to_f32(b[i] & 0xffffu), acc);
      acc = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), acc);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = fmaf(__uint_as_float(a[i]), __uint_as_float(b[i]), acc);
  }
  return acc;
}

// grid (r / 4, T): four waves, one rank each
template <int ES>
__global__ __launch_bounds__(256) void shrink_row_kernel(
    const char *__restrict__ x, const char *__restrict__ F, const float *__restrict__ scale,
    const int32_t *__restrict__ adapter, int K, int r, int n, float *__restrict__ v) {
  const int t = blockIdx.y, j = blockIdx.x * 4 + threadIdx.x / kWave, lane = lane_id();
  const int a = adapter[t];
  if (a < 0 || a >= n) {
    if (lane == 0) v[(size_t)t * r + j] = 0.f;
    return;
  }
  const int np = K * ES / 16;
  const u32x4 *xp = reinterpret_cast<const u32x4 *>(x + (size_t)t * K * ES);
  const u32x4 *fp = reinterpret_cast<const u32x4 *>(F + ((size_t)a * r + j) * K * ES);
  constexpr int U = 8;
  float acc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) acc[u] = 0.f;
  for (int p0 = lane; p0 < np; p0 += U * kWave) {
    u32x4 xa[U], fa[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + u * kWave;
      xa[u] = p < np ? xp[p] : u32x4{};
      fa[u] = p < np ? fp[p] : u32x4{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] = dot_piece<ES>(xa[u], fa[u], acc[u]);
  }
#pragma unroll
  for (int u = 1; u < U; ++u) acc[0] += acc[u];
  const float sum = wave_sum(acc[0]);
  if (lane == 0) v[(size_t)t * r + j] = scale[a] * sum;
}

// one 16-byte piece per lane of both operands: 16 x 16 outputs += 64 / ES * 2
// terms.  Row (column) lane % 16 of the 16; lane / 16 picks the piece.  The
// operands agree on which k a piece holds, which is all the product needs.
template <int ES>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 acc) {
  if constexpr (ES == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i], fb[i], acc, 0, 0, 0);
    return acc;
  }
}

constexpr int kShrinkWaves = 8;

// NR: blocks of 16 ranks
template <int ES, int NR>
__global__ __launch_bounds__(kShrinkWaves *kWave) void shrink_tile_kernel(
    const char *__restrict__ x, const char *__restrict__ F, const float *__restrict__ scale,
    const int32_t *__restrict__ adapter, int T, int K, int r, int n, float *__restrict__ v) {
  constexpr int RP = NR * 16;
  __shared__ float red[kShrinkWaves][16][RP + 1];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int fr = lane & 15, fq = lane >> 4;
  const int t0 = blockIdx.x * 16;
  const int t = min(t0 + fr, T - 1);
  int a_mine = t0 + fr < T ? adapter[t] : -1;
  if (a_mine < 0 || a_mine >= n) a_mine = -1;
  // rows without an adapter get zeros
  for (int i = tid; i < 16 * r; i += kShrinkWaves * kWave) {
    const int row = i / r;
    const int a = t0 + row < T ? adapter[t0 + row] : 0;
    if (t0 + row < T && (a < 0 || a >= n)) v[(size_t)(t0 + row) * r + (i - row * r)] = 0.f;
  }
  unsigned todo = (unsigned)__ballot(a_mine >= 0) & 0xffffu;  // the same in every wave
  const int np = K * ES / 16;
  const u32x4 *xp = reinterpret_cast<const u32x4 *>(x + (size_t)t * K * ES);
  while (todo) {
    const int a = __builtin_amdgcn_readlane(a_mine, __builtin_ctz(todo));
    const unsigned same = (unsigned)__ballot(a_mine == a) & todo;
    todo &= ~same;
    const u32x4 *fp[NR];
#pragma unroll
    for (int b = 0; b < NR; ++b)  // ranks behind r repeat the last one and are not stored
      fp[b] = reinterpret_cast<const u32x4 *>(F + ((size_t)a * r + min(b * 16 + fr, r - 1)) * K * ES);
    f32x4 acc[NR];
#pragma unroll
    for (int b = 0; b < NR; ++b) acc[b] = f32x4{};
    // a wave takes two neighbouring groups of 4 pieces (whole 128-byte lines
    // of every row) out of each 16
    constexpr int U = NR <= 2 ? 4 : 2;
    for (int g0 = 2 * wv; g0 * 4 < np; g0 += (U / 2) * 2 * kShrinkWaves) {
      u32x4 xa[U], fa[U][NR];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = (g0 + (u & 1) + (u >> 1) * 2 * kShrinkWaves) * 4 + fq;
        xa[u] = p < np ? xp[p] : u32x4{};
#pragma unroll
        for (int b = 0; b < NR; ++b) fa[u][b] = p < np ? fp[b][p] : u32x4{};
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < NR; ++b) acc[b] = mma16<ES>(xa[u], fa[u][b], acc[b]);
    }
#pragma unroll
    for (int b = 0; b < NR; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wv][4 * fq + i][b * 16 + fr] = acc[b][i];
    __syncthreads();
    const float s = scale[a];
    for (int i = tid; i < 16 * RP; i += kShrinkWaves * kWave) {
      const int row = i / RP, j = i - row * RP;
      if (!((same >> row) & 1) || j >= r) continue;
      float sum = red[0][row][j];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) sum += red[w][row][j];
      v[(size_t)(t0 + row) * r + j] = s * sum;
    }
    __syncthreads();
  }
}

template <int ES>
void launch_t(const void *x, const void *F, const float *scale, const int32_t *adapter, int T, int K,
              int r, int n, float *v, hipStream_t s) {
  const char *xb = static_cast<const char *>(x), *fb = static_cast<const char *>(F);
  if (T <= kShrinkRowMax) {
    hipLaunchKernelGGL((shrink_row_kernel<ES>), dim3(r / 4, T), dim3(256), 0, s, xb, fb, scale,
                       adapter, K, r, n, v);
    return;
  }
  const dim3 grid((T + 15) / 16), block(kShrinkWaves * kWave);
#define MOE_SHRINK(NR)                                                                              \
  hipLaunchKernelGGL((shrink_tile_kernel<ES, NR>), grid, block, 0, s, xb, fb, scale, adapter, T, K, \
                     r, n, v)
  if (r <= 16) MOE_SHRINK(1);
  else if (r <= 32) MOE_SHRINK(2);
  else if (r <= 64) MOE_SHRINK(4);
  else MOE_SHRINK(8);
#undef MOE_SHRINK
}

}  // namespace

hipError_t launch_lora_shrink(const void *x, const void *F, int dt, const float *scale,
                              const int32_t *adapter, int T, int K, int r, int n, float *v,
                              hipStream_t s) {
  if (dt == MOE_BF16) launch_t<2>(x, F, scale, adapter, T, K, r, n, v, s);
  else launch_t<4>(x, F, scale, adapter, T, K, r, n, v, s);
  return hipGetLastError();
}
