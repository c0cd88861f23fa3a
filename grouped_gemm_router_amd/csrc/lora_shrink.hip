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
//   * many rows: 16 rows and 16 ranks per workgroup of eight waves.  Where
//     the rows have few adapters (prompts), the waves cut K and the matrix
//     cores multiply, one adapter after the other; partial sums meet in LDS
//     in wave order.  Otherwise each wave takes a row and reads that row's
//     own factors.
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
      xa[u] = load_piece(xp, p, np);
      fa[u] = load_piece(fp, p, np);
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

// Sum of each of a lane's eight values over the wave: the result for value
// lane & 7 (bit-reversed: value 4 (lane & 1) + 2 (lane >> 1 & 1) + (lane >> 2
// & 1)).  Each of the first three steps halves the values that a lane still
// holds, ten exchanges in all instead of 48; the order is fixed.
__device__ __forceinline__ float sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int h = 4, o = 1; h > 0; h >>= 1, o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h];
      v[i] = (up ? v[i + h] : v[i]) + __shfl_xor(send, o, kWave);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = 8; o < kWave; o <<= 1) s += __shfl_xor(s, o, kWave);
  return s;
}

constexpr int kShrinkWaves = 8;

// Adapters among 16 rows up to which the tile takes them one after the other
// on the matrix cores: a pass costs its latency and 32 rows of operands, the
// other way 17 rows of operands per row.
__device__ __forceinline__ bool few_adapters(int kinds, int row_bytes) {
  return kinds <= 1 || kinds * 2048 <= row_bytes;
}

// one chunk's pieces of a wave: two neighbouring groups of 4 pieces (whole
// 128-byte lines of every row) out of each 2 kShrinkWaves groups
constexpr int kShrinkU = 4, kShrinkChunk = kShrinkU * kShrinkWaves * 4;

struct ShrinkPieces {
  u32x4 x[kShrinkU], f[kShrinkU];
  static __device__ __forceinline__ int at(int u, int wv, int fq) {
    return (2 * wv + (u & 1) + (u >> 1) * 2 * kShrinkWaves) * 4 + fq;
  }
  __device__ __forceinline__ void load(const u32x4 *xp, const u32x4 *fp, int p0, int wv, int fq) {
#pragma unroll
    for (int u = 0; u < kShrinkU; ++u) {
      x[u] = xp[p0 + at(u, wv, fq)];
      f[u] = fp[p0 + at(u, wv, fq)];
    }
  }
  // the last chunk: zeros behind the row's np pieces
  __device__ __forceinline__ void load_tail(const u32x4 *xp, const u32x4 *fp, int p0, int np, int wv,
                                            int fq) {
#pragma unroll
    for (int u = 0; u < kShrinkU; ++u) {
      x[u] = load_piece(xp, p0 + at(u, wv, fq), np);
      f[u] = load_piece(fp, p0 + at(u, wv, fq), np);
    }
  }
  template <int ES>
  __device__ __forceinline__ f32x4 multiply(f32x4 acc) const {
#pragma unroll
    for (int u = 0; u < kShrinkU; ++u) acc = mma16<ES>(x[u], f[u], acc);
    return acc;
  }
};

// A workgroup per 16 rows and 16 ranks.  The rank blocks of a row tile run
// next to each other on one XCD (workgroups are dealt to the 8 XCDs in turn),
// so x comes from HBM once.
template <int ES>
__global__ __launch_bounds__(kShrinkWaves *kWave, 4) void shrink_tile_kernel(
    const char *__restrict__ x, const char *__restrict__ F, const float *__restrict__ scale,
    const int32_t *__restrict__ adapter, int T, int K, int r, int n, float *__restrict__ v) {
  __shared__ float red[kShrinkWaves][16][17];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int fr = lane & 15, fq = lane >> 4;
  const int blocks = (r + 15) / 16, i8 = blockIdx.x / 8;
  const int t0 = ((i8 / blocks) * 8 + blockIdx.x % 8) * 16, j0 = (i8 % blocks) * 16;
  if (t0 >= T) return;
  const int np = K * ES / 16;
  // the tile's adapters, the same answer in every wave (rows past T repeat
  // the last one)
  int a_mine = adapter[min(t0 + fr, T - 1)];
  if (a_mine < 0 || a_mine >= n) a_mine = -1;
  unsigned todo = (unsigned)__ballot(a_mine >= 0) & 0xffffu;
  int kinds = 0;
  for (unsigned left = todo; left; ++kinds)
    left &= ~(unsigned)__ballot(a_mine == __builtin_amdgcn_readlane(a_mine, __builtin_ctz(left)));
  if (few_adapters(kinds, K * ES)) {
    if (tid < 256) {  // rows without an adapter
      const int row = tid >> 4, j = tid & 15;
      if (!((todo >> row) & 1) && t0 + row < T && j0 + j < r) v[(size_t)(t0 + row) * r + j0 + j] = 0.f;
    }
    const u32x4 *xp = reinterpret_cast<const u32x4 *>(x + (size_t)min(t0 + fr, T - 1) * K * ES);
    while (todo) {
      const int a = __builtin_amdgcn_readlane(a_mine, __builtin_ctz(todo));
      const unsigned same = (unsigned)__ballot(a_mine == a) & 0xffffu;
      todo &= ~same;
      // ranks behind r repeat the last one and are not stored
      const u32x4 *fp =
          reinterpret_cast<const u32x4 *>(F + ((size_t)a * r + min(j0 + fr, r - 1)) * K * ES);
      f32x4 acc = f32x4{};
      int p0 = 0;
      for (; p0 + kShrinkChunk <= np; p0 += kShrinkChunk) {
        ShrinkPieces c;
        c.load(xp, fp, p0, wv, fq);
        __builtin_amdgcn_sched_barrier(0);  // every load is issued first
        acc = c.multiply<ES>(acc);
      }
      if (p0 < np) {
        ShrinkPieces c;
        c.load_tail(xp, fp, p0, np, wv, fq);
        __builtin_amdgcn_sched_barrier(0);
        acc = c.multiply<ES>(acc);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wv][4 * fq + i][fr] = acc[i];
      __syncthreads();
      if (tid < 256) {
        const int row = tid >> 4, j = tid & 15;
        float sum = red[0][row][j];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; ++w) sum += red[w][row][j];
        if (((same >> row) & 1) && t0 + row < T && j0 + j < r)
          v[(size_t)(t0 + row) * r + j0 + j] = scale[a] * sum;
      }
      __syncthreads();
    }
    return;
  }
  // rows of many adapters: a row per wave at a time, eight ranks of it
  for (int t = t0 + wv; t < min(t0 + 16, T); t += kShrinkWaves) {
    const int a = adapter[t];
    const bool none = a < 0 || a >= n;
    const u32x4 *xp = reinterpret_cast<const u32x4 *>(x + (size_t)t * K * ES);
    for (int j = j0; j < min(j0 + 16, r); j += 8) {
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      if (!none) {
        const u32x4 *fp = reinterpret_cast<const u32x4 *>(F + ((size_t)a * r + j) * K * ES);
        constexpr int U = 1;
        for (int p0 = lane; p0 < np; p0 += U * kWave) {
          u32x4 xa[U], fa[U][8];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            xa[u] = load_piece(xp, p0 + u * kWave, np);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              fa[u][i] = load_piece(fp + (size_t)i * np, p0 + u * kWave, np);
          }
          __builtin_amdgcn_sched_barrier(0);  // every load is issued first
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = dot_piece<ES>(xa[u], fa[u][i], acc[i]);
        }
      }
      const float s = sum8(acc, lane);
      const int which = 4 * (lane & 1) + (lane & 2) + ((lane >> 2) & 1);
      if (lane < 8) v[(size_t)t * r + j + which] = none ? 0.f : scale[a] * s;
    }
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
  hipLaunchKernelGGL((shrink_tile_kernel<ES>), dim3(((T + 15) / 16 + 7) / 8 * 8 * ((r + 15) / 16)),
                     dim3(kShrinkWaves * kWave), 0, s, xb, fb, scale, adapter, T, K, r, n, v);
}

}  // namespace

hipError_t launch_lora_shrink(const void *x, const void *F, int dt, const float *scale,
                              const int32_t *adapter, int T, int K, int r, int n, float *v,
                              hipStream_t s) {
  if (dt == MOE_BF16) launch_t<2>(x, F, scale, adapter, T, K, r, n, v, s);
  else launch_t<4>(x, F, scale, adapter, T, K, r, n, v, s);
  return hipGetLastError();
}
