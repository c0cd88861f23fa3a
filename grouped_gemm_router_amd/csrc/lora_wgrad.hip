// lora_wgrad.hip -- the adapters' gradients: for every adapter a,
//   dA[a][j] = sum over its rows t of u[t][j] x[t],
//   dB[a][j] = sum over its rows t of v[t][j] dy[t].
//
// The rows are read in the plan's order, adapter by adapter, and each
// adapter's rows are cut into units of at most TS.  A workgroup takes a unit,
// 128 columns and 16 or 32 ranks, and its four waves take 32 rows in turn (a
// short unit's take 128 columns each).  The sum runs over rows, so a lane loads
// 16 bytes (8 columns) of 8 rows and turns that 8 x 8 block in registers into
// eight matrix-core fragments; x and dy are read once, in whole lines, which
// is what bounds this (2 r flops per 2 bytes).  u and v are fp32 and enter as
// three bf16 terms each, so no bit of them is lost.  A unit that is all of
// its adapter writes the gradient itself; the slices of a longer one go to
// the workspace and a second launch adds them in order.  Measured: 4096 rows,
// 8192 columns (67 MB), 8 adapters of rank 16: 18 to 20 us + 4.8.
#include "lora_internal.h"

namespace {

using namespace moe;

constexpr int kColTile = 128;
// Rows of a unit up to which a workgroup's waves take 128 columns each and all
// of the unit's rows, instead of 128 columns together and 32 rows in turn: most
// of the waves would have none (777 rows of 33 adapters of rank 32, 9216
// columns: 23.2 us, so 15.6).
constexpr int kShortUnit = 64;

// the slices behind the plan: an adapter of c > TS rows has fewer than
// 2 c / TS units
size_t slices_bytes(const LoraPlan &p, int T, int N, int K, int r) {
  const size_t slots = T <= p.TS ? 0 : 2 * (size_t)T / p.TS + 1;
  return slots * r * ((size_t)K + N) * 4;
}

// grid (units, column tiles of x then of dy, rank groups of 16 NR)
template <int ES, int NR>
__global__ __launch_bounds__(256) void wgrad_kernel(
    const char *__restrict__ x, const char *__restrict__ dy, const float *__restrict__ u,
    const float *__restrict__ v, const int32_t *__restrict__ order, const LoraUnit *__restrict__ units,
    const int32_t *__restrict__ n_units, int N, int K, int r, float *__restrict__ dA,
    float *__restrict__ dB, float *__restrict__ part) {
  __shared__ float red[4][16][kColTile + 4];
  if ((int)blockIdx.x >= *n_units) return;
  const LoraUnit un = units[blockIdx.x];
  const int ka = (K + kColTile - 1) / kColTile;
  const bool is_a = (int)blockIdx.y < ka, cut = un.count > kShortUnit;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int ct = is_a ? blockIdx.y : blockIdx.y - ka;
  if (!cut && ct % 4 != 0) return;
  const int C = is_a ? K : N, c0 = (cut ? ct : ct + wv) * kColTile;
  if (!cut && c0 >= C) return;
  const int j0 = blockIdx.z * 16 * NR;
  const char *q = is_a ? x : dy;
  const float *p = is_a ? u : v;
  const int fr = lane & 15, fq = lane >> 4;
  const int col = min(c0 + 8 * fr, C - 8);  // C is a multiple of 8
  f32x4 acc[NR][8];
#pragma unroll
  for (int b = 0; b < NR; ++b)
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[b][f] = f32x4{};

  for (int s = cut ? wv * 32 : 0; s < un.count; s += cut ? 4 * 32 : 32) {
    // rows past the unit's end load the last one and count as zero in both
    // operands (no load is under a condition: the loads are in flight
    // together); columns past C and ranks past r load the last ones and are
    // not stored
    size_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = order[un.pos + min(s + fq * 8 + i, un.count - 1)];
    u32x4 qv[8][ES / 2];
    float pv[NR][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int h = 0; h < ES / 2; ++h)
        qv[i][h] = *reinterpret_cast<const u32x4 *>(q + (t[i] * C + col) * ES + 16 * h);
#pragma unroll
      for (int b = 0; b < NR; ++b) pv[b][i] = p[t[i] * r + min(j0 + b * 16 + fr, r - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = s + fq * 8 + i < un.count;
#pragma unroll
      for (int h = 0; h < ES / 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) qv[i][h][c] = in ? qv[i][h][c] : 0u;
#pragma unroll
      for (int b = 0; b < NR; ++b) pv[b][i] = in ? pv[b][i] : 0.f;
    }
    if constexpr (ES == 2) {
      bf16x8 pt[NR][3];
#pragma unroll
      for (int b = 0; b < NR; ++b) split_bf16<3>(pv[b], pt[b]);
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        // column f of the lane's 8 x 8 block: row pairs into words
        const unsigned sel = (f & 1) ? 0x07060302u : 0x05040100u;
        u32x4 w;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          w[d] = __builtin_amdgcn_perm(qv[2 * d + 1][0][f >> 1], qv[2 * d][0][f >> 1], sel);
        const bf16x8 qf = __builtin_bit_cast(bf16x8, w);
#pragma unroll
        for (int b = 0; b < NR; ++b)
#pragma unroll
          for (int k = 0; k < 3; ++k)
            acc[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pt[b][k], qf, acc[b][f], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int f = 0; f < 8; ++f)
#pragma unroll
          for (int b = 0; b < NR; ++b)
            acc[b][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                pv[b][i], __uint_as_float(qv[i][f >> 2 & (ES / 2 - 1)][f & 3]), acc[b][f], 0, 0, 0);
    }
  }
  const int width = un.slot < 0 ? C : K + N;
  float *out = un.slot < 0 ? (is_a ? dA : dB) + (size_t)un.adapter * r * C + c0
                           : part + (size_t)un.slot * r * width + (is_a ? c0 : K + c0);
  if (!cut) {
#pragma unroll
    for (int b = 0; b < NR; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + b * 16 + 4 * fq + i;
        if (j >= r || c0 + 8 * fr >= C) continue;
        f32x4 *const to = reinterpret_cast<f32x4 *>(out + (size_t)j * width + 8 * fr);
        to[0] = f32x4{acc[b][0][i], acc[b][1][i], acc[b][2][i], acc[b][3][i]};
        to[1] = f32x4{acc[b][4][i], acc[b][5][i], acc[b][6][i], acc[b][7][i]};
      }
    return;
  }
  // the four waves' sums, in wave order
#pragma unroll
  for (int b = 0; b < NR; ++b) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int f = 0; f < 8; ++f) red[wv][4 * fq + i][8 * fr + f] = acc[b][f][i];
    __syncthreads();
    for (int e = tid; e < 16 * kColTile / 4; e += 256) {
      const int jr = e / (kColTile / 4), c = (e % (kColTile / 4)) * 4, j = j0 + b * 16 + jr;
      if (j >= r || c0 + c >= C) continue;
      f32x4 sum = *reinterpret_cast<const f32x4 *>(&red[0][jr][c]);
#pragma unroll
      for (int w = 1; w < 4; ++w) sum += *reinterpret_cast<const f32x4 *>(&red[w][jr][c]);
      *reinterpret_cast<f32x4 *>(out + (size_t)j * width + c) = sum;
    }
  }
}

// grid (pieces of r (K + N) / 4, adapters)
__global__ __launch_bounds__(256) void wgrad_reduce_kernel(const int2 *__restrict__ adapters,
                                                           const float *__restrict__ part, int N,
                                                           int K, int r, float *__restrict__ dA,
                                                           float *__restrict__ dB) {
  const int a = blockIdx.y;
  const int2 s = adapters[a];
  if (s.y <= 1) return;
  const int wide = (K + N) / 4;
  const long long q = (long long)blockIdx.x * 256 + threadIdx.x;
  if (q >= (long long)r * wide) return;
  const int j = (int)(q / wide), c = (int)(q - (long long)j * wide) * 4;
  f32x4 sum = f32x4{};
  const float *src = part + (size_t)s.x * r * (K + N) + (size_t)j * (K + N) + c;
  for (int i = 0; i < s.y; ++i)
    sum += *reinterpret_cast<const f32x4 *>(src + (size_t)i * r * (K + N));
  float *out = c < K ? dA + ((size_t)a * r + j) * K + c : dB + ((size_t)a * r + j) * N + (c - K);
  *reinterpret_cast<f32x4 *>(out) = sum;
}

template <int ES>
void launch_t(const void *dy, const void *x, const float *u, const float *v, const LoraPlan &p,
              char *ws, int N, int K, int r, float *dA, float *dB, hipStream_t s) {
  const int cols = (K + kColTile - 1) / kColTile + (N + kColTile - 1) / kColTile;
  const int32_t *order = reinterpret_cast<const int32_t *>(ws + p.order);
  const LoraUnit *units = reinterpret_cast<const LoraUnit *>(ws + p.units);
  const int32_t *nu = reinterpret_cast<const int32_t *>(ws + p.n_units);
  float *part = reinterpret_cast<float *>(ws + p.bytes);
  const char *xb = static_cast<const char *>(x), *db = static_cast<const char *>(dy);
  if (r <= 16)
    hipLaunchKernelGGL((wgrad_kernel<ES, 1>), dim3(p.max_units, cols, 1), dim3(256), 0, s, xb, db, u,
                       v, order, units, nu, N, K, r, dA, dB, part);
  else
    hipLaunchKernelGGL((wgrad_kernel<ES, 2>), dim3(p.max_units, cols, (r + 31) / 32), dim3(256), 0, s,
                       xb, db, u, v, order, units, nu, N, K, r, dA, dB, part);
}

}  // namespace

size_t lora_wgrad_ws_bytes(int T, int N, int K, int r, int n, int es) {
  const LoraPlan p = lora_plan(T, N, K, r, n, es, true);
  return p.bytes + slices_bytes(p, T, N, K, r);
}

hipError_t launch_lora_wgrad(const void *dy, const void *x, int dt, const float *u, const float *v,
                             int T, int N, int K, int r, int n, float *dA, float *dB, void *ws,
                             hipStream_t s) {
  const LoraPlan p = lora_plan(T, N, K, r, n, dt == MOE_BF16 ? 2 : 4, true);
  char *b = static_cast<char *>(ws);
  if (dt == MOE_BF16) launch_t<2>(dy, x, u, v, p, b, N, K, r, dA, dB, s);
  else launch_t<4>(dy, x, u, v, p, b, N, K, r, dA, dB, s);
  if (T <= p.TS) return hipGetLastError();
  const long long pieces = (long long)r * ((K + N) / 4);
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3((unsigned)((pieces + 255) / 256), n), dim3(256), 0, s,
                     reinterpret_cast<const int2 *>(b + p.adapters),
                     reinterpret_cast<const float *>(b + p.bytes), N, K, r, dA, dB);
  return hipGetLastError();
}
