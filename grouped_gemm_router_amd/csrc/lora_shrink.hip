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
//   * many rows, sorted by adapter (the plan): a workgroup takes up to 64 rows
//     of one adapter, up to 64 ranks and a slice of K.  What bounds this is
//     the rate at which a CU takes in operands (some 20 bytes a ns from beyond
//     its L1, measured): 64 rows share each factor load, and K is cut so that
//     every CU has its share; a second launch adds the slices in order.
//
// Measured: one row of 4096, rank 16, 3.4 us; 128 rows on 64 adapters 5.6 us;
// through the plan, 1331 rows of 7168, rank 64, 12.6 + 4.8 us (16 rows and 16
// ranks a wave instead: 29), 4096 rows of 7168, rank 8, 14 us and more (x is
// 59 MB from HBM) + 4.8.
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

// grid T r / 4: four waves, one (row, rank) each
template <int ES>
__global__ __launch_bounds__(256) void shrink_row_kernel(
    const char *__restrict__ x, const char *__restrict__ F, const float *__restrict__ scale,
    const int32_t *__restrict__ adapter, int K, int r, int n, float *__restrict__ v) {
  const int t = blockIdx.x / (r / 4), j = blockIdx.x % (r / 4) * 4 + threadIdx.x / kWave;
  const int lane = lane_id();
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
      xa[u] = load_piece(xp, p0 + u * kWave, np);
      fa[u] = load_piece(fp, p0 + u * kWave, np);
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

constexpr int kTileWaves = 4, kTileThreads = kTileWaves * kWave, kTileBlocks = kShrinkTile / 16;

// One wave's share of a tile's sums over the pieces [p0, p_end): RB blocks of
// 16 rows times NR blocks of 16 ranks, to red[row][rank].
template <int ES, int RB, int NR>
__device__ __forceinline__ void shrink_slice(const char *x, const char *F, const int *s_row, int K,
                                             int r, int a, int j0, int p0, int p_end, int wv,
                                             float (*red)[NR * 16 + 1]) {
  const int lane = lane_id(), fr = lane & 15, fq = lane >> 4;
  const u32x4 *xp[RB], *fp[NR];
#pragma unroll
  for (int b = 0; b < RB; ++b)
    xp[b] = reinterpret_cast<const u32x4 *>(x + (size_t)s_row[b * 16 + fr] * K * ES);
#pragma unroll
  for (int q = 0; q < NR; ++q)  // ranks behind r repeat the last one and are not stored
    fp[q] = reinterpret_cast<const u32x4 *>(F + ((size_t)a * r + min(j0 + q * 16 + fr, r - 1)) * K * ES);
  f32x4 acc[RB][NR];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int q = 0; q < NR; ++q) acc[b][q] = f32x4{};
  // a wave takes U / 2 lines of every row at a time
  constexpr int U = NR == 1 ? 4 : 2, CHUNK = U * kTileWaves * 4;
  auto at = [&](int p, int u) {
    return p + (2 * wv + (u & 1) + (u >> 1) * 2 * kTileWaves) * 4 + fq;
  };
  auto multiply = [&](const u32x4(&xa)[U][RB], const u32x4(&fa)[U][NR]) {
    __builtin_amdgcn_sched_barrier(0);  // every load of the chunk is issued first
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int q = 0; q < NR; ++q) acc[b][q] = mma16<ES>(xa[u][b], fa[u][q], acc[b][q]);
  };
  for (; p0 + CHUNK <= p_end; p0 += CHUNK) {
    u32x4 xa[U][RB], fa[U][NR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int b = 0; b < RB; ++b) xa[u][b] = xp[b][at(p0, u)];
#pragma unroll
      for (int q = 0; q < NR; ++q) fa[u][q] = fp[q][at(p0, u)];
    }
    multiply(xa, fa);
  }
  if (p0 < p_end) {  // zeros behind the slice's end
    u32x4 xa[U][RB], fa[U][NR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int b = 0; b < RB; ++b) xa[u][b] = load_piece(xp[b], at(p0, u), p_end);
#pragma unroll
      for (int q = 0; q < NR; ++q) fa[u][q] = load_piece(fp[q], at(p0, u), p_end);
    }
    multiply(xa, fa);
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[b * 16 + 4 * fq + i][q * 16 + fr] = acc[b][q][i];
}

// A tile's adapter (n: none, n + 1: no such tile), first place in the order and
// number of rows.  tiles[a]: the adapters' first tiles (tiles[n]: of the rows
// without an adapter, tiles[n + 1]: all); starts[a]: their first rows in the
// order.  The adapter a with tiles[a] <= tile < tiles[a + 1] is found 64 probes at a time.
// Must be called by whole waves.
struct TileRows {
  int a, first, rows;
};
__device__ __forceinline__ TileRows tile_rows(const int32_t *starts, const int32_t *tiles, int n,
                                              int tile) {
  int lo = 0, cnt = n + 1;
  while (cnt > 0) {
    const int step = (cnt + kWave - 1) / kWave;
    const int i = lo + min(((int)lane_id() + 1) * step, cnt) - 1;
    const unsigned long long behind = __ballot(tiles[i + 1] > tile);
    if (behind == 0) {
      lo += cnt;
      break;
    }
    const int f = __builtin_ctzll(behind), hit = lo + min((f + 1) * step, cnt) - 1;
    lo += f * step;
    cnt = hit - lo;
  }
  if (lo > n) return {lo, 0, 0};
  const int first = starts[lo] + (tile - tiles[lo]) * kShrinkTile;
  return {lo, first, min(starts[lo + 1] - first, kShrinkTile)};
}

// grid (tiles times K slices, rank groups of 16 NR)
template <int ES, int NR>
__global__ __launch_bounds__(kTileThreads) void shrink_tile_kernel(
    const char *__restrict__ x, const char *__restrict__ F, const float *__restrict__ scale,
    const int32_t *__restrict__ order, const int32_t *__restrict__ starts,
    const int32_t *__restrict__ tiles, int T, int slices, int K, int r, int n,
    float *__restrict__ part, float *__restrict__ v) {
  constexpr int RP = NR * 16;
  __shared__ float red[kTileWaves][kShrinkTile][RP + 1];
  __shared__ int s_row[kShrinkTile];
  const int tid = threadIdx.x, wv = tid / kWave;
  const int tile = blockIdx.x / slices, ks = blockIdx.x % slices, j0 = blockIdx.y * RP;
  const TileRows tr = tile_rows(starts, tiles, n, tile);
  const int a = tr.a, rows = tr.rows;
  if (a > n) return;
  if (a == n) {  // rows without an adapter
    if (ks == 0)
      for (int i = tid; i < rows * RP; i += kTileThreads) {
        const int j = j0 + i % RP;
        if (j < r) v[(size_t)order[tr.first + i / RP] * r + j] = 0.f;
      }
    return;
  }
  if (tid < kShrinkTile) s_row[tid] = order[tr.first + min(tid, rows - 1)];
  __syncthreads();
  const int np = K * ES / 16;
  // this slice's pieces: whole lines of 8, the same number for every slice
  const int per = ((np + 7) / 8 + slices - 1) / slices * 8;
  const int p_end = min(np, (ks + 1) * per);
  const int live = (rows + 15) / 16;  // row blocks
  const int p0 = ks * per;
  if (live <= 1) shrink_slice<ES, 1, NR>(x, F, s_row, K, r, a, j0, p0, p_end, wv, red[wv]);
  else if (live <= 2) shrink_slice<ES, 2, NR>(x, F, s_row, K, r, a, j0, p0, p_end, wv, red[wv]);
  else shrink_slice<ES, kTileBlocks, NR>(x, F, s_row, K, r, a, j0, p0, p_end, wv, red[wv]);
  __syncthreads();
  float *mine = part + (((size_t)blockIdx.y * slices + ks) * T + tr.first) * RP;
  for (int i = tid; i < rows * RP; i += kTileThreads) {
    const int row = i / RP, j = i % RP;
    float sum = red[0][row][j];
#pragma unroll
    for (int w = 1; w < kTileWaves; ++w) sum += red[w][row][j];
    if (slices > 1)
      mine[i] = sum;
    else if (j0 + j < r)
      v[(size_t)s_row[row] * r + j0 + j] = scale[a] * sum;
  }
}

// The slices of the sums added in slice order, four ranks of a row a thread.
// A launch of its own: a flag between workgroups of the same launch needs
// their XCDs' L2 written back, which took five times as long as the products.
// grid (pieces of T RP, rank groups).  Rows without an adapter have their
// zeros already.
__global__ __launch_bounds__(256) void shrink_sum_kernel(
    const float *__restrict__ part, const float *__restrict__ scale,
    const int32_t *__restrict__ adapter, const int32_t *__restrict__ order, int T, int slices, int RP,
    int r, int n, float *__restrict__ v) {
  const int i = blockIdx.x * 256 + threadIdx.x, row = i / (RP / 4), jr = i % (RP / 4) * 4,
            j = blockIdx.y * RP + jr;
  if (row >= T || j >= r) return;
  const float *const all = part + ((size_t)blockIdx.y * slices * T + row) * RP + jr;
  f32x4 p[kShrinkSlices];
#pragma unroll
  for (int k = 0; k < kShrinkSlices; ++k)
    p[k] = *reinterpret_cast<const f32x4 *>(all + (size_t)min(k, slices - 1) * T * RP);
  const int t = order[row], a = adapter[t];
  if (a < 0 || a >= n) return;
  f32x4 sum = p[0];
#pragma unroll
  for (int k = 1; k < kShrinkSlices; ++k)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[c] += k < slices ? p[k][c] : 0.f;
  *reinterpret_cast<f32x4 *>(v + (size_t)t * r + j) = scale[a] * sum;
}

template <int ES>
void launch_t(const void *x, const void *F, const float *scale, const int32_t *adapter,
              const LoraPlan *p, char *ws, int T, int K, int r, int n, float *v, hipStream_t s) {
  const char *xb = static_cast<const char *>(x), *fb = static_cast<const char *>(F);
  if (!p) {
    hipLaunchKernelGGL((shrink_row_kernel<ES>), dim3((unsigned)T * (r / 4)), dim3(256), 0, s, xb, fb,
                       scale, adapter, K, r, n, v);
    return;
  }
  const int NR = r <= 16 ? 1 : r <= 32 ? 2 : 4, groups = (r + 16 * NR - 1) / (16 * NR);
  const int slices = lora_shrink_slices(T, K * ES, r);
  const dim3 grid((unsigned)p->max_tiles * slices, groups), block(kTileThreads);
  const int32_t *order = reinterpret_cast<const int32_t *>(ws + p->order);
  const int32_t *starts = reinterpret_cast<const int32_t *>(ws + p->starts);
  const int32_t *tiles = reinterpret_cast<const int32_t *>(ws + p->tiles);
  float *part = reinterpret_cast<float *>(ws + p->part);
#define MOE_SHRINK(NR)                                                                          \
  hipLaunchKernelGGL((shrink_tile_kernel<ES, NR>), grid, block, 0, s, xb, fb, scale, order, starts, \
                     tiles, T, slices, K, r, n, part, v)
  if (NR == 1) MOE_SHRINK(1);
  else if (NR == 2) MOE_SHRINK(2);
  else MOE_SHRINK(4);
#undef MOE_SHRINK
  if (slices > 1)
    hipLaunchKernelGGL(shrink_sum_kernel, dim3((unsigned)(((size_t)T * 4 * NR + 255) / 256), groups),
                       dim3(256), 0, s, part, scale, adapter, order, T, slices, 16 * NR, r, n, v);
}

}  // namespace

hipError_t launch_lora_shrink(const void *x, const void *F, int dt, const float *scale,
                              const int32_t *adapter, const LoraPlan *p, char *ws, int T, int K,
                              int r, int n, float *v, hipStream_t s) {
  if (dt == MOE_BF16) launch_t<2>(x, F, scale, adapter, p, ws, T, K, r, n, v, s);
  else launch_t<4>(x, F, scale, adapter, p, ws, T, K, r, n, v, s);
  return hipGetLastError();
}
