// lora_expand.hip -- y[t] = W x[t] + sum_j v[t][j] F[a][j], a = adapter[t]:
// the shared projection and, in its epilogue, each row's low-rank part.
//
// The low-rank vector v (fp32, r values a row) is ready when this launch
// starts.  Fusing its product with F into the projection writes y once, with
// one rounding, where a second pass would read and write it again.
//
// The low-rank part of a 32-row block that belongs to one adapter (a prompt's
// rows) goes through the matrix cores: v is split into bf16 terms (two for
// a bf16 y, three for an fp32 y, so that the product keeps 16 or 24 bits of
// v) and multiplied like 16 more columns of x.  In any other block every row
// reads its own adapter's rows of F on the vector ALUs.  No row ever meets
// another adapter's values, not even multiplied by zero: an infinity in one
// request's adapter stays in that request's rows.
#include "lora_internal.h"

namespace {

using namespace moe;

__device__ __forceinline__ int swz(int row, int p) { return p ^ ((row >> 1) & 7); }

// element i of a factor or of y as fp32
template <int ES>
__device__ __forceinline__ float ld1(const char *p, size_t i) {
  if constexpr (ES == 2) return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
  else return reinterpret_cast<const float *>(p)[i];
}

// eight consecutive elements; vec: the address is 16-byte aligned and all
// eight exist, else the first `have` exist
template <int ES>
__device__ __forceinline__ void ld8(const char *p, size_t i, bool vec, int have, float (&f)[8]) {
  if (vec) {
    if constexpr (ES == 2) {
      const u32x4 q = *reinterpret_cast<const u32x4 *>(p + i * 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[2 * c] = bf16_bits_to_f32(q[c] & 0xffffu);
        f[2 * c + 1] = __uint_as_float(q[c] & 0xffff0000u);
      }
    } else {
      const f32x4 q0 = *reinterpret_cast<const f32x4 *>(p + i * 4);
      const f32x4 q1 = *reinterpret_cast<const f32x4 *>(p + i * 4 + 16);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[c] = q0[c];
        f[4 + c] = q1[c];
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = c < have ? ld1<ES>(p, i + c) : 0.f;
  }
}

template <int OS>
__device__ __forceinline__ void st8(char *p, size_t i, bool vec, int have, const float (&f)[8]) {
  if (vec) {
    if constexpr (OS == 2) {
      bf16x8 q;
#pragma unroll
      for (int c = 0; c < 8; ++c) q[c] = (__bf16)f[c];  // round to nearest even
      *reinterpret_cast<bf16x8 *>(p + i * 2) = q;
    } else {
      *reinterpret_cast<f32x4 *>(p + i * 4) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4 *>(p + i * 4 + 16) = f32x4{f[4], f[5], f[6], f[7]};
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= have) break;
      if constexpr (OS == 2) reinterpret_cast<__bf16 *>(p)[i + c] = (__bf16)f[c];
      else reinterpret_cast<float *>(p)[i + c] = f[c];
    }
  }
}

// f[0..7] += sum_j vr[j] F[j][n .. n + 7] for one row's adapter
template <int ES>
__device__ __forceinline__ void add_low_rank(float (&f)[8], const float *vr, const char *F, int r,
                                             int N, int n, bool vec, int have) {
  for (int j0 = 0; j0 < r; j0 += 8) {
    float w[8][8];
    const f32x4 v0 = *reinterpret_cast<const f32x4 *>(vr + j0);
    const f32x4 v1 = *reinterpret_cast<const f32x4 *>(vr + j0 + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) ld8<ES>(F, (size_t)(j0 + j) * N + n, vec, have, w[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = fmaf(j < 4 ? v0[j & 3] : v1[j & 3], w[j][c], f[c]);
  }
}

// acc[nb] += v F over one 32-row block that belongs to adapter a: 16 ranks a
// step.  t: the lane's row, n[nb]: its columns.
template <int TERMS, int NB>
__device__ __forceinline__ void mma_low_rank(f32x16 (&acc)[NB], const float *v, const char *F, int r,
                                             int N, size_t t, const int (&n)[NB], int fh) {
  for (int j0 = 0; j0 < r; j0 += 16) {
    const int j = j0 + 8 * fh;
    const bool in = j < r;  // r is a multiple of 8: a lane's eight ranks exist or not
    float f[8];
    const f32x4 v0 = in ? *reinterpret_cast<const f32x4 *>(v + t * r + j) : f32x4{};
    const f32x4 v1 = in ? *reinterpret_cast<const f32x4 *>(v + t * r + j + 4) : f32x4{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = v0[i];
      f[4 + i] = v1[i];
    }
    uint16_t w[NB][8];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[nb][i] = in ? reinterpret_cast<const uint16_t *>(F)[(size_t)(j + i) * N + n[nb]] : 0;
    bf16x8 va[TERMS];
    split_bf16<TERMS>(f, va);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      bf16x8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = __builtin_bit_cast(__bf16, w[nb][i]);
#pragma unroll
      for (int k = 0; k < TERMS; ++k)
        acc[nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[k], b, acc[nb], 0, 0, 0);
    }
  }
}

// tile of workgroup id: the axis with more tiles is dealt over the 8 XCDs
// (consecutive workgroups go to the XCDs in turn), each XCD walking the other
// axis inside: the operand tile that its workgroups share stays in its L2
struct TileAt {
  int mt, nt;
};
__device__ __forceinline__ TileAt tile_at(int id, int MT, int NT) {
  const int major = max(MT, NT), minor = min(MT, NT);
  const int i = id / 8, a = (i / minor) * 8 + id % 8, b = i % minor;
  if (a >= major) return {-1, -1};
  return MT > NT ? TileAt{a, b} : TileAt{b, a};
}
unsigned tile_grid(int MT, int NT) {
  const int major = MT > NT ? MT : NT, minor = MT > NT ? NT : MT;
  return (unsigned)((major + 7) / 8 * 8) * (unsigned)minor;
}

// ---------------------------------------------------------------------------
// tiles of BM x BN on 4 waves (WM x WN), operands through LDS 128 bytes of a
// row at a time: the next step's pieces are loaded into registers while this
// step is multiplied.  Pieces past K read as zero; rows past T and columns
// past N repeat the last one and are not stored.
// ---------------------------------------------------------------------------
template <int ES, int OS, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256) void expand_tile_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter, int T, int N, int K, int r,
    int n, char *__restrict__ y, int MT, int NT) {
  constexpr int MI = BM / WM / 32, NB = BN / WN / 32;
  constexpr int NLD = (BM + BN) * 8 / 256;
  constexpr int SP = BN + 4;  // row pitch of the staged fp32 tile
  constexpr int RING = 2 * (BM + BN) * 128, STAGE = BM * SP * 4;
  static_assert(WM * WN == 4 && MI >= 1 && NB >= 1, "four waves of 32 x 32 blocks");
  __shared__ __align__(16) char smem[RING > STAGE ? RING : STAGE];
  __shared__ int s_ad[BM];
  __shared__ int s_hom[BM / 32];
  const TileAt at = tile_at(blockIdx.x, MT, NT);
  if (at.mt < 0) return;
  const int m0 = at.mt * BM, n0 = at.nt * BN;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int wm = wv / WN, wn = wv % WN, fr = lane & 31, fh = lane >> 5;

  if (tid < BM) {
    const int a = adapter[min(m0 + tid, T - 1)];
    s_ad[tid] = a >= 0 && a < n ? a : -1;
  }
  f32x16 acc[MI][NB];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};

  if (W) {
    const int KP = K * ES / 16, KT = (KP + 7) / 8;
    const u32x4 *src[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int row = (tid + 256 * i) >> 3;
      src[i] = row < BM
                   ? reinterpret_cast<const u32x4 *>(x + (size_t)min(m0 + row, T - 1) * K * ES)
                   : reinterpret_cast<const u32x4 *>(W + (size_t)min(n0 + row - BM, N - 1) * ldw * ES);
    }
    u32x4 reg[NLD];
    auto fetch = [&](int kt) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int p = kt * 8 + (tid & 7);
        reg[i] = p < KP ? src[i][p] : u32x4{};
      }
    };
    auto put = [&](int b) {
      u32x4 *l = reinterpret_cast<u32x4 *>(smem) + b * (BM + BN) * 8;
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int row = (tid + 256 * i) >> 3;
        l[row * 8 + swz(row, tid & 7)] = reg[i];
      }
    };
    fetch(0);
    put(0);
    __syncthreads();
    for (int kt = 0; kt < KT; ++kt) {
      if (kt + 1 < KT) fetch(kt + 1);
      const u32x4 *l = reinterpret_cast<const u32x4 *>(smem) + (kt & 1) * (BM + BN) * 8;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        u32x4 a[MI], b[NB];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const int row = wm * (MI * 32) + i * 32 + fr;
          a[i] = l[row * 8 + swz(row, 2 * ks + fh)];
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int row = BM + wn * (NB * 32) + j * 32 + fr;
          b[j] = l[row * 8 + swz(row, 2 * ks + fh)];
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            if constexpr (ES == 2) {
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(bf16x8, a[i]), __builtin_bit_cast(bf16x8, b[j]), acc[i][j], 0,
                  0, 0);
            } else {
              // component c of the two halves' pieces: k = 8 ks + 4 fh + c
              const f32x4 fa = __builtin_bit_cast(f32x4, a[i]), fb = __builtin_bit_cast(f32x4, b[j]);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[c], fb[c], acc[i][j], 0, 0, 0);
            }
          }
      }
      if (kt + 1 < KT) put((kt + 1) & 1);
      __syncthreads();
    }
  } else {
    __syncthreads();  // s_ad
  }

#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = wm * (MI * 32) + i * 32 + fr;
    const int a = s_ad[row], a0 = __builtin_amdgcn_readfirstlane(a);
    const bool hom = ES == 2 && a0 >= 0 && __all(a == a0);
    if (lane == 0 && wn == 0) s_hom[wm * MI + i] = hom;
    if constexpr (ES == 2) {
      if (hom) {
        int nn[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) nn[j] = min(n0 + wn * (NB * 32) + j * 32 + fr, N - 1);
        mma_low_rank<OS == 2 ? 2 : 3, NB>(acc[i], v, F + (size_t)a0 * r * N * ES, r, N,
                                          (size_t)min(m0 + row, T - 1), nn, fh);
      }
    }
  }
  // the tile meets in LDS in fp32 (the ring is free after the last barrier),
  // then every thread finishes whole 8-column pieces of rows
  float *stage = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        stage[(wm * (MI * 32) + i * 32 + 8 * (e >> 2) + 4 * fh + (e & 3)) * SP + wn * (NB * 32) +
              j * 32 + fr] = acc[i][j][e];
  __syncthreads();
  const bool vec = N % 8 == 0;  // rows of F and of y are then 16-byte aligned
  constexpr int CG = BN / 8;
  for (int q = tid; q < BM * CG; q += 256) {
    const int row = q / CG, c = (q % CG) * 8, t = m0 + row, col = n0 + c;
    if (t >= T || col >= N) continue;
    const int have = N - col;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = stage[row * SP + c + i];
    const int a = s_ad[row];
    if (a >= 0 && !s_hom[row / 32])
      add_low_rank<ES>(f, v + (size_t)t * r, F + (size_t)a * r * N * ES, r, N, col, vec, have);
    if (!W) {
      float old[8];
      ld8<OS>(y, (size_t)t * N + col, vec, have, old);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += old[i];
    }
    st8<OS>(y, (size_t)t * N + col, vec, have, f);
  }
}

// ---------------------------------------------------------------------------
// few rows (bf16): 16 columns per workgroup, MB blocks of 16 rows, eight
// waves cutting K.  W is read once, by the whole chip at once, straight into
// the matrix cores' fragments; x comes from L2.
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;

template <int OS, int MB>
__global__ __launch_bounds__(kRowWaves *kWave) void expand_rows_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter, int T, int N, int K, int r,
    int n, char *__restrict__ y) {
  __shared__ float red[kRowWaves][MB * 16][17];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int fr = lane & 15, fq = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int KP = K / 8;
  const u32x4 *wp = reinterpret_cast<const u32x4 *>(W + (size_t)min(n0 + fr, N - 1) * ldw * 2);
  const u32x4 *xp[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b)
    xp[b] = reinterpret_cast<const u32x4 *>(x + (size_t)min(b * 16 + fr, T - 1) * K * 2);
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4{};
  // a wave takes two neighbouring groups of 4 pieces (whole 128-byte lines)
  // out of each 16
  constexpr int U = MB <= 2 ? 8 : 4;
  for (int g0 = 2 * wv; g0 * 4 < KP; g0 += U * kRowWaves) {
    u32x4 wa[U], xa[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = (g0 + (u & 1) + (u >> 1) * 2 * kRowWaves) * 4 + fq;
      wa[u] = p < KP ? wp[p] : u32x4{};
#pragma unroll
      for (int b = 0; b < MB; ++b) xa[u][b] = p < KP ? xp[b][p] : u32x4{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa[u][b]),
                                                         __builtin_bit_cast(bf16x8, wa[u]), acc[b],
                                                         0, 0, 0);
  }
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wv][b * 16 + 4 * fq + i][fr] = acc[b][i];
  __syncthreads();
  for (int q = tid; q < MB * 256; q += kRowWaves * kWave) {
    const int t = q >> 4, c = q & 15, col = n0 + c;
    if (t >= T || col >= N) continue;
    float f = red[0][t][c];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) f += red[w][t][c];
    const int a = adapter[t];
    if (a >= 0 && a < n) {
      const char *Fa = F + (size_t)a * r * N * 2;
      for (int j0 = 0; j0 < r; j0 += 8) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = ld1<2>(Fa, (size_t)(j0 + j) * N + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) f = fmaf(v[(size_t)t * r + j0 + j], w[j], f);
      }
    }
    if constexpr (OS == 2) reinterpret_cast<__bf16 *>(y)[(size_t)t * N + col] = (__bf16)f;
    else reinterpret_cast<float *>(y)[(size_t)t * N + col] = f;
  }
}

// rows up to which expand_rows_kernel runs (bf16 with a W)
constexpr int kExpandRowsMax = 64;

struct Shape {
  int BM, BN;
};

// The tile shape whose rounds over the CUs cost least: a K step of 128 bytes
// takes the larger of its matrix-core time and its L2 time.
Shape pick_tile(int T, int N, int cus, bool f32) {
  const Shape all[] = {{128, 128}, {128, 64}, {64, 64}, {32, 128}};
  Shape best = all[0];
  double least = 1e300;
  for (const Shape &s : all) {
    const double tiles = (double)((T + s.BM - 1) / s.BM) * ((N + s.BN - 1) / s.BN);
    const double rounds = tiles <= cus ? 1.0 : tiles / cus > 4 ? tiles / cus : (double)((long long)(tiles + cus - 1) / cus);
    const double mma = s.BM * s.BN / (f32 ? 4.0 : 20.0), l2 = (s.BM + s.BN) * 2.7;
    const double cost = rounds * (mma > l2 ? mma : l2);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

template <int ES, int OS, int BM, int BN, int WM, int WN>
void launch_tile(const char *x, const char *W, int ldw, const char *F, const float *v,
                 const int32_t *adapter, int T, int N, int K, int r, int n, char *y, hipStream_t s) {
  const int MT = (T + BM - 1) / BM, NT = (N + BN - 1) / BN;
  hipLaunchKernelGGL((expand_tile_kernel<ES, OS, BM, BN, WM, WN>), dim3(tile_grid(MT, NT)), dim3(256),
                     0, s, x, W, ldw, F, v, adapter, T, N, K, r, n, y, MT, NT);
}

template <int ES, int OS>
void launch_t(const char *x, const char *W, int ldw, const char *F, const float *v,
              const int32_t *adapter, int T, int N, int K, int r, int n, char *y, int cus,
              hipStream_t s) {
  if constexpr (ES == 2) {
    if (W && T <= kExpandRowsMax) {
      const dim3 grid((N + 15) / 16), block(kRowWaves * kWave);
#define MOE_ROWS(MB)                                                                             \
  hipLaunchKernelGGL((expand_rows_kernel<OS, MB>), grid, block, 0, s, x, W, ldw, F, v, adapter, T, \
                     N, K, r, n, y)
      if (T <= 16) MOE_ROWS(1);
      else if (T <= 32) MOE_ROWS(2);
      else MOE_ROWS(4);
#undef MOE_ROWS
      return;
    }
  }
  const Shape p = pick_tile(T, N, cus, ES == 4);
#define MOE_TILE(BM, BN, WM, WN) \
  launch_tile<ES, OS, BM, BN, WM, WN>(x, W, ldw, F, v, adapter, T, N, K, r, n, y, s)
  if (p.BM == 128 && p.BN == 128) MOE_TILE(128, 128, 2, 2);
  else if (p.BM == 128) MOE_TILE(128, 64, 2, 2);
  else if (p.BM == 64) MOE_TILE(64, 64, 2, 2);
  else MOE_TILE(32, 128, 1, 4);
#undef MOE_TILE
}

}  // namespace

hipError_t launch_lora_expand(const void *x, const void *W, int ldw, const void *F, int dt,
                              const float *v, const int32_t *adapter, int T, int N, int K, int r,
                              int n, void *y, int y_dt, int cus, hipStream_t s) {
  const char *xb = static_cast<const char *>(x), *wb = static_cast<const char *>(W),
             *fb = static_cast<const char *>(F);
  char *yb = static_cast<char *>(y);
  if (dt == MOE_F32) launch_t<4, 4>(xb, wb, ldw, fb, v, adapter, T, N, K, r, n, yb, cus, s);
  else if (y_dt == MOE_F32) launch_t<2, 4>(xb, wb, ldw, fb, v, adapter, T, N, K, r, n, yb, cus, s);
  else launch_t<2, 2>(xb, wb, ldw, fb, v, adapter, T, N, K, r, n, yb, cus, s);
  return hipGetLastError();
}
