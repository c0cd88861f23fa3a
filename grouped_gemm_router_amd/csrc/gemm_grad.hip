// gemm_grad.hip -- the gradients of the grouped products on bf16 MFMA.
//
//   dgrad  dA[r][k] = sum_n dC[r][n] B[g][n][k] (+ dC2 B2), r in group g,
//          with SwiGLU's gradient behind it or not
//   wgrad  dB[g][n][k] (+)= sum_{r in group g} dC[r][n] A[r][k]
//
// The forward product reads both operands along the sum (C = A B^T).  Here
// dgrad's weights and both of wgrad's operands lie across it: their rows are
// terms of the sum.  Such a tile goes to LDS as it lies in memory, whole
// 512-byte row pieces by LDS-direct loads, and is turned on the way to the
// registers by ds_read_b64_tr_b16, which hands each lane four terms of one
// column; no operand is transposed in memory.
#include "backward_internal.h"

namespace {

using namespace moe;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int BN = 256;              // output columns of a tile
constexpr int BK = 32;               // terms of the sum a stage
constexpr int NS = 5;                // stages in LDS
constexpr int NW = 4;                // waves, 2 x 2
constexpr int SLOT = 2 * BN * BK / 8; // 16-byte pieces a stage: both operands, 32 KB

// what loads behind the last term of a sum read
__device__ u32x4 g_zeros[1];

// An operand whose rows are terms: 32 rows of 256 columns (32 pieces of 16
// bytes).  The 64-byte blocks of a row are stored at block ^ (row & 3): the
// four rows that a transposing read takes then lie in different banks.
// fragment of 32 columns: terms 8 (lane / 32) .. + 7 of a 16-term step
struct CrossOperand {
  uint32_t at[4];  // byte offset of each of the wave's 32-column blocks
  __device__ __forceinline__ void init(int first_block, int lane) {
    const int kk = (lane % 16) / 4;
    const int row = 8 * (lane / 32) + kk;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      at[b] = row * 512 + ((first_block + b) ^ kk) * 64 + ((lane / 16) & 1) * 32 + (lane % 4) * 8;
  }
  __device__ __forceinline__ bf16x8 read(const u32x4 *slot, int b, int ks) const {
    const char *p = reinterpret_cast<const char *>(slot) + at[b] + ks * (16 * 512);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 512));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// An operand whose rows are outputs: rows of 32 terms (4 pieces), piece p of
// row r at p ^ ((r >> 2) & 3).
struct AlongOperand {
  uint32_t at[2];
  __device__ __forceinline__ void init(int first_row, int lane) {
    const int r = first_row + lane % 32;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      at[ks] = r * 64 + (((ks * 2 + lane / 32) ^ ((r >> 2) & 3)) * 16);
  }
  __device__ __forceinline__ bf16x8 read(const u32x4 *slot, int b, int ks) const {
    const char *p = reinterpret_cast<const char *>(slot) + at[ks] + b * (32 * 64);
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
  }
};

template <int MI>
struct Frag {
  bf16x8 a[MI], b[4];
};

template <int MI, class OpA>
__device__ __forceinline__ void read_frag(Frag<MI> &f, const OpA &oa, const CrossOperand &ob,
                                          const u32x4 *slot, int ks) {
#pragma unroll
  for (int i = 0; i < MI; ++i) f.a[i] = oa.read(slot, i, ks);
#pragma unroll
  for (int i = 0; i < 4; ++i) f.b[i] = ob.read(slot + SLOT / 2, i, ks);
}

template <int MI>
__device__ __forceinline__ void mfma_frag(f32x16 (&acc)[MI][4], const Frag<MI> &f) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Runs the sum's `stages` stages through the ring and leaves it in acc.
// issue(stage, slot) starts IL loads of a wave; stages past the last one read
// zeros, so that the counts never change.
template <int MI, int IL, class OpA, class Issue>
__device__ __forceinline__ void run_sum(f32x16 (&acc)[MI][4], const OpA &oa, const CrossOperand &ob,
                                        int stages, u32x4 *s0, u32x4 *s1, u32x4 *s2, u32x4 *s3,
                                        u32x4 *s4, Issue issue) {
  issue(0, s0);
  issue(1, s1);
  issue(2, s2);
  issue(3, s3);
  issue(4, s4);
  wait_vmcnt<(NS - 1) * IL>();
  stage_barrier();
  Frag<MI> f0, f1;
  read_frag(f0, oa, ob, s0, 0);
  // Stage s in slot `cur`: its second half is read while the first is
  // multiplied; then stage s + 1 has landed for every wave, and `cur`, which
  // every wave has read, takes stage s + 5.
#define MOE_STAGE(s, cur, nxt)                   \
  read_frag(f1, oa, ob, cur, 1);                 \
  mfma_frag(acc, f0);                            \
  wait_vmcnt_lgkm0<(NS - 2) * IL>();             \
  stage_barrier();                               \
  issue((s) + NS, cur);                          \
  read_frag(f0, oa, ob, nxt, 0);                 \
  mfma_frag(acc, f1);
  int s = 0;
  for (; s + NS <= stages; s += NS) {
    MOE_STAGE(s, s0, s1)
    MOE_STAGE(s + 1, s1, s2)
    MOE_STAGE(s + 2, s2, s3)
    MOE_STAGE(s + 3, s3, s4)
    MOE_STAGE(s + 4, s4, s0)
  }
  if (s < stages) {
    MOE_STAGE(s, s0, s1)
    if (s + 1 < stages) {
      MOE_STAGE(s + 1, s1, s2)
      if (s + 2 < stages) {
        MOE_STAGE(s + 2, s2, s3)
        if (s + 3 < stages) {
          MOE_STAGE(s + 3, s3, s4)
        }
      }
    }
  }
#undef MOE_STAGE
  wait_vmcnt<0>();  // no LDS-direct load may still be landing in what comes next
}

__device__ __forceinline__ void load_lds(const uint16_t *g, u32x4 *l) {
  __builtin_amdgcn_global_load_lds((const void *)g, (lds_void *)l, 16, 0, 0);
}

// live ? p : the zeros, without a branch (written as a choice of addresses,
// the compiler makes two loads of it, each under its own lanes)
__device__ __forceinline__ const uint16_t *or_zeros(bool live, const uint16_t *p) {
  const uint64_t z = reinterpret_cast<uint64_t>(g_zeros), m = live ? ~0ull : 0ull;
  return reinterpret_cast<const uint16_t *>(z ^ ((z ^ reinterpret_cast<uint64_t>(p)) & m));
}

// The tile's sums, 32 rows of every wave at a time, through LDS: f(row, first
// column, 8 values) for pieces of 8 columns, 16 bytes of bf16.  32 x 32
// accumulator layout: lane holds column lane % 32, register r row 8 (r / 4) +
// 4 (lane / 32) + r % 4; rows 4 apart go to different halves of 256 bytes.
template <int MI, class F>
__device__ __forceinline__ void each_piece(const f32x16 (&acc)[MI][4], u32x4 *s0, u32x4 *s1, F f) {
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int wm = wv / 2, wn = wv % 2;
  float *const mine = reinterpret_cast<float *>(wm == 0 ? s0 : s1);
  __syncthreads();  // every wave is done reading the ring
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r / 4) + 4 * (lane / 32) + r % 4;
        const int col = wn * 128 + j * 32 + lane % 32;
        mine[row * BN + (col ^ (((row >> 2) & 1) << 5))] = acc[i][j][r];
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2 * 32 * 32 / (NW * 64); ++q) {
      const int id = q * (NW * 64) + tid;
      const int half = id / (32 * 32), row = id / 32 % 32, pc = id % 32;
      const float *p = reinterpret_cast<const float *>(half == 0 ? s0 : s1) + row * BN +
                       ((pc * 8) ^ (((row >> 2) & 1) << 5));
      float v[8];
      *reinterpret_cast<f32x4 *>(v) = *reinterpret_cast<const f32x4 *>(p);
      *reinterpret_cast<f32x4 *>(v + 4) = *reinterpret_cast<const f32x4 *>(p + 4);
      f(half * (MI * 32) + i * 32 + row, pc * 8, v);
    }
    __syncthreads();  // the rows are rewritten
  }
}

__device__ __forceinline__ void load8(const uint16_t *p, float v[8]) {
  const u32x4 raw = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(raw[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
  }
}

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void store8(uint16_t *p, const float v[8]) {
  bf16x8v o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];  // round to nearest even
  *reinterpret_cast<bf16x8v *>(p) = o;
}

__device__ __forceinline__ void store8(float *p, const float v[8]) {
  *reinterpret_cast<f32x4 *>(p) = *reinterpret_cast<const f32x4 *>(v);
  *reinterpret_cast<f32x4 *>(p + 4) = *reinterpret_cast<const f32x4 *>(v + 4);
}

// One dgrad tile of at most BM rows.  TAIL: N is not a multiple of a stage.
template <int BM, bool TAIL, class Out>
__device__ __forceinline__ void dgrad_tile(const GradArgs &a, const Tile &tile, u32x4 *s0, u32x4 *s1,
                                           u32x4 *s2, u32x4 *s3, u32x4 *s4, Out out) {
  constexpr int MI = BM / 64;
  constexpr int IA = BM * 4 / 64 / NW, IB = SLOT / 2 / 64 / NW;  // loads a wave and stage
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = wv / 2, wn = wv % 2;
  // rows past the tile's last repeat it, columns past the last the last piece
  const int n_a = ((lane % 4) ^ ((lane / 16) & 3)) * 8;  // first term of this lane's A pieces
  const uint16_t *ga[IA], *gb[IB];
  int n_b[IB];
#pragma unroll
  for (int i = 0; i < IA; ++i) {
    const int r = (wv * IA + i) * 16 + lane / 4;
    ga[i] = static_cast<const uint16_t *>(a.dC) +
            (size_t)min(tile.m0 + r, tile.mend - 1) * a.N + n_a;
  }
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int n = (wv * IB + i) * 2 + lane / 32;
    const int col = tile.nt * BN + (((lane % 32) ^ ((n & 3) << 2))) * 8;
    n_b[i] = n;
    gb[i] = static_cast<const uint16_t *>(a.B) + ((size_t)tile.g * a.N + n) * a.ldb +
            min(col, a.K - 8);
  }
  const int span = (a.N + BK - 1) / BK;  // stages of one product
  const ptrdiff_t second_a = static_cast<const uint16_t *>(a.dC2) - static_cast<const uint16_t *>(a.dC);
  const ptrdiff_t second_b = static_cast<const uint16_t *>(a.B2) - static_cast<const uint16_t *>(a.B);
  const int stages = a.dC2 ? 2 * span : span;
  auto issue = [&](int st, u32x4 *slot) {
    st = min(st, stages - 1);
    const bool second = st >= span;
    const int n0 = (second ? st - span : st) * BK;
    const ptrdiff_t oa = n0 + (second ? second_a : 0);
    const ptrdiff_t ob = (ptrdiff_t)n0 * a.ldb + (second ? second_b : 0);
#pragma unroll
    for (int i = 0; i < IA; ++i)
      load_lds(TAIL ? or_zeros(n0 + n_a < a.N, ga[i] + oa) : ga[i] + oa, slot + (wv * IA + i) * 64);
#pragma unroll
    for (int i = 0; i < IB; ++i)
      load_lds(TAIL ? or_zeros(n0 + n_b[i] < a.N, gb[i] + ob) : gb[i] + ob,
               slot + SLOT / 2 + (wv * IB + i) * 64);
  };
  AlongOperand oa;
  CrossOperand ob;
  oa.init(wm * (MI * 32), lane);
  ob.init(wn * 4, lane);
  f32x16 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
  run_sum<MI, IA + IB>(acc, oa, ob, stages, s0, s1, s2, s3, s4, issue);
  each_piece(acc, s0, s1, [&](int r, int c, const float *v) {
    const int m = tile.m0 + r, k = tile.nt * BN + c;
    if (m < tile.mend && k < a.K) out((size_t)m * a.K + k, v);
  });
}

// silu's factor with the hardware's exp2 and reciprocal (each within 1 ulp,
// far below the bf16 rounding)
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

template <bool SWIGLU, bool OUT_F32, bool TAIL>
__global__ __launch_bounds__(NW * 64, 1) void dgrad_kernel(const GradArgs a, int nt) {
  __shared__ u32x4 s0[SLOT], s1[SLOT], s2[SLOT], s3[SLOT], s4[SLOT];
  // (the scheduler's result lies in the last slot until the ring starts)
  const Sched sc = sched_lookup(a.offsets, a.G, a.rows, 256, nt, kTileChunk, false,
                                reinterpret_cast<int *>(s4),
                                [](int total) { return tile_of_workgroup(blockIdx.x, total); });
  if (sc.L < 0) return;
  __syncthreads();
  const Tile tile = sc.tile;
  auto out = [&](size_t at, const float *v) {
    if constexpr (SWIGLU) {
      float z[8], u[8], dg[8], du[8], h[8];
      load8(static_cast<const uint16_t *>(a.gate) + at, z);
      load8(static_cast<const uint16_t *>(a.up) + at, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid(z[i]), zs = z[i] * s;
        dg[i] = v[i] * u[i] * s * (1.f + z[i] * (1.f - s));
        du[i] = v[i] * zs;
        h[i] = zs * u[i];
      }
      store8(static_cast<uint16_t *>(a.out) + at, dg);
      store8(static_cast<uint16_t *>(a.out2) + at, du);
      if (a.h) store8(static_cast<uint16_t *>(a.h) + at, h);
    } else if constexpr (OUT_F32) {
      store8(static_cast<float *>(a.out) + at, v);
    } else {
      store8(static_cast<uint16_t *>(a.out) + at, v);
    }
  };
  const int rows = tile.mend - tile.m0;
  if (rows > 128) dgrad_tile<256, TAIL>(a, tile, s0, s1, s2, s3, s4, out);
  else if (rows > 64) dgrad_tile<128, TAIL>(a, tile, s0, s1, s2, s3, s4, out);
  else dgrad_tile<64, TAIL>(a, tile, s0, s1, s2, s3, s4, out);
}

template <bool OUT_F32>
__global__ __launch_bounds__(NW * 64, 1) void wgrad_kernel(const GradArgs a, int nt, int kt) {
  __shared__ u32x4 s0[SLOT], s1[SLOT], s2[SLOT], s3[SLOT], s4[SLOT];
  constexpr int IL = SLOT / 2 / 64 / NW;  // loads a wave, stage and operand
  int w = blockIdx.x;
  const int k0 = w % kt * BN;
  w /= kt;
  const int n0 = w % nt * BN;
  w /= nt;
  const int g = w % a.G, slice = w / a.G;
  int *const s_rows = reinterpret_cast<int *>(s4);
  group_rows(a.offsets, a.rows, g, s_rows);
  int r0 = s_rows[0], r1 = s_rows[1];
  __syncthreads();
  if (a.part) slice_rows(&r0, &r1, slice, a.slices);
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = wv / 2, wn = wv % 2;
  const uint16_t *ga[IL], *gb[IL];
  int r_of[IL];
#pragma unroll
  for (int i = 0; i < IL; ++i) {
    const int r = (wv * IL + i) * 2 + lane / 32;
    const int col = ((lane % 32) ^ ((r & 3) << 2)) * 8;
    r_of[i] = r;
    ga[i] = static_cast<const uint16_t *>(a.dC) + (size_t)(r0 + r) * a.N + min(n0 + col, a.N - 8);
    gb[i] = static_cast<const uint16_t *>(a.A) + (size_t)(r0 + r) * a.K + min(k0 + col, a.K - 8);
  }
  const int terms = r1 - r0;
  auto issue = [&](int st, u32x4 *slot) {
    const int t0 = st * BK;
    const size_t oa = (size_t)t0 * a.N, ob = (size_t)t0 * a.K;
#pragma unroll
    for (int i = 0; i < IL; ++i) {
      const bool live = t0 + r_of[i] < terms;
      load_lds(or_zeros(live, ga[i] + oa), slot + (wv * IL + i) * 64);
      load_lds(or_zeros(live, gb[i] + ob), slot + SLOT / 2 + (wv * IL + i) * 64);
    }
  };
  CrossOperand oa, ob;
  oa.init(wm * 4, lane);
  ob.init(wn * 4, lane);
  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
  run_sum<4, 2 * IL>(acc, oa, ob, (terms + BK - 1) / BK, s0, s1, s2, s3, s4, issue);
  each_piece(acc, s0, s1, [&](int r, int c, const float *v) {
    const int n = n0 + r, k = k0 + c;
    if (n >= a.N || k >= a.K) return;
    const size_t at = ((size_t)g * a.N + n) * a.K + k;
    if (a.part) {
      store8(a.part + (size_t)slice * a.G * a.N * a.K + at, v);
      return;
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
    if (a.accumulate) {
      float b[8];
      if constexpr (OUT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = static_cast<const float *>(a.out)[at + i];
      } else {
        load8(static_cast<const uint16_t *>(a.out) + at, b);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += b[i];
    }
    if constexpr (OUT_F32) store8(static_cast<float *>(a.out) + at, o);
    else store8(static_cast<uint16_t *>(a.out) + at, o);
  });
}

}  // namespace

hipError_t launch_dgrad_bf16(const GradArgs &a, hipStream_t s) {
  const int nt = (a.K + BN - 1) / BN;
  const dim3 grid((unsigned)(host_row_tile_bound(a.rows, a.G, 256) * (long long)nt)), block(NW * 64);
  const bool tail = a.N % BK != 0;
#define MOE_LAUNCH(SW, F32)                                                                    \
  if (tail) hipLaunchKernelGGL((dgrad_kernel<SW, F32, true>), grid, block, 0, s, a, nt);       \
  else hipLaunchKernelGGL((dgrad_kernel<SW, F32, false>), grid, block, 0, s, a, nt)
  if (a.gate) {
    MOE_LAUNCH(true, false);
  } else if (a.out_dt == MOE_F32) {
    MOE_LAUNCH(false, true);
  } else {
    MOE_LAUNCH(false, false);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_wgrad_bf16(const GradArgs &a, hipStream_t s) {
  const int nt = (a.N + BN - 1) / BN, kt = (a.K + BN - 1) / BN;
  const dim3 grid((unsigned)((long long)a.slices * a.G * nt * kt)), block(NW * 64);
  if (a.out_dt == MOE_F32) hipLaunchKernelGGL(wgrad_kernel<true>, grid, block, 0, s, a, nt, kt);
  else hipLaunchKernelGGL(wgrad_kernel<false>, grid, block, 0, s, a, nt, kt);
  return hipGetLastError();
}
