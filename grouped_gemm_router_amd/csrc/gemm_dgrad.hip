// gemm_dgrad.hip -- the gradient of a grouped product's input on bf16 MFMA:
//   dA[r][k] = sum_n dC[r][n] B[g][n][k] (+ dC2 B2), r in group g,
// with SwiGLU's gradient behind it or not.
//
// Design (what is shared with gemm_wgrad.hip stands in gemm_grad.h):
//   * tiles of 256 x 256 outputs, one workgroup of 4 waves (128 x 128 each) a
//     CU, and tiles of 192, 128 or 64 rows for what a group leaves; the device
//     reads the offsets (the tile scheduler of the forward product);
//   * stages of 64 terms: dC, whose rows lie along the sum, moves as whole
//     128-byte lines (as 64-byte halves, twice the requests: 8 groups of 1024,
//     N 4096, K 14336 took 842 us instead of 779), the weights as they lie;
//   * half a stage's LDS reads go between the first MFMAs of the half before
//     (left to the compiler, each half waited for its own reads: 887 -> 847);
//   * a sum that ends inside a stage moves its last stage back instead of
//     testing every load (that arithmetic, 10 instructions a load, no longer
//     fitted beside the MFMAs); the second of two products follows in the same
//     run of stages.
// Measured on that shape: 750-880 us, from card to card, 1.09-1.28 PFLOP/s (the library's
// dense product of the same sizes 1.31, its 8192^3 with both operands along the
// sum 1.51).  The matrix cores are busy 66 % of the cycles, at 1.70 GHz: the
// chip lowers its clock under this load, so that fewer stalls buy less than
// their share.  SwiGLU's gradient reads and writes 0.94 GB more than the product
// does (186 us at 5.05 TB/s) and adds 137 us to it, 100 without h, in turn in one
// process (813, 950 and 914 us); a workgroup does nothing else meanwhile.
// Measured and not kept for it: eight waves of 128 x 64 (no faster, the product 3 % slower),
// two workgroups a CU of 256 x 128 tiles (1136 against 989 us at the time),
// loads asked for further ahead (no change, then spills), workgroups started
// apart (1078 -> 1068 at best), 32 instead of 16 columns of tiles in turn.
#include "gemm_grad.h"

namespace {

// An operand whose rows are outputs: W rows of 64 terms, a 128-byte line (8
// pieces), piece p of row r at p ^ ((r >> 1) & 7).
template <int W>
struct AlongOperand {
  static constexpr int NB = W / 64;
  static constexpr int IL = pieces(W, 64) / 64 / NW;
  static constexpr int READS = NB;
  uint32_t row, turn;
  __device__ __forceinline__ void init(int half, int lane) {
    const int r = half * (W / 2) + lane % 32;
    row = r * 128;
    turn = ((lane / 32) ^ ((r >> 1) & 7)) * 16;
  }
  __device__ __forceinline__ bf16x8 read(const u32x4 *slot, int b, int ks) const {
    const char *p = reinterpret_cast<const char *>(slot) + row + (turn ^ (ks * 32)) + b * (32 * 128);
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
  }
  // the first z terms as zeros (z a multiple of 8)
  static __device__ __forceinline__ void zero(u32x4 *slot, int z) {
    for (int i = threadIdx.x; i < W * 8; i += NW * 64) {
      const int r = i / 8, p = i % 8;
      if (p * 8 < z) slot[r * 8 + (p ^ ((r >> 1) & 7))] = u32x4{};
    }
  }
  // row and first term of what load i of wave wv brings this lane
  static __device__ __forceinline__ int load_row(int wv, int i, int lane) {
    return (wv * IL + i) * 8 + lane / 8;
  }
  static __device__ __forceinline__ int load_term(int row, int lane) {
    return ((lane % 8) ^ ((row >> 1) & 7)) * 8;
  }
};

// dgrad's ring: stages of 64 terms, so that the operand whose rows lie along
// the sum moves as whole 128-byte lines: two slots of it, three of the weights,
// all 160 KB.  Stage d reads A slot d % 2 and B slot d % 3 in four steps.  In
// the last of them stage d + 1 has landed for every wave and every wave has
// read stage d: A slot d % 2 takes A's stage d + 2.  B's stage d + 2 goes into
// the slot of stage d - 1 during the first steps of stage d.
struct Ring23 {
  u32x4 *a0, *a1, *b0, *b1, *b2;
};

#define MOE_STEP(sa, sb, ks, from, to, loads, load)         \
  load;                                                     \
  read_frag(to, oa, ob, r.sa, r.sb, ks);                    \
  mfma_frag(acc, from);                                     \
  interleave<MI * NB, OpA::READS + OpB::READS, loads>();    \
  __builtin_amdgcn_sched_barrier(0);
#define MOE_STAGE(d, sa, sb, na, nb, pb, check)             \
  MOE_STEP(sa, sb, 1, f0, f1, OpB::IL / 2, issue_b((d) + 2, r.pb, 0)) \
  MOE_STEP(sa, sb, 2, f1, f0, OpB::IL / 2, issue_b((d) + 2, r.pb, 1)) \
  MOE_STEP(sa, sb, 3, f0, f1, 0, )                          \
  wait_vmcnt_lgkm0<OpB::IL>();                              \
  stage_barrier();                                          \
  if (check && z && (d) + 2 == stages) zero_terms<OpA, OpB>(r.na, r.nb, z); \
  MOE_STEP(na, nb, 0, f1, f0, OpA::IL, issue_a((d) + 2, r.sa))
template <int MI, int NB, class OpA, class OpB, class IssueA, class IssueB>
__device__ __forceinline__ void run_sum(f32x16 (&acc)[MI][NB], const OpA &oa, const OpB &ob,
                                        int stages, int z, const Ring23 &r, IssueA issue_a,
                                        IssueB issue_b) {
  issue_b(0, r.b0, 0);
  issue_b(0, r.b0, 1);
  issue_a(0, r.a0);
  issue_b(1, r.b1, 0);
  issue_b(1, r.b1, 1);
  issue_a(1, r.a1);
  wait_vmcnt<OpA::IL + OpB::IL>();
  stage_barrier();
  if (z && stages == 1) zero_terms<OpA, OpB>(r.a0, r.b0, z);
  Frag<MI, NB> f0, f1;
  read_frag(f0, oa, ob, r.a0, r.b0, 0);
  int d = 0;
  for (; d + 7 < stages; d += 6) {
    MOE_STAGE(d, a0, b0, a1, b1, b2, false)
    MOE_STAGE(d + 1, a1, b1, a0, b2, b0, false)
    MOE_STAGE(d + 2, a0, b2, a1, b0, b1, false)
    MOE_STAGE(d + 3, a1, b0, a0, b1, b2, false)
    MOE_STAGE(d + 4, a0, b1, a1, b2, b0, false)
    MOE_STAGE(d + 5, a1, b2, a0, b0, b1, false)
  }
  if (d < stages) {
    MOE_STAGE(d, a0, b0, a1, b1, b2, true)
    if (d + 1 < stages) {
      MOE_STAGE(d + 1, a1, b1, a0, b2, b0, true)
      if (d + 2 < stages) {
        MOE_STAGE(d + 2, a0, b2, a1, b0, b1, true)
        if (d + 3 < stages) {
          MOE_STAGE(d + 3, a1, b0, a0, b1, b2, true)
          if (d + 4 < stages) {
            MOE_STAGE(d + 4, a0, b1, a1, b2, b0, true)
            if (d + 5 < stages) {
              MOE_STAGE(d + 5, a1, b2, a0, b0, b1, true)
              if (d + 6 < stages) {
                MOE_STAGE(d + 6, a0, b0, a1, b1, b2, true)
              }
            }
          }
        }
      }
    }
  }
  wait_vmcnt<0>();  // no LDS-direct load may still be landing in what comes next
}
#undef MOE_STAGE
#undef MOE_STEP

// One dgrad tile of at most BM rows and 256 columns.  SHORT: N is less than a
// stage.
template <int BM, bool SHORT, class Out>
__device__ __forceinline__ void dgrad_tile(const GradArgs &a, const Tile &tile, int slice,
                                           const Ring23 &ring) {
  typedef AlongOperand<BM> OpA;
  typedef CrossOperand<256, 64> OpB;
  constexpr int IA = OpA::IL, IB = OpB::IL;
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  // bytes from the stage's first term in the tile's first row and column; rows
  // past the tile's last repeat it, columns past the last the last piece
  const int k0 = tile.nt * 256;
  uint32_t at_a[IA], at_b[IB];
#pragma unroll
  for (int i = 0; i < IA; ++i) {
    const int r = OpA::load_row(wv, i, lane);
    at_a[i] = ((uint32_t)min(r, tile.mend - 1 - tile.m0) * a.N + OpA::load_term(r, lane)) * 2;
  }
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int n = OpB::load_row(wv, i, lane);
    at_b[i] = ((uint32_t)n * a.ldb + min(OpB::load_col(n, lane), a.K - 8 - k0)) * 2;
  }
  const Span<64> span(a.N);
  const size_t first_a = (size_t)tile.m0 * a.N, first_b = (size_t)tile.g * a.N * a.ldb + k0;
  // this slice's stages of one product; both products in one run of stages, or,
  // where each ends inside a stage or is cut, one after the other
  const int per = (span.stages + a.slices - 1) / a.slices, st0 = slice * per;
  const int count = min(per, span.stages - st0);
  const int back = st0 + count == span.stages ? span.back : 0;
  const bool joined = a.dC2 && !span.back && a.slices == 1;
  const int parts = a.dC2 && !joined ? 2 : 1;
  const int stages = joined ? 2 * count : count;
  int part = 0;
  auto issue_a = [&](int st, u32x4 *slot) {
    st = min(st, stages - 1) + st0;
    const bool second = part || st >= span.stages;
    st -= second && !part ? span.stages : 0;
    const uint16_t *const p = static_cast<const uint16_t *>(second ? a.dC2 : a.dC) + first_a +
                              (SHORT ? 0 : span.first(st));
#pragma unroll
    for (int i = 0; i < IA; ++i) {
      u32x4 *const to = slot + (wv * IA + i) * 64;
      if constexpr (SHORT)
        load_lds(or_zeros(OpA::load_term(OpA::load_row(wv, i, lane), lane) < a.N, p + at_a[i] / 2),
                 0, to);
      else load_lds(p, at_a[i], to);
    }
  };
  auto issue_b = [&](int st, u32x4 *slot, int half) {
    st = min(st, stages - 1) + st0;
    const bool second = part || st >= span.stages;
    st -= second && !part ? span.stages : 0;
    const uint16_t *const p = static_cast<const uint16_t *>(second ? a.B2 : a.B) + first_b +
                              (size_t)(SHORT ? 0 : span.first(st)) * a.ldb;
#pragma unroll
    for (int j = 0; j < IB / 2; ++j) {
      const int i = half * (IB / 2) + j;
      u32x4 *const to = slot + (wv * IB + i) * 64;
      if constexpr (SHORT)
        load_lds(or_zeros(OpB::load_row(wv, i, lane) < a.N, p + at_b[i] / 2), 0, to);
      else load_lds(p, at_b[i], to);
    }
  };
  OpA oa;
  OpB ob;
  oa.init(wv / 2, lane);
  ob.init(wv % 2, lane);
  f32x16 acc[OpA::NB][OpB::NB];
#pragma unroll
  for (int i = 0; i < OpA::NB; ++i)
#pragma unroll
    for (int j = 0; j < OpB::NB; ++j) acc[i][j] = f32x16{};
  for (; part < parts; ++part) {
    run_sum(acc, oa, ob, stages, back, ring, issue_a, issue_b);
    stage_barrier();  // every wave is done reading the ring
  }
  const Out out = {a, tile.m0, tile.mend, k0, (size_t)slice * a.rows * a.K};
  u32x4 *const mine = wv == 0 ? ring.a0 : wv == 1 ? ring.a1 : wv == 2 ? ring.b0 : ring.b1;
  if (tile.mend - tile.m0 == BM && k0 + 256 <= a.K) each_piece<true, 64>(acc, mine, out);
  else each_piece<false, 64>(acc, mine, out);
}

// silu's factor with the hardware's exp2 and reciprocal (each within 1 ulp,
// far below the bf16 rounding)
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

// what becomes of the sums of a dgrad tile
template <bool SWIGLU, bool OUT_F32, bool STREAM>
struct DgradOut {
  static constexpr int COLS = OUT_F32 ? 4 : 8, UN = 4, DEPTH = 2;
  const GradArgs &a;
  int m0, mend, k0;
  size_t first;  // where the slice's outputs begin
  struct Held {
    u32x4 gate, up;
  };
  template <bool FULL>
  __device__ __forceinline__ Held begin(int r, int c) const {
    Held x{};
    if constexpr (SWIGLU) {
      if (FULL || (m0 + r < mend && k0 + c < a.K)) {
        const size_t at = (size_t)(m0 + r) * a.K + k0 + c;
        x.gate = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.gate) + at);
        x.up = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.up) + at);
      }
    }
    return x;
  }
  template <bool FULL>
  __device__ __forceinline__ void finish(int r, int c, const Held &x, const float *v) const {
    if (!FULL && (m0 + r >= mend || k0 + c >= a.K)) return;
    const size_t at = first + (size_t)(m0 + r) * a.K + k0 + c;
    if constexpr (SWIGLU) {
      float z[8], u[8], dg[8], du[8], h[8];
      widen8(x.gate, z);
      widen8(x.up, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid(z[i]), zs = z[i] * s;
        dg[i] = v[i] * u[i] * fmaf(zs, 1.f - s, s);  // s (1 + z (1 - s))
        du[i] = v[i] * zs;
        h[i] = zs * u[i];
      }
      store<STREAM>(static_cast<uint16_t *>(a.out) + at, dg);
      store<STREAM>(static_cast<uint16_t *>(a.out2) + at, du);
      if (a.h) store<STREAM>(static_cast<uint16_t *>(a.h) + at, h);
    } else if constexpr (OUT_F32) {
      store<STREAM>(static_cast<float *>(a.out) + at, v);
    } else {
      store<STREAM>(static_cast<uint16_t *>(a.out) + at, v);
    }
  }
};

template <bool SWIGLU, bool OUT_F32, bool STREAM, bool SHORT>
__global__ __launch_bounds__(NW * 64, 1) void dgrad_kernel(const GradArgs a, int nt,
                                                                int run) {
  constexpr int SLOT = pieces(256, 64);
  __shared__ u32x4 a0[SLOT], a1[SLOT], b0[SLOT], b1[SLOT], b2[SLOT];
  const Ring23 ring = {a0, a1, b0, b1, b2};
  const int w = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  // (the scheduler's result lies in a slot that the ring fills later)
  const Sched sc = sched_lookup(a.offsets, a.G, a.rows, 256, nt, kTileChunk, false,
                                reinterpret_cast<int *>(b2),
                                [&](int total) {
                                  if (w >= total / (8 * run) * (8 * run))
                                    return tile_of_workgroup(w, total);
                                  return w / (8 * run) * (8 * run) + w % 8 * run + w / 8 % run;
                                });
  if (sc.L < 0) return;
  const Tile tile = sc.tile;
  typedef DgradOut<SWIGLU, OUT_F32, STREAM> Out;
  const int rows = tile.mend - tile.m0;
  if (rows > 192) dgrad_tile<256, SHORT, Out>(a, tile, slice, ring);
  else if (rows > 128) dgrad_tile<192, SHORT, Out>(a, tile, slice, ring);
  else if (rows > 64) dgrad_tile<128, SHORT, Out>(a, tile, slice, ring);
  else dgrad_tile<64, SHORT, Out>(a, tile, slice, ring);
}

}  // namespace

hipError_t launch_dgrad_bf16(const GradArgs &args, hipStream_t s) {
  const GradArgs a = to_slices(args);
  const int nt = (a.K + 255) / 256;
  const dim3 grid((unsigned)(row_tiles(a.rows, a.G, 256) * (long long)nt * a.slices)), block(NW * 64);
  const bool brief = a.N < 64;
  // Tiles go to the 8 XCDs in turn (runs of 1: their concurrent tiles share
  // columns of one group's weights), or, for groups of few row tiles, in runs of
  // 32, so that a group's weights are fetched into one or two L2s (64 groups of
  // 384 rows, N 2048, K 7168: 970 -> 919 us, of 430 rows 846 -> 797; 8 groups of
  // 1024, N 4096, K 14336: 753 -> 766 us, with SwiGLU 1058 -> 1114)
  const int run = a.rows <= 512ll * a.G ? 32 : 1;
  const bool stream = a.slices == 1 && streams(a.rows, a.K * (a.out_dt == MOE_F32 ? 4 : 2), a.gate ? 2 + (a.h != nullptr) : 1);
#define MOE_LAUNCH(SW, F32)                                                                          \
  if (brief) hipLaunchKernelGGL((dgrad_kernel<SW, F32, false, true>), grid, block, 0, s, a, nt, run);     \
  else if (stream) hipLaunchKernelGGL((dgrad_kernel<SW, F32, true, false>), grid, block, 0, s, a, nt, run); \
  else hipLaunchKernelGGL((dgrad_kernel<SW, F32, false, false>), grid, block, 0, s, a, nt, run)
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
