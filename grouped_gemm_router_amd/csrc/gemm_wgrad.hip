// gemm_wgrad.hip -- the gradient of a grouped product's weights on bf16 MFMA:
//   dB[g][n][k] (+)= sum_{r in group g} dC[r][n] A[r][k]
//
// Design (what is shared with gemm_dgrad.hip stands in gemm_grad.h): sums are
// as long as a group has rows (1024 on the Mixtral shapes, some hundreds for
// fine-grained experts), so what a tile does besides its sum counts: tiles of
// 128 x 256 weights, 4 waves of 64 x 128, two workgroups a CU, so that one's
// sum runs beside the other's start and stores (256 x 256 tiles, one a CU: 8
// groups of 1024 rows, 14336 x 4096: 999 against 946 us in one process; 64
// groups of 384, 1408 x 2048: 250 against 193).  Both operands' rows are terms;
// stages of 32 rows of whole 256- and 512-byte pieces.
// Measured: 14336 x 4096 in bf16, 8192 rows of 8 groups 935-1000 us (1.0
// PFLOP/s; the library's single product of a group 0.84): matrix cores 58 %
// busy at 1.68 GHz, 0.94 GB of weights written (186 us at 5.05 TB/s) partly
// beside the sums.  1416 x 2056 in fp32, 24271 rows of 64 groups 361-395 us:
// 1.18 GB fetched and written (233 us at 5.05 TB/s), matrix cores 20 % busy; a
// tile's start, its 12 stages and its stores mostly follow each other.  Rows that
// begin inside a 128-byte line are 70 us of it (in turn: 1416 x 2056 377, 1416 x
// 2080 307), the tiles for the last 8 and 32 columns 47 (1408 x 2048: 260).
// Added to fp32 sums, 14336 x 4096 takes 1217-1273: 1.9 GB read and as much
// written (805 us at the copy's rate).
#include <type_traits>

#include "gemm_grad.h"

namespace {

// wgrad's ring: three stages of 32 terms of both operands, 24 KB each, so that
// two workgroups share a CU.  Stage s in slot `cur`: its second half is read
// while the first is multiplied; then stage s + 1 has landed for every wave,
// and `cur`, which every wave has read, takes stage s + 3.
struct Ring3 {
  u32x4 *s0, *s1, *s2;
};
constexpr int SB = pieces(128, 32);  // where the second operand begins in a slot

#define MOE_HALF_0(s, cur, prv)                        \
  issue_b((s) + 2, r.prv + SB);                        \
  read_frag(f1, oa, ob, r.cur, r.cur + SB, 1);         \
  mfma_frag(acc, f0);                                  \
  interleave<MI * NB, OpA::READS + OpB::READS, OpB::IL>(); \
  __builtin_amdgcn_sched_barrier(0);                   \
  wait_vmcnt_lgkm0<IL>();                              \
  stage_barrier();
#define MOE_HALF_1(s, cur, nxt)                        \
  issue_a((s) + 3, r.cur);                             \
  read_frag(f0, oa, ob, r.nxt, r.nxt + SB, 0);         \
  mfma_frag(acc, f1);                                  \
  interleave<MI * NB, OpA::READS + OpB::READS, OpA::IL>();
#define MOE_STAGE(s, cur, nxt, prv)                    \
  MOE_HALF_0(s, cur, prv)                              \
  MOE_HALF_1(s, cur, nxt)
#define MOE_LAST_STAGES(s, cur, nxt, prv)              \
  MOE_HALF_0(s, cur, prv)                              \
  if (z && (s) + 2 == stages) zero_terms<OpA, OpB>(r.nxt, r.nxt + SB, z); \
  MOE_HALF_1(s, cur, nxt)
template <int MI, int NB, class OpA, class OpB, class IssueA, class IssueB>
__device__ __forceinline__ void run_sum(f32x16 (&acc)[MI][NB], const OpA &oa, const OpB &ob,
                                        int stages, int z, const Ring3 &r, IssueA issue_a,
                                        IssueB issue_b) {
  constexpr int IL = OpA::IL + OpB::IL;
  issue_a(0, r.s0);
  issue_b(0, r.s0 + SB);
  issue_a(1, r.s1);
  issue_b(1, r.s1 + SB);
  issue_a(2, r.s2);
  wait_vmcnt<IL + OpA::IL>();
  stage_barrier();
  if (z && stages == 1) zero_terms<OpA, OpB>(r.s0, r.s0 + SB, z);
  Frag<MI, NB> f0, f1;
  read_frag(f0, oa, ob, r.s0, r.s0 + SB, 0);
  int s = 0;
  for (; s + 4 < stages; s += 3) {
    MOE_STAGE(s, s0, s1, s2)
    MOE_STAGE(s + 1, s1, s2, s0)
    MOE_STAGE(s + 2, s2, s0, s1)
  }
  if (s < stages) {
    MOE_LAST_STAGES(s, s0, s1, s2)
    if (s + 1 < stages) {
      MOE_LAST_STAGES(s + 1, s1, s2, s0)
      if (s + 2 < stages) {
        MOE_LAST_STAGES(s + 2, s2, s0, s1)
        if (s + 3 < stages) {
          MOE_LAST_STAGES(s + 3, s0, s1, s2)
        }
      }
    }
  }
  wait_vmcnt<0>();  // no LDS-direct load may still be landing in what comes next
}
#undef MOE_LAST_STAGES
#undef MOE_STAGE
#undef MOE_HALF_1
#undef MOE_HALF_0

// Tiles run in strips of kStrip tiles of n, along k, and an XCD takes 64
// consecutive ones (what its 32 CUs hold), so that its L2 is asked for few
// columns of either operand (columns of k in turn over all XCDs: 1013 -> 986 us
// on 8 groups of 14336 x 4096; strips of 4, 8 or 12, or along n: within 3 %).
constexpr int kStrip = 6, kRun = 64;

// how the sums of a wgrad tile are stored
enum Mode { PLAIN, STREAM, ADD };  // past the caches; added to what is there

template <bool OUT_F32, Mode MODE>
struct WgradOut {
  static constexpr int COLS = OUT_F32 ? 4 : 8, UN = 4, DEPTH = 2;
  typedef typename std::conditional<OUT_F32, float, uint16_t>::type T;
  T *out;  // the group's weights
  int N, K, n0, k0;
  typedef u32x4 Held;
  template <bool FULL>
  __device__ __forceinline__ Held begin(int r, int c) const {
    if (MODE != ADD || (!FULL && (n0 + r >= N || k0 + c >= K))) return u32x4{};
    return *reinterpret_cast<const u32x4 *>(out + (size_t)(n0 + r) * K + k0 + c);
  }
  template <bool FULL>
  __device__ __forceinline__ void finish(int r, int c, const Held &held, float *v) const {
    if (!FULL && (n0 + r >= N || k0 + c >= K)) return;
    if constexpr (MODE == ADD) {
      float b[COLS];
      if constexpr (OUT_F32) *reinterpret_cast<u32x4 *>(b) = held;
      else widen8(held, b);
#pragma unroll
      for (int i = 0; i < COLS; ++i) v[i] += b[i];
    }
    store<MODE == STREAM>(out + (size_t)(n0 + r) * K + k0 + c, v);
  }
};

// Tiles of 128 x 256 weights.
template <bool OUT_F32, Mode MODE>
__global__ __launch_bounds__(NW * 64, 2) void wgrad_kernel(const GradArgs a, int nt, int kt) {
  constexpr int SLOT = SB + pieces(256, 32);
  typedef CrossOperand<128, 32> OpA;
  typedef CrossOperand<256, 32> OpB;
  constexpr int IA = OpA::IL, IB = OpB::IL;
  __shared__ u32x4 s0[SLOT], s1[SLOT], s2[2048];  // 80 KB
  const Ring3 ring = {s0, s1, s2};
  const int all = nt * kt * a.G * a.slices;
  int w = blockIdx.x;
  if (w < all / (8 * kRun) * (8 * kRun))
    w = w / (8 * kRun) * (8 * kRun) + w % 8 * kRun + w / 8 % kRun;
  const int per = nt * kt;
  const int t = w % per;
  w /= per;
  const int strip = t / (kStrip * kt), wide = min(kStrip, nt - strip * kStrip);
  const int in = t - strip * kStrip * kt;
  const int k0 = in / wide * 256;
  const int n0 = (strip * kStrip + in % wide) * 128;
  const int g = w % a.G, slice = w / a.G;
  int r0, r1;
  group_rows(a.offsets, a.rows, g, &r0, &r1);
  if (a.slices > 1) slice_rows(&r0, &r1, slice, a.slices);
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  // bytes from the stage's first row in the tile's first column; columns past
  // the last repeat the last piece
  uint32_t at_a[IA], at_b[IB];
#pragma unroll
  for (int i = 0; i < IA; ++i) {
    const int r = OpA::load_row(wv, i, lane);
    at_a[i] = ((uint32_t)r * a.N + min(OpA::load_col(r, lane), a.N - 8 - n0)) * 2;
  }
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int r = OpB::load_row(wv, i, lane);
    at_b[i] = ((uint32_t)r * a.K + min(OpB::load_col(r, lane), a.K - 8 - k0)) * 2;
  }
  const Span<32> span(r1 - r0);
  const uint16_t *const dC = static_cast<const uint16_t *>(a.dC) + (size_t)r0 * a.N + n0;
  const uint16_t *const A = static_cast<const uint16_t *>(a.A) + (size_t)r0 * a.K + k0;
  OpA oa;
  OpB ob;
  oa.init(wv / 2, lane);
  ob.init(wv % 2, lane);
  f32x16 acc[OpA::NB][OpB::NB];
#pragma unroll
  for (int i = 0; i < OpA::NB; ++i)
#pragma unroll
    for (int j = 0; j < OpB::NB; ++j) acc[i][j] = f32x16{};
  u32x4 *const mine = wv == 0 ? s0 : wv == 1 ? s1 : wv == 2 ? s2 : s2 + 1024;
  typedef WgradOut<OUT_F32, MODE> Out;
  // (slices write their partial sums one behind the other)
  const Out out = {static_cast<typename Out::T *>(a.out) + ((size_t)slice * a.G + g) * a.N * a.K, a.N,
                   a.K, n0, k0};
  const bool full = n0 + 128 <= a.N && k0 + 256 <= a.K;
  if (span.terms < 32) {  // one stage, of which each row is loaded or zero
#pragma unroll
    for (int i = 0; i < IA; ++i)
      load_lds(or_zeros(OpA::load_row(wv, i, lane) < span.terms, dC + at_a[i] / 2), 0,
               ring.s0 + (wv * IA + i) * 64);
#pragma unroll
    for (int i = 0; i < IB; ++i)
      load_lds(or_zeros(OpB::load_row(wv, i, lane) < span.terms, A + at_b[i] / 2), 0,
               ring.s0 + SB + (wv * IB + i) * 64);
    wait_vmcnt<0>();
    stage_barrier();
    Frag<OpA::NB, OpB::NB> f;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      read_frag(f, oa, ob, ring.s0, ring.s0 + SB, ks);
      mfma_frag(acc, f);
    }
    __syncthreads();  // every wave is done reading
    each_piece<false, 32>(acc, mine, out);
    return;
  }
  auto issue_a = [&](int st, u32x4 *slot) {
    const uint16_t *const p = dC + (size_t)span.first(min(st, span.stages - 1)) * a.N;
#pragma unroll
    for (int i = 0; i < IA; ++i) load_lds(p, at_a[i], slot + (wv * IA + i) * 64);
  };
  auto issue_b = [&](int st, u32x4 *slot) {
    const uint16_t *const p = A + (size_t)span.first(min(st, span.stages - 1)) * a.K;
#pragma unroll
    for (int i = 0; i < IB; ++i) load_lds(p, at_b[i], slot + (wv * IB + i) * 64);
  };
  run_sum(acc, oa, ob, span.stages, span.back, ring, issue_a, issue_b);
  stage_barrier();  // every wave is done reading the ring
  if (full) each_piece<true, 32>(acc, mine, out);
  else each_piece<false, 32>(acc, mine, out);
}

}  // namespace

hipError_t launch_wgrad_bf16(const GradArgs &args, hipStream_t s) {
  const GradArgs a = to_slices(args);
  const int nt = (a.N + 127) / 128, kt = (a.K + 255) / 256;
  const dim3 grid((unsigned)((long long)a.slices * a.G * nt * kt)), block(NW * 64);
  const bool f32 = a.out_dt == MOE_F32;
  const Mode mode = a.accumulate ? ADD
                    : a.slices == 1 && streams((size_t)a.G * a.N, a.K * (f32 ? 4 : 2), 1) ? STREAM
                                                                                           : PLAIN;
#define MOE_LAUNCH(M)                                                                           \
  if (f32) hipLaunchKernelGGL((wgrad_kernel<true, M>), grid, block, 0, s, a, nt, kt);           \
  else hipLaunchKernelGGL((wgrad_kernel<false, M>), grid, block, 0, s, a, nt, kt)
  if (mode == ADD) {
    MOE_LAUNCH(ADD);
  } else if (mode == STREAM) {
    MOE_LAUNCH(STREAM);
  } else {
    MOE_LAUNCH(PLAIN);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}
