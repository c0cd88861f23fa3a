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

constexpr int NW = 4;   // waves, 2 x 2

// what loads behind the last term of a sum read
__device__ u32x4 g_zeros[1];

// s_waitcnt lgkmcnt(0) alone: this wave's LDS writes are done
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// 16-byte pieces of `terms` terms of `width` outputs
constexpr int pieces(int width, int terms) { return width * terms / 8; }

// An operand whose rows are terms: T rows of W columns (16-byte pieces of 8).
// The 64-byte blocks of a row are stored at block ^ (row & 3): the four rows
// that a transposing read takes then lie in different banks.
// fragment of 32 columns: terms 8 (lane / 32) .. + 7 of a 16-term step
template <int W, int T>
struct CrossOperand {
  static constexpr int NB = W / 64;                    // 32-column blocks a wave
  static constexpr int IL = pieces(W, T) / 64 / NW;    // loads a wave
  static constexpr int READS = 2 * NB;                 // LDS reads a 16-term step
  static constexpr int RPL = 64 / (W / 8);             // rows a load
  uint32_t at[NB];  // byte offset of each of the wave's blocks
  __device__ __forceinline__ void init(int half, int lane) {
    const int kk = (lane % 16) / 4;
    const int row = 8 * (lane / 32) + kk;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      at[b] = row * (2 * W) + ((half * NB + b) ^ kk) * 64 + ((lane / 16) & 1) * 32 + (lane % 4) * 8;
  }
  // block b of step ks
  __device__ __forceinline__ bf16x8 read(const u32x4 *slot, int b, int ks) const {
    const char *p = reinterpret_cast<const char *>(slot) + at[b] + ks * (16 * 2 * W);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * W));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // the first z terms as zeros
  static __device__ __forceinline__ void zero(u32x4 *slot, int z) {
    for (int i = threadIdx.x; i < z * (W / 8); i += NW * 64) slot[i] = u32x4{};
  }
  // row and first column of what load i of wave wv brings this lane
  static __device__ __forceinline__ int load_row(int wv, int i, int lane) {
    return (wv * IL + i) * RPL + lane / (W / 8);
  }
  static __device__ __forceinline__ int load_col(int row, int lane) {
    return ((lane % (W / 8)) ^ ((row & 3) << 2)) * 8;
  }
};

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

template <int MI, int NB>
struct Frag {
  bf16x8 a[MI], b[NB];
};

template <int MI, int NB, class OpA, class OpB>
__device__ __forceinline__ void read_frag(Frag<MI, NB> &f, const OpA &oa, const OpB &ob,
                                          const u32x4 *sa, const u32x4 *sb, int ks) {
#pragma unroll
  for (int i = 0; i < MI; ++i) f.a[i] = oa.read(sa, i, ks);
#pragma unroll
  for (int i = 0; i < NB; ++i) f.b[i] = ob.read(sb, i, ks);
}

template <int MI, int NB>
__device__ __forceinline__ void mfma_frag(f32x16 (&acc)[MI][NB], const Frag<MI, NB> &f) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
}

// Scheduling hint for half a stage: its LDS reads go between the first of its
// MFMAs, two each, so that they are back when the next half needs them, then
// its loads, one each.
template <int NMFMA, int NREAD, int NLOAD>
__device__ __forceinline__ void interleave() {
  constexpr int R = (NREAD + 1) / 2 < NMFMA ? (NREAD + 1) / 2 : NMFMA;
  constexpr int PER = (NREAD + R - 1) / R;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
  }
  constexpr int V = NLOAD < NMFMA - R ? NLOAD : NMFMA - R;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
  if (NMFMA - R - V > 0) __builtin_amdgcn_sched_group_barrier(0x008, NMFMA - R - V, 0);
}

template <class OpA, class OpB>
__device__ __forceinline__ void zero_terms(u32x4 *sa, u32x4 *sb, int z) {
  OpA::zero(sa, z);
  OpB::zero(sb, z);
  wait_lgkm0();
  stage_barrier();
}

// The rings' slots are arrays of their own: the compiler then knows that a
// read of one does not wait for loads into another.  In both, a sum's stages
// past the last load the last one again, so that the counts of loads in
// flight never change, and the last stage's first z terms are ones that the
// stage before has had: they are overwritten with zeros, in both operands (an
// infinity times zero would be NaN).

// wgrad's ring: three stages of 32 terms of both operands, 24 KB each, so that
// two workgroups share a CU.  Stage s in slot `cur`: its second half is read
// while the first is multiplied; then stage s + 1 has landed for every wave,
// and `cur`, which every wave has read, takes stage s + 3.
struct Ring3 {
  u32x4 *s0, *s1, *s2;
};
constexpr int SB = pieces(256, 32);  // where the second operand begins in a slot

#define MOE_HALF_0(cur)                                \
  read_frag(f1, oa, ob, r.cur, r.cur + SB, 1);         \
  mfma_frag(acc, f0);                                  \
  interleave<MI * NB, OpA::READS + OpB::READS, 0>();   \
  __builtin_amdgcn_sched_barrier(0);                   \
  wait_vmcnt_lgkm0<IL>();                              \
  stage_barrier();
#define MOE_HALF_1(s, cur, nxt)                        \
  issue((s) + 3, r.cur);                               \
  read_frag(f0, oa, ob, r.nxt, r.nxt + SB, 0);         \
  mfma_frag(acc, f1);                                  \
  interleave<MI * NB, OpA::READS + OpB::READS, IL>();
#define MOE_STAGE(s, cur, nxt)                         \
  MOE_HALF_0(cur)                                      \
  MOE_HALF_1(s, cur, nxt)
#define MOE_LAST_STAGES(s, cur, nxt)                   \
  MOE_HALF_0(cur)                                      \
  if (z && (s) + 2 == stages) zero_terms<OpA, OpB>(r.nxt, r.nxt + SB, z); \
  MOE_HALF_1(s, cur, nxt)
template <int MI, int NB, class OpA, class OpB, class Issue>
__device__ __forceinline__ void run_sum(f32x16 (&acc)[MI][NB], const OpA &oa, const OpB &ob,
                                        int stages, int z, const Ring3 &r, Issue issue) {
  constexpr int IL = OpA::IL + OpB::IL;
  issue(0, r.s0);
  issue(1, r.s1);
  issue(2, r.s2);
  wait_vmcnt<2 * IL>();
  stage_barrier();
  if (z && stages == 1) zero_terms<OpA, OpB>(r.s0, r.s0 + SB, z);
  Frag<MI, NB> f0, f1;
  read_frag(f0, oa, ob, r.s0, r.s0 + SB, 0);
  int s = 0;
  for (; s + 4 < stages; s += 3) {
    MOE_STAGE(s, s0, s1)
    MOE_STAGE(s + 1, s1, s2)
    MOE_STAGE(s + 2, s2, s0)
  }
  if (s < stages) {
    MOE_LAST_STAGES(s, s0, s1)
    if (s + 1 < stages) {
      MOE_LAST_STAGES(s + 1, s1, s2)
      if (s + 2 < stages) {
        MOE_LAST_STAGES(s + 2, s2, s0)
        if (s + 3 < stages) {
          MOE_LAST_STAGES(s + 3, s0, s1)
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
  MOE_STEP(sa, sb, 1, f0, f1, OpB::IL, issue_b((d) + 2, r.pb)) \
  MOE_STEP(sa, sb, 2, f1, f0, 0, )                          \
  MOE_STEP(sa, sb, 3, f0, f1, 0, )                          \
  wait_vmcnt_lgkm0<OpB::IL>();                              \
  stage_barrier();                                          \
  if (check && z && (d) + 2 == stages) zero_terms<OpA, OpB>(r.na, r.nb, z); \
  MOE_STEP(na, nb, 0, f1, f0, OpA::IL, issue_a((d) + 2, r.sa))
template <int MI, int NB, class OpA, class OpB, class IssueA, class IssueB>
__device__ __forceinline__ void run_sum(f32x16 (&acc)[MI][NB], const OpA &oa, const OpB &ob,
                                        int stages, int z, const Ring23 &r, IssueA issue_a,
                                        IssueB issue_b) {
  issue_b(0, r.b0);
  issue_a(0, r.a0);
  issue_b(1, r.b1);
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

// LDS-direct load of lane i's 16 bytes at base + at to l + 16 i; base is the
// wave's, so that only `at` needs a register and no arithmetic
__device__ __forceinline__ void load_lds(const uint16_t *base, uint32_t at, u32x4 *l) {
  __builtin_amdgcn_global_load_lds((const void *)(reinterpret_cast<const char *>(base) + at),
                                   (lds_void *)l, 16, 0, 0);
}

// live ? p : zeros, without a branch (written as a choice of addresses, the
// compiler makes two loads of it, each under its own lanes)
__device__ __forceinline__ const uint16_t *or_zeros(bool live, const uint16_t *p) {
  const uint64_t z = reinterpret_cast<uint64_t>(g_zeros), m = live ? ~0ull : 0ull;
  return reinterpret_cast<const uint16_t *>(z ^ ((z ^ reinterpret_cast<uint64_t>(p)) & m));
}

// The stages of BK terms of a sum of `terms` terms: all full, the last one
// moved back to end at the last term (its first `back` terms are then the
// stage before's).  A sum shorter than a stage has one, of which each term is
// loaded or zero.
template <int BK>
struct Span {
  int terms, stages, back;
  __device__ __forceinline__ explicit Span(int n)
      : terms(n), stages((n + BK - 1) / BK), back(n > BK ? stages * BK - n : 0) {}
  __device__ __forceinline__ int first(int st) const {  // (stages past the last: the last)
    return min(st * BK, terms - BK);
  }
};

// The wave's part of the tile, MI x NB blocks of 32 x 32 sums, through LDS:
// out.finish(row, first column, out.begin(row, column), 8 values) for pieces
// of 8 columns, row and column of the tile.  The blocks are held transposed (the second operand is the
// instruction's first): lane l has output row l % 32 and register r output
// column 8 (r / 4) + 4 (l / 32) + r % 4, so four registers are 16 bytes of one row.
// A wave writes and reads its own array only, so no wave waits for another:
// 16-byte piece p of row r lies at p ^ (r & 15), which spreads both the writes
// (32 rows of one piece) and the reads (whole rows) over all banks.
template <int ROWS, int MI, int NB, class Out>
__device__ __forceinline__ void each_piece(const f32x16 (&acc)[MI][NB], u32x4 *mine, const Out &out) {
  constexpr int W = NB * 32, PPR = W / 4;      // columns and 16-byte pieces a row
  constexpr int CH = MI < ROWS / 32 ? MI : ROWS / 32;  // 32-row blocks at a time
  constexpr int ALL = CH * 32 * (W / 8) / 64;  // pieces of 8 columns a lane
  constexpr int UN = ALL < 8 ? ALL : 8;        // of which in flight
  const int lane = lane_id(), wv = threadIdx.x / kWave;
  const int row0 = wv / 2 * (MI * 32), col0 = wv % 2 * W;
#pragma unroll
  for (int i0 = 0; i0 < MI; i0 += CH) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16 &c = acc[i0 + i][j];
          const int row = i * 32 + lane % 32, p = j * 8 + q * 2 + lane / 32;
          const f32x4 v = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
          mine[row * PPR + (p ^ (row & 15))] = __builtin_bit_cast(u32x4, v);
        }
#pragma unroll
    for (int n0 = 0; n0 < ALL; n0 += UN) {
      typename Out::Held held[UN];
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        const int id = (n0 + n) * 64 + lane;
        held[n] = out.begin(row0 + i0 * 32 + id / (W / 8), col0 + id % (W / 8) * 8);
      }
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        const int id = (n0 + n) * 64 + lane;
        const int row = id / (W / 8), p = id % (W / 8) * 2;
        float v[8];
        *reinterpret_cast<u32x4 *>(v) = mine[row * PPR + (p ^ (row & 15))];
        *reinterpret_cast<u32x4 *>(v + 4) = mine[row * PPR + ((p + 1) ^ (row & 15))];
        out.finish(row0 + i0 * 32 + row, col0 + id % (W / 8) * 8, held[n], v);
      }
    }
  }
}

__device__ __forceinline__ void widen8(const u32x4 &raw, float v[8]) {
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
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), reinterpret_cast<u32x4 *>(p));
}

__device__ __forceinline__ void store8(float *p, const float v[8]) {
  __builtin_nontemporal_store(*reinterpret_cast<const f32x4 *>(v), reinterpret_cast<f32x4 *>(p));
  __builtin_nontemporal_store(*reinterpret_cast<const f32x4 *>(v + 4),
                              reinterpret_cast<f32x4 *>(p + 4));
}

// One dgrad tile of at most BM rows and 256 columns.  SHORT: N is less than a
// stage.
template <int BM, bool SHORT, class Out>
__device__ __forceinline__ void dgrad_tile(const GradArgs &a, const Tile &tile, const Ring23 &ring) {
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
  // both products in one run of stages, or, where each ends inside a stage, one
  // after the other
  const int parts = a.dC2 && span.back ? 2 : 1;
  const int stages = a.dC2 && !span.back ? 2 * span.stages : span.stages;
  int part = 0;
  auto issue_a = [&](int st, u32x4 *slot) {
    st = min(st, stages - 1);
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
  auto issue_b = [&](int st, u32x4 *slot) {
    st = min(st, stages - 1);
    const bool second = part || st >= span.stages;
    st -= second && !part ? span.stages : 0;
    const uint16_t *const p = static_cast<const uint16_t *>(second ? a.B2 : a.B) + first_b +
                              (size_t)(SHORT ? 0 : span.first(st)) * a.ldb;
#pragma unroll
    for (int i = 0; i < IB; ++i) {
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
    run_sum(acc, oa, ob, stages, span.back, ring, issue_a, issue_b);
    stage_barrier();  // every wave is done reading the ring
  }
  const Out out = {a, tile.m0, tile.mend, k0};
  each_piece<64>(acc, wv == 0 ? ring.a0 : wv == 1 ? ring.a1 : wv == 2 ? ring.b0 : ring.b1, out);
}

// silu's factor with the hardware's exp2 and reciprocal (each within 1 ulp,
// far below the bf16 rounding)
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

// what becomes of the sums of a dgrad tile
template <bool SWIGLU, bool OUT_F32>
struct DgradOut {
  const GradArgs &a;
  int m0, mend, k0;
  struct Held {
    u32x4 gate, up;
  };
  __device__ __forceinline__ Held begin(int r, int c) const {
    Held x{};
    if constexpr (SWIGLU) {
      if (m0 + r < mend && k0 + c < a.K) {
        const size_t at = (size_t)(m0 + r) * a.K + k0 + c;
        x.gate = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.gate) + at);
        x.up = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.up) + at);
      }
    }
    return x;
  }
  __device__ __forceinline__ void finish(int r, int c, const Held &x, const float *v) const {
    if (m0 + r >= mend || k0 + c >= a.K) return;
    const size_t at = (size_t)(m0 + r) * a.K + k0 + c;
    if constexpr (SWIGLU) {
      float z[8], u[8], dg[8], du[8], h[8];
      widen8(x.gate, z);
      widen8(x.up, u);
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
  }
};

template <bool SWIGLU, bool OUT_F32, bool SHORT>
__global__ __launch_bounds__(NW * 64, 1) void dgrad_kernel(const GradArgs a, int nt) {
  constexpr int SLOT = pieces(256, 64);
  __shared__ u32x4 a0[SLOT], a1[SLOT], b0[SLOT], b1[SLOT], b2[SLOT];
  const Ring23 ring = {a0, a1, b0, b1, b2};
  // (the scheduler's result lies in a slot that the ring fills later)
  const Sched sc = sched_lookup(a.offsets, a.G, a.rows, 256, nt, kTileChunk, false,
                                reinterpret_cast<int *>(b2),
                                [](int total) { return tile_of_workgroup(blockIdx.x, total); });
  if (sc.L < 0) return;
  const Tile tile = sc.tile;
  typedef DgradOut<SWIGLU, OUT_F32> Out;
  const int rows = tile.mend - tile.m0;
  if (rows > 128) dgrad_tile<256, SHORT, Out>(a, tile, ring);
  else if (rows > 64) dgrad_tile<128, SHORT, Out>(a, tile, ring);
  else dgrad_tile<64, SHORT, Out>(a, tile, ring);
}

constexpr int kStrip = 6;

// what becomes of the sums of a wgrad tile
template <bool OUT_F32>
struct WgradOut {
  const GradArgs &a;
  int n0, k0;
  size_t first;  // row of the group's first
  float *part;
  struct Held {
    u32x4 x, y;
  };
  __device__ __forceinline__ Held begin(int r, int c) const {
    Held h{};
    if (a.accumulate && !part && n0 + r < a.N && k0 + c < a.K) {
      const size_t at = (first + n0 + r) * a.K + k0 + c;
      if constexpr (OUT_F32) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const float *>(a.out) + at);
        h.x = p[0];
        h.y = p[1];
      } else {
        h.x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.out) + at);
      }
    }
    return h;
  }
  __device__ __forceinline__ void finish(int r, int c, const Held &h, const float *v) const {
    if (n0 + r >= a.N || k0 + c >= a.K) return;
    const size_t at = (first + n0 + r) * a.K + k0 + c;
    if (part) {
      store8(part + at, v);
      return;
    }
    float o[8];
    if constexpr (OUT_F32) {
      *reinterpret_cast<u32x4 *>(o) = h.x;
      *reinterpret_cast<u32x4 *>(o + 4) = h.y;
    } else {
      widen8(h.x, o);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += v[i];  // (zero where nothing is added to)
    if constexpr (OUT_F32) store8(static_cast<float *>(a.out) + at, o);
    else store8(static_cast<uint16_t *>(a.out) + at, o);
  }
};

// Tiles of 256 x 128 weights.
template <bool OUT_F32>
__global__ __launch_bounds__(NW * 64, 2) void wgrad_kernel(const GradArgs a, int nt, int kt) {
  constexpr int BN = 128, SLOT = SB + pieces(BN, 32);
  typedef CrossOperand<256, 32> OpA;
  typedef CrossOperand<BN, 32> OpB;
  constexpr int IA = OpA::IL, IB = OpB::IL;
  __shared__ u32x4 s0[SLOT], s1[SLOT], s2[SLOT];
  const Ring3 ring = {s0, s1, s2};
  int *const s_rows = reinterpret_cast<int *>(s2);  // until the ring starts
  const int all = nt * kt * a.G * a.slices;
  int w = blockIdx.x;
  if (w < all / 256 * 256) w = w / 256 * 256 + (w % 8) * 32 + w % 256 / 8;
  const int per = nt * kt;
  const int t = w % per;
  w /= per;
  const int strip = t / (kStrip * kt), wide = min(kStrip, nt - strip * kStrip);
  const int in = t - strip * kStrip * kt;
  const int k0 = in / wide * BN;
  const int n0 = (strip * kStrip + in % wide) * 256;
  const int g = w % a.G, slice = w / a.G;
  group_rows(a.offsets, a.rows, g, s_rows);
  int r0 = s_rows[0], r1 = s_rows[1];
  __syncthreads();
  if (a.part) slice_rows(&r0, &r1, slice, a.slices);
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
  u32x4 *const mine = wv == 0 ? s0 : wv == 1 ? s1 : wv == 2 ? s2 : s2 + SLOT / 2;
  const WgradOut<OUT_F32> out = {a, n0, k0, (size_t)g * a.N,
                                 a.part ? a.part + (size_t)slice * a.G * a.N * a.K : nullptr};
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
    each_piece<32>(acc, mine, out);
    return;
  }
  auto issue = [&](int st, u32x4 *slot) {
    const int t0 = span.first(min(st, span.stages - 1));
    const uint16_t *const pa = dC + (size_t)t0 * a.N, *const pb = A + (size_t)t0 * a.K;
#pragma unroll
    for (int i = 0; i < IA; ++i) load_lds(pa, at_a[i], slot + (wv * IA + i) * 64);
#pragma unroll
    for (int i = 0; i < IB; ++i) load_lds(pb, at_b[i], slot + SB + (wv * IB + i) * 64);
  };
  run_sum(acc, oa, ob, span.stages, span.back, ring, issue);
  stage_barrier();  // every wave is done reading the ring
  each_piece<32>(acc, mine, out);
}

}  // namespace

hipError_t launch_dgrad_bf16(const GradArgs &a, hipStream_t s) {
  const int nt = (a.K + 255) / 256;
  const dim3 grid((unsigned)(host_row_tile_bound(a.rows, a.G, 256) * (long long)nt)), block(NW * 64);
  const bool brief = a.N < 64;
#define MOE_LAUNCH(SW, F32)                                                                 \
  if (brief) hipLaunchKernelGGL((dgrad_kernel<SW, F32, true>), grid, block, 0, s, a, nt);   \
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
  const int nt = (a.N + 255) / 256, kt = (a.K + 127) / 128;
  const dim3 grid((unsigned)((long long)a.slices * a.G * nt * kt)), block(NW * 64);
  if (a.out_dt == MOE_F32) hipLaunchKernelGGL(wgrad_kernel<true>, grid, block, 0, s, a, nt, kt);
  else hipLaunchKernelGGL(wgrad_kernel<false>, grid, block, 0, s, a, nt, kt);
  return hipGetLastError();
}
