// gemm_bf16_tile.h -- the K loop of a BM x 256 bf16 output tile through LDS
// rings, shared by the grouped GEMM (gemm_bf16.hip, which documents the
// design) and the shared projection with adapters (lora_expand.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int BM_MAX = 256, BN = 256, BK = 32;
constexpr int PIECES = BK / 8;             // 16-byte pieces per operand row and stage
constexpr int PIECES_B = 2 * PIECES;       // 128-byte row pieces covering two stages
constexpr int SLOTS_A2MAX = BM_MAX * PIECES_B; // 16-byte slots per A double stage (32 KB)
constexpr int SLOTS_B2 = BN * PIECES_B;    // 16-byte slots per B double stage (32 KB)

__device__ __forceinline__ int swzb(int row, int p) { return p ^ ((row >> 1) & 7); }

// B-tile row of wave column wn (of NWN), 32-row block nb
template <bool SWIGLU, int NWN>
__device__ __forceinline__ int b_row(int wn, int nb) {
  if (SWIGLU) {
    constexpr int per = 128 / NWN;  // gate rows per wave column
    constexpr int half = per / 32;  // 32-row blocks in each half
    return ((nb >= half) ? 128 : 0) + wn * per + (nb % half) * 32;
  }
  return wn * (BN / NWN) + nb * 32;
}

template <int MI, int NB>
struct Frag {
  bf16x8 a[MI];
  bf16x8 b[NB];
};

// live: the wave's 32-row blocks that hold rows of the group (wave-uniform;
// MI except in the short SwiGLU tiles that skip); blocks past the group end
// are neither read from LDS nor multiplied
template <bool SWIGLU, int MI, int NB, int NWN>
__device__ __forceinline__ void read_frag(Frag<MI, NB> &f, const u32x4 *tA, const u32x4 *tB,
                                          int ks, int par, int wm, int wn, int fr, int fh,
                                          int live) {
  const int pc = ks * 2 + fh;
  const int pb = par * PIECES + pc;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    if (mi >= live) break;
    const int r = wm * (MI * 32) + mi * 32 + fr;
    f.a[mi] = __builtin_bit_cast(bf16x8, tA[r * PIECES_B + swzb(r, pb)]);
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = b_row<SWIGLU, NWN>(wn, nb) + fr;
    f.b[nb] = __builtin_bit_cast(bf16x8, tB[r * PIECES_B + swzb(r, pb)]);
  }
}

template <int MI, int NB>
__device__ __forceinline__ void mfma_frag(f32x16 (&acc)[MI][NB], const Frag<MI, NB> &f,
                                          int live) {
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
    if (mi < live)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        acc[mi][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[mi], f.b[nb], acc[mi][nb], 0, 0, 0);
}

// scheduling hint: two LDS reads after each of the first MFMAs, so the
// next 16-deep step's fragments are requested early in this step's MFMAs
// (measured against one read per MFMA: Mixtral-shape down 0.90 -> 0.88 ms,
// gate/up unchanged; all reads first or three per MFMA were no better)
template <int NMFMA, int NREAD>
__device__ __forceinline__ void interleave_mfma_ds_read() {
#pragma unroll
  for (int i = 0; i < (NREAD + 1) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, NMFMA - (NREAD + 1) / 2, 0);
}

// acc += A B^T of one tile over KT steps of BK (a multiple of 4), through the
// A ring of two and the B ring of three double-stage slots.  ga / gb: the
// lane's sources of its IA / IB pieces per double stage, at K offset 0;
// dma_a / dma_b: where lane 0's pieces land in a slot (in 16-byte units).
// Every wave of the workgroup calls it; on return no load is in flight, and
// other waves may still read the slots.
template <bool SWIGLU, int MI, int NB, int NWN, int IA, int IB>
__device__ __forceinline__ void tile_k_loop(f32x16 (&acc)[MI][NB], const uint16_t *(&ga)[IA],
                                            const uint16_t *(&gb)[IB], int KT, int dma_a, int dma_b,
                                            int wm, int wn, int fr, int fh, int live, u32x4 *sA0,
                                            u32x4 *sA1, u32x4 *sB0, u32x4 *sB1, u32x4 *sB2) {
  constexpr int NM = MI * NB;                 // MFMAs per 16-deep step
  constexpr int NR = MI + NB;                 // fragment reads per 16-deep step
#define MOE_ISSUE_A(dA, k0)                                                                \
  _Pragma("unroll") for (int i = 0; i < IA; ++i)                                          \
    __builtin_amdgcn_global_load_lds((const void *)(ga[i] + (k0)),                        \
                                     (lds_void *)((dA) + dma_a + i * 64), 16, 0, 0);
#define MOE_ISSUE_B(dB, k0)                                                                \
  _Pragma("unroll") for (int i = 0; i < IB; ++i)                                          \
    __builtin_amdgcn_global_load_lds((const void *)(gb[i] + (k0)),                        \
                                     (lds_void *)((dB) + dma_b + i * 64), 16, 0, 0);

  const int KT2 = KT / 2;  // double stages
  MOE_ISSUE_B(sB0, 0);
  MOE_ISSUE_A(sA0, 0);
  MOE_ISSUE_B(sB1, 2 * BK);
  MOE_ISSUE_A(sA1, 2 * BK);
  wait_vmcnt<IA + IB>();  // A and B double stage 0 landed
  stage_barrier();
  Frag<MI, NB> f0, f1;
  read_frag<SWIGLU, MI, NB, NWN>(f0, sA0, sB0, 0, 0, wm, wn, fr, fh, live);

  // One stage s: A from double-stage slot (s / 2) % 2, B from slot (s / 2) %
  // 3, half s % 2.  The barrier in the middle makes stage s+1 visible.  An
  // odd s has just read the second half of its A slot: its wait also covers
  // this wave's LDS reads, and after the barrier the slot takes A double
  // stage (s + 3) / 2.  An even s frees B slot (s/2 + 2) % 3 (read last in
  // stage s-1) and refills it with double stage s/2 + 2.  Loads are issued
  // in the order A(d), B(d+1), A(d+1), B(d+2), ...: an odd s needs A and B
  // double stage (s+1)/2, after which only B((s+1)/2 + 1) was issued (IB
  // loads may stay in flight); an even s needs nothing new (IB + IA).  Past
  // the end the last double stage is re-loaded into slots nobody reads, so
  // the counts never change.
#define MOE_STAGE(tA, tB, tp, nA, nB, np, s, ODD, dA, dB)                                   \
  read_frag<SWIGLU, MI, NB, NWN>(f1, tA, tB, 1, tp, wm, wn, fr, fh, live);                   \
  mfma_frag<MI, NB>(acc, f0, live);                                                           \
  interleave_mfma_ds_read<NM, NR>();                                                          \
  if (ODD) { wait_vmcnt_lgkm0<IB>(); } else { wait_vmcnt<IB + IA>(); }                        \
  stage_barrier();                                                                            \
  if (ODD) { MOE_ISSUE_A(dA, min(((s) + 3) / 2, KT2 - 1) * 2 * BK); }                         \
  else { MOE_ISSUE_B(dB, min((s) / 2 + 2, KT2 - 1) * 2 * BK); }                               \
  read_frag<SWIGLU, MI, NB, NWN>(f0, nA, nB, 0, np, wm, wn, fr, fh, live);                   \
  mfma_frag<MI, NB>(acc, f1, live);                                                           \
  interleave_mfma_ds_read<NM, NR>();

// stage s: A slot (s/2)%2, B slot (s/2)%3, half s%2; odd s refills A slot
// ((s+3)/2)%2 (the one just read), even s refills B slot (s/2+2)%3
#define MOE_STAGES_0_3(kt)                                         \
  MOE_STAGE(sA0, sB0, 0, sA0, sB0, 1, (kt), 0, sA0, sB2)           \
  MOE_STAGE(sA0, sB0, 1, sA1, sB1, 0, (kt) + 1, 1, sA0, sB2)       \
  MOE_STAGE(sA1, sB1, 0, sA1, sB1, 1, (kt) + 2, 0, sA1, sB0)       \
  MOE_STAGE(sA1, sB1, 1, sA0, sB2, 0, (kt) + 3, 1, sA1, sB0)
#define MOE_STAGES_4_7(kt)                                         \
  MOE_STAGE(sA0, sB2, 0, sA0, sB2, 1, (kt) + 4, 0, sA0, sB1)       \
  MOE_STAGE(sA0, sB2, 1, sA1, sB0, 0, (kt) + 5, 1, sA0, sB1)       \
  MOE_STAGE(sA1, sB0, 0, sA1, sB0, 1, (kt) + 6, 0, sA1, sB2)       \
  MOE_STAGE(sA1, sB0, 1, sA0, sB1, 0, (kt) + 7, 1, sA1, sB2)
#define MOE_STAGES_8_11(kt)                                        \
  MOE_STAGE(sA0, sB1, 0, sA0, sB1, 1, (kt) + 8, 0, sA0, sB0)       \
  MOE_STAGE(sA0, sB1, 1, sA1, sB2, 0, (kt) + 9, 1, sA0, sB0)       \
  MOE_STAGE(sA1, sB2, 0, sA1, sB2, 1, (kt) + 10, 0, sA1, sB1)      \
  MOE_STAGE(sA1, sB2, 1, sA0, sB0, 0, (kt) + 11, 1, sA1, sB1)

  int kt = 0;
  for (; kt + 12 <= KT; kt += 12) {
    MOE_STAGES_0_3(kt)
    MOE_STAGES_4_7(kt)
    MOE_STAGES_8_11(kt)
  }
  if (kt + 4 <= KT) {  // KT % 12 is 0, 4 or 8
    MOE_STAGES_0_3(kt)
    if (kt + 8 <= KT) {
      MOE_STAGES_4_7(kt)
    }
  }
  wait_vmcnt<0>();  // no LDS-direct load may still be landing when the tile ends
#undef MOE_STAGES_0_3
#undef MOE_STAGES_4_7
#undef MOE_STAGES_8_11
#undef MOE_STAGE
#undef MOE_ISSUE_A
#undef MOE_ISSUE_B
}

}  // namespace moe
