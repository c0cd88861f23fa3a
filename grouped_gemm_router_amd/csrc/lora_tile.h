// lora_tile.h -- the K loops' shared parts, and the K loop of a 256 x 256
// bf16 tile.
#pragma once

#include "lora_internal.h"

namespace moe {

// A row of a slot is 8 pieces of 16 bytes, piece p of row r at place p ^ ((r
// >> 1) & 7): the loads write whole rows and the fragment reads (16 rows x one
// piece per phase) hit distinct banks.
__device__ __forceinline__ int swzb(int row, int p) { return p ^ ((row >> 1) & 7); }

// one 16-deep step's fragments of MI x NB blocks of 32 x 32
template <int MI, int NB>
struct Frag {
  bf16x8 a[MI], b[NB];
};

template <int MI, int NB>
__device__ __forceinline__ void mfma_frag(f32x16 (&acc)[MI][NB], const Frag<MI, NB> &f) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// scheduling hint: two LDS reads after each of the first multiplies, so the
// next step's fragments are requested early in this step's
template <int NMFMA, int NREAD>
__device__ __forceinline__ void interleave_mfma_ds_read() {
#pragma unroll
  for (int i = 0; i < (NREAD + 1) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, NMFMA - (NREAD + 1) / 2, 0);
}

// ---------------------------------------------------------------------------
// The 256 x 256 tile: four waves of 128 x 128, K in stages of 32.  Both
// operands move by LDS-direct loads of whole 128-byte row pieces (two stages),
// A through a ring of two such double stages, B through three: together the
// 160 KB of LDS.  The grouped GEMM's schedule (gemm_bf16.hip), for one dense
// group.
// ---------------------------------------------------------------------------
constexpr int kBig = 256, kBigK = 32;
constexpr int kBigSlot = kBig * 8;            // 16-byte pieces per operand and double stage
constexpr int kBigLoads = kBigSlot / 4 / 64;  // loads per wave and double stage
constexpr int kBigBlocks = 4;                 // 32-row (column) blocks of a wave

// acc += A B^T over KT stages (a multiple of 4).  ga / gb: the lane's sources
// of its pieces of a double stage, at K offset 0; wave wv of the four fills
// pieces [wv kBigSlot / 4, ...) of every slot.  Every wave of the workgroup
// calls it; on return no load is in flight, and other waves may still read
// the slots.
__device__ __forceinline__ void big_k_loop(f32x16 (&acc)[kBigBlocks][kBigBlocks],
                                           const uint16_t *(&ga)[kBigLoads],
                                           const uint16_t *(&gb)[kBigLoads], int KT, int wv, int fr,
                                           int fh, u32x4 *sA0, u32x4 *sA1, u32x4 *sB0, u32x4 *sB1,
                                           u32x4 *sB2) {
  constexpr int MI = kBigBlocks, NB = kBigBlocks, IL = kBigLoads;
  const int wm = wv / 2, wn = wv % 2, dma = wv * (kBigSlot / 4);
  const int KT2 = KT / 2;  // double stages
  auto read = [&](Frag<MI, NB> &f, const u32x4 *tA, const u32x4 *tB, int piece) {
    const int p = piece + fh;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = wm * (MI * 32) + i * 32 + fr;
      f.a[i] = __builtin_bit_cast(bf16x8, tA[r * 8 + swzb(r, p)]);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int r = wn * (NB * 32) + j * 32 + fr;
      f.b[j] = __builtin_bit_cast(bf16x8, tB[r * 8 + swzb(r, p)]);
    }
  };
#define MOE_BIG_ISSUE(slot, src, k0)                                                       \
  _Pragma("unroll") for (int i = 0; i < IL; ++i)                                         \
    __builtin_amdgcn_global_load_lds((const void *)((src)[i] + (k0)),                    \
                                     (lds_void *)((slot) + dma + i * 64), 16, 0, 0);
  MOE_BIG_ISSUE(sB0, gb, 0)
  MOE_BIG_ISSUE(sA0, ga, 0)
  MOE_BIG_ISSUE(sB1, gb, 2 * kBigK)
  MOE_BIG_ISSUE(sA1, ga, 2 * kBigK)
  wait_vmcnt<2 * IL>();  // double stage 0 has landed
  stage_barrier();
  Frag<MI, NB> f0, f1;
  read(f0, sA0, sB0, 0);
  // Stage s reads A from slot (s / 2) % 2 and B from slot (s / 2) % 3, half s
  // % 2.  The barrier in its middle makes stage s + 1 visible.  An odd s has
  // just read the second half of its A slot: its wait also covers this wave's
  // LDS reads, and after the barrier the slot takes A double stage (s + 3) /
  // 2.  An even s refills the B slot read last in stage s - 1 with double
  // stage s / 2 + 2.  Loads are issued in the order A(d), B(d + 1), A(d + 1),
  // B(d + 2), ...: an odd s needs A and B double stage (s + 1) / 2, after
  // which only one B was issued (IL loads may stay in flight); an even s
  // needs nothing new (2 IL).  Past the end the last double stage is loaded
  // again into slots that nobody reads, so the counts never change.
#define MOE_BIG_STAGE(tA, tB, half, nA, nB, nhalf, s, ODD, dst)                              \
  read(f1, tA, tB, 4 * (half) + 2);                                                        \
  mfma_frag<MI, NB>(acc, f0);                                                              \
  interleave_mfma_ds_read<MI * NB, MI + NB>();                                             \
  if (ODD) { wait_vmcnt_lgkm0<IL>(); } else { wait_vmcnt<2 * IL>(); }                      \
  stage_barrier();                                                                         \
  if (ODD) { MOE_BIG_ISSUE(dst, ga, min(((s) + 3) / 2, KT2 - 1) * 2 * kBigK) }             \
  else { MOE_BIG_ISSUE(dst, gb, min((s) / 2 + 2, KT2 - 1) * 2 * kBigK) }                   \
  read(f0, nA, nB, 4 * (nhalf));                                                           \
  mfma_frag<MI, NB>(acc, f1);                                                              \
  interleave_mfma_ds_read<MI * NB, MI + NB>();
  // four stages on the B slots b0 (now), b1 and b2
#define MOE_BIG_FOUR(kt, b0, b1, b2)                               \
  MOE_BIG_STAGE(sA0, b0, 0, sA0, b0, 1, (kt), 0, b2)               \
  MOE_BIG_STAGE(sA0, b0, 1, sA1, b1, 0, (kt) + 1, 1, sA0)          \
  MOE_BIG_STAGE(sA1, b1, 0, sA1, b1, 1, (kt) + 2, 0, b0)           \
  MOE_BIG_STAGE(sA1, b1, 1, sA0, b2, 0, (kt) + 3, 1, sA1)
  int kt = 0;
  for (; kt + 12 <= KT; kt += 12) {  // one period of both rings
    MOE_BIG_FOUR(kt, sB0, sB1, sB2)
    MOE_BIG_FOUR(kt + 4, sB2, sB0, sB1)
    MOE_BIG_FOUR(kt + 8, sB1, sB2, sB0)
  }
  if (kt + 4 <= KT) {  // KT % 12 is 0, 4 or 8
    MOE_BIG_FOUR(kt, sB0, sB1, sB2)
    if (kt + 8 <= KT) {
      MOE_BIG_FOUR(kt + 4, sB2, sB0, sB1)
    }
  }
  wait_vmcnt<0>();  // no LDS-direct load may still be landing when the tile ends
#undef MOE_BIG_FOUR
#undef MOE_BIG_STAGE
#undef MOE_BIG_ISSUE
}

}  // namespace moe
