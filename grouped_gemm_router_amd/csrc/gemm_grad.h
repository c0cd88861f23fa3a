// gemm_grad.h -- what the products' gradients on bf16 MFMA (gemm_dgrad.hip,
// gemm_wgrad.hip) share.
//
// The forward product reads both operands along the sum (C = A B^T).  Here
// dgrad's weights and both of wgrad's operands lie across it: their rows are
// terms of the sum.  Such a tile goes to LDS as it lies in memory, in pieces of
// whole rows by LDS-direct loads, and is turned on the way to the registers by
// ds_read_b64_tr_b16, which hands each lane four terms of one column; no
// operand is transposed in memory.
#pragma once

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
// out.finish<FULL>(row, first column, out.begin<FULL>(row, column), values)
// for pieces of Out::COLS columns, row and column of the tile; FULL: the whole
// tile lies inside the output.  The blocks are held transposed (the second
// operand is the instruction's first): lane l has output row l % 32 and
// register r output column 8 (r / 4) + 4 (l / 32) + r % 4, so four registers
// are 16 bytes of one row.  A wave writes and reads its own array only, so no
// wave waits for another: 16-byte piece p of row r lies at p ^ (r & 15), which
// spreads both the writes (32 rows of one piece) and the reads (whole rows)
// over all banks.
// What begin() loads is asked for DEPTH batches ahead, behind the stores of the
// batch then done: a load behind a store is not back before the store is, and
// stores take microseconds (asked for one batch ahead, behind the stores that it
// then waited for, a tile's epilogue took 10 us).
template <bool FULL, int ROWS, int MI, int NB, class Out>
__device__ __forceinline__ void each_piece(const f32x16 (&acc)[MI][NB], u32x4 *mine, const Out &out) {
  constexpr int W = NB * 32, PPR = W / 4;      // columns and 16-byte pieces a row
  constexpr int C = Out::COLS;                 // columns a lane takes: 16 bytes of the output
  constexpr int CH = MI % (ROWS / 32) == 0 ? ROWS / 32 : 1;  // 32-row blocks at a time
  constexpr int ALL = CH * 32 * (W / C) / 64;  // pieces a lane and chunk
  constexpr int UN = Out::UN, DEPTH = Out::DEPTH;  // pieces a batch, batches asked for ahead
  constexpr int BATCHES = ALL / UN * (MI / CH);
  static_assert(ALL % UN == 0 && MI % CH == 0, "whole batches");
  const int lane = lane_id(), wv = threadIdx.x / kWave;
  const int row0 = wv / 2 * (MI * 32), col0 = wv % 2 * W;
  typename Out::Held held[DEPTH][UN];
  auto begin = [&](int b) {
#pragma unroll
    for (int n = 0; n < UN; ++n) {
      const int id = (b * UN + n) * 64 + lane;  // (chunks follow each other row by row)
      held[b % DEPTH][n] = out.template begin<FULL>(row0 + id / (W / C), col0 + id % (W / C) * C);
    }
  };
#pragma unroll
  for (int b = 0; b < (DEPTH < BATCHES ? DEPTH : BATCHES); ++b) begin(b);
#pragma unroll
  for (int b = 0; b < BATCHES; ++b) {
    if (b % (ALL / UN) == 0) {
      const int i0 = b / (ALL / UN) * CH;
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
    }
    float v[UN][C];
#pragma unroll
    for (int n = 0; n < UN; ++n) {
      const int id = (b % (ALL / UN) * UN + n) * 64 + lane;
      const int row = id / (W / C), p = id % (W / C) * (C / 4);
#pragma unroll
      for (int h = 0; h < C / 4; ++h)
        *reinterpret_cast<u32x4 *>(v[n] + 4 * h) = mine[row * PPR + ((p + h) ^ (row & 15))];
    }
#pragma unroll
    for (int n = 0; n < UN; ++n) {
      const int id = (b * UN + n) * 64 + lane;
      out.template finish<FULL>(row0 + id / (W / C), col0 + id % (W / C) * C, held[b % DEPTH][n], v[n]);
    }
    if (b + DEPTH < BATCHES) begin(b + DEPTH);
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

// 16 bytes of outputs; STREAM: past the caches
template <bool STREAM>
__device__ __forceinline__ void store16(void *p, const u32x4 &o) {
  if constexpr (STREAM) __builtin_nontemporal_store(o, static_cast<u32x4 *>(p));
  else *static_cast<u32x4 *>(p) = o;
}

// 8 values rounded to bf16, or 4 as they are
template <bool STREAM>
__device__ __forceinline__ void store(uint16_t *p, const float *v) {
  bf16x8v o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];  // round to nearest even
  store16<STREAM>(p, __builtin_bit_cast(u32x4, o));
}
template <bool STREAM>
__device__ __forceinline__ void store(float *p, const float *v) {
  const f32x4 o = {v[0], v[1], v[2], v[3]};
  store16<STREAM>(p, __builtin_bit_cast(u32x4, o));
}

// Outputs that the 256 MB last-level cache cannot keep for their reader go past
// it, where rows are whole 128-byte lines (64 groups' weights of 1408 x 2048 in
// bf16 271 -> 210 us, 14336 x 4096 1013 -> 980; a line that two stores fill
// costs more that way: 1416 x 2056 in fp32 434 -> 474).
inline bool streams(size_t rows, int row_bytes, int arrays) {
  return row_bytes % 128 == 0 && rows * row_bytes * arrays > (256u << 20);
}

}  // namespace
