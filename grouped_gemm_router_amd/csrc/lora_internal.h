// lora_internal.h -- what the translation units of the low-rank adapters
// share.
#pragma once

#include "moe_internal.h"
#include "../../include/moe_lora.h"

namespace moe {

// rows of a tile of the sorted shrink, and the most slices that it cuts K into
constexpr int kShrinkTile = 64, kShrinkSlices = 8;

// Piece p of a row of np pieces, zero behind the row's end.  The load itself is
// unconditional: under a condition, each load of a batch gets its own branch
// and wait.
__device__ __forceinline__ u32x4 load_piece(const u32x4 *row, int p, int np) {
  const u32x4 q = row[min(p, np - 1)];
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = p < np ? q[i] : 0u;
  return r;
}

// fp32 -> the bf16 terms of a sum that holds it: f = t[0] + t[1] (+ t[2]),
// each the rounded rest of the one before.  Two terms keep 16 bits of f,
// three all 24.
template <int TERMS>
__device__ __forceinline__ void split_bf16(const float (&f)[8], bf16x8 (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = f[i];
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      t[k][i] = (__bf16)rest;  // round to nearest even
      rest -= (float)t[k][i];
    }
  }
}

}  // namespace moe

// One run of an adapter's rows in the plan's order: the backward pass's work
// item.  slot < 0: the adapter's only unit.
struct LoraUnit {
  int adapter, pos, count, slot;
};

// Slices of K that the sorted shrink cuts a tile into: enough workgroups for
// one per CU, at least 1 KB of every row each.
inline int lora_shrink_slices(int T, int row_bytes, int r) {
  const int tiles = (T + moe::kShrinkTile - 1) / moe::kShrinkTile * (r > 64 ? 2 : 1);
  int s = 1;
  while (s < moe::kShrinkSlices && tiles * s < 256 && row_bytes / (2 * s) >= 1024) s *= 2;
  return s;
}

// Where the plan of a batch lies in a workspace, and the size of its units.
// starts, tiles [n + 2]: each adapter's first row in the order and first
// shrink tile, then those of the rows without an adapter, then the ends;
// part: the slices of the shrink's sums, [rank group][slice][row of the
// order][rank].
struct LoraPlan {
  size_t order, starts, tiles, units, adapters, n_units, part, bytes;
  int TS, max_units, max_tiles;
};

// rows per unit: at most 32 slices of an adapter to add; batches of up to 1024
// rows are never sliced and need no launch that adds slices
inline LoraPlan lora_plan(int T, int N, int K, int r, int n, int es, bool backward) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  LoraPlan p;
  const int by = ((T + 31) / 32 + 31) / 32 * 32;
  p.TS = by > 1024 ? by : 1024;
  p.max_units = T / p.TS + n;  // (an adapter without rows has one of no rows)
  p.max_tiles = T / moe::kShrinkTile + (n + 1 < T ? n + 1 : T);
  p.order = 0;
  p.starts = up((size_t)T * 4);
  p.tiles = p.starts + up((size_t)(n + 2) * 4);
  p.units = p.tiles + up((size_t)(n + 2) * 4);
  p.adapters = p.units + (backward ? up((size_t)p.max_units * sizeof(LoraUnit)) : 0);
  p.n_units = p.adapters + (backward ? up((size_t)n * 8) : 0);
  p.part = p.n_units + (backward ? 256 : 0);
  const int slices = lora_shrink_slices(T, (backward ? N : K) * es, r);
  const int RP = r <= 16 ? 16 : r <= 32 ? 32 : 64;
  const size_t sums = (size_t)T * (r > 64 ? 2 : 1) * slices * RP;
  p.bytes = p.part + up(slices > 1 ? sums * 4 : 0);
  return p;
}

// Whether the forward pass reads its rows through a plan: not where a wave per
// row and rank takes less than the plan's launch and the longer way through it.
// That is so up to a number of waves, whatever N and K are (they cost their
// launch even where a row is short), and up to the bytes that rows in any order
// can cost.  Measured in order / through a plan, us, rows in any order:
//   bf16, T r = 8192, 16384, 32768, 131072: K and N 64, r 8 13.8 / 17.4, 18.6 /
//   18.5, 28.3 / 21.0, 84 / 40; K 512, N 512, r 64 21.3 / 20.5, 26.1 / 20.3, 35.2 /
//   21.5, 88 / 23; K and N 2048, r 16 19.6 / 24.4, 31.1 / 30.2, 52.5 / 38.8, 174 / 94;
//   fp32, T r = 16384, 32768, 131072: K 256, N 64, r 8 15.9 / 16.3, 23.8 / 19.0,
//   83 / 47; K 512, N 512, r 64 20.0 / 26.5, 26.5 / 27.9, 91 / 45; K 2048, N 512,
//   r 16 52.5 / 48.8, 89 / 81, 331 / 295;
//   bytes, bf16: 128 rows of N 14336, K 4096 (75e6) 48 / 55; N and K 4096: 512 rows
//   of rank 16 (134e6) 39 / 44 on 64 adapters, 37 / 40 on 8; 1024 rows (268e6) 65 /
//   62 on 100 adapters, 66 / 67 on 160.
inline bool lora_sorts(int T, int N, int K, int r, int es) {
  return (long long)T * r >= (es == 2 ? 16384 : 32768) ||
         (double)T * r * ((double)N + K) * es > 250e6;
}

hipError_t launch_lora_plan(const int32_t *adapter, int T, int n, const LoraPlan &p, bool units,
                            char *ws, hipStream_t s);

// p: the plan in ws, or null (rows as they come)
hipError_t launch_lora_shrink(const void *x, const void *F, int dt, const float *scale,
                              const int32_t *adapter, const LoraPlan *p, char *ws, int T, int K,
                              int r, int n, float *v, hipStream_t s);

// y (+)= x W^T + v F: W null adds to y
hipError_t launch_lora_expand(const void *x, const void *W, int ldw, const void *F, int dt,
                              const float *v, const int32_t *adapter, const int32_t *order, int T,
                              int N, int K, int r, int n, void *y, int y_dt, int cus, hipStream_t s);

// the plan (with its units), then the slices of adapters of several units
size_t lora_wgrad_ws_bytes(int T, int N, int K, int r, int n, int es);
hipError_t launch_lora_wgrad(const void *dy, const void *x, int dt, const float *u, const float *v,
                             int T, int N, int K, int r, int n, float *dA, float *dB, void *ws,
                             hipStream_t s);
