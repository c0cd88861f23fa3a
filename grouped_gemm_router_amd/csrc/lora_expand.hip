// lora_expand.hip -- y[t] = W x[t] + sum_j v[t][j] F[a][j], a = adapter[t]:
// the shared projection and, in its epilogue, each row's low-rank part.
//
// The low-rank vector v (fp32, r values a row) is ready when this launch
// starts.  Fusing its product with F into the projection writes y once, with
// one rounding, where a second pass would read and write it again.
//
// The low-rank part of a 32-row block of one or a few adapters (rows come
// sorted by adapter) goes through the matrix cores: v is split into bf16
// terms (two for a bf16 y, three for an fp32 y, so that the product keeps 16
// or 24 bits of v) and multiplied like 16 more columns of x.  (Three for a bf16
// y, which rounds to 8 bits: 1331 rows of rank 64 78.3 us instead of 75.4, 777
// rows of 33 adapters of rank 32 58.6 -> 60.4, 4096 rows of rank 16 141.7 instead
// of 141.0; the error of y stays.)  In a block of many adapters every row reads
// its own adapter's rows of F on the vector ALUs, with all of v.  An infinity or NaN in one request's adapter stays in that request's
// rows, and changes no bit of the others.
#include "lora_tile.h"

namespace {

using namespace moe;

// element i of a factor or of y as fp32
template <int ES>
__device__ __forceinline__ float ld1(const char *p, size_t i) {
  if constexpr (ES == 2) return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
  else return reinterpret_cast<const float *>(p)[i];
}

// Eight consecutive elements as they are stored.  VEC: 16-byte loads of all
// eight (the address is aligned and they exist); otherwise the first `have`
// exist and the others repeat the last of them.  No load is under a
// condition, so the loads of a batch are in flight together.
template <int ES, bool VEC>
struct Raw8 {
  u32x4 q[ES / 2];
  uint16_t h[VEC ? 1 : 8];
  float s[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const char *p, size_t i, int have) {
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < ES / 2; ++k) q[k] = *reinterpret_cast<const u32x4 *>(p + i * ES + 16 * k);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (ES == 2) h[c] = reinterpret_cast<const uint16_t *>(p)[i + min(c, have - 1)];
        else s[c] = reinterpret_cast<const float *>(p)[i + min(c, have - 1)];
      }
    }
  }
  __device__ __forceinline__ float get(int c) const {
    if constexpr (VEC && ES == 2)
      return c & 1 ? __uint_as_float(q[0][c >> 1] & 0xffff0000u) : bf16_bits_to_f32(q[0][c >> 1] & 0xffffu);
    else if constexpr (VEC)
      return __uint_as_float(q[(c >> 2) & (ES / 2 - 1)][c & 3]);
    else if constexpr (ES == 2)
      return bf16_bits_to_f32(h[c]);
    else
      return s[c];
  }
};

template <int OS, bool VEC>
__device__ __forceinline__ void st8(char *p, size_t i, int have, const float (&f)[8]) {
  if constexpr (VEC) {
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

// Adapters among 32 rows up to which they go through the matrix cores one
// after the other.  1024 rows of N and K 4096 with a limit of 2, 6 and 8: rank
// 16 of 100 adapters (4 a block) 63.1, 62.4, 62.3 us, of 160 65.1, 67.4, 67.1,
// of 250 67.8, 70.5, 74.0; rank 64 of 160 125, 117, 114.
constexpr int kBlockKinds = 6;

// The adapters of a tile's row blocks.  count: how many a block of 32 rows
// has, 0 if it does not go through the matrix cores (none, or more than
// kBlockKinds).  Its k-th adapter is that of slot base + k; neighbouring
// blocks share a slot where the one ends with the adapter that the next one
// begins with.
struct TileKinds {
  int count[8], base[8], ad[8][8], slot_ad[8 * kBlockKinds], slots;
  int bad;  // a staged factor holds an infinity or NaN
};

// by the whole workgroup of four waves; every thread may read it on return
__device__ __forceinline__ void find_kinds(TileKinds &tk, const int *s_ad, int blocks, int wv) {
  const int lane = lane_id();
  for (int blk = wv; blk < blocks; blk += 4) {
    const int mine = s_ad[blk * 32 + (lane & 31)];
    unsigned left = (unsigned)__ballot(mine >= 0);
    int kinds = 0, ids = -1;  // lane k: the k-th adapter
    while (left && kinds <= kBlockKinds) {
      const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
      ids = lane == kinds ? a : ids;
      left &= ~(unsigned)__ballot(mine == a);
      ++kinds;
    }
    if (lane < 8) tk.ad[blk][lane] = ids;
    if (lane == 0) tk.count[blk] = kinds <= kBlockKinds ? kinds : 0;
  }
  __syncthreads();
  if (wv == 0) {
    const int blk = lane >> 3, k = lane & 7, bc = min(blk, blocks - 1);
    const int cnt = blk < blocks ? tk.count[bc] : 0, mine = tk.ad[bc][k];
    const int before = bc > 0 ? tk.count[bc - 1] : 0;
    const int shares =
        cnt > 0 && before > 0 && tk.ad[max(bc - 1, 0)][max(before - 1, 0)] == tk.ad[bc][0];
    int total;
    const int sum = wave_exclusive_scan(k == 0 ? cnt - shares : 0, &total);
    const int base = __shfl(sum, lane & ~7, kWave) - shares;
    if (k < cnt) tk.slot_ad[base + k] = mine;  // (a shared slot: the same value twice)
    if (k == 0 && blk < blocks) tk.base[blk] = base;
    if (lane == 0) {
      tk.slots = total;
      tk.bad = 0;
    }
  }
  __syncthreads();
}

// The low-rank part of a tile's blocks on the matrix cores (those with a
// count in tk), BM x BN on 4 waves of MI x NB blocks: acc[i][nb] += v F for
// each of a block's adapters, the rows of v that are not its own as zeros.
// (Where a factor is not finite, zeros would not do: then the sums of those
// rows are kept aside.  The others' come out the same bit for bit.)
//
// v, split into its bf16 terms, and the adapters' rows of F (the tile's
// columns) are staged in LDS as the matrix cores' fragments, up to RC ranks of
// all the tile's adapters at once.  What counts here is the number of
// instructions: the code runs once a tile, from beyond the instruction cache,
// where it arrives at some 50 ns per 64 bytes.  By clock stamps inside a tile: 16
// ranks of one adapter on 256 x 256 6.6 us, with fragments built from single
// elements 9.2; 32 ranks of 2 to 3 adapters a block on 128 x 128 6.9 us, so built
// 9.2.  The launch grows by more: 4096 rows, N 4096, rank 16 by 10 us, 1331 rows,
// N 2048, rank 64 by 7, 777 rows of 33 adapters, N 7168, rank 32 by 13.5 (two
// rounds of tiles).
//
// v_of(row): 256 bytes for a row of the tile; slab_of(i), i < NSLAB: SLAB
// bytes each.  s_row, s_ad: the tile's rows and adapters (-1 for none).
// Called by the whole workgroup; other waves may still read what is staged on
// return.
template <int TERMS, int MI, int NB, int BM, int BN, int NSLAB, int SLAB, class VOf, class SlabOf>
__device__ __forceinline__ void low_rank_blocks(f32x16 (&acc)[MI][NB], TileKinds &tk,
                                                const int *s_row, const int *s_ad, int wm, int wn,
                                                VOf v_of, SlabOf slab_of, int n0, const char *F,
                                                const float *v, int N, int r) {
  const int tid = threadIdx.x, lane = lane_id(), fr = lane & 31, fh = lane >> 5;
  constexpr int NT = 256, CG = BN / 8;  // threads; groups of 8 columns
  // ranks that are staged at once, in eights: the terms of a row of v are at
  // most 16 pieces
  constexpr int RO = TERMS == 2 ? 8 : 4, RC = 8 * RO;
  static_assert(NSLAB <= 3, "slab() counts up to three");
  static_assert(SLAB >= RC * BN * 2, "a chunk of an adapter's ranks must fit a slab");
  const int slots = __builtin_amdgcn_readfirstlane(tk.slots);
  const uint16_t *const Fw = reinterpret_cast<const uint16_t *>(F);
  // column c of a slab's row of eight ranks: the threads of the transposition
  // write 8 columns apart, to distinct banks
  auto place = [](int c) { return c ^ ((c >> 3) & 7); };
  int at[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) at[nb] = fh * BN + place(wn * (NB * 32) + nb * 32 + fr);
  // the wave's blocks: the lane's row's adapter, and in lane k the k-th one
  int mine[MI], ids[MI], count[MI], base0[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int blk = wm * MI + i;
    mine[i] = s_ad[blk * 32 + fr];
    ids[i] = tk.ad[blk][lane & 7];
    count[i] = tk.count[blk];
    base0[i] = tk.base[blk];
  }
  for (int rc = 0; slots > 0 && rc < r; rc += RC) {
    // eights of ranks: those of the chunk, and the same with a zero one to make
    // whole steps of 16
    const int ro = min(RO, (r - rc) / 8), oc = (ro + 1) & ~1;
    const int per = SLAB / (oc * BN * 16), inv = (65536 + oc - 1) / oc;
    auto slab = [&](int slot) {
      const int i = (slot >= per) + (NSLAB > 2 && slot >= 2 * per);
      return slab_of(i) + (slot - i * per) * oc * BN;
    };
    for (int first = 0; first < slots; first += NSLAB * per) {
      const int ns = min(NSLAB * per, slots - first);
      if (rc > 0 || first > 0) __syncthreads();  // what is staged has been used
      const int vn = first == 0 ? BM * oc : 0, fn = ns * oc * CG;
      constexpr int U = 2;
#pragma unroll 1
      for (int b = tid; b - tid < fn || b - tid < (vn + U - 1) / U; b += NT) {
        // eight ranks of eight columns
        const int fi = min(b, fn - 1), cg = fi % CG, rest = fi / CG;
        const int slot = (rest * inv) >> 16, o = rest - slot * oc;  // (rest is below 100: exact)
        const uint16_t *const f0 =
            Fw + ((size_t)tk.slot_ad[first + slot] * r + rc + min(o, ro - 1) * 8) * N;
        const int c = n0 + cg * 8;
        u32x4 q[8];
        if (N % 8 == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            q[i] = *reinterpret_cast<const u32x4 *>(f0 + (size_t)i * N + min(c, N - 8));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < 4; ++h)
              q[i][h] = (uint32_t)f0[(size_t)i * N + min(c + 2 * h, N - 1)] |
                        ((uint32_t)f0[(size_t)i * N + min(c + 2 * h + 1, N - 1)] << 16);
        }
        // eight ranks of U rows
        f32x4 v0[U], v1[U];
        int row[U], ov[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min((b - tid) * U + u * NT + tid, BM * oc - 1);
          ov[u] = i / BM;
          row[u] = i % BM;
          const float *const vr = v + (size_t)s_row[row[u]] * r + rc + min(ov[u], ro - 1) * 8;
          v0[u] = *reinterpret_cast<const f32x4 *>(vr);
          v1[u] = *reinterpret_cast<const f32x4 *>(vr + 4);
        }
        __builtin_amdgcn_sched_barrier(0);  // every load is issued first
        if (first == 0) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float f[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) f[h] = ov[u] < ro ? (h < 4 ? v0[u][h] : v1[u][h - 4]) : 0.f;
            bf16x8 t[TERMS];
            split_bf16<TERMS>(f, t);
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
              v_of(row[u])[(k * RO + ov[u]) ^ (row[u] & 15)] = __builtin_bit_cast(u32x4, t[k]);
          }
        }
        unsigned bad = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            q[i][h] = o < ro ? q[i][h] : 0u;
            bad |= (q[i][h] & 0x7f807f80u) + 0x00800080u;  // an exponent of ones carries
          }
        if (b < fn) {
          u32x4 *const to = slab(slot) + o * BN;
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // column e: rank pairs into words
            const unsigned sel = (e & 1) ? 0x07060302u : 0x05040100u;
            u32x4 w;
#pragma unroll
            for (int d = 0; d < 4; ++d)
              w[d] = __builtin_amdgcn_perm(q[2 * d + 1][e >> 1], q[2 * d][e >> 1], sel);
            to[place(cg * 8 + e)] = w;
          }
          if (bad & 0x80008000u) tk.bad = 1;
        }
      }
      __syncthreads();
      const bool finite = __builtin_amdgcn_readfirstlane(tk.bad) == 0;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int row = (wm * MI + i) * 32 + fr;
        const int num = __builtin_amdgcn_readfirstlane(count[i]);
        const int base = __builtin_amdgcn_readfirstlane(base0[i]) - first;
        const u32x4 *const vr = v_of(row);
#pragma unroll 1
        for (int k = max(0, -base); k < num && base + k < ns; ++k) {
          const u32x4 *const sl = slab(base + k);
          const bool takes = mine[i] == __builtin_amdgcn_readlane(ids[i], k);
          const unsigned same = (unsigned)__ballot(takes);
          if (finite || same == ~0u) {
#pragma unroll 1
            for (int o = 0; o < oc; o += 2) {
              u32x4 va[TERMS];
#pragma unroll
              for (int t = 0; t < TERMS; ++t) {
                const u32x4 q = vr[(t * RO + o + fh) ^ (row & 15)];
#pragma unroll
                for (int h = 0; h < 4; ++h) va[t][h] = takes ? q[h] : 0u;
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const bf16x8 w = __builtin_bit_cast(bf16x8, sl[o * BN + at[nb]]);
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                  acc[i][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                      __builtin_bit_cast(bf16x8, va[t]), w, acc[i][nb], 0, 0, 0);
              }
            }
            continue;
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            f32x16 all = acc[i][nb];
#pragma unroll 1
            for (int o = 0; o < oc; o += 2)
#pragma unroll
              for (int t = 0; t < TERMS; ++t)
                all = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, vr[(t * RO + o + fh) ^ (row & 15)]),
                    __builtin_bit_cast(bf16x8, sl[o * BN + at[nb]]), all, 0, 0, 0);
            // register e holds row 8 (e / 4) + 4 fh + e % 4
            const unsigned rows = same >> (4 * fh);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              acc[i][nb][e] = (rows >> (8 * (e >> 2) + (e & 3))) & 1 ? all[e] : acc[i][nb][e];
          }
        }
      }
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

// row i of a tile: where it lies in the batch (rows past T repeat the last
// one) and its adapter, -1 for none
__device__ __forceinline__ void load_row(int *s_row, int *s_ad, int i, int m0, const int32_t *adapter,
                                         const int32_t *order, int T, int n) {
  int t = min(m0 + i, T - 1);
  if (order) t = order[t];
  const int a = adapter[t];
  s_row[i] = t;
  s_ad[i] = a >= 0 && a < n ? a : -1;
}

// rows [32 blk, 32 blk + 32) of a tile, staged in fp32 with row pitch SP, for
// WM row blocks at once (stage_of(w) holds tile row block first + w * stride):
// add what is left of the low-rank part (blocks without `done`) and of y,
// round, store 8-column pieces.  The rows' own factors are what bounds a block
// of many adapters: 64 rows of 64 adapters of 16 ranks, 128 columns, are 256 KB
// a tile, in 9 us (two pieces a thread at once: the same).
template <int ES, int OS, int BN, int SP, int WM, bool VEC, class StageOf>
__device__ __forceinline__ void finish_pieces(StageOf stage_of, int first, int stride, int m0, int n0,
                                              const int *s_row, const int *s_ad, const int *done,
                                              bool add_y, const char *F, const float *v, int T, int N,
                                              int r, char *y) {
  constexpr int CG = BN / 8;
  for (int q = threadIdx.x; q < WM * 32 * CG; q += blockDim.x) {
    const int w = q / (32 * CG), rr = (q / CG) % 32, c = (q % CG) * 8;
    const int blk = first + w * stride, row = blk * 32 + rr, col = n0 + c;
    if (m0 + row >= T || col >= N) continue;
    const int t = s_row[row], a = s_ad[row], have = N - col;
    const float *st = stage_of(w) + rr * SP + c;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = st[i];
    if (a >= 0 && !done[blk]) {
      const float *const vr = v + (size_t)t * r;
      const char *const Fa = F + ((size_t)a * r * N + col) * ES;
      // 16 ranks a step, all loads of a step before its first product
      for (int j0 = 0; j0 < r; j0 += 16) {
        Raw8<ES, VEC> fv[16];
        f32x4 vv[4];
        const int j8 = min(j0 + 8, r - 8);  // (r % 16 == 8: loaded again, not used)
#pragma unroll
        for (int j = 0; j < 16; ++j) fv[j].load(Fa, (size_t)(j < 8 ? j0 + j : j8 + j - 8) * N, have);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          vv[j] = *reinterpret_cast<const f32x4 *>(vr + (j < 2 ? j0 : j8 - 8) + 4 * j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && j0 + 8 >= r) break;
#pragma unroll
          for (int j = 8 * h; j < 8 * h + 8; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf(vv[j >> 2][j & 3], fv[j].get(i), f[i]);
        }
      }
    }
    const size_t at = (size_t)t * N + col;
    if (add_y) {
      Raw8<OS, VEC> old;
      old.load(y, at, have);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += old.get(i);
    }
    st8<OS, VEC>(y, at, have, f);
  }
}

template <int ES, int OS, int BN, int SP, int WM, class StageOf>
__device__ __forceinline__ void finish_rows(StageOf stage_of, int first, int stride, int m0, int n0,
                                            const int *s_row, const int *s_ad, const int *done,
                                            bool add_y, const char *F, const float *v, int T, int N,
                                            int r, char *y) {
  if (N % 8 == 0)  // rows of F and of y are then 16-byte aligned
    finish_pieces<ES, OS, BN, SP, WM, true>(stage_of, first, stride, m0, n0, s_row, s_ad, done, add_y,
                                            F, v, T, N, r, y);
  else
    finish_pieces<ES, OS, BN, SP, WM, false>(stage_of, first, stride, m0, n0, s_row, s_ad, done, add_y,
                                             F, v, T, N, r, y);
}

// ---------------------------------------------------------------------------
// fp32: every row's low-rank part runs on the vector ALUs in fp32, and no sum
// over K is longer than K / 2, or K / 8, terms before it meets the others.
// ---------------------------------------------------------------------------

// acc += a b over the lane's 16-byte pieces: component c of the two halves'
// pieces is k = 8 i + 4 (lane / 32) + c
__device__ __forceinline__ f32x16 mma_f32(u32x4 a, u32x4 b, f32x16 acc) {
  const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int c = 0; c < 4; ++c) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[c], fb[c], acc, 0, 0, 0);
  return acc;
}

// Tiles of 64 x 64 on two groups of 4 waves of 32 x 32, operands through LDS
// 256 bytes of a row at a time, 128 of them for each group: the next step's
// pieces are loaded into registers while this step is multiplied.  Pieces past
// K read as zero; rows past T and columns past N repeat the last one and are
// not stored.
constexpr int kF32Threads = 512;

__global__ __launch_bounds__(kF32Threads) void expand_f32_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter,
    const int32_t *__restrict__ order, int T, int N, int K, int r, int n, char *__restrict__ y, int MT,
    int NT) {
  constexpr int BM = 64, BNF = 64, SP = BNF + 4, ROWS = BM + BNF, NLD = 2 * ROWS * 8 / kF32Threads;
  __shared__ u32x4 ring[2][2][ROWS * 8];  // step parity, group
  __shared__ int s_row[BM], s_ad[BM];
  __shared__ int s_done[BM / 32];
  const TileAt at = tile_at(blockIdx.x, MT, NT);
  if (at.mt < 0) return;
  const int m0 = at.mt * BM, n0 = at.nt * BNF;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int grp = wv / 4, wm = wv / 2 % 2, wn = wv % 2, fr = lane & 31, fh = lane >> 5;
  if (tid < BM) load_row(s_row, s_ad, tid, m0, adapter, order, T, n);
  if (tid < BM / 32) s_done[tid] = 0;
  f32x16 acc = f32x16{};
  __syncthreads();
  if (W) {
    const int KP = K / 4, KT = (KP + 15) / 16;
    const u32x4 *src[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int row = (tid + kF32Threads * i) >> 4;  // 16 pieces a row and step
      src[i] = row < BM
                   ? reinterpret_cast<const u32x4 *>(x + (size_t)s_row[row] * K * 4)
                   : reinterpret_cast<const u32x4 *>(W + (size_t)min(n0 + row - BM, N - 1) * ldw * 4);
    }
    u32x4 reg[NLD];
    auto fetch = [&](int kt) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) reg[i] = load_piece(src[i], kt * 16 + (tid & 15), KP);
    };
    auto put = [&](int b) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int row = (tid + kF32Threads * i) >> 4;
        ring[b][(tid >> 3) & 1][row * 8 + swzb(row, tid & 7)] = reg[i];
      }
    };
    fetch(0);
    put(0);
    __syncthreads();
    for (int kt = 0; kt < KT; ++kt) {
      if (kt + 1 < KT) fetch(kt + 1);
      const u32x4 *l = ring[kt & 1][grp];
      const int ra = wm * 32 + fr, rb = BM + wn * 32 + fr;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        acc = mma_f32(l[ra * 8 + swzb(ra, 2 * ks + fh)], l[rb * 8 + swzb(rb, 2 * ks + fh)], acc);
      if (kt + 1 < KT) put((kt + 1) & 1);
      __syncthreads();
    }
  }
  // the second group's sums join the first's
  float *stage = reinterpret_cast<float *>(&ring[0][0][0]);
  for (int g = 1; g >= 0; --g) {
    if (grp == g)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float *p = stage + (wm * 32 + 8 * (e >> 2) + 4 * fh + (e & 3)) * SP + wn * 32 + fr;
        *p = g == 1 ? acc[e] : *p + acc[e];
      }
    __syncthreads();
  }
  finish_rows<4, 4, BNF, SP, 2>([&](int w) { return stage + w * 32 * SP; }, 0, 1, m0, n0, s_row,
                                s_ad, s_done, W == nullptr, F, v, T, N, r, y);
}

// Tiles of 32 x 32 whose eight waves cut K, operands straight from memory:
// where tiles of 64 x 64 would not fill the chip.
constexpr int kF32Waves = 8;

__global__ __launch_bounds__(kF32Waves *kWave) void expand_f32_small_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter,
    const int32_t *__restrict__ order, int T, int N, int K, int r, int n, char *__restrict__ y, int MT,
    int NT) {
  constexpr int BM = 32, BNF = 32, SP = BNF + 4;
  __shared__ float red[kF32Waves][BM * SP];
  __shared__ int s_row[BM], s_ad[BM];
  __shared__ int s_done[1];
  const TileAt at = tile_at(blockIdx.x, MT, NT);
  if (at.mt < 0) return;
  const int m0 = at.mt * BM, n0 = at.nt * BNF;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int fr = lane & 31, fh = lane >> 5;
  if (tid < BM) load_row(s_row, s_ad, tid, m0, adapter, order, T, n);
  if (tid == 0) s_done[0] = 0;
  f32x16 acc = f32x16{};
  __syncthreads();
  if (W) {
    const int KP = K / 4;
    const u32x4 *xp = reinterpret_cast<const u32x4 *>(x + (size_t)s_row[fr] * K * 4);
    const u32x4 *wp = reinterpret_cast<const u32x4 *>(W + (size_t)min(n0 + fr, N - 1) * ldw * 4);
    // a wave takes whole lines of 8 pieces
    constexpr int U = 4, CHUNK = 2 * U * kF32Waves;
    int p0 = 0;
    for (; p0 + CHUNK <= KP; p0 += CHUNK) {
      u32x4 xa[U], wa[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xa[u] = xp[p0 + (wv * U + u) * 2 + fh];
        wa[u] = wp[p0 + (wv * U + u) * 2 + fh];
      }
      __builtin_amdgcn_sched_barrier(0);  // every load of the chunk is issued first
#pragma unroll
      for (int u = 0; u < U; ++u) acc = mma_f32(xa[u], wa[u], acc);
    }
    if (p0 < KP) {  // zeros behind K
      u32x4 xa[U], wa[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xa[u] = load_piece(xp, p0 + (wv * U + u) * 2 + fh, KP);
        wa[u] = load_piece(wp, p0 + (wv * U + u) * 2 + fh, KP);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u) acc = mma_f32(xa[u], wa[u], acc);
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) red[wv][(8 * (e >> 2) + 4 * fh + (e & 3)) * SP + fr] = acc[e];
  __syncthreads();
  for (int i = tid; i < BM * BNF; i += kF32Waves * kWave) {
    const int o = (i / BNF) * SP + i % BNF;
    float sum = red[0][o];
#pragma unroll
    for (int w = 1; w < kF32Waves; ++w) sum += red[w][o];
    red[0][o] = sum;
  }
  __syncthreads();
  finish_rows<4, 4, BNF, SP, 1>([&](int) { return &red[0][0]; }, 0, 1, m0, n0, s_row, s_ad, s_done,
                                W == nullptr, F, v, T, N, r, y);
}

// ---------------------------------------------------------------------------
// bf16: tiles of BM x BN on 4 waves (WM x WN), operands by LDS-direct loads
// through a ring of four slots of one 64-deep K step each, one barrier a step.
// The ring's slots are separate LDS arrays, so that the compiler does not wait
// for a load into one slot before it reads another.  What bounds it is the
// rate at which a CU takes in operands: about 80 bytes a ns where they come from
// L2 and the memory-side cache, whatever the shape, 50 to 65 with all CUs on
// 128 x 128 and a long K.  1331 rows, N 2048, K 7168 on 128 x 128 without
// adapters: 51 us, 42 of them for 112 steps of 32 KB on 176 CUs (with rank 64
// 62 us, the matrix cores busy 27 % of the chip's cycles, 39 % of those of the
// CUs that have a tile).  128 rows, N 14336, K 4096 without adapters: 36 us, W
// from HBM at 3.3 TB/s.
//
// rot: workgroups of different columns begin at different K, so that their
// loads of W do not all hit the same memory channels.  That is so where W's rows
// lie a multiple of 4 KB apart, and those rows go this way.  Without / with, us:
// 128 rows of N 14336, K 4096 39.1 / 36.6, 64 rows 30.2 / 27.7; 64 rows of N
// 28672, K 4096 57.1 / 45.5, of N and K 8192 46.9 / 41.4, of N 14336, K 6144
// 46.8 / 40.8.  Other pitches lose by it or gain nothing: the same N and K 8192
// with 256 bytes behind each row 44.3 / 50.2, N 14336, K 4096 so padded 28.5 /
// 30.8, dense K 7168 46.1 / 46.3.  With more rows the tiles that share x want the
// same part of it at the same time: 512 rows of 4096 x 4096 36.3 us instead of
// 29.6.
//
// Pieces past K come from a zero in memory (the last steps only); rows past T
// and columns past N repeat the last one and are not stored.
// ---------------------------------------------------------------------------
__device__ u32x4 g_zero;

template <int OS, int BM, int BNT, int WM, int WN>
__global__ __launch_bounds__(256) void expand_ring_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter,
    const int32_t *__restrict__ order, int T, int N, int K, int r, int n, char *__restrict__ y, int MT,
    int NT, int rot) {
  constexpr int MI = BM / WM / 32, NB = BNT / WN / 32;
  constexpr int IL = (BM + BNT) / 32;  // loads per wave and step
  constexpr int SLOT = (BM + BNT) * 8, SP = BNT + 4, NS = 4;
  static_assert(WM * WN == 4 && MI >= 1 && NB >= 1, "four waves of 32 x 32 blocks");
  static_assert(32 * SP * 4 <= SLOT * 16 && WM <= 2, "a staged row block must fit a slot");
  static_assert(BM * 16 <= SLOT, "64 floats for each row must fit a slot");
  __shared__ u32x4 s0[SLOT], s1[SLOT], s2[SLOT], s3[SLOT];
  __shared__ int s_row[BM], s_ad[BM];
  __shared__ TileKinds kinds;
  const TileAt at = tile_at(blockIdx.x, MT, NT);
  if (at.mt < 0) return;
  const int m0 = at.mt * BM, n0 = at.nt * BNT;
  const int tid = threadIdx.x, lane = lane_id(),
            wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wv / WN, wn = wv % WN, fr = lane & 31, fh = lane >> 5;

  if (tid < BM) load_row(s_row, s_ad, tid, m0, adapter, order, T, n);
  f32x16 acc[MI][NB];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};

  __syncthreads();  // s_row
  if (W) {
    const int KP = K / 8, KT = (KP + 7) / 8, KF = KP / 8;  // steps, whole steps
    const int k_first = rot && KT == KF ? (int)(at.nt * 5u % (unsigned)KT) : 0;
    const u32x4 *src[IL];
    int pc[IL];
    const int dma = wv * (SLOT / 4);
#pragma unroll
    for (int i = 0; i < IL; ++i) {
      const int sl = dma + i * 64 + lane, row = sl / 8;
      pc[i] = swzb(row, sl % 8);
      src[i] = (row < BM
                    ? reinterpret_cast<const u32x4 *>(x + (size_t)s_row[row] * K * 2)
                    : reinterpret_cast<const u32x4 *>(W + (size_t)min(n0 + row - BM, N - 1) * ldw * 2)) +
               pc[i];
    }
    const u32x4 *const zero = &g_zero;
    // the lane's fragment pieces of its first row blocks (32 rows are 256
    // pieces further on, under the same swizzle)
    int ra[4], rb[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      ra[ks] = (wm * (MI * 32) + fr) * 8 + swzb(fr, 2 * ks + fh);
      rb[ks] = (BM + wn * (NB * 32) + fr) * 8 + swzb(fr, 2 * ks + fh);
    }
#define MOE_ISSUE(slot, kl, TAIL)                                                            \
  _Pragma("unroll") for (int i = 0; i < IL; ++i) {                                         \
    const int kr = (kl) + k_first, ku = kr >= KT ? kr - KT : kr;                           \
    const u32x4 *g = src[i] + ku * 8;                                                      \
    if (TAIL && (kl) * 8 + pc[i] >= KP) g = zero;                                          \
    __builtin_amdgcn_global_load_lds((const void *)g, (lds_void *)((slot) + dma + i * 64), 16, 0, 0); \
  }
#define MOE_READ(f, slot, ks)                                                                \
  _Pragma("unroll") for (int i = 0; i < MI; ++i)                                           \
    f.a[i] = __builtin_bit_cast(bf16x8, (slot)[ra[ks] + i * 256]);                         \
  _Pragma("unroll") for (int j = 0; j < NB; ++j)                                           \
    f.b[j] = __builtin_bit_cast(bf16x8, (slot)[rb[ks] + j * 256]);
#define MOE_MMA(f)                             \
  mfma_frag<MI, NB>(acc, f);                   \
  interleave_mfma_ds_read<MI * NB, MI + NB>();
// Step kt, whose first fragments are in f0: each 16-deep part is multiplied
// while the next one's fragments are read.  Before the last part, every wave
// has read its slot out and the next step's loads have landed; the barrier
// makes both known, the slot takes step kt + NS, and the next step's first
// fragments are read under the last multiplies.
#define MOE_STEP(cur, nxt, kt, TAIL)                                       \
  MOE_READ(f1, cur, 1)                                                     \
  MOE_MMA(f0)                                                              \
  MOE_READ(f0, cur, 2)                                                     \
  MOE_MMA(f1)                                                              \
  MOE_READ(f1, cur, 3)                                                     \
  MOE_MMA(f0)                                                              \
  wait_vmcnt_lgkm0<(NS - 2) * IL>();                                       \
  stage_barrier();                                                         \
  MOE_ISSUE(cur, (kt) + NS, TAIL)                                          \
  MOE_READ(f0, nxt, 0)                                                     \
  MOE_MMA(f1)
#define MOE_PERIOD(kt, TAIL)             \
  MOE_STEP(s0, s1, kt, TAIL)             \
  MOE_STEP(s1, s2, (kt) + 1, TAIL)       \
  MOE_STEP(s2, s3, (kt) + 2, TAIL)       \
  MOE_STEP(s3, s0, (kt) + 3, TAIL)
    MOE_ISSUE(s0, 0, true)
    MOE_ISSUE(s1, 1, true)
    MOE_ISSUE(s2, 2, true)
    MOE_ISSUE(s3, 3, true)
    wait_vmcnt<(NS - 1) * IL>();
    stage_barrier();
    Frag<MI, NB> f0, f1;
    MOE_READ(f0, s0, 0)
    int kt = 0;
    // a period loads up to step kt + 2 NS - 1; the steps past the last one
    // multiply zeros
    for (; kt + 2 * NS <= KF; kt += NS) {
      MOE_PERIOD(kt, false)
    }
    for (; kt < KT; kt += NS) {
      MOE_PERIOD(kt, true)
    }
    wait_vmcnt<0>();  // no LDS-direct load may still be landing
#undef MOE_PERIOD
#undef MOE_STEP
#undef MOE_MMA
#undef MOE_READ
#undef MOE_ISSUE
  }
  __syncthreads();  // every wave is done with the ring

  find_kinds(kinds, s_ad, BM / 32, wv);
  low_rank_blocks<OS == 2 ? 2 : 3, MI, NB, BM, BNT, 3, SLOT * 16>(
      acc, kinds, s_row, s_ad, wm, wn, [&](int row) { return s0 + row * 16; },
      [&](int i) { return i == 0 ? s1 : i == 1 ? s2 : s3; }, n0, F, v, N, r);
  if (kinds.slots > 0) __syncthreads();
  // 32 rows of every wave row at a time meet in LDS in fp32
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    float *mine = reinterpret_cast<float *>(wm == 0 ? s0 : s1);
    if (i > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        mine[(8 * (e >> 2) + 4 * fh + (e & 3)) * SP + wn * (NB * 32) + j * 32 + fr] = acc[i][j][e];
    __syncthreads();
    finish_rows<2, OS, BNT, SP, WM>(
        [&](int w) { return reinterpret_cast<const float *>(w == 0 ? s0 : s1); }, i, MI, m0, n0,
        s_row, s_ad, kinds.count, W == nullptr, F, v, T, N, r, y);
  }
}

// ---------------------------------------------------------------------------
// bf16, large batches: 256 x 256 tiles (four waves of 128 x 128, which read
// half as many operand bytes from LDS per multiply as 64 x 64).  K % 128 == 0.
// 4096 rows, N and K 4096, one tile a CU, rank 16: 124 to 131 us, the matrix
// cores busy 53 % of it at the 1.9 GHz that this load leaves.  Without adapters
// 115: 17 before and behind the K loop (start, rows, y), 98 in it (23 per 1024 of
// K up to 2048, 26 from there on).
// ---------------------------------------------------------------------------
template <int OS>
__global__ __launch_bounds__(256, 1) void expand_big_kernel(
    const char *__restrict__ x, const char *__restrict__ W, int ldw, const char *__restrict__ F,
    const float *__restrict__ v, const int32_t *__restrict__ adapter,
    const int32_t *__restrict__ order, int T, int N, int K, int r, int n, char *__restrict__ y, int MT,
    int NT) {
  constexpr int MI = kBigBlocks, NB = kBigBlocks;
  __shared__ u32x4 sA0[kBigSlot], sA1[kBigSlot];
  __shared__ u32x4 sB0[kBigSlot], sB1[kBigSlot], sB2[kBigSlot];
  const TileAt at = tile_at(blockIdx.x, MT, NT);
  if (at.mt < 0) return;
  const int m0 = at.mt * kBig, n0 = at.nt * kBig;
  const int tid = threadIdx.x, lane = lane_id(),
            wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wv / 2, wn = wv % 2, fr = lane & 31, fh = lane >> 5;
  // the tile's rows wait in the last B slot, which the K loop fills last
  int *const rows = reinterpret_cast<int *>(sB2);
  load_row(rows, rows + kBig, tid, m0, adapter, order, T, n);
  __syncthreads();
  const uint16_t *ga[kBigLoads], *gb[kBigLoads];
#pragma unroll
  for (int i = 0; i < kBigLoads; ++i) {
    const int sl = wv * (kBigSlot / 4) + i * 64 + lane, row = sl / 8, p = swzb(row, sl % 8);
    ga[i] = reinterpret_cast<const uint16_t *>(x) + (size_t)rows[row] * K + p * 8;
    gb[i] = reinterpret_cast<const uint16_t *>(W) + (size_t)min(n0 + row, N - 1) * ldw + p * 8;
  }
  f32x16 acc[MI][NB];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
  big_k_loop(acc, ga, gb, K / kBigK, wv, fr, fh, sA0, sA1, sB0, sB1, sB2);
  __syncthreads();  // every wave is done with the rings
  int *const s_row = rows, *const s_ad = rows + kBig;
  TileKinds &kinds = *reinterpret_cast<TileKinds *>(rows + 2 * kBig);
  load_row(s_row, s_ad, tid, m0, adapter, order, T, n);
  __syncthreads();
  find_kinds(kinds, s_ad, kBig / 32, wv);
  low_rank_blocks<OS == 2 ? 2 : 3, MI, NB, kBig, kBig, 2, kBigSlot * 16>(
      acc, kinds, s_row, s_ad, wm, wn,
      [&](int row) { return (row < kBig / 2 ? sA0 : sA1) + row % (kBig / 2) * 16; },
      [&](int i) { return i == 0 ? sB0 : sB1; }, n0, F, v, N, r);
  if (kinds.slots > 0) __syncthreads();
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    // 32 rows of both wave rows: 32 x 256 fp32 are one B slot
    float *mine = reinterpret_cast<float *>(wm == 0 ? sB0 : sB1);
    if (i > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        mine[(8 * (e >> 2) + 4 * fh + (e & 3)) * kBig + wn * (NB * 32) + j * 32 + fr] = acc[i][j][e];
    __syncthreads();
    finish_rows<2, OS, kBig, kBig, 2>(
        [&](int w) { return reinterpret_cast<const float *>(w == 0 ? sB0 : sB1); }, i, MI, m0, n0,
        s_row, s_ad, kinds.count, false, F, v, T, N, r, y);
  }
}

// ---------------------------------------------------------------------------
// few rows (bf16): 16 columns per workgroup, MB blocks of 16 rows, eight
// waves cutting K.  W is read once, by the whole chip at once, straight into
// the matrix cores' fragments; x comes from L2.  One row of 4096 x 4096: 8.8
// us, W at 3.8 TB/s.
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
  // out of each 16; the last, partial chunk reads zeros behind K
  constexpr int U = MB == 1 ? 16 : 8;
  constexpr int CHUNK = U * kRowWaves * 4;  // pieces that the workgroup takes at once
  auto multiply = [&](const u32x4 (&wa)[U], const u32x4 (&xa)[U][MB]) {
    __builtin_amdgcn_sched_barrier(0);  // every load of the chunk is issued first
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa[u][b]),
                                                         __builtin_bit_cast(bf16x8, wa[u]), acc[b],
                                                         0, 0, 0);
  };
  int p0 = 0;
  for (; p0 + CHUNK <= KP; p0 += CHUNK) {
    u32x4 wa[U], xa[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + (2 * wv + (u & 1) + (u >> 1) * 2 * kRowWaves) * 4 + fq;
      wa[u] = wp[p];
#pragma unroll
      for (int b = 0; b < MB; ++b) xa[u][b] = xp[b][p];
    }
    multiply(wa, xa);
  }
  if (p0 < KP) {
    u32x4 wa[U], xa[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + (2 * wv + (u & 1) + (u >> 1) * 2 * kRowWaves) * 4 + fq;
      wa[u] = load_piece(wp, p, KP);
#pragma unroll
      for (int b = 0; b < MB; ++b) xa[u][b] = load_piece(xp[b], p, KP);
    }
    multiply(wa, xa);
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

// Rows up to which expand_rows_kernel runs (bf16 with a W).  Every workgroup
// reads all of x, so above that the tiles are faster (N and K 4096: 64 rows
// 27.7 us here, 80 rows 23.4 us in tiles; 32 rows 18.9 us here).
constexpr int kExpandRowsMax = 32;

// Tile shapes of the bf16 kernels, and what pick_tile counts for a 64-deep K
// step and for the rest of a tile on a CU, in ns: measured with one tile per CU
// on 96 to 4096 rows, K from 2048 to 7168.  256 tiles whose operands stay in the
// memory-side cache take 1650, 490 to 640, 300 and 195 ns a step and 16, 7.6, 6.1
// and 5 us for the rest, so the smaller shapes are counted rather dear.
struct Shape {
  int BM, BN, step, fixed;
};
constexpr Shape kShapes[] = {
    {256, 256, 1750, 12000}, {128, 128, 700, 5000}, {64, 128, 480, 4000}, {64, 64, 310, 3000}};
constexpr int kNumShapes = sizeof(kShapes) / sizeof(kShapes[0]);

// The shape whose rounds over the CUs cost least.  (Without a W there are no K
// steps to pay, but the fixed part alone would choose otherwise for one size in
// 700, so they are counted all the same.)
int pick_tile(int T, int N, int K, bool with_w, int cus) {
  int best = 1;
  double least = 1e300;
  for (int i = K % 128 == 0 && with_w ? 0 : 1; i < kNumShapes; ++i) {
    const Shape &s = kShapes[i];
    const double tiles = (double)((T + s.BM - 1) / s.BM) * ((N + s.BN - 1) / s.BN);
    double rounds = tiles / (cus > 0 ? cus : 256);
    if (rounds < 8) rounds = (double)(long long)(rounds + 0.9999);
    const double cost = rounds * ((K + 63) / 64 * (double)s.step + s.fixed);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

template <class Kernel, class... More>
void launch_tiles(Kernel kernel, int threads, int BM, int BNT, const char *x, const char *W, int ldw,
                  const char *F, const float *v, const int32_t *adapter, const int32_t *order, int T,
                  int N, int K, int r, int n, char *y, hipStream_t s, More... more) {
  const int MT = (T + BM - 1) / BM, NT = (N + BNT - 1) / BNT;
  hipLaunchKernelGGL(kernel, dim3(tile_grid(MT, NT)), dim3(threads), 0, s, x, W, ldw, F, v, adapter,
                     order, T, N, K, r, n, y, MT, NT, more...);
}

template <int OS>
void launch_bf16(const char *x, const char *W, int ldw, const char *F, const float *v,
                 const int32_t *adapter, const int32_t *order, int T, int N, int K, int r, int n,
                 char *y, int cus, hipStream_t s) {
  if (W && T <= kExpandRowsMax) {
    const dim3 grid((N + 15) / 16), block(kRowWaves * kWave);
#define MOE_ROWS(MB)                                                                             \
  hipLaunchKernelGGL((expand_rows_kernel<OS, MB>), grid, block, 0, s, x, W, ldw, F, v, adapter, T, \
                     N, K, r, n, y)
    if (T <= 16) MOE_ROWS(1);
    else MOE_ROWS(2);
#undef MOE_ROWS
    return;
  }
  const int rot = T <= 128 && (size_t)ldw * 2 % 4096 == 0;
#define MOE_TILES(kernel, BM, BNT) \
  launch_tiles(kernel, 256, BM, BNT, x, W, ldw, F, v, adapter, order, T, N, K, r, n, y, s, rot)
  switch (pick_tile(T, N, K, W != nullptr, cus)) {
    case 0:
      launch_tiles(expand_big_kernel<OS>, 256, 256, 256, x, W, ldw, F, v, adapter, order, T, N, K, r, n, y,
                   s);
      break;
    case 1: MOE_TILES((expand_ring_kernel<OS, 128, 128, 2, 2>), 128, 128); break;
    case 2: MOE_TILES((expand_ring_kernel<OS, 64, 128, 1, 4>), 64, 128); break;
    default: MOE_TILES((expand_ring_kernel<OS, 64, 64, 2, 2>), 64, 64); break;
  }
#undef MOE_TILES
}

}  // namespace

hipError_t launch_lora_expand(const void *x, const void *W, int ldw, const void *F, int dt,
                              const float *v, const int32_t *adapter, const int32_t *order, int T,
                              int N, int K, int r, int n, void *y, int y_dt, int cus,
                              hipStream_t s) {
  const char *xb = static_cast<const char *>(x), *wb = static_cast<const char *>(W),
             *fb = static_cast<const char *>(F);
  char *yb = static_cast<char *>(y);
  if (dt == MOE_F32) {
    const long long tiles = (long long)((T + 63) / 64) * ((N + 63) / 64);
    if (tiles < cus)
      launch_tiles(expand_f32_small_kernel, kF32Waves * moe::kWave, 32, 32, xb, wb, ldw, fb, v, adapter,
                   order, T, N, K, r, n, yb, s);
    else
      launch_tiles(expand_f32_kernel, kF32Threads, 64, 64, xb, wb, ldw, fb, v, adapter, order, T, N, K,
                   r, n, yb, s);
  }
  else if (y_dt == MOE_F32)
    launch_bf16<4>(xb, wb, ldw, fb, v, adapter, order, T, N, K, r, n, yb, cus, s);
  else
    launch_bf16<2>(xb, wb, ldw, fb, v, adapter, order, T, N, K, r, n, yb, cus, s);
  return hipGetLastError();
}
