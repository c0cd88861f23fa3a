// balance.hip -- the load-balance loss of a routing decision with its
// per-expert counts, and the gradient of the router's logits.
//
// "DeepGEMM walkthrough" §2.2: L_aux = alpha E sum_e f_e P_e, here over each
// sequence of a packed batch.  The softmax p_t is recomputed from the logits
// in both directions (T E values of exp against T E 4 bytes of traffic for
// storing it).
//
// A wave takes 64 / L tokens at once, L lanes each; a lane holds NP groups of
// four neighbouring experts (16-byte loads; E % 4 == 0) or NP single ones.
// Everything is one pass over the logits, and no launch is long enough to
// stream: it is one burst of loads between its start and its end, so what
// counts is that every load is issued before anything is looked up, that the
// code is short, and that the sums over a token's lanes are DPP.  Measured:
// loss of 32749 tokens of 256 experts (34 MB) 15.9 + 5.3 us, of 256 tokens of
// 8 3.7 us; gradient of 16381 tokens of 256 (34 MB) 12.6 us, of 4096 of 8
// 4.0 us.
#include "balance_internal.h"

namespace {

using namespace moe;

constexpr int kWavesP = 8;              // waves per workgroup
constexpr int kThreadsP = kWavesP * kWave;

// e^x for x <= 0 by the hardware exp2 (within 1 ulp) of the rounded product
// x log2(e): |x| 2^-24 more, so that the large probabilities, whose x is
// small, keep all their bits.  -inf gives 0.  (With what the product loses put
// back, and the normaliser's reciprocal refined, the gradient of 16381 tokens of
// 256 experts is off by 7.2e-8 of its norm instead of 7.8e-8, and the loss of
// 32749 tokens takes 23.5 us instead of 21.)
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// The first sequence s with off[s + 1] > t, S if there is none: 64 probes at a
// time by the lanes of a wave (one round of loads for up to 64 sequences,
// three for any number).  Whatever the offsets hold, the result is in [0, S].
// Must be called by a whole wave.
__device__ __forceinline__ int sequence_of(const int32_t *off, int S, int t) {
  int lo = 0, n = S;  // sequences before lo end at t or before, those from lo + n on do not
  while (n > 0) {
    const int step = (n + kWave - 1) / kWave;
    const int i = lo + min(((int)lane_id() + 1) * step, n) - 1;
    const unsigned long long behind = __ballot(off[i + 1] > t);
    if (behind == 0) return lo + n;
    const int f = __builtin_ctzll(behind), hit = lo + min((f + 1) * step, n) - 1;
    lo += f * step;
    n = hit - lo;
  }
  return lo;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The lanes' share of one row of E values: a token has L lanes (a power of
// two); lane l's values are those of experts expert(i, l).
template <int L_, int NP, bool VEC>
struct Row {
  static constexpr int L = L_, V = VEC ? 4 * NP : NP;
  float v[V];
  static __device__ __forceinline__ int expert(int i, int l) {
    return VEC ? ((i >> 2) * L + l) * 4 + (i & 3) : i * L + l;
  }
  // -inf behind E
  __device__ __forceinline__ void load(const float *row, int l, int E) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = (i * L + l) * 4;
        const f32x4 q = *reinterpret_cast<const f32x4 *>(row + min(e, E - 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * i + c] = q[c];
      }
      if (E < L * V) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = expert(i, l) < E ? v[i] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float q = row[min(i * L + l, E - 1)];
        v[i] = i * L + l < E ? q : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void store(float *row, int l, int E) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = (i * L + l) * 4;
        if (e < E)
          *reinterpret_cast<f32x4 *>(row + e) =
              f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (i * L + l < E) row[i * L + l] = v[i];
    }
  }
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f;
  }
};

// f over the L lanes of a token, the same value in each of them: exchanges
// inside a row of 16 lanes by DPP (neighbours, pairs, mirrored halves), then
// the swaps of 16- and 32-lane halves.  The order is fixed.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int L, class T, class F>
__device__ __forceinline__ T over_lanes(T v, F f) {
  if constexpr (L >= 2) v = f(v, dpp<0xB1>(v));    // lane ^ 1
  if constexpr (L >= 4) v = f(v, dpp<0x4E>(v));    // lane ^ 2
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));   // 7 - lane of 8
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));  // 15 - lane of 16
  if constexpr (L >= 32) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto q = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned a = q[0], b = q[1];
    v = f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  }
  if constexpr (L >= 64) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = q[0], b = q[1];
    v = f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return over_lanes<L>(v, [](float a, float b) { return a + b; });
}
// the maximum by the bits as integers of the same order: one instruction an
// exchange, where a floating maximum first quiets both operands
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  int u = __float_as_int(v);
  u ^= (u >> 31) & 0x7fffffff;
  u = over_lanes<L>(u, [](int a, int b) { return max(a, b); });
  u ^= (u >> 31) & 0x7fffffff;
  return __int_as_float(u);
}

// logits -> probabilities in place; a row of -inf only becomes zeros
template <class R>
__device__ __forceinline__ void softmax_row(R &x) {
  float m = x.v[0];
#pragma unroll
  for (int i = 1; i < R::V; ++i) m = fmaxf(m, x.v[i]);
  m = lanes_max<R::L>(m);
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < R::V; ++i) {
    x.v[i] = exp_neg(x.v[i] - m);
    z += x.v[i];
  }
  z = lanes_sum<R::L>(z);
  const float inv = z != 0.f ? __builtin_amdgcn_rcpf(z) : 0.f;  // (within 1 ulp)
#pragma unroll
  for (int i = 0; i < R::V; ++i) x.v[i] *= inv;
}

// ---------------------------------------------------------------------------
// loss, first launch: block b (C tokens) writes, for every sequence s that
// has tokens in it, slot b + s: the sums of the probabilities, the counts
// and the number of tokens that take part.  b + s is a slot of its own for
// each such pair: going along the tokens, b or s grows from pair to pair and
// neither ever falls.  A batch of one block and one sequence is finished here.
// ---------------------------------------------------------------------------
struct LossOut {
  int32_t *counts;
  float *probs;
  int32_t *tokens;
  float *loss;
};

template <class R>
__global__ __launch_bounds__(kThreadsP) void balance_partial_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const int32_t *__restrict__ off, const uint8_t *__restrict__ mask, int T, int E, int k, int S,
    int C, float alpha, float *__restrict__ slot_p, int32_t *__restrict__ slot_c,
    int32_t *__restrict__ slot_n, int32_t *__restrict__ ticket, LossOut out) {
  constexpr int L = R::L, nq = kWave / L;
  __shared__ float s_p[kWavesP][MOE_MAX_EXPERTS];
  __shared__ int s_c[MOE_MAX_EXPERTS];
  __shared__ int s_n;
  __shared__ float s_w[kWavesP];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int l = lane & (L - 1), q = lane / L;
  const int b = blockIdx.x, b0 = b * C, b1 = min(T, b0 + C);
  const bool whole = gridDim.x == 1 && S == 1;
  if (b == 0 && tid == 0) *ticket = 0;
  constexpr int step = kWavesP * nq;  // token slots of the workgroup
  // A batch is one token of every slot: the other waves of the CU cover its
  // latency, in less code than several tokens a lane (which arrives slower
  // than the data; 32749 tokens of 256 experts: 17.4 us with four, 16.0 with
  // one).  The first one is loaded before anything else is looked up: which
  // tokens take part in which sequence is decided when its probabilities are
  // there.
  R x;
  bool on = false;
  auto load = [&](int t) {
    const int tc = max(min(t, b1 - 1), 0);
    if (b1 > b0) x.load(logits + (size_t)tc * E, l, E);
    on = t < b1;
    if (mask) on = on && mask[tc];
  };
  const int slot = b0 + wv * nq + q;  // the lane's first token
  load(slot);
  // entry i of the block: an expert, -1 if it counts for none
  const int entries = (b1 - b0) * k;
  auto entry = [&](int i) {
    const int ic = max(min(i, entries - 1), 0);
    const int e = entries > 0 ? topk_idx[(size_t)b0 * k + ic] : -1;
    bool in = i < entries && e >= 0 && e < E;
    if (mask && entries > 0) in = in && mask[b0 + ic / k];
    return in ? e : -1;
  };
  const int e0 = entry(tid);
  int s = off && !whole ? sequence_of(off, S, b0) : 0;
  bool first = true;
  for (; s < S; ++s) {
    const int lo = off ? off[s] : 0, hi = off ? off[s + 1] : T;
    if (lo >= b1 && !whole) break;
    const int ta = max(lo, b0), tb = min(hi, b1);
    if (ta >= tb && !whole) {  // empty: past all such at once
      s += max(sequence_of(off + s, S - s, max(lo, b0)) - 1, 0);
      continue;
    }
    for (int e = tid; e < E; e += kThreadsP) s_c[e] = 0;
    if (tid == 0) s_n = 0;
    __syncthreads();
    for (int i = tid; i < entries; i += kThreadsP) {
      const int e = i == tid ? e0 : entry(i), t = b0 + i / k;
      if (e >= 0 && t >= ta && t < tb) atomicAdd(&s_c[e], 1);
    }
    int n_mine = 0;  // tokens of the wave that take part
    float acc[R::V];
#pragma unroll
    for (int i = 0; i < R::V; ++i) acc[i] = 0.f;
    for (int t = slot; t - q < b1; t += step) {
      if (!first) load(t);
      first = b1 - b0 <= step;  // the block is one batch: it stays loaded
      const bool in = on && t >= ta && t < tb;
      n_mine += __popcll(__ballot(in && l == 0));
      R p = x;
      softmax_row(p);
#pragma unroll
      for (int i = 0; i < R::V; ++i) acc[i] += in ? p.v[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < R::V; ++i) {
      for (int o = L; o < kWave; o <<= 1) acc[i] += __shfl_xor(acc[i], o, kWave);
      const int e = R::expert(i, l);
      if (q == 0 && e < E) s_p[wv][e] = acc[i];
    }
    if (lane == 0) atomicAdd(&s_n, n_mine);
    __syncthreads();
    const size_t base = (size_t)(b + s) * E;
    float dot = 0.f;
    const float fn = (float)max(s_n, 1);
    for (int e = tid; e < E; e += kThreadsP) {
      float p = s_p[0][e];
#pragma unroll
      for (int w = 1; w < kWavesP; ++w) p += s_p[w][e];
      if (whole) {
        p /= fn;
        out.counts[e] = s_c[e];
        out.probs[e] = p;
        dot += (float)s_c[e] / (fn * (float)k) * p;
      } else {
        slot_p[base + e] = p;
        slot_c[base + e] = s_c[e];
      }
    }
    if (whole) {
      dot = wave_sum(dot);
      if (lane == 0) s_w[wv] = dot;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kWavesP; ++w) dot += s_w[w];
        out.tokens[0] = s_n;
        out.tokens[1] = s_n > 0;
        *out.loss = s_n > 0 ? alpha * (float)E * dot : 0.f;
      }
      return;
    }
    if (tid == 0) slot_n[b + s] = s_n;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// loss, second launch: workgroup (s, 64 experts) adds its sequence's slots
// in a fixed order; the last workgroup to finish adds the sequences' losses,
// again in a fixed order.  What a thread adds over its loop is held in 64 bits:
// a sequence may have a million slots of much the same size, whose roundings in
// 32 bits all fall on one side (2^24 equal tokens of 2 experts: 2^-14 of a
// probability).
// ---------------------------------------------------------------------------
constexpr int kGroupsF = 16;  // waves per workgroup, each a share of the slots

__global__ __launch_bounds__(kGroupsF *kWave) void balance_final_kernel(
    const float *__restrict__ slot_p, const int32_t *__restrict__ slot_c,
    const int32_t *__restrict__ slot_n, const int32_t *__restrict__ off, int T, int E, int k, int S,
    int C, int EC, float alpha, int32_t *__restrict__ counts, float *__restrict__ probs,
    int32_t *__restrict__ tokens, float *__restrict__ loss, float *__restrict__ dots,
    int32_t *__restrict__ ticket) {
  __shared__ float s_p[kGroupsF][kWave];
  __shared__ int s_c[kGroupsF][kWave];
  __shared__ int s_n[kGroupsF];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = lane_id(), g = tid / kWave;
  const int s = blockIdx.x / EC, ec = blockIdx.x - s * EC;
  const int e = ec * kWave + lane;
  const int lo = off ? clampi(off[s], 0, T) : 0, hi = off ? clampi(off[s + 1], 0, T) : T;
  float p = 0.f;
  int c = 0, n = 0;
  if (lo < hi) {
    double all = 0.;
    const int k1 = (hi - 1) / C;
    constexpr int U = 4;
    for (int k0 = lo / C + g; k0 <= k1; k0 += U * kGroupsF) {
      float pv[U];
      int cv[U], nv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kb = k0 + u * kGroupsF;
        const bool in = kb <= k1;
        const size_t at = (size_t)((in ? kb : k1) + s);
        nv[u] = in ? slot_n[at] : 0;
        pv[u] = in && e < E ? slot_p[at * E + e] : 0.f;
        cv[u] = in && e < E ? slot_c[at * E + e] : 0;
      }
#pragma unroll
      for (int u = 1; u < U; ++u) pv[0] += pv[u];
      all += (double)pv[0];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        c += cv[u];
        n += nv[u];
      }
    }
    p = (float)all;
  }
  s_p[g][lane] = p;
  s_c[g][lane] = c;
  if (lane == 0) s_n[g] = n;
  __syncthreads();
  if (g == 0) {
    p = s_p[0][lane];
    c = s_c[0][lane];
    n = s_n[0];
    for (int w = 1; w < kGroupsF; ++w) {
      p += s_p[w][lane];
      c += s_c[w][lane];
      n += s_n[w];
    }
    const float fn = (float)max(n, 1), mean = p / fn;
    if (e < E) {
      counts[(size_t)s * E + e] = c;
      probs[(size_t)s * E + e] = mean;
    }
    const float d = wave_sum(e < E ? (float)c / (fn * (float)k) * mean : 0.f);
    if (lane == 0) {
      // read by the last workgroup, perhaps on another XCD
      __hip_atomic_store(&dots[blockIdx.x], d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (ec == 0)
        __hip_atomic_store(&tokens[s], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = 1;
      if (gridDim.x > 1) {
        s_last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                 (int)gridDim.x - 1;
      }
    }
  }
  __syncthreads();
  if (!s_last) return;
  double part = 0.;
  int some = 0;
  for (int i = tid; i < (int)gridDim.x; i += kGroupsF * kWave)  // (0 for an empty sequence)
    part += (double)__hip_atomic_load(&dots[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < S; i += kGroupsF * kWave)
    some += __hip_atomic_load(&tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
  float sum = wave_sum((float)part);
  for (int o = 32; o > 0; o >>= 1) some += __shfl_xor(some, o, kWave);
  if (lane == 0) {
    s_p[0][g] = sum;
    s_c[0][g] = some;
  }
  __syncthreads();
  if (tid == 0) {
    sum = 0.f;
    some = 0;
    for (int w = 0; w < kGroupsF; ++w) {
      sum += s_p[0][w];
      some += s_c[0][w];
    }
    tokens[S] = some;
    *loss = alpha * (float)E * sum / (float)max(some, 1);
  }
}

// ---------------------------------------------------------------------------
// gradient of the logits
// ---------------------------------------------------------------------------
// The selected experts of one token, spread over its lanes: lane l holds
// entries l, l + L, ... (k <= E <= V L, so at most V of them), -1 for none.
template <class R, bool GATHER>
struct Picked {
  static constexpr int L = R::L, N = R::V < (MOE_MAX_TOPK + L - 1) / L ? R::V : (MOE_MAX_TOPK + L - 1) / L;
  int e[N];
  float d[N], z[GATHER ? N : 1];  // gradient of the weight; logit
  __device__ __forceinline__ void load(const int32_t *idx, const float *dw, const float *row, int k,
                                       int E, int l) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int j = c * L + l, jc = min(j, k - 1);
      const int en = idx[jc];
      const float dn = dw[jc];
      const bool in = j < k && en >= 0 && en < E;
      e[c] = in ? en : -1;
      d[c] = in ? dn : 0.f;
      if constexpr (GATHER) {
        const float zn = row[in ? en : 0];
        z[c] = in ? zn : -INFINITY;
      }
    }
  }
};

// LDS operations of one wave, in program order for the compiler too
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Tokens in flight per token slot: few, so that the code, which runs once a
// workgroup and arrives slower than the data, is short (4096 tokens of 8
// experts: 6.8 us with four, 4.8 with two, 3.9 with one; 16381 of 256: 12.9,
// 12.5, 13.3).
template <class R>
constexpr int backward_batch() { return R::L >= 32 && R::V <= 8 ? 2 : 1; }

template <class R, bool RENORM>
__global__ __launch_bounds__(256) void route_backward_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ dw, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ tokens, float alpha, const float *__restrict__ d_loss,
    const int32_t *__restrict__ off, const uint8_t *__restrict__ mask, int T, int E, int k, int S,
    int C, float *__restrict__ out) {
  constexpr int U = backward_batch<R>(), L = R::L, nq = kWave / L, NW = 256 / kWave;
  constexpr int step = NW * nq;
  using P = Picked<R, RENORM>;
  __shared__ __align__(16) float s_g[NW][U * kWave * R::V];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int l = lane & (L - 1), q = lane / L;
  const int b0 = blockIdx.x * C, b1 = min(T, b0 + C);
  const int first = wv * nq + q;
  // the balance term's factor, looked up beside the first loads
  const float some = counts ? (float)max(tokens[S], 1) : 1.f;
  const float scale = counts ? (d_loss ? *d_loss : 1.f) * alpha * (float)E / some : 0.f;
  const int s_first = off ? sequence_of(off, S, b0) : 0;
  for (int t0 = b0 + first; t0 - q < b1; t0 += U * step) {
    // every load of the batch first
    R x[U];
    P pick[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * step, tc = min(t, b1 - 1);
      on[u] = t < b1;
      if (mask) on[u] = on[u] && mask[tc];
      x[u].load(logits + (size_t)tc * E, l, E);
      if (dw)
        pick[u].load(topk_idx + (size_t)tc * k, dw + (size_t)tc * k, logits + (size_t)tc * E, k, E, l);
    }
    R g[U];  // the gate's part: of p (raw), of the logits (renormalised)
    if (dw) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u].fill(0.f);
        g[u].store(s_g[wv] + (u * nq + q) * (R::V * L), l, R::V * L);
      }
      wave_order();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dw) {
        if constexpr (RENORM) {
          // q over the selected logits, shifted by their own maximum; d
          // becomes the gradient of the entry's logit
          float m = pick[u].z[0], z = 0.f, dot = 0.f;
#pragma unroll
          for (int c = 1; c < P::N; ++c) m = fmaxf(m, pick[u].z[c]);
          m = lanes_max<L>(m);
          if (m == -INFINITY) m = 0.f;
#pragma unroll
          for (int c = 0; c < P::N; ++c) {
            pick[u].z[c] = exp_neg(pick[u].z[c] - m);
            z += pick[u].z[c];
            dot = fmaf(pick[u].z[c], pick[u].d[c], dot);
          }
          z = lanes_sum<L>(z);
          const float inv = z != 0.f ? 1.f / z : 0.f;
          dot = lanes_sum<L>(dot) * inv;
#pragma unroll
          for (int c = 0; c < P::N; ++c) pick[u].d[c] = pick[u].z[c] * inv * (pick[u].d[c] - dot);
        }
        // the entries meet their experts' lanes in the wave's own LDS (an
        // expert that is there twice takes both)
        float *sc = s_g[wv] + (u * nq + q) * (R::V * L);
#pragma unroll
        for (int c = 0; c < P::N; ++c)
          if (pick[u].e[c] >= 0)
            __hip_atomic_fetch_add(&sc[pick[u].e[c]], pick[u].d[c], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WAVEFRONT);
      }
      softmax_row(x[u]);
    }
    if (dw) wave_order();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      g[u].fill(0.f);
      if (dw) g[u].load(s_g[wv] + (u * nq + q) * (R::V * L), l, R::V * L);
    }
    // the batch's tokens sequence by sequence; b[e], the balance loss's
    // derivative by p_t[e], is the same for a whole sequence
    bool done[U] = {};
    for (int s = s_first; s < S; ++s) {
      const int lo = off ? off[s] : 0, hi = off ? off[s + 1] : T;
      if (lo >= b1) break;
      if (max(lo, b0) >= min(hi, b1)) {  // empty: past all such at once
        s += max(sequence_of(off + s, S - s, max(lo, b0)) - 1, 0);
        continue;
      }
      R bal;
      bal.fill(0.f);
      if (counts) {
        const float n = (float)max(tokens[s], 1);
#pragma unroll
        for (int i = 0; i < R::V; ++i) {
          const int e = R::expert(i, l), c = counts[(size_t)s * E + min(e, E - 1)];
          bal.v[i] = e < E ? scale / n * ((float)c / (n * (float)k)) : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * step;
        const bool mine = on[u] && t >= lo && t < hi;
        float dot = 0.f;
        R r;
#pragma unroll
        for (int i = 0; i < R::V; ++i) {
          r.v[i] = RENORM ? bal.v[i] : bal.v[i] + g[u].v[i];
          dot = fmaf(x[u].v[i], r.v[i], dot);
        }
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < R::V; ++i) {
          r.v[i] = x[u].v[i] * (r.v[i] - dot);
          if constexpr (RENORM) r.v[i] += g[u].v[i];
        }
        if (mine) {
          r.store(out + (size_t)t * E, l, E);
          done[u] = true;
        }
      }
    }
    R zero;  // tokens that take no part
    zero.fill(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u * step < b1 && !done[u]) zero.store(out + (size_t)(t0 + u * step) * E, l, E);
  }
}

// lanes per token
int lanes_for(int E) {
  const int pieces = E % 4 == 0 ? E / 4 : E;
  int L = 1;
  while (L < pieces && L < kWave) L <<= 1;
  return L;
}

// f(Row) with the compiled row shape for E experts
template <int NP, bool VEC, class F>
void with_lanes(int L, F f) {
  switch (L) {
    case 1: f(Row<1, NP, VEC>()); break;
    case 2: f(Row<2, NP, VEC>()); break;
    case 4: f(Row<4, NP, VEC>()); break;
    case 8: f(Row<8, NP, VEC>()); break;
    case 16: f(Row<16, NP, VEC>()); break;
    case 32: f(Row<32, NP, VEC>()); break;
    default: f(Row<64, NP, VEC>()); break;
  }
}
template <class F>
void with_row(int E, F f) {
  const int L = lanes_for(E);
  if (E % 4 == 0) {
    const int np = (E / 4 + L - 1) / L;
    if (np <= 1) with_lanes<1, true>(L, f);
    else if (np <= 2) f(Row<64, 2, true>());
    else f(Row<64, 4, true>());
  } else {
    const int np = (E + L - 1) / L;
    if (np <= 1) with_lanes<1, false>(L, f);
    else if (np <= 2) f(Row<64, 2, false>());
    else if (np <= 4) f(Row<64, 4, false>());
    else if (np <= 8) f(Row<64, 8, false>());
    else f(Row<64, 16, false>());
  }
}

// token slots of a workgroup of the loss's first launch
int loss_batch(int E) { return kWavesP * (kWave / lanes_for(E)); }

// Tokens per block of the loss's first launch.  A small batch is one block
// (a workgroup's loads of a few thousand values cost less than a second
// launch); otherwise one batch of the workgroup's token slots, at least 64
// tokens (the second launch reads as many slots as there are blocks: with 32
// it takes 6.3 us instead of 5.1 at 32749 tokens of 256 experts, the first as
// long as before), halved down to 16 while there are fewer than 512 blocks
// (two per CU; with one, of 128 tokens, the first takes 22.6 us instead of 16).
int loss_block(int T, int E, int S, int batch) {
  if (S == 1 && (long long)T * E <= 16384) return T > 0 ? T : 1;
  int C = batch > 64 ? batch : 64;
  while (C > 16 && (T + C - 1) / C < 512) C >>= 1;
  return C;
}

struct LossWs {
  size_t p, c, n, dots, ticket, bytes;
};

LossWs loss_ws(int T, int E, int S) {
  const int C = loss_block(T, E, S, loss_batch(E)), EC = (E + kWave - 1) / kWave;
  const size_t slots = (size_t)((T + C - 1) / C) + S;
  LossWs w;
  w.p = 0;
  w.c = w.p + slots * E * 4;
  w.n = w.c + slots * E * 4;
  w.dots = w.n + slots * 4;
  w.ticket = w.dots + (size_t)S * EC * 4;
  w.bytes = w.ticket + 4;
  return w;
}

}  // namespace

size_t balance_loss_ws_bytes(int T, int E, int S) { return loss_ws(T, E, S).bytes; }

hipError_t launch_balance_loss(const float *logits, const int32_t *topk_idx, const int32_t *off,
                               const uint8_t *mask, int T, int E, int k, int S, float alpha,
                               int32_t *counts, float *probs, int32_t *tokens, float *loss, void *ws,
                               hipStream_t s) {
  const int C = loss_block(T, E, S, loss_batch(E)), EC = (E + kWave - 1) / kWave;
  const LossWs w = loss_ws(T, E, S);
  char *base = static_cast<char *>(ws);
  float *p = reinterpret_cast<float *>(base + w.p);
  int32_t *c = reinterpret_cast<int32_t *>(base + w.c), *n = reinterpret_cast<int32_t *>(base + w.n);
  float *dots = reinterpret_cast<float *>(base + w.dots);
  int32_t *ticket = reinterpret_cast<int32_t *>(base + w.ticket);
  // (one block for an empty batch too)
  const int blocks = max(1, (T + C - 1) / C);
  const LossOut out = {counts, probs, tokens, loss};
  with_row(E, [&](auto row) {
    hipLaunchKernelGGL((balance_partial_kernel<decltype(row)>), dim3(blocks), dim3(kThreadsP), 0, s,
                       logits, topk_idx, off, mask, T, E, k, S, C, alpha, p, c, n, ticket, out);
  });
  if (blocks > 1 || S > 1)
    hipLaunchKernelGGL(balance_final_kernel, dim3(S * EC), dim3(kGroupsF * kWave), 0, s, p, c, n, off,
                       T, E, k, S, C, EC, alpha, counts, probs, tokens, loss, dots, ticket);
  return hipGetLastError();
}

hipError_t launch_route_backward(const float *logits, const int32_t *topk_idx, const float *dw,
                                 bool renorm, const int32_t *counts, const int32_t *tokens,
                                 float alpha, const float *d_loss, const int32_t *off,
                                 const uint8_t *mask, int T, int E, int k, int S, float *d_logits,
                                 hipStream_t s) {
  with_row(E, [&](auto row) {
    using R = decltype(row);
    // tokens per workgroup: one batch of its token slots, at least 8
    const int C = max(8, backward_batch<R>() * (256 / R::L));
    const dim3 grid((T + C - 1) / C), block(256);
    if (renorm)
      hipLaunchKernelGGL((route_backward_kernel<R, true>), grid, block, 0, s, logits, topk_idx, dw,
                         counts, tokens, alpha, d_loss, off, mask, T, E, k, S, C, d_logits);
    else
      hipLaunchKernelGGL((route_backward_kernel<R, false>), grid, block, 0, s, logits, topk_idx, dw,
                         counts, tokens, alpha, d_loss, off, mask, T, E, k, S, C, d_logits);
  });
  return hipGetLastError();
}
