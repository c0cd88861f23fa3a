// balance.hip -- the load-balance loss of a routing decision with its
// per-expert counts, and the gradient of the router's logits.
//
// "DeepGEMM walkthrough" §2.2: L_aux = alpha E sum_e f_e P_e, here over each
// sequence of a packed batch.  The softmax p_t is recomputed from the logits
// in both directions (T E values of exp against T E 4 bytes of traffic for
// storing it).
//
// A wave takes 64 / L tokens at once, L lanes each; a lane holds 4 NP
// consecutive-by-four experts (16-byte loads; E % 4 == 0) or NP strided ones.
// Everything is one pass over the logits: HBM-bound on large batches,
// latency-bound on small ones.
#include "moe_internal.h"
#include "../../include/moe_balance.h"

namespace {

using namespace moe;

constexpr int kWavesP = 8;              // waves per workgroup
constexpr int kThreadsP = kWavesP * kWave;

// e^x for x <= 0: exp2 of the rounded product x log2(e), corrected to first
// order by the product's rounding error and the low part of log2(e).  The
// hardware exp2 is within 1 ulp; without the correction the error grows to
// |x| ulp.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f, kLn2 = 0.693147182f;
  const float t = x * kHi;
  if (!(t > -150.f)) return x != x ? x : 0.f;  // underflows (also x = -inf)
  const float lo = fmaf(x, kHi, -t) + x * kLo;
  const float r = __builtin_amdgcn_exp2f(t);
  return fmaf(r, lo * kLn2, r);
}

// Token t's sequence: the first s with off[s + 1] > t, S if there is none
// (offsets as stored; whatever they hold, the result is in [0, S]).
__device__ __forceinline__ int sequence_of(const int32_t *off, int S, int t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The lanes' share of one row of E values.
template <int NP, bool VEC>
struct Row {
  static constexpr int V = VEC ? 4 * NP : NP;
  float v[V];
  static __device__ __forceinline__ int expert(int i, int l, int L) {
    return VEC ? ((i >> 2) * L + l) * 4 + (i & 3) : i * L + l;
  }
  __device__ __forceinline__ void load(const float *row, int l, int L, int E) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = (i * L + l) * 4;
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) q = *reinterpret_cast<const float4 *>(row + e);
        v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = i * L + l < E ? row[i * L + l] : -INFINITY;
    }
  }
  __device__ __forceinline__ void store(float *row, int l, int L, int E) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = (i * L + l) * 4;
        if (e < E)
          *reinterpret_cast<float4 *>(row + e) =
              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (i * L + l < E) row[i * L + l] = v[i];
    }
  }
};

// sum / maximum over the L lanes of a token (L a power of two)
__device__ __forceinline__ float lanes_sum(float v, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
__device__ __forceinline__ float lanes_max(float v, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

// logits -> probabilities in place; a row of -inf only becomes zeros
template <int NP, bool VEC>
__device__ __forceinline__ void softmax_row(Row<NP, VEC> &x, int L) {
  constexpr int V = Row<NP, VEC>::V;
  float m = x.v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, x.v[i]);
  m = lanes_max(m, L);
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x.v[i] = exp_neg(x.v[i] - m);
    z += x.v[i];
  }
  z = lanes_sum(z, L);
  const float inv = z != 0.f ? 1.f / z : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) x.v[i] *= inv;
}

// tokens in flight per token slot: enough loads to cover the latency without
// running out of registers
template <int NP, bool VEC>
constexpr int unroll_of() { return Row<NP, VEC>::V <= 4 ? 4 : (Row<NP, VEC>::V <= 8 ? 2 : 1); }

// ---------------------------------------------------------------------------
// loss, first launch: block b (C tokens) writes, for every sequence s that
// has tokens in it, slot b + s: the sums of the probabilities, the counts
// and the number of tokens that take part.  b + s is a slot of its own for
// each such pair: going along the tokens, b or s grows from pair to pair and
// neither ever falls.
// ---------------------------------------------------------------------------
template <int NP, bool VEC>
__global__ __launch_bounds__(kThreadsP) void balance_partial_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const int32_t *__restrict__ off, const uint8_t *__restrict__ mask, int T, int E, int k, int S,
    int C, int L, float *__restrict__ slot_p, int32_t *__restrict__ slot_c,
    int32_t *__restrict__ slot_n, int32_t *__restrict__ ticket) {
  using R = Row<NP, VEC>;
  constexpr int U = unroll_of<NP, VEC>();
  __shared__ float s_p[kWavesP][MOE_MAX_EXPERTS];
  __shared__ int s_c[MOE_MAX_EXPERTS];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int l = lane & (L - 1), q = lane / L, nq = kWave / L;
  const int b = blockIdx.x, b0 = b * C, b1 = min(T, b0 + C);
  if (b == 0 && tid == 0) *ticket = 0;
  int s = off ? sequence_of(off, S, b0) : 0;
  for (; s < S; ++s) {
    const int lo = off ? off[s] : 0, hi = off ? off[s + 1] : T;
    if (lo >= b1) break;
    const int ta = max(lo, b0), tb = min(hi, b1);
    if (ta >= tb) continue;
    for (int e = tid; e < E; e += kThreadsP) s_c[e] = 0;
    if (tid == 0) s_n = 0;
    __syncthreads();
    for (int i = tid; i < (tb - ta) * k; i += kThreadsP) {
      const int e = topk_idx[(size_t)ta * k + i];
      if ((!mask || mask[ta + i / k]) && e >= 0 && e < E) atomicAdd(&s_c[e], 1);
    }
    for (int t = ta + tid; t < tb; t += kThreadsP)
      if (!mask || mask[t]) atomicAdd(&s_n, 1);
    float acc[R::V];
#pragma unroll
    for (int i = 0; i < R::V; ++i) acc[i] = 0.f;
    const int step = kWavesP * nq;
    for (int t0 = ta + wv * nq + q; t0 - q < tb; t0 += U * step) {
      R x[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * step;
        on[u] = t < tb && (!mask || mask[t]);
        if (on[u]) {
          x[u].load(logits + (size_t)t * E, l, L, E);
        } else {
#pragma unroll
          for (int i = 0; i < R::V; ++i) x[u].v[i] = -INFINITY;  // probability 0
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        softmax_row(x[u], L);
#pragma unroll
        for (int i = 0; i < R::V; ++i) acc[i] += x[u].v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < R::V; ++i) {
      for (int o = L; o < kWave; o <<= 1) acc[i] += __shfl_xor(acc[i], o, kWave);
      const int e = R::expert(i, l, L);
      if (q == 0 && e < E) s_p[wv][e] = acc[i];
    }
    __syncthreads();
    const size_t base = (size_t)(b + s) * E;
    for (int e = tid; e < E; e += kThreadsP) {
      float p = s_p[0][e];
#pragma unroll
      for (int w = 1; w < kWavesP; ++w) p += s_p[w][e];
      slot_p[base + e] = p;
      slot_c[base + e] = s_c[e];
    }
    if (tid == 0) slot_n[b + s] = s_n;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// loss, second launch: workgroup (s, 64 experts) adds its sequence's slots
// in a fixed order; the last workgroup to finish adds the sequences' losses,
// again in a fixed order.
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
      for (int u = 0; u < U; ++u) {
        p += pv[u];
        c += cv[u];
        n += nv[u];
      }
    }
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
    const float fn = (float)max(n, 1);
    p = p / fn;
    if (e < E) {
      counts[(size_t)s * E + e] = c;
      probs[(size_t)s * E + e] = p;
    }
    const float d = wave_sum(e < E ? (float)c / (fn * (float)k) * p : 0.f);
    if (lane == 0) {
      // read by the last workgroup, perhaps on another XCD
      __hip_atomic_store(&dots[blockIdx.x], d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (ec == 0)
        __hip_atomic_store(&tokens[s], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __threadfence();
      s_last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float sum = 0.f;
  int some = 0;
  for (int i = tid; i < S; i += kGroupsF * kWave) {
    const int ns = __hip_atomic_load(&tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (ns <= 0) continue;
    ++some;
    for (int j = 0; j < EC; ++j)
      sum += __hip_atomic_load(&dots[i * EC + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  sum = wave_sum(sum);
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
template <int NP, bool VEC, bool RENORM>
__global__ __launch_bounds__(256) void route_backward_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ dw, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ tokens, float alpha, const float *__restrict__ d_loss,
    const int32_t *__restrict__ off, const uint8_t *__restrict__ mask, int T, int E, int k, int S,
    int C, int L, float *__restrict__ out) {
  using R = Row<NP, VEC>;
  constexpr int U = R::V <= 4 ? 2 : 1;
  constexpr int NW = 256 / kWave;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave;
  const int l = lane & (L - 1), q = lane / L, nq = kWave / L, step = NW * nq;
  const int b0 = blockIdx.x * C, b1 = min(T, b0 + C);
  const int first = wv * nq + q;
  R zero;
#pragma unroll
  for (int i = 0; i < R::V; ++i) zero.v[i] = 0.f;
  if (off) {  // rows outside every sequence
    const int lo = off[0], hi = off[S];
    for (int t = b0 + first; t < b1; t += step)
      if (t < lo || t >= hi) zero.store(out + (size_t)t * E, l, L, E);
  }
  int s = off ? sequence_of(off, S, b0) : 0;
  for (; s < S; ++s) {
    const int lo = off ? off[s] : 0, hi = off ? off[s + 1] : T;
    if (lo >= b1) break;
    const int ta = max(lo, b0), tb = min(hi, b1);
    if (ta >= tb) continue;
    // b[e], the balance loss's derivative by p_t[e], the same for the whole
    // sequence
    float bal[R::V];
#pragma unroll
    for (int i = 0; i < R::V; ++i) bal[i] = 0.f;
    if (counts) {
      const float n = (float)max(tokens[s], 1), some = (float)max(tokens[S], 1);
      const float coef = (d_loss ? *d_loss : 1.f) * alpha * (float)E / (some * n);
#pragma unroll
      for (int i = 0; i < R::V; ++i) {
        const int e = R::expert(i, l, L);
        if (e < E) bal[i] = coef * ((float)counts[(size_t)s * E + e] / (n * (float)k));
      }
    }
    for (int t0 = ta + first; t0 - q < tb; t0 += U * step) {
      R x[U];
      bool on[U], in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * step;
        in[u] = t < tb;
        on[u] = in[u] && (!mask || mask[t]);
        if (on[u]) {
          x[u].load(logits + (size_t)t * E, l, L, E);
        } else {
#pragma unroll
          for (int i = 0; i < R::V; ++i) x[u].v[i] = -INFINITY;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t t = (size_t)(t0 + u * step);
        float g[R::V];
#pragma unroll
        for (int i = 0; i < R::V; ++i) g[i] = bal[i];
        float add[RENORM ? R::V : 1];
        if (RENORM) {
#pragma unroll
          for (int i = 0; i < (RENORM ? R::V : 1); ++i) add[i] = 0.f;
        }
        if (dw && on[u]) {
          if (RENORM) {
            // q over the selected logits, shifted by their own maximum
            float m = -INFINITY, z = 0.f, dot = 0.f;
            for (int j = 0; j < k; ++j) {
              const int e = topk_idx[t * k + j];
              if (e >= 0 && e < E) m = fmaxf(m, logits[t * E + e]);
            }
            if (m == -INFINITY) m = 0.f;
            for (int j = 0; j < k; ++j) {
              const int e = topk_idx[t * k + j];
              if (e < 0 || e >= E) continue;
              const float w = exp_neg(logits[t * E + e] - m);
              z += w;
              dot = fmaf(w, dw[t * k + j], dot);
            }
            const float inv = z != 0.f ? 1.f / z : 0.f;
            dot *= inv;
            for (int j = 0; j < k; ++j) {
              const int e = topk_idx[t * k + j];
              if (e < 0 || e >= E) continue;
              const float part = exp_neg(logits[t * E + e] - m) * inv * (dw[t * k + j] - dot);
#pragma unroll
              for (int i = 0; i < (RENORM ? R::V : 1); ++i)
                add[i] += R::expert(i, l, L) == e ? part : 0.f;
            }
          } else {
            for (int j = 0; j < k; ++j) {
              const int e = topk_idx[t * k + j];
              const float d = dw[t * k + j];
#pragma unroll
              for (int i = 0; i < R::V; ++i) g[i] += R::expert(i, l, L) == e ? d : 0.f;
            }
          }
        }
        softmax_row(x[u], L);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < R::V; ++i) dot = fmaf(x[u].v[i], g[i], dot);
        dot = lanes_sum(dot, L);
        R r;
#pragma unroll
        for (int i = 0; i < R::V; ++i) {
          r.v[i] = x[u].v[i] * (g[i] - dot);
          if (RENORM) r.v[i] += add[RENORM ? i : 0];
          if (!on[u]) r.v[i] = 0.f;
        }
        if (in[u]) r.store(out + t * E, l, L, E);
      }
    }
  }
}

// lanes per token
int lanes_for(int E) {
  const int pieces = E % 4 == 0 ? E / 4 : E;
  int L = 1;
  while (L < pieces && L < kWave) L <<= 1;
  return L;
}

// tokens per block of the loss's first launch: 16 (as many workgroups as a
// small batch can give), doubled while more than 512 blocks remain (two per
// CU), so that the slots stay a small share of the logits' bytes
int loss_block(int T) {
  int C = 16;
  while ((T + C - 1) / C > 512 && C < 1024) C <<= 1;
  return C;
}

struct LossWs {
  size_t p, c, n, dots, ticket, bytes;
};

LossWs loss_ws(int T, int E, int S) {
  const int C = loss_block(T), EC = (E + kWave - 1) / kWave;
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

// the compiled row shape for E experts on L lanes: f(Row<NP, VEC>())
template <class F>
void with_row(int E, int L, F f) {
  if (E % 4 == 0) {
    const int np = (E / 4 + L - 1) / L;
    if (np <= 1) f(Row<1, true>());
    else if (np <= 2) f(Row<2, true>());
    else f(Row<4, true>());
  } else {
    const int np = (E + L - 1) / L;
    if (np <= 1) f(Row<1, false>());
    else if (np <= 2) f(Row<2, false>());
    else if (np <= 4) f(Row<4, false>());
    else if (np <= 8) f(Row<8, false>());
    else f(Row<16, false>());
  }
}

template <int NP, bool VEC>
void launch_partial(Row<NP, VEC>, int blocks, hipStream_t st, const float *logits,
                    const int32_t *idx, const int32_t *off, const uint8_t *mask, int T, int E,
                    int k, int S, int C, int L, float *p, int32_t *c, int32_t *n, int32_t *ticket) {
  hipLaunchKernelGGL((balance_partial_kernel<NP, VEC>), dim3(blocks), dim3(kThreadsP), 0, st, logits,
                     idx, off, mask, T, E, k, S, C, L, p, c, n, ticket);
}

template <bool RENORM, int NP, bool VEC>
void launch_backward(Row<NP, VEC>, int blocks, hipStream_t st, const float *logits,
                     const int32_t *idx, const float *dw, const int32_t *counts,
                     const int32_t *tokens, float alpha, const float *d_loss, const int32_t *off,
                     const uint8_t *mask, int T, int E, int k, int S, int C, int L, float *out) {
  hipLaunchKernelGGL((route_backward_kernel<NP, VEC, RENORM>), dim3(blocks), dim3(256), 0, st,
                     logits, idx, dw, counts, tokens, alpha, d_loss, off, mask, T, E, k, S, C, L,
                     out);
}

}  // namespace

size_t balance_loss_ws_bytes(int T, int E, int S) { return loss_ws(T, E, S).bytes; }

hipError_t launch_balance_loss(const float *logits, const int32_t *topk_idx, const int32_t *off,
                               const uint8_t *mask, int T, int E, int k, int S, float alpha,
                               int32_t *counts, float *probs, int32_t *tokens, float *loss, void *ws,
                               hipStream_t s) {
  const int C = loss_block(T), EC = (E + kWave - 1) / kWave, L = lanes_for(E);
  const LossWs w = loss_ws(T, E, S);
  char *base = static_cast<char *>(ws);
  float *p = reinterpret_cast<float *>(base + w.p);
  int32_t *c = reinterpret_cast<int32_t *>(base + w.c), *n = reinterpret_cast<int32_t *>(base + w.n);
  float *dots = reinterpret_cast<float *>(base + w.dots);
  int32_t *ticket = reinterpret_cast<int32_t *>(base + w.ticket);
  with_row(E, L, [&](auto row) {
    // (one block for an empty batch: it clears the ticket)
    launch_partial(row, max(1, (T + C - 1) / C), s, logits, topk_idx, off, mask, T, E, k, S, C, L, p, c, n,
                   ticket);
  });
  hipLaunchKernelGGL(balance_final_kernel, dim3(S * EC), dim3(kGroupsF * kWave), 0, s, p, c, n, off,
                     T, E, k, S, C, EC, alpha, counts, probs, tokens, loss, dots, ticket);
  return hipGetLastError();
}

hipError_t launch_route_backward(const float *logits, const int32_t *topk_idx, const float *dw,
                                 bool renorm, const int32_t *counts, const int32_t *tokens,
                                 float alpha, const float *d_loss, const int32_t *off,
                                 const uint8_t *mask, int T, int E, int k, int S, float *d_logits,
                                 hipStream_t s) {
  const int L = lanes_for(E);
  // tokens per workgroup: two passes of its token slots, at least 16
  const int C = max(16, 2 * (256 / kWave) * (kWave / L));
  with_row(E, L, [&](auto row) {
    if (renorm)
      launch_backward<true>(row, (T + C - 1) / C, s, logits, topk_idx, dw, counts, tokens, alpha,
                            d_loss, off, mask, T, E, k, S, C, L, d_logits);
    else
      launch_backward<false>(row, (T + C - 1) / C, s, logits, topk_idx, dw, counts, tokens, alpha,
                             d_loss, off, mask, T, E, k, S, C, L, d_logits);
  });
  return hipGetLastError();
}
