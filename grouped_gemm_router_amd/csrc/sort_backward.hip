// sort_backward.hip -- the gradients of the gather with gate weights
// (moe_combine) and of the scatter into expert order (moe_permute).
//
// "DeepGEMM walkthrough" §2.1: y = E_shared(x) + sum_i p_i E_i(x).  So the
// gradient of expert row E_i(x_t) is p_i dy_t, that of p_i the product of
// dy_t with the row, and x_t, copied to its k experts, collects its copies'
// gradients.
//
// Both are bound by HBM (4096 tokens of 7168 columns, 8 experts and a shared one:
// 1.53 GB in 313 us, 4.9 TB/s; 4096 of 4096, 2 experts, the sum of fp32 rows:
// 201 MB in 41 us): every row is read and written once.  One workgroup
// per token; a thread owns 8 consecutive columns at a time and issues the row
// loads of four entries together.
#include "backward_internal.h"

namespace {

using namespace moe;

constexpr int kMaxTerms = MOE_MAX_TOPK + 8;
constexpr int kMaxThreads = 1024;
constexpr int kDots = 8;  // entries whose products a thread keeps at a time

template <int ES>
__device__ __forceinline__ void load8(const void *base, size_t elem, float v[8]) {
  if constexpr (ES == 2) {
    const u32x4 raw = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32(raw[i] & 0xffffu);
      v[2 * i + 1] = bf16_bits_to_f32(raw[i] >> 16);
    }
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <int ES>
__device__ __forceinline__ void store8(void *base, size_t elem, const float v[8]) {
  if constexpr (ES == 2) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + elem) = o;
  } else {
    f32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = v[i];
      b[i] = v[4 + i];
    }
    *reinterpret_cast<f32x4 *>(static_cast<float *>(base) + elem) = a;
    *reinterpret_cast<f32x4 *>(static_cast<float *>(base) + elem + 4) = b;
  }
}

// rows of a token's entries, -1 for what is dropped or out of range
__device__ __forceinline__ void token_rows(const int32_t *flat_to_row, int t, int T, int k,
                                           int n_shared, int *s_row) {
  const long long nrows = (long long)T * (k + n_shared);
  for (int j = threadIdx.x; j < k + n_shared; j += blockDim.x) {
    const int row = j < k ? flat_to_row[(size_t)t * k + j]
                          : flat_to_row[(size_t)T * k + (size_t)(j - k) * T + t];
    s_row[j] = row >= 0 && row < nrows ? row : -1;
  }
}

// GS: element size of d_out and dY, YS of Y
template <int GS, int YS>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
    const void *__restrict__ d_out, const void *__restrict__ Y,
    const int32_t *__restrict__ flat_to_row, const float *topk_w, int T, int k, int d, int n_shared,
    void *__restrict__ dY, float *d_topk_w) {  // (the last may be topk_w: a token's are read first)
  __shared__ int s_row[kMaxTerms];
  __shared__ float s_w[kMaxTerms];
  __shared__ float s_dot[kMaxThreads / kWave][kDots];
  const int t = blockIdx.x;
  token_rows(flat_to_row, t, T, k, n_shared, s_row);
  for (int j = threadIdx.x; j < k; j += blockDim.x) s_w[j] = topk_w[(size_t)t * k + j];
  __syncthreads();
  const int npiece = d / 8, wave = threadIdx.x / kWave;
  for (int j0 = 0; j0 < k; j0 += kDots) {
    const int n = min(kDots, k - j0);
    float dot[kDots];
#pragma unroll
    for (int q = 0; q < kDots; ++q) dot[q] = 0.f;
    for (int p = threadIdx.x; p < npiece; p += blockDim.x) {
      float g[8];
      load8<GS>(d_out, (size_t)t * d + (size_t)p * 8, g);
#pragma unroll
      for (int q0 = 0; q0 < kDots; q0 += 4) {
        float y[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = q0 + q < n ? s_row[j0 + q0 + q] : -1;
          if (d_topk_w && row >= 0) load8<YS>(Y, (size_t)row * d + (size_t)p * 8, y[q]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = q0 + q < n ? s_row[j0 + q0 + q] : -1;
          if (row < 0) continue;
          if (d_topk_w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[q0 + q] = fmaf(g[i], y[q][i], dot[q0 + q]);
          }
          if (dY) {
            const float w = s_w[j0 + q0 + q];
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = w * g[i];
            store8<GS>(dY, (size_t)row * d + (size_t)p * 8, o);
          }
        }
      }
      if (j0 == 0 && dY)
        for (int s = 0; s < n_shared; ++s) {
          const int row = s_row[k + s];
          if (row >= 0) store8<GS>(dY, (size_t)row * d + (size_t)p * 8, g);
        }
    }
    if (d_topk_w) {
      if (j0) __syncthreads();  // the last entries' sums are read
#pragma unroll
      for (int q = 0; q < kDots; ++q) {
        dot[q] = wave_sum(dot[q]);
        if (lane_id() == 0) s_dot[wave][q] = dot[q];
      }
      __syncthreads();
      if ((int)threadIdx.x < n) {
        float v = 0.f;
        for (int w = 0; w < (int)blockDim.x / kWave; ++w) v += s_dot[w][threadIdx.x];
        d_topk_w[(size_t)t * k + j0 + threadIdx.x] = s_row[j0 + threadIdx.x] >= 0 ? v : 0.f;
      }
    }
  }
}

// PS: element size of dx_perm, XS of dx and addend
template <int PS, int XS>
__global__ __launch_bounds__(kMaxThreads) void permute_backward_kernel(
    const void *__restrict__ dx_perm, const int32_t *__restrict__ flat_to_row, int T, int k, int d,
    int n_shared, const void *addend, void *dx) {
  __shared__ int s_row[kMaxTerms];
  const int t = blockIdx.x, nterm = k + n_shared;
  token_rows(flat_to_row, t, T, k, n_shared, s_row);
  __syncthreads();
  for (int p = threadIdx.x; p < d / 8; p += blockDim.x) {
    const size_t at = (size_t)t * d + (size_t)p * 8;
    float acc[8], add[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (addend) load8<XS>(addend, at, add);
    for (int j0 = 0; j0 < nterm; j0 += 4) {
      float v[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = j0 + q < nterm ? s_row[j0 + q] : -1;
        if (row >= 0) {
          load8<PS>(dx_perm, (size_t)row * d + (size_t)p * 8, v[q]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[q][i] = 0.f;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[q][i];
    }
    if (addend) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += add[i];
    }
    store8<XS>(dx, at, acc);
  }
}

// 256 threads a token where there are tokens enough; with fewer, as many as it
// has 8-column pieces, so that the loads in flight do not fall with the tokens
// (203 tokens of 10 x 6960 fp32 rows: 29 -> 21 us)
unsigned threads_of(int T, int d) {
  const unsigned all = ((unsigned)d / 8 + kWave - 1) / kWave * kWave;
  const unsigned most = T < 1024 ? kMaxThreads : 256;
  return all < most ? all : most;
}

}  // namespace

hipError_t launch_combine_backward(const void *d_out, int dt, const void *Y, int y_dt,
                                   const int32_t *flat_to_row, const float *topk_w, int T, int k,
                                   int d, int n_shared, void *dY, float *d_topk_w, hipStream_t s) {
  const dim3 grid(T), block(threads_of(T, d));
#define MOE_LAUNCH(GS, YS)                                                                      \
  hipLaunchKernelGGL((combine_backward_kernel<GS, YS>), grid, block, 0, s, d_out, Y, flat_to_row, \
                     topk_w, T, k, d, n_shared, dY, d_topk_w)
  if (dt == MOE_BF16) {
    if (y_dt == MOE_BF16) MOE_LAUNCH(2, 2); else MOE_LAUNCH(2, 4);
  } else {
    if (y_dt == MOE_BF16) MOE_LAUNCH(4, 2); else MOE_LAUNCH(4, 4);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_permute_backward(const void *dx_perm, int p_dt, const int32_t *flat_to_row, int T,
                                   int k, int d, int n_shared, const void *addend, void *dx, int dt,
                                   hipStream_t s) {
  const dim3 grid(T), block(threads_of(T, d));
#define MOE_LAUNCH(PS, XS)                                                                       \
  hipLaunchKernelGGL((permute_backward_kernel<PS, XS>), grid, block, 0, s, dx_perm, flat_to_row, T, \
                     k, d, n_shared, addend, dx)
  if (p_dt == MOE_BF16) {
    if (dt == MOE_BF16) MOE_LAUNCH(2, 2); else MOE_LAUNCH(2, 4);
  } else {
    if (dt == MOE_BF16) MOE_LAUNCH(4, 2); else MOE_LAUNCH(4, 4);
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}
