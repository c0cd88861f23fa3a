// grad_norm.hip -- the global 2-norm of many gradients, and their scaling by
// min(1, max_norm / (norm + 1e-6)).
//
// The tensors' addresses, sizes and types travel in the kernel's arguments
// (kMany tensors a launch), so a call needs no table on the device and can be
// captured.  Every tensor is cut into chunks of kChunk elements, counted from
// the 16-byte boundary at or below its first element so that whole 16-byte
// pieces are aligned; a workgroup takes a run of consecutive chunks.
//
// Squares are summed in fp64: no finite fp32 or bf16 gradient overflows or
// underflows, and the sum of 2^30 of them keeps all bits of the fp32 result.
// Both passes are bound by HBM: 2.8 GB of bf16 in 453-465 us (6.1 TB/s); 201 MB
// of fp32 in 96 tensors 39 us for the norm (5.2 TB/s) and 66 for 403 MB of
// clipping (6.1, part of the reads from the last-level cache).  A call of many
// small tensors is bound by the host, which looks at each (0.3 us a tensor and
// list from Python).
#include "backward_internal.h"

namespace {

using namespace moe;

constexpr int kMany = 128;       // tensors a launch
constexpr int kChunk = 16384;    // elements a chunk
constexpr int kMaxGroups = 2048; // workgroups (and partial sums) a launch

struct Tensors {
  const void *p[kMany];
  void *out[kMany];
  int64_t n[kMany];
  int first[kMany + 1];  // first chunk of each tensor
  uint8_t bf16[kMany];
  int count;
  int in_place;  // every output is its gradient
};
static_assert(sizeof(Tensors) <= 4000, "kernel arguments hold 4 KB");

// elements between the 16-byte boundary below p and p
__host__ __device__ inline int misaligned(const void *p, int es) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / es);
}

// The tensor that chunk c lies in.
__device__ __forceinline__ int tensor_of(const Tensors &t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {  // the last tensor whose first chunk is not past c
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int ES>
__device__ __forceinline__ float element(const void *p, int64_t e) {
  if constexpr (ES == 2) return bf16_bits_to_f32(static_cast<const uint16_t *>(p)[e]);
  else return static_cast<const float *>(p)[e];
}

template <int ES>
__device__ __forceinline__ double chunk_squares(const void *p, int64_t n, int64_t c) {
  constexpr int PE = 16 / ES;  // elements a piece
  const int mis = misaligned(p, ES);
  const int64_t end = n + mis, v0 = c * kChunk, v1 = min(end, v0 + kChunk);
  const char *base = static_cast<const char *>(p) - (size_t)mis * ES;
  double sum[2] = {0., 0.};
  auto piece = [&](u32x4 raw) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ES == 2) {
        const double lo = bf16_bits_to_f32(raw[i] & 0xffffu), hi = __uint_as_float(raw[i] & 0xffff0000u);
        sum[0] = fma(lo, lo, sum[0]);
        sum[1] = fma(hi, hi, sum[1]);
      } else {
        const double v = __uint_as_float(raw[i]);
        sum[i & 1] = fma(v, v, sum[i & 1]);
      }
    }
  };
  const int64_t full0 = (v0 == 0 && mis) ? PE : v0;   // whole pieces
  const int64_t full1 = v1 - v1 % PE;
  constexpr int UN = 8;
  const int64_t step = (int64_t)blockDim.x * PE;
  int64_t v = full0 + (int64_t)threadIdx.x * PE;
  for (; v + (UN - 1) * step < full1; v += UN * step) {
    u32x4 raw[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u)
      raw[u] = *reinterpret_cast<const u32x4 *>(base + (size_t)(v + u * step) * ES);
#pragma unroll
    for (int u = 0; u < UN; ++u) piece(raw[u]);
  }
  for (; v < full1; v += step) piece(*reinterpret_cast<const u32x4 *>(base + (size_t)v * ES));
  // what is left at both ends of the tensor
  if (full0 > v0) {
    const int64_t e = (int64_t)threadIdx.x;
    if (e < min((int64_t)(PE - mis), n)) {
      const double x = element<ES>(p, e);
      sum[0] = fma(x, x, sum[0]);
    }
  }
  if (full1 >= full0) {
    const int64_t e = full1 + (int64_t)threadIdx.x;
    if (e < v1) {
      const double x = element<ES>(p, e - mis);
      sum[0] = fma(x, x, sum[0]);
    }
  }
  return sum[0] + sum[1];
}

// the workgroup's sum, in the order of the threads' tree; valid in thread 0
__device__ __forceinline__ double block_sum(double v, double *s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if (lane_id() == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  double r = 0.;
  for (int w = 0; w < (int)blockDim.x / kWave; ++w) r += s[w];
  __syncthreads();
  return r;
}

__device__ __forceinline__ double run_squares(const Tensors &t, int c0, int c1) {
  double sum = 0.;
  if (c0 >= c1) return sum;
  int i = tensor_of(t, c0);
  for (int c = c0; c < c1; ++c) {
    while (c >= t.first[i + 1]) ++i;
    sum += t.bf16[i] ? chunk_squares<2>(t.p[i], t.n[i], c - t.first[i])
                     : chunk_squares<4>(t.p[i], t.n[i], c - t.first[i]);
  }
  return sum;
}

__global__ __launch_bounds__(256) void norm_partial_kernel(const Tensors t, double *partial) {
  __shared__ double s[256 / kWave];
  const long long chunks = t.first[t.count];
  const int c0 = (int)(chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)(chunks * (blockIdx.x + 1) / gridDim.x);
  const double r = block_sum(run_squares(t, c0, c1), s);
  if (threadIdx.x == 0) partial[blockIdx.x] = r;
}

// few elements: the whole norm in one launch
__global__ __launch_bounds__(1024) void norm_small_kernel(const Tensors t, float *norm) {
  __shared__ double s[1024 / kWave];
  const double r = block_sum(run_squares(t, 0, t.first[t.count]), s);
  if (threadIdx.x == 0) *norm = (float)sqrt(r);
}

__global__ __launch_bounds__(1024) void norm_final_kernel(const double *partial, int n, float *norm) {
  __shared__ double s[1024 / kWave];
  double v = 0.;
  for (int i = threadIdx.x; i < n; i += 1024) v += partial[i];
  v = block_sum(v, s);
  if (threadIdx.x == 0) *norm = (float)sqrt(v);
}

template <int ES>
__device__ __forceinline__ void put(void *p, int64_t e, float v) {
  if constexpr (ES == 2) static_cast<uint16_t *>(p)[e] = f32_to_bf16_bits(v);
  else static_cast<float *>(p)[e] = v;
}

template <int ES, bool STREAM>
__device__ __forceinline__ void chunk_scale(const void *p, void *out, int64_t n, int64_t c, float f) {
  constexpr int PE = 16 / ES;
  const int mis = misaligned(p, ES);
  const int64_t end = n + mis, v0 = c * kChunk, v1 = min(end, v0 + kChunk);
  if (misaligned(out, ES) != mis) {  // no common 16-byte boundaries
    for (int64_t v = max(v0, (int64_t)mis) + threadIdx.x; v < v1; v += blockDim.x)
      put<ES>(out, v - mis, element<ES>(p, v - mis) * f);
    return;
  }
  const char *base = static_cast<const char *>(p) - (size_t)mis * ES;
  char *obase = static_cast<char *>(out) - (size_t)mis * ES;
  auto piece = [&](u32x4 raw) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ES == 2)
        o[i] = f32_to_bf16_bits(bf16_bits_to_f32(raw[i] & 0xffffu) * f) |
               ((uint32_t)f32_to_bf16_bits(__uint_as_float(raw[i] & 0xffff0000u) * f) << 16);
      else
        o[i] = __float_as_uint(__uint_as_float(raw[i]) * f);
    }
    return o;
  };
  const int64_t full0 = (v0 == 0 && mis) ? PE : v0;
  const int64_t full1 = v1 - v1 % PE;
  constexpr int UN = 4;
  const int64_t step = (int64_t)blockDim.x * PE;
  int64_t v = full0 + (int64_t)threadIdx.x * PE;
  for (; v + (UN - 1) * step < full1; v += UN * step) {
    u32x4 raw[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u)
      raw[u] = *reinterpret_cast<const u32x4 *>(base + (size_t)(v + u * step) * ES);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      u32x4 *const to = reinterpret_cast<u32x4 *>(obase + (size_t)(v + u * step) * ES);
      if constexpr (STREAM) __builtin_nontemporal_store(piece(raw[u]), to);
      else *to = piece(raw[u]);
    }
  }
  for (; v < full1; v += step)
    *reinterpret_cast<u32x4 *>(obase + (size_t)v * ES) =
        piece(*reinterpret_cast<const u32x4 *>(base + (size_t)v * ES));
  if (full0 > v0) {
    const int64_t e = (int64_t)threadIdx.x;
    if (e < min((int64_t)(PE - mis), n)) put<ES>(out, e, element<ES>(p, e) * f);
  }
  if (full1 >= full0) {
    const int64_t e = full1 + (int64_t)threadIdx.x;
    if (e < v1) put<ES>(out, e - mis, element<ES>(p, e - mis) * f);
  }
}

// STREAM: outputs past the caches
template <bool STREAM>
__global__ __launch_bounds__(256) void clip_kernel(const Tensors t, const float *norm, float max_norm) {
  const float q = max_norm / (*norm + 1e-6f);
  const float f = q >= 1.f ? 1.f : q;  // (a NaN stays)
  if (f == 1.f && t.in_place) return;
  const long long chunks = t.first[t.count];
  // from the end: the norm has read the last chunks last, so they are still in
  // the last-level cache (96 fp32 gradients, 201 MB: 132 -> 128 us a norm and
  // clip, with the outputs past the cache 111).  That is inside a launch: those
  // of a list of more than kMany tensors run in the list's order.
  const int b = gridDim.x - 1 - blockIdx.x;
  const int c0 = (int)(chunks * b / gridDim.x);
  const int c1 = (int)(chunks * (b + 1) / gridDim.x);
  if (c0 >= c1) return;
  int i = tensor_of(t, c1 - 1);
  for (int c = c1 - 1; c >= c0; --c) {
    while (c < t.first[i]) --i;
    if (f == 1.f && t.out[i] == t.p[i]) continue;  // nothing changes
    if (t.bf16[i]) chunk_scale<2, STREAM>(t.p[i], t.out[i], t.n[i], c - t.first[i], f);
    else chunk_scale<4, STREAM>(t.p[i], t.out[i], t.n[i], c - t.first[i], f);
  }
}

// Calls f(tensors, chunks, index of the launch) for every kMany tensors of
// the list that have an element.
template <class F>
hipError_t for_each_launch(const void *const *grads, const int64_t *sizes, const int *dts, int n,
                           void *const *out, F f) {
  Tensors t;
  int index = 0;
  long long chunks = 0;
  t.count = 0;
  t.in_place = 1;
  for (int i = 0; i <= n; ++i) {
    const bool full = t.count == kMany;
    const int es = i < n && dts[i] == MOE_BF16 ? 2 : 4;
    const long long add = i < n && sizes[i] > 0
                              ? (sizes[i] + misaligned(grads[i], es) + kChunk - 1) / kChunk : 0;
    if (t.count && (i == n || full || chunks + add > INT32_MAX)) {
      t.first[t.count] = (int)chunks;
      const hipError_t e = f(t, (int)chunks, index++);
      if (e != hipSuccess) return e;
      t.count = 0;
      t.in_place = 1;
      chunks = 0;
    }
    if (!add) continue;
    t.p[t.count] = grads[i];
    t.out[t.count] = out ? out[i] : const_cast<void *>(grads[i]);
    t.in_place &= t.out[t.count] == t.p[t.count];
    t.n[t.count] = sizes[i];
    t.bf16[t.count] = es == 2;
    t.first[t.count++] = (int)chunks;
    chunks += add;
  }
  return hipSuccess;
}

}  // namespace

// (a launch of kMany tensors, or one cut short by its chunk count: a tensor
// has at most 2^26 chunks, so 31 of them fit and no cut leaves fewer)
size_t grad_norm_ws_bytes(int n) {
  return (size_t)((n + 30) / 31) * kMaxGroups * sizeof(double);
}

hipError_t launch_grad_norm(const void *const *grads, const int64_t *sizes, const int *dts, int n,
                            float *norm, void *ws, hipStream_t s) {
  double *partial = static_cast<double *>(ws);
  int used = 0;
  bool done = false;
  hipError_t e = for_each_launch(
      grads, sizes, dts, n, nullptr, [&](Tensors &t, int chunks, int) {
        // a workgroup adds up to 4 chunks faster than a second launch starts
        if (used == 0 && t.count == n && chunks <= 4) {
          hipLaunchKernelGGL(norm_small_kernel, dim3(1), dim3(1024), 0, s, t, norm);
          done = true;
          return hipGetLastError();
        }
        const int grid = chunks < kMaxGroups ? chunks : kMaxGroups;
        hipLaunchKernelGGL(norm_partial_kernel, dim3(grid), dim3(256), 0, s, t, partial + used);
        used += grid;
        return hipGetLastError();
      });
  if (e != hipSuccess || done) return e;
  hipLaunchKernelGGL(norm_final_kernel, dim3(1), dim3(1024), 0, s, partial, used, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const void *const *grads, const int64_t *sizes, const int *dts, int n,
                            const float *norm, float max_norm, void *const *out, hipStream_t s) {
  // Gradients and outputs that the 256 MB last-level cache cannot both hold: the
  // outputs leave it to the gradients (norm and clip of 96 fp32 tensors into
  // others, stores through it and past it: 130 MB 127 and 127 us, 160 MB 168 and
  // 152, 200 MB 183 and 173, 300 MB 254 and 248, 400 MB and more the same).  In
  // place both take the same at every size, 32 MB to 1 GB: the lines are there.
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += sizes[i] * (dts[i] == MOE_BF16 ? 2 : 4);
  const bool stream = bytes > (128ll << 20);
  return for_each_launch(grads, sizes, dts, n, out, [&](Tensors &t, int chunks, int) {
    const int grid = chunks < kMaxGroups ? chunks : kMaxGroups;
    if (stream)
      hipLaunchKernelGGL(clip_kernel<true>, dim3(grid), dim3(256), 0, s, t, norm, max_norm);
    else
      hipLaunchKernelGGL(clip_kernel<false>, dim3(grid), dim3(256), 0, s, t, norm, max_norm);
    return hipGetLastError();
  });
}
