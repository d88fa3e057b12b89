// Global norm of many tensors, and the tensors clipped by it:
//   norm = sqrt(sum over all elements of g^2),  out = g * min(1, max_norm / (norm + 1e-6)).
//
// Two launches for up to kMaxTensors tensors. k_norm_partial: every CTA sums the squares of a
// fixed share of the elements (the tensors' 16-byte pieces, numbered through) and stores one
// double; k_norm_finish: every CTA adds all those partial sums in the same order, so the norm
// is the same on every run and needs no counter or zeroed state, and then scales its share.
// Bound by memory: 1 read for the norm, 1 read and 1 write for the scaling, of which the
// second read comes from L2 as far as the tensors fit it.
//
// Squares of 8 elements are added in fp32 and those sums in double, so neither long sums nor
// many tensors lose bits; a sum of 8 that overflows fp32 or falls to its smallest range is
// formed again in double.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "packed_fft.cuh"
#include "pdl.cuh"

namespace rdfft {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTensors = 512;               // per launch: 20 bytes each of kernel parameters
constexpr int kMaxGrid = 592;                  // partial sums per launch

// One launch's tensors. Work is numbered in units of 8 elements; units of tensor i are
// [first[i], first[i + 1]).
struct Tensors {
  const void* in[kMaxTensors];
  void* out[kMaxTensors];
  int64_t numel[kMaxTensors];
  int64_t first[kMaxTensors + 1];
  uint8_t bf16[kMaxTensors];
  int count;
};

__device__ __forceinline__ int tensor_of(const Tensors& t, int64_t unit) {
  int lo = 0, hi = t.count;                    // first[lo] <= unit < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= unit) lo = mid; else hi = mid;
  }
  return lo;
}

// The 8 elements of a unit as fp32, zeros beyond the tensor's end.
__device__ __forceinline__ void load_unit(const void* p, bool bf16, int64_t e, int64_t n, float (&v)[8]) {
  const char* at = static_cast<const char*>(p) + e * (bf16 ? 2 : 4);
  if (e + 8 <= n && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
    if (bf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(at);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = e + i < n ? (bf16 ? to_f32(reinterpret_cast<const bf16_t*>(at)[i]) : reinterpret_cast<const float*>(at)[i])
                     : 0.0f;
}

__device__ __forceinline__ void store_unit(void* p, bool bf16, int64_t e, int64_t n, const float (&v)[8]) {
  char* at = static_cast<char*>(p) + e * (bf16 ? 2 : 4);
  if (e + 8 <= n && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
    if (bf16) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = (uint32_t)from_f32<bf16_t>(v[2 * i]) | (uint32_t)from_f32<bf16_t>(v[2 * i + 1]) << 16;
      *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < n) {
      if (bf16) reinterpret_cast<bf16_t*>(at)[i] = from_f32<bf16_t>(v[i]);
      else reinterpret_cast<float*>(at)[i] = v[i];
    }
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += warp_sum[i];
  return s;
}

__global__ void __launch_bounds__(kThreads) k_norm_partial(const __grid_constant__ Tensors t,
                                                           double* __restrict__ partial) {
  griddep_wait();
  const int64_t units = t.first[t.count], step = (int64_t)gridDim.x * kThreads;
  double sum = 0.0;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const int i = tensor_of(t, u);
    float v[8];
    load_unit(t.in[i], t.bf16[i], 8 * (u - t.first[i]), t.numel[i], v);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(v[k], v[k], s);
    if (s > 1e-30f && s < 1e38f) {
      sum += s;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += (double)v[k] * (double)v[k];
    }
  }
  griddep_launch_dependents();
  const double s = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) k_norm_finish(const __grid_constant__ Tensors t,
                                                          const double* __restrict__ partial, int npartial,
                                                          float max_norm, float* norm) {
  griddep_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < npartial; i += kThreads) s += partial[i];
  const float nrm = (float)sqrt(block_sum(s));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  if (t.count == 0) return;
  // a NaN norm keeps the coefficient NaN, an infinite one makes it 0
  const float ratio = max_norm / (nrm + 1e-6f);
  const float coef = ratio > 1.0f ? 1.0f : ratio;
  const int64_t units = t.first[t.count], step = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const int i = tensor_of(t, u);
    const int64_t e = 8 * (u - t.first[i]);
    float v[8];
    load_unit(t.in[i], t.bf16[i], e, t.numel[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= coef;
    store_unit(t.out[i], t.bf16[i], e, t.numel[i], v);
  }
  griddep_launch_dependents();
}

int grid_of(int64_t units) {
  const int64_t b = (units + kThreads - 1) / kThreads;
  return (int)(b < 1 ? 1 : (b < kMaxGrid ? b : kMaxGrid));
}

}  // namespace

int64_t grad_norm_ws_doubles(int count) {
  return (int64_t)((count + kMaxTensors - 1) / kMaxTensors) * kMaxGrid;
}

cudaError_t launch_grad_norm(const void* const* grads, void* const* out, const int64_t* numels, const int* dtypes,
                             int count, float max_norm, float* norm, double* ws, cudaStream_t s) {
  // the largest number of parameters a kernel takes is 32764 bytes
  static_assert(sizeof(Tensors) <= 32000, "kernel parameters");
  Tensors t;
  auto gather = [&](int i0) {
    t.count = 0;
    t.first[0] = 0;
    for (int i = i0; i < count && i < i0 + kMaxTensors; ++i) {
      const int k = t.count++;
      t.in[k] = grads[i];
      t.out[k] = out ? out[i] : nullptr;
      t.numel[k] = numels[i];
      t.bf16[k] = dtypes[i] == 1;
      t.first[k + 1] = t.first[k] + (numels[i] + 7) / 8;
    }
  };
  int npartial = 0;
  for (int i = 0; i < count; i += kMaxTensors) {
    gather(i);
    const int grid = grid_of(t.first[t.count]);
    const cudaError_t e = launch_pdl(k_norm_partial, dim3(grid), dim3(kThreads), 0, s, t, ws + npartial);
    if (e != cudaSuccess) return e;
    npartial += grid;
  }
  if (out == nullptr || count == 0) {
    t.count = 0;
    t.first[0] = 0;
    return launch_pdl(k_norm_finish, dim3(1), dim3(kThreads), 0, s, t, ws, npartial, max_norm, norm);
  }
  for (int i = 0; i < count; i += kMaxTensors) {
    if (count > kMaxTensors) gather(i);
    const cudaError_t e = launch_pdl(k_norm_finish, dim3(grid_of(t.first[t.count])), dim3(kThreads), 0, s, t, ws,
                                     npartial, max_norm, i == 0 ? norm : static_cast<float*>(nullptr));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rdfft
