// Global norm of many tensors, and the tensors clipped by it:
//   norm = sqrt(sum over all elements of g^2),  out = g * min(1, max_norm / (norm + 1e-6)).
//
// Two launches for up to kMost tensors. The elements are cut into blocks of 8192 of one tensor.
// k_norm_partial: a CTA sums the squares of an equal run of blocks and stores one double;
// k_norm_finish: every CTA adds all those partial sums in the same order, so the norm is the
// same on every run and needs no counter or zeroed state, and then scales its blocks. It takes
// them in the opposite order: what the first pass read last is still in L2.
// Bound by memory: 1 read for the norm, 1 read and 1 write for the scaling, less what L2 keeps.
// 291 bf16 tensors, 456 MB: 88.7 + 147.9 us (5.1 and 6.2 TB/s); 64 fp32 tensors, 8.4 MB: 5.6 + 7.3.
// A thread requests its 4 pieces of 16 bytes (8 in fp32) of a block before it uses the first.
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
constexpr int kFew = 64, kMost = 1024;         // tensors per launch (kernel parameters: 32764 bytes at most)
constexpr int kMaxGrid = 2368;                 // CTAs, and partial sums, per launch (four waves of 4 per SM)
constexpr int kPer = 4;                        // units of 8 elements per thread and block
constexpr int kUnits = kPer * kThreads;        // units per block

// One launch's tensors: tensor i has the blocks [first[i], first[i + 1]), and its last block
// ends `tail` elements before its end.
template <int CAP>
struct Tensors {
  const void* in[CAP];
  void* out[CAP];
  int64_t first[CAP + 1];
  uint16_t tail[CAP];
  uint8_t bf16[CAP];
  int count;
};

template <int CAP>
__device__ __forceinline__ int tensor_of(const Tensors<CAP>& t, int64_t block) {
  int lo = 0, hi = t.count;                    // first[lo] <= block < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= block) lo = mid; else hi = mid;
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
      __stcs(reinterpret_cast<uint4*>(at), make_uint4(u[0], u[1], u[2], u[3]));
    } else {
      __stcs(reinterpret_cast<float4*>(at), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(at) + 1, make_float4(v[4], v[5], v[6], v[7]));
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

// Calls use(unit's first element, its 8 values) for this thread's units of one block, loads
// first. LAST: streaming loads, for data that no one reads again.
template <bool LAST, typename Use>
__device__ __forceinline__ void each_unit(const void* p, bool bf16, int64_t e0, int64_t n, Use use) {
  const char* base = static_cast<const char*>(p) + e0 * (bf16 ? 2 : 4);
  if ((reinterpret_cast<uintptr_t>(base) & 15) != 0) {
    for (int i = 0; i < kPer; ++i) {
      const int64_t e = e0 + 8 * (threadIdx.x + kThreads * i);
      if (e >= n) return;
      float v[8];
      load_unit(p, bf16, e, n, v);
      use(e, v);
    }
    return;
  }
  // whole units; the one that the tensor ends in, if any, is its thread's at the end
  const int whole = (int)min((n - e0) / 8, (int64_t)kUnits);
  const float4* src = reinterpret_cast<const float4*>(base);
  auto get = [&](int unit, int piece, int per_unit) {
    const float4* a = src + per_unit * unit + piece;
    return unit < whole ? (LAST ? __ldcs(a) : *a) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  if (bf16) {
    float4 w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = get(threadIdx.x + kThreads * i, 0, 1);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t u[4] = {__float_as_uint(w[i].x), __float_as_uint(w[i].y), __float_as_uint(w[i].z),
                             __float_as_uint(w[i].w)};
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
      if ((int)threadIdx.x + kThreads * i < whole) use(e0 + 8 * (threadIdx.x + kThreads * i), v);
    }
  } else {
    float4 w[2 * kPer];
#pragma unroll
    for (int i = 0; i < 2 * kPer; ++i) w[i] = get(threadIdx.x + kThreads * (i / 2), i & 1, 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float4 a = w[2 * i], b = w[2 * i + 1];
      float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const int unit = threadIdx.x + kThreads * i;
      if (unit < whole) use(e0 + 8 * unit, v);
    }
  }
  const int64_t e = e0 + 8 * (int64_t)whole;
  if (whole < kUnits && e < n && (int)threadIdx.x == whole % kThreads) {
    float v[8];
    load_unit(p, bf16, e, n, v);
    use(e, v);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) k_norm_partial(const __grid_constant__ Tensors<CAP> t,
                                                           double* __restrict__ partial) {
  griddep_wait();
  const int64_t blocks = t.first[t.count];
  const int64_t b0 = blocks * blockIdx.x / gridDim.x, b1 = blocks * (blockIdx.x + 1) / gridDim.x;
  double sum = 0.0;
  int i = b0 < b1 ? tensor_of(t, b0) : 0;
  for (int64_t b = b0; b < b1; ++b) {
    while (b >= t.first[i + 1]) ++i;
    const int64_t n = 8 * kUnits * (t.first[i + 1] - t.first[i]) - t.tail[i];
    each_unit<false>(t.in[i], t.bf16[i], 8 * kUnits * (b - t.first[i]), n, [&](int64_t, const float (&v)[8]) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(v[k], v[k], s);
      if (s > 1e-30f && s < 1e38f) {
        sum += s;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += (double)v[k] * (double)v[k];
      }
    });
  }
  griddep_launch_dependents();
  const double s = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) k_norm_finish(const __grid_constant__ Tensors<CAP> t,
                                                          const double* __restrict__ partial, int npartial,
                                                          float max_norm, float* norm) {
  griddep_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < npartial; i += kThreads) s += partial[i];
  const float nrm = (float)sqrt(block_sum(s));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  // a NaN norm keeps the coefficient NaN, an infinite one makes it 0
  const float ratio = max_norm / (nrm + 1e-6f);
  const float coef = ratio > 1.0f ? 1.0f : ratio;
  const int64_t blocks = t.first[t.count];
  const int64_t b0 = blocks * blockIdx.x / gridDim.x, b1 = blocks * (blockIdx.x + 1) / gridDim.x;
  int i = b0 < b1 ? tensor_of(t, b1 - 1) : 0;
  for (int64_t b = b1 - 1; b >= b0; --b) {
    while (b < t.first[i]) --i;
    const int64_t n = 8 * kUnits * (t.first[i + 1] - t.first[i]) - t.tail[i];
    each_unit<true>(t.in[i], t.bf16[i], 8 * kUnits * (b - t.first[i]), n, [&](int64_t e, float (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= coef;
      store_unit(t.out[i], t.bf16[i], e, n, v);
    });
  }
  griddep_launch_dependents();
}

int grid_of(int64_t blocks) { return (int)(blocks < 1 ? 1 : (blocks < kMaxGrid ? blocks : kMaxGrid)); }

template <int CAP>
cudaError_t run(const void* const* grads, void* const* out, const int64_t* numels, const int* dtypes, int count,
                float max_norm, float* norm, double* ws, cudaStream_t s) {
  static_assert(sizeof(Tensors<CAP>) + 64 <= 32764, "kernel parameters");
  Tensors<CAP> t;
  auto gather = [&](int i0) {
    t.count = 0;
    t.first[0] = 0;
    for (int i = i0; i < count && i < i0 + CAP; ++i) {
      const int k = t.count++;
      const int64_t blocks = (numels[i] + 8 * kUnits - 1) / (8 * kUnits);
      t.in[k] = grads[i];
      t.out[k] = out ? out[i] : nullptr;
      t.bf16[k] = dtypes[i] == 1;
      t.tail[k] = (uint16_t)(8 * kUnits * blocks - numels[i]);
      t.first[k + 1] = t.first[k] + blocks;
    }
  };
  int npartial = 0;
  for (int i = 0; i < count; i += CAP) {
    gather(i);
    const int grid = grid_of(t.first[t.count]);
    const cudaError_t e = launch_pdl(k_norm_partial<CAP>, dim3(grid), dim3(kThreads), 0, s, t, ws + npartial);
    if (e != cudaSuccess) return e;
    npartial += grid;
  }
  if (out == nullptr || count == 0) {
    t.count = 0;                                   // no blocks: the norm alone
    t.first[0] = 0;
    return launch_pdl(k_norm_finish<CAP>, dim3(1), dim3(kThreads), 0, s, t, ws, npartial, max_norm, norm);
  }
  for (int i = 0; i < count; i += CAP) {
    if (count > CAP) gather(i);
    const cudaError_t e = launch_pdl(k_norm_finish<CAP>, dim3(grid_of(t.first[t.count])), dim3(kThreads), 0, s, t, ws,
                                     npartial, max_norm, i == 0 ? norm : static_cast<float*>(nullptr));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int64_t grad_norm_ws_doubles(int count) { return (int64_t)((count + kMost - 1) / kMost) * kMaxGrid; }

cudaError_t launch_grad_norm(const void* const* grads, void* const* out, const int64_t* numels, const int* dtypes,
                             int count, float max_norm, float* norm, double* ws, cudaStream_t s) {
  // few tensors: a tenth of the parameters to copy per launch
  if (count <= kFew) return run<kFew>(grads, out, numels, dtypes, count, max_norm, norm, ws, s);
  return run<kMost>(grads, out, numels, dtypes, count, max_norm, norm, ws, s);
}

}  // namespace rdfft
