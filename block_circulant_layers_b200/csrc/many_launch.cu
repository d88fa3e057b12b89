// Many-adapter operators: dispatch on the block size or the dtype.
#include <cuda_runtime.h>

#include "internal.h"
#include "lora.cuh"

namespace rdfft {

#define RDFFT_MANY_P(X) X(64) X(128) X(256) X(512) X(1024) X(2048) X(4096)
#define RDFFT_MANY_DECL(PP) \
  cudaError_t circ_many_##PP(int op, const CircMany& a, int dtype, cudaStream_t s, GcSink* sink);
RDFFT_MANY_P(RDFFT_MANY_DECL)

cudaError_t launch_circ_many(int op, const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink) {
  switch (p) {
#define RDFFT_MANY_CASE(PP) \
  case PP: return circ_many_##PP(op, a, dtype, s, sink);
    RDFFT_MANY_P(RDFFT_MANY_CASE)
    default: return cudaErrorInvalidValue;
  }
}

// grad_c[a] = the slots of adapter a added in slice order: with S <= T' slices of T' planned tokens,
// slice s holds positions [T' s / S, T' (s + 1) / S), and its sums over adapter a lie in slot
// s + a, or already in grad_c if the slice holds all of a. Zeros for an adapter without tokens. kSplit threads share an element, each adding
// every kSplit-th slot, and their sums are added in order: the order depends on the plan alone.
constexpr int kSumThreads = 256, kSplit = 8;

__global__ void __launch_bounds__(kSumThreads) k_sum_slots(const float4* __restrict__ slots, int64_t n4, int slices,
                                                           float4* __restrict__ out, PlanView plan) {
  constexpr int EPB = kSumThreads / kSplit;
  __shared__ float4 sums[kSplit][EPB];
  griddep_wait();
  if (!plan_matches(plan)) return;
  const int ad = blockIdx.y, el = threadIdx.x % EPB, r = threadIdx.x / EPB;
  const int64_t e = (int64_t)blockIdx.x * EPB + el;
  const int64_t tokens = __ldg(plan.offsets() + plan.n);
  slices = (int)min((int64_t)slices, tokens);
  const int beg = __ldg(plan.offsets() + ad), end = __ldg(plan.offsets() + ad + 1);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // the slice of a position: the last s with tokens s / slices <= position
  const int first = beg < end ? (int)(((int64_t)(beg + 1) * slices - 1) / tokens) : 0;
  const int last = beg < end ? (int)(((int64_t)end * slices - 1) / tokens) : 0;
  if (beg < end && first == last) return;
  if (e < n4 && beg < end) {
#pragma unroll 4
    for (int s = first + r; s <= last; s += kSplit) {
      const float4 v = __ldcs(slots + (int64_t)(s + ad) * n4 + e);
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
  }
  sums[r][el] = acc;
  __syncthreads();
  griddep_launch_dependents();
  if (r == 0 && e < n4) {
    float4 t = sums[0][el];
#pragma unroll
    for (int j = 1; j < kSplit; ++j) {
      const float4 v = sums[j][el];
      t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    }
    out[(int64_t)ad * n4 + e] = t;
  }
}

cudaError_t launch_circ_many_bwd(const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink) {
  const int q = a.D / p;
  const bool both = a.out != nullptr && a.grad_c != nullptr;
  cudaError_t e = cudaSuccess;
  if (a.grad_c != nullptr) {
    e = both && circ_bwd_fused_supported(p, a.D, a.T) ? launch_circ_many_fused(a, p, dtype, s, sink)
                                                      : launch_circ_many(2, a, p, dtype, s, sink);
    if (e != cudaSuccess || sink->plan_only) return e;
    const int64_t floats = (int64_t)q * q * p, n4 = floats / 4;
    if ((int64_t)(sink->slices + a.n) * floats > sink->partial_floats) return cudaErrorInvalidValue;
    constexpr int EPB = kSumThreads / kSplit;
    e = launch_pdl(k_sum_slots, dim3((unsigned)((n4 + EPB - 1) / EPB), (unsigned)a.n), dim3(kSumThreads), 0, s,
                   reinterpret_cast<const float4*>(sink->partial), n4, sink->slices,
                   reinterpret_cast<float4*>(a.grad_c), plan_view(a.plan, a.T, a.n, 0));
    if (e != cudaSuccess) return e;
    e = launch_rows(a.grad_c, (int64_t)a.n * q * q, p, 0, true, s);
    if (e != cudaSuccess) return e;
  }
  if (a.out != nullptr && !(both && circ_bwd_fused_supported(p, a.D, a.T))) {
    CircMany x = a;
    x.in = a.g;
    e = launch_circ_many(1, x, p, dtype, s, nullptr);
  }
  return e;
}

cudaError_t lora_rows_bf16(const LoraRows<bf16_t>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s);
cudaError_t lora_rows_f32(const LoraRows<float>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s);
cudaError_t lora_wgrad_bf16(const LoraWgrad<bf16_t>& a, cudaStream_t s);
cudaError_t lora_wgrad_f32(const LoraWgrad<float>& a, cudaStream_t s);

template <typename T>
static LoraRows<T> rows_args(const void* in, const void* w1, const void* w2, const float* scale, const void* base,
                             void* out, float* mid, int K, int N, int r) {
  LoraRows<T> a = {};
  a.in = static_cast<const T*>(in);
  a.w1 = static_cast<const T*>(w1);
  a.w2 = static_cast<const T*>(w2);
  a.scale = scale;
  a.base = static_cast<const T*>(base);
  a.out = static_cast<T*>(out);
  a.mid = mid;
  a.K = K, a.N = N, a.r = r;
  return a;
}

cudaError_t launch_lora_rows(bool bwd, const void* in, const void* w1, const void* w2, const float* scale,
                             const void* base, void* out, float* mid, const int* plan, int64_t T, int K, int N,
                             int r, int n, int dtype, cudaStream_t s) {
  if (dtype == 0)
    return lora_rows_f32(rows_args<float>(in, w1, w2, scale, base, out, mid, K, N, r), bwd, plan, T, n, s);
  return lora_rows_bf16(rows_args<bf16_t>(in, w1, w2, scale, base, out, mid, K, N, r), bwd, plan, T, n, s);
}

template <typename T>
static LoraWgrad<T> wgrad_args(const void* g, const void* x, const float* u, const float* v, const float* scale,
                               float* grad_a, float* grad_b, bool after_rows, const int* plan, int64_t tokens, int K,
                               int N, int r, int n) {
  LoraWgrad<T> a = {};
  a.x = static_cast<const T*>(x);
  a.g = static_cast<const T*>(g);
  a.u = u, a.v = v, a.scale = scale;
  a.grad_a = grad_a, a.grad_b = grad_b;
  a.K = K, a.N = N, a.r = r;
  a.after_rows = after_rows;
  a.plan = plan_view(plan, tokens, n, 2);
  return a;
}

cudaError_t launch_lora_wgrad(const void* g, const void* x, const float* u, const float* v, const float* scale,
                              float* grad_a, float* grad_b, bool after_rows, const int* plan, int64_t T, int K, int N,
                              int r, int n, int dtype, cudaStream_t s) {
  if (dtype == 0)
    return lora_wgrad_f32(wgrad_args<float>(g, x, u, v, scale, grad_a, grad_b, after_rows, plan, T, K, N, r, n), s);
  return lora_wgrad_bf16(wgrad_args<bf16_t>(g, x, u, v, scale, grad_a, grad_b, after_rows, plan, T, K, N, r, n), s);
}

}  // namespace rdfft
