// Many-adapter operators: dispatch on the block size or the dtype, and the error words of
// their translation units.
#include <cuda_runtime.h>

#include "internal.h"
#include "lora.cuh"

namespace rdfft {

#define RDFFT_MANY_P(X) X(64) X(128) X(256) X(512) X(1024) X(2048) X(4096)
#define RDFFT_MANY_DECL(PP)                                                                      \
  cudaError_t circ_many_##PP(int op, const CircMany& a, int dtype, cudaStream_t s, GcSink* sink); \
  cudaError_t take_circ_many_error_##PP(unsigned int* flags);
RDFFT_MANY_P(RDFFT_MANY_DECL)

cudaError_t launch_circ_many(int op, const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink) {
  switch (p) {
#define RDFFT_MANY_CASE(PP) \
  case PP: return circ_many_##PP(op, a, dtype, s, sink);
    RDFFT_MANY_P(RDFFT_MANY_CASE)
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t lora_rows_bf16(const LoraRows<bf16_t>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s);
cudaError_t lora_rows_f32(const LoraRows<float>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s);
cudaError_t lora_wgrad_bf16(const LoraWgrad<bf16_t>& a, cudaStream_t s);
cudaError_t lora_wgrad_f32(const LoraWgrad<float>& a, cudaStream_t s);
cudaError_t take_lora_bf16_error(unsigned int* flags);
cudaError_t take_lora_f32_error(unsigned int* flags);

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
                               float* grad_a, float* grad_b, const int* plan, int64_t tokens, int K, int N, int r,
                               int n) {
  LoraWgrad<T> a = {};
  a.x = static_cast<const T*>(x);
  a.g = static_cast<const T*>(g);
  a.u = u, a.v = v, a.scale = scale;
  a.grad_a = grad_a, a.grad_b = grad_b;
  a.K = K, a.N = N, a.r = r;
  a.plan = plan_view(plan, tokens, n, 2);
  return a;
}

cudaError_t launch_lora_wgrad(const void* g, const void* x, const float* u, const float* v, const float* scale,
                              float* grad_a, float* grad_b, const int* plan, int64_t T, int K, int N, int r, int n,
                              int dtype, cudaStream_t s) {
  if (dtype == 0)
    return lora_wgrad_f32(wgrad_args<float>(g, x, u, v, scale, grad_a, grad_b, plan, T, K, N, r, n), s);
  return lora_wgrad_bf16(wgrad_args<bf16_t>(g, x, u, v, scale, grad_a, grad_b, plan, T, K, N, r, n), s);
}

cudaError_t take_plan_device_error(unsigned int* flags) {
  *flags = 0;
  cudaError_t (*const words[])(unsigned int*) = {
      take_lora_bf16_error,
      take_lora_f32_error,
#define RDFFT_MANY_WORD(PP) take_circ_many_error_##PP,
      RDFFT_MANY_P(RDFFT_MANY_WORD)};
  for (auto take : words) {
    unsigned int f = 0;
    const cudaError_t e = take(&f);
    if (e != cudaSuccess) return e;
    *flags |= f;
  }
  return cudaSuccess;
}

}  // namespace rdfft
