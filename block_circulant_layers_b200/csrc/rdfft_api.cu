// C ABI of the library: argument validation and dispatch (declared in rdfft.h).
// Every argument check happens before any CUDA call, so invalid calls enqueue
// nothing and need no GPU.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <mutex>

#include "rdfft.h"
#include "adapter_plan.h"
#include "internal.h"

namespace {

thread_local cudaError_t t_last_cuda = cudaSuccess;
thread_local char t_msg[256];

bool pow2_in_range(int p) { return p >= 2 && p <= 4096 && (p & (p - 1)) == 0; }
bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
bool dtype_ok(int dtype) { return dtype == RDFFT_F32 || dtype == RDFFT_BF16; }

int finish(cudaError_t e) {
  if (e == cudaSuccess) return RDFFT_OK;
  t_last_cuda = e;
  return RDFFT_ECUDA;
}

int rows_call(void* data, int64_t rows, int p, int dtype, rdfft_stream_t stream, bool inverse) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!pow2_in_range(p) || rows < 0) return RDFFT_EINVAL;
  if (rows == 0) return RDFFT_OK;
  if (data == nullptr) return RDFFT_ENULL;
  if (!aligned16(data)) return RDFFT_EALIGN;
  return finish(rdfft::launch_rows(data, rows, p, dtype, inverse, reinterpret_cast<cudaStream_t>(stream)));
}

int layer_shape_ok(int64_t B, int D, int p) {
  if (!pow2_in_range(p) || p < 64 || B < 0 || D < p || D > RDFFT_MAX_D || D % p != 0) return 0;
  return 1;
}

// Byte ranges [a, a + na) and [b, b + nb) intersect (null pointers never do).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

int convert_call(const void* in, void* out, int64_t rows, int p, int dtype, bool to_complex,
                 rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!pow2_in_range(p) || rows < 0) return RDFFT_EINVAL;
  if (rows == 0) return RDFFT_OK;
  if (in == nullptr || out == nullptr) return RDFFT_ENULL;
  if (!aligned16(in) || !aligned16(out)) return RDFFT_EALIGN;
  const size_t es = dtype == RDFFT_F32 ? 4 : 2;
  const size_t packed_bytes = (size_t)rows * p * es, cplx_bytes = (size_t)rows * (p + 2) * es;
  if (overlap(in, to_complex ? packed_bytes : cplx_bytes, out, to_complex ? cplx_bytes : packed_bytes))
    return RDFFT_EOVERLAP;
  return finish(rdfft::launch_convert(in, out, rows, p, dtype, to_complex, reinterpret_cast<cudaStream_t>(stream)));
}

// The 2-D transform: rows then columns (forward), columns then rows (inverse), in
// place; both halves are enqueued on the same stream.
int image_call(void* data, int64_t images, int R, int C, int dtype, rdfft_stream_t stream, bool inverse) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!pow2_in_range(R) || !pow2_in_range(C) || images < 0) return RDFFT_EINVAL;
  if (images > INT64_MAX / ((int64_t)R * C)) return RDFFT_EINVAL;
  if (images == 0) return RDFFT_OK;
  if (data == nullptr) return RDFFT_ENULL;
  if (!aligned16(data)) return RDFFT_EALIGN;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = images * R;
  if (!inverse) {
    const cudaError_t e = rdfft::launch_rows(data, rows, C, dtype, false, s);
    if (e != cudaSuccess) return finish(e);
    return finish(rdfft::launch_cols(data, images, R, C, dtype, false, s));
  }
  const cudaError_t e = rdfft::launch_cols(data, images, R, C, dtype, true, s);
  if (e != cudaSuccess) return finish(e);
  return finish(rdfft::launch_rows(data, rows, C, dtype, true, s));
}

// Bytes of c_hat or grad_c: q x q x p fp32.
size_t gc_bytes(int D, int p) { return sizeof(float) * (size_t)(D / p) * (D / p) * p; }

// Argument checks of the layer backward (circ_bwd, circ_bwd_deterministic). Returns
// kEnqueue when the call has work to enqueue, else the call's return code (an error, or
// RDFFT_OK when there is nothing to do or an empty batch only zeroed grad_c).
constexpr int kEnqueue = -1;
int bwd_args(const void* g, const void* x, const float* c_hat, void* grad_x, float* grad_c, int64_t B, int D,
             int p, int dtype, rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(B, D, p)) return RDFFT_EINVAL;
  if (grad_x == nullptr && grad_c == nullptr) return RDFFT_OK;
  const size_t cb = gc_bytes(D, p);
  if (B == 0) {
    // no tokens: grad_x is empty and grad_c is an empty sum
    if (grad_c == nullptr) return RDFFT_OK;
    if (!aligned16(grad_c)) return RDFFT_EALIGN;
    return finish(cudaMemsetAsync(grad_c, 0, cb, reinterpret_cast<cudaStream_t>(stream)));
  }
  if (g == nullptr || c_hat == nullptr) return RDFFT_ENULL;
  if (grad_c != nullptr && x == nullptr) return RDFFT_ENULL;
  if (!aligned16(g) || !aligned16(c_hat) || (x && !aligned16(x)) || (grad_x && !aligned16(grad_x)) ||
      (grad_c && !aligned16(grad_c)))
    return RDFFT_EALIGN;
  const size_t act = (size_t)B * D * (dtype == RDFFT_F32 ? 4 : 2);
  if (overlap(grad_x, act, g, act) || overlap(grad_x, act, x, act) || overlap(grad_x, act, c_hat, cb) ||
      overlap(grad_x, act, grad_c, cb) || overlap(grad_c, cb, g, act) || overlap(grad_c, cb, x, act) ||
      overlap(grad_c, cb, c_hat, cb))
    return RDFFT_EOVERLAP;
  return kEnqueue;
}

// Scratch of circ_bwd_deterministic_noalloc: its per-slice grad_c sums live here instead
// of in caller memory. Every device that loads the library holds it until the process exits.
constexpr size_t kNoAllocScratchBytes = RDFFT_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) float g_noalloc_scratch[kNoAllocScratchBytes / sizeof(float)];

// Device address of g_noalloc_scratch on the current device. In host code the array's name
// is only a stand-in, so the address is looked up with cudaGetSymbolAddress, once per
// device with that device current, and kept (no host or device allocation).
constexpr int kMaxDevices = 64;
cudaError_t noalloc_scratch(float** ptr) {
  static std::mutex mu;
  static float* addr[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (addr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return e;
    addr[dev] = static_cast<float*>(p);
  }
  *ptr = addr[dev];
  return cudaSuccess;
}

// ---- adapters of many requests

struct Range {
  const void* ptr;
  size_t bytes;
};

// Any of the first `nout` ranges intersects another range.
template <int N>
bool outputs_overlap(const Range (&r)[N], int nout) {
  for (int i = 0; i < nout; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlap(r[i].ptr, r[i].bytes, r[j].ptr, r[j].bytes)) return true;
  return false;
}

template <int N>
bool all_aligned16(const Range (&r)[N]) {
  for (int i = 0; i < N; ++i)
    if (!aligned16(r[i].ptr)) return false;
  return true;
}

bool plan_sizes_ok(int64_t T, int n) {
  return T >= 0 && T <= RDFFT_MAX_TOKENS && n >= 1 && n <= RDFFT_MAX_ADAPTERS;
}
size_t plan_bytes(int64_t T, int n) { return sizeof(int32_t) * (size_t)rdfft::plan_layout(T, n).words; }

bool lora_sizes_ok(int64_t T, int K, int N, int r, int n) {
  auto width = [](int w) { return w >= 8 && w <= 65536 && w % 8 == 0; };
  return plan_sizes_ok(T, n) && width(K) && width(N) && r >= 8 && r <= 128 && r % 8 == 0;
}

// Argument checks shared by grad_norm and clip_grad_norm.
int norm_args(const void* const* grads, const int64_t* numels, const int* dtypes, int count, float* norm,
              void* workspace, size_t workspace_bytes) {
  if (count < 0 || count > RDFFT_MAX_TENSORS) return RDFFT_EINVAL;
  if (norm == nullptr || (count > 0 && (grads == nullptr || numels == nullptr || dtypes == nullptr)))
    return RDFFT_ENULL;
  for (int i = 0; i < count; ++i) {
    if (!dtype_ok(dtypes[i])) return RDFFT_EDTYPE;
    if (numels[i] < 0 || numels[i] > (INT64_MAX >> 16)) return RDFFT_EINVAL;
    if (numels[i] > 0 && grads[i] == nullptr) return RDFFT_ENULL;
    if (reinterpret_cast<uintptr_t>(grads[i]) % (dtypes[i] == RDFFT_F32 ? 4 : 2)) return RDFFT_EALIGN;
  }
  if (reinterpret_cast<uintptr_t>(norm) % 4) return RDFFT_EALIGN;
  const size_t need = sizeof(double) * (size_t)rdfft::grad_norm_ws_doubles(count);
  if (need > 0) {
    if (workspace == nullptr) return RDFFT_ENULL;
    if (reinterpret_cast<uintptr_t>(workspace) % 8) return RDFFT_EALIGN;
    if (workspace_bytes < need) return RDFFT_ESPACE;
  }
  return RDFFT_OK;
}

struct Span {
  uintptr_t beg, end;
};

}  // namespace

extern "C" {

int rdfft_fwd(void* data, int64_t rows, int p, int dtype, rdfft_stream_t stream) {
  return rows_call(data, rows, p, dtype, stream, false);
}

int rdfft_inv(void* data, int64_t rows, int p, int dtype, rdfft_stream_t stream) {
  return rows_call(data, rows, p, dtype, stream, true);
}

int rdfft_to_complex(const void* packed, void* cplx, int64_t rows, int p, int dtype, rdfft_stream_t stream) {
  return convert_call(packed, cplx, rows, p, dtype, true, stream);
}

int rdfft_from_complex(const void* cplx, void* packed, int64_t rows, int p, int dtype, rdfft_stream_t stream) {
  return convert_call(cplx, packed, rows, p, dtype, false, stream);
}

int rdfft2_fwd(void* data, int64_t images, int R, int C, int dtype, rdfft_stream_t stream) {
  return image_call(data, images, R, C, dtype, stream, false);
}

int rdfft2_inv(void* data, int64_t images, int R, int C, int dtype, rdfft_stream_t stream) {
  return image_call(data, images, R, C, dtype, stream, true);
}

int circ_prepare(const float* c, float* c_hat, int D, int p, rdfft_stream_t stream) {
  if (!layer_shape_ok(0, D, p)) return RDFFT_EINVAL;
  if (c == nullptr || c_hat == nullptr) return RDFFT_ENULL;
  if (!aligned16(c) || !aligned16(c_hat)) return RDFFT_EALIGN;
  const size_t cb = sizeof(float) * (size_t)(D / p) * (D / p) * p;
  if (c != c_hat && overlap(c, cb, c_hat, cb)) return RDFFT_EOVERLAP;
  const int64_t rows = (int64_t)(D / p) * (D / p);
  return finish(rdfft::launch_rows_to(c, c_hat, rows, p, RDFFT_F32, false, reinterpret_cast<cudaStream_t>(stream)));
}

int circ_fwd(const void* x, const float* c_hat, void* y, int64_t B, int D, int p, int dtype,
             rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(B, D, p)) return RDFFT_EINVAL;
  if (B == 0) return RDFFT_OK;
  if (x == nullptr || c_hat == nullptr || y == nullptr) return RDFFT_ENULL;
  if (!aligned16(x) || !aligned16(c_hat) || !aligned16(y)) return RDFFT_EALIGN;
  const size_t act = (size_t)B * D * (dtype == RDFFT_F32 ? 4 : 2);
  const size_t cb = sizeof(float) * (size_t)(D / p) * (D / p) * p;
  if (overlap(y, act, x, act) || overlap(y, act, c_hat, cb)) return RDFFT_EOVERLAP;
  return finish(rdfft::launch_circ_fwd(x, c_hat, y, B, D, p, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int circ_bwd(const void* g, const void* x, const float* c_hat, void* grad_x, float* grad_c,
             int64_t B, int D, int p, int dtype, rdfft_stream_t stream) {
  const int chk = bwd_args(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, stream);
  if (chk != kEnqueue) return chk;
  return finish(rdfft::launch_circ_bwd(g, x, c_hat, grad_x, grad_c, B, D, p, dtype,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int circ_bwd_workspace_size(int64_t B, int D, int p, int dtype, int with_grad_x, size_t* bytes) {
  if (bytes == nullptr) return RDFFT_ENULL;
  *bytes = 0;
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(B, D, p)) return RDFFT_EINVAL;
  if (B == 0) return RDFFT_OK;
  int slices = 0;
  const cudaError_t e = rdfft::plan_circ_bwd(B, D, p, dtype, with_grad_x != 0, &slices);
  if (e != cudaSuccess) return finish(e);
  if (slices > 1) *bytes = (size_t)slices * gc_bytes(D, p);
  return RDFFT_OK;
}

int circ_bwd_deterministic(const void* g, const void* x, const float* c_hat, void* grad_x, float* grad_c,
                           int64_t B, int D, int p, int dtype, void* workspace, size_t workspace_bytes,
                           rdfft_stream_t stream) {
  const int chk = bwd_args(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, stream);
  if (chk != kEnqueue) return chk;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (grad_c == nullptr) return finish(rdfft::launch_circ_bwd(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, s));
  size_t need = 0;
  const int rc = circ_bwd_workspace_size(B, D, p, dtype, grad_x != nullptr, &need);
  if (rc != RDFFT_OK) return rc;
  rdfft::GcSink sink;
  if (need > 0) {
    if (workspace == nullptr) return RDFFT_ENULL;
    if (!aligned16(workspace)) return RDFFT_EALIGN;
    if (workspace_bytes < need) return RDFFT_ESPACE;
    const size_t act = (size_t)B * D * (dtype == RDFFT_F32 ? 4 : 2), cb = gc_bytes(D, p);
    if (overlap(workspace, need, g, act) || overlap(workspace, need, x, act) ||
        overlap(workspace, need, c_hat, cb) || overlap(workspace, need, grad_x, act) ||
        overlap(workspace, need, grad_c, cb))
      return RDFFT_EOVERLAP;
    sink.partial = static_cast<float*>(workspace);
    sink.partial_floats = (int64_t)(need / sizeof(float));
  }
  return finish(rdfft::launch_circ_bwd(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, s, &sink));
}

int circ_bwd_deterministic_noalloc(const void* g, const void* x, const float* c_hat, void* grad_x, float* grad_c,
                                   int64_t B, int D, int p, int dtype, rdfft_stream_t stream) {
  const int chk = bwd_args(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, stream);
  if (chk != kEnqueue) return chk;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (grad_c == nullptr) return finish(rdfft::launch_circ_bwd(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, s));
  size_t need = 0;
  const int rc = circ_bwd_workspace_size(B, D, p, dtype, grad_x != nullptr, &need);
  if (rc != RDFFT_OK) return rc;
  if (need > kNoAllocScratchBytes) return RDFFT_ESPACE;
  rdfft::GcSink sink;
  if (need > 0) {
    float* scratch = nullptr;
    const cudaError_t e = noalloc_scratch(&scratch);
    if (e != cudaSuccess) return finish(e);
    sink.partial = scratch;
    sink.partial_floats = (int64_t)(need / sizeof(float));
  }
  return finish(rdfft::launch_circ_bwd(g, x, c_hat, grad_x, grad_c, B, D, p, dtype, s, &sink));
}

int circ_fwd_tc(const void* x, const float* c_hat, void* y, int64_t B, int D, int p, int dtype,
                rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(B, D, p) || !rdfft::circ_tc_supported(p, D, dtype)) return RDFFT_EINVAL;
  if (B == 0) return RDFFT_OK;
  if (x == nullptr || c_hat == nullptr || y == nullptr) return RDFFT_ENULL;
  if (!aligned16(x) || !aligned16(c_hat) || !aligned16(y)) return RDFFT_EALIGN;
  const size_t act = (size_t)B * D * 2;
  const size_t cb = sizeof(float) * (size_t)(D / p) * (D / p) * p;
  if (overlap(y, act, x, act) || overlap(y, act, c_hat, cb)) return RDFFT_EOVERLAP;
  return finish(rdfft::launch_circ_x_tc(x, c_hat, y, B, false, reinterpret_cast<cudaStream_t>(stream)));
}

int circ_bwd_x_tc(const void* g, const float* c_hat, void* grad_x, int64_t B, int D, int p, int dtype,
                  rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(B, D, p) || !rdfft::circ_tc_supported(p, D, dtype)) return RDFFT_EINVAL;
  if (B == 0) return RDFFT_OK;
  if (g == nullptr || c_hat == nullptr || grad_x == nullptr) return RDFFT_ENULL;
  if (!aligned16(g) || !aligned16(c_hat) || !aligned16(grad_x)) return RDFFT_EALIGN;
  const size_t act = (size_t)B * D * 2;
  const size_t cb = sizeof(float) * (size_t)(D / p) * (D / p) * p;
  if (overlap(grad_x, act, g, act) || overlap(grad_x, act, c_hat, cb)) return RDFFT_EOVERLAP;
  return finish(rdfft::launch_circ_x_tc(g, c_hat, grad_x, B, true, reinterpret_cast<cudaStream_t>(stream)));
}

int adapter_plan_size(int64_t T, int n, int64_t* words) {
  if (words == nullptr) return RDFFT_ENULL;
  *words = 0;
  if (!plan_sizes_ok(T, n)) return RDFFT_EINVAL;
  *words = rdfft::plan_layout(T, n).words;
  return RDFFT_OK;
}

int adapter_plan(const int32_t* ids, int64_t T, int n, int32_t* plan, rdfft_stream_t stream) {
  if (!plan_sizes_ok(T, n)) return RDFFT_EINVAL;
  if (plan == nullptr || (T > 0 && ids == nullptr)) return RDFFT_ENULL;
  if (!aligned16(plan) || reinterpret_cast<uintptr_t>(ids) % 4) return RDFFT_EALIGN;
  if (overlap(plan, plan_bytes(T, n), ids, sizeof(int32_t) * (size_t)T)) return RDFFT_EOVERLAP;
  return finish(rdfft::launch_adapter_plan(ids, T, n, plan, reinterpret_cast<cudaStream_t>(stream)));
}

int lora_fwd(const void* x, const void* a, const void* b, const float* scale, const void* base, void* y, float* u,
             const int32_t* plan, int64_t T, int K, int N, int r, int n, int dtype, rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!lora_sizes_ok(T, K, N, r, n)) return RDFFT_EINVAL;
  if (T == 0) return RDFFT_OK;
  if (x == nullptr || a == nullptr || b == nullptr || y == nullptr || plan == nullptr) return RDFFT_ENULL;
  const size_t es = dtype == RDFFT_F32 ? 4 : 2;
  const Range args[] = {{y, es * T * N},
                        {u, sizeof(float) * T * r},
                        {x, es * T * K},
                        {a, es * n * r * K},
                        {b, es * n * r * N},
                        {plan, plan_bytes(T, n)},
                        {base == y ? nullptr : base, es * T * N}};
  if (!all_aligned16(args) || reinterpret_cast<uintptr_t>(scale) % 4) return RDFFT_EALIGN;
  if (outputs_overlap(args, 2) || overlap(scale, sizeof(float) * n, y, es * T * N) ||
      overlap(scale, sizeof(float) * n, u, sizeof(float) * T * r))
    return RDFFT_EOVERLAP;
  return finish(rdfft::launch_lora_rows(false, x, a, b, scale, base, y, u, plan, T, K, N, r, n, dtype,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int lora_bwd(const void* g, const void* x, const void* a, const void* b, const float* scale, const float* u, float* v,
             void* grad_x, float* grad_a, float* grad_b, const int32_t* plan, int64_t T, int K, int N, int r, int n,
             int dtype, rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!lora_sizes_ok(T, K, N, r, n)) return RDFFT_EINVAL;
  if (grad_x == nullptr && grad_a == nullptr && grad_b == nullptr) return RDFFT_OK;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t es = dtype == RDFFT_F32 ? 4 : 2;
  const size_t ga_bytes = sizeof(float) * n * r * K, gb_bytes = sizeof(float) * n * r * N;
  if (T == 0) {                                        // no tokens: empty sums
    if (!aligned16(grad_a) || !aligned16(grad_b)) return RDFFT_EALIGN;
    if (overlap(grad_a, ga_bytes, grad_b, gb_bytes)) return RDFFT_EOVERLAP;
    cudaError_t e = grad_a ? cudaMemsetAsync(grad_a, 0, ga_bytes, s) : cudaSuccess;
    if (e == cudaSuccess && grad_b) e = cudaMemsetAsync(grad_b, 0, gb_bytes, s);
    return finish(e);
  }
  const bool rows = grad_x != nullptr || grad_a != nullptr;
  if (g == nullptr || plan == nullptr || (rows && b == nullptr) || (grad_x && a == nullptr) ||
      (grad_a && (x == nullptr || v == nullptr)) || (grad_b && u == nullptr))
    return RDFFT_ENULL;
  const Range args[] = {{grad_x, es * T * K},
                        {grad_a, ga_bytes},
                        {grad_b, gb_bytes},
                        {rows ? v : nullptr, sizeof(float) * T * r},
                        {g, es * T * N},
                        {x, es * T * K},
                        {a, es * n * r * K},
                        {b, es * n * r * N},
                        {u, sizeof(float) * T * r},
                        {plan, plan_bytes(T, n)},
                        {scale, sizeof(float) * n}};
  for (const Range& r16 : args)
    if (r16.ptr != scale && !aligned16(r16.ptr)) return RDFFT_EALIGN;
  if (reinterpret_cast<uintptr_t>(scale) % 4) return RDFFT_EALIGN;
  if (outputs_overlap(args, 4)) return RDFFT_EOVERLAP;
  cudaError_t e = cudaSuccess;
  if (rows) e = rdfft::launch_lora_rows(true, g, b, a, scale, nullptr, grad_x, v, plan, T, N, K, r, n, dtype, s);
  if (e == cudaSuccess && (grad_a || grad_b))
    e = rdfft::launch_lora_wgrad(g, x, u, v, scale, grad_a, grad_b, rows, plan, T, K, N, r, n, dtype, s);
  return finish(e);
}

int circ_fwd_many(const void* x, const float* c_hat, const void* base, void* y, const int32_t* plan, int64_t T, int D,
                  int p, int n, int dtype, rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(T, D, p) || !plan_sizes_ok(T, n)) return RDFFT_EINVAL;
  if (T == 0) return RDFFT_OK;
  if (x == nullptr || c_hat == nullptr || y == nullptr || plan == nullptr) return RDFFT_ENULL;
  const size_t act = (size_t)T * D * (dtype == RDFFT_F32 ? 4 : 2);
  const Range args[] = {{y, act}, {x, act}, {c_hat, n * gc_bytes(D, p)}, {plan, plan_bytes(T, n)},
                        {base == y ? nullptr : base, act}};
  if (!all_aligned16(args)) return RDFFT_EALIGN;
  if (outputs_overlap(args, 1)) return RDFFT_EOVERLAP;
  rdfft::CircMany c;
  c.in = x, c.c_hat = c_hat, c.base = base, c.out = y, c.plan = plan;
  c.T = T, c.D = D, c.n = n;
  return finish(rdfft::launch_circ_many(0, c, p, dtype, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

int circ_bwd_many_workspace_size(int64_t T, int D, int p, int n, int dtype, int with_grad_x, size_t* bytes) {
  if (bytes == nullptr) return RDFFT_ENULL;
  *bytes = 0;
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(T, D, p) || !plan_sizes_ok(T, n)) return RDFFT_EINVAL;
  if (T == 0) return RDFFT_OK;
  rdfft::CircMany c;
  c.T = T, c.D = D, c.n = n;
  c.grad_c = reinterpret_cast<float*>(16);             // asked for; a plan touches no pointer
  if (with_grad_x) c.out = c.grad_c;
  rdfft::GcSink plan;
  plan.plan_only = true;
  const cudaError_t e = rdfft::launch_circ_many_bwd(c, p, dtype, nullptr, &plan);
  if (e == cudaSuccess) *bytes = (size_t)(plan.slices + n) * gc_bytes(D, p);
  return finish(e);
}

int circ_bwd_many(const void* g, const void* x, const float* c_hat, void* grad_x, float* grad_c, const int32_t* plan,
                  int64_t T, int D, int p, int n, int dtype, void* workspace, size_t workspace_bytes,
                  rdfft_stream_t stream) {
  if (!dtype_ok(dtype)) return RDFFT_EDTYPE;
  if (!layer_shape_ok(T, D, p) || !plan_sizes_ok(T, n)) return RDFFT_EINVAL;
  if (grad_x == nullptr && grad_c == nullptr) return RDFFT_OK;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t cb = n * gc_bytes(D, p);
  if (T == 0) {
    if (grad_c == nullptr) return RDFFT_OK;
    if (!aligned16(grad_c)) return RDFFT_EALIGN;
    return finish(cudaMemsetAsync(grad_c, 0, cb, s));
  }
  if (g == nullptr || plan == nullptr || (grad_x && c_hat == nullptr) || (grad_c && x == nullptr)) return RDFFT_ENULL;
  size_t need = 0;
  if (grad_c != nullptr) {
    const int rc = circ_bwd_many_workspace_size(T, D, p, n, dtype, grad_x != nullptr, &need);
    if (rc != RDFFT_OK) return rc;
    if (workspace == nullptr) return RDFFT_ENULL;
  }
  const size_t act = (size_t)T * D * (dtype == RDFFT_F32 ? 4 : 2);
  const Range args[] = {{grad_x, act}, {grad_c, cb}, {need ? workspace : nullptr, need}, {g, act}, {x, act},
                        {c_hat, cb}, {plan, plan_bytes(T, n)}};
  if (!all_aligned16(args)) return RDFFT_EALIGN;
  if (workspace_bytes < need) return RDFFT_ESPACE;
  if (outputs_overlap(args, 3)) return RDFFT_EOVERLAP;
  rdfft::CircMany c;
  c.in = x, c.g = g, c.c_hat = c_hat, c.out = grad_x, c.grad_c = grad_c, c.plan = plan;
  c.T = T, c.D = D, c.n = n;
  rdfft::GcSink sink;
  sink.partial = static_cast<float*>(workspace);
  sink.partial_floats = (int64_t)(need / sizeof(float));
  return finish(rdfft::launch_circ_many_bwd(c, p, dtype, s, &sink));
}

int grad_norm_workspace_size(int count, size_t* bytes) {
  if (bytes == nullptr) return RDFFT_ENULL;
  *bytes = 0;
  if (count < 0 || count > RDFFT_MAX_TENSORS) return RDFFT_EINVAL;
  *bytes = sizeof(double) * (size_t)rdfft::grad_norm_ws_doubles(count);
  return RDFFT_OK;
}

int grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes, int count, float* norm,
              void* workspace, size_t workspace_bytes, rdfft_stream_t stream) {
  const int rc = norm_args(grads, numels, dtypes, count, norm, workspace, workspace_bytes);
  if (rc != RDFFT_OK) return rc;
  const size_t ws = sizeof(double) * (size_t)rdfft::grad_norm_ws_doubles(count);
  if (overlap(norm, sizeof(float), workspace, ws)) return RDFFT_EOVERLAP;
  for (int i = 0; i < count; ++i) {
    const size_t bytes = (dtypes[i] == RDFFT_F32 ? 4 : 2) * (size_t)numels[i];
    if (overlap(grads[i], bytes, norm, sizeof(float)) || overlap(grads[i], bytes, workspace, ws)) return RDFFT_EOVERLAP;
  }
  return finish(rdfft::launch_grad_norm(grads, nullptr, numels, dtypes, count, 0.0f, norm,
                                        static_cast<double*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

int clip_grad_norm(const void* const* grads, void* const* out, const int64_t* numels, const int* dtypes, int count,
                   float max_norm, float* norm, void* workspace, size_t workspace_bytes, rdfft_stream_t stream) {
  if (!(max_norm >= 0.0f)) return RDFFT_EINVAL;
  const int rc = norm_args(grads, numels, dtypes, count, norm, workspace, workspace_bytes);
  if (rc != RDFFT_OK) return rc;
  if (count > 0 && out == nullptr) return RDFFT_ENULL;
  // outputs (and the norm and the workspace) sorted by address: neighbours must not overlap
  Span spans[RDFFT_MAX_TENSORS + 2];
  int ns = 0;
  auto span_of = [](const void* ptr, size_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(ptr);
    return Span{b, b + bytes};
  };
  spans[ns++] = span_of(norm, sizeof(float));
  if (count > 0) spans[ns++] = span_of(workspace, sizeof(double) * (size_t)rdfft::grad_norm_ws_doubles(count));
  for (int i = 0; i < count; ++i) {
    const size_t es = dtypes[i] == RDFFT_F32 ? 4 : 2;
    if (numels[i] > 0 && out[i] == nullptr) return RDFFT_ENULL;
    if (reinterpret_cast<uintptr_t>(out[i]) % es) return RDFFT_EALIGN;
    if (numels[i] > 0) spans[ns++] = span_of(out[i], es * (size_t)numels[i]);
  }
  auto by_begin = [](const Span& a, const Span& b) { return a.beg < b.beg; };
  std::sort(spans, spans + ns, by_begin);
  for (int i = 1; i < ns; ++i)
    if (spans[i].beg < spans[i - 1].end) return RDFFT_EOVERLAP;
  for (int i = 0; i < count; ++i) {
    if (numels[i] == 0) continue;
    const Span in = span_of(grads[i], (dtypes[i] == RDFFT_F32 ? 4 : 2) * (size_t)numels[i]);
    // the last span that begins before this tensor ends is the only one it can meet first
    const Span* at = std::upper_bound(spans, spans + ns, Span{in.end - 1, 0}, by_begin);
    if (at == spans) continue;
    const Span& o = *(at - 1);
    const bool own = out[i] == grads[i];
    if (own ? o.beg != in.beg : o.end > in.beg) return RDFFT_EOVERLAP;
  }
  return finish(rdfft::launch_grad_norm(grads, out, numels, dtypes, count, max_norm, norm,
                                        static_cast<double*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

const char* rdfft_strerror(int code) {
  switch (code) {
    case RDFFT_OK: return "ok";
    case RDFFT_EINVAL: return "invalid size: p must be a power of two in [2, 4096] (>= 64 for the layer), counts >= 0, D a multiple of p and <= RDFFT_MAX_D; adapters: 1 to 1024 of them, K and N multiples of 8 up to 65536, r a multiple of 8 up to 128; at most 4096 tensors, max_norm >= 0";
    case RDFFT_ENULL: return "a required pointer is NULL";
    case RDFFT_EALIGN: return "a pointer is not 16-byte aligned";
    case RDFFT_EDTYPE: return "dtype must be RDFFT_F32 (0) or RDFFT_BF16 (1)";
    case RDFFT_EOVERLAP: return "an output buffer overlaps an input buffer";
    case RDFFT_ETIMEOUT: return "a kernel's bounded wait for its data timed out; its rows were not transformed";
    case RDFFT_ESPACE:
      return "the workspace is smaller than circ_bwd_workspace_size (circ_bwd_many_workspace_size, "
             "grad_norm_workspace_size) reports for this call (for circ_bwd_deterministic_noalloc: the call needs "
             "more than its built-in 16 MiB of scratch)";
    case RDFFT_EPLAN: return "a kernel was given an adapter plan made for other sizes; its outputs are not valid";
    case RDFFT_ECUDA:
      snprintf(t_msg, sizeof(t_msg), "CUDA error while enqueuing: %s (%d)", cudaGetErrorString(t_last_cuda),
               (int)t_last_cuda);
      return t_msg;
    default: return "unknown rdfft error code";
  }
}

int rdfft_take_device_error(void) {
  unsigned int flags = 0, tc_flags = 0, fused_flags = 0, plan_flags = 0;
  cudaError_t e = rdfft::take_rows_device_error(&flags);
  if (e == cudaSuccess) e = rdfft::take_tc_device_error(&tc_flags);
  if (e == cudaSuccess) e = rdfft::take_fused_device_error(&fused_flags);
  if (e == cudaSuccess) e = rdfft::take_plan_device_error(&plan_flags);
  if (e != cudaSuccess) return finish(e);
  if ((flags | tc_flags | fused_flags) & 1u) return RDFFT_ETIMEOUT;
  return plan_flags ? RDFFT_EPLAN : RDFFT_OK;
}

int rdfft_selftest_wait_timeout(rdfft_stream_t stream) {
  return finish(rdfft::launch_wait_selftest(reinterpret_cast<cudaStream_t>(stream)));
}

int rdfft_version(void) { return 120; }

}  // extern "C"
