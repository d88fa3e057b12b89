// Launchers shared between the C ABI layer and the kernel translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rdfft {

// Batched in-place rdFFT (inverse = false) or rdIFFT (inverse = true) of `rows`
// rows of length p; dtype 0 = fp32, 1 = bf16. Arguments are already validated.
cudaError_t launch_rows(void* data, int64_t rows, int p, int dtype, bool inverse, cudaStream_t s);

// The same transform out of place: rows read from src, written to dst (dst == src is the
// in-place transform; any other overlap is the caller's to avoid).
cudaError_t launch_rows_to(const void* src, void* dst, int64_t rows, int p, int dtype, bool inverse, cudaStream_t s);

// Reads and clears the error word of the rows kernels (bit 0: a bounded wait timed out).
cudaError_t take_rows_device_error(unsigned int* flags);

// Launches a kernel whose bounded wait must time out (self-test of the error path).
cudaError_t launch_wait_selftest(cudaStream_t s);

// Packed <-> rFFT complex layout conversion (see rdfft_to_complex / rdfft_from_complex).
cudaError_t launch_convert(const void* in, void* out, int64_t rows, int p, int dtype, bool to_complex,
                           cudaStream_t s);

// Column half of the 2-D rdFFT of `images` images of R x C (see rdfft2_fwd / rdfft2_inv):
// forward column transform with the pair combine, or its inverse.
cudaError_t launch_cols(void* data, int64_t images, int R, int C, int dtype, bool inverse, cudaStream_t s);

// Tensor-core (tcgen05) forward / grad_x of the layer for the shape it covers
// (circ_tc_supported: p = 128, D = 4096, bf16; circ_fwd_tc / circ_bwd_x_tc in rdfft.h),
// and the error word of its bounded waits.
bool circ_tc_supported(int p, int D, int dtype);
cudaError_t launch_circ_x_tc(const void* in, const float* chat, void* out, int64_t B, bool bwdx, cudaStream_t s);
cudaError_t take_tc_device_error(unsigned int* flags);

// Where a grad_c launch puts its token slices' sums, and what it reports back. Without a
// sink (or with partial == nullptr) several slices add into a zeroed grad_c with fp32
// atomics; with partial, slice s stores its packed sums at partial + s q^2 p (the whole
// q x q x p spectrum over the slice's block groups) and the caller sums the slices in order.
struct GcSink {
  float* partial = nullptr;      // in: per-slice sums (deterministic mode), or nullptr
  int64_t partial_floats = 0;    // in: capacity of partial
  bool plan_only = false;        // in: work out the launch shape, enqueue nothing
  int slices = 0;                // out: token slices of the grad_c launch
  bool ifft_done = false;        // out: the kernel also ran grad_c's rdIFFT (one slice)
};

// Backward in one kernel (grad_x and the grad_c cross-spectrum from one transform of g
// and x per input-block group) for the shapes it covers (circ_bwd_fused_supported: D = 4096
// at p = 128, 512 or 1024, and layers of one or two blocks, D in {p, 2p},
// p >= 512); the caller runs the in-place rdIFFT of grad_c after it.
bool circ_bwd_fused_supported(int p, int D, int64_t B);
// Reads and clears the error word of the fused backward (bit 0: a bounded wait for its staged
// rows timed out).
cudaError_t take_fused_device_error(unsigned int* flags);
cudaError_t launch_circ_bwd_fused(const void* g, const void* x, const float* chat, void* grad_x, float* grad_c,
                                  int64_t B, int D, int p, int dtype, cudaStream_t s, GcSink* sink);

// Block-circulant layer forward: y = W x (see circ_fwd in rdfft.h).
cudaError_t launch_circ_fwd(const void* x, const float* c_hat, void* y, int64_t B, int D, int p,
                            int dtype, cudaStream_t s);

// Block-circulant layer backward (see circ_bwd in rdfft.h). grad_x / grad_c may be null.
// With a sink whose partial is set, grad_c's token slices are summed in slice order (see
// circ_bwd_deterministic).
cudaError_t launch_circ_bwd(const void* g, const void* x, const float* c_hat, void* grad_x,
                            float* grad_c, int64_t B, int D, int p, int dtype, cudaStream_t s,
                            GcSink* sink = nullptr);

// Token slices of the grad_c launch that launch_circ_bwd would make for these sizes with
// grad_c requested (and grad_x too if with_grad_x); enqueues nothing.
cudaError_t plan_circ_bwd(int64_t B, int D, int p, int dtype, bool with_grad_x, int* slices);

// ---- adapters of many requests (see adapter_plan, lora_* and circ_*_many in rdfft.h)

// Groups the T tokens of `ids` by adapter into `plan` (adapter_plan.h).
cudaError_t launch_adapter_plan(const int* ids, int64_t T, int n, int* plan, cudaStream_t s);

// One call of the many-adapter block-circulant layer. Forward: in = x. grad_x: in = g.
// grad_c: in = x and g.
struct CircMany {
  const void* in = nullptr;
  const void* g = nullptr;
  const float* c_hat = nullptr;
  const void* base = nullptr;
  void* out = nullptr;
  float* grad_c = nullptr;
  const int* plan = nullptr;
  int64_t T = 0;
  int D = 0, n = 0;
};
// op 0 = forward, 1 = grad_x, 2 = grad_c's slots: per-slice sums in the sink's partial buffer,
// (slices + n) x q x q x p floats; with plan_only the sink receives the slice count alone.
cudaError_t launch_circ_many(int op, const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink);
// grad_x (out) and grad_c's slots in one kernel, for the shapes of circ_bwd_fused_supported.
cudaError_t launch_circ_many_fused(const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink);
// The whole backward: grad_x if out, grad_c (spatial) if grad_c.
cudaError_t launch_circ_many_bwd(const CircMany& a, int p, int dtype, cudaStream_t s, GcSink* sink);

// Low-rank adapters: rows (forward: in = x, w1 = a, w2 = b; bwd: in = g, w1 = b, w2 = a) and
// weight gradients (after_rows: the rows kernel that writes v is the launch just before on s).
// Arguments as lora_fwd / lora_bwd in rdfft.h.
cudaError_t launch_lora_rows(bool bwd, const void* in, const void* w1, const void* w2, const float* scale,
                             const void* base, void* out, float* mid, const int* plan, int64_t T, int K, int N,
                             int r, int n, int dtype, cudaStream_t s);
cudaError_t launch_lora_wgrad(const void* g, const void* x, const float* u, const float* v, const float* scale,
                              float* grad_a, float* grad_b, bool after_rows, const int* plan, int64_t T, int K, int N,
                              int r, int n, int dtype, cudaStream_t s);

// The word of the current device in which the kernels that take a plan record that it was made
// for other sizes (nullptr if CUDA does not give it), and the call that reads and clears it (bit 0;
// no CUDA call while no such kernel has been launched on the device).
unsigned int* plan_error_word();
cudaError_t take_plan_device_error(unsigned int* flags);

// Global norm and clipping of many tensors (grad_norm, clip_grad_norm in rdfft.h). `ws` holds
// grad_norm_ws_doubles(count) doubles; out == nullptr computes the norm alone.
int64_t grad_norm_ws_doubles(int count);
cudaError_t launch_grad_norm(const void* const* grads, void* const* out, const int64_t* numels, const int* dtypes,
                             int count, float max_norm, float* norm, double* ws, cudaStream_t s);

}  // namespace rdfft
