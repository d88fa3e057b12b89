// Block-circulant adapters of many requests: the layer kernels of circ_kernels.cuh over a
// batch whose tokens each use one of n adapters, or none (a plan, adapter_plan.h).
//
//     forward : y_t = base_t + W(c_a) x_t      grad_x_t = W(c_a)^T g_t     a = adapter of t
//     grad_c  : grad_c[a] = the packed cross-spectrum summed over the tokens of a, inverted
//
// A CTA takes up to TT tokens of one adapter (a tile of the plan, or part of one) and runs the
// dense layer's body on them, reading its rows through the plan's order and its adapter's part
// of c_hat, so a c_hat read from L2 serves the same number of tokens as in the dense layer.
// The base row is added in fp32 as the last transform pass stores a row.
// D = 4096, p = 512, bf16, 4096 tokens of 8 adapters (512 each), one call after another: forward 75 us
// without base, 85 with (the dense layer 68; the difference is the plan's dependent loads per CTA, then
// the base rows), both gradients 118 us (dense 106). On uneven groups, both gradients: 107 us, and 182
// with a slice per adapter instead of slices of equal length.
#pragma once

#include "circ_kernels.cuh"
#include "lora.cuh"
#include "many_policy.h"

namespace rdfft {

struct PlannedTokens {
  const int* order;
  int ntok;
  __device__ __forceinline__ int64_t row(int t) const { return __ldg(order + t); }
};
struct PlannedPositions {
  const int* order;
  __device__ __forceinline__ int64_t row(int64_t pos) const { return __ldg(order + pos); }
};

// Requests `bytes` (a multiple of 16, as is the address) into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

template <int P, typename T, int NT, int TT, int NS, bool BWDX>
__global__ void __launch_bounds__(NT, NT >= 512 ? 1 : (NT >= 256 ? 2 : 1))
k_circ_many_x(const T* __restrict__ in, const float* __restrict__ chat, const T* base, T* out, int q, int QI,
              PlanView plan) {
  griddep_wait();
  if (!plan_matches(plan)) return;
  int pos, ad, m;
  if constexpr (TT == 1) {
    pos = blockIdx.x;                                       // one token per CTA: no tile list
    ad = __ldg(plan.group + pos);
    m = 1;
  } else {
    static_assert(TT == 2 || TT == 4, "a CTA takes a whole tile of the 4-token list, or half of it");
    const int sub = blockIdx.x % (4 / TT), tile = blockIdx.x / (4 / TT);
    const int2 te = __ldg(plan.tiles + tile);               // within the list's capacity
    if (tile >= __ldg(plan.header + 2 + plan.list)) return;
    pos = te.x + sub * TT, ad = te.y;
    m = min(__ldg(plan.offsets() + ad + 1) - pos, TT);
    if (m <= 0) return;
  }
  const int o0 = blockIdx.y * QI, D = q * P;
  PlannedTokens tok{plan.order + pos, m};
  // the base rows are added at the very end: into L2 meanwhile
  if (base != nullptr && ad < plan.n && threadIdx.x < m)
    prefetch_l2(base + tok.row(threadIdx.x) * (int64_t)D + (int64_t)o0 * P, QI * P * (int)sizeof(T));
  if (ad >= plan.n) {                                       // no adapter: the base row, or zeros
    if (base == out) return;
    for (int t = 0; t < m; ++t) {
      const int64_t at = tok.row(t) * D + (int64_t)o0 * P;
      for (int e = threadIdx.x * (16 / (int)sizeof(T)); e < QI * P; e += NT * (16 / (int)sizeof(T)))
        *reinterpret_cast<uint4*>(out + at + e) =
            base ? *reinterpret_cast<const uint4*>(base + at + e) : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const float* c = chat + (int64_t)ad * q * q * P;
  circ_x_body<P, T, NT, TT, NS, BWDX>(in, c, out, tok, q, QI, o0, [&](int r) -> const T* {
    const int t = r / QI, ol = r - t * QI;
    return (base != nullptr && t < m) ? base + tok.row(t) * (int64_t)D + (int64_t)(o0 + ol) * P : nullptr;
  });
}

// Token slices of the gradient kernels: slice blockIdx.x takes an equal part of the sorted
// positions that have an adapter, and walks it adapter by adapter (a part per adapter would
// leave the launch to the adapter with most tokens). No slice is empty but those beyond the
// number of tokens, so every slot that k_sum_slots reads has been written.
struct SliceWalk {
  int64_t pos, hi, beg, end;                                // [beg, end): tokens of adapter ad
  int ad;
  bool whole;                                               // all of them
  __device__ __forceinline__ explicit SliceWalk(const PlanView& v) {
    const int64_t tokens = __ldg(v.offsets() + v.n);
    const int64_t slices = min((int64_t)gridDim.x, tokens);
    pos = hi = 0;
    if (blockIdx.x < slices) {
      pos = tokens * blockIdx.x / slices;
      hi = tokens * (blockIdx.x + 1) / slices;
    }
    beg = end = pos;
    ad = 0;
    whole = false;
  }
  __device__ __forceinline__ bool next(const PlanView& v) {
    if (pos >= hi) return false;
    ad = __ldg(v.group + pos);
    beg = pos;
    const int64_t all = __ldg(v.offsets() + ad + 1);
    end = min(all, hi);
    whole = end == all && beg == __ldg(v.offsets() + ad);
    pos = end;
    return true;
  }
  // Where the sums over this piece go, `floats` of them: the gradient itself for a whole adapter,
  // else slot (slice + adapter). In the order of the positions each next piece has a larger
  // slice, adapter or both, so no two share a slot.
  __device__ __forceinline__ float* sums(float* grad_c, float* slots, int64_t floats) const {
    return whole ? grad_c + ad * floats : slots + ((int64_t)blockIdx.x + ad) * floats;
  }
};

// grad_x of the tokens without an adapter: zeros in blocks [j0, j0 + QJ), shared by the slices.
template <int P, typename T>
__device__ __forceinline__ void zero_unplanned(T* grad_x, const PlanView& v, int q, int j0, int QJ) {
  const int beg = __ldg(v.offsets() + v.n), end = __ldg(v.offsets() + v.n + 1), w = QJ * P;
  constexpr int V = 16 / (int)sizeof(T);
  for (int t = beg + blockIdx.x; t < end; t += gridDim.x) {
    T* const row = grad_x + (int64_t)__ldg(v.order + t) * q * P + (int64_t)j0 * P;
    for (int e = threadIdx.x * V; e < w; e += blockDim.x * V) *reinterpret_cast<uint4*>(row + e) = make_uint4(0, 0, 0, 0);
  }
}

// grid: token slices x input-block groups.
template <int P, typename T, int NT, int TT, int NG, int RI, int RJ>
__global__ void __launch_bounds__(NT, 1)
k_circ_many_gc(const T* __restrict__ g, const T* __restrict__ x, float* grad_c, float* slots, int q, int QJ,
               PlanView plan) {
  griddep_wait();
  if (!plan_matches(plan)) return;
  SliceWalk walk(plan);
  while (walk.next(plan)) {
    circ_gc_body<P, T, NT, TT, NG, RI, RJ>(g, x, walk.sums(grad_c, slots, (int64_t)q * q * P),
                                           PlannedPositions{plan.order}, walk.beg, walk.end, q, QJ, true, 0);
    __syncthreads();                                        // the segment's last tile is consumed
  }
}

// Records the slots of a launch in the sink; false when it was only to be planned.
static inline bool many_slots(GcSink* sink, int slices, const CircMany& a, int64_t floats) {
  sink->slices = slices;
  return !sink->plan_only && (int64_t)(slices + a.n) * floats <= sink->partial_floats;
}

template <int P, typename T, int NT, int TT, int NS, bool BWDX>
static cudaError_t launch_many_x_cfg(const CircMany& a, cudaStream_t s) {
  constexpr int QI_MAX = NS * NT / (P / 2);
  const int q = a.D / P;
  const PlanLayout lay = plan_layout(a.T, a.n);
  const int64_t gx = TT == 1 ? a.T : lay.cap[0] * (4 / TT);
  if (gx > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int QI = layer_qi(q, QI_MAX, gx, num_sms());
  const size_t smem = sizeof(float) * (size_t)LayerGeo<P>::words(TT * q);
  auto kern = k_circ_many_x<P, T, NT, TT, NS, BWDX>;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)gx, (unsigned)(q / QI)), dim3(NT), smem, s, static_cast<const T*>(a.in),
                    a.c_hat, static_cast<const T*>(a.base), static_cast<T*>(a.out), q, QI,
                    plan_view(a.plan, a.T, a.n, 0));
}

// The dense layer's shapes (launch_x_p), with the tokens per CTA bounded by the mean group.
template <int P, typename T, bool BWDX>
static cudaError_t launch_many_x_p(const CircMany& a, cudaStream_t s) {
  const int q = a.D / P;
  if constexpr (P <= 512) {
    constexpr int NT = 256;
    constexpr int NS = (8 * (P / 2)) / NT > 0 ? (8 * (P / 2)) / NT : 1;
    const int tt = circ_many_tokens(a.T, a.n, q, NS * NT / (P / 2), num_sms(), NS * 4 <= 32 ? 4 : 2);
    if constexpr (P == 128) {
      if (tt > 1 && a.T >= 256 && q >= 16) return launch_many_x_cfg<P, T, 512, 2, 4, BWDX>(a, s);
    }
    if constexpr (NS * 4 <= 32) {
      if (tt == 4) return launch_many_x_cfg<P, T, NT, 4, NS, BWDX>(a, s);
    }
    if (tt == 2) return launch_many_x_cfg<P, T, NT, 2, NS, BWDX>(a, s);
    return launch_many_x_cfg<P, T, NT, 1, NS, BWDX>(a, s);
  } else {
    constexpr int NT = 128;
    constexpr int NS1 = (P / 2) / NT;
    constexpr int NSM = P == 2048 ? 16 : (NS1 * 4 <= 32 ? NS1 * 4 : 32);
    if constexpr (P > 1024) {
      if (q == 1) return launch_many_x_cfg<P, T, NT, 1, NS1, BWDX>(a, s);
    }
    return launch_many_x_cfg<P, T, NT, 1, NSM, BWDX>(a, s);
  }
}

template <int P, typename T, int NT, int TT, int NG, int RI, int RJ>
static cudaError_t run_many_gc(const CircMany& a, int QJ, cudaStream_t s, GcSink* sink) {
  const int q = a.D / P;
  auto kern = k_circ_many_gc<P, T, NT, TT, NG, RI, RJ>;
  const size_t smem = sizeof(float) * (size_t)LayerGeo<P>::words(TT * (q + QJ));
  const int njgroups = q / QJ;
  const int slices = circ_many_slices(a.T, a.n, njgroups, TT, num_sms());
  if (!many_slots(sink, slices, a, (int64_t)q * q * P)) return cudaSuccess;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)slices, (unsigned)njgroups), dim3(NT), smem, s,
                    static_cast<const T*>(a.g), static_cast<const T*>(a.in), a.grad_c, sink->partial, q, QJ,
                    plan_view(a.plan, a.T, a.n, 0));
}

// Accumulator shapes as launch_gc_tt.
template <int P, typename T>
static cudaError_t launch_many_gc_p(const CircMany& a, cudaStream_t s, GcSink* sink) {
  constexpr int TT = (P >= 2048) ? 1 : (P >= 1024 ? 2 : 4);
  constexpr int NT = 512;
  constexpr int HB = P / 2;
  const int q = a.D / P;
  const int QJ = layer_qj(q, HB, 32LL * NT, (a.T + TT - 1) / TT, num_sms());
  if ((int64_t)HB * q * QJ > 32LL * NT) return cudaErrorInvalidConfiguration;
  const int64_t slots = (int64_t)HB * q * QJ;
  if (q % 4 == 0 && QJ % 8 == 0) return run_many_gc<P, T, NT, TT, 1, 4, 8>(a, QJ, s, sink);
  if (q % 4 == 0 && QJ % 4 == 0) {
    if (slots <= 16LL * NT) return run_many_gc<P, T, NT, TT, 1, 4, 4>(a, QJ, s, sink);
    return run_many_gc<P, T, NT, TT, 2, 4, 4>(a, QJ, s, sink);
  }
  if (q % 2 == 0 && QJ % 2 == 0) {
    if (slots <= 4LL * NT) return run_many_gc<P, T, NT, TT, 1, 2, 2>(a, QJ, s, sink);
    if (slots <= 8LL * NT) return run_many_gc<P, T, NT, TT, 2, 2, 2>(a, QJ, s, sink);
    if (slots <= 16LL * NT) return run_many_gc<P, T, NT, TT, 4, 2, 2>(a, QJ, s, sink);
    return run_many_gc<P, T, NT, TT, 8, 2, 2>(a, QJ, s, sink);
  }
  if (slots <= 1LL * NT) return run_many_gc<P, T, NT, TT, 1, 1, 1>(a, QJ, s, sink);
  if (slots <= 4LL * NT) return run_many_gc<P, T, NT, TT, 4, 1, 1>(a, QJ, s, sink);
  if (slots <= 8LL * NT) return run_many_gc<P, T, NT, TT, 8, 1, 1>(a, QJ, s, sink);
  if (slots <= 16LL * NT) return run_many_gc<P, T, NT, TT, 16, 1, 1>(a, QJ, s, sink);
  return run_many_gc<P, T, NT, TT, 32, 1, 1>(a, QJ, s, sink);
}

// op 0 = forward (in = x), 1 = grad_x (in = g), 2 = grad_c slots (g, in = x).
template <int P>
cudaError_t circ_many_p(int op, const CircMany& a, int dtype, cudaStream_t s, GcSink* sink) {
  if (dtype == 0) {
    if (op == 0) return launch_many_x_p<P, float, false>(a, s);
    if (op == 1) return launch_many_x_p<P, float, true>(a, s);
    return launch_many_gc_p<P, float>(a, s, sink);
  }
  if (op == 0) return launch_many_x_p<P, bf16_t, false>(a, s);
  if (op == 1) return launch_many_x_p<P, bf16_t, true>(a, s);
  return launch_many_gc_p<P, bf16_t>(a, s, sink);
}

#define RDFFT_CIRC_MANY_INSTANCE(PP)                                                               \
  cudaError_t circ_many_##PP(int op, const CircMany& a, int dtype, cudaStream_t s, GcSink* sink) { \
    return circ_many_p<PP>(op, a, dtype, s, sink);                                                 \
  }

}  // namespace rdfft
