// Shared pieces of the low-rank adapter kernels (lora_bf16.cu, lora_f32.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "adapter_plan.h"
#include "internal.h"
#include "packed_fft.cuh"
#include "pdl.cuh"

namespace rdfft {

// The parts of a plan that one kernel reads, and the sizes it must have been made for.
struct PlanView {
  const int* header;
  const int* order;
  const int* group;
  const int2* tiles;
  unsigned int* error;     // plan_error_word()
  int list;
  int T, n;
  // Behind the header in every plan, so not a field: with one more, the 64-token rows kernels spill.
  __device__ __forceinline__ const int* offsets() const { return header + kPlanHeader; }
};

inline PlanView plan_view(const int* plan, int64_t T, int n, int list) {
  const PlanLayout l = plan_layout(T, n);
  PlanView v;
  v.header = plan;
  v.order = plan + l.order;
  v.group = plan + l.group;
  v.tiles = reinterpret_cast<const int2*>(plan + l.tiles[list]);
  v.error = plan_error_word();
  v.list = list;
  v.T = (int)T;
  v.n = n;
  return v;
}

// False, and recorded for rdfft_take_device_error, when the plan was made for other sizes; the
// kernel then writes nothing. Uniform over the grid.
__device__ __forceinline__ bool plan_matches(const PlanView& v) {
  if (__ldg(v.header) == v.T && __ldg(v.header + 1) == v.n) return true;
  if (threadIdx.x == 0 && v.error != nullptr) atomicOr(v.error, 1u);
  return false;
}

// One direction of a low-rank adapter: rows of `in` (T x K) through w1 and w2 to rows of
// `out` (T x N):  mid_t = w1 in_t (r values), out_t = base_t + scale w2 mid_t.
// Forward: w1 = A (r x K), w2 = B (N x r). Backward for the input: in = g, w1 = B^T,
// w2 = A^T, both read where A and B lie (the kernels' BWD), and no base.
template <typename T>
struct LoraRows {
  const T* in;
  const T* w1;
  const T* w2;
  const float* scale;      // n, or nullptr for 1
  const T* base;           // T x N or nullptr; may be `out`
  T* out;                  // T x N, or nullptr to compute mid alone
  float* mid;              // T x r or nullptr: forward u = A x, backward v = scale B^T g
  int K, N, r;
  PlanView plan;
};

// Weight gradients over the tokens of each adapter:
//   grad_a[a] (r x K) = sum_t v_t x_t^T,  grad_b[a] (N x r) = scale_a sum_t g_t u_t^T.
template <typename T>
struct LoraWgrad {
  const T* x;
  const T* g;
  const float* u;
  const float* v;
  const float* scale;
  float* grad_a;
  float* grad_b;
  int K, N, r;
  bool after_rows;         // the rows kernel that writes v is the launch just before
  PlanView plan;
};

// The part for grad_b reads nothing that the rows kernel writes, so its CTAs need not wait for
// it: the rows kernel lets them start only after all work before it has completed. They wait
// before they exit, on every path, so that the grid still ends after the rows kernel (a launch
// behind it might otherwise write the plan or v while the rows kernel reads them).
__device__ __forceinline__ bool starts_early(bool after_rows, bool is_a) { return after_rows && !is_a; }

// The weight gradients share the batch evenly: CTA `rank` of a cluster of C takes an equal part
// [lo, hi) of the plan's 64-token tiles, whatever adapters they belong to. (A CTA per adapter
// would leave the launch to the adapter with most tokens.) Tiles lie in the order of their
// positions, so a tile ends where the next begins, and consecutive tiles of one adapter are one
// sum. kWindow tiles and their neighbours are looked up at a time.
constexpr int kWindow = 254;
struct TileShare {
  int lo, hi, all, end;                     // of `all` tiles with an adapter, whose positions end at `end`
  __device__ __forceinline__ TileShare(const PlanView& v, unsigned rank, unsigned C) {
    end = __ldg(v.offsets() + v.n);
    const int none = __ldg(v.offsets() + v.n + 1) - end;
    all = __ldg(v.header + 2 + v.list) - (none + 63) / 64;
    lo = (int)((int64_t)all * rank / C);
    hi = (int)((int64_t)all * (rank + 1) / C);
  }
  // desc[i] = tile w0 - 1 + i (position, adapter) for the window's tiles and one on either side;
  // before the first: adapter -1; after the last: `end`, adapter -1. Needs blockDim >= kWindow + 2.
  __device__ __forceinline__ void window(const PlanView& v, int w0, int2* desc) const {
    const int k = w0 - 1 + (int)threadIdx.x;
    if (threadIdx.x < kWindow + 2)
      desc[threadIdx.x] = (k >= 0 && k < all) ? __ldg(v.tiles + k) : make_int2(k < 0 ? 0 : end, -1);
  }
};

// Asynchronous copies to shared memory.
__device__ __forceinline__ uint32_t shared_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros when !in (src is then not read, but must be a valid pointer).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// The same for 4 bytes.
__device__ __forceinline__ void cp4(uint32_t dst, const int* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Cluster of this CTA (one-dimensional).
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned v;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
  return v;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned v;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(v));
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_rank(const void* p, unsigned rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ int ld_cluster_i1(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Sum over the cluster's CTAs of the four floats at `p`, in rank order; the loads go out together.
__device__ __forceinline__ float4 cluster_sum_f4(const float* p, unsigned C) {
  float4 v[8];
#pragma unroll
  for (unsigned c = 0; c < 8; ++c)
    if (c < C) v[c] = ld_cluster_f4(map_rank(p, c));
  float4 s = v[0];
#pragma unroll
  for (unsigned c = 1; c < 8; ++c)
    if (c < C) s.x += v[c].x, s.y += v[c].y, s.z += v[c].z, s.w += v[c].w;
  return s;
}

// Adds the N sums of this thread that CTA `rank` left at head[e][thread].
template <int N>
__device__ __forceinline__ void add_from(float (&acc)[N], const float* head, unsigned rank) {
  const uint32_t src = map_rank(head, rank) + 4 * threadIdx.x;
  constexpr int B = N < 16 ? N : 16;                          // loads in flight
#pragma unroll
  for (int e0 = 0; e0 < N; e0 += B) {
    float v[B];
#pragma unroll
    for (int e = 0; e < B; ++e) v[e] = ld_cluster_f1(src + 4 * blockDim.x * (e0 + e));
#pragma unroll
    for (int e = 0; e < B; ++e) acc[e0 + e] += v[e];
  }
}

// Allows KERNEL `bytes` of dynamic shared memory on the current device. The attribute stays with
// the loaded kernel, so it is set once per device (bytes is the same in every call).
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (set.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// launch_pdl with the grid cut into clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
static cudaError_t launch_cluster_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                                      cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace rdfft
