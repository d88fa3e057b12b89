// Grouping of a batch's tokens by adapter: a stable counting sort of T keys in [0, n], and
// the tile lists that the adapter kernels' CTAs read (layout in adapter_plan.h).
//
// One cluster of 1 to 8 CTAs of 32 warps; every warp owns a contiguous range of tokens, so
// counting per warp and then scanning the warps' counts of a bin (over the cluster through
// distributed shared memory) gives every token a rank that keeps the batch's order, with no
// atomics and the same result on every run. Lanes with equal keys find each other with a match;
// the first of them moves the warp's counter. The keys are read twice (4 T bytes, the second
// time from cache) and 8 T bytes and the lists are written, but a few microseconds of latency,
// not the bytes, are the time: a warp's steps of 32 tokens depend on one another (about 0.35 us
// a step over both passes), so the CTAs are chosen for few steps per warp: T = 32768, 200
// adapters: one CTA 24 us, eight 8.0 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "adapter_plan.h"
#include "internal.h"
#include "lora.cuh"
#include "pdl.cuh"
#include "rdfft.h"

namespace rdfft {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads, 1) k_adapter_plan(const int* __restrict__ ids, int T, int n, int* plan,
                                                           PlanLayout lay) {
  extern __shared__ int sm[];
  const int bins = n + 1;
  int* hist = sm;                             // [kWarps][bins]: counts, then next sorted position
  int* first = sm + kWarps * bins;            // [bins + 1]: offsets
  int* tile0 = first + bins + 1;              // [kPlanLists][bins + 1]: first tile of each group
  int* mine_all = tile0 + kPlanLists * (bins + 1);   // [bins]: this CTA's counts
  int* before = mine_all + bins;              // [bins]: tokens of the group in earlier CTAs
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int i = threadIdx.x; i < kWarps * bins; i += kThreads) hist[i] = 0;
  griddep_wait();                             // ids are complete, readers of the old plan are done
  __syncthreads();

  const int per = (T / (kThreads * (int)C) + 1) * 32;                 // tokens per warp, whole steps
  const int64_t beg64 = ((int64_t)rank * kWarps + w) * per;
  const int beg = beg64 < T ? (int)beg64 : T, end = T - beg < per ? T : beg + per;
  int* mine = hist + w * bins;
  auto key_at = [&](int t) {                  // an id outside [0, n) is "no adapter": bin n
    const int id = t < end ? __ldg(ids + t) : -1;
    return (unsigned)id < (unsigned)n ? id : n;
  };
  // kAhead steps' keys are requested together, so a step does not wait for memory
  constexpr int kAhead = 8;
  for (int t0 = beg; t0 < end; t0 += 32 * kAhead) {
    int key[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) key[s] = key_at(t0 + 32 * s + lane);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int t = t0 + 32 * s + lane;
      const unsigned in = __ballot_sync(~0u, t < end);
      if (in == 0) break;
      const unsigned same = __match_any_sync(~0u, key[s]) & in;
      if (t < end && lane == __ffs(same) - 1) mine[key[s]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();

  // per bin: the warps' counts become ranks within the CTA's part of the group
  for (int b = threadIdx.x; b < bins; b += kThreads) {
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < kWarps; ++i) {
      const int c = hist[i * bins + b];
      hist[i * bins + b] = sum;
      sum += c;
    }
    mine_all[b] = sum;
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int b = threadIdx.x; b < bins; b += kThreads) {
    int sum = 0, ahead = 0, v[8];
#pragma unroll
    for (unsigned c = 0; c < 8; ++c) v[c] = c < C ? ld_cluster_i1(map_rank(mine_all + b, c)) : 0;
#pragma unroll
    for (unsigned c = 0; c < 8; ++c) {
      if (c < rank) ahead += v[c];
      sum += v[c];
    }
    before[b] = ahead;
    first[b] = sum;
#pragma unroll
    for (int l = 0; l < kPlanLists; ++l) tile0[l * (bins + 1) + b] = (sum + plan_tile(l) - 1) / plan_tile(l);
  }
  if (C > 1) cluster_arrive();                // done with the others' counts
  __syncthreads();
  // exclusive scans of the counts (warp 0) and of each list's tiles (warps 1 to 3)
  if (w <= kPlanLists) {
    int* v = w == 0 ? first : tile0 + (w - 1) * (bins + 1);
    int carry = 0;
    for (int b0 = 0; b0 < bins; b0 += 32) {
      const int b = b0 + lane;
      const int x = b < bins ? v[b] : 0;
      int s = x;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(~0u, s, d);
        if (lane >= d) s += o;
      }
      if (b < bins) v[b] = carry + s - x;
      carry += __shfl_sync(~0u, s, 31);
    }
    if (lane == 0) {
      v[bins] = carry;
      if (w > 0 && rank == 0) plan[1 + w] = carry;
    }
  }
  if (threadIdx.x == 0 && rank == 0) {
    plan[0] = T;
    plan[1] = n;
  }
  __syncthreads();
  if (rank == 0)
    for (int b = threadIdx.x; b <= bins; b += kThreads) plan[lay.offsets + b] = first[b];

  // the ranks place the tokens; the first token of every tile writes the tile
  for (int t0 = beg; t0 < end; t0 += 32 * kAhead) {
    int key[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) key[s] = key_at(t0 + 32 * s + lane);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int t = t0 + 32 * s + lane;
      const unsigned in = __ballot_sync(~0u, t < end);
      if (in == 0) break;
      const unsigned same = __match_any_sync(~0u, key[s]) & in;
      int base = 0;
      if (t < end) base = mine[key[s]];
      __syncwarp();
      if (t < end) {
        const int at = before[key[s]] + base + __popc(same & ((1u << lane) - 1));
        const int pos = first[key[s]] + at;
        plan[lay.order + pos] = t;
        plan[lay.group + pos] = key[s];
#pragma unroll
        for (int l = 0; l < kPlanLists; ++l)
          if (at % plan_tile(l) == 0) {
            const int64_t tile = tile0[l * (bins + 1) + key[s]] + at / plan_tile(l);
            *reinterpret_cast<int2*>(plan + lay.tiles[l] + 2 * tile) = make_int2(pos, key[s]);
          }
        if (lane == __ffs(same) - 1) mine[key[s]] = base + __popc(same);
      }
      __syncwarp();
    }
  }
  if (C > 1) cluster_wait();
}

}  // namespace

// Beside the plan's kernel: whoever has a plan has loaded this module.
static __device__ unsigned int g_plan_error;
constexpr int kDevices = 64;
static std::atomic<unsigned int*> g_words[kDevices];

unsigned int* plan_error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return nullptr;
  unsigned int* word = g_words[dev].load(std::memory_order_acquire);
  if (word == nullptr) {
    void* at = nullptr;
    if (cudaGetSymbolAddress(&at, g_plan_error) != cudaSuccess) return nullptr;
    word = static_cast<unsigned int*>(at);
    g_words[dev].store(word, std::memory_order_release);
  }
  return word;
}

cudaError_t take_plan_device_error(unsigned int* flags) {
  *flags = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev >= kDevices || g_words[dev].load(std::memory_order_acquire) == nullptr) return e;
  e = cudaMemcpyFromSymbol(flags, g_plan_error, sizeof(*flags));
  if (e != cudaSuccess || *flags == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_plan_error, &zero, sizeof(zero));
}

cudaError_t launch_adapter_plan(const int* ids, int64_t T, int n, int* plan, cudaStream_t s) {
  const int bins = n + 1;
  const size_t smem = sizeof(int) * ((size_t)(kWarps + 2) * bins + (size_t)(kPlanLists + 1) * (bins + 1));
  // the most that any n needs
  const cudaError_t e = allow_smem<k_adapter_plan>(sizeof(int) * (size_t)(kWarps + 6) * (RDFFT_MAX_ADAPTERS + 2));
  if (e != cudaSuccess) return e;
  // about two steps per warp (2048 tokens per CTA)
  int cluster = 1;
  while (cluster < 8 && (int64_t)cluster * 2048 < T) cluster *= 2;
  return launch_cluster_pdl(k_adapter_plan, dim3(cluster), dim3(kThreads), cluster, smem, s, ids, (int)T, n, plan,
                            plan_layout(T, n));
}

}  // namespace rdfft
