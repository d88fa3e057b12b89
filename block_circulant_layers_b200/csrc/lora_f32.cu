// Low-rank adapters of many requests, fp32: rows kernel (forward, grad_x) and weight
// gradients. The same split as lora_bf16.cu (one cluster per tile of the plan, one launch),
// with the products as fp32 FMAs on register tiles fed from shared memory: the parity bar of
// fp32 leaves no room for tf32 operands. Operand chunks lie in shared memory with the
// contraction index outermost, so a thread's rows and columns are one vector each.
#include "lora.cuh"

#include "many_policy.h"

namespace rdfft {

namespace {

constexpr int kThreads = 256;
constexpr int kKC = 32;                        // contraction indices per chunk

// N consecutive floats of shared memory.
template <int N>
__device__ __forceinline__ void lds(const float* p, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = p[0];
  } else if constexpr (N == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x, v[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(p + 4 * i);
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  }
}

__device__ __forceinline__ float4 ldg4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void put(float* p, int stride, float4 v) {
  p[0] = v.x, p[stride] = v.y, p[2 * stride] = v.z, p[3 * stride] = v.w;
}

template <int R, int M>
struct RowsShape {
  static constexpr int KG = 64 / M;                         // thread groups that share a chunk's indices
  static constexpr int XS = M + 4, WS = R + 4;              // padded strides
  static constexpr int NC = 4096 / M, NS = NC + 4;          // output columns per pass
  static constexpr int kChunk = kKC * (XS + WS), kExpand = kKC * NS, kPart = KG * M * R;
  static constexpr int kStage = kChunk > kExpand ? kChunk : kExpand;
  static constexpr size_t smem = sizeof(float) * (size_t)(kStage + kPart + R * XS);
};

template <int R, int M, bool BWD>
__global__ void __launch_bounds__(kThreads) k_lora_rows_f32(LoraRows<float> a) {
  using S = RowsShape<R, M>;
  constexpr int RT = R / 16;                                // r values per thread
  extern __shared__ __align__(16) float sm[];
  float* const xs = sm;                                     // [kKC][XS]
  float* const ws = sm + kKC * S::XS;                       // [kKC][WS]
  float* const part = sm + S::kStage;                       // [KG][M][R]
  float* const mid = part + S::kPart;                       // [R][XS]

  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int tile = blockIdx.x / C;
  const int2 te = __ldg(a.plan.tiles + tile);               // within the list's capacity
  if (tile >= __ldg(a.plan.header + 2 + a.plan.list)) return;   // the whole cluster leaves
  const int pos0 = te.x, ad = te.y;
  const int m = min(__ldg(a.plan.offsets + ad + 1) - pos0, M);
  const int tid = threadIdx.x, K = a.K, N = a.N, r = a.r;
  const bool adapted = ad < a.plan.n;

  if (adapted) {
    // ---- mid = in w1^T over this CTA's units of 32 columns: 4 rows x RT values per thread
    constexpr int GT = 4 * M;                               // threads of one k group
    const int kg = tid / GT, rg = tid % GT / 16, cg = tid % 16;
    const int units = (K + 31) / 32;
    const int u0 = (int)((int64_t)units * rank / C), u1 = (int)((int64_t)units * (rank + 1) / C);
    const float* const w1 = a.w1 + (int64_t)ad * r * K;
    float acc[4][RT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = 0.0f;
    constexpr int XL = (M * 8 + kThreads - 1) / kThreads, WL = (R * 8 + kThreads - 1) / kThreads;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int64_t xrow[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int t = (tid + kThreads * i) / 8;
      xrow[i] = t < m ? (int64_t)__ldg(a.plan.order + pos0 + t) * K : -1;
    }
    float4 xv[XL], wv[WL];
    auto fetch = [&](int u) {
      const int k0 = 32 * u;
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int k = k0 + (tid + kThreads * i) % 8 * 4;
        xv[i] = (xrow[i] >= 0 && k < K) ? ldg4(a.in + xrow[i] + k) : zero;
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        const int e = tid + kThreads * i;
        if constexpr (!BWD) {
          const int rho = e / 8, k = k0 + e % 8 * 4;
          wv[i] = (rho < r && k < K) ? ldg4(w1 + (int64_t)rho * K + k) : zero;
        } else {
          const int k = k0 + e / (R / 4), rho = e % (R / 4) * 4;
          wv[i] = (e < R * 8 && rho < r && k < K) ? ldg4(w1 + (int64_t)k * r + rho) : zero;
        }
      }
    };
    if (u0 < u1) fetch(u0);
    for (int u = u0; u < u1; ++u) {
      __syncthreads();                                      // the previous chunk is consumed
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int e = tid + kThreads * i;
        if (e < M * 8) put(xs + e % 8 * 4 * S::XS + e / 8, S::XS, xv[i]);
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        const int e = tid + kThreads * i;
        if (e >= R * 8) continue;
        if constexpr (!BWD)
          put(ws + e % 8 * 4 * S::WS + e / 8, S::WS, wv[i]);
        else
          *reinterpret_cast<float4*>(ws + e / (R / 4) * S::WS + e % (R / 4) * 4) = wv[i];
      }
      __syncthreads();
      if (u + 1 < u1) fetch(u + 1);
#pragma unroll 8
      for (int k = kg * (kKC / S::KG); k < (kg + 1) * (kKC / S::KG); ++k) {
        float xr[4], wr[RT];
        lds<4>(xs + k * S::XS + 4 * rg, xr);
        lds<RT>(ws + k * S::WS + RT * cg, wr);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] = fmaf(xr[i], wr[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) part[(kg * M + 4 * rg + i) * R + RT * cg + j] = acc[i][j];
    __syncthreads();
    if constexpr (S::KG > 1) {
      for (int e = tid; e < M * R; e += kThreads) {
        float s = part[e];
#pragma unroll
        for (int k = 1; k < S::KG; ++k) s += part[k * M * R + e];
        part[e] = s;
      }
    }
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // the cluster's sum in rank order, every CTA for itself
    const float scale = a.scale ? __ldg(a.scale + ad) : 1.0f;
    for (int e = 4 * tid; e < M * R; e += 4 * kThreads) {
      float4 s = zero;
      if (C > 1) {
        for (unsigned c = 0; c < C; ++c) {
          const float4 v = ld_cluster_f4(map_rank(part + e, c));
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
      } else {
        s = *reinterpret_cast<const float4*>(part + e);
      }
      const int t = e / R, c = e % R;
      // columns beyond r stay zero even where a row holds an infinity (0 x inf)
      const float4 ss = c < r ? make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w) : zero;
      if (a.mid && t < m && c < r && (unsigned)(t % C) == rank)
        *reinterpret_cast<float4*>(a.mid + (int64_t)__ldg(a.plan.order + pos0 + t) * r + c) = BWD ? ss : s;
      put(mid + c * S::XS + t, S::XS, ss);
    }
    if (C > 1) cluster_arrive();                            // done with the others' memory
    __syncthreads();
  } else if (a.mid) {
    for (int e = tid; e < m * r; e += kThreads) {           // tokens without an adapter: mid is zero
      const int t = e / r;
      if ((unsigned)(t % C) == rank) a.mid[(int64_t)__ldg(a.plan.order + pos0 + t) * r + e % r] = 0.0f;
    }
  }
  griddep_launch_dependents();

  // ---- out = base + mid w2^T over this CTA's columns: 4 rows x 4 columns per thread
  if (a.out != nullptr && (adapted || a.base != a.out)) {
    const int rg = tid % (M / 4), cg = tid / (M / 4);
    const int groups = (N + S::NC - 1) / S::NC;
    const int g0 = (int)((int64_t)groups * rank / C), g1 = (int)((int64_t)groups * (rank + 1) / C);
    const float* const w2 = a.w2 + (int64_t)(adapted ? ad : 0) * r * N;
    for (int gr = g0; gr < g1; ++gr) {
      const int n0 = S::NC * gr, c = n0 + 4 * cg;
      float acc[4][4];
      int64_t orow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * rg + i;
        orow[i] = (t < m && c < N) ? (int64_t)__ldg(a.plan.order + pos0 + t) * N + c : -1;
        float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.base && orow[i] >= 0) b = *reinterpret_cast<const float4*>(a.base + orow[i]);
        acc[i][0] = b.x, acc[i][1] = b.y, acc[i][2] = b.z, acc[i][3] = b.w;
      }
      for (int r0 = 0; adapted && r0 < r; r0 += kKC) {
        __syncthreads();
        for (int e = tid; e < S::NC * 8; e += kThreads) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if constexpr (!BWD) {
            const int cc = e / 8, rho = r0 + e % 8 * 4;
            if (n0 + cc < N && rho < r) v = ldg4(w2 + (int64_t)(n0 + cc) * r + rho);
            put(sm + e % 8 * 4 * S::NS + cc, S::NS, v);
          } else {
            const int rho = e / (S::NC / 4), cc = e % (S::NC / 4) * 4;
            if (n0 + cc < N && r0 + rho < r) v = ldg4(w2 + (int64_t)(r0 + rho) * N + n0 + cc);
            *reinterpret_cast<float4*>(sm + rho * S::NS + cc) = v;
          }
        }
        __syncthreads();
        const int kn = min(kKC, R - r0);
#pragma unroll 8
        for (int k = 0; k < kn; ++k) {
          float mr[4], wr[4];
          lds<4>(mid + (r0 + k) * S::XS + 4 * rg, mr);
          lds<4>(sm + k * S::NS + 4 * cg, wr);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(mr[i], wr[j], acc[i][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (orow[i] >= 0)
          *reinterpret_cast<float4*>(a.out + orow[i]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
  }
  if (adapted && C > 1) cluster_wait();                     // the others are done with this CTA's memory
}

// ------------------------------------------------------------------- weight gradients
// One cluster: 64 columns of x (grad_a) or of g (grad_b) over all tokens, its CTAs sharing the
// plan's 64-token tiles evenly (TileShare); 4 columns x R / 16 values of r per thread. An
// adapter whose tiles lie in several CTAs is written by the first of them, as in lora_bf16.cu.
constexpr int kTok = 64;
template <int R>
constexpr size_t wgrad_smem() { return sizeof(float) * (kTok * (64 + 4) + kTok * (R + 4) + R * 64); }

template <int R>
__global__ void __launch_bounds__(kThreads) k_lora_wgrad_f32(LoraWgrad<float> a, int blocks_a) {
  constexpr int RT = R / 16, XS = 64 + 4, WS = R + 4;
  extern __shared__ __align__(16) float sm[];
  float* const xs = sm;                                     // [kTok][XS]
  float* const ws = sm + kTok * XS;                         // [kTok][WS]
  float* const head = ws + kTok * WS;                       // [4 RT][kThreads]
  __shared__ int2 desc[kWindow + 2];
  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int r = a.r, tid = threadIdx.x, block = blockIdx.x / C;
  const bool is_a = block < blocks_a;
  const int n0 = 64 * (is_a ? block : block - blocks_a);
  const int W = is_a ? a.K : a.N;
  const float* const rows = is_a ? a.x : a.g;
  const float* const mid = is_a ? a.v : a.u;
  // consecutive threads write consecutive elements: columns for grad_a, r for grad_b
  const int cg = is_a ? tid % 16 : tid / 16, rg = is_a ? tid / 16 : tid % 16;
  const TileShare share(a.plan, rank, C);
  float acc[4][RT];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = 0.0f;
  };
  auto write = [&](int ad) {
    const float scale = (!is_a && a.scale) ? __ldg(a.scale + ad) : 1.0f;
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rho = RT * rg + j, c = n0 + 4 * cg + i;
        if (rho >= r || c >= W) continue;
        if (is_a)
          a.grad_a[((int64_t)ad * r + rho) * W + c] = acc[i][j];
        else
          a.grad_b[((int64_t)ad * W + c) * r + rho] = scale * acc[i][j];
      }
  };
  constexpr int XL = kTok * 16 / kThreads, WL = kTok * R / 4 / kThreads;
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float4 xv[XL], wv[WL];
  auto fetch = [&](int p0, int tokens) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int e = tid + kThreads * i, k = e / 16, c = n0 + e % 16 * 4;
      xv[i] = (k < tokens && c < W) ? ldg4(rows + (int64_t)__ldg(a.plan.order + p0 + k) * W + c) : zero;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int e = tid + kThreads * i, k = e / (R / 4), rho = e % (R / 4) * 4;
      wv[i] = (k < tokens && rho < r) ? ldg4(mid + (int64_t)__ldg(a.plan.order + p0 + k) * r + rho) : zero;
    }
  };
  clear();
  int open = -1;                                            // adapter whose sums go on in the next CTA
  bool from_before = false;                                 // the sum at hand began in an earlier CTA
  for (int w0 = share.lo; w0 < share.hi; w0 += kWindow) {
    const int count = min(kWindow, share.hi - w0);
    __syncthreads();
    share.window(a.plan, w0, desc);
    __syncthreads();
    if (w0 == share.lo) from_before = desc[0].y == desc[1].y;
    fetch(desc[1].x, desc[2].x - desc[1].x);
    for (int i = 0; i < count; ++i) {
      __syncthreads();                                      // the last tile is consumed
#pragma unroll
      for (int h = 0; h < XL; ++h) {
        const int e = tid + kThreads * h;
        *reinterpret_cast<float4*>(xs + e / 16 * XS + e % 16 * 4) = xv[h];
      }
#pragma unroll
      for (int h = 0; h < WL; ++h) {
        const int e = tid + kThreads * h;
        *reinterpret_cast<float4*>(ws + e / (R / 4) * WS + e % (R / 4) * 4) = wv[h];
      }
      __syncthreads();
      const int tokens = desc[i + 2].x - desc[i + 1].x, ad = desc[i + 1].y;
      if (i + 1 < count) fetch(desc[i + 2].x, desc[i + 3].x - desc[i + 2].x);
#pragma unroll 8
      for (int k = 0; k < tokens; ++k) {
        float xr[4], wr[RT];
        lds<4>(xs + k * XS + 4 * cg, xr);
        lds<RT>(ws + k * WS + RT * rg, wr);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[x][j] = fmaf(xr[x], wr[j], acc[x][j]);
      }
      const bool goes_on = desc[i + 2].y == ad;             // the next tile is the same adapter's
      if (w0 + i + 1 == share.hi && goes_on && !from_before) {
        open = ad;                                          // its sums stay here
      } else if (!goes_on || w0 + i + 1 == share.hi) {
        if (from_before) {                                  // an earlier CTA writes it
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < RT; ++j) head[(x * RT + j) * kThreads + tid] = acc[x][j];
          from_before = false;
        } else {
          write(ad);
        }
        clear();
      }
    }
  }
  griddep_launch_dependents();
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (open >= 0) {
      // the CTAs after this one up to the adapter's end hold its other sums
      for (unsigned k = rank + 1; k < C; ++k) {
        const int klo = (int)((int64_t)share.all * k / C), khi = (int)((int64_t)share.all * (k + 1) / C);
        if (klo == khi) continue;                           // no tiles there
        if (__ldg(a.plan.tiles + klo).y != open) break;
        const uint32_t src = map_rank(head, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] += ld_cluster_f1(src + 4 * ((i * RT + j) * kThreads + tid));
      }
      write(open);
    }
    cluster_arrive();
  }
  clear();
  for (int ad = rank; ad < a.plan.n; ad += C)               // adapters without tokens
    if (__ldg(a.plan.offsets + ad) == __ldg(a.plan.offsets + ad + 1)) write(ad);
  if (C > 1) cluster_wait();                                // the others are done with this CTA's memory
}

template <int R, int M, bool BWD>
cudaError_t run_rows(const LoraRows<float>& a, int64_t tiles, int cluster, cudaStream_t s) {
  constexpr size_t smem = RowsShape<R, M>::smem;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_lora_rows_f32<R, M, BWD>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_cluster_pdl(k_lora_rows_f32<R, M, BWD>, dim3((unsigned)(tiles * cluster)), dim3(kThreads), cluster,
                            smem, s, a);
}

template <int R, bool BWD>
cudaError_t rows_m(LoraRows<float> a, const int* plan, int64_t T, int n, cudaStream_t s) {
  const int list = lora_list(T, n);
  a.plan = plan_view(plan, T, n, list);
  const int64_t tiles = plan_layout(T, n).cap[list];
  const int cluster = lora_cluster(tiles, a.K, a.N);
  if (list == 1) return run_rows<R, 16, BWD>(a, tiles, cluster, s);
  return run_rows<R, 64, BWD>(a, tiles, cluster, s);
}

template <bool BWD>
cudaError_t rows_r(const LoraRows<float>& a, const int* plan, int64_t T, int n, cudaStream_t s) {
  if (a.r <= 16) return rows_m<16, BWD>(a, plan, T, n, s);
  if (a.r <= 32) return rows_m<32, BWD>(a, plan, T, n, s);
  if (a.r <= 64) return rows_m<64, BWD>(a, plan, T, n, s);
  return rows_m<128, BWD>(a, plan, T, n, s);
}

template <int R>
cudaError_t run_wgrad(const LoraWgrad<float>& a, cudaStream_t s) {
  const int ka = (a.K + 63) / 64, nb = (a.N + 63) / 64;
  const int ba = a.grad_a ? ka : 0, bb = a.grad_b ? nb : 0;
  constexpr size_t smem = wgrad_smem<R>();
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_lora_wgrad_f32<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  // by both widths, so that a gradient does not depend on whether the other is asked for
  const int cluster = lora_token_split(a.plan.T, ka + nb, kTok);
  return launch_cluster_pdl(k_lora_wgrad_f32<R>, dim3((unsigned)((ba + bb) * cluster)), dim3(kThreads), cluster, smem, s,
                            a, ba);
}

}  // namespace

cudaError_t lora_rows_f32(const LoraRows<float>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s) {
  return bwd ? rows_r<true>(a, plan, T, n, s) : rows_r<false>(a, plan, T, n, s);
}

cudaError_t lora_wgrad_f32(const LoraWgrad<float>& a, cudaStream_t s) {
  if (a.r <= 16) return run_wgrad<16>(a, s);
  if (a.r <= 32) return run_wgrad<32>(a, s);
  if (a.r <= 64) return run_wgrad<64>(a, s);
  return run_wgrad<128>(a, s);
}

cudaError_t take_lora_f32_error(unsigned int* flags) { return take_error_word(flags); }

}  // namespace rdfft
