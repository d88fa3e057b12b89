// Low-rank adapters of many requests, fp32: rows kernel (forward, grad_x) and weight
// gradients. The same split as lora_bf16.cu (one cluster per tile of the plan, one launch),
// with the products as fp32 FMAs on register tiles fed from shared memory: the parity bar of
// fp32 leaves no room for tf32 operands. Steps of 32 or 64 contraction indices, then of 64
// output columns, pass through one ring of cp.async stages; operands keep their own row order, padded
// by 16 bytes a row, and are read 4 contraction indices at a time; sums are kept on packed fp32
// pairs. Shared-memory reads and their latency bound it: K = N = 2048, r = 16, 4096 tokens 39.2 us
// forward (101 MB: 15 us); K = N = 4096, r = 64 163 us (26 TFLOP/s).
#include "lora.cuh"

#include "many_policy.h"

namespace rdfft {

namespace {

constexpr int kThreads = 256;
constexpr int kNC = 64;                        // output columns per step

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

template <int R, int M, bool BWD>
struct RowsShape {
  static constexpr int kKC = M == 16 && R <= 64 ? 64 : 32;  // contraction indices per step
  static constexpr int KG = 64 / M;                         // thread groups that share a step's indices
  static constexpr int XS = kKC + 4;                        // padded strides: in,
  static constexpr int W1S = BWD ? R + 4 : kKC + 4;         // w1 (backward: contraction index outermost),
  static constexpr int W2S = BWD ? kNC + 4 : R + 4;         // w2 (the same),
  static constexpr int MS = R + 4;                          // mid
  static constexpr int kFirst = M * XS + (BWD ? kKC : R) * W1S, kSecond = (BWD ? R : kNC) * W2S;
  static constexpr int kStage = kFirst > kSecond ? kFirst : kSecond;
  static constexpr int kStages = R <= 64 ? 4 : 3;
  static constexpr int kPart = KG * M * R;
  static constexpr size_t smem = sizeof(float) * (size_t)(kStage * kStages + kPart + M * MS);
};

template <int R, int M, bool BWD>
__global__ void __launch_bounds__(kThreads) k_lora_rows_f32(LoraRows<float> a) {
  using S = RowsShape<R, M, BWD>;
  constexpr int RT = R / 16, kKC = S::kKC, KU = kKC / 4;    // r values per thread; 16-byte units per row of a step
  extern __shared__ __align__(16) float sm[];               // ring
  float* const part = sm + S::kStage * S::kStages;          // [KG][M][R]
  float* const mid = part + S::kPart;                       // [M][MS]

  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int tile = blockIdx.x / C;
  const int2 te = __ldg(a.plan.tiles + tile);               // within the list's capacity
  if (tile >= __ldg(a.plan.header + 2 + a.plan.list)) return;   // the whole cluster leaves
  const int pos0 = te.x, ad = te.y;
  const int m = min(__ldg(a.plan.offsets() + ad + 1) - pos0, M);
  const int tid = threadIdx.x, K = a.K, N = a.N, r = a.r;
  const bool adapted = ad < a.plan.n;

  // this CTA's steps: [0, n1) of kKC columns of in and w1, then [n1, n1 + n2) of 64 of w2
  const int ks = (K + kKC - 1) / kKC, ns = (N + kNC - 1) / kNC;
  const int k_first = (int)((int64_t)ks * rank / C), n_first = (int)((int64_t)ns * rank / C);
  const int n1 = adapted ? (int)((int64_t)ks * (rank + 1) / C) - k_first : 0;
  const int n2 = (a.out != nullptr && (adapted || a.base != a.out)) ? (int)((int64_t)ns * (rank + 1) / C) - n_first : 0;
  const float* const w1 = a.w1 + (adapted ? (int64_t)ad * r * K : 0);
  const float* const w2 = a.w2 + (adapted ? (int64_t)ad * r * N : 0);
  constexpr int XL = (M * KU + kThreads - 1) / kThreads;
  int xtok[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int t = (tid + kThreads * i) / KU;
    xtok[i] = t < m ? __ldg(a.plan.order + pos0 + t) : -1;
  }
  auto request = [&](int step) {
    if (adapted && step < n1 + n2) {
      const uint32_t dst = shared_at(sm + step % S::kStages * S::kStage);
      if (step < n1) {
        const int k0 = kKC * (k_first + step);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          const int e = tid + kThreads * i, k = k0 + e % KU * 4;
          const bool in = xtok[i] >= 0 && k < K;
          if (e < M * KU) cp16(dst + (e / KU * S::XS + e % KU * 4) * 4, in ? a.in + (int64_t)xtok[i] * K + k : a.in, in);
        }
        const uint32_t wdst = dst + M * S::XS * 4;
#pragma unroll
        for (int i = 0; i < (R * KU + kThreads - 1) / kThreads; ++i) {
          const int e = tid + kThreads * i;
          if (R * KU < kThreads && e >= R * KU) break;
          if constexpr (!BWD) {
            const int rho = e / KU, k = k0 + e % KU * 4;
            const bool in = rho < r && k < K;
            cp16(wdst + (rho * S::W1S + e % KU * 4) * 4, in ? w1 + (int64_t)rho * K + k : w1, in);
          } else {
            const int k = k0 + e / (R / 4), rho = e % (R / 4) * 4;
            const bool in = rho < r && k < K;
            cp16(wdst + (e / (R / 4) * S::W1S + rho) * 4, in ? w1 + (int64_t)k * r + rho : w1, in);
          }
        }
      } else {
        const int n0 = kNC * (n_first + step - n1);
#pragma unroll
        for (int i = 0; i < kNC * R / 4 / kThreads; ++i) {
          const int e = tid + kThreads * i;
          if constexpr (!BWD) {
            const int c = e / (R / 4), rho = e % (R / 4) * 4;
            const bool in = n0 + c < N && rho < r;
            cp16(dst + (c * S::W2S + rho) * 4, in ? w2 + (int64_t)(n0 + c) * r + rho : w2, in);
          } else {
            const int rho = e / (kNC / 4), c = e % (kNC / 4) * 4;
            const bool in = n0 + c < N && rho < r;
            cp16(dst + (rho * S::W2S + c) * 4, in ? w2 + (int64_t)rho * N + n0 + c : w2, in);
          }
        }
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) request(s);

  if (adapted) {
    // ---- mid = in w1^T: 4 rows x RT values per thread, rows 4 rg + i, values cg + 16 j (backward RT cg + j)
    constexpr int GT = 4 * M;                               // threads of one k group
    const int kg = tid / GT, rg = tid % GT / 16, cg = tid % 16;
    // sums on packed fp32 pairs: the even and the odd contraction indices (added at the end), or,
    // backward with several values of r per thread, which lie side by side, two of those
    constexpr bool PAIR_R = BWD && RT > 1;
    constexpr int PJ = PAIR_R ? RT / 2 : RT;
    f2 acc[4][PJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < PJ; ++j) acc[i][j] = f2_bc(0.0f);
    for (int step = 0; step < n1; ++step) {
      cp_wait<S::kStages - 2>();
      __syncthreads();
      request(step + S::kStages - 1);
      const float* const xs = sm + step % S::kStages * S::kStage;
      const float* const ws = xs + M * S::XS;
#pragma unroll 2
      for (int k = kg * (kKC / S::KG); k < (kg + 1) * (kKC / S::KG); k += 4) {
        float xr[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) lds<4>(xs + (4 * rg + i) * S::XS + k, xr[i]);
        if constexpr (!BWD) {
#pragma unroll
          for (int j = 0; j < RT; ++j) {
            float wr[4];
            lds<4>(ws + (cg + 16 * j) * S::W1S + k, wr);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 4; e += 2)
                acc[i][j] = f2_fma(f2_mk(xr[i][e], xr[i][e + 1]), f2_mk(wr[e], wr[e + 1]), acc[i][j]);
          }
        } else if constexpr (!PAIR_R) {
          float wr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) wr[e] = ws[(k + e) * S::W1S + cg];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              acc[i][0] = f2_fma(f2_mk(xr[i][e], xr[i][e + 1]), f2_mk(wr[e], wr[e + 1]), acc[i][0]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float wr[RT];
            lds<RT>(ws + (k + e) * S::W1S + RT * cg, wr);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < PJ; ++j)
                acc[i][j] = f2_fma(f2_bc(xr[i][e]), f2_mk(wr[(2 * j) % RT], wr[(2 * j + 1) % RT]), acc[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j)
        part[(kg * M + 4 * rg + i) * R + (BWD ? RT * cg + j : cg + 16 * j)] =
            PAIR_R ? (j & 1 ? acc[i][(j / 2) % PJ].y : acc[i][(j / 2) % PJ].x) : acc[i][j % PJ].x + acc[i][j % PJ].y;
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
      const float4 s = C > 1 ? cluster_sum_f4(part + e, C) : *reinterpret_cast<const float4*>(part + e);
      const int t = e / R, c = e % R;
      // columns beyond r stay zero even where a row holds an infinity (0 x inf)
      const float4 ss = c < r ? make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (a.mid && t < m && c < r && (unsigned)(t % C) == rank)
        *reinterpret_cast<float4*>(a.mid + (int64_t)__ldg(a.plan.order + pos0 + t) * r + c) = BWD ? ss : s;
      *reinterpret_cast<float4*>(mid + t * S::MS + c) = ss;
    }
    if (C > 1) cluster_arrive();                            // done with the others' memory
  } else if (a.mid) {
    for (int e = tid; e < m * r; e += kThreads) {           // tokens without an adapter: mid is zero
      const int t = e / r;
      if ((unsigned)(t % C) == rank) a.mid[(int64_t)__ldg(a.plan.order + pos0 + t) * r + e % r] = 0.0f;
    }
  }
  griddep_launch_dependents();

  // ---- out = base + mid w2^T: RM rows x 4 columns per thread, columns cg + 16 j (backward 4 cg + j)
  constexpr int RM = M / 16;
  const int rg = tid / 16, cg = tid % 16;
  int otok[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) otok[i] = RM * rg + i < m ? __ldg(a.plan.order + pos0 + RM * rg + i) : -1;
  for (int step = n1; step < n1 + n2; ++step) {
    const int n0 = kNC * (n_first + step - n1);
    // as above: forward pairs of even and odd contraction indices, backward pairs of columns
    constexpr int PJ = BWD ? 2 : 4;
    float b[RM][4];
    f2 acc[RM][PJ];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + (BWD ? 4 * cg + j : cg + 16 * j);
        b[i][j] = (a.base && otok[i] >= 0 && c < N) ? a.base[(int64_t)otok[i] * N + c] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < PJ; ++j) acc[i][j] = f2_bc(0.0f);
    }
    cp_wait<S::kStages - 2>();
    __syncthreads();                                        // the stage, and at first mid, is complete
    request(step + S::kStages - 1);
    const float* const ws = sm + step % S::kStages * S::kStage;
    if (adapted) {
#pragma unroll 2
      for (int k = 0; k < R; k += 4) {
        float mr[RM][4];
#pragma unroll
        for (int i = 0; i < RM; ++i) lds<4>(mid + (RM * rg + i) * S::MS + k, mr[i]);
        if constexpr (!BWD) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float wr[4];
            lds<4>(ws + (cg + 16 * j) * S::W2S + k, wr);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
              for (int e = 0; e < 4; e += 2)
                acc[i][j % PJ] = f2_fma(f2_mk(mr[i][e], mr[i][e + 1]), f2_mk(wr[e], wr[e + 1]), acc[i][j % PJ]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float wr[4];
            lds<4>(ws + (k + e) * S::W2S + 4 * cg, wr);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
              for (int j = 0; j < PJ; ++j)
                acc[i][j] = f2_fma(f2_bc(mr[i][e]), f2_mk(wr[(2 * j) % 4], wr[(2 * j + 1) % 4]), acc[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      if (otok[i] < 0) continue;
      float* const o = a.out + (int64_t)otok[i] * N + n0;
      if constexpr (BWD) {
        if (n0 + 4 * cg < N)
          *reinterpret_cast<float4*>(o + 4 * cg) = make_float4(b[i][0] + acc[i][0].x, b[i][1] + acc[i][0].y,
                                                               b[i][2] + acc[i][1].x, b[i][3] + acc[i][1].y);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + cg + 16 * j < N) o[cg + 16 * j] = b[i][j] + (acc[i][j % PJ].x + acc[i][j % PJ].y);
      }
    }
  }
  cp_wait<0>();
  if (adapted && C > 1) cluster_wait();                     // the others are done with this CTA's memory
}

// ------------------------------------------------------------------- weight gradients
// One cluster: 64 columns of x (grad_a) or of g (grad_b) over all tokens, its CTAs sharing the
// plan's 64-token tiles evenly (TileShare), as in lora_bf16.cu: tiles through a ring of two
// cp.async stages, an adapter whose tiles lie in several CTAs written by the first of them. A
// thread has 4 columns x RT values of r, of a share of the tile's tokens while r <= 32 (a
// smaller register tile would read shared memory as often as it multiplies); the shares are
// added in order when an adapter is complete.
// K = N = 4096, 4096 tokens of 8 adapters, from cold L2: r = 16 57 us (134 MB: 21 us), r = 64 143 us.
template <int R>
struct WgradF32 {
  static constexpr int kTok = 64, kStages = 2, kOrders = 8;
  static constexpr int RT = R <= 64 ? 4 : 8;                // values of r per thread
  static constexpr int TG = kThreads / (16 * (R / RT));     // token shares
  static constexpr int XS = 64 + 4, WS = R + 4;
  static constexpr int kStage = kTok * (XS + WS);
  static constexpr int SS = 64 + 1;                         // padded row of a share's sums
  static constexpr int kShare = R * SS;
  static constexpr int kPerSM = R == 16 ? 3 : (R <= 64 ? 2 : 1);          // CTAs that fit
  static constexpr size_t smem = sizeof(float) * (size_t)(kStage * kStages + R * 64 + (TG > 1 ? TG * kShare : 0));
};

template <int R>
__global__ void __launch_bounds__(kThreads, WgradF32<R>::kPerSM) k_lora_wgrad_f32(LoraWgrad<float> a, int blocks_b) {
  using S = WgradF32<R>;
  constexpr int RT = S::RT, TG = S::TG, NA = R * 64 / kThreads;
  extern __shared__ __align__(16) float sm[];               // ring
  float* const head = sm + S::kStage * S::kStages;          // [NA][kThreads]
  float* const shares = head + R * 64;                      // [TG][R][SS]
  __shared__ int2 desc[kWindow + 2];
  __shared__ __align__(16) int order[S::kOrders][S::kTok];
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int r = a.r, tid = threadIdx.x, block = blockIdx.x / C;
  const bool is_a = block >= blocks_b;                         // grad_b's blocks first: they start early
  const bool early = starts_early(a.after_rows, is_a);
  if (!early) griddep_wait();
  if (!plan_matches(a.plan)) {
    if (early) griddep_wait();
    return;
  }
  const int n0 = 64 * (is_a ? block - blocks_b : block);
  const int W = is_a ? a.K : a.N;
  const float* const rows = is_a ? a.x : a.g;
  const float* const mid = is_a ? a.v : a.u;
  const int tg = tid / (kThreads / TG), cg = tid % 16, rg = tid % (kThreads / TG) / 16;
  const TileShare share(a.plan, rank, C);
  f2 accp[2][RT];                                           // packed pairs of columns
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) accp[i][j] = f2_bc(0.0f);
  };
  auto acc_at = [&](int i, int j) { return i & 1 ? accp[i / 2][j].y : accp[i / 2][j].x; };
  // The complete sums, four consecutive elements of the gradient (columns for grad_a, r for
  // grad_b) at a time: sum[4 v..] belongs at (rho, c) and after. One share: the register tile as
  // it is. Several: values of all of them, added in order through shared memory.
  float sum[NA];
  auto index = [&](int v, int& rho, int& c) {
    if constexpr (TG == 1) {
      rho = RT * rg + (is_a ? v : v % (RT / 4) * 4);
      c = 4 * cg + (is_a ? 0 : v / (RT / 4));
    } else {
      const int k = tid + kThreads * v;
      rho = is_a ? k / 16 : k % (R / 4) * 4;
      c = is_a ? k % 16 * 4 : k / (R / 4);
    }
  };
  auto collect = [&] {
    if constexpr (TG == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const float v = acc_at(i, j);
          if (is_a) sum[4 * j + i] = v;
          else sum[RT * i + j] = v;
        }
    } else {
      float* const to = shares + tg * S::kShare;
      __syncthreads();                                      // the last sums have been read
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(RT * rg + j) * S::SS + 4 * cg + i] = acc_at(i, j);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NA / 4; ++v) {
        int rho, c;
        index(v, rho, c);
        const float* from = shares + rho * S::SS + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int o = e * (is_a ? 1 : S::SS);
          float t = from[o];
#pragma unroll
          for (int k = 1; k < TG; ++k) t += from[k * S::kShare + o];
          sum[4 * v + e] = t;
        }
      }
    }
  };
  auto scale_of = [&](int ad) { return (!is_a && a.scale) ? __ldg(a.scale + ad) : 1.0f; };
  auto write = [&](int ad, float scale) {
#pragma unroll
    for (int v = 0; v < NA / 4; ++v) {
      int rho, c;
      index(v, rho, c);
      if (rho >= r || n0 + c >= W) continue;                // r and W are multiples of 8: all four or none
      float* const dst = is_a ? a.grad_a + ((int64_t)ad * r + rho) * W + n0 + c
                              : a.grad_b + ((int64_t)ad * W + n0 + c) * r + rho;
      *reinterpret_cast<float4*>(dst) = make_float4(scale * sum[4 * v], scale * sum[4 * v + 1], scale * sum[4 * v + 2],
                                                    scale * sum[4 * v + 3]);
    }
  };

  clear();
  int open = -1;                                            // adapter whose sums go on in the next CTA
  bool from_before = false;                                 // the sum at hand began in an earlier CTA
  for (int w0 = share.lo; w0 < share.hi; w0 += kWindow) {
    const int count = min(kWindow, share.hi - w0);
    __syncthreads();                                        // the last window is consumed
    share.window(a.plan, w0, desc);
    __syncthreads();
    auto request_order = [&](int i) {
      if (i < count && tid < S::kTok) {
        const int pos = desc[i + 1].x + tid;
        const bool in = pos < desc[i + 2].x;
        cp4(shared_at(&order[i % S::kOrders][tid]), in ? a.plan.order + pos : a.plan.order, in);
      }
    };
    auto request = [&](int i) {
      if (i < count) {
        const int tokens = desc[i + 2].x - desc[i + 1].x;
        const int* const ord = order[i % S::kOrders];
        const uint32_t xs = shared_at(sm + i % S::kStages * S::kStage), ws = xs + S::kTok * S::XS * 4;
#pragma unroll
        for (int h = 0; h < S::kTok * 16 / kThreads; ++h) {
          const int e = tid + kThreads * h, t = e / 16, c = n0 + e % 16 * 4;
          const bool in = t < tokens && c < W;
          cp16(xs + (t * S::XS + e % 16 * 4) * 4, in ? rows + (int64_t)ord[t] * W + c : rows, in);
        }
#pragma unroll
        for (int h = 0; h < S::kTok * R / 4 / kThreads; ++h) {
          const int e = tid + kThreads * h, t = e / (R / 4), c = e % (R / 4) * 4;
          const bool in = t < tokens && c < r;
          cp16(ws + (t * S::WS + c) * 4, in ? mid + (int64_t)ord[t] * r + c : mid, in);
        }
      }
    };
    request_order(0);
    request_order(1);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    request(0);
    request_order(2);
    cp_commit();
    if (w0 == share.lo) from_before = desc[0].y == desc[1].y;
    for (int i = 0; i < count; ++i) {
      cp_wait<0>();                                         // rows i and order i + 1 have arrived
      __syncthreads();
      const bool goes_on = desc[i + 2].y == desc[i + 1].y;  // the next tile is the same adapter's
      const bool ends = !goes_on || w0 + i + 1 == share.hi;
      request(i + 1);
      request_order(i + 3);
      cp_commit();
      const int tokens = desc[i + 2].x - desc[i + 1].x, ad = desc[i + 1].y;
      const float* const xs = sm + i % S::kStages * S::kStage;
      const float* const ws = xs + S::kTok * S::XS;
      const int t1 = min(tokens, (tg + 1) * (S::kTok / TG));
#pragma unroll 4
      for (int k = tg * (S::kTok / TG); k < t1; ++k) {
        float xr[4], wr[RT];
        lds<4>(xs + k * S::XS + 4 * cg, xr);
        lds<RT>(ws + k * S::WS + RT * rg, wr);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const f2 w = f2_bc(wr[j]);
          accp[0][j] = f2_fma(f2_mk(xr[0], xr[1]), w, accp[0][j]);
          accp[1][j] = f2_fma(f2_mk(xr[2], xr[3]), w, accp[1][j]);
        }
      }
      if (ends) {
        collect();
        clear();
        if (goes_on && !from_before) {
          open = ad;                                        // its sums stay here
        } else if (from_before) {                           // an earlier CTA writes it
#pragma unroll
          for (int e = 0; e < NA; ++e) head[e * kThreads + tid] = sum[e];
          from_before = false;
        } else {
          write(ad, scale_of(ad));
        }
      }
    }
    cp_wait<0>();
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
        add_from(sum, head, k);
      }
      write(open, scale_of(open));
    }
    cluster_arrive();
  }
#pragma unroll
  for (int e = 0; e < NA; ++e) sum[e] = 0.0f;
  for (int ad = rank; ad < a.plan.n; ad += C)               // adapters without tokens: zeros, whatever their scale holds
    if (__ldg(a.plan.offsets() + ad) == __ldg(a.plan.offsets() + ad + 1)) write(ad, 1.0f);
  if (C > 1) cluster_wait();                                // the others are done with this CTA's memory
  if (early) griddep_wait();
}

template <int R, int M, bool BWD>
cudaError_t run_rows(const LoraRows<float>& a, int64_t tiles, int cluster, cudaStream_t s) {
  constexpr size_t smem = RowsShape<R, M, BWD>::smem;
  const cudaError_t e = allow_smem<k_lora_rows_f32<R, M, BWD>>(smem);
  if (e != cudaSuccess) return e;
  return launch_cluster_pdl(k_lora_rows_f32<R, M, BWD>, dim3((unsigned)(tiles * cluster)), dim3(kThreads), cluster,
                            smem, s, a);
}

template <int R, bool BWD>
cudaError_t rows_m(LoraRows<float> a, const int* plan, int64_t T, int n, cudaStream_t s) {
  const int list = lora_list(T, n);
  a.plan = plan_view(plan, T, n, list);
  const int64_t tiles = plan_layout(T, n).cap[list];
  const int cluster = lora_cluster(tiles, list, true, a.K, a.N);
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
  using S = WgradF32<R>;
  const cudaError_t e = allow_smem<k_lora_wgrad_f32<R>>(S::smem);
  if (e != cudaSuccess) return e;
  const int ka = (a.K + 63) / 64, nb = (a.N + 63) / 64;
  const int ba = a.grad_a ? ka : 0, bb = a.grad_b ? nb : 0;
  // by both widths, so that a gradient does not depend on whether the other is asked for
  const int cluster = lora_token_split(a.plan.T, a.plan.n, ka + nb, S::kTok, S::kPerSM);
  return launch_cluster_pdl(k_lora_wgrad_f32<R>, dim3((unsigned)((ba + bb) * cluster)), dim3(kThreads), cluster,
                            S::smem, s, a, bb);
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

}  // namespace rdfft
