// Low-rank adapters of many requests, bf16: rows kernel (forward, grad_x) and weight
// gradients. fp32 accumulation throughout.
//
// A tile of the plan is up to M tokens of one adapter. One cluster of CTAs computes it in one
// launch: each CTA multiplies its share of the K columns of the tile's rows with its share of
// w1 (mid = in w1^T, r columns), the partial sums are added over the cluster through
// distributed shared memory in rank order, and each CTA then expands mid to its share of the N
// output columns (out = base + scale mid w2^T). So every row is read once and written once,
// and A and B once per tile; the sums do not depend on timing.
//
// The products run on mma.m16n8k16 with operand fragments loaded straight from global memory:
// the contraction index may be taken in any order as long as both operands agree, so a lane
// takes 16 consecutive bytes of a row where the instruction's layout would scatter them. With
// r <= 128 the work is 2 r flops per byte of a row at most, and the rows, not the tensor
// pipe, set the time; tensor memory would only add a trip for a result of r columns.
#include "lora.cuh"

#include "many_policy.h"

namespace rdfft {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const bf16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// N consecutive 32-bit words (N = 1, 2, 4, 8) through the read-only path.
template <int N>
__device__ __forceinline__ void ldg_words(const bf16_t* p, uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (N == 2) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = t.x, v[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 t = ldg16(p + 8 * i);
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  }
}

// Element j of the vectors lo and hi (rows k and k + 1 of a row-major operand), as the pair
// that an operand with consecutive contraction indices holds.
template <int N>
__device__ __forceinline__ uint32_t pair_of(const uint32_t (&lo)[N], const uint32_t (&hi)[N], int j) {
  return __byte_perm(lo[j / 2], hi[j / 2], (j & 1) ? 0x7632 : 0x5410);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Row stride, in elements, of mid in shared memory: 8-byte reads of 8 rows x 4 lanes are then
// free of bank conflicts (32-byte rows are so already).
template <int R>
constexpr int mid_stride() { return R == 16 ? 16 : R + 16; }

template <int R, int M>
constexpr size_t rows_smem() {
  constexpr int MT = M == 16 ? 1 : (R <= 32 ? 4 : 128 / R);
  constexpr int WK = kWarps / (M / (16 * MT));
  return sizeof(float) * WK * M * R + 2 * sizeof(bf16_t) * M * mid_stride<R>();
}

// R: r rounded up to 16, 32, 64 or 128. M: tokens per tile, 16 or 64 (the plan's list).
template <int R, int M, bool BWD>
__global__ void __launch_bounds__(kThreads) k_lora_rows(LoraRows<bf16_t> a) {
  constexpr int MT = M == 16 ? 1 : (R <= 32 ? 4 : 128 / R);   // 16-row tiles per warp: 64 accumulators at most
  constexpr int WM = M / (16 * MT), WK = kWarps / WM;          // row groups x shares of K
  constexpr int NJ = R / 8;
  constexpr int V = R / 8;                                     // r values per lane of a w1 row, backward
  constexpr int MS = mid_stride<R>();
  extern __shared__ __align__(16) float part[];                // [WK][M][R]
  bf16_t* const mid_hi = reinterpret_cast<bf16_t*>(part + WK * M * R);
  bf16_t* const mid_lo = mid_hi + M * MS;

  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int tile = blockIdx.x / C;
  const int2 te = __ldg(a.plan.tiles + tile);                  // within the list's capacity
  if (tile >= __ldg(a.plan.header + 2 + a.plan.list)) return;  // the whole cluster leaves
  const int pos0 = te.x, ad = te.y;
  const int m = min(__ldg(a.plan.offsets + ad + 1) - pos0, M);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int K = a.K, N = a.N, r = a.r;
  const bool adapted = ad < a.plan.n;

  if (adapted) {
    // ---- mid = in w1^T over this CTA's units of 32 columns
    const int wm = warp % WM, wk = warp / WM;
    const int units = (K + 31) / 32;
    const int u0 = (int)((int64_t)units * rank / C), u1 = (int)((int64_t)units * (rank + 1) / C);
    const bf16_t* row[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = (wm * MT + i) * 16 + g + 8 * h;
        row[i][h] = t < m ? a.in + (int64_t)__ldg(a.plan.order + pos0 + t) * K : nullptr;
      }
    const bf16_t* const w1 = a.w1 + (int64_t)ad * r * K;
    float acc[MT][NJ][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;

    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int u = u0 + wk; u < u1; u += WK) {
      const int k0 = 32 * u + 8 * q;                           // this lane's 8 columns
      const bool in = k0 < K;
      uint4 xa[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[i][h] = (in && row[i][h]) ? ldg16(row[i][h] + k0) : zero;
      if constexpr (!BWD) {
        // w1 row 8 j + g, the same 8 columns
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int rho = 8 * j + g;
          const uint4 wb = (in && rho < r) ? ldg16(w1 + (int64_t)rho * K + k0) : zero;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            mma16816(acc[i][j], xa[i][0].x, xa[i][1].x, xa[i][0].y, xa[i][1].y, wb.x, wb.y);
            mma16816(acc[i][j], xa[i][0].z, xa[i][1].z, xa[i][0].w, xa[i][1].w, wb.z, wb.w);
          }
        }
      } else {
        // w1 is read where B lies: column k0 + e of w1 is row k0 + e of B, r values of which
        // this lane takes V, so tile j holds the r index V g + j at its column g
        uint32_t wr[8][V / 2];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int x = 0; x < V / 2; ++x) wr[e][x] = 0;
          if (in) {
            if constexpr (V <= 8) {
              if (V * g < r) ldg_words<V / 2>(w1 + (int64_t)(k0 + e) * r + V * g, wr[e]);
            } else {
#pragma unroll
              for (int hv = 0; hv < 2; ++hv) {
                uint32_t t[4] = {0, 0, 0, 0};
                if (V * g + 8 * hv < r) ldg_words<4>(w1 + (int64_t)(k0 + e) * r + V * g + 8 * hv, t);
#pragma unroll
                for (int x = 0; x < 4; ++x) wr[e][4 * hv + x] = t[x];
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            mma16816(acc[i][j], xa[i][0].x, xa[i][1].x, xa[i][0].y, xa[i][1].y, pair_of(wr[0], wr[1], j),
                     pair_of(wr[2], wr[3], j));
            mma16816(acc[i][j], xa[i][0].z, xa[i][1].z, xa[i][0].w, xa[i][1].w, pair_of(wr[4], wr[5], j),
                     pair_of(wr[6], wr[7], j));
          }
      }
    }
    // the column of tile j that a lane holds is 2 q + e
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = (wm * MT + i) * 16 + g + 8 * (e / 2), c = 2 * q + (e & 1);
          part[(wk * M + t) * R + (BWD ? V * c + j : 8 * j + c)] = acc[i][j][e];
        }
    __syncthreads();
    // this CTA's sum, in place of the first share
    for (int e = 4 * threadIdx.x; e < M * R; e += 4 * kThreads) {
      float4 s = *reinterpret_cast<float4*>(part + e);
#pragma unroll
      for (int k = 1; k < WK; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(part + k * M * R + e);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      *reinterpret_cast<float4*>(part + e) = s;
    }
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // the cluster's sum in rank order, every CTA for itself; mid is scaled and kept as the sum
    // of two bf16, hi + lo (16 mantissa bits), so its rounding stays far below the output's
    const float scale = a.scale ? __ldg(a.scale + ad) : 1.0f;
    for (int e = 4 * threadIdx.x; e < M * R; e += 4 * kThreads) {
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
      const float4 ss = c < r ? make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (a.mid && t < m && c < r && (unsigned)(t % C) == rank) {
        float* dst = a.mid + (int64_t)__ldg(a.plan.order + pos0 + t) * r + c;
        *reinterpret_cast<float4*>(dst) = BWD ? ss : s;
      }
      const uint32_t h0 = pack2(ss.x, ss.y), h1 = pack2(ss.z, ss.w);
      *reinterpret_cast<uint2*>(mid_hi + t * MS + c) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(mid_lo + t * MS + c) =
          make_uint2(pack2(ss.x - lo_f32(h0), ss.y - hi_f32(h0)), pack2(ss.z - lo_f32(h1), ss.w - hi_f32(h1)));
    }
    if (C > 1) cluster_arrive();                               // done with the others' memory
    __syncthreads();
  } else if (a.mid) {
    // tokens without an adapter: mid is zero
    for (int e = threadIdx.x; e < m * r; e += kThreads) {
      const int t = e / r;
      if ((unsigned)(t % C) == rank) a.mid[(int64_t)__ldg(a.plan.order + pos0 + t) * r + e % r] = 0.0f;
    }
  }
  griddep_launch_dependents();

  // ---- out = base + mid w2^T over this CTA's groups of 64 columns
  if (a.out != nullptr && (adapted || a.base != a.out)) {
    constexpr int MT2 = M == 16 ? 1 : 2;
    constexpr int RG = M / (16 * MT2);                         // row groups; the other warps take columns
    const int rg = warp % RG, cw = warp / RG;
    const int groups = (N + 63) / 64;
    const int g0 = (int)((int64_t)groups * rank / C), g1 = (int)((int64_t)groups * (rank + 1) / C);
    const bf16_t* const w2 = a.w2 + (int64_t)(adapted ? ad : 0) * r * N;
    int64_t orow[MT2][2];
#pragma unroll
    for (int i = 0; i < MT2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = (rg * MT2 + i) * 16 + g + 8 * h;
        orow[i][h] = t < m ? (int64_t)__ldg(a.plan.order + pos0 + t) * N : -1;
      }
    for (int gr = g0 + cw; gr < g1; gr += kWarps / RG) {
      const int n0 = 64 * gr;
      // a lane ends with two runs of 8 columns of each of its rows: 8 (2 q + run) + [0, 8)
      uint4 bs[MT2][2][2];
#pragma unroll
      for (int i = 0; i < MT2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int run = 0; run < 2; ++run) {
            const int c = n0 + 16 * q + 8 * run;
            bs[i][h][run] = make_uint4(0, 0, 0, 0);
            if (a.base && orow[i][h] >= 0 && c < N)
              bs[i][h][run] = *reinterpret_cast<const uint4*>(a.base + orow[i][h] + c);
          }
      float acc[MT2][8][4];
#pragma unroll
      for (int i = 0; i < MT2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
      if (adapted) {
        const int col = n0 + 8 * g;                            // tile j's column g is output column col + j
#pragma unroll
        for (int s = 0; s < R / 16; ++s) {
          const int rho = 16 * s + 4 * q;                      // this lane's 4 contraction indices
          uint32_t b0[8], b1[8];
          if constexpr (!BWD) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t t[2] = {0, 0};
              if (col < N && rho < r) ldg_words<2>(w2 + (int64_t)(col + j) * r + rho, t);
              b0[j] = t[0], b1[j] = t[1];
            }
          } else {
            uint32_t wr[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
              for (int x = 0; x < 4; ++x) wr[e][x] = 0;
              if (col < N && rho < r) ldg_words<4>(w2 + (int64_t)(rho + e) * N + col, wr[e]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) b0[j] = pair_of(wr[0], wr[1], j), b1[j] = pair_of(wr[2], wr[3], j);
          }
#pragma unroll
          for (int i = 0; i < MT2; ++i) {
            const int t = (rg * MT2 + i) * 16 + g;
            const uint2 h0 = *reinterpret_cast<const uint2*>(mid_hi + t * MS + rho);
            const uint2 h1 = *reinterpret_cast<const uint2*>(mid_hi + (t + 8) * MS + rho);
            const uint2 l0 = *reinterpret_cast<const uint2*>(mid_lo + t * MS + rho);
            const uint2 l1 = *reinterpret_cast<const uint2*>(mid_lo + (t + 8) * MS + rho);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              mma16816(acc[i][j], h0.x, h1.x, h0.y, h1.y, b0[j], b1[j]);
              mma16816(acc[i][j], l0.x, l1.x, l0.y, l1.y, b0[j], b1[j]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int run = 0; run < 2; ++run) {
            const int c = n0 + 16 * q + 8 * run;
            if (orow[i][h] < 0 || c >= N) continue;
            const uint32_t b[4] = {bs[i][h][run].x, bs[i][h][run].y, bs[i][h][run].z, bs[i][h][run].w};
            uint32_t o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              o[x] = pack2(acc[i][2 * x][2 * h + run] + lo_f32(b[x]), acc[i][2 * x + 1][2 * h + run] + hi_f32(b[x]));
            *reinterpret_cast<uint4*>(a.out + orow[i][h] + c) = make_uint4(o[0], o[1], o[2], o[3]);
          }
    }
  }
  if (adapted && C > 1) cluster_wait();                        // the others are done with this CTA's memory
}

// ------------------------------------------------------------------- weight gradients
// One CTA: 64 columns of x (grad_a) or of g (grad_b) over all tokens of one adapter. D[rho,
// column] = sum_t mid[t, rho] row[t, column]: tokens are the contraction index, so the rows'
// fragments are pairs of tokens, built from 16-byte pieces of four rows. The 8 warps share
// the tokens (and, from r > 32 on, the rho range) and add their sums in a fixed order.
// mid is fp32; it enters the product as three bf16 summing to it exactly in all but the last
// bits (24 mantissa bits), since the gradients are fp32.
template <int R>
__global__ void __launch_bounds__(kThreads) k_lora_wgrad(LoraWgrad<bf16_t> a, int blocks_a) {
  constexpr int MT = R == 16 ? 1 : 2;                          // 16-row tiles of rho per warp
  constexpr int WR = R / (16 * MT), WT = kWarps / WR;          // rho groups x shares of the tokens
  extern __shared__ __align__(16) float part[];                // [WT][R][64]
  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const int ad = blockIdx.y, r = a.r;
  const bool is_a = (int)blockIdx.x < blocks_a;
  const int n0 = 64 * (is_a ? blockIdx.x : blockIdx.x - blocks_a);
  const int W = is_a ? a.K : a.N;                              // columns of the rows read
  const bf16_t* const rows = is_a ? a.x : a.g;
  const float* const mid = is_a ? a.v : a.u;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int wr = warp % WR, wt = warp / WR;
  const int beg = __ldg(a.plan.offsets + ad), end = __ldg(a.plan.offsets + ad + 1);
  const int col = n0 + 8 * g;

  float acc[MT][8][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
#pragma unroll 2
  for (int p0 = beg + 16 * wt; p0 < end; p0 += 16 * WT) {
    int64_t tok[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int pos = p0 + 4 * q + e;
      tok[e] = pos < end ? __ldg(a.plan.order + pos) : -1;
    }
    uint32_t w[4][4];
    float mv[MT][2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int x = 0; x < 4; ++x) w[e][x] = 0;
      if (tok[e] >= 0 && col < W) ldg_words<4>(rows + tok[e] * W + col, w[e]);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rho = (wr * MT + i) * 16 + g + 8 * h;
          mv[i][h][e] = (tok[e] >= 0 && rho < r) ? __ldg(mid + tok[e] * r + rho) : 0.0f;
        }
    }
    uint32_t b0[8], b1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b0[j] = pair_of(w[0], w[1], j), b1[j] = pair_of(w[2], w[3], j);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        uint32_t f[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float &v0 = mv[i][h][2 * x], &v1 = mv[i][h][2 * x + 1];
            f[h][x] = pack2(v0, v1);
            v0 -= lo_f32(f[h][x]);
            v1 -= hi_f32(f[h][x]);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16816(acc[i][j], f[0][0], f[1][0], f[0][1], f[1][1], b0[j], b1[j]);
      }
  }
  griddep_launch_dependents();
  // [rho][column] sums of each share, then their sum; column 8 (2 q + e) + j of the group
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* dst = part + ((wt * R + (wr * MT + i) * 16 + g + 8 * h) * 64 + 16 * q + 8 * e);
        *reinterpret_cast<float4*>(dst) =
            make_float4(acc[i][0][2 * h + e], acc[i][1][2 * h + e], acc[i][2][2 * h + e], acc[i][3][2 * h + e]);
        *reinterpret_cast<float4*>(dst + 4) =
            make_float4(acc[i][4][2 * h + e], acc[i][5][2 * h + e], acc[i][6][2 * h + e], acc[i][7][2 * h + e]);
      }
  __syncthreads();
  const float scale = (!is_a && a.scale) ? __ldg(a.scale + ad) : 1.0f;
  for (int e = threadIdx.x; e < R * 64; e += kThreads) {
    // grad_a is written along the columns, grad_b along rho
    const int rho = is_a ? e / 64 : e % R, c = is_a ? e % 64 : e / R;
    if (rho >= r || n0 + c >= W) continue;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < WT; ++k) s += part[(k * R + rho) * 64 + c];
    if (is_a)
      a.grad_a[((int64_t)ad * r + rho) * W + n0 + c] = s;
    else
      a.grad_b[((int64_t)ad * W + n0 + c) * r + rho] = scale * s;
  }
}

template <typename KernelT>
cudaError_t set_smem(KernelT kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int R, int M, bool BWD>
cudaError_t run_rows(const LoraRows<bf16_t>& a, int64_t tiles, int cluster, cudaStream_t s) {
  constexpr size_t smem = rows_smem<R, M>();
  const cudaError_t e = set_smem(k_lora_rows<R, M, BWD>, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster_pdl(k_lora_rows<R, M, BWD>, dim3((unsigned)(tiles * cluster)), dim3(kThreads), cluster, smem, s, a);
}

template <int R, bool BWD>
cudaError_t rows_m(LoraRows<bf16_t> a, const int* plan, int64_t T, int n, cudaStream_t s) {
  const int list = lora_list(T, n);
  a.plan = plan_view(plan, T, n, list);
  const int64_t tiles = plan_layout(T, n).cap[list];
  const int cluster = lora_cluster(tiles, a.K, a.N);
  if (list == 1) return run_rows<R, 16, BWD>(a, tiles, cluster, s);
  return run_rows<R, 64, BWD>(a, tiles, cluster, s);
}

template <int R>
cudaError_t run_wgrad(const LoraWgrad<bf16_t>& a, cudaStream_t s) {
  constexpr int MT = R == 16 ? 1 : 2;
  constexpr size_t smem = sizeof(float) * 64 * R * (kWarps / (R / (16 * MT)));
  const cudaError_t e = set_smem(k_lora_wgrad<R>, smem);
  if (e != cudaSuccess) return e;
  const int ba = a.grad_a ? (a.K + 63) / 64 : 0, bb = a.grad_b ? (a.N + 63) / 64 : 0;
  return launch_pdl(k_lora_wgrad<R>, dim3((unsigned)(ba + bb), (unsigned)a.plan.n), dim3(kThreads), smem, s, a, ba);
}

template <bool BWD>
cudaError_t rows_r(const LoraRows<bf16_t>& a, const int* plan, int64_t T, int n, cudaStream_t s) {
  if (a.r <= 16) return rows_m<16, BWD>(a, plan, T, n, s);
  if (a.r <= 32) return rows_m<32, BWD>(a, plan, T, n, s);
  if (a.r <= 64) return rows_m<64, BWD>(a, plan, T, n, s);
  return rows_m<128, BWD>(a, plan, T, n, s);
}

}  // namespace

cudaError_t lora_rows_bf16(const LoraRows<bf16_t>& a, bool bwd, const int* plan, int64_t T, int n, cudaStream_t s) {
  return bwd ? rows_r<true>(a, plan, T, n, s) : rows_r<false>(a, plan, T, n, s);
}

cudaError_t lora_wgrad_bf16(const LoraWgrad<bf16_t>& a, cudaStream_t s) {
  if (a.r <= 16) return run_wgrad<16>(a, s);
  if (a.r <= 32) return run_wgrad<32>(a, s);
  if (a.r <= 64) return run_wgrad<64>(a, s);
  return run_wgrad<128>(a, s);
}

cudaError_t take_lora_bf16_error(unsigned int* flags) { return take_error_word(flags); }

}  // namespace rdfft
