// Low-rank adapters of many requests, bf16: rows kernels (forward, grad_x) and weight
// gradients. fp32 accumulation throughout.
//
// A tile of the plan is up to 16 or 64 tokens of one adapter. One cluster of CTAs computes it
// in one launch: each CTA multiplies its share of the K columns of the tile's rows with its
// share of w1 (mid = in w1^T, r columns), the partial sums are added over the cluster through
// distributed shared memory in rank order, and each CTA then expands mid to its share of the N
// output columns (out = base + scale mid w2^T). So every row is read once and written once,
// and A and B once per tile; the sums do not depend on timing.
//
// The products run on mma.m16n8k16. With r <= 128 the work is 2 r flops per byte of a row at
// most, and the rows, not the tensor pipe, set the time; tensor memory would only add a trip
// for a result of r columns.
//  * k_lora_rows16 (decode, small groups): operand fragments straight from global memory. The
//    contraction index may be taken in any order as long as both operands agree, so a lane
//    takes 16 consecutive bytes of a row where the instruction's layout would scatter them.
//    No staging and one barrier before the cluster's: few tokens are a matter of latency
//    (K = N = 4096, r = 16, 32 tokens of 16 adapters from cold L2: 7.5 us, five dependent loads
//    and two cluster barriers; 5 MB would take 0.8).
//  * k_lora_rows64: steps of 64 or 128 columns of rows and weights through a ring of cp.async
//    stages, the second half's steps (base, w2) requested while the cluster adds up the first
//    half's (K = N = 4096, r = 16, 4096 tokens of 8 adapters: 21.6 us, 4.8 TB/s of the 103 MB;
//    with fragments straight from global memory, as above, 39: eight warps of 142 registers per
//    SM kept too little in flight; r = 64: 38 us).
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

// The additions inside mma truncate: a sum left in its accumulator loses up to a step (2^-23) at
// each of them, always towards zero (262144 tokens of one adapter: gradients 2e-4 too small). So an
// accumulator takes the products of one step of a loop only (4 to 12 mma), and the steps' sums
// are added by FADD, rounded to nearest.
__device__ __forceinline__ void add4(float (&acc)[4], const float (&d)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] += d[e];
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

template <int R>
constexpr size_t rows16_smem() {
  return sizeof(float) * kWarps * 16 * R + 2 * sizeof(bf16_t) * 16 * mid_stride<R>();
}

// R: r rounded up to 16, 32, 64 or 128.
template <int R, bool BWD>
__global__ void __launch_bounds__(kThreads, R <= 64 ? 2 : 1) k_lora_rows16(LoraRows<bf16_t> a) {
  constexpr int M = 16, WK = kWarps;                           // the warps share the K columns
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
  const int m = min(__ldg(a.plan.offsets() + ad + 1) - pos0, M);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int K = a.K, N = a.N, r = a.r;
  const bool adapted = ad < a.plan.n;

  // the output's rows, columns and first base values: requested early, used in the second half
  const int groups = (N + 63) / 64;
  const int gr0 = (int)((int64_t)groups * rank / C) + warp, g1 = (int)((int64_t)groups * (rank + 1) / C);
  int tok[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) tok[h] = g + 8 * h < m ? __ldg(a.plan.order + pos0 + g + 8 * h) : -1;
  // a lane holds two runs of 8 columns of each of its rows: 8 (2 q + run) + [0, 8)
  uint4 next[2][2];
  auto load_base = [&](int gr) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int run = 0; run < 2; ++run) {
        const int c = 64 * gr + 16 * q + 8 * run;
        next[h][run] = make_uint4(0, 0, 0, 0);
        if (a.base && tok[h] >= 0 && c < N)
          next[h][run] = *reinterpret_cast<const uint4*>(a.base + (int64_t)tok[h] * N + c);
      }
  };

  if (adapted) {
    // ---- mid = in w1^T over this CTA's units of 32 columns
    const int units = (K + 31) / 32;
    const int u0 = (int)((int64_t)units * rank / C), u1 = (int)((int64_t)units * (rank + 1) / C);
    const bf16_t* const row0 = a.in + (int64_t)tok[0] * K;
    const bf16_t* const row1 = a.in + (int64_t)tok[1] * K;
    const bf16_t* const w1 = a.w1 + (int64_t)ad * r * K;
    // in runs of kRun units (2 kRun mma), each run's sums added to this warp's in shared memory
    constexpr int kRun = 4;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int u = u0 + warp;
    for (bool first = true; first || u < u1; first = false) {
      float acc[NJ][4];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
      const int end = min(u1, u + kRun * WK);
#pragma unroll (R <= 32 ? 2 : 1)
      for (; u < end; u += WK) {
        const int k0 = 32 * u + 8 * q;                         // this lane's 8 columns
        const bool in = k0 < K;
        const uint4 x0 = (in && tok[0] >= 0) ? ldg16(row0 + k0) : zero;
        const uint4 x1 = (in && tok[1] >= 0) ? ldg16(row1 + k0) : zero;
        if constexpr (!BWD) {
          // w1 row 8 j + g, the same 8 columns
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int rho = 8 * j + g;
            const uint4 wb = (in && rho < r) ? ldg16(w1 + (int64_t)rho * K + k0) : zero;
            mma16816(acc[j], x0.x, x1.x, x0.y, x1.y, wb.x, wb.y);
            mma16816(acc[j], x0.z, x1.z, x0.w, x1.w, wb.z, wb.w);
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
          for (int j = 0; j < NJ; ++j) {
            mma16816(acc[j], x0.x, x1.x, x0.y, x1.y, pair_of(wr[0], wr[1], j), pair_of(wr[2], wr[3], j));
            mma16816(acc[j], x0.z, x1.z, x0.w, x1.w, pair_of(wr[4], wr[5], j), pair_of(wr[6], wr[7], j));
          }
        }
      }
      // the column of tile j that a lane holds is 2 q + e
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = g + 8 * (e / 2), c = 2 * q + (e & 1);
          float& sum = part[(warp * M + t) * R + (BWD ? V * c + j : 8 * j + c)];
          sum = first ? acc[j][e] : sum + acc[j][e];
        }
    }
    if (gr0 < g1) load_base(gr0);
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
      const float4 s = C > 1 ? cluster_sum_f4(part + e, C) : *reinterpret_cast<const float4*>(part + e);
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
  } else {
    if (gr0 < g1) load_base(gr0);
    for (int e = threadIdx.x; a.mid != nullptr && e < m * r; e += kThreads) {   // mid is zero
      const int t = e / r;
      if ((unsigned)(t % C) == rank) a.mid[(int64_t)__ldg(a.plan.order + pos0 + t) * r + e % r] = 0.0f;
    }
  }
  griddep_launch_dependents();

  // ---- out = base + mid w2^T over this CTA's groups of 64 columns
  if (a.out != nullptr && (adapted || a.base != a.out)) {
    const bf16_t* const w2 = a.w2 + (int64_t)(adapted ? ad : 0) * r * N;
    for (int gr = gr0; gr < g1; gr += kWarps) {
      const int n0 = 64 * gr;
      uint4 bs[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int run = 0; run < 2; ++run) bs[h][run] = next[h][run];
      if (gr + kWarps < g1) load_base(gr + kWarps);
      float acc[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
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
          const uint2 h0 = *reinterpret_cast<const uint2*>(mid_hi + g * MS + rho);
          const uint2 h1 = *reinterpret_cast<const uint2*>(mid_hi + (g + 8) * MS + rho);
          const uint2 l0 = *reinterpret_cast<const uint2*>(mid_lo + g * MS + rho);
          const uint2 l1 = *reinterpret_cast<const uint2*>(mid_lo + (g + 8) * MS + rho);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mma16816(acc[j], h0.x, h1.x, h0.y, h1.y, b0[j], b1[j]);
            mma16816(acc[j], l0.x, l1.x, l0.y, l1.y, b0[j], b1[j]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int run = 0; run < 2; ++run) {
          const int c = n0 + 16 * q + 8 * run;
          if (tok[h] < 0 || c >= N) continue;
          const uint32_t b[4] = {bs[h][run].x, bs[h][run].y, bs[h][run].z, bs[h][run].w};
          uint32_t o[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            o[x] = pack2(acc[2 * x][2 * h + run] + lo_f32(b[x]), acc[2 * x + 1][2 * h + run] + hi_f32(b[x]));
          *reinterpret_cast<uint4*>(a.out + (int64_t)tok[h] * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
  }
  if (adapted && C > 1) cluster_wait();                        // the others are done with this CTA's memory
}

// ----------------------------------------------------------------- tiles and fragments
__device__ __forceinline__ void ldsm4(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// Four 8 x 8 matrices to shared memory, held as ldsm4 loads them.
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// Byte offset of 16-byte unit `unit` of row `row` in a tile of W bf16 columns. The units of a
// row are permuted by the row so that 8 rows' units of one column fall into different banks.
// Moving by 16 rows adds 32 W; moving by an even number u of units from an even unit, or from
// the odd one after it, flips 16 u in the offset.
template <int W>
__device__ __forceinline__ uint32_t at(int row, int unit) {
  const int f = W == 16 ? (row >> 2) & 1 : (W == 32 ? (row >> 1) & 3 : row & 7);
  return row * 2 * W + 16 * (unit ^ f);
}

// Fragments from a tile of W columns: 16 rows from row0, 16 columns from col0 (multiples of 16).
// A lane's address is an offset worked out once (lane_rows or lane_cols) moved to (row0, col0).
// As ldsm4 gives them, lane_rows yields an A fragment whose rows are the tile's rows or, loaded
// transposed, {b0, b1} of B columns col0..+7 and col0 + 8..+15 with the contraction index down the
// rows; lane_cols yields {b0, b1} of B columns row0..+7 and row0 + 8..+15 that are the tile's rows
// or, loaded transposed, an A fragment with the contraction index down the rows.
template <int W>
__device__ __forceinline__ uint32_t lane_rows(int lane) { return at<W>((lane / 8 & 1) * 8 + lane % 8, lane / 16); }
template <int W>
__device__ __forceinline__ uint32_t lane_cols(int lane) { return at<W>(lane / 16 * 8 + lane % 8, lane / 8 & 1); }
template <int W>
__device__ __forceinline__ uint32_t moved(uint32_t offset, int row0, int col0) {
  return (offset ^ (2 * col0)) + row0 * 2 * W;
}

// ----------------------------------------------------------------- rows, 64-token tiles
template <int R>
struct Rows64 {
  static constexpr int kCols = R <= 32 ? 128 : 64;           // columns per step
  static constexpr int kRowBytes = 64 * kCols * 2;           // 64 rows of in or base
  static constexpr int kStage = kRowBytes + kCols * R * 2;   // and those columns of w1 or w2
  static constexpr int kStages = R == 64 ? 4 : 3;
  static constexpr size_t smem = (size_t)kStage * kStages + sizeof(float) * 2 * 64 * R + 2 * 64 * R * sizeof(bf16_t);
};

template <int R, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) k_lora_rows64(LoraRows<bf16_t> a) {
  using S = Rows64<R>;
  constexpr int M = 64, COLS = S::kCols, UNITS = COLS / 8, ROWS = kThreads / UNITS, NH = M / ROWS;
  extern __shared__ __align__(128) unsigned char ring[];
  float* const part = reinterpret_cast<float*>(ring + S::kStage * S::kStages);     // [2][M][R]
  const uint32_t ring_at = shared_at(ring);
  const uint32_t hi_at = shared_at(part + 2 * M * R), lo_at = hi_at + M * R * 2;   // mid, tiles of R columns
  unsigned char* const mid_hi = reinterpret_cast<unsigned char*>(part + 2 * M * R);
  unsigned char* const mid_lo = mid_hi + M * R * 2;

  griddep_wait();
  if (!plan_matches(a.plan)) return;
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int tile = blockIdx.x / C;
  const int2 te = __ldg(a.plan.tiles + tile);                  // within the list's capacity
  if (tile >= __ldg(a.plan.header + 2 + a.plan.list)) return;  // the whole cluster leaves
  const int pos0 = te.x, ad = te.y;
  const int m = min(__ldg(a.plan.offsets() + ad + 1) - pos0, M);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int K = a.K, N = a.N, r = a.r;
  const bool adapted = ad < a.plan.n;

  // this CTA's steps of COLS columns, every C-th (the cluster reads a row's columns side by side):
  // [0, n1) of in and w1, then [n1, n1 + n2) of base and w2
  const int ks = (K + COLS - 1) / COLS, ns = (N + COLS - 1) / COLS;
  const auto mine = [&](int all) { return (all - (int)rank + (int)C - 1) / (int)C; };
  const int n1 = adapted ? mine(ks) : 0;
  const int n2 = (a.out != nullptr && (adapted || a.base != a.out)) ? mine(ns) : 0;
  const bf16_t* const w1 = a.w1 + (adapted ? (int64_t)ad * r * K : 0);
  const bf16_t* const w2 = a.w2 + (adapted ? (int64_t)ad * r * N : 0);
  // A thread moves one unit of every ROWS-th row of a row tile, and WL units of a weight tile:
  // r rows of COLS columns (w1 forward, w2 backward), or COLS rows of r columns. Its addresses go
  // from step to step by a fixed distance. Rows beyond the tile's tokens are left as they are:
  // they reach only their own rows of the products, which nobody stores.
  constexpr int WL = (UNITS * R + kThreads - 1) / kThreads;
  const int trow = tid / UNITS, tunit = tid % UNITS;
  int tok[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) tok[h] = trow + ROWS * h < m ? __ldg(a.plan.order + pos0 + trow + ROWS * h) : -1;
  const uint32_t x_dst = ring_at + at<COLS>(trow, tunit);
  const bf16_t *px[NH], *pw[WL];
  uint32_t w_dst[WL];
  int64_t w_go;                                                // per step, in elements
  int rcol, wcol[WL];                                          // columns the next request begins with
  bool w_in[WL];
  int rstep = 0, rslot = 0, RW;
  auto aim = [&](bool first) {                                 // at the first step of a half
    const bf16_t* const rows = first || a.base == nullptr ? a.in : a.base;
    const bf16_t* const w = first ? w1 : w2;
    const bool along = first != BWD;
    RW = first ? K : N;
    rcol = COLS * (int)rank + 8 * tunit;
#pragma unroll
    for (int h = 0; h < NH; ++h) px[h] = rows + (int64_t)max(tok[h], 0) * RW + rcol;
    w_go = (int64_t)COLS * C * (along ? 1 : r);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int e = tid + kThreads * i;
      const int rho = along ? e / UNITS : e % (R / 8) * 8, c = along ? e % UNITS * 8 : e / (R / 8);
      wcol[i] = COLS * (int)rank + c;
      w_in[i] = rho < r;
      pw[i] = along ? w + (int64_t)rho * RW + wcol[i] : w + (int64_t)wcol[i] * r + rho;
      w_dst[i] = ring_at + S::kRowBytes + (along ? at<COLS>(rho, c / 8) : at<R>(c, rho / 8));
    }
  };
  auto request = [&] {
    if (rstep < n1 + n2) {
      if (rstep == n1) aim(false);
      const uint32_t slot = rslot * S::kStage;
      if (rstep < n1 || a.base != nullptr) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (tok[h] >= 0) cp16(x_dst + slot + h * ROWS * COLS * 2, rcol < RW ? px[h] : a.in, rcol < RW);
          px[h] += COLS * C;
        }
      }
      if (adapted) {
#pragma unroll
        for (int i = 0; i < WL; ++i) {
          const bool in = w_in[i] && wcol[i] < RW;
          if (UNITS * R >= kThreads || tid < UNITS * R) cp16(w_dst[i] + slot, in ? pw[i] : a.w1, in);
          pw[i] += w_go;
          wcol[i] += COLS * C;
        }
      }
      rcol += COLS * C;
      ++rstep;
      rslot = rslot + 1 == S::kStages ? 0 : rslot + 1;
    }
    cp_commit();
  };
  if (n1 > 0) aim(true);
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) request();

  const int wm = warp % 4, wh = warp / 4;                      // 16 rows; half of a step's columns
  // fragment offsets: rows of in or base; w1; mid; w2
  const uint32_t x_off = moved<COLS>(lane_rows<COLS>(lane), 16 * wm, 0);
  const uint32_t w1_off = BWD ? lane_rows<R>(lane) : lane_cols<COLS>(lane);
  const uint32_t mid_off = moved<R>(lane_rows<R>(lane), 16 * wm, 0);
  const uint32_t w2_off = BWD ? lane_rows<COLS>(lane) : lane_cols<R>(lane);
  int slot = 0;                                                // stage of the step at hand
  if (adapted) {
    float acc[R / 8][4];
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    for (int step = 0; step < n1; ++step) {
      cp_wait<S::kStages - 2>();
      __syncthreads();
      request();
      const uint32_t x_at = ring_at + slot * S::kStage, w_at = x_at + S::kRowBytes;
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      uint32_t x[COLS / 32][4];
#pragma unroll
      for (int s = 0; s < COLS / 32; ++s) ldsm4(x[s], x_at + moved<COLS>(x_off, 0, COLS / 2 * wh + 16 * s));
#pragma unroll
      for (int j = 0; j < R / 16; ++j) {
        float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // this step's sums
#pragma unroll
        for (int s = 0; s < COLS / 32; ++s) {
          const int k = COLS / 2 * wh + 16 * s;
          uint32_t w[4];
          if constexpr (!BWD) ldsm4(w, w_at + moved<COLS>(w1_off, 16 * j, k));
          else ldsm4t(w, w_at + moved<R>(w1_off, k, 16 * j));
          mma16816(d0, x[s][0], x[s][1], x[s][2], x[s][3], w[0], w[1]);
          mma16816(d1, x[s][0], x[s][1], x[s][2], x[s][3], w[2], w[3]);
        }
        add4(acc[2 * j], d0);
        add4(acc[2 * j + 1], d1);
      }
    }
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(part + (wh * M + 16 * wm + g + 8 * h) * R + 8 * j + 2 * q) =
            make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    __syncthreads();
    // this CTA's sum, in place of the first half's
    for (int e = 4 * tid; e < M * R; e += 4 * kThreads) {
      float4 s = *reinterpret_cast<float4*>(part + e);
      const float4 v = *reinterpret_cast<const float4*>(part + M * R + e);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
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
    for (int e = 4 * tid; e < M * R; e += 4 * kThreads) {
      const float4 s = C > 1 ? cluster_sum_f4(part + e, C) : *reinterpret_cast<const float4*>(part + e);
      const int t = e / R, c = e % R;
      // columns beyond r stay zero even where a row holds an infinity (0 x inf)
      const float4 ss = c < r ? make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (a.mid && t < m && c < r && (unsigned)(t % C) == rank)
        *reinterpret_cast<float4*>(a.mid + (int64_t)__ldg(a.plan.order + pos0 + t) * r + c) = BWD ? ss : s;
      const uint32_t h0 = pack2(ss.x, ss.y), h1 = pack2(ss.z, ss.w);
      const uint32_t o = at<R>(t, c / 8) + (c & 4) * 2;
      *reinterpret_cast<uint2*>(mid_hi + o) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(mid_lo + o) =
          make_uint2(pack2(ss.x - lo_f32(h0), ss.y - hi_f32(h0)), pack2(ss.z - lo_f32(h1), ss.w - hi_f32(h1)));
    }
    if (C > 1) cluster_arrive();                               // done with the others' memory
  } else if (a.mid != nullptr) {
    for (int e = tid; e < m * r; e += kThreads) {              // mid is zero
      const int t = e / r;
      if ((unsigned)(t % C) == rank) a.mid[(int64_t)__ldg(a.plan.order + pos0 + t) * r + e % r] = 0.0f;
    }
  }
  for (int step = n1; step < n1 + n2; ++step) {
    cp_wait<S::kStages - 2>();
    __syncthreads();                                           // the stage, and at first mid, is complete
    request();
    unsigned char* const tile_p = ring + slot * S::kStage;
    const uint32_t out_at = ring_at + slot * S::kStage, w_at = out_at + S::kRowBytes;
    slot = slot + 1 == S::kStages ? 0 : slot + 1;
    if (adapted) {
      // the sums start from base, whose fragments lie in the stage as the results will
      float acc[COLS / 16][4];
#pragma unroll
      for (int j = 0; j < COLS / 32; ++j) {
        uint32_t b[4] = {0, 0, 0, 0};
        if (a.base != nullptr) ldsm4(b, out_at + moved<COLS>(x_off, 0, COLS / 2 * wh + 16 * j));
#pragma unroll
        for (int e = 0; e < 4; ++e) {                          // rows g + 8 (e & 1), columns 8 (e / 2) + 2 q
          acc[2 * j + e / 2][2 * (e & 1)] = lo_f32(b[e]);
          acc[2 * j + e / 2][2 * (e & 1) + 1] = hi_f32(b[e]);
        }
      }
#pragma unroll
      for (int k = 0; k < R; k += 16) {
        uint32_t h[4], l[4];
        ldsm4(h, hi_at + moved<R>(mid_off, 0, k));
        ldsm4(l, lo_at + moved<R>(mid_off, 0, k));
#pragma unroll
        for (int j = 0; j < COLS / 32; ++j) {
          uint32_t w[4];
          if constexpr (!BWD) ldsm4(w, w_at + moved<R>(w2_off, COLS / 2 * wh + 16 * j, k));
          else ldsm4t(w, w_at + moved<COLS>(w2_off, k, COLS / 2 * wh + 16 * j));
          mma16816(acc[2 * j], h[0], h[1], h[2], h[3], w[0], w[1]);
          mma16816(acc[2 * j + 1], h[0], h[1], h[2], h[3], w[2], w[3]);
          mma16816(acc[2 * j], l[0], l[1], l[2], l[3], w[0], w[1]);
          mma16816(acc[2 * j + 1], l[0], l[1], l[2], l[3], w[2], w[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < COLS / 32; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack2(acc[2 * j + e / 2][2 * (e & 1)], acc[2 * j + e / 2][2 * (e & 1) + 1]);
        stsm4(out_at + moved<COLS>(x_off, 0, COLS / 2 * wh + 16 * j), o);
      }
      __syncthreads();
    }
    const int c = COLS * ((int)rank + (int)C * (step - n1)) + 8 * tunit;
#pragma unroll
    for (int h = 0; h < NH; ++h)
      if (tok[h] >= 0 && c < N)
        *reinterpret_cast<uint4*>(a.out + (int64_t)tok[h] * N + c) =
            adapted || a.base != nullptr
                ? *reinterpret_cast<const uint4*>(tile_p + at<COLS>(trow + ROWS * h, tunit))
                : make_uint4(0, 0, 0, 0);
  }
  // Here and not before the columns: the next launch's CTAs would take SMs from this one's columns
  // (forward, 4096 tokens, r = 16: 21.6 against 22.2 us; backward, inputs changing, 1500 tokens, D = 2048, r = 8:
  // 22.3 against 24.9, 4096 tokens, D = 4096, r = 16: 48.0 both, r = 64: 113.5 against 111.3).
  griddep_launch_dependents();
  cp_wait<0>();
  if (adapted && C > 1) cluster_wait();                        // the others are done with this CTA's memory
}

// ------------------------------------------------------------------- weight gradients
// One cluster: 128 (64 at r > 32) columns of x (grad_a) or of g (grad_b) over all tokens, its
// CTAs sharing the plan's 64-token tiles evenly (TileShare). D[rho, column] = sum_t mid[t, rho]
// row[t, column]: tokens are the contraction index, and both operands are read transposed. A
// warp has 16 columns and every rho (half of them at r > 32), so no sums are shared inside a
// CTA. An adapter whose tiles lie in several CTAs is written by the first of them, which adds
// the others' sums in rank order through distributed shared memory.
// Tiles pass through a ring of cp.async stages: a tile's rows are requested one to three
// steps ahead, its token numbers two or three steps before that.
// mid is fp32; it enters the product as three bf16 that sum to it in all but its last bits
// (24 mantissa bits), since the gradients are fp32.
// K = N = 4096, 4096 tokens of 8 adapters, from cold L2: r = 16 26 us for the 67 MB of x and g (10 at the
// copy rate; start and end take about 8), r = 64 78 us, r = 128 163 us. A CTA per adapter and column
// group, whatever the group's size, took 41 us on uneven groups where this takes 26 (r = 16).
template <int R>
struct Wgrad {
  static constexpr int kCols = R <= 32 ? 128 : 64, kTok = 64, kOrders = 8;
  static constexpr int kStages = R == 16 ? 4 : (R == 64 ? 2 : 3), kAhead = kStages - 1;   // row tiles requested ahead
  // A tile's token numbers come with the rows of the tile kOrder before it, which have arrived
  // when its own rows are requested (kOrder >= kAhead).
  static constexpr int kOrder = kAhead < 2 ? 2 : kAhead;
  static_assert(kAhead + kOrder < kOrders, "order ring");
  static constexpr int kPerSM = R <= 64 ? 2 : 1;              // CTAs that fit
  static constexpr int kWC = kCols / 16, kNI = R / 16 / (kWarps / kWC);   // column groups; rho tiles per warp
  static constexpr int kRowBytes = kTok * kCols * 2;
  static constexpr int kStage = kRowBytes + kTok * R * 4;     // rows, and mid in fp32
  static constexpr int kMid = 3 * kTok * R * 2;               // mid as three tiles of R columns
  static constexpr int kHead = R * kCols * 4;
  static constexpr size_t smem = (size_t)kStage * kStages + kMid + kHead;
};

template <int R>
__global__ void __launch_bounds__(kThreads, Wgrad<R>::kPerSM)
k_lora_wgrad(LoraWgrad<bf16_t> a, int blocks_b) {
  using S = Wgrad<R>;
  constexpr int COLS = S::kCols, UNITS = COLS / 8, NI = S::kNI;
  constexpr int NA = NI * 8;                                   // sums per thread
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ int2 desc[kWindow + 2];
  __shared__ __align__(16) int order[S::kOrders][S::kTok];
  unsigned char* const mid_p = ring + S::kStage * S::kStages;
  float* const head = reinterpret_cast<float*>(mid_p + S::kMid);   // [NA][kThreads]
  const uint32_t ring_at = shared_at(ring), mid_at = shared_at(mid_p);
  const unsigned C = cluster_size(), rank = cluster_rank();
  const int r = a.r, block = blockIdx.x / C;
  const bool is_a = block >= blocks_b;                         // grad_b's blocks first: they start early
  const bool early = starts_early(a.after_rows, is_a);
  if (!early) griddep_wait();
  if (!plan_matches(a.plan)) {
    if (early) griddep_wait();
    return;
  }
  const int n0 = S::kCols * (is_a ? block - blocks_b : block);
  const int W = is_a ? a.K : a.N;                              // columns of the rows read
  const bf16_t* const rows = is_a ? a.x : a.g;
  const float* const mid = is_a ? a.v : a.u;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int wc = warp % S::kWC, rho0 = 16 * NI * (warp / S::kWC);
  const uint32_t x_off = moved<COLS>(lane_rows<COLS>(lane), 0, 16 * wc);
  const uint32_t m_off = moved<R>(lane_cols<R>(lane), 0, rho0);
  const TileShare share(a.plan, rank, C);

  float acc[NA];
  auto clear = [&] {
#pragma unroll
    for (int e = 0; e < NA; ++e) acc[e] = 0.0f;
  };
  // sums of adapter ad to global memory; acc[8 i + 4 j + 2 h + e] is row rho0 + 16 i + g + 8 h,
  // column 16 wc + 8 j + 2 q + e
  auto scale_of = [&](int ad) { return (!is_a && a.scale) ? __ldg(a.scale + ad) : 1.0f; };
  auto write = [&](int ad, float scale) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rho = rho0 + 16 * i + g + 8 * h, c = n0 + 16 * wc + 8 * j + 2 * q;
          if (rho >= r || c >= W) continue;
          const float* v = acc + 8 * i + 4 * j + 2 * h;
          if (is_a) {
            *reinterpret_cast<float2*>(a.grad_a + ((int64_t)ad * r + rho) * W + c) = make_float2(v[0], v[1]);
          } else {
            float* dst = a.grad_b + ((int64_t)ad * W + c) * r + rho;
            dst[0] = scale * v[0];
            dst[r] = scale * v[1];
          }
        }
  };

  clear();
  int open = -1;                                               // adapter whose sums go on in the next CTA
  bool from_before = false;                                    // the sum at hand began in an earlier CTA
  for (int w0 = share.lo; w0 < share.hi; w0 += kWindow) {
    const int count = min(kWindow, share.hi - w0);
    __syncthreads();                                           // the last window is consumed
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
        const uint32_t dst = ring_at + i % S::kStages * S::kStage;
#pragma unroll
        for (int h = 0; h < S::kTok * UNITS / kThreads; ++h) {
          const int t = tid / UNITS + kThreads / UNITS * h, c = n0 + tid % UNITS * 8;
          const bool in = t < tokens && c < W;
          cp16(dst + at<COLS>(t, tid % UNITS), in ? rows + (int64_t)ord[t] * W + c : rows, in);
        }
#pragma unroll
        for (int h = 0; h < R / 16; ++h) {
          const int e = tid + kThreads * h, t = e / (R / 4), c = e % (R / 4) * 4;
          const bool in = t < tokens && c < r;
          cp16(dst + S::kRowBytes + (t * R + c) * 4, in ? mid + (int64_t)ord[t] * r + c : mid, in);
        }
      }
    };
#pragma unroll
    for (int s = 0; s < S::kOrder; ++s) request_order(s);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S::kAhead; ++s) {
      request(s);
      request_order(s + S::kOrder);
      cp_commit();
    }
    if (w0 == share.lo) from_before = desc[0].y == desc[1].y;
    for (int i = 0; i < count; ++i) {
      cp_wait<S::kAhead - 1>();                                // rows i and order i + kAhead have arrived
      __syncthreads();
      request(i + S::kAhead);
      request_order(i + S::kAhead + S::kOrder);
      cp_commit();
      const unsigned char* const stage = ring + i % S::kStages * S::kStage;
#pragma unroll
      for (int h = 0; h < R / 16; ++h) {
        const int e = tid + kThreads * h, t = e / (R / 4), c = e % (R / 4) * 4;
        float4 v = *reinterpret_cast<const float4*>(stage + S::kRowBytes + (t * R + c) * 4);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          const uint32_t p0 = pack2(v.x, v.y), p1 = pack2(v.z, v.w);
          *reinterpret_cast<uint2*>(mid_p + s * S::kTok * R * 2 + at<R>(t, c / 8) + (c & 4) * 2) = make_uint2(p0, p1);
          v.x -= lo_f32(p0), v.y -= hi_f32(p0), v.z -= lo_f32(p1), v.w -= hi_f32(p1);
        }
      }
      __syncthreads();
      const uint32_t x_at = ring_at + i % S::kStages * S::kStage;
      const int tokens = desc[i + 2].x - desc[i + 1].x, ad = desc[i + 1].y;
      float d[NI][2][4];                                       // this tile's sums
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[j][e / 4][e % 4] = 0.0f;
#pragma unroll
      for (int k = 0; k < S::kTok; k += 16) {
        if (k >= tokens) break;
        uint32_t b[4];
        ldsm4t(b, x_at + moved<COLS>(x_off, k, 0));
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            uint32_t f[4];
            ldsm4t(f, mid_at + s * S::kTok * R * 2 + moved<R>(m_off, k, 16 * j));
            mma16816(d[j][0], f[0], f[1], f[2], f[3], b[0], b[1]);
            mma16816(d[j][1], f[0], f[1], f[2], f[3], b[2], b[3]);
          }
      }
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[8 * j + e] += d[j][e / 4][e % 4];
      const bool goes_on = desc[i + 2].y == ad;                // the next tile is the same adapter's
      if (w0 + i + 1 == share.hi && goes_on && !from_before) {
        open = ad;                                             // its sums stay here
      } else if (!goes_on || w0 + i + 1 == share.hi) {
        if (from_before) {                                     // an earlier CTA writes it
#pragma unroll
          for (int e = 0; e < NA; ++e) head[e * kThreads + tid] = acc[e];
          from_before = false;
        } else {
          write(ad, scale_of(ad));
        }
        clear();
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
        if (klo == khi) continue;                              // no tiles there
        if (__ldg(a.plan.tiles + klo).y != open) break;
        add_from(acc, head, k);
      }
      write(open, scale_of(open));
    }
    cluster_arrive();
  }
  // adapters without tokens, shared by the cluster: zeros, whatever their scale holds
  clear();
  for (int ad = rank; ad < a.plan.n; ad += C)
    if (__ldg(a.plan.offsets() + ad) == __ldg(a.plan.offsets() + ad + 1)) write(ad, 1.0f);
  if (C > 1) cluster_wait();                                   // the others are done with this CTA's memory
  if (early) griddep_wait();
}

template <auto KERNEL>
cudaError_t run_rows(size_t smem, const LoraRows<bf16_t>& a, int64_t tiles, int cluster, cudaStream_t s) {
  const cudaError_t e = allow_smem<KERNEL>(smem);
  if (e != cudaSuccess) return e;
  return launch_cluster_pdl(KERNEL, dim3((unsigned)(tiles * cluster)), dim3(kThreads), cluster, smem, s, a);
}

template <int R, bool BWD>
cudaError_t rows_m(LoraRows<bf16_t> a, const int* plan, int64_t T, int n, cudaStream_t s) {
  const int list = lora_list(T, n);
  a.plan = plan_view(plan, T, n, list);
  const int64_t tiles = plan_layout(T, n).cap[list];
  const int cluster = lora_cluster(tiles, list, false, a.K, a.N);
  if (list == 1) return run_rows<k_lora_rows16<R, BWD>>(rows16_smem<R>(), a, tiles, cluster, s);
  return run_rows<k_lora_rows64<R, BWD>>(Rows64<R>::smem, a, tiles, cluster, s);
}

template <int R>
cudaError_t run_wgrad(const LoraWgrad<bf16_t>& a, cudaStream_t s) {
  using S = Wgrad<R>;
  const cudaError_t e = allow_smem<k_lora_wgrad<R>>(S::smem);
  if (e != cudaSuccess) return e;
  const int ka = (a.K + S::kCols - 1) / S::kCols, nb = (a.N + S::kCols - 1) / S::kCols;
  const int ba = a.grad_a ? ka : 0, bb = a.grad_b ? nb : 0;
  // by both widths, so that a gradient does not depend on whether the other is asked for
  const int cluster = lora_token_split(a.plan.T, a.plan.n, ka + nb, S::kTok, S::kPerSM);
  return launch_cluster_pdl(k_lora_wgrad<R>, dim3((unsigned)((ba + bb) * cluster)), dim3(kThreads), cluster, S::smem, s,
                            a, bb);
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

}  // namespace rdfft
