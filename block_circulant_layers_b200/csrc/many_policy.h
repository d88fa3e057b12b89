// Launch-shape rules of the many-adapter kernels. Plain host arithmetic, checked on the CPU.
#pragma once

#include <stdint.h>

#include "layer_policy.h"

namespace rdfft {

// Tile list of the low-rank rows kernels (adapter_plan.h): tiles of 64 tokens (list 2) from
// T = 1024 on while the mean group has 32, else of 16 (list 1). A tile reads its adapter's A and
// B once, so longer tiles read them less often; short batches lack tiles to fill the SMs, and a
// group far below 64 leaves most of a tile's rows empty. bf16, K = N = 4096, r = 64, 4 adapters,
// tiles of 16 against 64: T = 777 22.4 and 28.6 us, T = 1500 36.4 and 30.1; fp32, K = N = 2048,
// r = 16: T = 777 17.9 and 23.2, T = 1500 24.9 and 25.4, T = 4096 52.5 and 41.6.
inline int lora_list(int64_t T, int n) { return T >= 1024 && T >= 32 * (int64_t)n ? 2 : 1; }

// CTAs per cluster (per tile) of the low-rank rows kernels: as many as let the clusters start
// together (a cluster's CTAs take separate SMs of one GPC), so that a tile's columns spread
// over more SMs, and not so many that a CTA has less than 256 columns (fp32: 64). A 64-token
// tile of bf16 has a long pipeline in each CTA and gains nothing from 8. bf16, r = 64 as above,
// 8, 4 and 2 CTAs: T = 16 12.1, 16.9, 27.8 us (2 tiles), T = 777 30.0, 22.4, 28.0 (52), T = 1500 44.9,
// 41.7, 36.4 (97), T = 4096 63.7, 43.6, 52.4 (65 tiles of 64); fp32: T = 777 83.2, 75.7, 90.7,
// T = 1500 88.5, 104.7, 196.9 (26 tiles of 64), T = 4096 217, 160, 200.
inline int lora_cluster(int64_t tiles, int list, bool f32, int K, int N) {
  int c;
  if (list == 1) c = tiles <= (f32 ? 48 : 20) ? 8 : (tiles <= (f32 ? 150 : 56) ? 4 : 2);
  else c = (f32 && tiles <= 40) ? 8 : (tiles <= 111 ? 4 : 2);
  const int widest = K > N ? K : N;
  while (c > 1 && (int64_t)c * (f32 ? 64 : 256) > widest) c /= 2;
  return c;
}

// CTAs per cluster of the low-rank weight gradients, which share the batch's tokens (and the
// adapters that have none): as many as keep the grid of `blocks` clusters within one wave of
// 148 x per_sm CTAs, at most 8, and no more than there are tiles of `chunk` tokens or adapters.
// bf16, K = N = 4096, r = 16, T = 4096, 64 clusters of 1, 2, 4, 6, 8 CTAs, three of which fit an
// SM (6 fill the wave): 65.6, 40.1, 29.6, 27.6, 41.9 us; r = 64, one (2 fill it): 138, 77.7, 86.0,
// 88.6, 129.
inline int lora_token_split(int64_t T, int n, int blocks, int chunk, int per_sm) {
  int64_t c = 148 * per_sm / blocks;
  const int64_t tiles = (T + chunk - 1) / chunk, most = tiles > n ? tiles : n;
  if (c > most) c = most;
  return c < 1 ? 1 : (c > 8 ? 8 : (int)c);
}

// Tokens per CTA of the many-adapter layer kernels at p <= 512: as layer_x_tokens for T
// tokens, but 1 while the mean group is below 2 and at most 2 below 12 (a CTA's tokens share
// one adapter, and unfilled places cost their transforms). bf16 forward, 64 adapters, 1, 2 and 4
// tokens per CTA: D = 4096, p = 512, mean 1 12.1, 14.2, 15.5 us, mean 8 24.2, 18.2, 20.3, mean 16
// 43.1, 32.0, 27.4; D = 4096, p = 128, mean 2 24.5, 21.6, 22.0; D = 1024, p = 256, mean 8 13.1,
// 8.9, 10.1, mean 16 23.4, 15.6, 11.0.
inline int circ_many_tokens(int64_t T, int n, int q, int qi_max, int n_sm, int tt_max) {
  const int64_t mean = T / (n > 0 ? n : 1);
  const int by_group = mean >= 12 ? 4 : (mean >= 2 ? 2 : 1);
  return layer_x_tokens(T, q, qi_max, n_sm, by_group < tt_max ? by_group : tt_max);
}

// Token slices of the many-adapter gradient kernels: one CTA per SM over njgroups groups, no
// more than the batch has token tiles (or adapters in use, a tile each, if those are more).
// D = 4096, p = 512, 4096 tokens of 8 adapters, both gradients: 115 us; half as many slices 207,
// twice as many 122; p = 128: 391, 748, 399.
inline int circ_many_slices(int64_t T, int n, int njgroups, int tt, int n_sm) {
  int64_t s = n_sm / njgroups;
  const int64_t tiles = (T + tt - 1) / tt, used = T < n ? T : n, most = tiles > used ? tiles : used;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

}  // namespace rdfft
