// Launch-shape rules of the many-adapter kernels. Plain host arithmetic, checked on the CPU.
#pragma once

#include <stdint.h>

#include "layer_policy.h"

namespace rdfft {

// Tile list of the low-rank rows kernels (adapter_plan.h): tiles of 64 tokens (list 2) from
// T = 1024 on while the mean group has 32, else of 16 (list 1). A tile reads its adapter's A and
// B once, so longer tiles read them less often; short batches lack tiles to fill the SMs, and a
// group far below 64 leaves most of a tile's rows empty. Forward from cold L2, 4 adapters, tiles of
// 16 against 64: bf16, K = N = 4096, r = 16: T = 777 12.7 and 16.4 us, T = 1500 19.2 and 17.5, T = 4096 37.6
// and 26.3; r = 64: T = 777 24.0 and 25.2, T = 1500 40.9 and 25.8; fp32, K = N = 2048, r = 16: T = 777 19.3
// and 21.5, T = 1500 24.1 and 23.4, T = 4096 60.3 and 38.9.
inline int lora_list(int64_t T, int n) { return T >= 1024 && T >= 32 * (int64_t)n ? 2 : 1; }

// CTAs per cluster (per tile) of the low-rank rows kernels: as many as let the clusters start
// together (a cluster's CTAs take separate SMs of one GPC), so that a tile's columns spread
// over more SMs, and not so many that a CTA has less than 256 columns (fp32: 64). A 64-token
// tile of bf16 has a long pipeline in each CTA and gains nothing from 8. K = N = 4096, r = 64, else as
// above, 8, 4 and 2 CTAs: bf16: T = 16 13.2, 20.0, 34.5 us (2 adapters), T = 777 32.5, 23.9, 34.1 (52
// tiles of 16), T = 1500 29.6, 26.0, 42.1 (27 tiles of 64), T = 4096 60.0, 39.2, 43.9 (68); fp32: T = 777
// 78.0, 76.4, 84.7, T = 1500 80.5, 91.0, 168.8, T = 4096 170.0, 163.4, 173.0.
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
// T = 4096 of 8 adapters, from cold L2, clusters of 1, 2, 3, 4, 6, 8 CTAs: bf16, K = N = 4096, r = 16 (64
// clusters, two CTAs per SM: 4) 58.4, 32.5, 34.1, 26.1, 39.0, 29.5 us; r = 64 (128, two: 2) 100.1, 78.0, 91.2,
// 80.9, 91.5, 87.0; r = 128 (128, one: 1) 163, 165, 181, 173, 201, 208; K = N = 1024, r = 16 (16, two: 8)
// 58.2, 31.7, 24.3, 18.1, 15.5, 14.4; fp32, K = N = 4096, r = 16 (128, three: 3) 71.8, 56.4, 57.1, 56.4, 60.7,
// 60.9; r = 64 (128, two: 2) 176, 143, 160, 146, 157, 151.
inline int lora_token_split(int64_t T, int n, int blocks, int chunk, int per_sm) {
  int64_t c = 148 * per_sm / blocks;
  const int64_t tiles = (T + chunk - 1) / chunk, most = tiles > n ? tiles : n;
  if (c > most) c = most;
  return c < 1 ? 1 : (c > 8 ? 8 : (int)c);
}

// Tokens per CTA of the many-adapter layer kernels at p <= 512: as layer_x_tokens for T
// tokens, but 1 while the mean group is below 2 and at most 2 below 12 (a CTA's tokens share
// one adapter, and unfilled places cost their transforms). bf16 forward, 64 adapters, 1, 2 and 4
// tokens per CTA: D = 4096, p = 512, mean 1 12.1, 14.3, 15.5 us, mean 8 23.8, 18.1, 20.3, mean 16
// 43.1, 31.7, 27.1; D = 4096, p = 128, mean 2 24.4, 21.5, 22.0; D = 1024, p = 256, mean 8 13.0,
// 9.1, 9.9, mean 16 23.5, 15.6, 11.1.
inline int circ_many_tokens(int64_t T, int n, int q, int qi_max, int n_sm, int tt_max) {
  const int64_t mean = T / (n > 0 ? n : 1);
  const int by_group = mean >= 12 ? 4 : (mean >= 2 ? 2 : 1);
  return layer_x_tokens(T, q, qi_max, n_sm, by_group < tt_max ? by_group : tt_max);
}

// Token slices of the many-adapter gradient kernels: one CTA per SM over njgroups groups, no
// more than the batch has token tiles (or adapters in use, a tile each, if those are more).
// D = 4096, p = 512, 4096 tokens of 8 adapters (512 each), both gradients, one call after another:
// 118 us; half as many slices 210, twice as many 127; p = 128: 397, 774, 405.
inline int circ_many_slices(int64_t T, int n, int njgroups, int tt, int n_sm) {
  int64_t s = n_sm / njgroups;
  const int64_t tiles = (T + tt - 1) / tt, used = T < n ? T : n, most = tiles > used ? tiles : used;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

}  // namespace rdfft
