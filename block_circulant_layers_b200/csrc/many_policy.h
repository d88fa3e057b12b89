// Launch-shape rules of the many-adapter kernels. Plain host arithmetic, checked on the CPU.
#pragma once

#include <stdint.h>

#include "layer_policy.h"

namespace rdfft {

// Tile list of the low-rank rows kernels (adapter_plan.h): tiles of 64 tokens once the mean
// group has 32, else of 16. A tile reads its adapter's A and B once, so longer tiles read them
// less often; a group far below 64 would leave most of a tile's rows empty.
inline int lora_list(int64_t T, int n) { return T >= 32 * (int64_t)n ? 2 : 1; }

// CTAs per cluster (per tile) of the low-rank rows kernels: 8 while the tiles are few, so
// that a tile's columns spread over more SMs, fewer when narrow rows would leave a CTA less
// than 256 columns (one step of its 8 warps).
inline int lora_cluster(int64_t tiles, int K, int N) {
  int c = tiles <= 64 ? 8 : 4;
  const int widest = K > N ? K : N;
  while (c > 1 && (int64_t)c * 256 > widest) c /= 2;
  return c;
}

// CTAs per cluster of the low-rank weight gradients, which share the batch's tokens: as many as
// keep the grid of `blocks` clusters within about three CTAs per SM (one wave), at most 8, and
// no more than the batch has pieces of `chunk` tokens.
inline int lora_token_split(int64_t T, int blocks, int chunk) {
  int64_t c = 444 / blocks;
  const int64_t pieces = (T + chunk - 1) / chunk;
  if (c > pieces) c = pieces;
  return c < 1 ? 1 : (c > 8 ? 8 : (int)c);
}

// Tokens per CTA of the many-adapter layer kernels at p <= 512: as layer_x_tokens for T
// tokens, but 1 while the mean group is below 2 and at most 2 below 4 (a CTA's tokens share
// one adapter, and unfilled places cost their transforms).
inline int circ_many_tokens(int64_t T, int n, int q, int qi_max, int n_sm, int tt_max) {
  const int64_t mean = T / (n > 0 ? n : 1);
  const int by_group = mean >= 4 ? 4 : (mean >= 2 ? 2 : 1);
  return layer_x_tokens(T, q, qi_max, n_sm, by_group < tt_max ? by_group : tt_max);
}

// Token slices per adapter of the grad_c kernel: about two CTAs per SM over njgroups groups of
// n adapters (uneven groups then still spread), no more than the batch's tiles.
inline int circ_many_slices(int64_t T, int n, int njgroups, int tt, int n_sm) {
  const int64_t ctas = (int64_t)njgroups * n, tiles = (T + tt - 1) / tt;
  int64_t s = 2 * n_sm / ctas;
  if (s > tiles) s = tiles;
  return s < 1 ? 1 : (int)s;
}

}  // namespace rdfft
