// Layout of an adapter plan: the tokens of a batch grouped by adapter, as int32 words in one
// device buffer (adapter_plan in rdfft.h). Plain host arithmetic, shared by the C ABI, the
// launchers and the host tests.
//
//   [0, 16)      header: T, n, then the tile counts of the three lists below
//   offsets      n + 2 words: sorted positions [offsets[a], offsets[a+1]) use adapter a;
//                a = n is the group of tokens without an adapter
//   order        T words: the token at each sorted position (stable within a group)
//   group        T words: the adapter (or n) of each sorted position
//   tiles[l]     pairs (first sorted position, adapter): a group cut into tiles of at most
//                plan_tile(l) tokens, no tile crossing a group; l = 0, 1, 2
#pragma once

#include <stdint.h>

namespace rdfft {

constexpr int kPlanHeader = 16;
constexpr int kPlanLists = 3;
constexpr int plan_tile(int list) { return 4 << (2 * list); }   // 4, 16, 64

struct PlanLayout {
  int64_t offsets, order, group, tiles[kPlanLists], words;
  int64_t cap[kPlanLists];                  // tiles a list can hold, and launchers' tile grids
};

// Groups are at most min(T, n + 1), and each adds at most one partial tile.
inline int64_t plan_tile_cap(int64_t T, int n, int tile) {
  const int64_t groups = T < n + 1 ? T : n + 1;
  const int64_t c = T / tile + groups;
  return c < T ? c : T;
}

inline PlanLayout plan_layout(int64_t T, int n) {
  PlanLayout l;
  int64_t at = kPlanHeader;
  auto take = [&](int64_t words) {
    const int64_t here = at;
    at += (words + 3) / 4 * 4;              // every part starts on 16 bytes
    return here;
  };
  l.offsets = take(n + 2);
  l.order = take(T);
  l.group = take(T);
  for (int i = 0; i < kPlanLists; ++i) {
    l.cap[i] = plan_tile_cap(T, n, plan_tile(i));
    l.tiles[i] = take(2 * l.cap[i]);
  }
  l.words = at;
  return l;
}

}  // namespace rdfft
