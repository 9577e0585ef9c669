// window_split.cuh -- the keys that attention with windows visits, for the cut of
// tree_split.cuh.
//
// New row i of a head with n cached tokens sees the keys t <= n + i that lie among
// the first `sinks` or in (n + i - window, n + i]. Of all its rows together a head
// visits the tiles of the sinks and those from the first row's window (or the first
// new row: its accumulated weight starts here) to the end; the tiles between, the
// gap, are not read. Visited tile j is tile j of the head for j < lead, else j + gap.
#pragma once

#include "tree_split.cuh"
#include "window.h"

namespace kvx {

// A tile of 64 keys against an item, in the same units as tree_split.cuh's.
__device__ __forceinline__ constexpr int tile_cost(const WindowParams &) { return 1; }
__device__ __forceinline__ constexpr int item_cost(const WindowParams &) { return 1; }

struct Window {
  int sinks, width;
};
__device__ __forceinline__ void tree_raw_window(const WindowParams &p, int h, TreeRaw &r) {
  r.sinks = p.sinks ? p.sinks[h] : 0;
  r.width = p.window ? p.window[h] : INT32_MAX;
}
__device__ __forceinline__ Window window_of(const TreeHead &t) { return {t.sinks, t.width}; }
// Whether the row at position pos sees key t.
__device__ __forceinline__ bool window_sees(const Window &w, int pos, int t) {
  return t <= pos && (t < w.sinks || t > pos - w.width);
}

template <int kTile>
__device__ __forceinline__ void tree_tiles(const WindowParams &, const TreeRaw &r, TreeHead &t) {
  t.sinks = max(0, r.sinks);
  t.width = max(0, r.width);
  t.tiles = t.lead = t.gap = 0;
  if (t.T <= 0) return;
  const int all = (t.n + t.T + kTile - 1) / kTile;
  const int from = max(0, min(t.n, t.n - t.width + 1)) / kTile;
  t.lead = min(all, t.sinks / kTile + (t.sinks % kTile ? 1 : 0));
  t.gap = max(0, from - t.lead);
  t.tiles = all - t.gap;
}
// The head's tile that visited tile j is.
__device__ __forceinline__ int window_tile(const TreeHead &t, int j) {
  return j < t.lead ? j : j + t.gap;
}

// Whether every row [i0, i1] of an item sees all of the keys [t0, t0 + len).
__device__ __forceinline__ bool window_all_seen(const Window &w, int n, int i0, int i1, int t0,
                                                int len) {
  return t0 + len - 1 <= n + i0 && (t0 + len <= w.sinks || t0 > n + i1 - w.width);
}

// Whether one of the rows [i0, i1] sees key t.
__device__ __forceinline__ bool window_any_sees(const Window &w, int n, int i0, int i1, int t) {
  return t <= n + i1 && (t < w.sinks || (t > n + i0 - w.width && w.width > 0));
}
// The keys base .. base + 31 that the row at position pos sees, as bits.
__device__ __forceinline__ uint32_t window_bits(const Window &w, int pos, int base) {
  auto ones = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
  const int from = max(0, pos - w.width + 1);
  return ones(pos + 1 - base) & (ones(w.sinks - base) | ~ones(from - base));
}

// Scores of an item's visited key `key` (tile * kTile + place): one row group's.
__device__ __forceinline__ float *window_scores(const WindowParams &p, const TreeHead &t, int group,
                                                int64_t key) {
  const int64_t bh = (int64_t)t.b * p.c.Hkv + t.h;
  return p.scores + ((bh * p.score_groups + group) * p.score_keys + key) * p.score_rows;
}

}  // namespace kvx
