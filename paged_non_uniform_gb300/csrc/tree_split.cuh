// tree_split.cuh -- how tree attention is cut over the thread blocks, from
// device lengths, and how the pieces of a head are merged.
//
// A head (b, h) with T_b new rows has T_b * g query rows, in groups of
// group_tokens new rows, and n[b][h] + T_b keys, in tiles of kTile. A row group costs
// kItemCost for being worked on at all (queries, pipeline fill, epilogue) and kTileCost
// a tile. All costs are laid end to end -- heads in order, row groups within a head,
// tiles within a row group -- and block c of `blocks` takes the tiles that start in
// [c * U / blocks, (c + 1) * U / blocks): the flat cut with a charge per item of the
// ahead-of-time plan ("Tangram: Unlocking Non-Uniform KV Cache for Efficient
// Multi-turn LLM Serving", AOT Load Balancing, Fig. 13), but found by every
// block itself from one pass over the lengths, so that nothing is planned on
// the host. A row group whose tiles span blocks leaves one partial (max in
// log2 units, sum, un-normalised output) per block; a second, small kernel folds
// them in block order. A block leaves at most two partials: of the row group
// that runs into it (slot 2c) and of one that begins in it and runs on (slot 2c +
// 1), which it also describes for the second kernel.
#pragma once

#include <math.h>

#include "ptx.cuh"
#include "tree.h"

namespace kvx {

// Measured with the tensor-core kernel on 256 sequences of 100 to 1000 tokens / 32 of 1k to
// 32k with trees of up to 48 tokens: an item charged as 4 fifths of a tile 101.4 / 176 us,
// 6: 102 / 175, 8: 104.6 / 174; an earlier form without a charge took 130 instead of 117.
constexpr int kTileCost = 5;
constexpr int kItemCost = 6;

struct TreeHead {
  int b, h;      // sequence, KV head
  int q0, T;     // first new row, new rows (0: nothing to do)
  int n;         // cached tokens
  int tiles, groups;
  // windows (window_split.cuh): tiles before the gap, tiles left out, and the head's window
  int lead, gap, sinks, width;
};

// The lengths of a head as they are in memory: loaded ahead of their use.
struct TreeRaw {
  int q0, q1, n, sinks, width;
};
__device__ __forceinline__ void tree_raw_window(const TreeParams &, int, TreeRaw &) {}
template <class Prm>
__device__ __forceinline__ TreeRaw tree_raw(const Prm &p, int hd) {
  TreeRaw r = {0, 0, 0, 0, 0};
  if (hd < p.c.B * p.c.Hkv) {
    const int b = hd / p.c.Hkv;
    r.q0 = p.q_start[b];
    r.q1 = p.q_start[b + 1];
    r.n = p.kv_len[hd];
    tree_raw_window(p, hd - b * p.c.Hkv, r);
  }
  return r;
}

// What a tile and an item cost, by the kind of attention.
__device__ __forceinline__ constexpr int tile_cost(const TreeParams &) { return kTileCost; }
__device__ __forceinline__ constexpr int item_cost(const TreeParams &) { return kItemCost; }
// A head's tiles: all of its keys.
template <int kTile>
__device__ __forceinline__ void tree_tiles(const TreeParams &, const TreeRaw &, TreeHead &t) {
  t.tiles = t.T > 0 ? (t.n + t.T + kTile - 1) / kTile : 0;
  t.lead = t.gap = t.sinks = t.width = 0;
}

// Cost of a row group, and of the head.
template <class Prm>
__device__ __forceinline__ int tree_seg(const Prm &p, const TreeHead &t) {
  return t.tiles ? item_cost(p) + tile_cost(p) * t.tiles : 0;
}
template <class Prm>
__device__ __forceinline__ int64_t tree_cost(const Prm &p, const TreeHead &t) {
  return (int64_t)tree_seg(p, t) * t.groups;
}

// Head `hd` from its lengths; lengths that do not fit their arrays give T = 0
// and set KVX_DEV_BAD_LENGTH (in the one block that reports).
template <int kTile, class Prm>
__device__ __forceinline__ TreeHead tree_head(const Prm &p, int hd, const TreeRaw &r,
                                              bool report) {
  TreeHead t;
  t.b = hd / p.c.Hkv;
  t.h = hd - t.b * p.c.Hkv;
  t.q0 = r.q0;
  t.n = r.n;
  t.T = r.q1 - r.q0;
  const CacheGroup &g = p.c.grp[p.c.head_grp[t.h]];
  const bool ok = r.q0 >= 0 && r.q1 >= r.q0 && r.q1 <= p.max_rows && t.T <= p.max_q && r.n >= 0 &&
                  r.n <= g.tokens - t.T;
  if (!ok) {
    if (report) atomicOr(p.status, KVX_DEV_BAD_LENGTH);
    t.T = t.n = 0;
  }
  tree_tiles<kTile>(p, r, t);
  t.groups = t.T <= p.group_tokens ? 1 : (t.T + p.group_tokens - 1) / p.group_tokens;
  return t;
}

struct TreeRange {
  int units;       // cost of all heads (little work: to whole parts)
  int blocks;      // blocks with work
  int begin, end;  // this block's part of it
  int head;        // the head that holds `begin`
  int base;        // where that head starts
  TreeHead first;  // that head
};

// Where block c begins: floor(c * units / blocks) without 64 bits.
__device__ __forceinline__ int tree_bound(int units, int blocks, int c) {
  const int q = units / blocks, r = units - q * blocks;
  return c * q + c * r / blocks;  // blocks is at most a few hundred
}
// The block that holds position u.
__device__ __forceinline__ int tree_block_of(int units, int blocks, int u) {
  return (int)((((int64_t)u + 1) * blocks - 1) / units);
}

// Sums the costs of all heads over the block's NT threads and finds this block's range.
// `min_tiles`: a block gets at least the cost of that many (one at least, so that every
// block between a row group's first and last has a tile of it).
template <int NT, int kTile, class Prm>
__device__ __forceinline__ TreeRange tree_range(const Prm &p, int min_tiles,
                                                int64_t *warp_sum /* shared, NT / 32 */,
                                                TreeRange *shared) {
  // Each warp takes a run of heads, its lanes one head in turn.
  const int heads = p.c.B * p.c.Hkv, run = (heads + NT / 32 - 1) / (NT / 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = min(heads, warp * run), hi = min(heads, lo + run);
  int64_t s = 0;
  TreeRaw raw = tree_raw(p, lo + lane), raw1 = tree_raw(p, lo + lane + 32);
  for (int i = lo + lane; i < hi; i += 32) {  // (lengths loaded two steps ahead)
    const TreeRaw raw2 = tree_raw(p, i + 64);
    s += tree_cost(p, tree_head<kTile>(p, i, raw, blockIdx.x == 0));
    raw = raw1;
    raw1 = raw2;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  // More units than an int holds are refused whole. Distinct pages cannot hold that many, but the
  // margin is small: an fp32 cache of 288 GB with D = 64, g = 8 and 128 new rows a sequence has 32
  // row groups a head and 32 KB a tile, 1.5e9 units with 262,144 heads,
  // 1.4 times less (bf16: 5.7 times). Dearer tiles or items, or larger trees, need more bits.
  if (all > INT32_MAX) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, KVX_DEV_BAD_LENGTH);
    all = 0;
  }
  // Little work: parts of exactly `least`, so that a block has no more tiles than that
  // stands for (the last part may be shorter).
  const int least = min_tiles * tile_cost(p), total = (int)all;
  const bool little = total / least < (int)gridDim.x;
  const int blocks = little ? (total + least - 1) / least : (int)gridDim.x;
  const int units = little ? blocks * least : total;
  const bool work = (int)blockIdx.x < blocks;
  const int begin = work ? tree_bound(units, blocks, blockIdx.x) : 0;
  const int end = work ? min(total, tree_bound(units, blocks, blockIdx.x + 1)) : 0;
  if (!work) {
    if (tid == 0) *shared = {units, blocks, 0, 0, 0, 0, {}};
  } else if (begin >= before && begin < before + s) {
    // this warp's run holds it: 32 heads at a time
    if (lane == 0) *shared = {units, blocks, 0, 0, 0, 0, {}};
    __syncwarp();
    int base = (int)before;
    for (int i0 = lo; i0 < hi && base <= begin; i0 += 32) {
      const int i = i0 + lane;
      TreeHead t = {};
      if (i < hi) t = tree_head<kTile>(p, i, tree_raw(p, i), false);
      const int u = (int)tree_cost(p, t);
      int x = u;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (begin >= base + x - u && begin < base + x)
        *shared = {units, blocks, begin, end, i, base + x - u, t};
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  return *shared;
}

// One block's items in order: (head, row group, tiles [t0, t1)).
struct TreeItem {
  TreeHead head;
  int group, t0, t1;
  int seg;  // where the row group starts
};

// Walks a block's items. The lengths of the two heads after the current one are
// already in flight, so that short heads do not wait for them.
template <int kTile>
struct TreeCursor {
  int at, end, base, hd;
  TreeHead head;
  TreeRaw raw1, raw2;
  template <class Prm>
  __device__ __forceinline__ TreeCursor(const Prm &p, const TreeRange &r)
      : at(r.begin), end(r.end), base(r.base), hd(r.head), head(r.first) {
    if (at < end) {
      raw1 = tree_raw(p, hd + 1);
      raw2 = tree_raw(p, hd + 2);
    }
  }
  template <class Prm>
  __device__ __forceinline__ bool next(const Prm &p, TreeItem &it) {
    while (at < end) {
      const int seg = tree_seg(p, head);
      if (at - base >= seg * head.groups) {
        base += seg * head.groups;
        ++hd;
        head = tree_head<kTile>(p, hd, raw1, false);
        raw1 = raw2;
        raw2 = tree_raw(p, hd + 2);
        continue;
      }
      const int group = head.groups == 1 ? 0 : (at - base) / seg;
      const int start = base + group * seg, first = start + item_cost(p);  // of its tile 0
      const int c = tile_cost(p), t0 = max(0, at - first + c - 1) / c;
      const int t1 = min(head.tiles, (max(0, end - first) + c - 1) / c);
      at = start + seg;  // (past `end` where the row group runs on)
      if (t0 >= t1) continue;
      it.head = head;
      it.group = group;
      it.t0 = t0;
      it.t1 = t1;
      it.seg = start;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ bool tree_whole(const TreeItem &it) {
  return it.t0 == 0 && it.t1 == it.head.tiles;
}
__device__ __forceinline__ int tree_slot(const TreeItem &it) {
  return 2 * (int)blockIdx.x + (it.t0 == 0 ? 1 : 0);
}

// Scale of a partial with maximum m when the merged maximum is M (a partial
// that has seen no token has m = -inf and contributes nothing).
__device__ __forceinline__ float tree_weight(float m, float M) {
  return m == -INFINITY ? 0.f : ex2(m - M);
}

// First new row, and query rows, of an item.
__device__ __forceinline__ int tree_first(const TreeParams &p, const TreeItem &it) {
  return it.group * p.group_tokens;
}
__device__ __forceinline__ int tree_rows(const TreeParams &p, const TreeItem &it) {
  return min(p.group_tokens, it.head.T - it.group * p.group_tokens) * p.c.g;
}
// r / g for the query rows r of an item.
__device__ __forceinline__ int tree_div_g(const TreeParams &p, int r) {
  return (r * p.recip_g) >> 16;
}
// The output row of query row r of the item whose first new row is row0 of the
// row arrays.
__device__ __forceinline__ float *tree_out(const TreeParams &p, int row0, int h, int r) {
  const int i = tree_div_g(p, r), j = r - i * p.c.g;
  return p.out + ((size_t)(row0 + i) * p.c.Hq + (size_t)h * p.c.g + j) * p.c.D;
}

// Where its maximum and sum go (window attention with weights).
__device__ __forceinline__ int tree_ml_row(const TreeParams &p, int b, int first) {
  return b * p.max_q + first;  // of a sequence's new row `first`
}
__device__ __forceinline__ float2 *tree_row_ml(const TreeParams &p, int row0, int h, int r) {
  const int i = tree_div_g(p, r), j = r - i * p.c.g;
  return p.row_ml + (size_t)(row0 + i) * p.c.Hq + (size_t)h * p.c.g + j;
}

// Describes the row group that starts in this block and runs past its end (one
// thread; `it` is the block's last item, or null if it has none).
template <class Prm>
__device__ __forceinline__ void tree_describe(const Prm &p, const TreeRange &r,
                                              const TreeItem *it) {
  TreeSplit s = {0, 0, 0, 0};
  if (it && it->t0 == 0 && !tree_whole(*it)) {
    const int last = tree_block_of(
        r.units, r.blocks, it->seg + item_cost(p) + tile_cost(p) * (it->head.tiles - 1));
    s = {last - (int)blockIdx.x + 1, it->head.q0 + tree_first(p, *it), it->head.h,
         tree_rows(p, *it)};
    if (p.row_ml) p.split_row[blockIdx.x] = tree_ml_row(p, it->head.b, tree_first(p, *it));
  }
  p.split[blockIdx.x] = s;
}

// Word `w` of the visibility mask of new row i of a sequence of T rows (bits
// from T on cleared); without masks row i sees rows 0 .. i.
__device__ __forceinline__ uint32_t tree_mask_word(const TreeParams &p, const TreeHead &t, int i,
                                                   int w) {
  uint32_t m;
  int last = t.T - 1;
  if (p.mask) {
    m = w < p.words ? p.mask[(size_t)(t.q0 + i) * p.words + w] : 0u;
  } else {
    m = 0xffffffffu;
    last = i;
  }
  const int n = last + 1 - 32 * w;
  return n <= 0 ? 0u : n >= 32 ? m : m & ((1u << n) - 1u);
}

}  // namespace kvx
