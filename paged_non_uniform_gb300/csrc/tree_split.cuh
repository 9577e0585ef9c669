// tree_split.cuh -- how tree attention is cut over the thread blocks, from
// device lengths, and how the pieces of a head are merged.
//
// A head (b, h) with T_b new rows has T_b * g query rows, in groups of kRows,
// and n[b][h] + T_b keys, in tiles of kTile. A unit is one tile for one row
// group. All units are laid end to end -- heads in order, row groups within a
// head, tiles within a row group -- and block c of `blocks` takes units
// [c * U / blocks, (c + 1) * U / blocks): the flat equal cut of the
// ahead-of-time plan ("Tangram: Unlocking Non-Uniform KV Cache for Efficient
// Multi-turn LLM Serving", AOT Load Balancing, Fig. 13), but found by every
// block itself from one pass over the lengths, so that nothing is planned on
// the host. A row group whose tiles span blocks leaves one partial (max in
// log2 units, sum, un-normalised output) per block; the block that finishes
// last folds them in block order. A block leaves at most two partials: of the
// row group that its range begins in (slot 2c) and of one that begins inside
// its range and runs past its end (slot 2c + 1).
#pragma once

#include <math.h>

#include "ptx.cuh"
#include "tree.h"

namespace kvx {

struct TreeHead {
  int b, h;      // sequence, KV head
  int q0, T;     // first new row, new rows (0: nothing to do)
  int n;         // cached tokens
  int tiles, groups;
};

// Reads the lengths of head `hd`; lengths that do not fit their arrays give
// T = 0 and set KVX_DEV_BAD_LENGTH (in the one block that reports).
template <int kTile, int kRows>
__device__ __forceinline__ TreeHead tree_head(const TreeParams &p, int hd, bool report) {
  TreeHead t;
  t.b = hd / p.c.Hkv;
  t.h = hd - t.b * p.c.Hkv;
  t.q0 = __ldg(p.q_start + t.b);
  const int q1 = __ldg(p.q_start + t.b + 1);
  t.n = __ldg(p.kv_len + hd);
  t.T = q1 - t.q0;
  const CacheGroup &g = p.c.grp[p.c.head_grp[t.h]];
  const bool ok = t.q0 >= 0 && q1 >= t.q0 && q1 <= p.max_rows && t.T <= p.max_q && t.n >= 0 &&
                  (int64_t)t.n + t.T <= ((int64_t)g.stride << p.c.lgP);
  if (!ok) {
    if (report) atomicOr(p.status, KVX_DEV_BAD_LENGTH);
    t.T = t.n = 0;
  }
  t.tiles = t.T > 0 ? (t.n + t.T + kTile - 1) / kTile : 0;
  t.groups = (t.T * p.c.g + kRows - 1) / kRows;
  return t;
}

struct TreeRange {
  int64_t units;    // of all heads
  int blocks;       // blocks with work
  int64_t begin, end;  // this block's units
  int head;         // the head that holds `begin`
  int64_t base;     // first unit of that head
};

// First unit of block c.
__device__ __forceinline__ int64_t tree_bound(int64_t units, int blocks, int c) {
  return (int64_t)c * units / blocks;
}
// The block that holds unit u.
__device__ __forceinline__ int tree_block_of(int64_t units, int blocks, int64_t u) {
  return (int)(((u + 1) * blocks - 1) / units);
}

// Sums the units of all heads over the block's NT threads and finds this block's range.
// `min_units`: a block gets at least that many where there are few in all.
template <int NT, int kTile, int kRows>
__device__ __forceinline__ TreeRange tree_range(const TreeParams &p, int min_units,
                                                int64_t *warp_sum /* shared, NT / 32 */,
                                                TreeRange *shared) {
  const int heads = p.c.B * p.c.Hkv;
  const int per = (heads + NT - 1) / NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = min(heads, tid * per), hi = min(heads, lo + per);
  int64_t s = 0;
  for (int i = lo; i < hi; ++i) {
    const TreeHead t = tree_head<kTile, kRows>(p, i, blockIdx.x == 0);
    s += (int64_t)t.tiles * t.groups;
  }
  int64_t x = s;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  const int64_t want = all / min_units;
  const int blocks = (int)(want < 1 ? 1 : want < (int64_t)gridDim.x ? want : (int64_t)gridDim.x);
  const bool work = (int)blockIdx.x < blocks && all > 0;
  const int64_t begin = work ? tree_bound(all, blocks, blockIdx.x) : 0;
  const int64_t end = work ? tree_bound(all, blocks, blockIdx.x + 1) : 0;
  const int64_t mine = before + x - s;
  if (!work) {
    if (tid == 0) *shared = {all, blocks, 0, 0, 0, 0};
  } else if (begin >= mine && begin < mine + s) {
    int64_t base = mine;
    for (int i = lo; i < hi; ++i) {
      const TreeHead t = tree_head<kTile, kRows>(p, i, false);
      const int64_t u = (int64_t)t.tiles * t.groups;
      if (begin < base + u) {
        *shared = {all, blocks, begin, end, i, base};
        break;
      }
      base += u;
    }
  }
  __syncthreads();
  return *shared;
}

// One block's items in order: (head, row group, tiles [t0, t1)).
struct TreeItem {
  TreeHead head;
  int hd, group, t0, t1;
  int64_t seg;  // first unit of the row group
};

template <int kTile, int kRows>
struct TreeCursor {
  int64_t at, end, base;
  int hd;
  TreeHead head;
  __device__ __forceinline__ TreeCursor(const TreeParams &p, const TreeRange &r)
      : at(r.begin), end(r.end), base(r.base), hd(r.head) {
    if (at < end) head = tree_head<kTile, kRows>(p, hd, false);
  }
  __device__ __forceinline__ bool next(const TreeParams &p, TreeItem &it) {
    if (at >= end) return false;
    while (at - base >= (int64_t)head.tiles * head.groups) {
      base += (int64_t)head.tiles * head.groups;
      head = tree_head<kTile, kRows>(p, ++hd, false);
    }
    const int v = (int)(at - base);
    it.head = head;
    it.hd = hd;
    it.group = v / head.tiles;
    it.t0 = v - it.group * head.tiles;
    it.seg = at - it.t0;
    const int64_t left = end - at;
    it.t1 = left < head.tiles - it.t0 ? it.t0 + (int)left : head.tiles;
    at += it.t1 - it.t0;
    return true;
  }
};

__device__ __forceinline__ bool tree_whole(const TreeItem &it) {
  return it.t0 == 0 && it.t1 == it.head.tiles;
}
__device__ __forceinline__ int tree_slot(const TreeRange &r, const TreeItem &it) {
  return 2 * (int)blockIdx.x + (it.seg > r.begin ? 1 : 0);
}

// Scale of a partial with maximum m when the merged maximum is M (a partial
// that has seen no token has m = -inf and contributes nothing).
__device__ __forceinline__ float tree_weight(float m, float M) {
  return m == -INFINITY ? 0.f : ex2(m - M);
}

// The output row of query row `r` (new row r / g, query head r % g).
__device__ __forceinline__ float *tree_out(const TreeParams &p, const TreeHead &t, int r) {
  const int i = r / p.c.g, j = r - i * p.c.g;
  return p.out + ((size_t)(t.q0 + i) * p.c.Hq + (size_t)t.h * p.c.g + j) * p.c.D;
}

// Publishes this block's partial of a split row group, written by the NT
// threads, and merges the row group in the block that published last. All NT
// threads call it; sync() is a barrier over them, *flag a shared int.
template <int D, int NT, int kTile, int kRows, typename Sync>
__device__ __forceinline__ void tree_publish(const TreeParams &p, const TreeRange &r,
                                             const TreeItem &it, int tid, int *flag, Sync sync) {
  const int64_t seg_end = it.seg + it.head.tiles;
  const int c0 = tree_block_of(r.units, r.blocks, it.seg);
  const int c1 = tree_block_of(r.units, r.blocks, seg_end - 1);
  int *counter = p.counters + (size_t)it.hd * p.row_groups + it.group;
  // the barrier orders the partial's writes before the ticket, whose release
  // publishes them; in the last block its acquire, passed on by the second
  // barrier, makes the other partials visible
  sync();
  if (tid == 0) *flag = ticket_acq_rel(counter) == c1 - c0;
  sync();
  if (*flag) {
    const int rows = min(kRows, it.head.T * p.c.g - it.group * kRows);
    const int first = 2 * c0 + (it.seg > tree_bound(r.units, r.blocks, c0) ? 1 : 0);
    // Each thread owns float4 groups q = tid, tid + NT, ...; kQ of them and
    // kC partials of each load before any is folded, so that the fold is not a chain
    // of L2 round trips.
    constexpr int kQ = 4, kC = 4;
    const int n4 = rows * (D / 4);
    for (int q0 = tid; q0 < n4; q0 += kQ * NT) {
      float M[kQ], L[kQ];
      float4 O[kQ];
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        M[k] = -INFINITY;
        L[k] = 0.f;
        O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (int c = c0; c <= c1; c += kC) {
        float2 ml[kC][kQ];
        float4 o[kC][kQ];
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            const int q = q0 + k * NT;
            ml[i][k] = make_float2(-INFINITY, 0.f);
            o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + i <= c1 && q < n4) {
              const size_t at =
                  (size_t)(c + i == c0 ? first : 2 * (c + i)) * kRows + q / (D / 4);
              ml[i][k] = __ldcg(p.part_ml + at);
              o[i][k] = __ldcg((const float4 *)(p.part_o + at * D) + q % (D / 4));
            }
          }
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            // (a partial that saw nothing is (-inf, 0, 0): weight 0)
            const float m = fmaxf(M[k], ml[i][k].x);
            const float a = tree_weight(M[k], m), f = tree_weight(ml[i][k].x, m);
            L[k] = L[k] * a + f * ml[i][k].y;
            O[k].x = O[k].x * a + f * o[i][k].x;
            O[k].y = O[k].y * a + f * o[i][k].y;
            O[k].z = O[k].z * a + f * o[i][k].z;
            O[k].w = O[k].w * a + f * o[i][k].w;
            M[k] = m;
          }
      }
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const int q = q0 + k * NT;
        if (q >= n4) continue;
        const float s = L[k] == 0.f ? 0.f : 1.f / L[k];
        float *out = tree_out(p, it.head, it.group * kRows + q / (D / 4));
        *((float4 *)out + q % (D / 4)) =
            make_float4(O[k].x * s, O[k].y * s, O[k].z * s, O[k].w * s);
      }
    }
    if (tid == 0) *counter = 0;
  }
  sync();
}

// Word `w` of the visibility mask of new row i of a sequence of T rows (bits
// from T on cleared); without masks row i sees rows 0 .. i.
__device__ __forceinline__ uint32_t tree_mask_word(const TreeParams &p, const TreeHead &t, int i,
                                                   int w) {
  uint32_t m;
  int last = t.T - 1;
  if (p.mask) {
    m = w < p.words ? __ldg(p.mask + (size_t)(t.q0 + i) * p.words + w) : 0u;
  } else {
    m = 0xffffffffu;
    last = i;
  }
  const int n = last + 1 - 32 * w;
  return n <= 0 ? 0u : n >= 32 ? m : m & ((1u << n) - 1u);
}

}  // namespace kvx
