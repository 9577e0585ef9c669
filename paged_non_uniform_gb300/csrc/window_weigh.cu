// window_weigh.cu -- accumulates the attention weights of cached tokens.
//
// w_t = (t < n ? w_t : 0) + sum over the rows r (new rows and query heads of the KV head) of
// 2^(x_rt - M_r) / L_r, from the scores x that the attention launch left and the row's
// maximum and sum, which are only known when all of a head's pieces are merged: hence
// the stored scores and a launch of its own. A thread owns a token and adds its rows in
// order, so nothing depends on timing. Blocks take equal parts of all heads' visited tiles.
#include <math.h>

#include "window_split.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kWindowTile;

struct Smem {
  int64_t warp_sum[kThreads / 32];
  TreeRange range;
};

__global__ void __launch_bounds__(kThreads) weigh_kernel(const __grid_constant__ WindowParams p,
                                                         int group_tokens) {
  __shared__ Smem sm;
  extern __shared__ float2 row[];  // the head's rows: (maximum, 1 / sum)
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  // (the params count a head as one row group here; group_tokens are the attention launch's)
  const TreeRange range = tree_range<kThreads, kTile>(p, 1, sm.warp_sum, &sm.range);
  TreeCursor<kTile> cur(p, range);
  TreeItem it;
  while (cur.next(p, it)) {
    const TreeHead &hd = it.head;
    const int gi = p.c.head_grp[hd.h], rank = p.c.head_row[hd.h], rows = hd.T * p.c.g;
    const CacheGroup &grp = p.c.grp[gi];
    const int32_t *table = grp.table + (size_t)hd.b * grp.stride;
    __syncthreads();  // the item before is done
    for (int r = tid; r < rows; r += kThreads) {
      const float2 ml = __ldcg(tree_row_ml(p, tree_ml_row(p, hd.b, 0), hd.h, r));
      row[r] = make_float2(ml.x, ml.y == 0.f ? 0.f : 1.f / ml.y);
    }
    __syncthreads();
    const int per = group_tokens * p.c.g;
    for (int i = it.t0 * kTile + tid; i < it.t1 * kTile; i += kThreads) {
      const int t = window_tile(hd, i / kTile) * kTile + i % kTile;
      if (t >= hd.n + hd.T) continue;
      float w = 0.f;
      for (int r0 = 0, group = 0; r0 < rows; r0 += per, ++group) {
        const float *x = window_scores(p, hd, group, i);
        const int k = min(per, rows - r0);
        for (int r = 0; r < k; ++r) {
          const float xr = __ldcg(x + r);
          if (xr != -INFINITY) w += ex2(xr - row[r0 + r].x) * row[r0 + r].y;
        }
      }
      const int page = table[t >> p.c.lgP];
      if (page < 0 || page >= grp.pages) continue;  // (reported by the attention launch)
      float *at = p.weights[gi] + pool_row(p.c, grp, page, rank, t & (p.c.P - 1));
      *at = t < hd.n ? *at + w : w;
    }
  }
}

}  // namespace

cudaError_t launch_weigh(const WindowParams &p, int blocks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.max_q * p.c.g * sizeof(float2);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  WindowParams w = p;
  w.group_tokens = p.max_q;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weigh_kernel, w, (int)p.group_tokens);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvx
