// window_weigh.cu -- accumulates the attention weights of cached tokens.
//
// w_t = (t < n ? w_t : 0) + sum over the rows r (new rows and query heads of the KV head) of
// 2^(x_rt - M_r) / L_r, from the scores x that the attention launch left and the row's
// maximum and sum, which are only known when all of a head's pieces are merged: hence
// the stored scores and a launch of its own. A token's rows are added in a fixed order, so
// nothing depends on timing. Blocks take equal parts of all heads' visited tiles.
// Recomputing the scores instead would read K again, 256 bytes a token (bf16, D 128), where storing and reading them
// is 8 a query row: 32 for a decode step of four heads. From 32 rows a head on that reason is gone (32 rows of
// four heads: 1024 bytes); the form that would recompute them is not built. Measured on one GB300, in a graph: 16
// sequences of 8k to 32k, one row of 4 heads, 89 us with weights, 71 without (this launch by itself 17); 4 sequences,
// 32 rows (200 MB of scores) 253 and 155 (60).
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

// kLanes lanes share a token: four rows of every row group each (a 16-byte load), so that a
// token's scores are one stretch of memory to neighbouring lanes; several tokens in flight.
// Measured, the call in a graph: a decode step (one lane a token) with two tokens in flight and four
// blocks an SM 84.7 us, four tokens 86.2, four and no more blocks 89.2; 32 rows voting (eight
// lanes) 258, 270, 249. Lanes: as many as a row group has fours of rows; 8 rows with two, four and eight lanes
// 105, 117, 141 us, 16 rows with four and eight 127, 154 (16 sequences of 8k to 32k).
template <int kLanes>
__global__ void __launch_bounds__(kThreads, kLanes == 1 ? 4 : 3) weigh_kernel(const __grid_constant__ WindowParams p,
                                                         int group_tokens) {
  constexpr int kBatch = kLanes == 1 ? 2 : 4, kTokens = kThreads / kLanes;  // tokens of a block's step
  __shared__ Smem sm;
  extern __shared__ float2 row[];  // the head's rows: (maximum, 1 / sum)
  const int tid = threadIdx.x, sub = tid % kLanes;
  pdl_launch_dependents();
  pdl_wait();
  // After a wait that ran out the scores of the stages left out are an earlier call's: the weights,
  // which are the sum of all calls, stay as they are.
  if (*(volatile const uint32_t *)p.status & KVX_DEV_TIMEOUT) return;
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
    const int per = group_tokens * p.c.g, end = it.t1 * kTile;
    // (warps stay whole: lanes of a token meet in shuffles)
    for (int i0 = it.t0 * kTile; i0 < end; i0 += kBatch * kTokens) {
      int t[kBatch];
      float w[kBatch], old[kBatch];
      float *at[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * kTokens + tid / kLanes;
        t[b] = i < end ? window_tile(hd, i / kTile) * kTile + i % kTile : INT32_MAX;
        w[b] = 0.f;
        at[b] = nullptr;
        if (t[b] < hd.n + hd.T && sub == 0) {
          const int page = table[t[b] >> p.c.lgP];
          // (a page outside the pool was reported by the attention launch)
          if (page >= 0 && page < grp.pages)
            at[b] = p.weights[gi] + pool_row(p.c, grp, page, rank, t[b] & (p.c.P - 1));
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) old[b] = at[b] && t[b] < hd.n ? *at[b] : 0.f;
      for (int r0 = 0, group = 0; r0 < rows; r0 += per, ++group) {
        const int k = min(per, rows - r0) - 4 * sub;  // rows left from this lane's first
        const float2 *rw = row + r0 + 4 * sub;
        float4 x[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (k > 0 && t[b] < hd.n + hd.T)
            x[b] = __ldcg((const float4 *)(window_scores(p, hd, group, i0 + b * kTokens + tid / kLanes) + 4 * sub));
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (k <= 0 || t[b] >= hd.n + hd.T) continue;
          const float v[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < k && v[e] != -INFINITY) w[b] = fmaf(ex2(v[e] - rw[e].x), rw[e].y, w[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
#pragma unroll
        for (int sh = 1; sh < kLanes; sh <<= 1) w[b] += __shfl_xor_sync(0xffffffffu, w[b], sh);
        if (at[b]) *at[b] = old[b] + w[b];
      }
    }
  }
}

template <int kLanes>
cudaError_t launch_lanes(const WindowParams &p, int blocks, cudaStream_t st) {
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weigh_kernel<kLanes>, w, (int)p.group_tokens);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh(const WindowParams &p, int blocks, cudaStream_t st) {
  const int n = p.score_rows / 4;  // lanes with work
  if (n <= 1) return launch_lanes<1>(p, 2 * blocks, st);
  if (n <= 2) return launch_lanes<2>(p, 2 * blocks, st);
  if (n <= 4) return launch_lanes<4>(p, 2 * blocks, st);
  return launch_lanes<8>(p, 2 * blocks, st);
}

}  // namespace kvx
