// window_simt.cu -- attention with a sliding window and sink tokens over a paged
// fp32 cache, on the CUDA cores.
//
// out[row] = sum_t softmax(scale * <q_row, k_t>)_t v_t over the keys that the row sees
// (window_split.cuh), in one pass over the visited tiles of 64 keys per group of 32 query
// rows (running maximum and sum in fp32). K and V tiles are gathered from their
// pages into shared memory; each thread computes a 4 x 4 block of scores and
// accumulates 4 rows x D/16 dims of the output. Keys that no row of the item sees are not read.
// In a tile that some row sees only in part, unseen scores become -inf; where such a tile's V is
// not all finite, a separate path skips what a row does not see instead of multiplying it by
// zero, so that NaN and infinities in unseen rows have no influence.
// Latency bounds short inputs: two sequences of 37 to 100 tokens 16.5 us with the merge, in a graph (18.6 when
// every edge tile took the separate path). Longer ones are bound by the multiplications, 32 rows
// whatever the call has: 16 sequences of 8k to 32k, windows of 4096 in six of eight heads, 945 MB, one row of 4
// heads 887 us (1.1 TB/s), eight rows 990 us.
#include <math.h>

#include "window_split.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = kWindowTile;
constexpr int kRows = 32;
constexpr int kMinTiles = 2;

template <int D>
struct Smem {
  float q[kRows][D + 4];
  float k[kTile][D + 4];
  float v[kTile][D + 4];
  float p[kRows][kTile + 4];
  uint32_t seen[kRows][2];  // visible keys of the tile, by row
  int64_t warp_sum[kThreads / 32];
  TreeRange range;
};

template <int D>
__global__ void __launch_bounds__(kThreads, kWindowBlocksPerSm)
    window_simt_kernel(const __grid_constant__ WindowParams p) {
  extern __shared__ float4 smem_raw[];
  Smem<D> &sm = *(Smem<D> *)smem_raw;
  constexpr int CPR = D / 4;  // 4-element chunks of a row
  constexpr int ND = D / 64;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  pdl_launch_dependents();
  pdl_wait();
  const TreeRange range = tree_range<kThreads, kTile>(p, kMinTiles, sm.warp_sum, &sm.range);
  TreeCursor<kTile> cur(p, range);
  TreeItem it;
  bool any = false;
  while (cur.next(p, it)) {
    any = true;
    const TreeHead &hd = it.head;
    const CacheGroup &grp = p.c.grp[p.c.head_grp[hd.h]];
    const Window win = window_of(hd);
    const int rank = p.c.head_row[hd.h], g = p.c.g, P = p.c.P;
    const int32_t *table = grp.table + (size_t)hd.b * grp.stride;
    const int i0 = tree_first(p, it), rows = tree_rows(p, it);
    const int i1 = i0 + tree_div_g(p, rows - 1);
    __syncthreads();  // the item before is done with shared memory
    for (int i = tid; i < kRows * CPR; i += kThreads) {
      const int r = i / CPR, c = i - r * CPR;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int nr = tree_div_g(p, r), j = r - nr * g;
        x = *(const float4 *)(p.q + (size_t)(hd.q0 + i0 + nr) * p.q_stride +
                              ((size_t)hd.h * g + j) * (D * 4) + c * 16);
      }
      *(float4 *)&sm.q[r][c * 4] = x;
    }
    float m[4], l[4], o[4][ND][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[a][d][0] = o[a][d][1] = o[a][d][2] = o[a][d][3] = 0.f;
    }
    for (int tile = it.t0; tile < it.t1; ++tile) {
      const int t0 = window_tile(hd, tile) * kTile, valid = min(kTile, hd.n + hd.T - t0);
      const bool edge = !window_all_seen(win, hd.n, i0, i1, t0, kTile);
      bool odd = false;  // infinities or NaN in V (or sums past fp32's range)
      __syncthreads();   // the tile before is consumed
      for (int i = tid; i < kTile * CPR; i += kThreads) {
        const int t = i / CPR, c = i - t * CPR;
        float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
        const int tok = t0 + t;
        // (what no row sees is not read)
        if (t < valid && (!edge || window_any_sees(win, hd.n, i0, i1, tok))) {
          const int page = table[tok >> p.c.lgP];
          if (page >= 0 && page < grp.pages) {
            const int64_t at = pool_row(p.c, grp, page, rank, tok & (P - 1)) * (D * 4) + c * 16;
            dk = *(const float4 *)(grp.k + at);
            dv = *(const float4 *)(grp.v + at);
            odd |= !(fabsf(dv.x) + fabsf(dv.y) + fabsf(dv.z) + fabsf(dv.w) < INFINITY);
          } else if (c == 0) {
            atomicOr(p.status, KVX_DEV_BAD_PAGE);
          }
        }
        *(float4 *)&sm.k[t][c * 4] = dk;
        *(float4 *)&sm.v[t][c * 4] = dv;
      }
      if (edge && tid < 2 * kRows) {
        // visible keys of row r, word w: bits [32w, 32w + 32) of the tile
        const int r = tid >> 1, w = tid & 1;
        uint32_t bits = 0;
        if (r < rows) bits = window_bits(win, hd.n + i0 + tree_div_g(p, r), t0 + 32 * w);
        sm.seen[r][w] = bits;
      }
      const bool skip = __syncthreads_or(edge && odd);
      float s[4][4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[a][b] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 qa[4], kb[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) qa[a] = *(const float4 *)&sm.q[ty * 4 + a][d];
#pragma unroll
        for (int b = 0; b < 4; ++b) kb[b] = *(const float4 *)&sm.k[tx + 16 * b][d];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            s[a][b] = fmaf(qa[a].x, kb[b].x, s[a][b]);
            s[a][b] = fmaf(qa[a].y, kb[b].y, s[a][b]);
            s[a][b] = fmaf(qa[a].z, kb[b].z, s[a][b]);
            s[a][b] = fmaf(qa[a].w, kb[b].w, s[a][b]);
          }
      }
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float mx = m[a];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int t = tx + 16 * b;
          float x = s[a][b] * p.scale_log2;
          if (edge && !((sm.seen[ty * 4 + a][t >> 5] >> (t & 31)) & 1u)) x = -INFINITY;
          s[a][b] = x;
          mx = fmaxf(mx, x);
          if (p.scores && ty * 4 + a < rows)
            window_scores(p, hd, it.group, (int64_t)tile * kTile + t)[ty * 4 + a] = x;
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float ref = mx == -INFINITY ? 0.f : mx;  // a row that has seen nothing
        const float al = tree_weight(m[a], ref);
        m[a] = mx;
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float e = ex2(s[a][b] - ref);
          sm.p[ty * 4 + a][tx + 16 * b] = e;
          sum += e;
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[a] = l[a] * al + sum;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          o[a][d][0] *= al;
          o[a][d][1] *= al;
          o[a][d][2] *= al;
          o[a][d][3] *= al;
        }
      }
      __syncwarp();  // a row's scores are written and read by one half-warp
      if (!skip) {
#pragma unroll 2
        for (int t = 0; t < kTile; t += 4) {
          float pa[4][4];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float4 x = *(const float4 *)&sm.p[ty * 4 + a][t];
            pa[a][0] = x.x;
            pa[a][1] = x.y;
            pa[a][2] = x.z;
            pa[a][3] = x.w;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const float4 vv = *(const float4 *)&sm.v[t + u][tx * 4 + 64 * d];
#pragma unroll
              for (int a = 0; a < 4; ++a) {
                o[a][d][0] = fmaf(pa[a][u], vv.x, o[a][d][0]);
                o[a][d][1] = fmaf(pa[a][u], vv.y, o[a][d][1]);
                o[a][d][2] = fmaf(pa[a][u], vv.z, o[a][d][2]);
                o[a][d][3] = fmaf(pa[a][u], vv.w, o[a][d][3]);
              }
            }
        }
      } else {
        for (int t = 0; t < valid; ++t) {
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (!((sm.seen[ty * 4 + a][t >> 5] >> (t & 31)) & 1u)) continue;
            const float x = sm.p[ty * 4 + a][t];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const float4 vv = *(const float4 *)&sm.v[t][tx * 4 + 64 * d];
              o[a][d][0] = fmaf(x, vv.x, o[a][d][0]);
              o[a][d][1] = fmaf(x, vv.y, o[a][d][1]);
              o[a][d][2] = fmaf(x, vv.z, o[a][d][2]);
              o[a][d][3] = fmaf(x, vv.w, o[a][d][3]);
            }
          }
        }
      }
    }
    const bool whole = tree_whole(it);
    const int slot = whole ? 0 : tree_slot(it);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = ty * 4 + a;
      if (r >= rows) continue;
      float *dst;
      float f = 1.f;
      if (whole) {
        dst = tree_out(p, hd.q0 + i0, hd.h, r);
        f = l[a] == 0.f ? 0.f : 1.f / l[a];
        if (p.row_ml && tx == 0)
          *tree_row_ml(p, tree_ml_row(p, hd.b, i0), hd.h, r) = make_float2(m[a], l[a]);
      } else {
        const size_t at = (size_t)slot * kRows + r;
        dst = p.part_o + at * D;
        if (tx == 0) p.part_ml[at] = make_float2(m[a], l[a]);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *(float4 *)(dst + tx * 4 + 64 * d) =
            make_float4(o[a][d][0] * f, o[a][d][1] * f, o[a][d][2] * f, o[a][d][3] * f);
    }
  }
  if (tid == 0) tree_describe(p, range, any ? &it : nullptr);
}

template <int D>
cudaError_t launch_d(const WindowParams &p, int blocks, cudaStream_t st) {
  const int bytes = (int)sizeof(Smem<D>);
  static int8_t done[64];
  cudaError_t e = raise_smem_limit(done, (const void *)window_simt_kernel<D>, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, window_simt_kernel<D>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int window_simt_rows() { return kRows; }

cudaError_t launch_window_simt(const WindowParams &p, int blocks, cudaStream_t st) {
  return p.c.D == 128 ? launch_d<128>(p, blocks, st) : launch_d<64>(p, blocks, st);
}

}  // namespace kvx
