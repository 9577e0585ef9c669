// tree_merge.cu -- folds the partials of row groups that tree attention cut over
// several blocks.
//
// out[row] = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over the partials c of the
// row group in block order (M the largest m_c), so the result does not depend on
// timing. One warp takes a row: lanes hold the partials' weights, then each lane one
// float4 (D = 128) or float2 of the row, four partials' loads in flight: more of them
// cost registers, and with those the blocks that start while attention still runs. Figures
// for one sequence of 2k / 16 of 8k to 32k, attention and merge: two rows a warp and eight
// loads 17.7 / 85.3 us, one row and eight 15.6 / 85.2, one row and four 16.0 / 83.2, 16
// loads 16.1 / 87.9.
// Why a launch of its own: the block that finishes a head last used to fold it inside
// the attention launch. With eight heads cut in seven pieces of 64 rows that took 20 us,
// because a few blocks folded several heads one after the other, in code that no cache
// held yet; spread over all SMs it is one L2 round trip for the weights and one for
// the rows. The launch overlaps the attention kernel's tail (programmatic dependent).
#include "tree_split.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;  // elements of a lane
  pdl_launch_dependents();
  pdl_wait();
  const TreeSplit s = p.split[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);
  if (r < s.rows) {
    // row r of partial c: the first is its block's last piece, the others are their
    // blocks' first
    auto at = [&](int c) {
      return (size_t)(2 * ((int)blockIdx.y + c) + (c == 0 ? 1 : 0)) * p.group_rows + r;
    };
    float M = -INFINITY;
    for (int c = lane; c < s.parts; c += 32) M = fmaxf(M, __ldcg(p.part_ml + at(c)).x);
#pragma unroll
    for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int c0 = 0; c0 < s.parts; c0 += 32) {
      float f = 0.f;
      if (c0 + lane < s.parts) {
        const float2 ml = __ldcg(p.part_ml + at(c0 + lane));
        f = tree_weight(ml.x, M);
        L = fmaf(f, ml.y, L);
      }
      const int n = min(32, s.parts - c0);
      for (int c = 0; c < n; c += 4) {
        alignas(16) float v[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float *src = p.part_o + at(c0 + c + u) * D + lane * E;
          if (c + u >= n) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
          } else if constexpr (E == 4) {
            *(float4 *)v[u] = __ldcg((const float4 *)src);
          } else {
            *(float2 *)v[u] = __ldcg((const float2 *)src);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float w = __shfl_sync(0xffffffffu, f, (c + u) & 31);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
        }
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
    const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing
    if (p.row_ml && lane == 0)
      *tree_row_ml(p, p.split_row[blockIdx.y], s.h, r) = make_float2(M, L);
    float *out = tree_out(p, s.row0, s.h, r) + lane * E;
    if constexpr (E == 4)
      *(float4 *)out = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    else
      *(float2 *)out = make_float2(acc[0] * inv, acc[1] * inv);
  }
}

}  // namespace

cudaError_t launch_tree_merge(const TreeParams &p, int blocks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int rows = p.group_rows < p.max_q * p.c.g ? p.group_rows : p.max_q * p.c.g;
  cfg.gridDim = dim3((unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock), (unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.c.D == 128 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<128>, p)
                                     : cudaLaunchKernelEx(&cfg, tree_merge_kernel<64>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvx
