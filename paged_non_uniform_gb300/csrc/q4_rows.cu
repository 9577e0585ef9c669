// q4_rows.cu -- rows of a cache as values: new rows quantised into the pages of a 4-bit
// cache, and rows of any cache read back from their slots.
//
// Quantisation of a group of 64 elements x: lo = min x (a bf16 number, so exact), step =
// bf16((max x - lo) / 15), code = min(15, rint((x - lo) / step)) in fp32 with IEEE division;
// codes 0 where step is 0. A group with a non-finite element, or whose range is not finite,
// gets step 0 and lo NaN, so that all of it reads as NaN. Eight lanes hold a group,
// eight elements (a 16-byte load, a 4-byte word of codes) each; minimum and maximum
// meet in three shuffles. Memory bounds both kernels.
#include <math.h>

#include "ptx.cuh"
#include "window.h"

namespace kvx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t pool_rows(const CacheDev &c, int grp) {
  return c.grp[grp].pages * c.grp[grp].size * c.P;
}

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
  const float2 a = unpack_bf16(x.x), b = unpack_bf16(x.y), c = unpack_bf16(x.z), d = unpack_bf16(x.w);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}

struct Quantised {
  uint32_t codes, params;  // (lo << 16 | step, of the group)
};
// This lane's eight elements of its group; eight neighbouring lanes hold one.
__device__ __forceinline__ Quantised quantise(const uint4 &x) {
  float f[8];
  unpack8(x, f);
  float lo = f[0], hi = f[0];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
    finite = finite && isfinite(f[i]);
  }
#pragma unroll
  for (int w = 1; w < 8; w <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, w));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, w));
    finite = __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, w) && finite;
  }
  const float range = hi - lo;
  if (!finite || !isfinite(range)) return {0u, 0x7fc00000u};
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
  const float step = __bfloat162float(sb);
  uint32_t codes = 0;
  if (step > 0.f)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(15.f, rintf(__fdiv_rn(f[i] - lo, step)));
      codes |= (uint32_t)c << (4 * i);
    }
  return {codes, pack_bf16(step, lo)};
}

// One lane per eight elements of a (row, head), K and V together.
template <int D>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;  // of a row
  pdl_wait();
  const CacheDev &c = p.c;
  const int stated = p.q_start[c.B], rows = min(stated, p.max_rows);
  if ((stated < 0 || stated > p.max_rows) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  if (rows <= 0) return;
  const int64_t total = (int64_t)rows * c.Hkv * kLanes;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  // whole warps stay in the loop: lanes meet in shuffles
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); i0 < total; i0 += step) {
    const int64_t i = i0 + (threadIdx.x & 31);
    const bool in = i < total;
    const int64_t rh = in ? i / kLanes : 0;
    const int w = (int)(threadIdx.x % kLanes);  // the row's word
    const int64_t r = rh / c.Hkv;
    const int h = (int)(rh - r * c.Hkv);
    const int64_t slot = in ? p.slots[rh] : -1;
    const int grp = c.head_grp[h];
    const bool have = slot >= 0 && slot < pool_rows(c, grp);
    if (!have && slot != -1 && w == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (have) {
      const int64_t src = (int64_t)h * (D * 2) + w * 16;
      kx = *(const uint4 *)(p.k + r * p.k_stride + src);
      vx = *(const uint4 *)(p.v + r * p.v_stride + src);
    }
    const Quantised k = quantise(kx), v = quantise(vx);
    if (!have) continue;
    const int at = D == 128 ? 2 * (w & 7) + (w >> 3) : w;
    const int64_t co = q4_codes(c, slot) + at * 4, po = q4_params(c, slot) + (w >> 3) * 4;
    *(uint32_t *)(c.grp[grp].k + co) = k.codes;
    *(uint32_t *)(c.grp[grp].v + co) = v.codes;
    if ((w & 7) == 0) {
      *(uint32_t *)(c.grp[grp].k + po) = k.params;
      *(uint32_t *)(c.grp[grp].v + po) = v.params;
    }
  }
  __threadfence();
}

// Eight values of a 4-bit row as bf16.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t params) {
  const float2 s = unpack_bf16(params);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_bf16(fmaf(s.x, (float)(codes >> (8 * i) & 15u), s.y),
                     fmaf(s.x, (float)(codes >> (8 * i + 4) & 15u), s.y));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// out[r][h] = pool_h[slots[r][h]] for K and V; one lane per 16 bytes of a value row.
template <bool kQ4>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheDev &c = p.c;
  const int lanes = c.row_bytes >> 4;
  const int stated = p.q_start[c.B], rows = min(stated, p.max_rows);
  if ((stated < 0 || stated > p.max_rows) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  if (rows <= 0) return;
  const int64_t total = (int64_t)rows * c.Hkv * lanes;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t rh = i / lanes;
    const int w = (int)(i - rh * lanes);
    const int64_t r = rh / c.Hkv;
    const int h = (int)(rh - r * c.Hkv);
    const int64_t slot = p.slots[rh];
    const CacheGroup &g = c.grp[c.head_grp[h]];
    if (slot < 0 || slot >= pool_rows(c, c.head_grp[h])) {
      if (slot != -1 && w == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
      continue;
    }
    uint4 k, v;
    if constexpr (kQ4) {
      const int at = c.D == 128 ? 2 * (w & 7) + (w >> 3) : w;
      const int64_t co = q4_codes(c, slot) + at * 4, po = q4_params(c, slot) + (w >> 3) * 4;
      const uint32_t kc = *(const uint32_t *)(g.k + co), kp = *(const uint32_t *)(g.k + po);
      const uint32_t vc = *(const uint32_t *)(g.v + co), vp = *(const uint32_t *)(g.v + po);
      k = values8(kc, kp);
      v = values8(vc, vp);
    } else {
      k = *(const uint4 *)(g.k + slot * c.row_bytes + w * 16);
      v = *(const uint4 *)(g.v + slot * c.row_bytes + w * 16);
    }
    const int64_t dst = (int64_t)h * c.row_bytes + w * 16;
    *(uint4 *)(p.k + r * p.k_stride + dst) = k;
    *(uint4 *)(p.v + r * p.v_stride + dst) = v;
  }
}

// A dependent launch over `lanes` 16-byte pieces, at most 32 blocks per SM.
template <class Params>
cudaError_t launch(void (*kernel)(Params), const Params &p, int64_t lanes, cudaStream_t st) {
  const int64_t blocks = (lanes + kThreads - 1) / kThreads, most = 32 * 152;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_q4_append(const AppendParams &p, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int64_t lanes = (int64_t)p.max_rows * p.c.Hkv * (p.c.D / 8);
  return p.c.D == 128 ? launch(q4_append_kernel<128>, p, lanes, st)
                      : launch(q4_append_kernel<64>, p, lanes, st);
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int64_t lanes = (int64_t)p.max_rows * p.c.Hkv * (p.c.row_bytes >> 4);
  return p.q4 ? launch(read_kernel<true>, p, lanes, st) : launch(read_kernel<false>, p, lanes, st);
}

}  // namespace kvx
