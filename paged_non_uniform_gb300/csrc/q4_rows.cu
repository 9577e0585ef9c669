// q4_rows.cu -- rows of a cache as values: new rows quantised into the pages of a 4-bit
// cache, and rows of any cache read back from their slots.
//
// Quantisation of a group of 64 elements x: lo = min x (a bf16 number, so exact), step =
// bf16((max x - lo) / 15), code = min(15, rint((x - lo) / step)) in fp32; codes 0 where step is
// 0. A group with a non-finite element, or whose range is not finite, gets step 0 and lo NaN, so that all of it reads as NaN. Four lanes hold a group,
// sixteen elements (32 bytes in, two 4-byte words of codes out) each; minimum and maximum
// meet in two shuffles.
// Measured on one GB300: 43k rows of 8 heads quantised in 75 us (230 MB; instructions bound it: with
// eight elements a lane, 94 us, 74 % of the issue slots were taken), read back in 47 us (230 MB, 4.9 TB/s).
// bf16 rows of the same shape are read back in 66 us (352 MB, 5.3 TB/s), fp32 in 117 (701 MB, 6.0 TB/s).
#include <math.h>

#include "ptx.cuh"
#include "window.h"

namespace kvx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t pool_rows(const CacheDev &c, int grp) {
  return c.grp[grp].pages * c.grp[grp].size * c.P;
}

struct Quantised {
  uint32_t codes[2], params;  // two words; (lo << 16 | step, of the group)
};
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *(const __nv_bfloat162 *)&x; }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *(const uint32_t *)&x; }
// fl(range / 15) to bf16: the product with a rounded 1 / 15 is within two units in the last place of
// the quotient, which matters only next to the middle of two bf16 numbers.
__device__ __forceinline__ __nv_bfloat16 step_of(float range) {
  float q = range * (1.f / 15.f);
  if (((__float_as_uint(q) + 4u) & 0xffffu) - 0x8000u <= 8u || q < 0x1p-100f) q = __fdiv_rn(range, 15.f);
  return __float2bfloat16_rn(q);
}
// Settles an element whose estimated code c leaves e, half a step or nearly (quantise).
__device__ __noinline__ float settle(float c, float e, float past, float step) {
  const float middle = c + copysignf(0.5f, e);
  // half a unit in the last place of the middle, twice
  const float near = __uint_as_float((__float_as_uint(middle) & 0x7f800000u) - (23u << 23)) * step;
  return past > near || (past >= -near && ((int)c & 1)) ? 2.f * middle - c : c;
}

// This lane's sixteen elements of its group; four neighbouring lanes hold one.
__device__ __forceinline__ Quantised quantise(const uint4 (&x)[2]) {
  // (least, -greatest) of the group; NaN stays NaN
  __nv_bfloat162 a = as_bf2(x[0].x), b = a;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a = __hmin2_nan(__hmin2_nan(a, as_bf2(x[i].x)), as_bf2(x[i].y));
    a = __hmin2_nan(__hmin2_nan(a, as_bf2(x[i].z)), as_bf2(x[i].w));
    b = __hmax2_nan(__hmax2_nan(b, as_bf2(x[i].x)), as_bf2(x[i].y));
    b = __hmax2_nan(__hmax2_nan(b, as_bf2(x[i].z)), as_bf2(x[i].w));
  }
  b = __hneg2(b);
  a = __hmin2_nan(__lows2bfloat162(a, b), __highs2bfloat162(a, b));
#pragma unroll
  for (int w = 1; w < 4; w <<= 1) a = __hmin2_nan(a, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(a), w)));
  const float lo = __low2float(a), range = -__high2float(a) - lo;
  if (!isfinite(range)) return {{0u, 0u}, 0x7fc00000u};
  const __nv_bfloat16 sb = step_of(range);
  const float step = __bfloat162float(sb);
  Quantised q = {{0u, 0u}, pack_bf16(step, lo)};
  // rint(fl(d / step)) without the division: c, the nearest integer to an estimate of the
  // quotient, and e = d - c * step, exact in one multiply-add. Where 2 |e| is below step, c it
  // is. Else d lies past the middle between c and its neighbour on e's side (the estimate was
  // off), or so near it that the quotient would be rounded to it: then the even one of the two.
  const bool usual = step >= 0x1p-120f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(step));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16(i == 0 ? x[k].x : i == 1 ? x[k].y : i == 2 ? x[k].z : x[k].w);
      f[2 * i] = v.x - lo;
      f[2 * i + 1] = v.y - lo;
    }
    if (usual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float c = fmaf(f[i], r, 12582912.f) - 12582912.f;  // 1.5 * 2^23
        const float e = fmaf(-c, step, f[i]), past = fmaf(2.f, fabsf(e), -step);
        if (past > -0x1p-20f * step) c = settle(c, e, past, step);
        f[i] = c;
      }
      const float l = fmaf(fmaf(fmaf(f[3], 16.f, f[2]), 16.f, f[1]), 16.f, f[0]);
      const float h = fmaf(fmaf(fmaf(f[7], 16.f, f[6]), 16.f, f[5]), 16.f, f[4]);
      q.codes[k] = __byte_perm(__float_as_uint(l + 8388608.f), __float_as_uint(h + 8388608.f), 0x5410);
    } else if (step > 0.f) {
      for (int i = 0; i < 8; ++i)
        q.codes[k] |= (uint32_t)fminf(15.f, rintf(__fdiv_rn(f[i], step))) << (4 * i);
    }
  }
  return q;
}

// Steps through the (row, head) pairs of a call, `step` pairs at a time, without dividing.
struct Pairs {
  int64_t rh;    // row * Hkv + head
  int32_t r, h;  // (rows fit in 30 bits)
  int32_t dr, dh;
  int64_t step;
  __device__ __forceinline__ Pairs(int64_t first, int64_t step_, int Hkv) : rh(first), step(step_) {
    r = (int32_t)(first / Hkv);
    h = (int32_t)(first - (int64_t)r * Hkv);
    dr = (int32_t)(step_ / Hkv);
    dh = (int32_t)(step_ - (int64_t)dr * Hkv);
  }
  __device__ __forceinline__ void next(int Hkv) {
    rh += step;
    r += dr;
    h += dh;
    if (h >= Hkv) h -= Hkv, ++r;
  }
};

// One lane per sixteen elements of a (row, head), K and V together (with eight, what a lane does
// once took as long as its elements).
template <int D>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16;  // of a row
  pdl_wait();
  const CacheDev &c = p.c;
  const int stated = p.q_start[c.B], rows = min(stated, p.max_rows);
  if ((stated < 0 || stated > p.max_rows) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  if (rows <= 0) return;
  const int64_t total = (int64_t)rows * c.Hkv;
  const int l = (int)(threadIdx.x % kLanes);  // words 2l and 2l + 1 of the row
  const int at = D == 128 ? 4 * (l & 3) + (l >> 2) : 2 * l, next = D == 128 ? 2 : 1;
  // (lanes meet in shuffles: whole warps stay in the loop, a warp's first pair decides)
  const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int64_t lead = ((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31)) / kLanes;
  Pairs q(first, (int64_t)gridDim.x * (kThreads / kLanes), c.Hkv);
  for (int64_t i = lead; i < total; i += q.step, q.next(c.Hkv)) {
    uint4 kx[2] = {}, vx[2] = {};
    int64_t slot = -1;
    if (q.rh < total) {
      slot = p.slots[q.rh];
      const int64_t src = (int64_t)q.h * (D * 2) + l * 32;
      const uint4 *ks = (const uint4 *)(p.k + q.r * p.k_stride + src);
      const uint4 *vs = (const uint4 *)(p.v + q.r * p.v_stride + src);
      kx[0] = ks[0], kx[1] = ks[1], vx[0] = vs[0], vx[1] = vs[1];
    }
    const Quantised k = quantise(kx), v = quantise(vx);
    const CacheGroup &g = c.grp[c.head_grp[q.h]];
    if (slot < 0 || slot >= pool_rows(c, c.head_grp[q.h])) {
      if (slot != -1 && l == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t co = q4_codes(c, slot) + at * 4, po = q4_params(c, slot) + (l >> 2) * 4;
    *(uint32_t *)(g.k + co) = k.codes[0];
    *(uint32_t *)(g.k + co + next * 4) = k.codes[1];
    *(uint32_t *)(g.v + co) = v.codes[0];
    *(uint32_t *)(g.v + co + next * 4) = v.codes[1];
    if ((l & 3) == 0) {
      *(uint32_t *)(g.k + po) = k.params;
      *(uint32_t *)(g.v + po) = v.params;
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

// out[r][h] = pool_h[slots[r][h]] for K and V; one lane per 16 bytes of a value row (kLanes a
// row), two (row, head) pairs in flight.
template <bool kQ4, int kLanes>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheDev &c = p.c;
  const int stated = p.q_start[c.B], rows = min(stated, p.max_rows);
  if ((stated < 0 || stated > p.max_rows) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  if (rows <= 0) return;
  const int64_t total = (int64_t)rows * c.Hkv;
  const int w = (int)(threadIdx.x % kLanes);
  const int at = kLanes == 16 ? 2 * (w & 7) + (w >> 3) : w;  // (4 bits: D / 8 lanes)
  Pairs q(((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes,
          (int64_t)gridDim.x * (kThreads / kLanes), c.Hkv);
  while (q.rh < total) {
    int64_t slot[2];
    int32_t r[2], h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      slot[u] = q.rh < total ? p.slots[q.rh] : -1;
      r[u] = q.r;
      h[u] = q.h;
      q.next(c.Hkv);
    }
    uint4 k[2], v[2];
    uint32_t kp[2], vp[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const CacheGroup &g = c.grp[c.head_grp[h[u]]];
      if (slot[u] < 0 || slot[u] >= pool_rows(c, c.head_grp[h[u]])) {
        if (slot[u] != -1 && w == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
        slot[u] = -1;
      } else if constexpr (kQ4) {
        const int64_t co = q4_codes(c, slot[u]) + at * 4, po = q4_params(c, slot[u]) + (w >> 3) * 4;
        k[u].x = *(const uint32_t *)(g.k + co), kp[u] = *(const uint32_t *)(g.k + po);
        v[u].x = *(const uint32_t *)(g.v + co), vp[u] = *(const uint32_t *)(g.v + po);
      } else {
        k[u] = *(const uint4 *)(g.k + slot[u] * (kLanes * 16) + w * 16);
        v[u] = *(const uint4 *)(g.v + slot[u] * (kLanes * 16) + w * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (slot[u] < 0) continue;
      const int64_t dst = (int64_t)h[u] * (kLanes * 16) + w * 16;
      *(uint4 *)(p.k + r[u] * p.k_stride + dst) = kQ4 ? values8(k[u].x, kp[u]) : k[u];
      *(uint4 *)(p.v + r[u] * p.v_stride + dst) = kQ4 ? values8(v[u].x, vp[u]) : v[u];
    }
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
  const int64_t lanes = (int64_t)p.max_rows * p.c.Hkv * (p.c.D / 16);
  return p.c.D == 128 ? launch(q4_append_kernel<128>, p, lanes, st)
                      : launch(q4_append_kernel<64>, p, lanes, st);
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int64_t lanes = (int64_t)p.max_rows * p.c.Hkv * (p.c.row_bytes >> 4);
  if (p.q4)
    return p.c.D == 128 ? launch(read_kernel<true, 16>, p, lanes, st) : launch(read_kernel<true, 8>, p, lanes, st);
  switch (p.c.row_bytes) {
    case 512: return launch(read_kernel<false, 32>, p, lanes, st);
    case 256: return launch(read_kernel<false, 16>, p, lanes, st);
    default: return launch(read_kernel<false, 8>, p, lanes, st);
  }
}

}  // namespace kvx
