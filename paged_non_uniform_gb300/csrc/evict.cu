// evict.cu -- eviction of cached tokens by accumulated attention weight.
//
// A head with n cached tokens and a budget of m < n keeps its first f and last r tokens and,
// of those between, the m - f - r with the largest weights (equal weights: lower index first),
// in their order; kept token number i becomes token i.
//
// First launch: a cluster of blocks per head, each with a run of the head's tokens. Weights
// become 32-bit keys of the same order; four passes of 8-bit digits find the cut (histograms
// of the cluster's blocks are added through distributed shared memory), counts of the
// runs give every 64-token chunk its place. It leaves a list of units: chunk, tokens that
// stay, where they go.
// Second launch: blocks take units by ticket. A unit reads its rows, says so, waits until
// the units that hold its targets have read theirs (rows move towards the front, so those are
// earlier units of the head, which running blocks have taken before, and no unit waits
// before it has read), and writes. So a head moves on all SMs at once, in place, with
// one read and one write of every row that moves.
// Bounded by memory where much moves, by the latency of the passes where little does.
#include <math.h>

#include "ptx.cuh"
#include "window.h"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kEvictChunk;
constexpr int kKeys = 8192;  // keys of a block's run that are kept in shared memory
static_assert(kThreads == 4 * kChunk, "a step of the placing pass is four chunks");

// Order-preserving key: larger weight, larger key; -0 as 0; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

struct Head {
  int b, h, n, m, first, last;  // cached, kept; tokens kept at the front and from `last` on
  bool evict;
};

__device__ __forceinline__ Head load_head(const EvictParams &p, int bh, bool report) {
  Head hd;
  hd.b = bh / p.c.Hkv;
  hd.h = bh - hd.b * p.c.Hkv;
  hd.n = p.kv_len[bh];
  const int budget = p.budget[bh];
  const bool ok = hd.n >= 0 && hd.n <= p.c.grp[p.c.head_grp[hd.h]].tokens && budget >= 0;
  if (!ok && report) atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  hd.m = ok ? min(hd.n, budget) : hd.n;
  hd.evict = hd.m < hd.n;
  const int r = min(hd.m, p.recent);
  hd.first = min(hd.m - r, p.sinks);
  hd.last = hd.n - r;
  if (!ok) hd.n = hd.m = hd.first = hd.last = 0;
  return hd;
}

struct SelectSmem {
  uint32_t keys[kKeys];
  uint32_t hist[2][256];
  uint32_t total[256];
  uint32_t warp_sum[8];
  uint32_t count[2];  // keys of this block's run above the cut, equal to it
  uint32_t cut, left;  // digits found; keys still to take among those that share them
  uint32_t start;      // rank 0: the head's first unit
  uint32_t words[2][8];
};

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ SelectSmem sm;
  pdl_launch_dependents();
  pdl_wait();
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = (int)(blockIdx.x / C);
  const Head hd = load_head(p, bh, rank == 0 && tid == 0);
  const int gi = p.c.head_grp[hd.h], row = p.c.head_row[hd.h];
  const CacheGroup &grp = p.c.grp[gi];
  const int32_t *table = grp.table + (size_t)hd.b * grp.stride;
  const float *weights = p.weights[gi];
  const int chunks = (hd.n + kChunk - 1) / kChunk, per = (chunks + (int)C - 1) / (int)C;
  const int c_lo = min(chunks, (int)rank * per), c_hi = min(chunks, c_lo + per);
  const int t_lo = c_lo * kChunk, t_hi = min(hd.n, c_hi * kChunk);
  const int first_chunk = p.copy_weights ? 0 : hd.first / kChunk;
  const int units = hd.evict || p.copy_weights ? max(0, chunks - first_chunk) : 0;

  auto load_key = [&](int t) -> uint32_t {
    const int page = table[t >> p.c.lgP];
    if (page < 0 || page >= grp.pages) return 0u;
    return weight_key(weights[pool_row(p.c, grp, page, row, t & (p.c.P - 1))]);
  };
  auto key = [&](int t) -> uint32_t {
    return t - t_lo < kKeys ? sm.keys[t - t_lo] : load_key(t);
  };
  const int a_lo = max(t_lo, hd.first), a_hi = min(t_hi, hd.last);  // this run's part that competes
  if (rank == 0 && tid == 0) {
    sm.start = units ? atomicAdd(p.counters, (uint32_t)units) : 0u;
    sm.cut = 0;
  }
  uint32_t prefix = 0, left = 0;  // found digits; keys to take among those that share them
  if (hd.evict) {
    left = (uint32_t)(hd.m - hd.first - (hd.n - hd.last));
    for (int t = t_lo + tid; t < min(t_hi, t_lo + kKeys); t += kThreads) sm.keys[t - t_lo] = load_key(t);
  }
  // left = 0: nothing of the middle stays (no key passes the cut)
  for (int pass = 0; pass < 4 && hd.evict && left; ++pass) {
    uint32_t *hist = sm.hist[pass & 1];
    hist[tid] = 0;
    __syncthreads();
    const int shift = 24 - 8 * pass;
    for (int t = a_lo + tid; t < a_hi; t += kThreads) {
      const uint32_t k = key(t);
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[k >> shift & 255u], 1u);
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    // bin 255 - tid of all blocks, and the keys in higher bins
    uint32_t own = 0;
    const uint32_t at = smem_u32(&hist[255 - tid]);
    for (uint32_t r = 0; r < C; ++r) own += ld_cluster_u32(mapa_shared(at, r));
    uint32_t x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sm.warp_sum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += sm.warp_sum[w];
    if (x >= left && x - own < left) {
      sm.cut = prefix | (uint32_t)(255 - tid) << shift;
      sm.left = left - (x - own);
    }
    __syncthreads();
    prefix = sm.cut;
    left = sm.left;
    __syncthreads();
  }
  const bool none = hd.evict && left == 0;
  // Kept are: the front, the tail, keys above the cut, and the first `left` keys equal to it.
  auto above = [&](int t) {
    return t < hd.n && (!hd.evict || t < hd.first || t >= hd.last || (!none && key(t) > prefix));
  };
  auto equal = [&](int t) {
    return hd.evict && !none && t >= hd.first && t < hd.last && key(t) == prefix;
  };
  uint32_t na = 0, ne = 0;
  for (int t = t_lo + tid; t < t_hi; t += kThreads) {
    na += above(t);
    ne += equal(t);
  }
  if (tid < 2) sm.count[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    na += __shfl_xor_sync(0xffffffffu, na, d);
    ne += __shfl_xor_sync(0xffffffffu, ne, d);
  }
  if (lane == 0) {
    atomicAdd(&sm.count[0], na);
    atomicAdd(&sm.count[1], ne);
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  uint32_t before = 0, equals = 0;  // kept, and keys equal to the cut, in the runs before
  for (uint32_t r = 0; r < rank; ++r) {
    before += ld_cluster_u32(mapa_shared(smem_u32(&sm.count[0]), r));
    equals += ld_cluster_u32(mapa_shared(smem_u32(&sm.count[1]), r));
  }
  before += min(equals, left);
  const uint32_t start = ld_cluster_u32(mapa_shared(smem_u32(&sm.start), 0));
  if (rank == 0 && tid == 0)  // (all blocks of the head have read its length)
    p.kv_out[bh] = hd.n ? hd.m : p.kv_len[bh];
  if (units)
    for (int c0 = c_lo; c0 < c_hi; c0 += kThreads / kChunk) {
      const int t = c0 * kChunk + tid;
      const bool in = t < t_hi, ab = in && above(t), eq = in && equal(t);
      const uint32_t eb = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) sm.words[0][warp] = __popc(eb);
      __syncthreads();
      uint32_t e = equals, e_all = 0;
      for (int w = 0; w < 8; ++w) {
        if (w < warp) e += sm.words[0][w];
        e_all += sm.words[0][w];
      }
      const bool keep = ab || (eq && e + __popc(eb & ((1u << lane) - 1u)) < left);
      const uint32_t bits = __ballot_sync(0xffffffffu, keep);
      if (lane == 0) sm.words[1][warp] = bits;
      __syncthreads();
      if (tid < kThreads / kChunk && c0 + tid < c_hi && c0 + tid >= first_chunk) {
        uint32_t k = before;
        for (int w = 0; w < 2 * tid; ++w) k += __popc(sm.words[1][w]);
        const uint32_t u = start + (uint32_t)(c0 + tid - first_chunk);
        EvictUnit un;
        un.bh = bh;
        un.chunk = c0 + tid;
        un.first = (int)k;
        un.first_chunk = first_chunk;
        un.keep[0] = sm.words[1][2 * tid];
        un.keep[1] = sm.words[1][2 * tid + 1];
        un.pad[0] = un.pad[1] = 0;
        p.units[u] = un;
        p.read_done[u] = 0;
      }
      for (int w = 0; w < 8; ++w) before += __popc(sm.words[1][w]);
      equals += e_all;
      __syncthreads();
    }
  cluster_arrive();  // nobody leaves while its shared memory may be read
  cluster_wait();
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// kPieces pieces of type V make a row's K, as many its V. 4-bit rows: the last piece is the
// row's parameters.
template <class V, int kPieces, bool kQ4>
__global__ void __launch_bounds__(kThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kRow = 2 * kPieces;
  constexpr int kEach = (kChunk * kRow + kThreads - 1) / kThreads;  // pieces of a thread
  __shared__ int64_t src[kChunk], dst[kChunk];  // pool rows; dst -1: stays where it is
  __shared__ uint32_t ticket;
  __shared__ int ok_all;
  pdl_wait();
  const int tid = threadIdx.x;
  const uint32_t total = p.counters[0];
  for (;;) {
    __syncthreads();  // the unit before is done
    if (tid == 0) ticket = atomicAdd(p.counters + 1, 1u);
    __syncthreads();
    const uint32_t u = ticket;
    if (u >= total) break;
    const EvictUnit un = p.units[u];
    const int b = un.bh / p.c.Hkv, h = un.bh - b * p.c.Hkv;
    const int gi = p.c.head_grp[h], row = p.c.head_row[h];
    const CacheGroup &grp = p.c.grp[gi];
    const int n0 = __popc(un.keep[0]), cnt = n0 + __popc(un.keep[1]);
    float w = 0.f;
    int64_t w_to = -1;
    if (tid < kChunk && (un.keep[tid >> 5] >> (tid & 31) & 1u)) {
      const int32_t *table = grp.table + (size_t)b * grp.stride;
      const int j = (tid >> 5 ? n0 : 0) + __popc(un.keep[tid >> 5] & ((1u << (tid & 31)) - 1u));
      const int from = un.chunk * kChunk + tid, to = un.first + j;
      const int pf = table[from >> p.c.lgP], pt = table[to >> p.c.lgP];
      const bool have = pf >= 0 && pf < grp.pages && pt >= 0 && pt < grp.pages;
      if (!have) atomicOr(p.status, KVX_DEV_BAD_PAGE);
      src[j] = have ? pool_row(p.c, grp, pf, row, from & (p.c.P - 1)) : 0;
      const int64_t at = have ? pool_row(p.c, grp, pt, row, to & (p.c.P - 1)) : -1;
      dst[j] = from == to ? -1 : at;
      if (have && (p.copy_weights || from != to)) {
        w_to = at;
        w = p.weights[gi][src[j]];
      }
    }
    if (tid == 0) ok_all = 1;
    __syncthreads();
    V x[kEach];
    auto place = [&](int64_t r, int q) -> char * {
      char *pool = q < kPieces ? grp.k : grp.v;
      const int i = q < kPieces ? q : q - kPieces;
      if constexpr (kQ4)
        return pool + (i < kPieces - 1 ? q4_codes(p.c, r) + i * (int)sizeof(V) : q4_params(p.c, r));
      return pool + (r * kPieces + i) * (int)sizeof(V);
    };
    const int pieces = cnt * kRow;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid + e * kThreads;
      if (i < pieces && dst[i / kRow] >= 0) x[e] = *(const V *)place(src[i / kRow], i % kRow);
    }
    __syncthreads();  // the block has read its rows and weights
    if (tid == 0) st_release(p.read_done + u, 1u);
    // The chunks before this one that hold targets of its rows.
    const int lo = max(un.first_chunk, un.first / kChunk);
    if (cnt) {
      for (int c = lo + tid; c < un.chunk; c += kThreads) {
        const uint32_t *flag = p.read_done + (u - (uint32_t)(un.chunk - c));
        if (ld_acquire(flag)) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!ld_acquire(flag))
          if (globaltimer_ns() - t0 > p.wait_ns) {
            atomicOr(p.status, KVX_DEV_TIMEOUT);
            ok_all = 0;
            break;
          }
      }
    }
    __syncthreads();
    if (ok_all) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = tid + e * kThreads;
        if (i < pieces && dst[i / kRow] >= 0) *(V *)place(dst[i / kRow], i % kRow) = x[e];
      }
      if (w_to >= 0) p.weights_out[gi][w_to] = w;
    }
  }
  __threadfence();
  // The last block to leave resets the counters for the next call.
  if (tid == 0 && atomicAdd(p.counters + 2, 1u) == gridDim.x - 1)
    p.counters[0] = p.counters[1] = p.counters[2] = 0;
}

template <class V, int kPieces, bool kQ4>
cudaError_t launch_move(const EvictParams &p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.max_units < 4 * 152 ? p.max_units : 4 * 152));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_move_kernel<V, kPieces, kQ4>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t st) {
  const int heads = p.c.B * p.c.Hkv;
  // A head's blocks: more where there are few heads to fill the GPU with.
  const int C = heads <= 64 ? 8 : heads <= 256 ? 4 : heads <= 1024 ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool wide = p.c.D == 128;
  if (p.q4) return wide ? launch_move<uint2, 9, true>(p, st) : launch_move<uint32_t, 9, true>(p, st);
  if (p.c.row_bytes == 512) return launch_move<uint4, 32, false>(p, st);
  if (p.c.row_bytes == 256) return launch_move<uint4, 16, false>(p, st);
  return launch_move<uint4, 8, false>(p, st);
}

}  // namespace kvx
