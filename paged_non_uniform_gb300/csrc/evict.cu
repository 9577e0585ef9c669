// evict.cu -- eviction of cached tokens by accumulated attention weight.
//
// A head with n cached tokens and a budget of m < n keeps its first f and last r tokens and,
// of those between, the m - f - r with the largest weights (equal weights: lower index first),
// in their order; kept token number i becomes token i.
//
// First launch: a cluster of blocks per head, each with a run of the head's tokens. Weights
// become 32-bit keys of the same order; three passes of 11, 11 and 10 bits find the cut (histograms
// of the cluster's blocks are added through distributed shared memory), counts of the
// runs give every kept token its place. It leaves the list of kept tokens and a list of units:
// 64 places of a head each, with how many tokens stay before token 64 k of the head.
// Second launch: blocks take units by ticket. A unit reads its rows, says so, waits until
// the units that read its places have done so (rows move towards the front, so those are
// earlier units of the head, which running blocks have taken before, and no unit waits
// before it has read), and writes. So a head moves on all SMs at once, in place, with
// one read and one write of every row that moves.
// Measured on one GB300 (a call in a graph): 128 heads of 8k to 32k tokens cut to 10 to 50 % (a quarter
// keep all), 419 MB, 128 us: 50 of it the first launch (latency of
// the loads and the three passes), 80 the second (356 MB, 4.4 TB/s: two blocks an SM, each with two units
// of 32 KB under way, are bound by the latency of a unit's steps). 512 short heads, half of them
// cut to an eighth, 61 MB, 37 us: latency. With the weights in place 122 and 31 us; the 128 heads in fp32 (908 MB)
// 290, in 4 bits (189 MB) 180. All in page tables as wide as the longest head; launch_evict has wider ones.
#include <math.h>

#include "ptx.cuh"
#include "window.h"

namespace kvx {
namespace {

constexpr int kChunk = kEvictChunk;
constexpr int kBins = 2048;  // of a histogram: 11 bits of a key

// Order-preserving key: larger weight, larger key; -0 as 0; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

// The weight that a key other than 0 was made of (-0 as 0).
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
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

constexpr int kSmallKeys = 4096, kLargeKeys = 16384;  // in a block's shared memory

// Blocks of a head of n tokens, `most` at most: as many as its keys fill, or, where heads are few, as
// give each kSmallKeys of them. Measured, the call in a graph with 1 / 2 / 4 / 8 blocks a head: 32 heads of 8000
// tokens 33 / 27 / 25 / 35 us, of 16,000 54 / 39 / 32 / 41, of 32,000 147 / 62 / 46 / 52; 8 heads of 60,000
// 295 / 138 / 56 / 44; 128 heads of 16,000 82 / 76 / 77 / 112, of 32,000 201 / 130 / 125 / 151, of 60,000
// 406 / 277 / 210 / 229 (keys past a block's shared memory are read again in every pass).
__host__ __device__ constexpr uint32_t select_blocks(int n, int heads, uint32_t most) {
  uint32_t C = 1;
  while (C < most && (((int64_t)C * heads < 152 && (int64_t)C * kSmallKeys < n) || (int64_t)C * kLargeKeys < n)) C *= 2;
  return C;
}

// kThreads threads, kKeys keys of a block's run kept in shared memory (a longer run reads the
// others again in every pass).
template <int kThreads, int kKeys>
struct SelectSmem {
  uint32_t keys[kKeys];
  uint32_t hist[2][kBins];
  uint32_t warp_sum[2][kThreads / 32];
  uint32_t count[2];     // keys of this block's run that stay for certain, and equal to the cut
  uint32_t cut, left;    // digits found; keys still to take among those that share them
  uint32_t start;        // rank 0: the head's first unit
  uint32_t above[kKeys / 32], equal[kKeys / 32];
};

template <int kThreads, int kKeys>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 smem_raw[];
  SelectSmem<kThreads, kKeys> &sm = *(SelectSmem<kThreads, kKeys> *)smem_raw;
  pdl_launch_dependents();
  pdl_wait();
  uint32_t most;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(most));
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = (int)(blockIdx.x / most);
  const Head hd = load_head(p, bh, rank == 0 && tid == 0);
  // The cluster is as large as the page tables' room may ask for; the head's length says how many of
  // its blocks take part. The others leave at once (nobody reads their shared memory, and the cluster's barrier
  // waits for the blocks that have not left; a length that rank 0 has already replaced is smaller).
  const uint32_t C = select_blocks(hd.n, p.c.B * p.c.Hkv, most);
  if (rank >= C) return;
  const int gi = p.c.head_grp[hd.h], row = p.c.head_row[hd.h];
  const CacheGroup &grp = p.c.grp[gi];
  const int32_t *table = grp.table + (size_t)hd.b * grp.stride;
  const float *weights = p.weights[gi];
  // place of token t of page `page` in a pool of weights (pool_row, in fewer operations)
  const int page_step = grp.size << p.c.lgP, tok_step = p.c.token_major ? grp.size : 1;
  const int first_at = p.c.token_major ? row : row << p.c.lgP;
  auto place = [&](int page, int t) {
    return (int64_t)page * page_step + ((t & (p.c.P - 1)) * tok_step + first_at);
  };
  const int chunks = (hd.n + kChunk - 1) / kChunk, per = (chunks + (int)C - 1) / (int)C;
  const int c_lo = min(chunks, (int)rank * per), c_hi = min(chunks, c_lo + per);
  const int t_lo = c_lo * kChunk, t_hi = min(hd.n, c_hi * kChunk);
  const int first_unit = hd.first / kChunk;
  const int units = hd.evict ? max(0, (hd.m + kChunk - 1) / kChunk - first_unit) : 0;
  const int64_t base = (int64_t)hd.b * p.chunks_seq + p.chunk_off[hd.h];  // of the head's chunks

  auto load_key = [&](int t, int page) -> uint32_t {
    if (page < 0 || page >= grp.pages) return 0u;
    return weight_key(weights[place(page, t)]);
  };
  const int a_lo = max(t_lo, hd.first), a_hi = min(t_hi, hd.last);  // this run's part that competes
  const int k_hi = min(t_hi, t_lo + kKeys);                         // keys in shared memory
  if (rank == 0 && tid == 0) sm.start = units ? atomicAdd(p.counters, (uint32_t)units) : 0u;
  // All blocks of the head have written what the others read next.
  auto meet = [&]() {
    __syncthreads();
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    }
  };
  uint32_t prefix = 0, left = 0;  // found digits; keys to take among those that share them
  if (hd.evict) {
    left = (uint32_t)(hd.m - hd.first - (hd.n - hd.last));
    const int end = k_hi;
    for (int t0 = t_lo + tid; t0 < end; t0 += 8 * kThreads) {  // eight in flight
      int page[8];
      uint32_t k[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) page[u] = t0 + u * kThreads < end ? table[(t0 + u * kThreads) >> p.c.lgP] : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u) k[u] = load_key(t0 + u * kThreads, page[u]);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t0 + u * kThreads < end) sm.keys[t0 + u * kThreads - t_lo] = k[u];
    }
  }
  // (left = 0: nothing of the middle stays)
  for (int pass = 0; pass < 3 && hd.evict && left; ++pass) {
    uint32_t *hist = sm.hist[pass & 1];
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    auto count = [&](bool in, uint32_t k) {
      const uint32_t digit = k >> shift & ((1u << bits) - 1u);
      if (pass == 0) {
        // Weights share leading digits: one add for all lanes of a digit (adds to one address go
        // one after the other).
        const uint32_t same = __match_any_sync(0xffffffffu, in ? digit : (uint32_t)kBins);
        if (in && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&hist[digit], (uint32_t)__popc(same));
      } else if (in && (k >> (shift + bits)) == (prefix >> (shift + bits))) {
        atomicAdd(&hist[digit], 1u);
      }
    };
    const int split = min(a_hi, max(a_lo, k_hi));
    for (int t0 = a_lo + 32 * warp; t0 < split; t0 += kThreads) {
      const int t = t0 + lane;
      count(t < split, t < split ? sm.keys[t - t_lo] : 0u);
    }
    for (int t0 = split + 32 * warp; t0 < a_hi; t0 += kThreads) {
      const int t = t0 + lane;
      count(t < a_hi, t < a_hi ? load_key(t, table[t >> p.c.lgP]) : 0u);
    }
    meet();
    // Bins from the last down, kEach to a thread, of all blocks; the keys in higher bins.
    constexpr int kEach = kBins / kThreads;
    uint32_t own[kEach], x = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) own[e] = 0;
    for (uint32_t r = 0; r < C; ++r)
#pragma unroll
      for (int e = 0; e < kEach; e += 4) {  // four bins a load, the highest last
        const uint32_t at = smem_u32(&hist[kBins - 4 - (tid * kEach + e)]);
        const float4 v = ld_cluster_f4(C == 1 ? at : mapa_shared(at, r));
        own[e] += __float_as_uint(v.w);
        own[e + 1] += __float_as_uint(v.z);
        own[e + 2] += __float_as_uint(v.y);
        own[e + 3] += __float_as_uint(v.x);
      }
#pragma unroll
    for (int e = 0; e < kEach; ++e) x += own[e];
    const uint32_t mine = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sm.warp_sum[0][warp] = x;
    __syncthreads();
    x -= mine;
    for (int w = 0; w < warp; ++w) x += sm.warp_sum[0][w];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (x < left && x + own[e] >= left) {
        sm.cut = prefix | (uint32_t)(kBins - 1 - (tid * kEach + e)) << shift;
        sm.left = left - x;
      }
      x += own[e];
    }
    __syncthreads();
    prefix = sm.cut;
    left = sm.left;
    __syncthreads();
  }
  const bool some = hd.evict && left > 0;
  // Kept are: the front, the tail, keys above the cut, and the first `left` keys equal to it.
  // Bits of the words of 32 tokens from t0 on, kKeys tokens at most; counts of both kinds.
  uint32_t na = 0, ne = 0;
  auto mark = [&](int t0) {
    for (int w0 = warp; w0 < kKeys / 32 && t0 + 32 * w0 < t_hi; w0 += kThreads / 32) {
      const int t = t0 + 32 * w0 + lane;
      const bool in = t < t_hi, mid = in && hd.evict && t >= hd.first && t < hd.last;
      const uint32_t k = !mid || !some ? 0u
                         : t0 == t_lo  ? sm.keys[t - t_lo]
                                       : load_key(t, table[t >> p.c.lgP]);
      const uint32_t ab = __ballot_sync(0xffffffffu, in && (!mid || (some && k > prefix)));
      const uint32_t eq = __ballot_sync(0xffffffffu, mid && some && k == prefix);
      if (lane == 0) {
        sm.above[w0] = ab;
        sm.equal[w0] = eq;
      }
      na += __popc(ab);
      ne += __popc(eq);
    }
  };
  if (tid < 2) sm.count[tid] = 0;
  __syncthreads();
  for (int t0 = t_lo; t0 < t_hi; t0 += kKeys) mark(t0);
  if (lane == 0) {
    atomicAdd(&sm.count[0], na);
    atomicAdd(&sm.count[1], ne);
  }
  meet();
  uint32_t before = 0, equals = 0;  // kept for certain, and equal to the cut, in the runs before
  for (uint32_t r = 0; r < rank; ++r) {
    before += ld_cluster_u32(mapa_shared(smem_u32(&sm.count[0]), r));
    equals += ld_cluster_u32(mapa_shared(smem_u32(&sm.count[1]), r));
  }
  const uint32_t start = C == 1 ? sm.start : ld_cluster_u32(mapa_shared(smem_u32(&sm.start), 0));
  if (rank == 0 && tid == 0)  // (all blocks of the head have read its length)
    p.kv_out[bh] = hd.n ? hd.m : p.kv_len[bh];
  // Places: exclusive sums over the words of a segment of kKeys tokens.
  static_assert(kKeys / 32 <= kThreads, "a thread a word");
  for (int t0 = t_lo; t0 < t_hi && (units || p.copy_weights); t0 += kKeys) {
    if (t_hi - t_lo > kKeys) {  // (else the words are still there)
      __syncthreads();
      mark(t0);
    }
    __syncthreads();
    const bool in = tid < kKeys / 32 && t0 + 32 * tid < t_hi;
    const uint32_t ab = in ? sm.above[tid] : 0u, eq = in ? sm.equal[tid] : 0u;
    uint32_t xa = __popc(ab), xe = __popc(eq);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t ya = __shfl_up_sync(0xffffffffu, xa, d), ye = __shfl_up_sync(0xffffffffu, xe, d);
      if (lane >= d) xa += ya, xe += ye;
    }
    if (lane == 31) sm.warp_sum[0][warp] = xa, sm.warp_sum[1][warp] = xe;
    __syncthreads();
    uint32_t all_a = 0, all_e = 0;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t sa = sm.warp_sum[0][w], se = sm.warp_sum[1][w];
      if (w < warp) xa += sa, xe += se;
      all_a += sa, all_e += se;
    }
    const uint32_t e0 = equals + xe - __popc(eq);  // equal keys before this word
    uint32_t keep = ab, take = min(left > e0 ? left - e0 : 0u, (uint32_t)__popc(eq));
    for (uint32_t rest = eq; take; --take, rest &= rest - 1) keep |= rest & (0u - rest);
    const uint32_t at = before + xa - __popc(ab) + min(e0, left);  // kept before this word
    __syncthreads();  // (the words and sums have been read)
    if (in) {
      sm.above[tid] = keep;
      sm.equal[tid] = at;
      const int c = (t0 >> 6) + (tid >> 1);
      if ((tid & 1) == 0 && c >= first_unit && c < first_unit + units) {
        p.units[start + (c - first_unit)] = {bh, c, min(kChunk, hd.m - c * kChunk), (int)at / kChunk};
        p.read_done[start + (c - first_unit)] = 0;
      }
    }
    before += all_a;
    equals += all_e;
    __syncthreads();
    const int words = min(kKeys / 32, (t_hi - t0 + 31) / 32);
    for (int w0 = warp; w0 < words; w0 += 8 * kWarps) {  // eight words in flight
      int from[8], to[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int w = w0 + u * kWarps;
        const uint32_t k = w < words ? sm.above[w] : 0u;
        from[u] = t0 + 32 * w + lane;
        to[u] = -1;
        if (k >> lane & 1u) {
          to[u] = (int)(sm.equal[w] + __popc(k & ((1u << lane) - 1u)));
          p.source[base * kChunk + to[u]] = from[u];
        }
      }
      if (!p.copy_weights) continue;  // (in place, weights move with their rows)
      int pf[8], pt[8];
      float wt[8];
      bool look[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t k = to[u] >= 0 && hd.evict && t0 == t_lo ? sm.keys[from[u] - t_lo] : 0u;
        wt[u] = key_weight(k);
        pt[u] = to[u] >= 0 ? table[to[u] >> p.c.lgP] : 0;
        // (key 0: not in shared memory, NaN, or a page outside the pool)
        look[u] = to[u] >= 0 && k == 0u;
        pf[u] = look[u] ? table[from[u] >> p.c.lgP] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool ok = pt[u] >= 0 && pt[u] < grp.pages && pf[u] >= 0 && pf[u] < grp.pages;
        if (!ok) {
          atomicOr(p.status, KVX_DEV_BAD_PAGE);
          to[u] = -1;
        }
        if (ok && look[u]) wt[u] = weights[place(pf[u], from[u])];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (to[u] >= 0) p.weights_out[gi][place(pt[u], to[u])] = wt[u];
    }
  }
  meet();  // nobody leaves while its shared memory may be read
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// What is known of a unit before its rows are read.
struct Places {
  int64_t src[kChunk], dst[kChunk];  // pool rows; -1: a page outside the pool
  EvictUnit un;
  uint32_t unit, end;  // end: no unit, nothing comes after it
};
constexpr int kMovers = 256, kScouts = kChunk;
constexpr int kRing = 3;  // units whose places are known: written, read, looked up

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Named barriers: a ring slot's places are there (1 ..), the slot is free (4 ..), movers (7).
constexpr int kFull = 1, kFree = kFull + kRing, kMove = kFree + kRing;

// kPieces pieces of type V make a row's K, as many its V. 4-bit rows: the last piece is the
// row's parameters. Two warps look up the places of the units to come; the others read unit
// i + 1 before they wait for the units before unit i and write it, so that a unit is
// read long before another one needs that (said only after unit i is written, a call took 228 us instead of 183).
template <class V, int kPieces, bool kQ4>
__global__ void __launch_bounds__(kMovers + kScouts) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kRow = 2 * kPieces;
  constexpr int kEach = (kChunk * kRow + kMovers - 1) / kMovers;  // pieces of a thread
  __shared__ Places ring[kRing];
  __shared__ uint32_t ticket;
  __shared__ uint32_t failed;
  const int tid = threadIdx.x;
  if (tid == 0) failed = 0;
  __syncthreads();
  pdl_wait();
  if (tid >= kMovers) {
    const int j = tid - kMovers;  // the unit's row
    const uint32_t total = p.counters[0];
    // The ticket is taken two units ahead, the unit read one ahead.
    auto take = [&]() { return j == 0 ? atomicAdd(p.counters + 1, 1u) : 0u; };
    auto tell = [&](uint32_t t) {
      if (j == 0) ticket = t;
      bar_sync(kMove + 1, kScouts);
      const uint32_t u = ticket;
      bar_sync(kMove + 1, kScouts);
      return u;
    };
    uint32_t u = tell(take()), u1 = tell(take());
    EvictUnit un = {}, un1 = {};
    if (u < total) un = p.units[u];
    for (int i = 0;; ++i) {
      Places &m = ring[i % kRing];
      const uint32_t t2 = take();
      if (u1 < total) un1 = p.units[u1];
      if (i >= kRing) bar_sync(kFree + i % kRing, kMovers + kScouts);
      if (u < total) {
        const int b = un.bh / p.c.Hkv, h = un.bh - b * p.c.Hkv, row = p.c.head_row[h];
        const CacheGroup &grp = p.c.grp[p.c.head_grp[h]];
        const int64_t base = (int64_t)b * p.chunks_seq + p.chunk_off[h];
        const int32_t *table = grp.table + (size_t)b * grp.stride;
        const int to = un.chunk * kChunk + j;
        int64_t src = -1, dst = -1;
        if (j < un.count) {
          const int from = p.source[base * kChunk + to];
          const int pt = table[to >> p.c.lgP], pf = table[from >> p.c.lgP];
          if (pf >= 0 && pf < grp.pages && pt >= 0 && pt < grp.pages) {
            src = pool_row(p.c, grp, pf, row, from & (p.c.P - 1));
            dst = pool_row(p.c, grp, pt, row, to & (p.c.P - 1));
          } else {
            atomicOr(p.status, KVX_DEV_BAD_PAGE);
          }
        }
        m.src[j] = src;
        m.dst[j] = dst;
        if (j == 0) {
          m.un = un;
          m.unit = u;
        }
      }
      if (j == 0) m.end = u >= total;
      bar_arrive(kFull + i % kRing, kMovers + kScouts);
      if (u >= total) break;
      u = u1;
      un = un1;
      u1 = tell(t2);
    }
  } else {
    auto place = [&](const CacheGroup &grp, int64_t r, int q) -> char * {
      char *pool = q < kPieces ? grp.k : grp.v;
      const int i = q < kPieces ? q : q - kPieces;
      if constexpr (kQ4)
        return pool + (i < kPieces - 1 ? q4_codes(p.c, r) + i * (int)sizeof(V) : q4_params(p.c, r));
      return pool + (r * kPieces + i) * (int)sizeof(V);
    };
    auto moves = [&](const Places &m, int i) {
      return i < m.un.count * kRow && m.dst[i / kRow] != m.src[i / kRow];
    };
    auto weighs = [&](const Places &m) {
      return !p.copy_weights && tid < m.un.count && m.dst[tid] != m.src[tid];
    };
    auto read = [&](const Places &m, V(&v)[kEach], float &wt) {
      const int gi = p.c.head_grp[m.un.bh % p.c.Hkv];
      const CacheGroup &grp = p.c.grp[gi];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = tid + e * kMovers;
        if (moves(m, i)) v[e] = *(const V *)place(grp, m.src[i / kRow], i % kRow);
      }
      if (weighs(m)) wt = p.weights[gi][m.src[tid]];
    };
    // (the barrier after its use lies before the next unit's)
    volatile uint32_t *const given_up = &failed;  // one more than the last unit whose wait ran out, or 0
    auto write = [&](const Places &m, const V(&v)[kEach], float wt) {
      // Units before this one that read what it overwrites. A block that has given up once looks, but
      // waits no more, so that it ends; only units whose places are still needed stay unwritten.
      for (int c = m.un.wait_from + tid; c < m.un.chunk; c += kMovers) {
        const uint32_t *flag = p.read_done + (m.unit - (uint32_t)(m.un.chunk - c));
        if (ld_acquire(flag)) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!ld_acquire(flag))
          if (*given_up || globaltimer_ns() - t0 > p.wait_ns) {
            atomicOr(p.status, KVX_DEV_TIMEOUT);
            *given_up = m.unit + 1u;
            break;
          }
      }
      bar_sync(kMove, kMovers);
      if (*given_up == m.unit + 1u) return;
      const int gi = p.c.head_grp[m.un.bh % p.c.Hkv];
      const CacheGroup &grp = p.c.grp[gi];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = tid + e * kMovers;
        if (moves(m, i)) *(V *)place(grp, m.dst[i / kRow], i % kRow) = v[e];
      }
      if (weighs(m)) p.weights_out[gi][m.dst[tid]] = wt;
    };
    // Reads unit i (false: there is none) and writes the unit before it, whose rows are in `prev`.
    auto step = [&](int i, V(&mine)[kEach], float &w_mine, const V(&prev)[kEach], float w_prev) {
      const Places &m = ring[i % kRing], &before = ring[(i + kRing - 1) % kRing];
      bar_sync(kFull + i % kRing, kMovers + kScouts);
      const bool more = !m.end;
      if (more) {
        read(m, mine, w_mine);
        bar_sync(kMove, kMovers);  // the block has read its rows and weights
        // (failure-detection test: the chosen block keeps its first unit's to itself)
        const bool stall = i == 0 && (int)blockIdx.x == p.stall_block;
        if (tid == 0 && !stall) st_release(p.read_done + m.unit, 1u);
      }
      if (i > 0) {
        write(before, prev, w_prev);
        if (more) bar_arrive(kFree + (i + kRing - 1) % kRing, kMovers + kScouts);
      }
      return more;
    };
    V xa[kEach], xb[kEach];
    float wa = 0.f, wb = 0.f;
    for (int i = 0; step(i, xa, wa, xb, wb) && step(i + 1, xb, wb, xa, wa); i += 2) {
    }
  }
  __threadfence();
  __syncthreads();
  // The last block to leave resets the counters for the next call.
  if (tid == 0 && atomicAdd(p.counters + 2, 1u) == gridDim.x - 1)
    p.counters[0] = p.counters[1] = p.counters[2] = 0;
}

template <class V, int kPieces, bool kQ4>
cudaError_t launch_move(const EvictParams &p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.chunks < 2 * 152 ? p.chunks : 2 * 152));
  cfg.blockDim = dim3(kMovers + kScouts);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_move_kernel<V, kPieces, kQ4>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kThreads, int kKeys>
cudaError_t launch_select(const EvictParams &p, int C, cudaStream_t st) {
  static int8_t done[64];
  const int bytes = (int)sizeof(SelectSmem<kThreads, kKeys>);
  const auto kernel = evict_select_kernel<kThreads, kKeys>;
  cudaError_t e = raise_smem_limit(done, (const void *)kernel, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.B * p.c.Hkv * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
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
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t st) {
  // Rooms of page tables are all that is known here. Heads that no table lets pass 4096 tokens, and
  // many: a small block each, many to an SM (512 heads of 2000 tokens 34 us, in large blocks 42; of 4000 64 and
  // 70, 256 of them 39 and 37). Else clusters for the longest head that fits; blocks that a head's
  // length does not need still cost their launch. 512 heads of 1000 to 2500 tokens in tables 1, 4, 8 and 32
  // times as wide: 37, 41, 56, 75 us (243 with all blocks of the clusters at work); 128 heads of 8k to 32k:
  // 128, 145, 146, 144 (181).
  const int heads = p.c.B * p.c.Hkv;
  int room = 0;
  for (int g = 0; g < p.c.G; ++g) room = p.c.grp[g].tokens > room ? p.c.grp[g].tokens : room;
  cudaError_t e = room <= kSmallKeys && heads >= 152
                      ? launch_select<256, kSmallKeys>(p, 1, st)
                      : launch_select<512, kLargeKeys>(p, (int)select_blocks(room, heads, 8), st);
  if (e != cudaSuccess) return e;
  const bool wide = p.c.D == 128;
  if (p.q4) return wide ? launch_move<uint2, 9, true>(p, st) : launch_move<uint32_t, 9, true>(p, st);
  if (p.c.row_bytes == 512) return launch_move<uint4, 32, false>(p, st);
  if (p.c.row_bytes == 256) return launch_move<uint4, 16, false>(p, st);
  return launch_move<uint4, 8, false>(p, st);
}

}  // namespace kvx
