// tree_mma.cu -- attention for a tree of drafted tokens, bf16 cache, on the
// 5th-generation tensor cores (tcgen05).
//
// out[row] = sum_t softmax(scale * <q_row, k_t>)_t v_t over the cached tokens
// of the row's KV head and the drafts its mask shows. The T_b * g query rows of
// a KV head share its keys, so both products are dense: S [128 rows][128 keys]
// = Q K^T and O [128 rows][D] += P V, with S, P and O in tensor memory. One
// pass over the keys with a running maximum and sum per row. One block per SM
// walks its items (tree_split.cuh) in tiles of 128 keys:
//  * warps 8 and 9 load K and V tiles from their pages into two rings (bulk
//    tensor loads, one box of min(P, 128) rows x 64 dims per lane, landing as
//    [half][128 rows][128 bytes], 128-byte swizzled);
//  * warp 10 issues the MMAs: S(j), then O += P V of job j - 1, so that one warp
//    group's softmax runs under the other's products;
//  * warps 0-3 and 4-7 are two softmax groups, one query row per thread. Up to
//    128 query rows, both hold all rows and take the tiles in turn (their (m, l, O) are
//    merged at the item's end); above, each holds half the rows and takes
//    every tile. A job is one tile for one group;
//  * warp 11 cleans the V tiles that hold drafts or the head's end: rows past
//    the end are zeroed (stale or padding data), and non-finite values of drafts
//    are replaced by zero and noted, because a weight of 0 does not silence them
//    for rows that do not see the draft; the epilogue adds them to the rows that do.
// P is kept as a bf16 high part and a bf16 residual (two products): with the
// high part alone the weights would be off by 2^-9, with both by 2^-18, below
// the fp32 output's other errors. They overwrite the scores they came from, column
// block by column block.
// The output is rescaled only when a row's maximum has grown by more than 2^8 since
// its reference (the weights are then at most 2^8, exact in scale), which
// after a row's first tile is rare; a row's sum and output share one reference.
// Every mbarrier wait gives up after two seconds, sets KVX_DEV_TIMEOUT and lets
// all roles run to their end without waiting, loading or multiplying.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "tcgen05.cuh"
#include "tree_split.cuh"

namespace kvx {
namespace {

constexpr int kTile = 128;       // keys of a tile
constexpr int kThreads = 384;
constexpr int kSoft = 256;       // threads of the softmax groups
constexpr int kMinUnits = 2;     // tiles a block takes at least
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kGrow = 8.f;     // log2 growth of the maximum that triggers a rescale
// Tiles of a group after which its output leaves tensor memory for an fp32 sum: the
// tensor cores truncate each of the 16 additions a tile makes to every output
// element, which over 200 tiles was measured as 5e-5 of the output, growing
// linearly; over 16 tiles it stays below 5e-6.
constexpr int kFold = 16;
constexpr int kItems = 16;       // item slots: more than V tiles in flight, plus one

constexpr int kCtlBytes = 1408;

// kTwo: launches with more than 128 query rows a head (two Q tiles).
template <int D, bool kTwo>
struct Cfg {
  static constexpr int kRows = kTwo ? 256 : 128;  // query rows of an item
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTile * 128;            // bytes of 64 dims of a tile
  static constexpr int kTileBytes = kHalves * kHalf;   // a K, V or Q tile
  static constexpr int kSlots = 7 * 2 / kHalves - (kTwo ? 2 : 1);  // of 224 KB, after Q
  static constexpr int kV = (kSlots + 1) / 2, kK = kSlots - kV;
  static_assert(kV + 1 < kItems, "items in flight");
  static constexpr int kBars = 2 * kK + 3 * kV + 8 + kItems;
  static constexpr int kQ = 0, kKs = (kTwo ? 2 : 1) * kTileBytes;
  static constexpr int kVs = kKs + kK * kTileBytes, kCtl = kVs + kV * kTileBytes;
  static_assert((kCtl - kKs) / (kTreeMmaBlocks * (D * 4 + 8)) >= 2, "two rows of every partial fit");
  static constexpr int kSmem = 1024 + kCtl + kBars * 8 + kCtlBytes;
};

struct Ctl {  // small shared state behind the barriers
  uint32_t tmem;
  int abort;
  int last[2];
  int more[2];
  int64_t warp_sum[kThreads / 32];
  TreeRange range;
  TreeItem split[2];          // items shared with other blocks
  TreeItem item[kItems];      // written by warp 11, ahead of the others
  uint32_t notes[kItems][4];  // drafts of an item whose V is not finite
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

struct alignas(128) MmaParams {
  CUtensorMap tmK[KVX_MAX_GROUPS];
  CUtensorMap tmV[KVX_MAX_GROUPS];
  TreeParams t;
};

// Bounded wait for the phase of `bar` with the given parity. When it runs out, or
// another role's has, waits end at once and the block runs down.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                     uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return;
    if (*abort) return;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *abort = 1;
      atomicOr(status, KVX_DEV_TIMEOUT);
      return;
    }
  }
}

// How an item is worked: two groups over all rows (tiles in turn), or a half of
// the rows each (every tile).
struct Jobs {
  int rows, tiles, jobs;
  bool halves;
  __device__ __forceinline__ Jobs(const TreeItem &it, int g, int max_rows) {
    rows = min(max_rows, it.head.T * g - it.group * max_rows);
    tiles = it.t1 - it.t0;
    halves = rows > 128;
    jobs = halves ? 2 * tiles : tiles;
  }
  __device__ __forceinline__ int tile(int j) const { return halves ? j >> 1 : j; }
  __device__ __forceinline__ bool opens(int j) const { return !halves || (j & 1) == 0; }
  __device__ __forceinline__ bool closes(int j) const { return !halves || (j & 1) == 1; }
};

// Visible keys among the 32 from draft `u0` on (negative: that many cached
// tokens first) for new row i.
__device__ __forceinline__ uint32_t seen_word(const TreeParams &p, const TreeHead &t, int i,
                                              int u0) {
  if (u0 <= -32) return 0xffffffffu;
  const int w = u0 >> 5, s = u0 & 31;  // u0 < 0: w = -1, cached tokens
  const uint32_t lo = w < 0 ? 0xffffffffu : tree_mask_word(p, t, i, w);
  return s ? __funnelshift_r(lo, tree_mask_word(p, t, i, w + 1), s) : lo;
}

// The loops below are kept rolled: the kernel's roles run side by side on one
// instruction cache, and with a tile's softmax unrolled (1,500 instructions) its warps
// mostly waited for instructions.

// Scores of keys that the row does not see become -inf (a tile with drafts or
// the head's end).
__device__ __forceinline__ void hide_keys(const TreeParams &p, const TreeHead &t, int row_i,
                                          bool row_ok, int u0, uint32_t s_at) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_ld32(s_at + 32 * c, x);
    const uint32_t seen = row_ok ? seen_word(p, t, row_i, u0 + 32 * c) : 0u;
    tmem_wait_ld(x);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((seen >> e) & 1u)) x[e] = __float_as_uint(-INFINITY);
    tmem_st32(s_at + 32 * c, x);
  }
  tmem_wait_st();
}

// One row's softmax of one tile: scores (TMEM) to weights (TMEM, in place), the
// running reference m and sum l. have: O holds products of earlier tiles, which a
// new reference rescales.
template <int D>
__device__ __forceinline__ void soft_tile(uint32_t s_at, uint32_t o_at, float scale, bool have,
                                          float &m, float &l) {
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32], y[32];
    tmem_ld32(s_at + 64 * c, x);
    tmem_ld32(s_at + 64 * c + 32, y);
    tmem_wait_ld(x);
    tmem_wait_ld(y);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      mx0 = fmaxf(mx0, __uint_as_float(x[e]));
      mx1 = fmaxf(mx1, __uint_as_float(y[e]));
    }
  }
  const float top = fmaxf(mx0, mx1) * scale;
  // a new reference for rows that have seen nothing before, or whose maximum
  // has grown by more than kGrow
  const bool move = top > m + kGrow;
  const float mn = move ? top : m;
  const float f = move ? tree_weight(m, mn) : 1.f;
  l *= f;
  if (have && __any_sync(0xffffffffu, move && m != -INFINITY)) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t y[32];
      tmem_ld32(o_at + 32 * c, y);
      tmem_wait_ld(y);
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
      tmem_st32(o_at + 32 * c, y);
    }
  }
  m = mn;
  const float ref = m == -INFINITY ? 0.f : m;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {  // of 16 keys: 8 columns of high parts, 8 of residuals
    uint32_t x[32], y[32];
    tmem_ld32(s_at + 32 * c, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float a = ex2(fmaf(__uint_as_float(x[e]), scale, -ref));
      const float b = ex2(fmaf(__uint_as_float(x[e + 1]), scale, -ref));
      sum[e & 2] += a;
      sum[(e & 2) + 1] += b;
      const uint32_t hi = pack_bf16(a, b);
      const int at = (e & 16) + ((e & 15) >> 1);
      y[at] = hi;
      y[at + 8] = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
    }
    tmem_st32(s_at + 32 * c, y);
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  tmem_wait_st();
}

// Folds the partials of a row group into its output rows, through the K and V
// rings (idle by now): bulk copies bring the partials of as many rows as fit, all
// in flight at once, so that the fold waits for L2 once a round and not once a
// partial. Partials are added in block order.
template <int D, int kRows, int kBytes>
__device__ __forceinline__ void merge_parts(const TreeParams &p, const TreeRange &r,
                                            const TreeItem &it, uint8_t *buf, uint32_t bar,
                                            int &phase, volatile int *abort, int tid) {
  const int c0 = tree_block_of(r.units, r.blocks, it.seg);
  const int n = tree_block_of(r.units, r.blocks, it.seg + it.head.tiles - 1) - c0 + 1;
  const int rows = min(kRows, it.head.T * p.c.g - it.group * kRows);
  const bool odd = it.seg > tree_bound(r.units, r.blocks, c0);
  // a round: (m, l) of `fit` rows of every partial, then their outputs
  const int fit = min((rows + 1) & ~1, (kBytes / (n * (D * 4 + 8))) & ~1);
  float2 *ml = (float2 *)buf;
  float4 *o = (float4 *)(buf + (size_t)n * fit * 8);
  for (int r0 = 0; r0 < rows; r0 += fit) {
    const int now = min(fit, rows - r0), even = (now + 1) & ~1;  // 16-byte copies
    if (tid < 32) {
      asm volatile("fence.proxy.async;" ::: "memory");  // the others' writes, then bulk reads
      if (tid == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * (now * D * 4 + even * 8)));
      __syncwarp();
      for (int c = tid; c < n; c += 32) {
        const size_t at = (size_t)(2 * (c0 + c) + (c == 0 && odd)) * kRows + r0;
        bulk_load(smem_u32(ml + c * fit), p.part_ml + at, even * 8, bar);
        bulk_load(smem_u32(o + (size_t)c * fit * (D / 4)), p.part_o + at * D, now * D * 4, bar);
      }
    }
    wait(bar, phase & 1, abort, p.status);
    ++phase;
    for (int q = tid; q < now; q += kSoft) {  // weights, divided by the sum
      float M = -INFINITY, L = 0.f;
      for (int c = 0; c < n; ++c) M = fmaxf(M, ml[c * fit + q].x);
      for (int c = 0; c < n; ++c) {
        const float2 v = ml[c * fit + q];
        L = fmaf(tree_weight(v.x, M), v.y, L);
      }
      const float s = L == 0.f ? 0.f : 1.f / L;
      for (int c = 0; c < n; ++c) ml[c * fit + q].x = tree_weight(ml[c * fit + q].x, M) * s;
    }
    named_sync(1, kSoft);
    for (int q = tid; q < now * (D / 4); q += kSoft) {
      const int row = q / (D / 4), d4 = q % (D / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < n; ++c) {
        const float f = ml[c * fit + row].x;
        const float4 v = o[(c * fit + row) * (D / 4) + d4];
        x.x = fmaf(f, v.x, x.x);
        x.y = fmaf(f, v.y, x.y);
        x.z = fmaf(f, v.z, x.z);
        x.w = fmaf(f, v.w, x.w);
      }
      *((float4 *)tree_out(p, it.head, it.group * kRows + r0 + row) + d4) = x;
    }
    fence_async_shared();  // the next round's copies land where these reads were
    named_sync(1, kSoft);
  }
}

// The block's tiles one by one.
template <int kRows>
struct TileWalk {
  TreeCursor<kTile, kRows> cur;
  TreeItem it;
  int tile;
  bool more;
  __device__ __forceinline__ TileWalk(const TreeParams &p, const TreeRange &r) : cur(p, r) {
    more = cur.next(p, it);
    tile = it.t0;
  }
  __device__ __forceinline__ void step(const TreeParams &p) {
    if (++tile < it.t1) return;
    more = cur.next(p, it);
    tile = it.t0;
  }
};

// One warp's part of one role's loads: all K (or V) tiles of the block.
template <int D, bool kTwo, bool kIsV>
__device__ __forceinline__ void produce(const MmaParams &mp, const TreeRange &range,
                                        uint32_t ring, uint32_t full0, uint32_t empty0,
                                        volatile int *abort, int lane) {
  using C = Cfg<D, kTwo>;
  constexpr int kN = kIsV ? C::kV : C::kK;
  const TreeParams &p = mp.t;
  const uint64_t pol = policy_evict_first();
  const int P = p.c.P, box = min(P, kTile);
  const int per = kTile / box;  // boxes of a tile and half
  // lane -> (box, half); a tile has at most 16 * 2 of them
  const int bx = lane % per, half = lane / per;
  // Two walks over the tiles: `ahead` runs kAhead tiles before `now` and reads
  // the page ids, so that neither the lengths nor the page table hold up a load.
  constexpr int kAhead = 3;
  TileWalk<C::kRows> now(p, range), ahead(p, range);
  auto page_of = [&]() {
    if (!ahead.more) return 0;
    const TreeHead &h = ahead.it.head;
    const CacheGroup &grp = p.c.grp[p.c.head_grp[h.h]];
    const int tok = ahead.tile * kTile + bx * box;
    const int page = half < C::kHalves && tok < h.n + h.T
                         ? __ldg(grp.table + (size_t)h.b * grp.stride + (tok >> p.c.lgP))
                         : 0;
    ahead.step(p);
    return page;
  };
  int pages[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) pages[i] = page_of();
  for (int n = 0; now.more; ++n) {
    const TreeHead &h = now.it.head;
    const int gi = p.c.head_grp[h.h], rank = p.c.head_row[h.h];
    const int slot = n % kN, valid = min(kTile, h.n + h.T - now.tile * kTile);
    const int boxes = (valid + box - 1) / box;
    int page = pages[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) pages[i] = pages[i + 1];
    pages[kAhead - 1] = page_of();
    if (n >= kN) wait(empty0 + 8 * slot, ((n / kN) - 1) & 1, abort, p.status);
    if (__any_sync(0xffffffffu, *abort)) return;
    const uint32_t full = full0 + 8 * slot;
    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(boxes * box * 128 * C::kHalves));
    __syncwarp();
    if (half < C::kHalves && bx < boxes) {
      const int64_t have = p.c.grp[gi].pages;
      if (page < 0 || (int64_t)page >= have) {
        atomicOr(p.status, KVX_DEV_BAD_PAGE);
        page = (int)have;  // past the last page: loads zeros
      }
      const int tok = now.tile * kTile + bx * box;
      tma_load_5d(ring + slot * C::kTileBytes + half * C::kHalf + bx * box * 128,
                  kIsV ? &mp.tmV[gi] : &mp.tmK[gi], 0, tok & (P - 1), half, rank, page, full, pol);
    }
    now.step(p);
  }
}

template <int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1) tree_mma_kernel(const __grid_constant__ MmaParams mp) {
  using C = Cfg<D, kTwo>;
  const TreeParams &p = mp.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  uint64_t *bars = (uint64_t *)(smem + C::kCtl);
  Ctl &ctl = *(Ctl *)(bars + C::kBars);
  volatile int *abort = &ctl.abort;
  const uint32_t k_full = smem_u32(bars), k_empty = k_full + 8 * C::kK;
  const uint32_t v_full = k_empty + 8 * C::kK, v_empty = v_full + 8 * C::kV;
  const uint32_t v_ready = v_empty + 8 * C::kV;  // loaded, and cleaned where it has to be
  const uint32_t s_full = v_ready + 8 * C::kV;   // [2] scores of a group are ready
  const uint32_t p_ready = s_full + 16;         // [2] weights of a group are ready
  const uint32_t o_full = p_ready + 16;         // [2] a group's output of the item is complete
  const uint32_t q_ready = o_full + 16;         // Q of the item is loaded, O may be overwritten
  const uint32_t m_full = q_ready + 8;          // partials to merge are loaded
  const uint32_t i_full = m_full + 8;           // [kItems] an item is written
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(v_ready + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, 4);
      mbar_init(o_full + 8 * i, 1);
    }
    mbar_init(q_ready, kSoft / 32);
    mbar_init(m_full, 1);
    for (int i = 0; i < kItems; ++i) mbar_init(i_full + 8 * i, 1);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == 10) tmem_alloc(smem_u32(&ctl.tmem), 512);
  if (warp >= 8 && warp < 10 && lane < p.c.G)
    prefetch_tensormap(warp == 8 ? &mp.tmK[lane] : &mp.tmV[lane]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // columns: S of both groups, O of both groups
  const uint32_t tS = tmem, tO = tmem + 2 * kTile;
  pdl_wait();
  const TreeRange range =
      tree_range<kThreads, kTile, C::kRows>(p, kMinUnits, ctl.warp_sum, &ctl.range);
  const int g = p.c.g;
  // Item i of the block (the last is followed by one without tiles).
  auto item_at = [&](int i) -> const TreeItem & {
    wait(i_full + 8 * (i % kItems), (i / kItems) & 1, abort, p.status);
    return ctl.item[i % kItems];
  };

  // the softmax groups take registers from the other roles: 256 * 208 + 128 * 88
  // = 384 * 168, the launch's
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 8) {
    produce<D, kTwo, false>(mp, range, base + C::kKs, k_full, k_empty, abort, lane);
  } else if (warp == 9) {
    produce<D, kTwo, true>(mp, range, base + C::kVs, v_full, v_empty, abort, lane);
  } else if (warp == 10) {
    if (lane == 0) {
      constexpr uint32_t kS = mma_desc(128, kTile, false), kO = mma_desc(128, D, true);
      int nk = 0, nv = 0;
      int np[2] = {0, 0};
      for (int items = 0;; ++items) {
        const TreeItem it = item_at(items);
        if (*abort || it.t0 >= it.t1) break;
        const Jobs jb(it, g, C::kRows);
        wait(q_ready, items & 1, abort, p.status);
        tc_fence_after();
        auto weigh = [&](int j) {  // O += P V of job j
          const int w = j & 1, slot = nv % C::kV;
          if (jb.opens(j)) wait(v_ready + 8 * slot, (nv / C::kV) & 1, abort, p.status);
          wait(p_ready + 8 * w, np[w]++ & 1, abort, p.status);
          tc_fence_after();
          if (!*abort) {
            const bool first = ((j >> 1) % kFold) == 0;  // overwrites O
            const uint32_t v = base + C::kVs + slot * C::kTileBytes;
            const uint32_t a = tS + w * kTile, d = tO + w * 128;
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i) {
              const uint64_t b = smem_desc(v + i * 16 * 128, C::kHalf);
              mma_ts(d, a + 16 * i, b, kO, !(first && i == 0));
              mma_ts(d, a + 16 * i + 8, b, kO, true);
            }
          }
          if (jb.closes(j)) {
            mma_commit(v_empty + 8 * slot);
            ++nv;
          }
          if (j + 2 >= jb.jobs) mma_commit(o_full + 8 * w);
        };
        for (int j = 0; j < jb.jobs; ++j) {
          const int w = j & 1, slot = nk % C::kK;
          if (jb.opens(j)) wait(k_full + 8 * slot, (nk / C::kK) & 1, abort, p.status);
          if (!*abort) {
            // S of this group was last read by the products of job j - 2, issued before:
            // MMAs of one thread run in the order of issue
            const uint32_t q = base + C::kQ + (jb.halves ? w * C::kTileBytes : 0);
            const uint32_t k = base + C::kKs + slot * C::kTileBytes;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t off = (i >> 2) * C::kHalf + (i & 3) * 32;
              mma_ss(tS + w * kTile, smem_desc(q + off, 16), smem_desc(k + off, 16), kS, i > 0);
            }
          }
          mma_commit(s_full + 8 * w);
          if (jb.closes(j)) {
            mma_commit(k_empty + 8 * slot);
            ++nk;
          }
          if (j > 0) weigh(j - 1);
        }
        weigh(jb.jobs - 1);
      }
    }
    __syncwarp();
  } else {
    // items for the other roles, and the V tiles that have to be cleaned
    TreeCursor<kTile, C::kRows> cur(p, range);
    TreeItem it;
    bool more = true;
    for (int items = 0, n = 0; more; ++items) {
      more = cur.next(p, it) && !__any_sync(0xffffffffu, *abort);
      if (!more) it.t0 = it.t1 = 0;
      if (lane == 0) {
        ctl.item[items % kItems] = it;
        mbar_arrive(i_full + 8 * (items % kItems));
      }
      const int len = it.head.n + it.head.T;
      uint32_t notes[4] = {0, 0, 0, 0};
      for (int tile = it.t0; tile < it.t1; ++tile, ++n) {
        const int slot = n % C::kV, t0 = tile * kTile;
        wait(v_full + 8 * slot, (n / C::kV) & 1, abort, p.status);
        if (t0 + kTile > it.head.n) {
          const int first = max(0, it.head.n - t0), valid = min(kTile, len - t0);
          // chunk (16 bytes) x of a row: half x >> 3, place x & 7
          constexpr int CPR = D / 8, RPW = 32 / CPR;  // rows a warp covers at once
          const int x = lane % CPR;
          uint8_t *v = smem + C::kVs + slot * C::kTileBytes + (x >> 3) * C::kHalf + (x & 7) * 16;
#pragma unroll 4
          for (int row = valid + lane / CPR; row < kTile; row += RPW)
            *(uint4 *)(v + row * 128) = make_uint4(0, 0, 0, 0);
          for (int r0 = first; r0 < valid; r0 += 4 * RPW) {
            uint4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = r0 + k * RPW + lane / CPR;
              y[k] = row < valid ? *(const uint4 *)(v + row * 128) : make_uint4(0, 0, 0, 0);
            }
            bool odd = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t e[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                odd |= (e[i] & 0x7f80u) == 0x7f80u || (e[i] & 0x7f800000u) == 0x7f800000u;
            }
            if (!__any_sync(0xffffffffu, odd)) continue;
            // rare: zero the elements and note their drafts
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const int row = r0 + k * RPW + lane / CPR;
              bool hit = false;
              if (row < valid) {
                uint32_t *at = (uint32_t *)(v + row * 128);
                for (int i = 0; i < 4; ++i) {
                  const uint32_t e = at[i];
                  const uint32_t bad = ((e & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                                       ((e & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
                  if (bad) at[i] = e & ~bad;
                  hit |= bad != 0;
                }
              }
              const uint32_t who = __ballot_sync(0xffffffffu, hit);
              for (int rr = 0; rr < RPW; ++rr) {
                const int u = t0 + r0 + k * RPW + rr - it.head.n;
                const uint32_t part = CPR == 32 ? ~0u : (1u << (CPR % 32)) - 1u;
                if (!(who & (part << (rr * CPR)))) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (i == (u >> 5)) notes[i] |= 1u << (u & 31);
              }
            }
          }
          if (lane < 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i == lane) ctl.notes[items % kItems][i] = notes[i];
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready + 8 * slot);
      }
    }
  }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int w = warp >> 2;                       // group
    const int lr = (warp & 3) * 32 + lane;         // TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tS + w * kTile + lanes, o_at = tO + w * 128 + lanes;
    auto fold_at = [&](int grp, int r) {  // float4 index: a thread's are 128 apart
      return ((size_t)blockIdx.x * 2 + grp) * (D / 4) * 128 + r;
    };
    constexpr int CPR = D / 8;  // 16-byte chunks of a query row
    constexpr int kQn = C::kRows * CPR / kSoft;
    uint4 qn[kQn];
    auto new_row = [&](int r) { return (r * p.recip_g) >> 16; };  // r / g, r < 1024
    auto load_q = [&](const TreeItem &t) {
      const int r0 = t.group * C::kRows, n = min(C::kRows, t.head.T * g - r0) * CPR;
#pragma unroll
      for (int k = 0; k < kQn; ++k) {
        const int i = tid + k * kSoft, r = i / CPR, c = i - r * CPR;
        qn[k] = make_uint4(0, 0, 0, 0);
        if (i >= n) continue;
        const int nr = new_row(r0 + r), j = (r0 + r) - nr * g;
        qn[k] = __ldg((const uint4 *)(p.q + (size_t)(t.head.q0 + nr) * p.q_stride +
                                      ((size_t)t.head.h * g + j) * (D * 2) + c * 16));
      }
    };
    int ns = 0, splits = 0;
    int no[2] = {0, 0};
    // One thread says whether item i is worked on, so that all agree even while
    // a wait runs out; a barrier follows.
    auto decide = [&](int i) {
      if (tid != 0) return;
      const TreeItem &t = item_at(i);
      ctl.more[i & 1] = !*abort && t.t0 < t.t1;
    };
    decide(0);
    named_sync(1, kSoft);
    if (ctl.more[0]) load_q(ctl.item[0]);
    for (int items = 0; ctl.more[items & 1]; ++items) {
      const TreeItem &it = ctl.item[items % kItems];  // in shared memory: not worth registers
      const TreeHead &hd = it.head;
      const Jobs jb(it, g, C::kRows);
      const int r0 = it.group * C::kRows;
      // ---- Q rows into shared memory (rows past the last keep what was there:
      // they only reach their own lanes, which nothing reads)
#pragma unroll
      for (int k = 0; k < kQn; ++k) {
        const int i = tid + k * kSoft, r = i / CPR, c = i - r * CPR;
        if (i < jb.rows * CPR)
          *(uint4 *)(smem + C::kQ + (r >> 7) * C::kTileBytes + (c >> 3) * C::kHalf +
                     (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)) = qn[k];
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      const int row = jb.halves ? 128 * w + lr : lr;
      const bool live = (jb.halves ? 128 * w : 0) + (warp & 3) * 32 < jb.rows;  // of the warp
      float m = -INFINITY, l = 0.f;  // reference of the weights (log2 units), sum
      float m_acc = -INFINITY;       // reference of the folded output
      bool folded = false;           // (of the group: every thread folds at the same tiles)
      for (int j = w; j < jb.jobs; j += 2) {
        const int tile = it.t0 + jb.tile(j), t0 = tile * kTile;
        wait(s_full + 8 * w, ns++ & 1, abort, p.status);
        tc_fence_after();
        if (live) {
          const bool turn = j >= 2 && ((j >> 1) % kFold) == 0;  // O starts afresh
          if (turn) {
            // fold the tensor cores' sum of the last kFold tiles into fp32 (see kFold)
            const float f = tree_weight(m_acc, m);
            float4 *acc = (float4 *)p.fold + fold_at(w, lr);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t x[32];
              tmem_ld32(o_at + 32 * c, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (folded) v = __ldcg(acc + (8 * c + e) * 128);
                v.x = fmaf(v.x, f, __uint_as_float(x[4 * e]));
                v.y = fmaf(v.y, f, __uint_as_float(x[4 * e + 1]));
                v.z = fmaf(v.z, f, __uint_as_float(x[4 * e + 2]));
                v.w = fmaf(v.w, f, __uint_as_float(x[4 * e + 3]));
                __stcg(acc + (8 * c + e) * 128, v);
              }
            }
            m_acc = m;
            folded = true;
          }
          if (t0 + kTile > hd.n)
            hide_keys(p, hd, new_row(r0 + row), row < jb.rows, t0 - hd.n, s_at);
          soft_tile<D>(s_at, o_at, p.scale_log2, j >= 2 && !turn, m, l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * w);
      }
      // ---- epilogue (the next item's Q is on its way meanwhile)
      decide(items + 1);
      const TreeItem &nx = item_at(items + 1);
      if (!*abort && nx.t0 < nx.t1) load_q(nx);
      // (a half waits for its own output alone; the barrier before the next item
      // makes the other's phase known)
      if (!jb.halves || w == 0) wait(o_full, no[0] & 1, abort, p.status);
      if (jb.halves ? w == 1 : jb.jobs > 1) wait(o_full + 8, no[1] & 1, abort, p.status);
      ++no[0];
      no[1] += jb.jobs > 1;
      tc_fence_after();
      const bool whole = tree_whole(it);
      uint32_t any = 0;
      if (it.t1 * kTile > hd.n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ctl.notes[items % kItems][i];
      }
      // Weights of the groups' outputs and of their folded parts; which groups this
      // thread's output comes from.
      float M = m, L = l, f0 = 1.f, f1 = 1.f;
      float fa0 = tree_weight(m_acc, m), fa1 = fa0;
      bool use0 = w == 0, use1 = w == 1;
      if (!jb.halves) {
        // both groups hold partial states of the same rows; Q is no longer read
        float4 *st = (float4 *)(smem + C::kQ);
        st[w * 128 + lr] = make_float4(m, l, fa0, 0.f);
        named_sync(1, kSoft);
        const float4 a = st[lr], b = st[128 + lr];
        M = fmaxf(a.x, b.x);
        f0 = tree_weight(a.x, M);
        f1 = tree_weight(b.x, M);
        L = f0 * a.y + f1 * b.y;
        fa0 = a.z;
        fa1 = b.z;
        use0 = true;
        use1 = jb.jobs > 1;
      }
      if (live) {
        const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
        const size_t part = (size_t)tree_slot(range, it) * C::kRows + row;
        float *dst = nullptr;
        if (row < jb.rows) {
          dst = whole ? tree_out(p, hd, r0 + row) : p.part_o + part * D;
          if (!whole && (jb.halves || w == 0)) p.part_ml[part] = make_float2(M, L);
        }
        const int c0 = jb.halves ? 0 : w * (D / 64), c1 = jb.halves ? D / 32 : c0 + D / 64;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            if (!(i ? use1 : use0)) continue;
            const float fi = i ? f1 : f0;
            uint32_t x[32];
            tmem_ld32(tO + i * 128 + lanes + 32 * c, x);
            tmem_wait_ld(x);
            if (jb.jobs > 2 * kFold + i) {
              const float4 *acc = (const float4 *)p.fold + fold_at(i, lr) + 8 * c * 128;
              const float fa = i ? fa1 : fa0;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 v = __ldcg(acc + e * 128);
                x[4 * e] = __float_as_uint(fmaf(v.x, fa, __uint_as_float(x[4 * e])));
                x[4 * e + 1] = __float_as_uint(fmaf(v.y, fa, __uint_as_float(x[4 * e + 1])));
                x[4 * e + 2] = __float_as_uint(fmaf(v.z, fa, __uint_as_float(x[4 * e + 2])));
                x[4 * e + 3] = __float_as_uint(fmaf(v.w, fa, __uint_as_float(x[4 * e + 3])));
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(fi, __uint_as_float(x[e]), o[e]);
          }
          if (any && row < jb.rows) {
            // non-finite values of drafts this row sees (their weight is positive)
            const CacheGroup &grp = p.c.grp[p.c.head_grp[hd.h]];
#pragma unroll 1
            for (int u = 0; u < hd.T; ++u) {
              const uint32_t bit = 1u << (u & 31);
              if (!(ctl.notes[items % kItems][u >> 5] & bit) ||
                  !(tree_mask_word(p, hd, new_row(r0 + row), u >> 5) & bit))
                continue;
              const int tok = hd.n + u;
              const int64_t pg = grp.table[(size_t)hd.b * grp.stride + (tok >> p.c.lgP)];
              if (pg < 0 || pg >= grp.pages) continue;
              const char *v = grp.v + pool_row(p.c, grp, pg, p.c.head_row[hd.h],
                                               tok & (p.c.P - 1)) * (D * 2);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float b = __uint_as_float(
                    (uint32_t)__ldg((const uint16_t *)v + 32 * c + e) << 16);
                if (!isfinite(b)) o[e] += b;
              }
            }
          }
          if (dst) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *(float4 *)(dst + 32 * c + e) =
                  make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        if (tid == 0) ctl.split[splits] = it;
        ++splits;
      }
      named_sync(1, kSoft);  // (m, l) in Q's place are read
    }
    // ---- row groups shared with other blocks, at most two: the last block merges
    if (splits > 0) {
      if (tid < splits) ctl.last[tid] = !*abort && tree_ticket(p, range, ctl.split[tid]);
      named_sync(1, kSoft);
      int phase = 0;
      for (int i = 0; i < splits; ++i)
        if (ctl.last[i])
          merge_parts<D, C::kRows, C::kCtl - C::kKs>(p, range, ctl.split[i], smem + C::kKs, m_full,
                                                     phase, abort, tid);
    }
  }
  __syncthreads();
  // Run-down: nothing of this block may still be landing when it leaves. The
  // roles above end with every load consumed and every product waited for,
  // unless a wait ran out.
  if (*abort) {
    if (tid == 0) {
      // bounded: bulk loads land within microseconds of their issue
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 20000000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == 10) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <int D, bool kTwo>
cudaError_t launch_dt(const MmaParams &mp, int blocks, cudaStream_t st) {
  using C = Cfg<D, kTwo>;
  cudaError_t e = cudaFuncSetAttribute(tree_mma_kernel<D, kTwo>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_mma_kernel<D, kTwo>, mp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int tree_mma_rows(int query_rows) { return query_rows > 128 ? 256 : 128; }

cudaError_t launch_tree_mma(const TreeParams &p, const CUtensorMap *k_maps,
                            const CUtensorMap *v_maps, int blocks, cudaStream_t st) {
  MmaParams mp;
  memcpy(mp.tmK, k_maps, sizeof(mp.tmK));
  memcpy(mp.tmV, v_maps, sizeof(mp.tmV));
  mp.t = p;
  const bool two = p.max_q * p.c.g > 128;
  if (p.c.D == 128)
    return two ? launch_dt<128, true>(mp, blocks, st) : launch_dt<128, false>(mp, blocks, st);
  return two ? launch_dt<64, true>(mp, blocks, st) : launch_dt<64, false>(mp, blocks, st);
}

}  // namespace kvx
