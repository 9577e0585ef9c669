// tree_mma.cu -- attention for a tree of drafted tokens, bf16 cache, on the
// 5th-generation tensor cores (tcgen05).
//
// out[row] = sum_t softmax(scale * <q_row, k_t>)_t v_t over the cached tokens
// of the row's KV head and the drafts its mask shows. The T_b * g query rows of
// a KV head share its keys, so both products are dense: S [128 rows][128 keys]
// = Q K^T and O [128 rows][D] += P V, with S, P and O in tensor memory. One
// pass over the keys with a running reference and sum per row. Two blocks per SM,
// independent of each other, so that one's item changes and softmax run under the
// other's loads and products; each walks its items (tree_split.cuh) in tiles of
// 128 keys:
//  * warps 8 and 9 load K and V tiles from their pages into two rings (bulk
//    tensor loads, one box a page of at most 128 rows, landing as [8-row group][half
//    of the dims][8 rows][128 bytes], 128-byte swizzled);
//  * warp 10 issues the MMAs: S, then O += P V of the tile. An item's first scores are
//    computed under the epilogue of the item before;
//  * warps 0-3 and 4-7 do the softmax: a query row belongs to two threads, one for each
//    half of a tile's keys (a thread can only reach one lane of TMEM). They agree on
//    the row's reference in one barrier with an OR a tile, and keep sums of their own;
//  * warp 11 hands out the items, loads their queries ([half][rows][128 bytes], boxes of
//    8 new rows x the g heads) and cleans the V tiles that hold drafts or the
//    head's end: rows past the end are zeroed to a whole step of 16 keys (stale or
//    padding data; the products stop there), and non-finite values of drafts are
//    replaced by zero and noted, because a weight of 0 does not silence them for rows
//    that do not see the draft; the epilogue adds them to the rows that do.
// P is kept as a bf16 high part and a bf16 residual (two products): with the
// high part alone the weights would be off by 2^-9, with both by 2^-18, below
// the fp32 output's other errors. They overwrite the scores they came from, column
// block by column block.
// Loops are kept rolled, rare paths out of line and the waits small: the roles run side by
// side on one instruction cache. With the output products and the waits unrolled, 256
// short sequences took 121 us instead of 102 (ragged trees 171 instead of 175).
// Measured on one GB300 (a call in a graph): 16 sequences of 8k to 32k, 16 drafts, 4
// query heads a KV head, 84.5 us for 427 MB, of which about 15 are the ramp, the last output
// and the merge (tensor pipe 39 % busy); 8 x 122k, 24 drafts, 650 to 720 us by GPU for 4.0
// GB (5.6 to 6.1 TB/s); 256 of 100 to 1000, 1 to 8 drafts, 102 us for 448 MB; one of 2k,
// 16.1 us. A tile takes a block about 3.3 us: scores, softmax and output products one
// after the other, which two blocks per SM hide from each other for the most part. Tried
// and slower: tiles or V slots of 64 keys; a second V slot where 64 query rows leave room
// for it; the products transposed, so that few query rows fill the tensor cores (a tile
// 2.6 us, but an item 3 to 4 us more); prefetching tiles into L2. (Measured against
// 86 us for the first and 120 for the short sequences.)
// Every mbarrier wait gives up after p.wait_ns (2 s unless a test shortens it), sets
// KVX_DEV_TIMEOUT and lets all roles run to their end without waiting, loading or
// multiplying.
#include <cuda_bf16.h>
#include <math.h>
#include <stddef.h>
#include <string.h>

#include "tcgen05.cuh"
#include "tree_split.cuh"

namespace kvx {
namespace {

constexpr int kTile = 128;       // keys of a tile
constexpr int kThreads = 384;
constexpr int kSoft = 256;       // threads of the softmax warps
constexpr int kMinTiles = 1;     // tiles a block takes at least
constexpr float kGrow = 16.f;    // log2 growth of the maximum that raises the reference
// Tiles after which the output leaves tensor memory for an fp32 sum: the
// tensor cores truncate each of the 16 additions a tile makes to every output
// element, which over 200 tiles was measured as 5e-5 of the output, growing
// linearly; over 16 tiles it stays below 5e-6.
constexpr int kFold = 16;
constexpr int kItems = 4;        // item slots: the epilogue is at most three items behind

struct alignas(16) Ctl {  // small shared state
  uint64_t bars[28];
  uint32_t tmem;
  int abort;
  int more[2];
  int64_t warp_sum[kThreads / 32];
  TreeRange range;
  TreeItem item[kItems];                  // written by warp 11, ahead of the others
  alignas(16) uint32_t notes[kItems][4];  // drafts of an item whose V is not finite
  float swap[2][128];                     // between the two threads of a row
};
static_assert(offsetof(Ctl, notes) % 16 == 0, "read as vectors");

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = D * 2 * 128;       // a Q, K or V tile
  static constexpr int kQHalf = 128 * 128;             // Q: 64 dims of all rows together
  static constexpr int kGroup = 1024 * kHalves;        // K, V: all dims of 8 rows together
  static constexpr int kSlots = (111 * 1024 - kTileBytes) / kTileBytes;  // K and V tiles
  static constexpr int kV = (kSlots + 1) / 2, kK = kSlots - kV;
  static_assert(kK >= 1, "ring depths");
  static constexpr int kBars = 2 * kK + 3 * kV + 5 + kItems;
  static constexpr int kKs = kTileBytes, kVs = kKs + kK * kTileBytes;
  static constexpr int kCtl = kVs + kV * kTileBytes;
  // Two blocks with the 1 KB that the system keeps in each have to fit in 228 KB.
  static constexpr int kSmem = kCtl + (int)sizeof(Ctl);
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks per SM");
};

struct alignas(128) MmaParams {
  CUtensorMap tmK[KVX_MAX_GROUPS];
  CUtensorMap tmV[KVX_MAX_GROUPS];
  CUtensorMap tmQ;
  TreeParams t;
};

// Bounded wait for the phase of `bar` with the given parity. When it runs out, or
// another role's has, waits end at once, the block runs down and reports it at its end.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                     const TreeParams &p) {
  if (mbar_try_wait(bar, parity)) return;
  const uint32_t t0 = timer_ns32();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return;
    if (timer_ns32() - t0 > p.wait_ns) *abort = 1;
  }
}

// Visible keys among the 32 from draft `u0` on (negative: that many cached
// tokens first) for new row i.
__device__ __forceinline__ uint32_t seen_word(const TreeParams &p, const TreeHead &t, int i,
                                              int u0) {
  if (u0 <= -32) return 0xffffffffu;
  const int w = u0 >> 5, s = u0 & 31;  // u0 < 0: w = -1, cached tokens
  const uint32_t lo = w < 0 ? 0xffffffffu : tree_mask_word(p, t, i, w);
  return s ? __funnelshift_r(lo, tree_mask_word(p, t, i, w + 1), s) : lo;
}

// Scores of keys that the row does not see become -inf, in 64 columns whose first key is
// draft u0 (a tile with drafts or the head's end).
__device__ __forceinline__ void hide_keys(const TreeParams &p, const TreeHead &t, int row_i,
                                          bool row_ok, int u0, uint32_t s_at) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    uint32_t x[32];
    const uint32_t seen = row_ok ? seen_word(p, t, row_i, u0 + c) : 0u;
    tmem_get32(s_at + c, x);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((seen >> e) & 1u)) x[e] = __float_as_uint(-INFINITY);
    tmem_st32(s_at + c, x);
  }
  tmem_wait_st();
}

// The largest of 64 scores of a row.
__device__ __forceinline__ float top_score(uint32_t s_at) {
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    uint32_t x[32];
    tmem_get32(s_at + c, x);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      mx0 = max3(mx0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
      mx1 = max3(mx1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
    }
  }
  return fmaxf(mx0, mx1);
}

// x *= f over `cols` TMEM columns.
__device__ __noinline__ void rescale(uint32_t at, int cols, float f) {
  for (int c = 0; c < cols; c += 16) {
    uint32_t y[16];
    tmem_get16(at + c, y);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
    tmem_st16(at + c, y);
  }
  tmem_wait_st();
}

// Weights of keys (at most 64, whole steps of 16) of a row from their scores, in place:
// per 16 keys, 8 columns of high parts and 8 of residuals (two keys a column), the A
// operands of two products. Returns their sum.
__device__ __forceinline__ float weigh(uint32_t s_at, int keys, float scale, float ref) {
  const uint64_t scale2 = pack2(scale, scale), ref2 = pack2(-ref, -ref);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int c = 0; c < keys; c += 16) {
    uint32_t x[16], y[16];
    tmem_get16(s_at + c, x);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float a, b;
      unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, ref2), a, b);
      a = ex2(a);
      b = ex2(b);
      const uint64_t ab = pack2(a, b);
      sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], ab);
      const uint32_t hi = pack_bf16(a, b);
      float ra, rb;
      unpack2(add2(ab, pack2(__uint_as_float((hi << 16) ^ 0x80000000u),
                             __uint_as_float((hi & 0xffff0000u) ^ 0x80000000u))),
              ra, rb);
      y[e >> 1] = hi;
      y[8 + (e >> 1)] = pack_bf16(ra, rb);
    }
    tmem_st16(s_at + c, y);
  }
  float s0, s1, s2, s3;
  unpack2(sum[0], s0, s1);
  unpack2(sum[1], s2, s3);
  tmem_wait_st();
  return (s0 + s1) + (s2 + s3);
}

// x += f * (16 folded output elements), from an acc whose float4s are 128 apart.
__device__ __forceinline__ void add_fold(uint32_t (&x)[16], const float4 *acc, float f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = __ldcg(acc + e * 128);
    x[4 * e] = __float_as_uint(fmaf(v.x, f, __uint_as_float(x[4 * e])));
    x[4 * e + 1] = __float_as_uint(fmaf(v.y, f, __uint_as_float(x[4 * e + 1])));
    x[4 * e + 2] = __float_as_uint(fmaf(v.z, f, __uint_as_float(x[4 * e + 2])));
    x[4 * e + 3] = __float_as_uint(fmaf(v.w, f, __uint_as_float(x[4 * e + 3])));
  }
}

// Adds half an output row to its fp32 sum, scaled by f where there is one yet.
template <int D>
__device__ __noinline__ void fold_out(uint32_t o_at, float4 *acc, bool more, float f) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t x[16];
    tmem_get16(o_at + 16 * c, x);
    if (more) add_fold(x, acc + 4 * c * 128, f);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __stcg((uint4 *)acc + (4 * c + e) * 128,
             make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]));
  }
}

// The other way round: adds the fp32 sum, scaled by f, to the half row.
template <int D>
__device__ __noinline__ void unfold_out(uint32_t o_at, const float4 *acc, float f) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t x[16];
    tmem_get16(o_at + 16 * c, x);
    add_fold(x, acc + 4 * c * 128, f);
    tmem_st16(o_at + 16 * c, x);
  }
  tmem_wait_st();
}

// Adds to half an output row (from dim d0 on) the non-finite values of the noted drafts
// that new row i sees: their weight is positive, so the sum is what they are.
template <int D>
__device__ __noinline__ void add_notes(const TreeParams &p, const TreeHead &hd, int i, int d0,
                                       const uint32_t *notes, float *out) {
  const CacheGroup &grp = p.c.grp[p.c.head_grp[hd.h]];
  for (int u = 0; u < hd.T; ++u) {
    const uint32_t bit = 1u << (u & 31);
    if (!(notes[u >> 5] & bit) || !(tree_mask_word(p, hd, i, u >> 5) & bit)) continue;
    const int tok = hd.n + u;
    const int64_t pg = grp.table[(size_t)hd.b * grp.stride + (tok >> p.c.lgP)];
    if (pg < 0 || pg >= grp.pages) continue;
    const uint16_t *v = (const uint16_t *)(grp.v + pool_row(p.c, grp, pg, p.c.head_row[hd.h],
                                                            tok & (p.c.P - 1)) * (D * 2));
    for (int d = 0; d < D / 2; ++d) {
      const float b = __uint_as_float((uint32_t)v[d0 + d] << 16);
      if (!isfinite(b)) out[d] += b;
    }
  }
}

// Zeroes the non-finite elements of rows r0 .. of a V tile (32 rows' worth of chunks, lanes as in
// the loop that found one) and notes their drafts.
template <int D>
__device__ __noinline__ void note_rows(uint8_t *v0, int r0, int valid, int u0, int lane,
                                       uint32_t *notes) {
  constexpr int CPR = D / 8, RPW = 32 / CPR;
  for (int k = 0; k < 4; ++k) {
    const int row = r0 + k * RPW + lane / CPR;
    bool hit = false;
    if (row < valid) {
      uint32_t *at = (uint32_t *)(v0 + (row >> 3) * (D * 16) + (row & 7) * 128);
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = at[i];
        const uint32_t bad = ((e & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                             ((e & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
        if (bad) at[i] = e & ~bad;
        hit |= bad != 0;
      }
    }
    if (hit) atomicOr(notes + ((u0 + row) >> 5), 1u << ((u0 + row) & 31));
  }
}

// The block's tiles one by one.
struct TileWalk {
  TreeCursor<kTile> cur;
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
template <int D, bool kIsV>
__device__ __forceinline__ void produce(const MmaParams &mp, const TreeRange &range,
                                        uint32_t ring, uint32_t full0, uint32_t empty0,
                                        volatile int *abort, int lane) {
  using C = Cfg<D>;
  constexpr int kN = kIsV ? C::kV : C::kK;
  const TreeParams &p = mp.t;
  const uint64_t pol = policy_evict_first();
  const int P = p.c.P, box = min(P, kTile);
  const int per = kTile / box;  // boxes of a tile: lane i loads box i
  // Two walks over the tiles: `ahead` runs kAhead tiles before `now` and reads
  // the page ids, so that neither the lengths nor the page table hold up a load (but
  // the first tile is on its way before the others' are looked up).
  constexpr int kAhead = 3;
  TileWalk now(p, range), ahead(p, range);
  auto page_of = [&]() {
    if (!ahead.more) return 0;
    const TreeHead &h = ahead.it.head;
    const CacheGroup &grp = p.c.grp[p.c.head_grp[h.h]];
    const int tok = ahead.tile * kTile + lane * box;
    const int page = lane < per && tok < h.n + h.T
                         ? grp.table[(size_t)h.b * grp.stride + (tok >> p.c.lgP)]
                         : 0;
    ahead.step(p);
    return page;
  };
  int pages[kAhead];
  pages[0] = page_of();
  for (int n = 0; now.more; ++n) {
    const TreeHead &h = now.it.head;
    const int gi = p.c.head_grp[h.h], rank = p.c.head_row[h.h];
    const int slot = n % kN, valid = min(kTile, h.n + h.T - now.tile * kTile);
    const int boxes = (valid + box - 1) / box;
    int page = pages[0];
    if (n >= kN) wait(empty0 + 8 * slot, ((n / kN) - 1) & 1, abort, p);
    if (__any_sync(0xffffffffu, *abort)) return;
    const uint32_t full = full0 + 8 * slot;
    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(boxes * box * 128 * C::kHalves));
    __syncwarp();
    if (lane < boxes) {
      if (page < 0 || (int64_t)page >= p.c.grp[gi].pages) {
        atomicOr(p.status, KVX_DEV_BAD_PAGE);
        page = (int)p.c.grp[gi].pages;  // past the last page: loads zeros
      }
      // the box's first 8-row group in the map's last two dims
      const int off = ((now.tile * kTile + lane * box) & (P - 1)) >> 3;
      const int c3 = p.c.token_major ? page * (P >> 3) + off : off;
      const int c4 = p.c.token_major ? rank : page * p.c.grp[gi].size + rank;
      tma_load_5d(ring + slot * C::kTileBytes + lane * box * (D * 2),
                  kIsV ? &mp.tmV[gi] : &mp.tmK[gi], 0, 0, 0, c3, c4, full, pol);
    }
    now.step(p);
#pragma unroll 1
    for (int k = n ? 1 : kAhead; k; --k) {
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) pages[i] = pages[i + 1];
      pages[kAhead - 1] = page_of();
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    tree_mma_kernel(const __grid_constant__ MmaParams mp) {
  using C = Cfg<D>;
  const TreeParams &p = mp.t;
  extern __shared__ __align__(1024) uint8_t smem[];  // tiles start on 1024 bytes
  Ctl &ctl = *(Ctl *)(smem + C::kCtl);
  static_assert(C::kBars <= sizeof(ctl.bars) / 8, "barriers");
  const uint32_t base = smem_u32(smem);
  volatile int *abort = &ctl.abort;
  const uint32_t k_full = smem_u32(ctl.bars), k_empty = k_full + 8 * C::kK;
  const uint32_t v_full = k_empty + 8 * C::kK, v_empty = v_full + 8 * C::kV;
  const uint32_t v_ready = v_empty + 8 * C::kV;  // loaded, and cleaned where it has to be
  const uint32_t s_full = v_ready + 8 * C::kV;   // scores of a tile are ready
  const uint32_t p_ready = s_full + 8;           // weights of a tile are ready
  const uint32_t o_full = p_ready + 8;           // the output of an item is complete
  const uint32_t q_full = o_full + 8;            // queries of an item are loaded
  const uint32_t q_empty = q_full + 8;           // the last scores of an item are done
  const uint32_t i_full = q_empty + 8;           // [kItems] an item is written
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (base & 1023u) {  // no toolchain places it so; nothing below would hold
    if (tid == 0) atomicOr(p.status, KVX_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) {
      // (failure-detection test: one arrival more than will come, so that the wait
      // for this block's first K tile runs out)
      mbar_init(k_full + 8 * i, i == 0 && (int)blockIdx.x == p.stall_block ? 2 : 1);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(v_ready + 8 * i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_ready, kSoft / 32);
    mbar_init(o_full, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < kItems; ++i) mbar_init(i_full + 8 * i, 1);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp >= 8 && warp < 10 && lane < p.c.G)
    prefetch_tensormap(warp == 8 ? &mp.tmK[lane] : &mp.tmV[lane]);
  if (warp == 11 && lane == 0) prefetch_tensormap(&mp.tmQ);
  pdl_wait();
  // (only now: a kernel before that has yet to allocate tensor memory must not find it taken)
  if (warp == 10) {
    tmem_alloc(smem_u32(&ctl.tmem), 256);
    tc_fence_before();
  }
  const TreeRange range = tree_range<kThreads, kTile>(p, kMinTiles, ctl.warp_sum, &ctl.range);
  tc_fence_after();  // (the search for the block's part synchronises it)
  const uint32_t tS = ctl.tmem, tO = tS + kTile;  // TMEM columns of S and O
  // Item i of the block (the last is followed by one without tiles).
  auto item_at = [&](int i) -> const TreeItem & {
    wait(i_full + 8 * (i % kItems), (i / kItems) & 1, abort, p);
    return ctl.item[i % kItems];
  };

  if (warp == 8) {
    produce<D, false>(mp, range, base + C::kKs, k_full, k_empty, abort, lane);
  } else if (warp == 9) {
    produce<D, true>(mp, range, base + C::kVs, v_full, v_empty, abort, lane);
  } else if (warp == 10) {
    if (lane == 0) {
      constexpr uint32_t kS = mma_desc(128, 0, false), kO = mma_desc(128, D, true);
      int n = 0;
      for (int i = 0;; ++i) {
        const TreeItem &it = item_at(i);
        const int tiles = it.t1 - it.t0;
        // keys from the item's first tile on
        const int keys = it.head.n + it.head.T - it.t0 * kTile;
        if (*abort || tiles <= 0) break;
        wait(q_full, i & 1, abort, p);
        for (int j = 0; j < tiles; ++j, ++n) {
          const int ks = n % C::kK, vs = n % C::kV;
          const int steps = min(kTile, keys - j * kTile + 15) / 16;  // of 16 keys
          wait(k_full + 8 * ks, (n / C::kK) & 1, abort, p);
          tc_fence_after();
          if (!*abort) {
            // (P of the tile before was read by products issued before: MMAs of one
            // thread run in the order of issue)
            const uint32_t k = base + C::kKs + ks * C::kTileBytes;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const uint32_t off = (e & 3) * 32;
              mma_ss(tS, smem_desc(base + (e >> 2) * C::kQHalf + off, 0, 1024),
                     smem_desc(k + (e >> 2) * 1024 + off, 0, C::kGroup), kS + (steps << 18),
                     e > 0);
            }
          }
          mma_commit(s_full);
          mma_commit(k_empty + 8 * ks);
          if (j == tiles - 1) mma_commit(q_empty);
          wait(v_ready + 8 * vs, (n / C::kV) & 1, abort, p);
          wait(p_ready, n & 1, abort, p);
          tc_fence_after();
          if (!*abort) {
            // overwrites O (of the item before: its epilogue came before these weights)
            const bool first = j % kFold == 0;
            uint64_t v = smem_desc(base + C::kVs + vs * C::kTileBytes, 1024, C::kGroup);
#pragma unroll 1
            for (int k = 0; k < steps; ++k, v += 2 * C::kGroup / 16) {
              mma_ts(tO, tS + 16 * k, v, kO, !(first && k == 0));
              mma_ts(tO, tS + 16 * k + 8, v, kO, true);
            }
          }
          mma_commit(v_empty + 8 * vs);
        }
        mma_commit(o_full);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // items and queries for the other roles, and the V tiles that have to be cleaned
    TreeCursor<kTile> cur(p, range);
    TreeItem it;
    bool more = true, any_item = false;
    for (int i = 0, n = 0; more; ++i) {
      more = cur.next(p, it) && !__any_sync(0xffffffffu, *abort);
      if (!more) {
        if (lane == 0) tree_describe(p, range, any_item ? &it : nullptr);
        it.t0 = it.t1 = 0;
      }
      any_item = more;
      if (lane == 0) {
        ctl.item[i % kItems] = it;
        mbar_arrive(i_full + 8 * (i % kItems));
      }
      if (!more) break;
      if (i > 0) wait(q_empty, (i - 1) & 1, abort, p);
      if (!__any_sync(0xffffffffu, *abort)) {
        // lane -> (box of 8 new rows, half): at most 16 * 2 of them
        const int boxes = (tree_rows(p, it) + kTreeBox * p.c.g - 1) / (kTreeBox * p.c.g);
        const uint32_t bytes = kTreeBox * p.c.g * 128;
        if (lane == 0) mbar_arrive_expect_tx(q_full, boxes * bytes * C::kHalves);
        __syncwarp();
        const int bx = lane / C::kHalves, half = lane % C::kHalves;
        if (bx < boxes)
          tma_load_5d(base + half * C::kQHalf + bx * bytes, &mp.tmQ, 0, half, it.head.h * p.c.g,
                      it.head.q0 + tree_first(p, it) + bx * kTreeBox, 0, q_full,
                      policy_evict_first());
      }
      const int len = it.head.n + it.head.T;
      if (lane < 4) ctl.notes[i % kItems][lane] = 0;
      __syncwarp();
      for (int tile = it.t0; tile < it.t1; ++tile, ++n) {
        const int slot = n % C::kV, t0 = tile * kTile;
        wait(v_full + 8 * slot, (n / C::kV) & 1, abort, p);
        if (t0 + kTile > it.head.n) {
          const int first = max(0, it.head.n - t0), valid = min(kTile, len - t0);
          // chunk (16 bytes) x of a row: half x >> 3, place x & 7
          constexpr int CPR = D / 8, RPW = 32 / CPR;  // rows a warp covers at once
          const int x = lane % CPR;
          uint8_t *v0 = smem + C::kVs + slot * C::kTileBytes + (x >> 3) * 1024 + (x & 7) * 16;
          auto v = [&](int row) { return v0 + (row >> 3) * C::kGroup + (row & 7) * 128; };
#pragma unroll 1
          for (int row = valid + lane / CPR; row < ((valid + 15) & ~15); row += RPW)
            *(uint4 *)v(row) = make_uint4(0, 0, 0, 0);
          for (int r0 = first; r0 < valid; r0 += 4 * RPW) {
            uint4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = r0 + k * RPW + lane / CPR;
              y[k] = row < valid ? *(const uint4 *)v(row) : make_uint4(0, 0, 0, 0);
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
            note_rows<D>(v0, r0, valid, t0 - it.head.n, lane, ctl.notes[i % kItems]);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready + 8 * slot);
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;  // keys' half; TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tS + lanes + half * 64, o_at = tO + lanes + half * (D / 2);
    // this thread's half of the folded row: float4s, 128 apart
    float4 *acc = (float4 *)p.fold + ((size_t)blockIdx.x * 2 + half) * (D / 8) * 128 + row;
    int n = 0;
    // One thread says whether item i is worked on, so that all agree even while
    // a wait runs out; a barrier follows.
    auto decide = [&](int i) {
      if (tid != 0) return;
      const TreeItem &t = item_at(i);
      ctl.more[i & 1] = !*abort && t.t0 < t.t1;
    };
    decide(0);
    named_sync(1, kSoft);
    for (int i = 0; ctl.more[i & 1]; ++i) {
      const TreeItem &it = ctl.item[i % kItems];  // in shared memory: not worth registers
      const int rows = tree_rows(p, it), tiles = it.t1 - it.t0;
      const bool live = (warp & 3) * 32 < rows;
      float m = -INFINITY, l = 0.f;  // reference of the weights (log2 units), sum
      float m_acc = -INFINITY;       // reference of the folded output
      for (int j = 0; j < tiles; ++j) {
        const int u0 = (it.t0 + j) * kTile - it.head.n;  // the tile's first key as a draft
        // keys of this thread, to whole steps of 16; a tile past its head's end has fewer
        const int keys = live ? min(64, (it.head.T - u0 - half * 64 + 15) & ~15) : 0;
        wait(s_full, n++ & 1, abort, p);
        tc_fence_after();
        const bool turn = j > 0 && j % kFold == 0;  // O starts afresh
        float top = -INFINITY;
        if (live) {
          if (turn) {
            // fold the tensor cores' sum of the last kFold tiles into fp32 (see kFold)
            fold_out<D>(o_at, acc, j > kFold, tree_weight(m_acc, m));
            m_acc = m;
          }
          if (keys > 0) {
            if (u0 + kTile > 0)
              hide_keys(p, it.head, tree_first(p, it) + tree_div_g(p, row), row < rows,
                        u0 + half * 64, s_at);
            top = top_score(s_at) * p.scale_log2;
          }
        }
        // The reference is the maximum of a row's first tile and rises only when a score
        // passes it by more than kGrow: weights and sums are then at most 2^kGrow times
        // larger than with the running maximum, which fp32 and bf16 hold as exactly.
        if (named_or(1, kSoft, top > m + kGrow)) {
          ctl.swap[half][row] = top;
          named_sync(1, kSoft);
          top = fmaxf(top, ctl.swap[half ^ 1][row]);
          const float mn = top > m + kGrow ? top : m;
          const float f = mn == m ? 1.f : tree_weight(m, mn);
          l *= f;
          if (live && j > 0 && !turn && __any_sync(0xffffffffu, f != 1.f))
            rescale(o_at, D / 2, f);
          m = mn;
        }
        if (keys > 0) l += weigh(s_at, keys, p.scale_log2, m == -INFINITY ? 0.f : m);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
      // ---- epilogue
      decide(i + 1);
      wait(o_full, i & 1, abort, p);  // (all have left the last tile)
      tc_fence_after();
      ctl.swap[half][row] = l;
      named_sync(1, kSoft);
      if (live) {
        l += ctl.swap[half ^ 1][row];
        const bool whole = tree_whole(it), ok = row < rows, folded = tiles > kFold;
        float *dst = tree_out(p, it.head.q0 + tree_first(p, it), it.head.h, row);
        float f = 1.f;
        if (whole) {
          f = l == 0.f ? 0.f : 1.f / l;
        } else {
          const size_t at = (size_t)tree_slot(it) * p.group_rows + row;
          dst = p.part_o + at * D;
          if (ok && half == 0) p.part_ml[at] = make_float2(m, l);
        }
        dst += half * (D / 2);
        if (folded) unfold_out<D>(o_at, acc, tree_weight(m_acc, m));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[16];
          tmem_get16(o_at + 16 * c, x);
          if (ok) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *(float4 *)(dst + 16 * c + 4 * e) =
                  make_float4(__uint_as_float(x[4 * e]) * f, __uint_as_float(x[4 * e + 1]) * f,
                              __uint_as_float(x[4 * e + 2]) * f, __uint_as_float(x[4 * e + 3]) * f);
          }
        }
        if (it.t1 * kTile > it.head.n) {
          const uint4 o = *(const uint4 *)ctl.notes[i % kItems];
          if ((o.x | o.y | o.z | o.w) && ok)
            add_notes<D>(p, it.head, tree_first(p, it) + tree_div_g(p, row), half * (D / 2),
                         ctl.notes[i % kItems], dst);
        }
      }
    }
  }
  __syncthreads();
  // Run-down: nothing of this block may still be landing when it leaves. The
  // roles above end with every load consumed and every product waited for,
  // unless a wait ran out.
  if (*abort) {
    if (tid == 0) {
      atomicOr(p.status, KVX_DEV_TIMEOUT);
      // bounded: bulk loads land within microseconds of their issue
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 20000000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == 10) {
    tc_fence_after();
    tmem_free(tS, 256);
  }
}

template <int D>
cudaError_t launch_d(const MmaParams &mp, int blocks, cudaStream_t st) {
  using C = Cfg<D>;
  constexpr int bytes = C::kSmem;
  static int8_t done[64];
  cudaError_t e = raise_smem_limit(done, (const void *)tree_mma_kernel<D>, bytes);
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
  e = cudaLaunchKernelEx(&cfg, tree_mma_kernel<D>, mp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int tree_mma_rows() { return 128; }
int tree_mma_tokens(int g) { return 128 / (kTreeBox * g) * kTreeBox; }
int tree_mma_blocks_per_sm() { return 2; }

cudaError_t launch_tree_mma(const TreeParams &p, const CUtensorMap *k_maps,
                            const CUtensorMap *v_maps, const CUtensorMap &q_map, int blocks,
                            cudaStream_t st) {
  MmaParams mp;
  memcpy(mp.tmK, k_maps, sizeof(mp.tmK));
  memcpy(mp.tmV, v_maps, sizeof(mp.tmV));
  mp.tmQ = q_map;
  mp.t = p;
  return p.c.D == 128 ? launch_d<128>(mp, blocks, st) : launch_d<64>(mp, blocks, st);
}

}  // namespace kvx
