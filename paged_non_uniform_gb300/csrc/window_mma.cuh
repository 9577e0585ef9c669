// window_mma.cuh -- attention with a sliding window and sink tokens over a paged
// cache, on warp-level tensor-core MMAs; bf16 and 4-bit caches.
//
// The keys that a head visits come in tiles of 64 (window_split.cuh), its query rows in
// groups of 4, 8, 16 or 32 (Cfg). Blocks take equal parts of all (row group, tile) units, found on
// the device from the lengths. In a block the producer warps walk the items and load stages of 32
// tokens (4 bits: 64) of K and V into a ring in shared memory; teams of one or more consumer
// warps, each warp with 8 of the group's rows, take the stages in turn. A team holds its own
// reference, sum and output, which meet in shared memory at an item's end. Per stage a warp computes
// S^T = K Q^T (m16n8k16: 16 tokens x 8 query rows), the softmax on the accumulators, turns P into the
// B operand with movmatrix, and O^T = V^T P^T in fresh accumulators that are then added to the
// output in fp32: the tensor cores truncate their sums, and a chain of two 16-token steps keeps
// that below the rounding of P. (mma.sync, not tcgen05: a decode step has 4 to 8 rows of the 128
// that an operand of tcgen05 has, and what it waits for is memory; and three parts of P beside S
// and O are more than tensor memory holds for two blocks an SM.)
// P is split into three bf16 parts (24 bits), 4-bit caches: two fp16 parts (22). With at most
// four query rows (a decode step of up to four heads a KV head) the columns 4 .. 7 repeat
// the rows 0 .. 3, so that one MMA multiplies two parts: high in the first four columns, next in
// the others.
//
// bf16 stages: bulk-tensor boxes of up to 32 tokens of one head, [8-token group][64-dim
// half][8 rows][128 B] with 128-byte swizzle. Tensor-core operands by ldmatrix.
//
// 4-bit stages: bulk copies of the codes and parameters of up to 64 tokens (window.h). Codes become
// fp16 in registers, two at a time: bits put under the exponent of 1024, and one subtraction
// or multiply-add (codes_k, codes_v). They go to the MMAs unscaled:
//   S = sum_g step_g sum_{d in g} q_d c_d + lo_g sum_{d in g} q_d
//   O_d = sum_t (p_t step_t / 2) (2 c_td - 15) + sum_t p_t (lo_t + 7.5 step_t),
// with the group's step and lo of the token, fp32 outside the MMAs. (7.5 centres the codes: with
// 0 .. 15, or 8, the two sums of O would nearly cancel, values having means near 0.) Queries
// and p * step are brought into fp16's range by powers of two, a query row's from its largest
// element, those of p from the largest step so far. V pairs two tokens in a register: a byte
// permute of their words brings equal elements side by side. The MMAs' inner dimension has no order
// of its own, so a lane takes the elements that its loads bring: eight neighbours of both
// groups of a row for V, sixteen for K.
//
// Measured on one GB300 (a call in a graph):
//  * bf16, 16 sequences of 8k to 32k, one token, two of eight heads unlimited, the others with
//    windows of 4096: 89 us for 526 MB (6.0 TB/s; the copy rate in the middle, about 10 us of
//    ramp, last output and merge). 8 x 122k without windows: 577 us for 4.0 GB (6.9 TB/s).
//  * bf16, up to 8 drafts of 5 query heads, windows of 1000 in half of the heads: 210 us for 676 MB.
//    Fixed instruction latencies bound it: 12 consumer warps an SM (128 registers) issue on 38 % of the
//    cycles, the tensor pipe is 38 % busy; products in shorter chains gain nothing. 32 rows in one warp took 413, 16 in one of two warps 254.
//  * 4 bits, 16 sequences of 8k to 32k: 48 us for 121 MB; 8 x 122k 270 us for 1.13 GB (4.2 TB/s).
//    Instructions bound it: about 760 for 32 tokens, 325 of them on the half-rate integer pipe. Without
//    any of that work the loads take 177 us, in batches of four stages; stage by stage they took 559.
//  * 4 bits, several rows of 4 heads, 16 sequences of 8k to 32k (107, 151 and 125 MB): two rows (groups of 8)
//    49 us, four (16) 136, eight 211. Groups of 16 are the slower ones (255 registers, 108 bytes
//    spilled at D 128): in groups of 8 four rows take 101 and eight 157; 8 x 122k, four rows, 579
//    instead of 863. What they have for them is half the row groups against the 2^31 units of a call.
// Tried and slower: with 4 bits (288 at that time) six consumer warps on stages of 32 tokens (334, 342
// in single 16-token steps), on as many stages of 64 as warps (505), four on stages of 32 tokens
// (298), single 16-token steps (297); for 32 rows four blocks an SM (209 -> 219).
#pragma once

#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "window_split.cuh"

namespace kvx {
namespace wmma {

constexpr uint32_t kAll = 0xffffffffu;

// kRows: query rows of a row group, 4 to 32. NB: column blocks of 8 that one warp takes; kCols:
// warps that share a stage, each with its own columns (32 rows in one warp left no registers for
// independent work: up to 8 drafts 413 us). kDup: 4 rows, repeated.
template <int D, bool kQ4, int kRows_>
struct Cfg {
  static constexpr int kRows = kRows_;
  static constexpr bool kDup = kRows == 4;
  static constexpr int kCols = kQ4 || kRows <= 8 ? 1 : kRows / 8;
  static constexpr int NB = kRows <= 8 ? 1 : kRows / 8 / kCols;
  static constexpr int kTokens = kQ4 ? 64 : 32;  // of a stage
  static constexpr int kBox = kWindowBox;        // of a bf16 load, at most
  static constexpr int kTokenBytes = kQ4 ? q4_row_bytes(D) : 2 * D;
  static constexpr int kTile = kTokens * kTokenBytes;  // K (or V) bytes of a stage
  static constexpr int kStage = 2 * kTile;
  static constexpr int kTeams = kQ4 ? (NB == 1 ? 4 : 2) : kCols == 1 ? 3 : kCols == 2 ? 2 : 1;  // takers of stages
  static constexpr int kCons = kTeams * kCols;                                 // consumer warps
  static constexpr int kBlocks = window_mma_blocks_per_sm(kRows);
  static constexpr int kSteps = 2;  // 16-token steps computed together
  static constexpr int kStages = kTeams == 1 ? 3 : 2 * kTeams;
  static constexpr int kProd = kQ4 ? 2 : 1;   // producer warps: K and V, or both in one
  static constexpr int kBatch = kQ4 ? 4 : 1;  // stages that a producer handles at once
  static constexpr int kThreads = 32 * (kCons + kProd);
  static constexpr int kMS = D + 4;  // floats of a row of a team's record
  static constexpr int kRec = kRows * kMS;
  static constexpr int kRing = kStages * kStage;
  // ring | records | (max, sum) [kTeams][kRows] | weights [kRows][8] | barriers, flag
  static constexpr int kSmem =
      1024 + kRing + 4 * kTeams * kRec + 8 * kTeams * kRows + 32 * kRows + 16 * kStages + 16;
  static_assert(kSmem + 2048 <= 227 * 1024 / kBlocks, "resident blocks per SM");
  static_assert(kTeams <= 7, "a row's eighth weight is 1 / sum");
};

__device__ __forceinline__ float bf_low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_high(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ uint32_t hfma2(uint32_t a, __half2 b, __half2 c) {
  const __half2 r = __hfma2(*(const __half2 *)&a, b, c);
  return *(const uint32_t *)&r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*(const __half2 *)&a, *(const __half2 *)&b);
  return *(const uint32_t *)&r;
}
// A word of eight codes as four fp16 pairs (code i, code i + 4), exact: code - 8 for even i, 16 * code
// for odd i. Bytes 0 and 2 (1 and 3) under the exponent of 1024 are 1024 + byte.
__device__ __forceinline__ void codes_k(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t both = __byte_perm(w, 0x64646464u, i ? 0x4341 : 0x4240), low = both & 0xff0fff0fu;
    o[2 * i] = hsub2(low, 0x64086408u);  // 1032
    o[2 * i + 1] = hsub2(both, low);
  }
}
// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
  return d;
}
// 2 * code - 15 of the four nibbles of both 16-bit halves, exact: a code's bits one place up, with
// a one below them, under the exponent of 1024 are 1024 + 2 code + 1, or 16 times that.
__device__ __forceinline__ void codes_v(uint32_t y, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t s = i ? y >> 7 : y << 1;
    o[2 * i] = hsub2(and_or(s, 0x001e001eu, 0x64016401u), 0x64106410u);  // 1040
    o[2 * i + 1] = hfma2(and_or(s, 0x01e001e0u, 0x64106410u), __float2half2_rn(0.0625f), __float2half2_rn(-80.f));
  }
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *(const uint32_t *)&v;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*(const __half2 *)&v); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*(unsigned long long *)&d)
      : "l"(*(unsigned long long *)&a), "l"(*(unsigned long long *)&b), "l"(*(unsigned long long *)&c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*(unsigned long long *)&d)
      : "l"(*(unsigned long long *)&a), "l"(*(unsigned long long *)&b));
  return d;
}
__device__ __forceinline__ void add4(float (&o)[4], const float (&a)[4]) {
  const float2 u = add2(make_float2(o[0], o[1]), make_float2(a[0], a[1]));
  const float2 v = add2(make_float2(o[2], o[3]), make_float2(a[2], a[3]));
  o[0] = u.x, o[1] = u.y, o[2] = v.x, o[3] = v.y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// d = a * b + (kFirst ? s of the column : d), m16n8k16, fp16 or bf16 inputs, fp32 accumulate.
template <bool kF16, bool kFirst>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1, float s0 = 0.f, float s1 = 0.f) {
  const float c0 = kFirst ? s0 : d[0], c1 = kFirst ? s1 : d[1], c2 = kFirst ? s0 : d[2],
              c3 = kFirst ? s1 : d[3];
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Bulk copy of `bytes` (a multiple of 16) to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                          uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}

__device__ __forceinline__ void zero16(uint32_t a) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
}

// The stages of an item: one a tile (kTokens 64), or two a tile, of which the last one's second is
// left out where the head ends before it.
template <int kTokens>
__device__ __forceinline__ int item_stages(const TreeItem &it) {
  constexpr int kPer = kWindowTile / kTokens;
  if constexpr (kPer == 1) return it.t1 - it.t0;
  const int end = it.head.n + it.head.T;
  const int last = window_tile(it.head, it.t1 - 1) * kWindowTile;
  return kPer * (it.t1 - it.t0) - (end - last <= kTokens ? 1 : 0);
}
template <int kTokens>
__device__ __forceinline__ int stage_token(const TreeItem &it, int st) {
  constexpr int kPer = kWindowTile / kTokens;
  return window_tile(it.head, it.t0 + st / kPer) * kWindowTile + st % kPer * kTokens;
}

// ---- producer ----------------------------------------------------------------
template <int D, bool kQ4, int kRows>
__device__ __forceinline__ void produce(const WindowMmaParams &mp, const TreeRange &range,
                                        uint32_t ring, uint32_t full0, uint32_t empty0,
                                        volatile int *abort_flag, int which, int lane) {
  using C = Cfg<D, kQ4, kRows>;
  const WindowParams &p = mp.w;
  const int P = p.c.P, box = min(P, kQ4 ? C::kTokens : C::kBox), lb = 31 - __clz(box);
  const uint32_t box_bytes = (uint32_t)box * C::kTokenBytes;
  // Keys of a window are read once, by one block (row groups past the first find them in L2).
  const uint64_t pol = policy_evict_first();
  TreeCursor<kWindowTile> cur(p, range);
  TreeItem it;
  int gs = 0;
  bool dead = false;
  while (!dead && cur.next(p, it)) {
    const TreeHead &hd = it.head;
    const int gi = p.c.head_grp[hd.h], rank = p.c.head_row[hd.h];
    const CacheGroup &grp = p.c.grp[gi];
    const int32_t *table = grp.table + (size_t)hd.b * grp.stride;
    const int end = hd.n + hd.T, nst = item_stages<C::kTokens>(it);
    // A batch of stages at a time, a lane for every box: the loop itself takes a warp some 700
    // cycles, three times what a 4-bit stage of 4.6 KB may take. The ids of a batch's pages are
    // looked up a batch ahead.
    const int sub = (lane << lb) / C::kTokens, off = (lane << lb) % C::kTokens;
    auto token = [&](int st) { return sub < C::kBatch && st + sub < nst ? stage_token<C::kTokens>(it, st + sub) + off : end; };
    auto look = [&](int st) {
      const int t = token(st);
      return t < end ? table[t >> p.c.lgP] : -2;
    };
    int next = look(0);
    for (int st = 0; st < nst; st += C::kBatch) {
      const int mine_gs = gs + sub, slot = mine_gs % C::kStages, page = next, t = token(st);
      const bool use = sub < C::kBatch && st + sub < nst;  // this lane's stage exists
      next = look(st + C::kBatch);
      bool ok = true;
      if (use && mine_gs >= C::kStages)
        ok = !*abort_flag && mbar_wait(empty0 + 8 * slot, ((mine_gs / C::kStages) - 1) & 1, p.wait_ns);
      if (!__all_sync(kAll, ok)) {
        if (lane == 0) {
          atomicOr(p.status, KVX_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        dead = true;
        break;
      }
      const uint32_t full = full0 + 8 * slot, tile = ring + slot * C::kStage;
      const bool mine = t < end, bad = mine && (page < 0 || page >= grp.pages);
      if (bad) atomicOr(p.status, KVX_DEV_BAD_PAGE);
      uint32_t live = __ballot_sync(kAll, mine);
      // 4-bit tiles: codes of the tokens, then their parameters
      constexpr int kCode = q4_code_bytes(D), kParam = q4_param_bytes(D);
      const uint32_t cd = tile + (uint32_t)off * kCode;
      const uint32_t pd = tile + C::kTokens * kCode + (uint32_t)off * kParam;
      if (kQ4 && __any_sync(kAll, bad)) {
        // no box to point past the pool's end: zeros from here
        if (bad)
          for (int k = which; k < 2; k += C::kProd) {
            for (uint32_t i = 0; i < (uint32_t)kCode << lb; i += 16) zero16(cd + k * C::kTile + i);
            for (uint32_t i = 0; i < (uint32_t)kParam << lb; i += 16) zero16(pd + k * C::kTile + i);
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        live = __ballot_sync(kAll, mine && !bad);
      }
      __syncwarp();
      if (use && off == 0) {
        const uint32_t boxes = __popc(live >> lane & ((2u << ((C::kTokens >> lb) - 1)) - 1u));
        mbar_arrive_expect_tx(full, (C::kProd == 2 ? 1u : 2u) * box_bytes * boxes);
      }
      __syncwarp();
      // Failure-detection test only: the chosen block arms its first stage but loads nothing.
      const bool stall = mine_gs == 0 && (int)blockIdx.x == p.stall_block;
      gs += min(C::kBatch, nst - st);
      if (!mine || stall) continue;
      if constexpr (kQ4) {
        if (!bad) {
          const int part = t & (P - 1);  // 0, or half of a page of 128
          const int64_t block = (((int64_t)page * grp.size + rank) * P) * q4_row_bytes(D);
          for (int k = which; k < 2; k += C::kProd) {  // K, V
            const char *src = (k ? grp.v : grp.k) + block;
            bulk_load(cd + k * C::kTile, src + part * kCode, (uint32_t)kCode << lb, full, pol);
            bulk_load(pd + k * C::kTile, src + P * kCode + part * kParam, (uint32_t)kParam << lb, full, pol);
          }
        }
      } else {
        const int row8 = (t & (P - 1)) >> 3;         // 8-row group in the page
        const int pg = bad ? (int)grp.pages : page;  // past the last page: zeros
        const int c3 = p.c.token_major ? pg * (P >> 3) + row8 : row8;
        const int c4 = p.c.token_major ? rank : pg * grp.size + rank;
        const uint32_t dst = tile + (uint32_t)off * C::kTokenBytes;
        tma_load_5d(dst, &mp.tmK[gi], 0, 0, 0, c3, c4, full, pol);
        tma_load_5d(dst + C::kTile, &mp.tmV[gi], 0, 0, 0, c3, c4, full, pol);
      }
    }
  }
  // Do not leave while a load of ours may still be landing.
  if (lane == 0)
    for (int s = 0; s < C::kStages && s < gs; ++s) {
      const int last = s + ((gs - 1 - s) / C::kStages) * C::kStages;
      if (!mbar_wait(full0 + 8 * s, (last / C::kStages) & 1, p.wait_ns))
        atomicOr(p.status, KVX_DEV_TIMEOUT);
    }
}

// ---- consumers -----------------------------------------------------------------
// What a consumer warp keeps of its item. Accumulator fragments: lane r * 4 + c holds rows r and
// r + 8 of a tile (tokens of S, dims of O) and the query rows 2c, 2c + 1 of each column block.
template <int D, bool kQ4, int NB>
struct State {
  static constexpr int NK = D / 16, NG = kQ4 ? D / 64 : 1;
  float o[NK][NB][4];
  float ref[NB][2], l[NB][2];  // weights are 2^(score - ref): the maximum, or a little less
  // 4-bit: sum of p (lo + 7.5 step) over this lane's tokens, by group (repeated rows: z[0], of
  // group 0 in lanes c < 2, else of the last); o is in units of 1 / vscale, good for steps up to vtop
  float z[NG][NB][2], vscale, vtop;
};

// Query fragments.
template <int D, int NB>
struct Queries {
  uint32_t f[NB][D / 16][2];
  __device__ __forceinline__ uint2 get(int nb, int j) const { return make_uint2(f[nb][j][0], f[nb][j][1]); }
};

// What the rows of an item see.
struct View {
  Window win;
  int n, i0, i1, rows;  // cached tokens, first and last new row, query rows of the item
  int recip_g;
  // position of query row r, -1 where there is none
  __device__ __forceinline__ int pos(int r) const { return r < rows ? n + i0 + ((r * recip_g) >> 16) : -1; }
};

// Scores of kSteps * 16 tokens, not yet scaled; `tile`: their first token's rows of K.
template <int D, int NB, int kSteps, class Q>
__device__ __forceinline__ void scores_bf16(uint32_t tile, const Q &q, float (&x)[kSteps][NB][4], int lane) {
  const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt) {
    const uint32_t row = tile + (uint32_t)(2 * mt + (mi & 1)) * (D * 16) + (uint32_t)lr * 128u;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4(row + (uint32_t)(j >> 2) * 1024u + ((uint32_t)(((2 * j) & 7) + (mi >> 1)) ^ (uint32_t)lr) * 16u,
              a0, a1, a2, a3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint2 b = q.get(nb, j);
        if (j == 0)
          mma<false, true>(x[mt][nb], a0, a1, a2, a3, b.x, b.y);
        else
          mma<false, false>(x[mt][nb], a0, a1, a2, a3, b.x, b.y);
      }
    }
  }
}

// qs: sums of the queries' elements by group, qe: 8 times those with even places.
template <int D, int NB, int kSteps, class Q>
__device__ __forceinline__ void scores_q4(const uint8_t *codes, const uint8_t *params, const Q &q,
                                          const float (&qs)[D / 64][NB][2], const float (&qe)[D / 64][NB][2],
                                          float (&x)[kSteps][NB][4], int lane) {
  constexpr int NG = D / 64, kCode = q4_code_bytes(D), kParam = q4_param_bytes(D);
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt) {
    // rows r and r + 8: words 2c and 2c + 1 of each group, [row][group][word]
    uint32_t w[2][NG][2], pr[2][NG];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 16 * mt + 8 * u + r;
      if constexpr (D == 128) {
        const uint4 v = *(const uint4 *)(codes + t * kCode + 16 * c);
        const uint2 pp = *(const uint2 *)(params + t * kParam);
        w[u][0][0] = v.x, w[u][NG - 1][0] = v.y, w[u][0][1] = v.z, w[u][NG - 1][1] = v.w;
        pr[u][0] = pp.x, pr[u][NG - 1] = pp.y;
      } else {
        const uint2 v = *(const uint2 *)(codes + t * kCode + 8 * c);
        w[u][0][0] = v.x, w[u][0][1] = v.y;
        pr[u][0] = *(const uint32_t *)(params + t * kParam);
      }
    }
#pragma unroll
    for (int gq = 0; gq < NG; ++gq) {
      float acc[NB][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[2][4];  // [row][pair]
        codes_k(w[0][gq][h], a[0]);
        codes_k(w[1][gq][h], a[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 b = q.get(nb, 4 * gq + 2 * h + j);
            if (h == 0 && j == 0)
              mma<true, true>(acc[nb], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y, qe[gq][nb][0], qe[gq][nb][1]);
            else
              mma<true, false>(acc[nb], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1], b.x, b.y);
          }
      }
      const float s0 = bf_low(pr[0][gq]), s1 = bf_low(pr[1][gq]), l0 = bf_high(pr[0][gq]), l1 = bf_high(pr[1][gq]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float l = e < 2 ? l0 : l1, v = qs[gq][nb][e & 1];
          x[mt][nb][e] = fmaf(e < 2 ? s0 : s1, acc[nb][e], gq == 0 ? l * v : fmaf(l, v, x[mt][nb][e]));
        }
    }
  }
}

// A stage's weights may be up to 2^kSlack before the reference rises to the maximum: most stages
// then need neither the columns' maxima nor a rescaled output. (4-bit caches: p * step stays
// below 2^(12 + kSlack) in fp16.)
constexpr float kSlack = 3.f;
constexpr float kNoRef = -FLT_MAX;  // of a row that has seen nothing

// x[mt][nb][e]: token mt * 16 + r (+ 8 for e >= 2), query row 8 nb + 2c + (e & 1). Masks and
// scales the scores, stores them where weights want them, and makes them weights. seen (kEdge):
// bit (mt * NB + nb) * 4 + e.
template <int D, bool kQ4, int NB, int kSteps, bool kDup, bool kEdge>
__device__ __forceinline__ void softmax(float (&x)[kSteps][NB][4], const float (&scale)[kQ4 ? NB : 1][2],
                                        const View &vw, int t0, State<D, kQ4, NB> &s,
                                        uint32_t &seen, float *scores, int score_rows, int row0, int lane) {
  const int r = lane >> 2, c = lane & 3;
  seen = 0;
  auto sc = [&](int nb, int k) { return scale[kQ4 ? nb : 0][k]; };
  if constexpr (kEdge) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = row0 + 8 * nb + 2 * c + (e & 1);
          const bool see = window_sees(vw.win, vw.pos(kDup ? q & 3 : q), t0 + mt * 16 + r + ((e >> 1) << 3));
          seen |= (see ? 1u : 0u) << ((mt * NB + nb) * 4 + e);
          x[mt][nb][e] = see ? x[mt][nb][e] : -INFINITY;
        }
  }
  if (scores) {
#pragma unroll
    for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (row0 + 8 * nb + 2 * c < score_rows) {
          float *at = scores + (size_t)(mt * 16 + r) * score_rows + row0 + 8 * nb + 2 * c;
          *(float2 *)at = make_float2(x[mt][nb][0] * sc(nb, 0), x[mt][nb][1] * sc(nb, 1));
          *(float2 *)(at + 8 * score_rows) =
              make_float2(x[mt][nb][2] * sc(nb, 0), x[mt][nb][3] * sc(nb, 1));
        }
  }
  float y[kSteps][NB][4];  // relative to the reference
  auto relate = [&]() {
    float top = -INFINITY;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          // The product is rounded as the reference was: one multiply-add would leave the reference's
          // rounding in all weights, which passes any number where scores are large. (A packed product
          // and sum are joined into one by the assembler; __fmul_rn is not.)
          const float2 v = add2(make_float2(__fmul_rn(x[mt][nb][e], sc(nb, 0)), __fmul_rn(x[mt][nb][e + 1], sc(nb, 1))),
                                make_float2(-s.ref[nb][0], -s.ref[nb][1]));
          y[mt][nb][e] = v.x, y[mt][nb][e + 1] = v.y;
          top = fmaxf(top, fmaxf(v.x, v.y));
        }
    return top;
  };
  if (__any_sync(kAll, relate() > kSlack)) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kSteps; ++mt) mx = fmaxf(mx, fmaxf(x[mt][nb][k], x[mt][nb][k + 2]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, sh));
        const float ref = fmaxf(s.ref[nb][k], mx * sc(nb, k)), f = ex2(s.ref[nb][k] - ref);
        s.ref[nb][k] = ref;
        s.l[nb][k] *= f;
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm) s.o[dm][nb][k] *= f, s.o[dm][nb][k + 2] *= f;
        if constexpr (kQ4) {
#pragma unroll
          for (int gq = 0; gq < D / 64; ++gq) s.z[gq][nb][k] *= f;
        }
      }
    relate();
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float2 sum = make_float2(s.l[nb][0], s.l[nb][1]), part = both(0.f);
#pragma unroll
    for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        x[mt][nb][e] = ex2(y[mt][nb][e]);
        x[mt][nb][e + 1] = ex2(y[mt][nb][e + 1]);
        part = add2(part, make_float2(x[mt][nb][e], x[mt][nb][e + 1]));
      }
    sum = add2(sum, part);
    s.l[nb][0] = sum.x, s.l[nb][1] = sum.y;
  }
}

// Whether some row of the item sees token t.
__device__ __forceinline__ bool any_sees(const View &vw, int t) {
  return window_any_sees(vw.win, vw.n, vw.i0, vw.i1, t);
}

template <int D, int NB, int kSteps, bool kDup, bool kEdge, class S>
__device__ __forceinline__ void values_bf16(uint32_t tile, const float (&x)[kSteps][NB][4],
                                            const View &vw, int t0, S &s, uint32_t seen, int lane) {
  const int c = lane & 3, mi = lane >> 3, lr = lane & 7;
  // P^T as the B operand (inner dimension tokens), in parts; repeated rows: the first two parts
  // in one operand, the third and zeros in another.
  constexpr int kParts = kDup ? 2 : 3;
  uint32_t b[kParts][kSteps][NB][2], bv[kSteps][NB][2];
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p0 = x[mt][nb][2 * u], p1 = x[mt][nb][2 * u + 1];
        const uint32_t h = pack_bf16(p0, p1);
        const float2 e = fma2(unpack_bf16(h), both(-1.f), make_float2(p0, p1));
        const uint32_t m = pack_bf16(e.x, e.y);
        const float2 f = fma2(unpack_bf16(m), both(-1.f), e);
        const uint32_t l = pack_bf16(f.x, f.y);
        if constexpr (kDup) {
          b[0][mt][nb][u] = movmatrix_t(c < 2 ? h : m);
          b[1][mt][nb][u] = movmatrix_t(c < 2 ? l : 0u);
        } else {
          b[0][mt][nb][u] = movmatrix_t(h);
          b[1][mt][nb][u] = movmatrix_t(m);
          b[kParts - 1][mt][nb][u] = movmatrix_t(l);
        }
        if constexpr (kEdge) {  // 1 where the row sees the token
          const uint32_t v = seen >> ((mt * NB + nb) * 4 + 2 * u);
          bv[mt][nb][u] = movmatrix_t((v & 1u ? 0x3f80u : 0u) | (v & 2u ? 0x3f800000u : 0u));
        }
      }
  // This lane's tokens in V^T fragments: 2c, 2c + 1 and 8 on; masked where no row sees them.
  uint32_t mask[kSteps][2];
  if constexpr (kEdge) {
#pragma unroll
    for (int k = 0; k < 2 * kSteps; ++k) {
      const int t = t0 + 8 * k + 2 * c;
      mask[k >> 1][k & 1] = (any_sees(vw, t) ? 0xffffu : 0u) | (any_sees(vw, t + 1) ? 0xffff0000u : 0u);
    }
  }
#pragma unroll
  for (int dm = 0; dm < D / 16; ++dm) {
    uint32_t a[kSteps][4];
#pragma unroll
    for (int mt = 0; mt < kSteps; ++mt) {
      const uint32_t row = tile + (uint32_t)(2 * mt + (mi >> 1)) * (D * 16) + (uint32_t)lr * 128u;
      ldsm_x4_t(row + (uint32_t)(dm >> 2) * 1024u +
                    ((uint32_t)(((2 * dm) & 7) + (mi & 1)) ^ (uint32_t)lr) * 16u,
                a[mt][0], a[mt][1], a[mt][2], a[mt][3]);
      if constexpr (kEdge) {
#pragma unroll
        for (int k = 0; k < 4; ++k) a[mt][k] &= mask[mt][k >> 1];
      }
    }
    // Non-finite elements of tokens that only some rows see: left out of the products, and
    // counted for the rows that see them, whose output becomes NaN.
    bool odd = false;
    if constexpr (kEdge) {
      if (vw.i1 > vw.i0) {
        uint32_t nf[kSteps][4], all = 0;
#pragma unroll
        for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t v = a[mt][k] & 0x7f807f80u;
            nf[mt][k] = ((v & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                        ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
            all |= nf[mt][k];
          }
        odd = __any_sync(kAll, all != 0);
        if (odd) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float cnt[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int mt = 0; mt < kSteps; ++mt)
              mma_bf16(cnt, nf[mt][0] & 0x3f803f80u, nf[mt][1] & 0x3f803f80u, nf[mt][2] & 0x3f803f80u,
                       nf[mt][3] & 0x3f803f80u, bv[mt][nb][0], bv[mt][nb][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cnt[e] != 0.f) s.o[dm][nb][e] = __uint_as_float(0x7fc00000u);
          }
#pragma unroll
          for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) a[mt][k] &= ~nf[mt][k];
        }
      }
    }
    float acc[NB][4];
#pragma unroll
    for (int k = kParts - 1; k >= 0; --k)  // small parts first; the column blocks side by side
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          if (k == kParts - 1 && mt == 0)
            mma<false, true>(acc[nb], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b[k][mt][nb][0], b[k][mt][nb][1]);
          else
            mma<false, false>(acc[nb], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b[k][mt][nb][0], b[k][mt][nb][1]);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) add4(s.o[dm][nb], acc[nb]);
  }
}

template <int D, int NB, int kSteps, bool kDup, bool kEdge, class S>
__device__ __forceinline__ void values_q4(const uint8_t *codes, const uint8_t *params,
                                          const float (&x)[kSteps][NB][4],
                                          const View &vw, int t0, S &s, uint32_t seen, int lane) {
  constexpr int NG = D / 64, kCode = q4_code_bytes(D), kParam = q4_param_bytes(D);
  const int r = lane >> 2, c = lane & 3;
  // Words r of tokens 2c, 2c + 1 of each half step; lanes with odd c read the odd one first, so
  // that a load's four tokens lie in all banks.
  uint32_t wa[kSteps][2][NG], wb[kSteps][2][NG];
  uint32_t pr[kSteps][2][NG];  // parameters of token r of each half step
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 16 * mt + 8 * u;
      const uint8_t *row = codes + t * kCode + r * (D / 16);
      const uint8_t *f = row + (2 * c + (c & 1)) * kCode, *g = row + (2 * c + 1 - (c & 1)) * kCode;
      const uint8_t *pa = params + (t + r) * kParam;
      if constexpr (D == 128) {
        const uint2 va = *(const uint2 *)f, vb = *(const uint2 *)g, vp = *(const uint2 *)pa;
        wa[mt][u][0] = va.x, wa[mt][u][NG - 1] = va.y;
        wb[mt][u][0] = vb.x, wb[mt][u][NG - 1] = vb.y;
        pr[mt][u][0] = vp.x, pr[mt][u][NG - 1] = vp.y;
      } else {
        wa[mt][u][0] = *(const uint32_t *)f;
        wb[mt][u][0] = *(const uint32_t *)g;
        pr[mt][u][0] = *(const uint32_t *)pa;
      }
      if constexpr (kEdge) {  // a token that no row sees may hold anything
        if (!any_sees(vw, t0 + t + r))
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) pr[mt][u][gq] = 0u;
      }
    }
  // Scale for p * step: the largest step so far becomes 2^11 to 2^12. (bf16 steps are compared as
  // numbers, two at a time with what shares their register.)
  __nv_bfloat162 most = *(const __nv_bfloat162 *)&pr[0][0][0];
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int gq = 0; gq < NG; ++gq) most = __hmax2(most, *(const __nv_bfloat162 *)&pr[mt][u][gq]);
  if (__any_sync(kAll, __low2float(most) > s.vtop)) {
    float top = __low2float(most);
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, sh));
    const uint32_t bits = __float_as_uint(top);
    s.vtop = __uint_as_float(bits | 0x007f0000u);  // (the largest bf16 of its exponent)
    const float scale = __uint_as_float((uint32_t)min(227, 265 - (int)(bits >> 23)) << 23);
    const float f = scale / s.vscale;
    s.vscale = scale;
#pragma unroll
    for (int dm = 0; dm < D / 16; ++dm)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.o[dm][nb][e] *= f;
  }
  // Sums with the middles: repeated rows' lanes c >= 2 take the second group's, so that every
  // lane has one (D 128).
  constexpr int kMid = kDup ? 1 : NG;
  float2 z[kMid][NB];
#pragma unroll
  for (int k = 0; k < kMid; ++k)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) z[k][nb] = make_float2(s.z[k][nb][0], s.z[k][nb][1]);
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < kMid; ++k) {
        const uint32_t q = kDup ? (c < 2 ? pr[mt][u][0] : pr[mt][u][NG - 1]) : pr[mt][u][k];
        const float mid = fmaf(7.5f, bf_low(q), bf_high(q));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float2 w = make_float2(x[mt][nb][2 * u], x[mt][nb][2 * u + 1]);
          if constexpr (kEdge) {  // what a row does not see may be anything
            const uint32_t v = seen >> ((mt * NB + nb) * 4 + 2 * u);
            z[k][nb].x += v & 1u ? w.x * mid : 0.f;
            z[k][nb].y += v & 2u ? w.y * mid : 0.f;
          } else {
            z[k][nb] = make_float2(fmaf(w.x, mid, z[k][nb].x), fmaf(w.y, mid, z[k][nb].y));
          }
        }
      }
#pragma unroll
  for (int k = 0; k < kMid; ++k)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s.z[k][nb][0] = z[k][nb].x, s.z[k][nb][1] = z[k][nb].y;
  const float lower = kDup && c >= 2 ? -1.f : 0.f;  // this lane's part of a split weight
  // two bytes of the even token, then of the odd one
  const uint32_t sel_lo = c & 1 ? 0x1054u : 0x5410u, sel_hi = c & 1 ? 0x3276u : 0x7632u;
#pragma unroll
  for (int gq = 0; gq < NG; ++gq) {
    uint32_t bh[kSteps][NB][2], bl[kSteps][NB][2];
#pragma unroll
    for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float sv = bf_low(pr[mt][u][gq]) * s.vscale;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float2 w = make_float2(x[mt][nb][2 * u] * sv, x[mt][nb][2 * u + 1] * sv);
          if constexpr (kEdge) {
            const uint32_t v = seen >> ((mt * NB + nb) * 4 + 2 * u);
            if (!(v & 1u)) w.x = 0.f;
            if (!(v & 2u)) w.y = 0.f;
          }
          const uint32_t h = pack_f16(w.x, w.y);
          const float2 rest = fma2(unpack_f16(h), both(kDup ? lower : -1.f), w);
          const uint32_t l = pack_f16(rest.x, rest.y);
          if constexpr (kDup) {
            bh[mt][nb][u] = movmatrix_t(l);  // (c < 2: the weight itself, so the high part)
          } else {
            bh[mt][nb][u] = movmatrix_t(h);
            bl[mt][nb][u] = movmatrix_t(l);
          }
        }
      }
#pragma unroll
    for (int e2 = 0; e2 < 2; ++e2) {  // elements 4 e2 .. 4 e2 + 3 of the words
      uint32_t a[kSteps][2][4];
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          codes_v(__byte_perm(wa[mt][u][gq], wb[mt][u][gq], e2 ? sel_hi : sel_lo), a[mt][u]);
#pragma unroll
      for (int e = 2 * e2; e < 2 * e2 + 2; ++e) {  // dims 8r + 2e and 8r + 2e + 1 of the group
      const int k0 = 2 * (e & 1);
      const int dm = 4 * gq + e;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float acc[4];
        if constexpr (!kDup) {
#pragma unroll
          for (int mt = 0; mt < kSteps; ++mt)
            if (mt == 0)
              mma<true, true>(acc, a[mt][0][k0], a[mt][0][k0 + 1], a[mt][1][k0], a[mt][1][k0 + 1], bl[mt][nb][0], bl[mt][nb][1]);
            else
              mma<true, false>(acc, a[mt][0][k0], a[mt][0][k0 + 1], a[mt][1][k0], a[mt][1][k0 + 1], bl[mt][nb][0], bl[mt][nb][1]);
        }
#pragma unroll
        for (int mt = 0; mt < kSteps; ++mt)
          if (kDup && mt == 0)
            mma<true, true>(acc, a[mt][0][k0], a[mt][0][k0 + 1], a[mt][1][k0], a[mt][1][k0 + 1], bh[mt][nb][0], bh[mt][nb][1]);
          else
            mma<true, false>(acc, a[mt][0][k0], a[mt][0][k0 + 1], a[mt][1][k0], a[mt][1][k0 + 1], bh[mt][nb][0], bh[mt][nb][1]);
        add4(s.o[dm][nb], acc);
      }
      }
    }
  }
}

// One stage. kEdge: some row does not see all of it.
template <int D, bool kQ4, int kRows, bool kEdge, int NB>
__device__ __forceinline__ void consume(const uint8_t *kt, const uint8_t *vt, const View &vw, int t0,
                                        const Queries<D, NB> &q, const float (&qs)[kQ4 ? D / 64 : 1][NB][2],
                                        const float (&qe)[kQ4 ? D / 64 : 1][NB][2],
                                        const float (&scale)[kQ4 ? NB : 1][2], State<D, kQ4, NB> &s,
                                        float *scores, int score_rows, int row0, int lane) {
  using C = Cfg<D, kQ4, kRows>;
  constexpr int kSteps = C::kSteps;
  constexpr bool kDup = C::kDup;
#pragma unroll 1
  for (int h = 0; h < C::kTokens; h += 16 * kSteps) {
    float x[kSteps][NB][4];
    uint32_t seen;
    constexpr int kCode = q4_code_bytes(D), kParam = q4_param_bytes(D);
    if constexpr (kQ4)
      scores_q4<D, NB, kSteps>(kt + h * kCode, kt + C::kTokens * kCode + h * kParam, q, qs, qe, x, lane);
    else
      scores_bf16<D, NB, kSteps>(smem_u32(kt) + h * (2 * D), q, x, lane);
    softmax<D, kQ4, NB, kSteps, kDup, kEdge>(x, scale, vw, t0 + h, s, seen, scores ? scores + h * score_rows : nullptr,
                                       score_rows, row0, lane);
    if constexpr (kQ4)
      values_q4<D, NB, kSteps, kDup, kEdge>(vt + h * kCode, vt + C::kTokens * kCode + h * kParam, x, vw, t0 + h, s,
                                            seen, lane);
    else
      values_bf16<D, NB, kSteps, kDup, kEdge>(smem_u32(vt) + h * (2 * D), x, vw, t0 + h, s, seen, lane);
  }
}

// First element of register e of query fragment j in a lane, and the distance to its second.
template <bool kQ4>
__device__ __forceinline__ int query_dim(int j, int e, int c) {
  // 4-bit: group j / 4, step j % 4: word 2c or 2c + 1 of the group, nibbles i and i + 4
  return kQ4 ? 64 * (j >> 2) + 8 * (2 * c + ((j >> 1) & 1)) + 2 * (j & 1) + e : 16 * j + 2 * c + 8 * e;
}

template <int D, bool kQ4, int kRows>
__global__ void __launch_bounds__((Cfg<D, kQ4, kRows>::kThreads), (Cfg<D, kQ4, kRows>::kBlocks))
    window_mma_kernel(const __grid_constant__ WindowMmaParams mp) {
  using C = Cfg<D, kQ4, kRows>;
  constexpr int NK = D / 16, NG = kQ4 ? D / 64 : 1, NB = C::NB, kCons = C::kCons, kTeams = C::kTeams;
  constexpr bool kDup = C::kDup;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t warp_sum[kCons + C::kProd];
  __shared__ TreeRange range_s;
  // Each consumer warp's place in the block's items, and its item: not worth registers.
  __shared__ alignas(16) uint8_t cur_s[kCons][sizeof(TreeCursor<kWindowTile>)];
  __shared__ TreeItem item_s[kCons];
  __shared__ View view_s[kCons];
  const WindowParams &p = mp.w;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *rec = (float *)(smem + C::kRing);
  float2 *ml = (float2 *)(rec + kTeams * C::kRec);
  float *wgt = (float *)(ml + kTeams * kRows);
  uint64_t *bars = (uint64_t *)(wgt + 8 * kRows);
  volatile int *abort_flag = (volatile int *)(bars + 2 * C::kStages);
  const uint32_t ring = smem_u32(smem), full0 = smem_u32(bars), empty0 = smem_u32(bars + C::kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full0 + 8 * i, C::kProd);
      mbar_init(empty0 + 8 * i, C::kCols);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (!kQ4 && warp == kCons && lane < p.c.G) {
    prefetch_tensormap(&mp.tmK[lane]);
    prefetch_tensormap(&mp.tmV[lane]);
  }
  pdl_wait();
  const TreeRange range = tree_range<C::kThreads, kWindowTile>(p, 1, warp_sum, &range_s);
  if (warp >= kCons) {
    produce<D, kQ4, kRows>(mp, range, ring, full0, empty0, abort_flag, warp - kCons, lane);
    return;
  }
  const int r = lane >> 2, c = lane & 3, g = p.c.g;
  const int team = warp / C::kCols, row0 = warp % C::kCols * (8 * NB);  // this warp's first row
  using Cursor = TreeCursor<kWindowTile>;
  Cursor &cur = *(Cursor *)cur_s[warp];
  const TreeItem &it = item_s[warp];
  const View &vw = view_s[warp];
  {
    const Cursor first(p, range);
    if (lane == 0) cur = first;
    __syncwarp();
  }
  bool any = false, dead = false;
  int gs = 0;
  for (;;) {
    {
      Cursor c1 = cur;
      TreeItem i1;
      const bool more = c1.next(p, i1);
      __syncwarp();
      if (!more) break;
      if (lane == 0) {
        cur = c1;
        item_s[warp] = i1;
        View v;
        v.win = window_of(i1.head);
        v.n = i1.head.n;
        v.i0 = tree_first(p, i1);
        v.rows = tree_rows(p, i1);
        v.i1 = v.i0 + tree_div_g(p, v.rows - 1);
        v.recip_g = p.recip_g;
        view_s[warp] = v;
      }
      __syncwarp();
    }
    any = true;
    const TreeHead &hd = it.head;
    const int i0 = tree_first(p, it), rows = tree_rows(p, it);
    // queries: column n = lane / 4 of each block; scale: of the scores of columns 2c, 2c + 1
    Queries<D, NB> q;
    float qs[NG][NB][2], qe[NG][NB][2], scale[kQ4 ? NB : 1][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      {
        const int row = kDup ? r & 3 : row0 + 8 * nb + r;
        const int nr = tree_div_g(p, row), j0 = row - nr * g;
        const uint16_t *src = (const uint16_t *)(p.q + (size_t)(hd.q0 + i0 + nr) * p.q_stride) +
                              ((size_t)hd.h * g + j0) * D;
        uint32_t f[NK][2];
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint16_t *at = src + query_dim<kQ4>(j, e, c);
            f[j][e] = row >= rows ? 0u : kQ4 ? (uint32_t)at[0] | (uint32_t)at[4] << 16 : *(const uint32_t *)at;
          }
        if constexpr (kQ4) {
          // to fp16: the row's largest element becomes 2^14 to 2^15
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              top = max(top, max((f[j][e] & 0x7fffu) << 16, f[j][e] & 0x7fff0000u));
          top = max(top, __shfl_xor_sync(kAll, top, 1));
          top = max(top, __shfl_xor_sync(kAll, top, 2));
          // (and no further than back, below, is a normal number: -inf times 0 would be NaN. Elements
          // that this leaves too small for fp16 move no score by more than 2^-45, see the header's limits.)
          const int most = min(254, (int)(__float_as_uint(p.scale_log2) >> 23) + 126);
          const int ex = max(1, min(most, 268 - (int)(top >> 23)));
          const float mul = __uint_as_float((uint32_t)ex << 23);
          float sum[NG], even[NG];
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) sum[gq] = even[gq] = 0.f;
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (codes of odd places come 16 times too large)
              const float lo = bf_low(f[j][e]) * mul, hi = bf_high(f[j][e]) * mul;
              f[j][e] = e ? pack_f16(lo * 0.0625f, hi * 0.0625f) : pack_f16(lo, hi);
              sum[j >> 2] += lo + hi;
              if (!e) even[j >> 2] += lo + hi;
            }
          const float back = p.scale_log2 / mul;
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) {
            sum[gq] += __shfl_xor_sync(kAll, sum[gq], 1);
            sum[gq] += __shfl_xor_sync(kAll, sum[gq], 2);
            even[gq] += __shfl_xor_sync(kAll, even[gq], 1);
            even[gq] += __shfl_xor_sync(kAll, even[gq], 2);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // from a lane of column 2c + k
            scale[nb][k] = __shfl_sync(kAll, back, 8 * c + 4 * k);
#pragma unroll
            for (int gq = 0; gq < NG; ++gq) {
              qs[gq][nb][k] = __shfl_sync(kAll, sum[gq], 8 * c + 4 * k);
              qe[gq][nb][k] = 8.f * __shfl_sync(kAll, even[gq], 8 * c + 4 * k);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          q.f[nb][j][0] = f[j][0];
          q.f[nb][j][1] = f[j][1];
        }
      }
    }
    if constexpr (!kQ4) scale[0][0] = scale[0][1] = p.scale_log2;
    State<D, kQ4, NB> s;
    s.vscale = 0x1p60f;
    s.vtop = 0.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int dm = 0; dm < NK; ++dm) s.o[dm][nb][0] = s.o[dm][nb][1] = s.o[dm][nb][2] = s.o[dm][nb][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s.ref[nb][k] = kNoRef;
        s.l[nb][k] = 0.f;
#pragma unroll
        for (int gq = 0; gq < NG; ++gq) s.z[gq][nb][k] = 0.f;
      }
    }
    const int nst = item_stages<C::kTokens>(it);
    // this warp's stages: gs = team (mod kTeams)
    int st = (team - gs) % kTeams;
    for (st += st < 0 ? kTeams : 0; st < nst && !dead; st += kTeams) {
      const int at = gs + st, slot = at % C::kStages;
      bool ok = !*abort_flag;
      if (ok) ok = mbar_wait(full0 + 8 * slot, (at / C::kStages) & 1, p.wait_ns);
      if (!__all_sync(kAll, ok)) {
        if (lane == 0) {
          atomicOr(p.status, KVX_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        dead = true;
        break;
      }
      const int t0 = stage_token<C::kTokens>(it, st);
      float *scores = p.scores ? window_scores(p, hd, it.group, (int64_t)it.t0 * kWindowTile + st * C::kTokens)
                               : nullptr;
      const uint8_t *kt = smem + slot * C::kStage, *vt = kt + C::kTile;
      if (row0 >= rows) {  // few rows: none for this warp
      } else if (window_all_seen(vw.win, hd.n, vw.i0, vw.i1, t0, C::kTokens)) {
        consume<D, kQ4, kRows, false>(kt, vt, vw, t0, q, qs, qe, scale, s, scores, p.score_rows, row0, lane);
      } else {
        consume<D, kQ4, kRows, true>(kt, vt, vw, t0, q, qs, qe, scale, s, scores, p.score_rows, row0, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * slot);
    }
    gs += nst;
    // ---- the consumer warps' states of this item meet
    float *mw = rec + team * C::kRec + row0 * C::kMS;
    const float back = kQ4 ? 0.5f / s.vscale : 1.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          s.l[nb][k] += __shfl_xor_sync(kAll, s.l[nb][k], sh);
          if constexpr (kQ4) {
#pragma unroll
            for (int gq = 0; gq < NG; ++gq) s.z[gq][nb][k] += __shfl_xor_sync(kAll, s.z[gq][nb][k], sh);
          }
        }
      float zsum[NG][2];
      if constexpr (kQ4) {
#pragma unroll
        for (int gq = 0; gq < NG; ++gq)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            zsum[gq][k] = !kDup ? s.z[gq][nb][k] : __shfl_sync(kAll, s.z[0][nb][k], (c & 1) + (gq ? 2 : 0));
      }
#pragma unroll
      for (int dm = 0; dm < NK; ++dm)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s.o[dm][nb][e];
          if constexpr (kDup) v += __shfl_xor_sync(kAll, v, 2);  // both parts of P
          if constexpr (kQ4) v = fmaf(v, back, zsum[dm >> 2][e & 1]);
          const int row = 8 * nb + 2 * c + (e & 1);
          const int d = kQ4 ? 64 * (dm >> 2) + 8 * r + 2 * (dm & 3) + (e >> 1) : 16 * dm + r + 8 * (e >> 1);
          if (!kDup || c < 2) mw[row * C::kMS + d] = v;
        }
      if (r == 0 && (!kDup || c < 2))
#pragma unroll
        for (int k = 0; k < 2; ++k)
          ml[team * kRows + row0 + 8 * nb + 2 * c + k] = make_float2(s.ref[nb][k], s.l[nb][k]);
    }
    consumer_sync(kCons * 32);
    const bool whole = tree_whole(it);
    const int slot0 = whole ? 0 : tree_slot(it);
    if (tid < rows) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kTeams; ++w) M = fmaxf(M, ml[w * kRows + tid].x);
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        const float2 v = ml[w * kRows + tid];
        const float f = v.x == v.x ? tree_weight(v.x, M) : v.x;
        wgt[tid * 8 + w] = f;
        L = fmaf(f, v.y, L);
      }
      wgt[tid * 8 + 7] = L == 0.f ? 0.f : 1.f / L;
      if (!whole)
        p.part_ml[(size_t)slot0 * p.group_rows + tid] = make_float2(M, L);
      else if (p.row_ml)
        *tree_row_ml(p, tree_ml_row(p, hd.b, i0), hd.h, tid) = make_float2(M, L);
    }
    consumer_sync(kCons * 32);
    for (int i = tid; i < rows * (D / 4); i += kCons * 32) {
      const int row = i / (D / 4), d4 = 4 * (i - row * (D / 4));
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        const float f = wgt[row * 8 + w];
        const float4 v = *(const float4 *)(rec + w * C::kRec + row * C::kMS + d4);
        O.x = fmaf(f, v.x, O.x);
        O.y = fmaf(f, v.y, O.y);
        O.z = fmaf(f, v.z, O.z);
        O.w = fmaf(f, v.w, O.w);
      }
      float *dst = p.part_o + ((size_t)slot0 * p.group_rows + row) * D;
      if (whole) {
        const float f = wgt[row * 8 + 7];
        O = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
        dst = tree_out(p, hd.q0 + i0, hd.h, row);
      }
      *(float4 *)(dst + d4) = O;
    }
    consumer_sync(kCons * 32);  // the records may be overwritten
  }
  if (tid == 0) tree_describe(p, range, any ? &it : nullptr);
}

template <int D, bool kQ4, int kRows>
cudaError_t launch_one(const WindowMmaParams &p, int blocks, cudaStream_t st) {
  using C = Cfg<D, kQ4, kRows>;
  static int8_t done[64];
  const auto kernel = window_mma_kernel<D, kQ4, kRows>;
  cudaError_t e = raise_smem_limit(done, (const void *)kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool kQ4>
cudaError_t launch_rows(const WindowMmaParams &p, int blocks, cudaStream_t st) {
  switch (p.w.group_rows) {  // window_mma_rows
    case 4: return launch_one<D, kQ4, 4>(p, blocks, st);
    case 8: return launch_one<D, kQ4, 8>(p, blocks, st);
    case 16: return launch_one<D, kQ4, 16>(p, blocks, st);
    default:
      if constexpr (kQ4) return cudaErrorInvalidValue;  // unreachable
      else return launch_one<D, kQ4, 32>(p, blocks, st);
  }
}

}  // namespace wmma
}  // namespace kvx
