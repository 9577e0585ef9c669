// window_mma.cuh -- attention with a sliding window and sink tokens over a paged
// cache, on warp-level tensor-core MMAs; bf16 and 4-bit caches.
//
// The keys that a head visits come in tiles of 64 (window_split.cuh), its query rows in
// groups of 8 * NB columns (or 4, below). Blocks take equal parts of all (row group, tile)
// units, found on the device from the lengths. In a block one producer warp walks the items and
// loads stages of 32 tokens (K and V) into a ring in shared memory; each consumer warp takes
// every kCons-th stage and holds its own running maximum, sum and output, which meet in
// shared memory at an item's end. Per stage a warp computes S^T = K Q^T (m16n8k16: 16 tokens x
// 8 query rows), the softmax on the accumulators (column maxima by shuffles), turns P into
// the B operand with movmatrix, and O^T = V^T P^T in fresh accumulators that are then added to
// the output in fp32: the tensor cores truncate their sums, and a chain of two 16-token
// steps keeps that below the rounding of P.
// P is split into a bf16 high part and a bf16 residual. With at most four query rows (a decode
// step of up to four heads a KV head) the columns 4 .. 7 repeat the rows 0 .. 3, so that
// one MMA multiplies both parts: high in the first four columns, residual in the others.
//
// bf16 stages: bulk-tensor boxes of up to 32 tokens of one head, [8-token group][64-dim
// half][8 rows][128 B] with 128-byte swizzle. Tensor-core operands by ldmatrix.
//
// 4-bit stages: bulk copies of page blocks (codes, then parameters: window.h). Codes become
// bf16 in registers with a mask, an or and a shift: a code in the top four bits of the
// mantissa of 16.0 is 16 + code. Two facts let the codes go to the MMAs without being scaled:
//   S = sum_g step_g (sum_{d in g} q_d (16 + c_d)) + (lo_g - 16 step_g) sum_{d in g} q_d
//   O_d = sum_t (p_t step_t) (c_td - 7.5) + sum_t p_t (lo_t + 7.5 step_t),
// with the group's step and lo of the token, fp32 outside the MMAs. (7.5 centres the codes: with
// 0 .. 15 the two sums would nearly cancel, values having means near 0.) V pairs two tokens in
// a register: one byte permute of their words brings equal elements side by side. The MMAs'
// inner dimension has no order of its own, so a lane takes the elements that its
// loads bring: eight neighbours of both groups of a row for V, sixteen for K.
#pragma once

#include <math.h>

#include "window_split.cuh"

namespace kvx {

namespace wmma {

constexpr int kStageTokens = kWindowBox;
constexpr uint32_t kAll = 0xffffffffu;

// NB: column blocks of 8 query rows. kDup: at most 4 rows, repeated (NB = 1).
template <int D, bool kQ4, int NB, bool kDup>
struct Cfg {
  static constexpr int kRows = kDup ? 4 : 8 * NB;  // query rows of a row group
  static constexpr int kTokenBytes = kQ4 ? q4_row_bytes(D) : 2 * D;
  static constexpr int kTile = kStageTokens * kTokenBytes;  // K (or V) bytes of a stage
  static constexpr int kStage = 2 * kTile;
  static constexpr int kCons = kQ4 ? (NB == 1 ? 7 : NB == 2 ? 5 : 3) : (NB == 1 ? 3 : 2);
  static constexpr int kStages = 2 * kCons;
  static constexpr int kThreads = 32 * (kCons + 1);
  static constexpr int kMS = D + 4;  // floats of a row of a warp's record
  static constexpr int kRec = kRows * kMS;
  static constexpr int kRing = kStages * kStage;
  static constexpr bool kQShared = NB > 2;  // query fragments in shared memory
  static constexpr int kQBytes = kQShared ? NB * (D / 16) * 32 * 8 : 0;
  // ring | records | (max, sum) [kCons][kRows] | weights [kRows][8] | queries | barriers, flag
  static constexpr int kSmem = 1024 + kRing + 4 * kCons * kRec + 8 * kCons * kRows + 32 * kRows +
                               kQBytes + 16 * kStages + 16;
  static_assert(kSmem + 2048 <= 227 * 1024 / kWindowBlocksPerSm, "resident blocks per SM");
  static_assert(kCons <= 7, "a row's eighth weight is 1 / sum");
};

// 16 + code of nibble i (0 .. 3) of both 16-bit halves, as two bf16.
template <int i>
__device__ __forceinline__ uint32_t code16(uint32_t w) {
  const uint32_t s = i == 0 ? w << 3 : w >> (i == 0 ? 0 : 4 * i - 3);
  return (s & 0x00780078u) | 0x41804180u;
}
__device__ __forceinline__ uint32_t code16_i(uint32_t w, int i) {  // i: a constant after unrolling
  return i == 0 ? code16<0>(w) : i == 1 ? code16<1>(w) : i == 2 ? code16<2>(w) : code16<3>(w);
}
// code - 7.5 (exact).
__device__ __forceinline__ uint32_t code_centred(uint32_t w, int i) {
  const uint32_t x = code16_i(w, i);
  const __nv_bfloat162 c = __hsub2(*(const __nv_bfloat162 *)&x, __floats2bfloat162_rn(23.5f, 23.5f));
  return *(const uint32_t *)&c;
}
__device__ __forceinline__ float bf_low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_high(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Bulk copy of `bytes` (a multiple of 16) to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                          uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}

// The stages of an item: st = 0 .. stages-1, two a tile; the last tile's second half is left out
// where the head ends before it.
__device__ __forceinline__ int item_stages(const TreeItem &it) {
  const int end = it.head.n + it.head.T;
  const int last = window_tile(it.head, it.t1 - 1) * kWindowTile;
  return 2 * (it.t1 - it.t0) - (end - last <= kStageTokens ? 1 : 0);
}
__device__ __forceinline__ int stage_token(const TreeItem &it, int st) {
  return window_tile(it.head, it.t0 + (st >> 1)) * kWindowTile + (st & 1) * kStageTokens;
}

// ---- producer ----------------------------------------------------------------
template <int D, bool kQ4, int NB, bool kDup>
__device__ __forceinline__ void produce(const WindowMmaParams &mp, const TreeRange &range,
                                        uint32_t ring, uint32_t full0, uint32_t empty0,
                                        volatile int *abort_flag, int lane) {
  using C = Cfg<D, kQ4, NB, kDup>;
  const WindowParams &p = mp.w;
  const int P = p.c.P, box = min(P, kStageTokens), lb = 31 - __clz(box);
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
    const int end = hd.n + hd.T, nst = item_stages(it);
    // lane i looks up the page of the stage's box i, a stage ahead
    auto look = [&](int st) {
      const int t = st < nst ? stage_token(it, st) + (lane << lb) : end;
      return lane < kStageTokens >> lb && t < end ? table[t >> p.c.lgP] : -2;
    };
    int next = look(0);
    for (int st = 0; st < nst; ++st, ++gs) {
      const int slot = gs % C::kStages, t0 = stage_token(it, st), page = next;
      next = look(st + 1);
      if (gs >= C::kStages) {
        bool ok = true;
        if (lane == 0)
          ok = !*abort_flag && mbar_wait(empty0 + 8 * slot, ((gs / C::kStages) - 1) & 1, p.wait_ns);
        if (!__shfl_sync(kAll, ok ? 1 : 0, 0)) {
          if (lane == 0) {
            atomicOr(p.status, KVX_DEV_TIMEOUT);
            *abort_flag = 1;
          }
          dead = true;
          break;
        }
      }
      const uint32_t full = full0 + 8 * slot, dst = ring + slot * C::kStage + (uint32_t)lane * box_bytes;
      const bool mine = page != -2, bad = mine && (page < 0 || page >= grp.pages);
      if (bad) atomicOr(p.status, KVX_DEV_BAD_PAGE);
      uint32_t live = __ballot_sync(kAll, mine);
      if (kQ4 && __any_sync(kAll, bad)) {
        // no box to point past the pool's end: zeros from here
        if (bad)
          for (uint32_t i = 0; i < box_bytes; i += 16) {
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + C::kTile + i), "r"(0)
                         : "memory");
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        live = __ballot_sync(kAll, mine && !bad);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, 2u * box_bytes * (uint32_t)__popc(live));
      __syncwarp();
      // Failure-detection test only: the chosen block arms its first stage but loads nothing.
      if (gs == 0 && (int)blockIdx.x == p.stall_block) continue;
      if constexpr (kQ4) {
        if (mine && !bad) {
          const int off = (t0 + (lane << lb)) & (P - 1);  // 0, or a part of a page of 64 or 128
          const int64_t at = (((int64_t)page * grp.size + rank) * P) * q4_row_bytes(D);
          if (P <= kStageTokens) {
            bulk_load(dst, grp.k + at, box_bytes, full, pol);
            bulk_load(dst + C::kTile, grp.v + at, box_bytes, full, pol);
          } else {
            constexpr uint32_t cb = kStageTokens * q4_code_bytes(D), pb = kStageTokens * q4_param_bytes(D);
            const int64_t ca = at + off * q4_code_bytes(D);
            const int64_t pa = at + P * q4_code_bytes(D) + off * q4_param_bytes(D);
            bulk_load(dst, grp.k + ca, cb, full, pol);
            bulk_load(dst + cb, grp.k + pa, pb, full, pol);
            bulk_load(dst + C::kTile, grp.v + ca, cb, full, pol);
            bulk_load(dst + C::kTile + cb, grp.v + pa, pb, full, pol);
          }
        }
      } else if (mine) {
        const int sub = ((t0 + (lane << lb)) & (P - 1)) >> 3;  // 8-row group in the page
        const int pg = bad ? (int)grp.pages : page;            // past the last page: zeros
        const int c3 = p.c.token_major ? pg * (P >> 3) + sub : sub;
        const int c4 = p.c.token_major ? rank : pg * grp.size + rank;
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
  float m[NB][2], l[NB][2];
  float z[NG][NB][2];  // 4-bit: sum of p (lo + 7.5 step), this lane's tokens
};

// Query fragments: registers, or shared memory where there are many.
template <int D, int NB, bool kShared>
struct Queries {
  uint32_t f[kShared ? 1 : NB][kShared ? 1 : D / 16][2];
  uint32_t at;  // shared: this lane's fragments
  __device__ __forceinline__ uint2 get(int nb, int j) const {
    if constexpr (kShared) return lds64(at + (uint32_t)(nb * (D / 16) + j) * 256u);
    return make_uint2(f[nb][j][0], f[nb][j][1]);
  }
};

// The two elements of register `e` of fragment j of a query row: first element, distance.
template <int D, bool kQ4>
__device__ __forceinline__ int query_dim(int j, int e, int c) {
  if constexpr (kQ4)  // group j / 4, step j % 4: word 2c or 2c + 1 of the group, nibbles i and i + 4
    return 64 * (j >> 2) + 8 * (2 * c + ((j >> 1) & 1)) + 2 * (j & 1) + e;
  return 16 * j + 2 * c + 8 * e;
}
template <bool kQ4>
__device__ __forceinline__ uint32_t query_pair(const __nv_bfloat16 *q, int d) {
  if constexpr (kQ4) {
    const uint16_t *u = (const uint16_t *)q;
    return (uint32_t)u[d] | (uint32_t)u[d + 4] << 16;
  }
  return *(const uint32_t *)(q + d);
}

// What a stage at the edge of some row's view needs: which rows see what.
struct Edge {
  Window win;
  int n, i0, i1;  // cached tokens, first and last new row of the item
  int t0;         // first token of the stage
};

// kEdge: some row does not see all of the stage.
template <int D, bool kQ4, int NB, bool kDup, bool kEdge>
__device__ __forceinline__ void consume(uint32_t kb, uint32_t vb, const int (&pos)[NB][2],
                                        const Edge &eg, int lb,
                                        const Queries<D, NB, Cfg<D, kQ4, NB, kDup>::kQShared> &q,
                                        const float (&qs)[kQ4 ? D / 64 : 1][NB][2],
                                        State<D, kQ4, NB> &s, float sl2, float *scores,
                                        int score_rows, int lane) {
  constexpr int NK = D / 16, NG = kQ4 ? D / 64 : 1;
  const int r = lane >> 2, c = lane & 3;
  // Byte offset of 8-token group t8 of a tile. 4-bit: of its codes; its parameters.
  auto group_at = [&](int t8) -> uint32_t {
    if constexpr (!kQ4) return (uint32_t)t8 * (D * 16);
    const int box = 1 << lb, t = 8 * t8;
    return (uint32_t)((t >> lb) * box * q4_row_bytes(D) + (t & (box - 1)) * q4_code_bytes(D));
  };
  auto params_at = [&](int t8) -> uint32_t {
    const int box = 1 << lb, t = 8 * t8;
    return (uint32_t)((t >> lb) * box * q4_row_bytes(D) + box * q4_code_bytes(D) +
                      (t & (box - 1)) * q4_param_bytes(D));
  };
  const int mi = lane >> 3, lr = lane & 7;
  float x[2][NB][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    if constexpr (!kQ4) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) x[mt][nb][0] = x[mt][nb][1] = x[mt][nb][2] = x[mt][nb][3] = 0.f;
      const uint32_t row = kb + group_at(2 * mt + (mi & 1)) + (uint32_t)lr * 128u;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(row + (uint32_t)(j >> 2) * 1024u + ((uint32_t)(((2 * j) & 7) + (mi >> 1)) ^ (uint32_t)lr) * 16u,
                a0, a1, a2, a3);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint2 b = q.get(nb, j);
          mma_bf16(x[mt][nb], a0, a1, a2, a3, b.x, b.y);
        }
      }
    } else {
      // rows r and r + 8: their words 2c and 2c + 1 of each group
      uint32_t w[2][NG][2], pr[2][NG];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t ca = kb + group_at(2 * mt + u) + (uint32_t)r * q4_code_bytes(D);
        const uint32_t pa = kb + params_at(2 * mt + u) + (uint32_t)r * q4_param_bytes(D);
        if constexpr (D == 128) {
          const uint4 v = lds128(ca + 16u * c);
          w[u][0][0] = v.x, w[u][NG - 1][0] = v.y, w[u][0][1] = v.z, w[u][NG - 1][1] = v.w;
          const uint2 pp = lds64(pa);
          pr[u][0] = pp.x, pr[u][NG - 1] = pp.y;
        } else {
          const uint2 v = lds64(ca + 8u * c);
          w[u][0][0] = v.x, w[u][0][1] = v.y;
          pr[u][0] = lds32(pa);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) x[mt][nb][0] = x[mt][nb][1] = x[mt][nb][2] = x[mt][nb][3] = 0.f;
#pragma unroll
      for (int gq = 0; gq < NG; ++gq) {
        float acc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = w[0][gq][j >> 1], w1 = w[1][gq][j >> 1];
          const int i = 2 * (j & 1);
          const uint32_t a0 = code16_i(w0, i), a1 = code16_i(w1, i), a2 = code16_i(w0, i + 1),
                         a3 = code16_i(w1, i + 1);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 b = q.get(nb, 4 * gq + j);
            mma_bf16(acc[nb], a0, a1, a2, a3, b.x, b.y);
          }
        }
        const float st0 = bf_low(pr[0][gq]), st1 = bf_low(pr[1][gq]);
        const float b0 = fmaf(-16.f, st0, bf_high(pr[0][gq])), b1 = fmaf(-16.f, st1, bf_high(pr[1][gq]));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          x[mt][nb][0] = fmaf(st0, acc[nb][0], fmaf(b0, qs[gq][nb][0], x[mt][nb][0]));
          x[mt][nb][1] = fmaf(st0, acc[nb][1], fmaf(b0, qs[gq][nb][1], x[mt][nb][1]));
          x[mt][nb][2] = fmaf(st1, acc[nb][2], fmaf(b1, qs[gq][nb][0], x[mt][nb][2]));
          x[mt][nb][3] = fmaf(st1, acc[nb][3], fmaf(b1, qs[gq][nb][1], x[mt][nb][3]));
        }
      }
    }
  }
  // x[mt][nb][e]: token mt * 16 + r (+ 8 for e >= 2), query row 8 nb + 2c + (e & 1)
  uint32_t seen = kAll;  // kEdge: bit (mt * NB + nb) * 4 + e
  if constexpr (kEdge) seen = 0;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = x[mt][nb][e] * sl2;
        if constexpr (kEdge) {
          const bool see = window_sees(eg.win, pos[nb][e & 1], eg.t0 + mt * 16 + r + ((e >> 1) << 3));
          seen |= (see ? 1u : 0u) << ((mt * NB + nb) * 4 + e);
          v = see ? v : -INFINITY;
        }
        x[mt][nb][e] = v;
      }
  if (scores) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (8 * nb + 2 * c < score_rows) {
          float *at = scores + (size_t)(mt * 16 + r) * score_rows + 8 * nb + 2 * c;
          *(float2 *)at = make_float2(x[mt][nb][0], x[mt][nb][1]);
          *(float2 *)(at + 8 * score_rows) = make_float2(x[mt][nb][2], x[mt][nb][3]);
        }
  }
  float al[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float mx = fmaxf(fmaxf(x[0][nb][k], x[0][nb][k + 2]), fmaxf(x[1][nb][k], x[1][nb][k + 2]));
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, sh));
      const float mn = fmaxf(s.m[nb][k], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing
      al[nb][k] = ex2(s.m[nb][k] - ref);
      s.m[nb][k] = mn;
      float sum = 0.f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = k; e < 4; e += 2) {
          const float pv = ex2(x[mt][nb][e] - ref);
          x[mt][nb][e] = pv;
          sum += pv;
        }
      s.l[nb][k] = fmaf(s.l[nb][k], al[nb][k], sum);
    }
  // P^T as the B operand (inner dimension tokens): high part and residual, or, repeated rows, the
  // part of this lane's columns.
  auto split = [&](float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    const float2 f = unpack_bf16(hi);
    lo = pack_bf16(a - f.x, b - f.y);
    if constexpr (kDup) hi = c < 2 ? hi : lo;
  };
  // Tokens of this lane in V^T fragments: 2c, 2c + 1 and 8 on, masked where no row sees them.
  uint32_t mask[2][2];
  if constexpr (kEdge) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = eg.t0 + 8 * k + 2 * c;
      auto any = [&](int u) {
        return u <= eg.n + eg.i1 && (u < eg.win.sinks || (u > eg.n + eg.i0 - eg.win.width && eg.win.width > 0));
      };
      mask[k >> 1][k & 1] = (any(t) ? 0xffffu : 0u) | (any(t + 1) ? 0xffff0000u : 0u);
    }
  }
  if constexpr (!kQ4) {
    uint32_t bh[2][NB][2], bl[2][NB][2], bv[2][NB][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t hi, lo;
          split(x[mt][nb][2 * u], x[mt][nb][2 * u + 1], hi, lo);
          bh[mt][nb][u] = movmatrix_t(hi);
          if constexpr (!kDup) bl[mt][nb][u] = movmatrix_t(lo);
          if constexpr (kEdge) {  // 1 where the row sees the token
            const uint32_t b = seen >> ((mt * NB + nb) * 4 + 2 * u);
            bv[mt][nb][u] = movmatrix_t((b & 1u ? 0x3f80u : 0u) | (b & 2u ? 0x3f800000u : 0u));
          }
        }
#pragma unroll
    for (int dm = 0; dm < NK; ++dm) {
      float acc[NB][4];
      uint32_t a[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t row = vb + group_at(2 * mt + (mi >> 1)) + (uint32_t)lr * 128u;
        ldsm_x4_t(row + (uint32_t)(dm >> 2) * 1024u +
                      ((uint32_t)(((2 * dm) & 7) + (mi & 1)) ^ (uint32_t)lr) * 16u,
                  a[mt][0], a[mt][1], a[mt][2], a[mt][3]);
        if constexpr (kEdge) {
          a[mt][0] &= mask[mt][0];
          a[mt][1] &= mask[mt][0];
          a[mt][2] &= mask[mt][1];
          a[mt][3] &= mask[mt][1];
        }
      }
      // Non-finite elements of tokens that only some rows see: left out of the products, and
      // counted for the rows that see them, whose output becomes NaN.
      float cnt[NB][4];
      bool odd = false;
      if constexpr (kEdge) {
        if (eg.i1 > eg.i0) {
          uint32_t nf[2][4], all = 0;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
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
              cnt[nb][0] = cnt[nb][1] = cnt[nb][2] = cnt[nb][3] = 0.f;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
                mma_bf16(cnt[nb], nf[mt][0] & 0x3f803f80u, nf[mt][1] & 0x3f803f80u,
                         nf[mt][2] & 0x3f803f80u, nf[mt][3] & 0x3f803f80u, bv[mt][nb][0], bv[mt][nb][1]);
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int k = 0; k < 4; ++k) a[mt][k] &= ~nf[mt][k];
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if constexpr (!kDup)
            mma_bf16(acc[nb], a[mt][0], a[mt][1], a[mt][2], a[mt][3], bl[mt][nb][0], bl[mt][nb][1]);
          mma_bf16(acc[nb], a[mt][0], a[mt][1], a[mt][2], a[mt][3], bh[mt][nb][0], bh[mt][nb][1]);
        }
        if constexpr (kEdge) {
          if (odd) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cnt[nb][e] != 0.f) acc[nb][e] = __uint_as_float(0x7fc00000u);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s.o[dm][nb][e] = fmaf(s.o[dm][nb][e], al[nb][e & 1], acc[nb][e]);
      }
    }
  } else {
    // V words of tokens 2c, 2c + 1 (lanes with odd c read the odd one first, so that a load's
    // four tokens lie in all banks), paired: x_lo elements 0 .. 3, x_hi 4 .. 7 of word r
    uint32_t xw[2][2][NG][2];  // [mt][8-token half][group][lo, hi]
    const uint32_t sel_lo = c & 1 ? 0x1054u : 0x5410u, sel_hi = c & 1 ? 0x3276u : 0x7632u;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t ca = vb + group_at(2 * mt + u) + (uint32_t)r * (D / 16);
        const uint32_t f = ca + (uint32_t)(2 * c + (c & 1)) * q4_code_bytes(D);
        const uint32_t g = ca + (uint32_t)(2 * c + 1 - (c & 1)) * q4_code_bytes(D);
        uint32_t a[NG], b[NG];
        if constexpr (D == 128) {
          const uint2 va = lds64(f), vb2 = lds64(g);
          a[0] = va.x, a[NG - 1] = va.y, b[0] = vb2.x, b[NG - 1] = vb2.y;
        } else {
          a[0] = lds32(f), b[0] = lds32(g);
        }
#pragma unroll
        for (int gq = 0; gq < NG; ++gq) {
          xw[mt][u][gq][0] = __byte_perm(a[gq], b[gq], sel_lo);
          xw[mt][u][gq][1] = __byte_perm(a[gq], b[gq], sel_hi);
        }
      }
#pragma unroll
    for (int gq = 0; gq < NG; ++gq) {
      uint32_t bh[2][NB][2], bl[2][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        s.z[gq][nb][0] *= al[nb][0];
        s.z[gq][nb][1] *= al[nb][1];
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t pr =
              lds32(vb + params_at(2 * mt + u) + (uint32_t)r * q4_param_bytes(D) + 4u * gq);
          const float st = bf_low(pr), mid = fmaf(7.5f, st, bf_high(pr));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float p0 = x[mt][nb][2 * u], p1 = x[mt][nb][2 * u + 1];
            float w0 = p0 * st, w1 = p1 * st, z0 = p0 * mid, z1 = p1 * mid;
            if constexpr (kEdge) {  // what a row does not see may be anything
              const uint32_t b = seen >> ((mt * NB + nb) * 4 + 2 * u);
              if (!(b & 1u)) w0 = z0 = 0.f;
              if (!(b & 2u)) w1 = z1 = 0.f;
            }
            s.z[gq][nb][0] += z0;
            s.z[gq][nb][1] += z1;
            uint32_t hi, lo;
            split(w0, w1, hi, lo);
            bh[mt][nb][u] = movmatrix_t(hi);
            if constexpr (!kDup) bl[mt][nb][u] = movmatrix_t(lo);
          }
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // dims 8r + 2e and 8r + 2e + 1 of the group
        uint32_t a[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            a[mt][k] = code_centred(xw[mt][k >> 1][gq][e >> 1], 2 * (e & 1) + (k & 1));
        const int dm = 4 * gq + e;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            if constexpr (!kDup) mma_bf16(acc, a[mt][0], a[mt][1], a[mt][2], a[mt][3], bl[mt][nb][0], bl[mt][nb][1]);
            mma_bf16(acc, a[mt][0], a[mt][1], a[mt][2], a[mt][3], bh[mt][nb][0], bh[mt][nb][1]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) s.o[dm][nb][k] = fmaf(s.o[dm][nb][k], al[nb][k & 1], acc[k]);
        }
      }
    }
  }
}

template <int D, bool kQ4, int NB, bool kDup>
__global__ void __launch_bounds__((Cfg<D, kQ4, NB, kDup>::kThreads), kWindowBlocksPerSm)
    window_mma_kernel(const __grid_constant__ WindowMmaParams mp) {
  using C = Cfg<D, kQ4, NB, kDup>;
  constexpr int NK = D / 16, NG = kQ4 ? D / 64 : 1, kCons = C::kCons;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t warp_sum[kCons + 1];
  __shared__ TreeRange range_s;
  const WindowParams &p = mp.w;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *rec = (float *)(smem + C::kRing);
  float2 *ml = (float2 *)(rec + kCons * C::kRec);
  float *wgt = (float *)(ml + kCons * C::kRows);
  uint8_t *qsm = (uint8_t *)(wgt + 8 * C::kRows);
  uint64_t *bars = (uint64_t *)(qsm + C::kQBytes);
  volatile int *abort_flag = (volatile int *)(bars + 2 * C::kStages);
  const uint32_t ring = smem_u32(smem), full0 = smem_u32(bars), empty0 = smem_u32(bars + C::kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
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
  if (warp == kCons) {
    produce<D, kQ4, NB, kDup>(mp, range, ring, full0, empty0, abort_flag, lane);
    return;
  }
  const int r = lane >> 2, c = lane & 3, g = p.c.g;
  const int lb = 31 - __clz(min(p.c.P, kStageTokens));
  TreeCursor<kWindowTile> cur(p, range);
  TreeItem it;
  bool any = false, dead = false;
  int gs = 0;
  while (cur.next(p, it)) {
    any = true;
    const TreeHead &hd = it.head;
    const int i0 = tree_first(p, it), rows = tree_rows(p, it);
    Edge eg;
    eg.win = window_of(p, hd.h);
    eg.n = hd.n;
    eg.i0 = i0;
    eg.i1 = i0 + tree_div_g(p, rows - 1);
    // queries: column n = lane / 4 of each block
    Queries<D, NB, C::kQShared> q;
    float qs[NG][NB][2];
    int pos[NB][2];
    if constexpr (C::kQShared) {
      consumer_sync(kCons * 32);  // the item before has read its queries
      q.at = smem_u32(qsm) + (uint32_t)lane * 8u;
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = kDup ? r & 3 : 8 * nb + r;
      const int nr = tree_div_g(p, row), j0 = row - nr * g;
      const __nv_bfloat16 *src = (const __nv_bfloat16 *)(p.q + (size_t)(hd.q0 + i0 + nr) * p.q_stride) +
                                 ((size_t)hd.h * g + j0) * D;
      float sum[NG];
#pragma unroll
      for (int gq = 0; gq < NG; ++gq) sum[gq] = 0.f;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        uint32_t f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = row < rows ? query_pair<kQ4>(src, query_dim<D, kQ4>(j, e, c)) : 0u;
          if constexpr (kQ4) sum[j >> 2] += bf_low(f[e]) + bf_high(f[e]);
        }
        if constexpr (C::kQShared) {
          // (each warp writes the blocks nb = warp, warp + kCons, ...)
          if (nb % kCons == warp) *(uint2 *)(qsm + ((nb * NK + j) * 32 + lane) * 8) = make_uint2(f[0], f[1]);
        } else {
          q.f[nb][j][0] = f[0];
          q.f[nb][j][1] = f[1];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 2 * c + k, own = kDup ? col & 3 : 8 * nb + col;
        pos[nb][k] = own < rows ? hd.n + i0 + tree_div_g(p, own) : -1;
      }
      if constexpr (kQ4) {
#pragma unroll
        for (int gq = 0; gq < NG; ++gq) {
          sum[gq] += __shfl_xor_sync(kAll, sum[gq], 1);
          sum[gq] += __shfl_xor_sync(kAll, sum[gq], 2);
          qs[gq][nb][0] = __shfl_sync(kAll, sum[gq], 8 * c);      // of column 2c
          qs[gq][nb][1] = __shfl_sync(kAll, sum[gq], 8 * c + 4);  // of column 2c + 1
        }
      }
    }
    if constexpr (C::kQShared) consumer_sync(kCons * 32);
    State<D, kQ4, NB> s;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int dm = 0; dm < NK; ++dm) s.o[dm][nb][0] = s.o[dm][nb][1] = s.o[dm][nb][2] = s.o[dm][nb][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s.m[nb][k] = -INFINITY;
        s.l[nb][k] = 0.f;
#pragma unroll
        for (int gq = 0; gq < NG; ++gq) s.z[gq][nb][k] = 0.f;
      }
    }
    const int nst = item_stages(it);
    for (int st = 0; st < nst; ++st, ++gs) {
      if (gs % kCons != warp || dead) continue;
      const int slot = gs % C::kStages;
      bool ok = !*abort_flag;
      if (ok) ok = mbar_wait(full0 + 8 * slot, (gs / C::kStages) & 1, p.wait_ns);
      if (!__all_sync(kAll, ok)) {
        if (lane == 0) {
          atomicOr(p.status, KVX_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        dead = true;
        continue;
      }
      eg.t0 = stage_token(it, st);
      float *scores = p.scores ? window_scores(p, hd, it.group, (int64_t)it.t0 * kWindowTile + st * kStageTokens)
                               : nullptr;
      const uint32_t kb = ring + slot * C::kStage;
      if (window_all_seen(eg.win, hd.n, eg.i0, eg.i1, eg.t0, kStageTokens))
        consume<D, kQ4, NB, kDup, false>(kb, kb + C::kTile, pos, eg, lb, q, qs, s, p.scale_log2, scores,
                                         p.score_rows, lane);
      else
        consume<D, kQ4, NB, kDup, true>(kb, kb + C::kTile, pos, eg, lb, q, qs, s, p.scale_log2, scores,
                                        p.score_rows, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * slot);
    }
    // ---- the consumer warps' states of this item meet
    float *mw = rec + warp * C::kRec;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          s.l[nb][k] += __shfl_xor_sync(kAll, s.l[nb][k], sh);
          if constexpr (kQ4)
#pragma unroll
            for (int gq = 0; gq < NG; ++gq) s.z[gq][nb][k] += __shfl_xor_sync(kAll, s.z[gq][nb][k], sh);
        }
#pragma unroll
      for (int dm = 0; dm < NK; ++dm)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s.o[dm][nb][e];
          if constexpr (kDup) v += __shfl_xor_sync(kAll, v, 2);  // both parts of P
          if constexpr (kQ4) v += s.z[dm >> 2][nb][e & 1];
          const int row = 8 * nb + 2 * c + (e & 1);
          const int d = kQ4 ? 64 * (dm >> 2) + 8 * r + 2 * (dm & 3) + (e >> 1) : 16 * dm + r + 8 * (e >> 1);
          if (!kDup || c < 2) mw[row * C::kMS + d] = v;
        }
      if (r == 0 && (!kDup || c < 2))
#pragma unroll
        for (int k = 0; k < 2; ++k)
          ml[warp * C::kRows + 8 * nb + 2 * c + k] = make_float2(s.m[nb][k], s.l[nb][k]);
    }
    consumer_sync(kCons * 32);
    const bool whole = tree_whole(it);
    const int slot0 = whole ? 0 : tree_slot(it);
    if (tid < rows) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kCons; ++w) M = fmaxf(M, ml[w * C::kRows + tid].x);
#pragma unroll
      for (int w = 0; w < kCons; ++w) {
        const float2 v = ml[w * C::kRows + tid];
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
      for (int w = 0; w < kCons; ++w) {
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

template <int D, bool kQ4, int NB, bool kDup>
cudaError_t launch_one(const WindowMmaParams &p, int blocks, cudaStream_t st) {
  using C = Cfg<D, kQ4, NB, kDup>;
  static int8_t done[64];
  const auto kernel = window_mma_kernel<D, kQ4, NB, kDup>;
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
    case 4: return launch_one<D, kQ4, 1, true>(p, blocks, st);
    case 8: return launch_one<D, kQ4, 1, false>(p, blocks, st);
    case 16: return launch_one<D, kQ4, 2, false>(p, blocks, st);
    default: return launch_one<D, kQ4, 4, false>(p, blocks, st);
  }
}

}  // namespace wmma
}  // namespace kvx
