// tables.cu -- page tables and slot maps from request lengths, on the GPU.
//
// Per head group g and sequence b, need = ceil(longest head / P) pages against
// the `have` held: rel = max(0, have - need) pages go back to the group's free
// list, alloc = max(0, need - have) come from it. With exclusive sums over b,
// released page r lands at list position F + r and allocation k takes position
// F + R - 1 - k (F free pages before the call, R released in all). So every
// page's place follows from the sums alone: no atomics, no order of arrival.
//
// One launch. Every block computes the sums of one group by itself (a few
// loads per thread; lengths are tiny and come from L2) and then does an equal
// share of the group's moved pages and slots. A popped position at or past F
// is a page released by this same call, perhaps by another block: it is found
// in its owner's table through the sums instead of the list, so no block waits
// for another. Table entries below `have` are never written, list entries below F
// neither, which is what makes a repeated call give the same result.
// Dependents start only when the tables are written (no early trigger, and a fence behind
// the writes): a decode call with early loads reads page ids before its dependency wait.
// Measured on one GB300: a verify step (16 sequences, 3 groups) 8.0 us, all latency: two
// passes of loads, the sums and their scan (6.7 when dependents were let go at once); 256
// prompts (1.17 M rows, 9.4 M slots of 8 bytes) 21.8 us, of which a plain fill with the slots'
// 75 MB would take 10 and the sums, which every block makes, 5.
#include "ptx.cuh"
#include "tree.h"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Exclusive sums of three arrays a[0..n), stride n + 1 apart, in place; a[n] becomes
// the total. Shared memory, all threads take part. Sums that pass int32 are caught by
// the caller's 64-bit totals.
__device__ void exclusive_scans(int *a, int n, int (*warp_sum)[kWarps]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int s[3], x[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = 0;
    for (int i = lo; i < hi; ++i) s[k] += a[k * (n + 1) + i];
    x[k] = s[k];
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, x[k], d);
      if (lane >= d) x[k] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) warp_sum[k][warp] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int run = x[k] - s[k], all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) run += warp_sum[k][w];
      all += warp_sum[k][w];
    }
    for (int i = lo; i < hi; ++i) {
      const int v = a[k * (n + 1) + i];
      a[k * (n + 1) + i] = run;
      run += v;
    }
    if (tid == 0) a[k * (n + 1) + n] = all;
  }
  __syncthreads();
}

// The entry b of exclusive sums s[0..n] with s[b] <= k < s[b + 1].
__device__ __forceinline__ int owner(const int *s, int n, int k) {
  int lo = 0, hi = n;  // s[lo] <= k < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ int sm[];
  // sums of alloc and release by group, and of the new rows: the low and the high 16
  // bits of the terms apart (a 64-bit shared atomic is a loop; with 256 threads on one
  // address it took 60 us)
  __shared__ unsigned total[2 * KVX_MAX_GROUPS + 1][2];
  __shared__ int warp_sum[3][kWarps];
  __shared__ int free_in[KVX_MAX_GROUPS];
  __shared__ int8_t heads[KVX_MAX_KV_HEADS];  // heads by group
  __shared__ int head_off[KVX_MAX_GROUPS + 1];
  const CacheDev &c = p.c;
  const int B = c.B, G = c.G, Hkv = c.Hkv, P = c.P, lgP = c.lgP, tid = threadIdx.x;
  const int own = blockIdx.y;  // this block's group
  int *a_start = sm, *r_start = sm + (B + 1), *q_start = sm + 2 * (B + 1);
  if (tid <= 2 * KVX_MAX_GROUPS) total[tid][0] = total[tid][1] = 0;
  auto add = [&](int k, int v) {
    if (v <= 0) return;
    atomicAdd(&total[k][0], (unsigned)v & 0xffffu);
    if (v >> 16) atomicAdd(&total[k][1], (unsigned)v >> 16);
  };
  auto sum_of = [&](int k) { return (int64_t)total[k][0] + ((int64_t)total[k][1] << 16); };
  if (tid == 0) {
    int n = 0;
    for (int g = 0; g < G; ++g) {
      head_off[g] = n;
      for (int h = 0; h < Hkv; ++h)
        if (c.head_grp[h] == g) heads[n++] = (int8_t)h;
    }
    head_off[G] = n;
  }
  __syncthreads();
  pdl_wait();
  if (tid < G) free_in[tid] = p.free_in[tid];

  // ---- lengths of every (group, sequence); sums of this block's group
  int bad = 0;
  for (int i = tid; i < G * B; i += kThreads) {
    const int g = i / B, b = i - g * B;
    const int t = p.new_len[b];
    const int have = p.pages_in[i];
    int64_t n = 0;
    for (int k = head_off[g]; k < head_off[g + 1]; ++k) {
      const int v = p.kv_len[(size_t)b * Hkv + heads[k]];
      bad |= v < 0;
      n = max(n, (int64_t)v);
    }
    n += t;
    bad |= t < 0 || have < 0 || have > c.grp[g].stride || n > ((int64_t)c.grp[g].stride << lgP);
    const int need = (int)((n + P - 1) >> lgP);
    const int alloc = max(0, need - have), rel = max(0, have - need);
    add(2 * g, alloc);
    add(2 * g + 1, rel);
    if (g == own) {
      a_start[b] = alloc;
      r_start[b] = rel;
      q_start[b] = t;
      add(2 * KVX_MAX_GROUPS, t);
    }
  }
  bad = __syncthreads_or(bad);
  int short_list = 0;
  if (!bad) {
    bad = sum_of(2 * KVX_MAX_GROUPS) > p.max_rows;
    for (int g = 0; g < G; ++g) {
      const int64_t f = free_in[g];
      const int64_t a = sum_of(2 * g), r = sum_of(2 * g + 1);
      bad |= f < 0 || f + r > c.grp[g].pages;
      short_list |= a > f + r;
    }
  }
  const bool first = blockIdx.x == 0;
  if (bad || short_list) {  // the same verdict in every block: nothing changes
    if (first) {
      for (int b = tid; b < B; b += kThreads)
        p.pages_out[(size_t)own * B + b] = p.pages_in[(size_t)own * B + b];
      if (tid == 0) p.free_out[own] = free_in[own];
      if (own == 0) {
        for (int b = tid; b <= B; b += kThreads) p.q_start[b] = 0;
        if (tid == 0) atomicOr(p.status, bad ? KVX_DEV_BAD_LENGTH : KVX_DEV_NO_PAGES);
      }
    }
    return;
  }
  const int32_t *pages_in = p.pages_in + (size_t)own * B;
  if (first)
    for (int b = tid; b < B; b += kThreads)
      p.pages_out[(size_t)own * B + b] = pages_in[b] + a_start[b] - r_start[b];
  __syncthreads();
  exclusive_scans(sm, B, warp_sum);
  const CacheGroup &grp = c.grp[own];
  int32_t *list = p.free_pages[own];
  const int F = free_in[own], A = a_start[B], R = r_start[B], N = q_start[B];
  if (first) {
    if (tid == 0) p.free_out[own] = F + R - A;
    if (own == 0)
      for (int b = tid; b <= B; b += kThreads) p.q_start[b] = q_start[b];
  }
  // Page j of sequence b after its release: the pages kept are the first
  // have - rel.
  auto released = [&](int r) {
    const int b = owner(r_start, B, r);
    const int j = pages_in[b] - (r_start[b + 1] - r_start[b]) + (r - r_start[b]);
    return grp.table[(size_t)b * grp.stride + j];
  };
  auto popped = [&](int k) {
    const int at = F + R - 1 - k;
    return at >= F ? released(at - F) : list[at];
  };
  const int step = (int)gridDim.x * kThreads, at0 = (int)blockIdx.x * kThreads + tid;
  for (int64_t r = at0; r < R; r += step) list[F + r] = released((int)r);
  for (int64_t k = at0; k < A; k += step) {
    const int b = owner(a_start, B, (int)k);
    const int j = pages_in[b] + ((int)k - a_start[b]);
    grp.table[(size_t)b * grp.stride + j] = popped((int)k);
  }
  // The page ids are in place before the block can count as finished. (Slots are read only
  // behind a dependency wait. A fence at the end, for all: 256 prompts 23.4 us instead of 21.7.)
  if (at0 < A) __threadfence();
  // ---- slots of this group's heads, rows [r0, r1) of this block: consecutive threads
  // take consecutive heads, then rows. A thread keeps its head and steps through
  // rows, mostly inside one sequence, whose lengths it then keeps too.
  const int nh = grp.size, dr = kThreads / nh;
  const int r0 = (int)((int64_t)blockIdx.x * N / gridDim.x);
  const int r1 = (int)((int64_t)(blockIdx.x + 1) * N / gridDim.x);
  const int rank = tid % nh, h = heads[head_off[own] + rank];
  // slot = page * page_rows + off * off_rows + first
  const int page_rows = nh << lgP, off_rows = c.token_major ? nh : 1;
  const int first_row = c.token_major ? rank : rank << lgP;
  const unsigned pages = (unsigned)grp.pages;
  const int top = F + R - 1;
  const int32_t *row_table = nullptr;
  int shift = 0, have = 0, fresh = 0, b_end = 0;  // of the sequence that holds the row
  const int stop = tid < dr * nh ? r1 : r0;
  int64_t *out = p.slots + ((size_t)r0 + tid / nh) * Hkv + h;
  const size_t out_step = (size_t)dr * Hkv;
  auto page_of = [&](int t) {
    const int j = t >> lgP, at = fresh - j;
    if (j >= have && at >= F) return released(at - F);
    return *(j < have ? row_table + j : list + at);
  };
  auto put = [&](int64_t *to, int t, int page) {
    int64_t slot = (int64_t)page * page_rows + ((t & (P - 1)) * off_rows + first_row);
    if ((unsigned)page >= pages) {
      slot = -1;
      atomicOr(p.status, KVX_DEV_BAD_PAGE);
    }
    *to = slot;
  };
  int row = r0 + tid / nh;
  while (row < stop) {
    if (row >= b_end) {
      const int b = owner(q_start, B, row);
      b_end = q_start[b + 1];
      shift = p.kv_len[(size_t)b * Hkv + h] - q_start[b];
      have = pages_in[b];
      fresh = top - a_start[b] + have;  // page j is at list position fresh - j
      row_table = grp.table + (size_t)b * grp.stride;
    }
    if (row + 3 * dr < min(stop, b_end)) {  // four at a time: their page ids load together
      int page[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) page[u] = page_of(row + u * dr + shift);
#pragma unroll
      for (int u = 0; u < 4; ++u) put(out + u * out_step, row + u * dr + shift, page[u]);
      row += 4 * dr;
      out += 4 * out_step;
    } else {
      put(out, row + shift, page_of(row + shift));
      row += dr;
      out += out_step;
    }
  }
}

}  // namespace

cudaError_t launch_tables(const TablesParams &p, cudaStream_t st) {
  const int64_t slots = (int64_t)p.max_rows * p.c.Hkv;
  const int64_t want = (slots / p.c.G + 8 * kThreads - 1) / (8 * kThreads);
  // four blocks per SM over all groups (256 prompts: two 23 us, four 21, six 27.5, eight 24.5)
  const int most = 608 / p.c.G;
  const unsigned blocks = (unsigned)(want < 1 ? 1 : want > most ? most : want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, (unsigned)p.c.G);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 3 * (size_t)(p.c.B + 1) * sizeof(int);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if (cfg.dynamicSmemBytes > 40 * 1024)  // (4096 + 1) * 12 bytes at most
    e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * (KVX_MAX_CACHE_SEQS + 1) * (int)sizeof(int));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, tables_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvx
