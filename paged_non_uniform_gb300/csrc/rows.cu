// rows.cu -- movement of new K/V rows: the append of a step's rows into their
// slots and the compaction of accepted tree branches. Both copy 16-byte chunks
// and do no arithmetic on them, so memory bounds them.
// Measured on one GB300: 751 MB of prompt rows appended in 117 us (6.4 TB/s, 95 % of a
// copy); a step of 16 x 16 rows 2.6 us; branches of 16 sequences committed in 4.4 us, of
// 256 sequences in 5.6 (three dependent loads, then the rows: latency). 0.5 to
// 0.7 us of each is the fence.
// Neither lets its dependents start early: a decode call with early loads reads pages before its
// dependency wait, and may stand behind kernels that do let theirs start, so that only a launch
// held back until the pages are written protects it. (The fence at the end has every write
// performed before the block counts as finished.)
#include "ptx.cuh"
#include "tree.h"

namespace kvx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t pool_rows(const CacheDev &c, int grp) {
  return c.grp[grp].pages * c.grp[grp].size * c.P;
}

// pool[slots[r][h]] = new[r][h] for K and V. One thread per 16-byte chunk of a
// (row, head), K and V together.
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  const CacheDev &c = p.c;
  const int cpr = c.row_bytes >> 4;  // chunks of a row: 8, 16 or 32
  const int stated = p.q_start[c.B], rows = min(stated, p.max_rows);
  if ((stated < 0 || stated > p.max_rows) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  if (rows <= 0) return;
  const int64_t total = (int64_t)rows * c.Hkv * cpr;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t rh = i / cpr;
    const int ch = (int)(i - rh * cpr);
    const int64_t r = rh / c.Hkv;
    const int h = (int)(rh - r * c.Hkv);
    const int64_t slot = p.slots[rh];
    const int grp = c.head_grp[h];
    if (slot < 0 || slot >= pool_rows(c, grp)) {
      if (slot != -1 && ch == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t src = (int64_t)h * c.row_bytes + ch * 16;
    const uint4 kv = *(const uint4 *)(p.k + r * p.k_stride + src);
    const uint4 vv = *(const uint4 *)(p.v + r * p.v_stride + src);
    const int64_t dst = slot * c.row_bytes + ch * 16;
    *(uint4 *)(c.grp[grp].k + dst) = kv;
    *(uint4 *)(c.grp[grp].v + dst) = vv;
  }
  __threadfence();
}

// row n + j <- row n + path[j]. One thread owns one 16-byte column of K or V of
// one head and walks j upwards: path ascends strictly, so path[j] >= j and
// every source of a later j lies past all targets written so far. A batch of
// eight loads therefore may precede its eight stores, and no thread reads what
// another writes. A block holds whole heads, whose lengths it checks and advances itself
// (kv_out may be kv_len).
__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  pdl_wait();
  const CacheDev &c = p.c;
  const int b = blockIdx.y;
  const int cpr = c.row_bytes >> 4;
  const int per_head = 2 * cpr;  // K chunks, then V chunks: 16, 32 or 64
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int h = i / per_head, x = i - h * per_head;
  const CacheGroup &g = c.grp[c.head_grp[min(h, c.Hkv - 1)]];
  const size_t bh = (size_t)b * c.Hkv + h;
  const int n = h < c.Hkv ? p.kv_len[bh] : 0;
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
  const int a = p.n_acc[b];
  const bool rows_ok = q0 >= 0 && q1 >= q0 && q1 <= p.max_rows;
  const int *path = p.path + (size_t)b * p.path_stride;
  int bad = !(rows_ok && a >= 0 && a <= q1 - q0 && a <= p.path_stride);
  if (!bad)
    for (int j = threadIdx.x; j < a; j += kThreads) {
      const int v = path[j], before = j ? path[j - 1] : -1;
      bad |= v <= before || v >= q1 - q0;
    }
  // of the sequence; the block has read its lengths before any of them is written
  const bool seq_ok = __syncthreads_or(bad) == 0;
  if (h >= c.Hkv) return;
  const bool ok = seq_ok && n >= 0 && (int64_t)n + (q1 - q0) <= ((int64_t)g.stride << c.lgP);
  if (x == 0) {
    p.kv_out[bh] = n + (ok ? a : 0);
    if (!ok) atomicOr(p.status, KVX_DEV_BAD_LENGTH);
  }
  if (!ok || a == 0) return;
  char *pool = (x < cpr ? g.k : g.v) + (x < cpr ? x : x - cpr) * 16;
  const int64_t limit = g.pages * g.size * c.P;
  const int64_t *slots = p.slots + (size_t)q0 * c.Hkv + h;
  for (int j0 = 0; j0 < a; j0 += 8) {
    uint4 v[8];
    int64_t to[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u;
      to[u] = -1;
      if (j >= a) continue;
      const int s = path[j];
      if (s == j) continue;
      const int64_t from = slots[(size_t)s * c.Hkv], t = slots[(size_t)j * c.Hkv];
      if (from < 0 || from >= limit || t < 0 || t >= limit) {
        if (x == 0) atomicOr(p.status, KVX_DEV_BAD_BLOCK);
        continue;
      }
      to[u] = t;
      v[u] = *(const uint4 *)(pool + from * c.row_bytes);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (to[u] >= 0) *(uint4 *)(pool + to[u] * c.row_bytes) = v[u];
  }
  __threadfence();
}

cudaLaunchConfig_t config(dim3 grid, cudaStream_t st, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int64_t chunks = (int64_t)p.max_rows * p.c.Hkv * (p.c.row_bytes >> 4);
  const int64_t blocks = (chunks + kThreads - 1) / kThreads;
  // At most 32 blocks per SM: the fence at a thread's end waits for its stores, which short
  // threads pay often (751 MB: 8 blocks 125 us, 16 123, 32 117, 64 118, one chunk a thread 133).
  const int64_t most = 32 * 152;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dim3((unsigned)(blocks < most ? blocks : most)), st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t st) {
  const int threads = p.c.Hkv * 2 * (p.c.row_bytes >> 4);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg =
      config(dim3((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)p.c.B), st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, commit_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvx
