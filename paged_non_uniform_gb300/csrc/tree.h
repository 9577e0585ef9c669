// tree.h -- structures shared by the cache handle, its entry points and the
// kernels of a speculative-decoding step (tables, append, tree attention,
// branch commit). Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx.h"

namespace kvx {

// Tokens of a head in tree attention, new rows included: the kernels' positions run past the last
// one by up to a tile, and those of the lanes that look up page ids by 31 boxes of 128 more,
// within int32.
constexpr int64_t kMaxTokens = INT32_MAX - 4096;

// One head group of a cache: its page table [B][stride] and its pools.
struct CacheGroup {
  int32_t *table;
  char *k, *v;
  int64_t pages;  // in each pool
  int32_t stride, size;
  int32_t tokens;  // a sequence's room in the table, at most kMaxTokens
};

// The cache as the kernels see it (passed by value in their parameters).
// The kernels are programmatic dependents: a grid may be resident while the kernel before it
// still writes the lengths, tables, slots and rows that it will read. They are therefore read
// with ordinary loads after the dependency wait, never through the non-coherent path (whose data
// must not change while the grid runs, and whose loads may move ahead of the wait).
struct CacheDev {
  CacheGroup grp[KVX_MAX_GROUPS];
  int32_t B, Hq, Hkv, D, g, G;
  int32_t P, lgP;       // page size and its log2
  int32_t token_major;  // page layout
  int32_t row_bytes;    // D elements
  int8_t head_grp[KVX_MAX_KV_HEADS];
  int8_t head_row[KVX_MAX_KV_HEADS];
};

// Row of a group's pool that holds token slot `off` of page `page` of the head
// with rank r.
__host__ __device__ inline int64_t pool_row(const CacheDev &c, const CacheGroup &g, int64_t page,
                                            int r, int off) {
  return c.token_major ? (page * c.P + off) * g.size + r
                       : ((page * g.size + r) << c.lgP) + off;
}

struct TablesParams {
  CacheDev c;
  int32_t *free_pages[KVX_MAX_GROUPS];
  const int32_t *kv_len, *new_len, *pages_in, *free_in;
  int32_t *pages_out, *free_out, *q_start;
  int64_t *slots;
  uint32_t *status;
  int32_t max_rows;
};

struct AppendParams {
  CacheDev c;
  const char *k, *v;
  int64_t k_stride, v_stride;  // bytes
  const int32_t *q_start;
  const int64_t *slots;
  uint32_t *status;
  int32_t max_rows;
};

struct CommitParams {
  CacheDev c;
  const int32_t *q_start, *path, *n_acc, *kv_len;
  const int64_t *slots;
  int32_t *kv_out;
  uint32_t *status;
  int32_t max_rows, path_stride;
};

// A row group that starts in block c and runs on: `parts` partials, the first in slot
// 2c + 1, the others in slots 2c of the blocks that follow (0: none).
struct TreeSplit {
  int32_t parts, row0, h, rows;
};

// Tree attention. A head's keys come in tiles, its query rows (new row i and
// query head j of the KV head: row i * g + j) in groups; tree_split.cuh
// says how the (row group, tile) units are cut over the blocks.
struct TreeParams {
  CacheDev c;
  const char *q;
  int64_t q_stride;  // bytes
  const int32_t *q_start, *kv_len;
  const uint32_t *mask;
  float *out;
  uint32_t *status;
  TreeSplit *split;   // [blocks] the row group that starts in the block and runs on
  float2 *part_ml;    // [2 * blocks][group_rows] = (max in log2 units, sum)
  float *part_o;      // [2 * blocks][group_rows][D]
  float *fold;        // tensor-core kernel: fp32 output sums of long items, [blocks][D / 4][128][4]
  int32_t max_rows, max_q, words;  // words: uint32 words of a mask row
  int32_t group_tokens;            // new rows of a row group
  int32_t group_rows;              // room for its query rows
  int32_t recip_g;                 // ceil(2^16 / g): r * recip_g >> 16 = r / g for r <= 1024
  float scale_log2;                // scale * log2(e)
  int32_t stall_block;             // failure-detection test (-1: none)
  uint32_t wait_ns;                // limit of every pipeline wait
};

// Workspace of tree attention: header | split row groups | partial (m, l) | partial o |
// folded o.
struct TreeWs {
  size_t split, part_ml, part_o, fold, total;
};

cudaError_t launch_tables(const TablesParams &p, cudaStream_t st);
cudaError_t launch_append(const AppendParams &p, cudaStream_t st);
cudaError_t launch_commit(const CommitParams &p, cudaStream_t st);
// fp32 caches: CUDA cores; bf16 caches: tensor cores.
cudaError_t launch_tree_simt(const TreeParams &p, int blocks, cudaStream_t st);
int tree_simt_tokens(int g);    // new rows of a row group; its query rows:
int tree_simt_rows();
int tree_simt_blocks_per_sm();  // resident blocks
constexpr int kTreeBox = 8;     // new rows of a query load
cudaError_t launch_tree_mma(const TreeParams &p, const CUtensorMap *k_maps,
                            const CUtensorMap *v_maps, const CUtensorMap &q_map, int blocks,
                            cudaStream_t st);
int tree_mma_tokens(int g);
int tree_mma_rows();
int tree_mma_blocks_per_sm();
// Raises a kernel's shared-memory limit on the current device, once (`done`: one flag per
// device, of that kernel).
cudaError_t raise_smem_limit(int8_t (&done)[64], const void *kernel, int bytes);
// Folds the partials of split row groups (after either kernel).
cudaError_t launch_tree_merge(const TreeParams &p, int blocks, cudaStream_t st);

}  // namespace kvx

struct kvx_cache {
  kvx_shape shape;
  kvx::CacheDev dev;
  // bf16 caches: maps of each group's pools (absent where no driver is loaded)
  CUtensorMap k_maps[KVX_MAX_GROUPS];
  CUtensorMap v_maps[KVX_MAX_GROUPS];
  bool have_maps;
  int32_t stall_block;  // kvx_cache_inject_stall
  uint32_t wait_ns;
};
