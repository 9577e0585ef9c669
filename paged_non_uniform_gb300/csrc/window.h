// window.h -- structures of the calls that keep a cache within a memory budget:
// attention with windows, sinks and accumulated weights, eviction, rows of 4-bit
// caches. Not part of the public interface.
#pragma once

#include "tree.h"

namespace kvx {

// ---- 4-bit rows -----------------------------------------------------------
// A row of D elements is D / 64 groups of 64: an element is lo + step * code, lo and step
// bf16 of its group. A head's P rows of a page are one block: the codes of all rows
// [P][D / 2 bytes], then their parameters [P][D / 64][step, lo]. Eight elements are
// a 32-bit word, lowest bits first; word w of a row of 128 is stored at 2 (w % 8) + w / 8, so
// that eight bytes hold the same eight elements of both groups: a thread's share of a
// row in either matrix product (window_mma.cuh).
constexpr int kQ4Group = 64;
__host__ __device__ constexpr int q4_code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int q4_param_bytes(int D) { return D / 16; }
__host__ __device__ constexpr int q4_row_bytes(int D) { return q4_code_bytes(D) + q4_param_bytes(D); }
// Byte offsets in its pool of the codes and the parameters of a row (pages are powers of two).
__host__ __device__ inline int64_t q4_codes(const CacheDev &c, int64_t row) {
  return (row >> c.lgP) * ((int64_t)q4_row_bytes(c.D) << c.lgP) + (row & (c.P - 1)) * q4_code_bytes(c.D);
}
__host__ __device__ inline int64_t q4_params(const CacheDev &c, int64_t row) {
  return (row >> c.lgP) * ((int64_t)q4_row_bytes(c.D) << c.lgP) + ((int64_t)q4_code_bytes(c.D) << c.lgP) +
         (row & (c.P - 1)) * q4_param_bytes(c.D);
}

// ---- attention ------------------------------------------------------------
constexpr int kWindowTile = 64;  // keys of a tile
constexpr int kWindowBox = 32;   // of a stage of bf16 caches, and of a load at most

struct WindowParams : TreeParams {
  const int32_t *sinks, *window;  // [Hkv], or null: no sinks, everything visible
  // With weights (scores not null): the scores of every (row, visited key) in log2 units,
  // [B * Hkv][row groups][score_keys][score_rows], -inf where the row does not see the key.
  float *scores;
  int64_t score_keys;  // a head's visited keys, rounded up to tiles, at most
  int32_t score_rows;  // rows of a row group, rounded up to a multiple of 4
  int32_t score_groups;
  float *weights[KVX_MAX_GROUPS];
};

// Workspace: tree attention's, then with weights (max, sum) of every row, where the split row
// groups begin in it, and the scores.
struct WindowShape {
  int blocks, tokens, rows;
  TreeWs ws;
  size_t row_ml, split_row, scores, total;
};

// Tensor-core kernels' parameters.
struct alignas(128) WindowMmaParams {
  CUtensorMap tmK[KVX_MAX_GROUPS];  // bf16 caches
  CUtensorMap tmV[KVX_MAX_GROUPS];
  WindowParams w;
};

// fp32 caches: CUDA cores; bf16 and 4-bit caches: tensor cores.
cudaError_t launch_window_simt(const WindowParams &p, int blocks, cudaStream_t st);
cudaError_t launch_window_bf16(const WindowMmaParams &p, int blocks, cudaStream_t st);
cudaError_t launch_window_q4(const WindowMmaParams &p, int blocks, cudaStream_t st);
int window_simt_rows();  // query rows of a row group
// of the tensor-core kernels, where a head has `rows` in all: one instance each
constexpr int window_mma_rows(int rows, bool q4) {
  return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 || q4 ? 16 : 32;
}
constexpr int kWindowBlocksPerSm = 2;
constexpr int window_mma_blocks_per_sm(int rows) { return rows == 32 ? 3 : 2; }
cudaError_t launch_weigh(const WindowParams &p, int blocks, cudaStream_t st);

// ---- rows of 4-bit caches, rows read back ----------------------------------
cudaError_t launch_q4_append(const AppendParams &p, cudaStream_t st);
struct ReadParams {
  CacheDev c;
  char *k, *v;
  int64_t k_stride, v_stride;  // bytes
  const int32_t *q_start;
  const int64_t *slots;
  uint32_t *status;
  int32_t max_rows, q4;
};
cudaError_t launch_read(const ReadParams &p, cudaStream_t st);

// ---- eviction ---------------------------------------------------------------
// A unit of the move: kEvictChunk target places of a head. A head's arrays hold a number per
// chunk of the tokens that its page table has room for, heads one after the other.
constexpr int kEvictChunk = 64;
struct alignas(16) EvictUnit {
  int32_t bh, chunk;  // head, first place / kEvictChunk
  int32_t count;      // places
  int32_t wait_from;  // first chunk whose unit reads what this one overwrites
};
struct EvictParams {
  CacheDev c;
  const int32_t *kv_len, *budget;
  int32_t *kv_out;
  int32_t sinks, recent;
  int32_t q4;            // 4-bit rows
  int32_t copy_weights;  // weights_out is not weights
  const float *weights[KVX_MAX_GROUPS];
  float *weights_out[KVX_MAX_GROUPS];
  uint32_t *status;
  uint32_t *counters;   // [0] units, [1] tickets, [2] blocks done
  EvictUnit *units;     // [chunks]
  uint32_t *read_done;  // [chunks] the unit's rows have been read
  int32_t *source;      // per head and kept token: the token that it was
  int64_t chunks;       // of all heads
  int64_t chunks_seq;   // of a sequence's heads
  int32_t chunk_off[KVX_MAX_KV_HEADS];  // where a KV head's begin among them
  int32_t stall_block;                  // failure-detection test (-1: none)
  uint32_t wait_ns;
};
// Workspace: header | units | read_done | source.
struct EvictWs {
  size_t read_done, source, total;
};
cudaError_t launch_evict(const EvictParams &p, cudaStream_t st);

}  // namespace kvx
