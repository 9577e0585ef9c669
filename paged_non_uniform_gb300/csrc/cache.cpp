// cache.cpp -- the cache handle and the entry points of a speculative-decoding
// step over it: argument validation (everything is checked before anything is
// launched) and launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>

#include "kvx_internal.h"
#include "tree.h"

namespace kvx {
namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// The int32 arrays of a call.
bool aligned_ints(std::initializer_list<const void *> arrays) {
  for (const void *p : arrays)
    if (!aligned(p, 4)) return false;
  return true;
}

bool is_pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

int elem_bytes(const kvx_cache *c) { return c->shape.dtype == KVX_BF16 ? 2 : 4; }

// A row array's stride in bytes, or 0 if it is not usable (from 2^40 bytes on no tensor map
// takes it).
int64_t row_stride(const kvx_cache *c, int64_t stride, int heads) {
  const int64_t es = elem_bytes(c), limit = (int64_t)1 << 40;
  if (stride < (int64_t)heads * c->shape.D || stride >= limit / es || stride * es % 16) return 0;
  return stride * es;
}

// Row arrays hold at most this many rows (row indices and their steps stay in int32).
constexpr int32_t kMaxRows = 1 << 30;

bool workspace_ok(const void *ws, size_t bytes, size_t need) {
  return ws && aligned(ws, 256) && bytes >= need;
}

bool encode(CUtensorMap *tm, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
  typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = []() -> Encode {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return (Encode)f;
  }();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn && fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A 5-D bf16 tensor map over one head group's pool, whose box is one head's rows of a
// page and lands as [8-row group][64-dim half][8 rows][128 bytes], 128-byte swizzled,
// zeros outside: the same distance between all 8-row groups of a tile, which one
// operand descriptor can express. Dims (innermost first):
//   head-major pages:  {64 elements, 8 rows, D/64 halves, P/8 groups, pages * |G|}
//   token-major pages: {64 elements, 8 rows, D/64 halves, pages * P/8 groups, |G|}
bool encode_map(CUtensorMap *tm, const kvx_cache *c, const void *pool, const CacheGroup &g) {
  const cuuint64_t row = (cuuint64_t)c->dev.row_bytes, P = (cuuint64_t)c->dev.P;
  const cuuint64_t n = (cuuint64_t)g.size, pages = (cuuint64_t)g.pages, halves = row / 128;
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, (cuuint32_t)P / 8, 1};
  if (c->dev.token_major) {
    const cuuint64_t dims[5] = {64, 8, halves, pages * P / 8, n};
    const cuuint64_t strides[4] = {row * n, 128, 8 * row * n, row};
    return encode(tm, pool, dims, strides, box);
  }
  const cuuint64_t dims[5] = {64, 8, halves, P / 8, pages * n};
  const cuuint64_t strides[4] = {row, 128, 8 * row, P * row};
  return encode(tm, pool, dims, strides, box);
}

// 5-D map over the query rows, dims {64 elements, D/64 halves, Hq heads, rows, 1}; one
// box {64, 1, g, 8, 1} is the g query heads of one KV head of 8 rows, one half.
bool encode_q_map(CUtensorMap *tm, const kvx_cache *c, const void *q, int64_t stride_bytes,
                  int max_rows) {
  const cuuint64_t row = (cuuint64_t)c->dev.row_bytes;
  const cuuint64_t dims[5] = {64, row / 128, (cuuint64_t)c->dev.Hq, (cuuint64_t)max_rows, 1};
  const cuuint64_t strides[4] = {128, row, (cuuint64_t)stride_bytes, (cuuint64_t)stride_bytes};
  const cuuint32_t box[5] = {64, 1, (cuuint32_t)c->dev.g, kTreeBox, 1};
  return encode(tm, q, dims, strides, box);
}

// Row groups, blocks and the workspace of a cache's attention calls.
struct TreeShape {
  int blocks, tokens, rows;
  TreeWs ws;
};
int tree_shape(const kvx_cache *c, TreeShape *t) {
  int32_t sms = 0;
  const int rc = kvx_device_sm_count(&sms);
  if (rc != KVX_OK) return rc;
  const int g = c->dev.g;
  const bool f32 = c->shape.dtype == KVX_F32;
  t->blocks = sms * (f32 ? tree_simt_blocks_per_sm() : tree_mma_blocks_per_sm());
  t->rows = f32 ? tree_simt_rows() : tree_mma_rows();
  t->tokens = f32 ? tree_simt_tokens(g) : tree_mma_tokens(g);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t slots = (size_t)2 * t->blocks, row = (size_t)c->shape.D * sizeof(float);
  TreeWs &w = t->ws;
  w.split = KVX_WS_HEADER_BYTES;
  w.part_ml = w.split + up(t->blocks * sizeof(TreeSplit));
  w.part_o = w.part_ml + up(slots * t->rows * sizeof(float2));
  w.fold = w.part_o + up(slots * t->rows * row);
  w.total = w.fold + (f32 ? 0 : up((size_t)t->blocks * 128 * row));
  return KVX_OK;
}

}  // namespace
}  // namespace kvx

namespace kvx {

cudaError_t raise_smem_limit(int8_t (&done)[64], const void *kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev] = 1;
  return e;
}

}  // namespace kvx

using namespace kvx;

extern "C" int kvx_cache_create(const kvx_shape *s, const int32_t *head_group,
                                void *const *k_pools, void *const *v_pools,
                                const int64_t *pool_pages, int32_t *const *page_tables,
                                const int32_t *page_table_stride, kvx_cache **out) {
  if (!out) return KVX_EINVAL;
  *out = nullptr;
  if (!s || !head_group || !k_pools || !v_pools || !pool_pages || !page_tables ||
      !page_table_stride)
    return KVX_EINVAL;
  if (s->B < 1 || s->Hkv < 1 || s->Hq < 1 || s->num_groups < 1) return KVX_EINVAL;
  if (s->B > KVX_MAX_CACHE_SEQS || s->Hkv > KVX_MAX_KV_HEADS ||
      s->num_groups > KVX_MAX_GROUPS || s->num_groups > s->Hkv)
    return KVX_EUNSUPPORTED;
  if (s->Hq % s->Hkv != 0) return KVX_EINVAL;
  if (s->Hq / s->Hkv > KVX_MAX_GQA) return KVX_EUNSUPPORTED;
  if (s->D != 64 && s->D != 128) return KVX_EUNSUPPORTED;
  if (!is_pow2(s->page_size) || s->page_size < 8 || s->page_size > 128) return KVX_EUNSUPPORTED;
  if (s->dtype != KVX_F32 && s->dtype != KVX_BF16) return KVX_EUNSUPPORTED;
  if (s->layout != KVX_LAYOUT_HEAD_MAJOR && s->layout != KVX_LAYOUT_TOKEN_MAJOR)
    return KVX_EUNSUPPORTED;
  const int G = s->num_groups, Hkv = s->Hkv;
  int32_t size[KVX_MAX_GROUPS] = {0};
  for (int h = 0; h < Hkv; ++h) {
    if (head_group[h] < 0 || head_group[h] >= G) return KVX_EINVAL;
    size[head_group[h]] += 1;
  }
  for (int gi = 0; gi < G; ++gi) {
    if (size[gi] == 0) return KVX_EINVAL;
    if (!k_pools[gi] || !v_pools[gi] || !page_tables[gi]) return KVX_EINVAL;
    if (!aligned(k_pools[gi], 16) || !aligned(v_pools[gi], 16) || !aligned(page_tables[gi], 4))
      return KVX_EINVAL;
    if (pool_pages[gi] < 1 || page_table_stride[gi] < 1) return KVX_EINVAL;
    if (pool_pages[gi] >= ((int64_t)1 << 31) - 1 ||
        (int64_t)page_table_stride[gi] * s->page_size > INT32_MAX)
      return KVX_ERANGE;
    // (coordinates of the tensor maps)
    if (s->dtype == KVX_BF16 &&
        (pool_pages[gi] + 1) * std::max(size[gi], s->page_size / 8) > INT32_MAX)
      return KVX_ERANGE;
  }
  kvx_cache *c = new (std::nothrow) kvx_cache();
  if (!c) return KVX_ENOMEM;
  c->shape = *s;
  CacheDev &d = c->dev;
  std::memset(&d, 0, sizeof(d));
  d.B = s->B;
  d.Hq = s->Hq;
  d.Hkv = Hkv;
  d.D = s->D;
  d.g = s->Hq / Hkv;
  d.G = G;
  d.P = s->page_size;
  while ((1 << d.lgP) < d.P) ++d.lgP;
  d.token_major = s->layout == KVX_LAYOUT_TOKEN_MAJOR;
  d.row_bytes = s->D * elem_bytes(c);
  int32_t seen[KVX_MAX_GROUPS] = {0};
  for (int h = 0; h < Hkv; ++h) {
    d.head_grp[h] = (int8_t)head_group[h];
    d.head_row[h] = (int8_t)seen[head_group[h]]++;
  }
  for (int gi = 0; gi < G; ++gi)
    d.grp[gi] = {page_tables[gi],
                 (char *)k_pools[gi],
                 (char *)v_pools[gi],
                 pool_pages[gi],
                 page_table_stride[gi],
                 size[gi],
                 (int32_t)std::min((int64_t)page_table_stride[gi] * s->page_size, kMaxTokens)};
  c->stall_block = -1;
  c->wait_ns = 2000000000u;
  c->have_maps = s->dtype == KVX_BF16;
  for (int gi = 0; gi < G && c->have_maps; ++gi)
    c->have_maps = encode_map(&c->k_maps[gi], c, d.grp[gi].k, d.grp[gi]) &&
                   encode_map(&c->v_maps[gi], c, d.grp[gi].v, d.grp[gi]);
  *out = c;
  return KVX_OK;
}

extern "C" void kvx_cache_destroy(kvx_cache *c) { delete c; }

extern "C" int kvx_cache_inject_stall(kvx_cache *c, int32_t block, uint64_t wait_limit_ns) {
  if (!c) return KVX_EINVAL;
  if (wait_limit_ns < 1000000ull || wait_limit_ns > 4000000000ull) return KVX_ERANGE;
  c->stall_block = block < 0 ? -1 : block;
  c->wait_ns = (uint32_t)wait_limit_ns;
  return KVX_OK;
}

extern "C" int kvx_build_tables(const kvx_cache *c, const int32_t *kv_len, const int32_t *new_len,
                                const int32_t *pages_in, int32_t *pages_out,
                                int32_t *const *free_pages, const int32_t *free_in,
                                int32_t *free_out, int32_t max_rows, int32_t *q_start,
                                int64_t *slots, void *workspace, size_t workspace_bytes,
                                void *stream) {
  if (!c || !kv_len || !new_len || !pages_in || !pages_out || !free_pages || !free_in ||
      !free_out || !q_start || max_rows < 0 || (max_rows > 0 && !slots))
    return KVX_EINVAL;
  if (max_rows > kMaxRows) return KVX_ERANGE;
  if (pages_in == pages_out || free_in == free_out || !aligned(slots, 8)) return KVX_EINVAL;
  if (!aligned_ints({kv_len, new_len, pages_in, pages_out, free_in, free_out, q_start}))
    return KVX_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, KVX_WS_HEADER_BYTES)) return KVX_EINVAL;
  TablesParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = c->dev;
  for (int gi = 0; gi < c->dev.G; ++gi) {
    if (!free_pages[gi] || !aligned(free_pages[gi], 4)) return KVX_EINVAL;
    p.free_pages[gi] = free_pages[gi];
  }
  p.kv_len = kv_len;
  p.new_len = new_len;
  p.pages_in = pages_in;
  p.pages_out = pages_out;
  p.free_in = free_in;
  p.free_out = free_out;
  p.q_start = q_start;
  p.slots = slots;
  p.status = (uint32_t *)workspace;
  p.max_rows = max_rows;
  const cudaError_t e = launch_tables(p, (cudaStream_t)stream);
  return e == cudaSuccess ? KVX_OK : set_cuda_error(e);
}

extern "C" int kvx_append_kv(const kvx_cache *c, const void *k_new, int64_t k_stride,
                             const void *v_new, int64_t v_stride, const int32_t *q_start,
                             const int64_t *slots, int32_t max_rows, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (!c || !q_start || max_rows < 0) return KVX_EINVAL;
  if (max_rows > 0 && (!k_new || !v_new || !slots)) return KVX_EINVAL;
  if (max_rows > kMaxRows) return KVX_ERANGE;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slots, 8)) return KVX_EINVAL;
  if (!aligned(q_start, 4)) return KVX_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, KVX_WS_HEADER_BYTES)) return KVX_EINVAL;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = c->dev;
  p.k = (const char *)k_new;
  p.v = (const char *)v_new;
  p.k_stride = row_stride(c, k_stride, c->dev.Hkv);
  p.v_stride = row_stride(c, v_stride, c->dev.Hkv);
  if (!p.k_stride || !p.v_stride) return KVX_EINVAL;
  p.q_start = q_start;
  p.slots = slots;
  p.status = (uint32_t *)workspace;
  p.max_rows = max_rows;
  const cudaError_t e = launch_append(p, (cudaStream_t)stream);
  return e == cudaSuccess ? KVX_OK : set_cuda_error(e);
}

extern "C" int kvx_tree_attn_workspace_bytes(const kvx_cache *c, int32_t max_q, size_t *bytes) {
  if (!c || !bytes) return KVX_EINVAL;
  if (max_q < 1 || max_q > KVX_MAX_TREE) return KVX_ERANGE;
  TreeShape t;
  const int rc = tree_shape(c, &t);
  if (rc == KVX_OK) *bytes = t.ws.total;
  return rc;
}

extern "C" int kvx_tree_attn(const kvx_cache *c, const void *q, int64_t q_stride,
                             const int32_t *q_start, int32_t max_rows, int32_t max_q,
                             const int32_t *kv_len, const uint32_t *mask, float scale, float *out,
                             void *workspace, size_t workspace_bytes, void *stream) {
  if (!c || !q_start || !kv_len || max_rows < 0) return KVX_EINVAL;
  if (max_rows > 0 && (!q || !out)) return KVX_EINVAL;
  if (max_q < 1 || max_q > KVX_MAX_TREE || max_rows > kMaxRows) return KVX_ERANGE;
  if (!std::isfinite(scale) || scale < 0.f) return KVX_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned_ints({mask, q_start, kv_len}))
    return KVX_EINVAL;
  TreeParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = c->dev;
  p.q_stride = row_stride(c, q_stride, c->dev.Hq);
  if (!p.q_stride) return KVX_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, KVX_WS_HEADER_BYTES)) return KVX_EINVAL;
  TreeShape t;
  const int rc = tree_shape(c, &t);
  if (rc != KVX_OK) return rc;
  const TreeWs &w = t.ws;
  if (workspace_bytes < w.total) return KVX_EINVAL;
  if (max_rows == 0) return KVX_OK;
  char *ws = (char *)workspace;
  p.q = (const char *)q;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.mask = mask;
  p.out = out;
  p.status = (uint32_t *)ws;
  p.split = (TreeSplit *)(ws + w.split);
  p.part_ml = (float2 *)(ws + w.part_ml);
  p.part_o = (float *)(ws + w.part_o);
  p.fold = (float *)(ws + w.fold);
  p.max_rows = max_rows;
  p.max_q = max_q;
  p.stall_block = c->stall_block;
  p.wait_ns = c->wait_ns;
  p.words = (max_q + 31) / 32;
  p.group_tokens = t.tokens;
  p.group_rows = t.rows;
  p.recip_g = (65536 + c->dev.g - 1) / c->dev.g;
  const float sc = scale == 0.f ? 1.0f / std::sqrt((float)c->dev.D) : scale;
  p.scale_log2 = (float)((double)sc * 1.4426950408889634);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaErrorInvalidValue;
  CUtensorMap q_map;
  if (c->shape.dtype == KVX_F32)
    e = launch_tree_simt(p, t.blocks, st);
  else if (c->have_maps && encode_q_map(&q_map, c, q, p.q_stride, max_rows))
    e = launch_tree_mma(p, c->k_maps, c->v_maps, q_map, t.blocks, st);
  if (e == cudaSuccess) e = launch_tree_merge(p, t.blocks, st);
  return e == cudaSuccess ? KVX_OK : set_cuda_error(e);
}

extern "C" int kvx_tree_commit(const kvx_cache *c, const int32_t *q_start, const int64_t *slots,
                               int32_t max_rows, const int32_t *path, int32_t path_stride,
                               const int32_t *n_acc, const int32_t *kv_len, int32_t *kv_len_out,
                               void *workspace, size_t workspace_bytes, void *stream) {
  if (!c || !q_start || !path || !n_acc || !kv_len || !kv_len_out || max_rows < 0 ||
      (max_rows > 0 && !slots) || path_stride < 1)
    return KVX_EINVAL;
  if (max_rows > kMaxRows) return KVX_ERANGE;
  if (!aligned(slots, 8) || !aligned_ints({q_start, path, n_acc, kv_len, kv_len_out}))
    return KVX_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, KVX_WS_HEADER_BYTES)) return KVX_EINVAL;
  CommitParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = c->dev;
  p.q_start = q_start;
  p.slots = slots;
  p.path = path;
  p.n_acc = n_acc;
  p.kv_len = kv_len;
  p.kv_out = kv_len_out;
  p.status = (uint32_t *)workspace;
  p.max_rows = max_rows;
  p.path_stride = path_stride;
  const cudaError_t e = launch_commit(p, (cudaStream_t)stream);
  return e == cudaSuccess ? KVX_OK : set_cuda_error(e);
}
