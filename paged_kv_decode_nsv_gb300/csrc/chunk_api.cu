// Host side of the chunk attention (nsv_chunk_workspace, nsv_paged_chunk,
// nsv_chunk_step): argument checks, workspace layout, tensor maps, launches.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "chunk.cuh"

namespace nsv {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_chunk(const nsv_shape* s, int64_t tokens) {
  const int rc = check_shape(s);
  if (rc) return rc;
  if (s->query_len > 1 || tokens < 0 || tokens >= kMaxTokens) return NSV_ERR_SHAPE;
  // the tensor maps' block coordinate is a signed 32-bit count of 8-token groups
  if (s->dtype == NSV_BF16 &&
      (s->num_blocks + 1) * (int64_t)s->num_kv_heads * 2 >= (int64_t(1) << 31))
    return NSV_ERR_SHAPE;
  return NSV_OK;
}

ChunkWs workspace_of(const nsv_shape* s, int64_t tokens, int num_sms) {
  return make_chunk_ws(s->rows, tokens, s->num_kv_heads, s->num_heads / s->num_kv_heads,
                       s->head_dim, s->dtype, num_sms);
}

// The pools for the bf16 kernel: the rows of [block][kv_head][token] seen as
// [64 dims][8 rows][64-dim halves][groups of 8 rows], so that one box (a block
// of one KV head) lands as [2 groups][half][8 rows][128 bytes].
bool encode_pool(const DeviceInfo& d, const nsv_shape* s, const void* pool, CUtensorMap* map) {
  const cuuint64_t D = (cuuint64_t)s->head_dim;
  const cuuint64_t groups = (cuuint64_t)(s->num_blocks + 1) * s->num_kv_heads * (kBlock / 8);
  const cuuint64_t dims[4] = {64u, 8u, D / 64, groups};
  const cuuint64_t strides[3] = {D * 2, 128u, D * 2 * 8};
  const cuuint32_t box[4] = {64u, 8u, (cuuint32_t)(D / 64), kBlock / 8};
  const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  return d.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The query tokens as [head_dim][heads][tokens]; one box is 64 dims of the
// query heads of one KV head for as many tokens as fit `rows` MMA rows (no map
// where not even one does).
bool chunk_encode_q(const DeviceInfo& d, const nsv_shape* s, int64_t tokens, int rows,
                    const void* q, CUtensorMap* map) {
  const int box_tokens = rows / (s->num_heads / s->num_kv_heads);
  if (box_tokens == 0) return true;
  const cuuint64_t D = (cuuint64_t)s->head_dim, H = (cuuint64_t)s->num_heads;
  const cuuint64_t dims[3] = {D, H, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {D * 2, D * 2 * H};
  const cuuint32_t box[3] = {64u, (cuuint32_t)(s->num_heads / s->num_kv_heads),
                             (cuuint32_t)box_tokens};
  const cuuint32_t one[3] = {1u, 1u, 1u};
  return d.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// All checks, then (with `append`) the append's launch, the plan's and the
// attention's.
int chunk_impl(const nsv_shape* s, const nsv_scores* sc, int64_t tokens, const void* q,
               const void* k_pool, const void* v_pool, const int32_t* block_tables,
               const int32_t* chunk_starts, const int32_t* context_lens, float scale, void* out,
               void* ws, size_t ws_bytes, cudaStream_t stream, const KvWriteParams* append) {
  int rc = check_chunk(s, tokens);
  if (rc) return rc;
  if (s->rows == 0 || tokens == 0) return NSV_OK;  // nothing to read or write
  if (!q || !k_pool || !v_pool || !block_tables || !chunk_starts || !context_lens || !out)
    return NSV_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(chunk_starts, 4) || !aligned(context_lens, 4))
    return NSV_ERR_ALIGN;
  if (sc) {
    if (sc->softcap != 0.f && !(sc->softcap >= 1e-6f && sc->softcap <= 1e6f)) return NSV_ERR_RANGE;
    if (!aligned(sc->slopes, 4) || !aligned(sc->see_begin, 4) || !aligned(sc->see_end, 4))
      return NSV_ERR_ALIGN;
  }
  DeviceInfo d;
  if ((rc = device_info(&d)) != NSV_OK) return rc;
  const ChunkWs W = workspace_of(s, tokens, d.num_sms);
  if (!ws || ws_bytes < W.total || !aligned(ws, 256)) return NSV_ERR_WORKSPACE;
  char* b = static_cast<char*>(ws);
  const int group = s->num_heads / s->num_kv_heads;
  ChunkParams p;
  memset(&p, 0, sizeof p);
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.block_tables = block_tables;
  p.chunk_starts = chunk_starts;
  p.context_lens = context_lens;
  p.slopes = sc ? sc->slopes : nullptr;
  p.see_begin = sc ? sc->see_begin : nullptr;
  p.see_end = sc ? sc->see_end : nullptr;
  p.out = out;
  p.ws_head = reinterpret_cast<long long*>(b);
  p.ws_prefix = reinterpret_cast<long long*>(b + W.off_prefix);
  p.ws_tiles = reinterpret_cast<int4*>(b + W.off_tiles);
  p.ws_cta = reinterpret_cast<int4*>(b + W.off_cta);
  p.ws_cnt = reinterpret_cast<int32_t*>(b + W.off_cnt);
  p.ws_ml = reinterpret_cast<float2*>(b + W.off_ml);
  p.ws_acc = reinterpret_cast<float*>(b + W.off_acc);
  p.status = d.status;
  p.pool_blocks = s->num_blocks + 1;
  p.tokens = tokens;
  p.rows = s->rows;
  p.heads = s->num_heads;
  p.kv_heads = s->num_kv_heads;
  p.group = group;
  p.max_blocks = s->max_blocks;
  p.max_tiles = W.max_tiles;
  p.tile_rows = W.tile_rows;
  p.tile_tokens = chunk_tile_tokens(s->dtype, group);
  p.keys = s->dtype == NSV_F32 ? kChunkKeysF32 : kChunkKeys;
  p.scale = scale;
  p.qscale = scale * 1.4426950408889634f;  // the kernels use exp2
  p.cap = sc ? sc->softcap : 0.f;
  p.grid = d.num_sms;  // one CTA per SM: it takes all the tensor memory
  p.tile_cost = s->dtype == NSV_F32 ? kChunkTileCostF32 : kChunkTileCost;
  p.pair_units = s->dtype == NSV_F32 ? 1 : kChunkPairUnits;
  p.half_units = s->dtype == NSV_F32 ? 1 : kChunkHalfUnits;
  p.ws_first = reinterpret_cast<long long*>(p.ws_cta + p.grid);
  if (s->dtype == NSV_BF16 &&
      (!chunk_encode_q(d, s, tokens, kChunkHalfRows, q, &p.tmap_q[0]) ||
       !chunk_encode_q(d, s, tokens, kChunkHalfRows / 2, q, &p.tmap_q[1]) ||
       !chunk_encode_q(d, s, tokens, kChunkHalfRows / 4, q, &p.tmap_q[2]) ||
       !encode_pool(d, s, k_pool, &p.tmap_k) || !encode_pool(d, s, v_pool, &p.tmap_v)))
    return cuda_fail();
  if (append && launch_kv_write(*append, stream) != cudaSuccess) return cuda_fail();
  if (launch_chunk_plan(p, stream) != cudaSuccess) return cuda_fail();
  const cudaError_t e = s->dtype == NSV_F32 ? launch_chunk_f32(p, s->head_dim, stream)
                                            : launch_chunk_bf16(p, s->head_dim, stream);
  return e == cudaSuccess ? NSV_OK : cuda_fail();
}

}  // namespace
}  // namespace nsv

using namespace nsv;

extern "C" {

NSV_API int nsv_chunk_workspace(const nsv_shape* shape, int64_t tokens, int num_sms,
                                int64_t* bytes) {
  if (!bytes) return NSV_ERR_NULLPTR;
  int rc = check_chunk(shape, tokens);
  if (rc) return rc;
  if (num_sms <= 0) {
    DeviceInfo d;
    if ((rc = device_info(&d)) != NSV_OK) return rc;
    num_sms = d.num_sms;
  }
  *bytes = (int64_t)workspace_of(shape, tokens, num_sms).total;
  return NSV_OK;
}

NSV_API int nsv_paged_chunk(const nsv_shape* shape, const nsv_scores* scores, int64_t tokens,
                            const void* q, const void* k_pool, const void* v_pool,
                            const int32_t* block_tables, const int32_t* chunk_starts,
                            const int32_t* context_lens, float scale, void* out, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  return chunk_impl(shape, scores, tokens, q, k_pool, v_pool, block_tables, chunk_starts,
                    context_lens, scale, out, workspace, workspace_bytes, stream, nullptr);
}

NSV_API int nsv_chunk_step(const nsv_shape* shape, const nsv_scores* scores, int64_t tokens,
                           const void* q, const void* k_new, const void* v_new,
                           const int64_t* write_slots, void* k_pool, void* v_pool,
                           const int32_t* block_tables, const int32_t* chunk_starts,
                           const int32_t* context_lens, float scale, void* out, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_chunk(shape, tokens);
  if (rc) return rc;
  if (shape->rows == 0 || tokens == 0) return NSV_OK;
  if (!k_new || !v_new || !write_slots || !k_pool || !v_pool) return NSV_ERR_NULLPTR;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(write_slots, 8)) return NSV_ERR_ALIGN;
  DeviceInfo d;
  if ((rc = device_info(&d)) != NSV_OK) return rc;
  KvWriteParams a;
  memset(&a, 0, sizeof a);
  a.k_new = k_new;
  a.v_new = v_new;
  a.write_slots = write_slots;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.status = d.status;
  a.pool_slots = (shape->num_blocks + 1) * (long long)shape->block_size;
  a.rows = (int)tokens;
  a.kv_heads = shape->num_kv_heads;
  a.vec_per_head = shape->head_dim * (shape->dtype == NSV_F32 ? 4 : 2) / 16;
  a.block_size = shape->block_size;
  return chunk_impl(shape, scores, tokens, q, k_pool, v_pool, block_tables, chunk_starts,
                    context_lens, scale, out, workspace, workspace_bytes, stream, &a);
}

}  // extern "C"
