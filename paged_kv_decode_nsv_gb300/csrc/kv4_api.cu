// Host side of the rotating appends and of the 4-bit cache: argument checks,
// workspace layout, launches.

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "kv4.cuh"

namespace nsv {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Null and alignment checks of one call's arguments.
struct Args {
  bool null = false, misaligned = false;
  void need(const void* p, uintptr_t a) {
    null |= !p;
    misaligned |= !aligned(p, a);
  }
  void may(const void* p, uintptr_t a) { misaligned |= !aligned(p, a); }
  int code() const { return null ? NSV_ERR_NULLPTR : misaligned ? NSV_ERR_ALIGN : NSV_OK; }
};

int check_tokens(const nsv_shape* s, int64_t tokens) {
  const int rc = check_shape(s);
  if (rc) return rc;
  return tokens < 0 || tokens >= kMaxTokens ? NSV_ERR_SHAPE : NSV_OK;
}

// A token's stride in elements: 0 stands for `heads` contiguous heads.  False for one
// that lets tokens overlap or takes their vectors off 16 bytes.
bool stride_of(const nsv_shape* s, int64_t given, int heads, long long* stride) {
  const int64_t least = (int64_t)heads * s->head_dim;
  *stride = given ? given : least;
  return *stride >= least && *stride % (s->dtype == NSV_F32 ? 4 : 8) == 0 &&
         *stride < (int64_t(1) << 31);
}

// Checks of an append's arguments; on NSV_OK `p` holds its parameters.  `nothing`:
// there is nothing to do.
int append_params(const nsv_shape* s, const nsv_rope* rope, int64_t tokens, const void* q,
                  const void* k_new, const void* v_new, int64_t q_stride, int64_t k_stride,
                  int64_t v_stride, const int64_t* write_slots, const float* k_scales,
                  const float* v_scales, void* k_pool, void* v_pool, void* q_out,
                  bool rope_needed, RopeParams* p, bool* nothing) {
  int rc = check_tokens(s, tokens);
  if (rc) return rc;
  memset(p, 0, sizeof *p);
  *nothing = tokens == 0;
  if (*nothing) return NSV_OK;
  Args a;
  a.need(k_new, 16), a.need(v_new, 16), a.need(write_slots, 8);
  a.need(k_pool, 16), a.need(v_pool, 16);
  a.may(k_scales, 4), a.may(v_scales, 4);
  if (rope) {
    a.need(rope->positions, 4), a.need(rope->table, 16);
  } else if (rope_needed) {
    return NSV_ERR_NULLPTR;
  }
  if (q || q_out) a.need(q, 16), a.need(q_out, 16);
  if ((rc = a.code()) != NSV_OK) return rc;
  if (q && !rope) return NSV_ERR_RANGE;  // queries are only ever rotated
  if (rope && (rope->rotary_dim < 16 || rope->rotary_dim > s->head_dim ||
               rope->rotary_dim % 16 != 0 || rope->num_positions < 1 ||
               (rope->interleaved != 0 && rope->interleaved != 1)))
    return NSV_ERR_RANGE;
  if (!stride_of(s, q_stride, s->num_heads, &p->q_stride) ||
      !stride_of(s, k_stride, s->num_kv_heads, &p->k_stride) ||
      !stride_of(s, v_stride, s->num_kv_heads, &p->v_stride))
    return NSV_ERR_SHAPE;
  // (a warp for 8 or 16 of a token's heads, two in a CTA; a grid holds 2^31 - 1 CTAs)
  if (tokens * ((int64_t)s->num_heads + 2 * (int64_t)s->num_kv_heads) >= (int64_t(1) << 33))
    return NSV_ERR_SHAPE;
  DeviceInfo d;
  if ((rc = device_info(&d)) != NSV_OK) return rc;
  p->q = q;
  p->k = k_new;
  p->v = v_new;
  if (rope) {
    p->positions = rope->positions;
    p->rotary = rope->table;
    p->num_positions = rope->num_positions;
    p->rotary_dim = rope->rotary_dim;
    p->interleaved = rope->interleaved;
  }
  p->write_slots = write_slots;
  p->k_scales = k_scales;
  p->v_scales = v_scales;
  p->q_out = q_out;
  p->k_pool = k_pool;
  p->v_pool = v_pool;
  p->status = d.status;
  p->tokens = tokens;
  p->pool_slots = (s->num_blocks + 1) * (long long)s->block_size;
  p->heads = s->num_heads;
  p->kv_heads = s->num_kv_heads;
  return NSV_OK;
}

// ------------------------------------------------------------------ attention

// How the vector form takes a shape: column tiles of 8 query vectors, the tokens of a
// tile, the parts that a KV head's query heads are taken in, and its workers.
struct VecForm {
  int col_tiles, tile_tokens, subs, heads_per_worker, workers_per_cta, workers;
};

VecForm vec_form(const nsv_shape* s, int col_tiles, int64_t tokens, int num_sms) {
  VecForm f;
  const int group = s->num_heads / s->num_kv_heads;
  f.col_tiles = col_tiles;
  const int vecs = 8 * col_tiles;
  f.subs = (group + vecs - 1) / vecs;
  f.tile_tokens = std::max(1, vecs / group);
  if (s->query_len > 0) f.tile_tokens = std::min(f.tile_tokens, (int)s->query_len);
  const int warps = kVecWarps;
  f.heads_per_worker = 1;
  for (int h = 2; h <= warps; ++h)
    if (s->num_kv_heads % h == 0) f.heads_per_worker = h;
  f.workers_per_cta = warps / f.heads_per_worker;
  f.workers = num_sms * kv4_vec_ctas_per_sm(s->dtype, col_tiles) * f.workers_per_cta;
  // (few tiles: pieces that are too many take longer to join than they save)
  const int64_t tiles = std::min(tokens, s->rows + tokens / f.tile_tokens);
  const int64_t most = tiles * (s->num_kv_heads / f.heads_per_worker) * f.subs * kVecMostPieces;
  f.workers = (int)std::max<int64_t>(1, std::min<int64_t>(f.workers, most));
  return f;
}

// fp32 takes one column tile (its operands are two parts each).  bf16 takes two where a
// KV head has more than 8 query heads or the caller says that rows bring more than 8 query
// vectors; where it does not say, most rows bring one token (a 509-token chunk among 32
// single tokens, 4 vectors each: 134 us with two column tiles, 131 with one).
int col_tiles_for(const nsv_shape* s) {
  if (s->dtype == NSV_F32) return 1;
  return s->num_heads / s->num_kv_heads * std::max(1, s->query_len) <= 8 ? 1 : 2;
}

struct VecWs {
  uint64_t off_prefix, off_tiles, off_cta, off_todo, off_ml, off_acc, total;
  int max_tiles;
};

VecWs vec_ws(const nsv_shape* s, const VecForm& f, int64_t tokens) {
  auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
  VecWs W;
  W.max_tiles = (int)(s->rows + tokens / f.tile_tokens);
  const uint64_t states = (uint64_t)f.workers * 2 * f.heads_per_worker * 8 * f.col_tiles;
  W.off_prefix = 256;
  W.off_tiles = W.off_prefix + up((uint64_t)(W.max_tiles + 1) * 8);
  W.off_cta = W.off_tiles + up((uint64_t)W.max_tiles * 32);
  W.off_todo = W.off_cta + up((uint64_t)f.workers * 24);
  W.off_ml = W.off_todo + up((uint64_t)f.workers * 16);
  W.off_acc = W.off_ml + up(states * 8);
  W.total = W.off_acc + states * s->head_dim * 4;
  return W;
}

// Most new tokens of a row that the vector form takes; rows that bring more go to the
// forms for many rows (chunk_bf16.cu, chunk_f32.cu).
int vec_tokens(const nsv_shape* s) {
  return (s->dtype == NSV_F32 ? kVecMostVectorsF32 : kVecMostVectors) /
         (s->num_heads / s->num_kv_heads);
}

ChunkWs tile_ws(const nsv_shape* s, int64_t tokens, int num_sms) {
  return make_chunk_ws(s->rows, tokens, s->num_kv_heads, s->num_heads / s->num_kv_heads,
                       s->head_dim, s->dtype, num_sms);
}

// The converted query vectors and their powers of two (bf16).
uint64_t queries_bytes(const nsv_shape* s, int64_t tokens) {
  if (s->dtype == NSV_F32) return 0;
  return ((uint64_t)tokens * s->num_heads * (s->head_dim * 2 + 4) + 255) / 256 * 256;
}

// The vector form's workspace, then the other form's, then the query vectors it converts.
// A larger batch's serves a smaller one, whichever form that takes.
uint64_t chunk4_ws_bytes(const nsv_shape* s, int64_t tokens, int num_sms) {
  nsv_shape any = *s;
  any.query_len = 0;
  uint64_t most = 0;
  for (int ct = 1; ct <= (s->dtype == NSV_F32 ? 1 : 2); ++ct) {
    nsv_shape one = any;
    one.query_len = 1;  // tiles of a single token: the longest list
    most = std::max({most, vec_ws(&any, vec_form(&any, ct, tokens, num_sms), tokens).total,
                     vec_ws(&one, vec_form(&one, ct, tokens, num_sms), tokens).total});
  }
  return (most + 255) / 256 * 256 + (tile_ws(s, tokens, num_sms).total + 255) / 256 * 256 +
         queries_bytes(s, tokens);
}

// What both forms' plans and kernels share of a call.
struct Call {
  const nsv_shape* s;
  const nsv_scores* sc;
  DeviceInfo d;
  int64_t tokens;
  const void* q;
  const int32_t* block_tables;
  const int32_t* chunk_starts;
  const int32_t* context_lens;
  float scale;
  void* out;
};

void common_params(const Call& a, ChunkParams* c) {
  const nsv_shape* s = a.s;
  c->q = a.q;
  c->block_tables = a.block_tables;
  c->chunk_starts = a.chunk_starts;
  c->context_lens = a.context_lens;
  c->slopes = a.sc ? a.sc->slopes : nullptr;
  c->see_begin = a.sc ? a.sc->see_begin : nullptr;
  c->see_end = a.sc ? a.sc->see_end : nullptr;
  c->out = a.out;
  c->status = a.d.status;
  c->pool_blocks = s->num_blocks + 1;
  c->tokens = a.tokens;
  c->rows = s->rows;
  c->heads = s->num_heads;
  c->group = s->num_heads / s->num_kv_heads;
  c->max_blocks = s->max_blocks;
  c->qscale = a.scale * 1.4426950408889634f;  // the kernels use exp2
  c->scale = a.scale;
  c->cap = a.sc ? a.sc->softcap : 0.f;
}

void vec_params(const Call& a, const VecForm& f, const VecWs& W, char* b, Kv4VecParams* p) {
  const nsv_shape* s = a.s;
  Chunk4Params& c = p->c;
  common_params(a, &c);
  c.ws_head = reinterpret_cast<long long*>(b);
  c.ws_prefix = reinterpret_cast<long long*>(b + W.off_prefix);
  c.ws_tiles = reinterpret_cast<int4*>(b + W.off_tiles);
  c.ws_cta = reinterpret_cast<int4*>(b + W.off_cta);
  c.ws_first = reinterpret_cast<long long*>(c.ws_cta + f.workers);
  c.kv_heads = s->num_kv_heads / f.heads_per_worker * f.subs;
  c.max_tiles = W.max_tiles;
  c.tile_tokens = f.tile_tokens;
  c.keys = kVecKeys;
  c.grid = f.workers;
  c.n_min = 0;
  c.n_max = vec_tokens(s);
  c.tile_cost = kVecTileCost;
  c.pair_units = c.half_units = 1;
  p->todo = reinterpret_cast<int4*>(b + W.off_todo);
  p->ml = reinterpret_cast<float2*>(b + W.off_ml);
  p->acc = reinterpret_cast<float*>(b + W.off_acc);
  p->kv_heads = s->num_kv_heads;
  p->heads_per_worker = f.heads_per_worker;
  p->workers_per_cta = f.workers_per_cta;
  p->subs = f.subs;
}

bool tile_params(const Call& a, const ChunkWs& W, char* b, const ChunkQueries& q,
                 Chunk4Params* c) {
  const nsv_shape* s = a.s;
  common_params(a, c);
  c->ws_head = reinterpret_cast<long long*>(b);
  c->ws_prefix = reinterpret_cast<long long*>(b + W.off_prefix);
  c->ws_tiles = reinterpret_cast<int4*>(b + W.off_tiles);
  c->ws_cta = reinterpret_cast<int4*>(b + W.off_cta);
  c->ws_cnt = reinterpret_cast<int32_t*>(b + W.off_cnt);
  c->ws_ml = reinterpret_cast<float2*>(b + W.off_ml);
  c->ws_acc = reinterpret_cast<float*>(b + W.off_acc);
  c->kv_heads = s->num_kv_heads;
  c->max_tiles = W.max_tiles;
  c->tile_rows = W.tile_rows;
  c->tile_tokens = chunk_tile_tokens(s->dtype, c->group);
  const bool f32 = s->dtype == NSV_F32;
  c->keys = f32 ? kChunkKeysF32 : kChunkKeys;
  c->grid = a.d.num_sms;  // one CTA per SM: it takes all the tensor memory
  c->n_min = vec_tokens(s) + 1;
  c->n_max = 0x7fffffff;
  c->tile_cost = f32 ? kChunkTileCostF32 : kChunkTileCost;
  c->pair_units = f32 ? 1 : kChunkPairUnits;
  c->half_units = f32 ? 1 : kChunkHalfUnits;
  c->ws_first = reinterpret_cast<long long*>(c->ws_cta + c->grid);
  if (f32) return true;
  c->q_up = q.up;
  return chunk_encode_q(a.d, s, a.tokens, kChunkHalfRows, q.half, &c->tmap_q[0]) &&
         chunk_encode_q(a.d, s, a.tokens, kChunkHalfRows / 2, q.half, &c->tmap_q[1]) &&
         chunk_encode_q(a.d, s, a.tokens, kChunkHalfRows / 4, q.half, &c->tmap_q[2]);
}

}  // namespace
}  // namespace nsv

using namespace nsv;

extern "C" {

NSV_API int nsv_rope_write(const nsv_shape* shape, const nsv_rope* rope, int64_t tokens,
                           const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int64_t* write_slots,
                           void* k_pool, void* v_pool, void* q_out, cudaStream_t stream) {
  RopeParams p;
  bool nothing;
  const int rc = append_params(shape, rope, tokens, q, k_new, v_new, q_stride, k_stride, v_stride,
                               write_slots, nullptr, nullptr, k_pool, v_pool, q_out, true, &p,
                               &nothing);
  if (rc || nothing) return rc;
  return launch_rope_write(p, shape->dtype, shape->head_dim, stream) == cudaSuccess ? NSV_OK
                                                                                     : cuda_fail();
}

NSV_API int nsv_kv4_write(const nsv_shape* shape, const nsv_rope* rope, const float* k_scales,
                          const float* v_scales, int64_t tokens, const void* q, const void* k_new,
                          const void* v_new, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                          const int64_t* write_slots, void* k_pool, void* v_pool, void* q_out,
                          cudaStream_t stream) {
  RopeParams p;
  bool nothing;
  const int rc = append_params(shape, rope, tokens, q, k_new, v_new, q_stride, k_stride, v_stride,
                               write_slots, k_scales, v_scales, k_pool, v_pool, q_out, false, &p,
                               &nothing);
  if (rc || nothing) return rc;
  return launch_kv4_write(p, shape->dtype, shape->head_dim, stream) == cudaSuccess ? NSV_OK
                                                                                    : cuda_fail();
}

NSV_API int nsv_kv4_read(const nsv_shape* shape, const float* k_scales, const float* v_scales,
                         int64_t tokens, const int64_t* slots, const void* k_pool,
                         const void* v_pool, void* k_out, void* v_out, cudaStream_t stream) {
  int rc = check_tokens(shape, tokens);
  if (rc) return rc;
  if (tokens == 0) return NSV_OK;
  Args a;
  a.need(slots, 8), a.need(k_pool, 16), a.need(v_pool, 16), a.need(k_out, 16), a.need(v_out, 16);
  a.may(k_scales, 4), a.may(v_scales, 4);
  if ((rc = a.code()) != NSV_OK) return rc;
  // (one thread for eight dimensions; a grid holds 2^31 - 1 CTAs)
  if ((tokens * (int64_t)shape->num_kv_heads) >= (int64_t(1) << 34)) return NSV_ERR_SHAPE;
  DeviceInfo d;
  if ((rc = device_info(&d)) != NSV_OK) return rc;
  Kv4ReadParams p;
  p.slots = slots;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = d.status;
  p.tokens = tokens;
  p.pool_slots = (shape->num_blocks + 1) * (long long)shape->block_size;
  p.kv_heads = shape->num_kv_heads;
  return launch_kv4_read(p, shape->dtype, shape->head_dim, stream) == cudaSuccess ? NSV_OK
                                                                                   : cuda_fail();
}

NSV_API int nsv_kv4_workspace(const nsv_shape* shape, int64_t tokens, int num_sms,
                              int64_t* bytes) {
  if (!bytes) return NSV_ERR_NULLPTR;
  int rc = check_tokens(shape, tokens);
  if (rc) return rc;
  if (num_sms <= 0) {
    DeviceInfo d;
    if ((rc = device_info(&d)) != NSV_OK) return rc;
    num_sms = d.num_sms;
  }
  *bytes = (int64_t)chunk4_ws_bytes(shape, tokens, num_sms);
  return NSV_OK;
}

NSV_API int nsv_kv4_chunk(const nsv_shape* s, const nsv_scores* sc, const float* k_scales,
                          const float* v_scales, int64_t tokens, const void* q, const void* k_pool,
                          const void* v_pool, const int32_t* block_tables,
                          const int32_t* chunk_starts, const int32_t* context_lens, float scale,
                          void* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_tokens(s, tokens);
  if (rc) return rc;
  if (s->rows == 0 || tokens == 0) return NSV_OK;
  Args a;
  a.need(q, 16), a.need(k_pool, 16), a.need(v_pool, 16), a.need(block_tables, 4);
  a.need(chunk_starts, 4), a.need(context_lens, 4), a.need(out, 16);
  a.may(k_scales, 4), a.may(v_scales, 4);
  if (sc) a.may(sc->slopes, 4), a.may(sc->see_begin, 4), a.may(sc->see_end, 4);
  if ((rc = a.code()) != NSV_OK) return rc;
  if (sc && sc->softcap != 0.f && !(sc->softcap >= 1e-6f && sc->softcap <= 1e6f))
    return NSV_ERR_RANGE;
  DeviceInfo d;
  if ((rc = device_info(&d)) != NSV_OK) return rc;
  const uint64_t ws_need = chunk4_ws_bytes(s, tokens, d.num_sms);
  if (!ws || ws_bytes < ws_need || !aligned(ws, 256)) return NSV_ERR_WORKSPACE;
  const Call call{s, sc, d, tokens, q, block_tables, chunk_starts, context_lens, scale, out};
  const VecForm f = vec_form(s, col_tiles_for(s), tokens, d.num_sms);
  const VecWs W = vec_ws(s, f, tokens);
  Kv4VecParams p;
  memset(&p, 0, sizeof p);
  vec_params(call, f, W, static_cast<char*>(ws), &p);
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  // Which forms rows of this call can take: both, unless the caller or the number of
  // tokens rules one out.
  const int64_t most = s->query_len > 0 ? s->query_len : tokens;
  const bool vec = vec_tokens(s) > 0, tiles = std::min(most, tokens) > vec_tokens(s);
  Chunk4Params c;
  memset(&c, 0, sizeof c);
  ChunkQueries conv{};
  if (tiles) {
    const ChunkWs T = tile_ws(s, tokens, d.num_sms);
    char* end = static_cast<char*>(ws) + ws_need - queries_bytes(s, tokens);
    if (s->dtype == NSV_BF16) {
      conv.q = q;
      conv.half = end;
      conv.vectors = tokens * s->num_heads;
      conv.up = reinterpret_cast<float*>(end + conv.vectors * s->head_dim * 2);
    }
    if (!tile_params(call, T, end - (T.total + 255) / 256 * 256, conv, &c)) return cuda_fail();
    c.k4 = p.k_pool;
    c.v4 = p.v_pool;
    c.k_units = k_scales;
    c.v_units = v_scales;
  }
  // a row of more tokens than the caller named is read as having none
  if (s->query_len > 0) {
    Chunk4Params& last = tiles ? c : p.c;
    last.n_max = s->query_len;
    last.flag_above = true;
  }
  // Few rows of few tokens need no list, which saves a launch (6 to 8 us of a call).
  if (!tiles && s->query_len > 0) {
    const int n = (s->query_len + f.tile_tokens - 1) / f.tile_tokens;
    if ((int64_t)s->rows * n <= kVecOwnTiles) p.row_tiles = n;
  }
  cudaError_t e = p.row_tiles ? cudaSuccess
                  : !tiles    ? launch_chunk_plan(p.c, stream)
                              : launch_chunk_plans(vec ? &p.c : nullptr, c, conv, s->head_dim,
                                                   d.num_sms, stream);
  if (e == cudaSuccess && tiles)
    e = s->dtype == NSV_F32 ? launch_chunk_kv4_f32(c, s->head_dim, stream)
                            : launch_chunk_kv4(c, s->head_dim, stream);
  if (e == cudaSuccess && vec)
    e = launch_kv4_vec(p, s->dtype, s->head_dim, f.col_tiles, stream);
  return e == cudaSuccess ? NSV_OK : cuda_fail();
}

}  // extern "C"
