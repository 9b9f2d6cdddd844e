// Internal declarations of the chunk attention (nsv_paged_chunk): parameters,
// workspace layout, the tile list that the planning kernel writes and the
// attention kernels walk, and the merge of tiles that were cut between CTAs.
//
// Work is cut into units: one tile of query tokens of one row, one KV head,
// one run of key positions (128 for bf16, 64 for fp32).  The planning kernel
// lists the tiles with their key ranges, because lengths live in device
// memory; the units of all tiles, KV head after KV head, are laid end to end
// and CTA c of a persistent grid takes [c*U/grid, (c+1)*U/grid).  So every
// CTA gets the same number of units whatever the mix of chunk and context
// lengths, and one long row with few query tokens is split over many CTAs.
//
// What the shares count is time: a bf16 run takes 4 units where the tile fills
// both halves and 3 where it fills one (measured 1.9 and 1.45 us), and what a
// tile costs besides its runs (its query rows, its output) as much as two runs,
// before the first.  Counting runs alone, CTAs that got many short tiles ended
// last.  No cost suits all mixes: prompts would have more, batches of single tokens
// less.  Times in us at costs of 0, 1, 2 and 4 runs (fp32: 0, 1, 2 and 3):
//   bf16  2048-token prompt, 32 heads over 8             73    -   56   57
//         5000-token prompt, 12 heads over 4, D 128     117  107   96   94
//         100 single tokens over 100 to 3000 positions  117  109  111  117
//         64 x 5 tokens over 300 to 4000 positions      104  102  105  107
//   fp32  2048-token prompt, 16 heads over 4, D 128     168  135  127  127
//         5000-token prompt, 12 heads over 4, D 128     516  470  428  421
//         638 tokens over up to 2048 positions           76   74   74   74
//         the same causal and capped, D 64               86   82   90   90
//         100 single tokens over 100 to 3000 positions  332  320  324  326
//         26 x 3 tokens over 22 to 7988 positions         -  356  373    -
// fp32 stays at one, because what prompts would gain by two other mixes would lose.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "nsv_common.cuh"
#include "sm103.cuh"

namespace nsv {

// bf16: a CTA works on two halves of 128 MMA rows (query tokens x query heads
// of one KV head); keys in runs of 128.  fp32: one set of 128 rows, runs of 64.
constexpr int kChunkHalfRows = 128;
constexpr int kChunkKeys = 128;
constexpr int kChunkRowsF32 = 128;
constexpr int kChunkKeysF32 = 64;

// Costs (see above): of a bf16 tile in runs, of its runs in units.
constexpr int kChunkTileCost = 2, kChunkPairUnits = 4, kChunkHalfUnits = 3;
constexpr int kChunkTileCostF32 = 1;
// Where there is a CTA for every tile and head, and no tile has more runs than
// this, each CTA gets one whole, which saves publishing and merging the pieces of cut
// tiles.  How many runs are worth that depends on how many CTAs would be left idle.
// Single tokens of 4 heads per KV head, D 128, in us with the tiles cut and whole:
//                        2 runs       4 runs       8 runs       16 runs
//   bf16  128 tiles    26.6  20.5   28.7  24.6   36.9  32.8   53.2  49.2
//         32 tiles     21.5  18.4   22.5  20.5   24.6  26.7   28.7  36.9
//         1 tile       18.4  16.4   20.5  18.8   20.5  24.6   20.5  34.8
//   fp32  128 tiles    36.9  26.6   41.0  32.8   53.2  45.1   75.8  69.6
//         32 tiles     26.6  24.6   30.7  30.7   30.7  43.0   36.9  65.5
//         1 tile       26.6  24.6   26.6  30.7   26.6  41.0   26.7  61.5
// Eight takes what many tiles gain (up to 8 us) and costs few long ones about as much in
// bf16 (4 us) and more in fp32 (14 us at 8 runs).
constexpr int kChunkWholeRuns = 8;

// Query tokens one tile holds.
__host__ __device__ constexpr int chunk_tile_tokens(int dtype, int group) {
  return dtype == NSV_F32 ? kChunkRowsF32 / group : 2 * (kChunkHalfRows / group);
}

// Workspace of one chunk attention (offsets are multiples of 256):
//   head    int64 units of one KV head, int64 tiles
//   prefix  int64 [max_tiles + 1]  units before each tile
//   tiles   int4 [max_tiles][2]    {row, first query token (global), tokens,
//           position of the first}, {first key, one past the last key, ctx,
//           units of a run}
//   cta     int4 [grid]  where each CTA starts: {units, KV head, tile, units of
//           the tile before}, and int64 [grid] its first unit
//   cnt     int32 [max_tiles][kv_heads]  pieces of a cut tile that finished
//   ml      float2 [grid][2][tile_rows]  running max (log2 units) and sum
//   acc     float4 [grid][2][head_dim / 4][tile_rows]  unnormalised outputs; the
//           rows are innermost, because a warp's lanes hold consecutive rows
struct ChunkWs {
  uint64_t off_prefix, off_tiles, off_cta, off_cnt, off_ml, off_acc, total;
  int max_tiles, tile_rows;
};

inline ChunkWs make_chunk_ws(int rows, long long tokens, int kv_heads, int group, int head_dim,
                             int dtype, int grid) {
  ChunkWs W;
  const int tt = chunk_tile_tokens(dtype, group);
  // Every row's last tile may be partial.
  W.max_tiles = (int)(rows + tokens / tt);
  W.tile_rows = (int)(tokens < tt ? tokens : tt) * group;
  auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
  W.off_prefix = 256;
  W.off_tiles = W.off_prefix + up((uint64_t)(W.max_tiles + 1) * 8);
  W.off_cta = W.off_tiles + up((uint64_t)W.max_tiles * 32);
  W.off_cnt = W.off_cta + up((uint64_t)grid * 24);
  W.off_ml = W.off_cnt + up((uint64_t)W.max_tiles * kv_heads * 4);
  W.off_acc = W.off_ml + up((uint64_t)grid * 2 * W.tile_rows * 8);
  W.total = W.off_acc + (uint64_t)grid * 2 * W.tile_rows * head_dim * 4;
  return W;
}

struct ChunkParams {
  // bf16 only; tmap_q: boxes of 128, 64 and 32 MMA rows.  (First: behind other fields they
  // cross 128-byte lines, which costs a call half a microsecond.)
  CUtensorMap tmap_q[3], tmap_k, tmap_v;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_tables;
  const int32_t* chunk_starts;
  const int32_t* context_lens;
  const float* slopes;       // [heads] or null
  const int32_t* see_begin;  // [tokens] or null
  const int32_t* see_end;    // [tokens] or null
  void* out;
  long long* ws_head;
  long long* ws_prefix;
  int4* ws_tiles;
  int4* ws_cta;
  long long* ws_first;
  int32_t* ws_cnt;  // null where a kernel of its own merges (kv4_vec.cu)
  float2* ws_ml;
  float* ws_acc;
  uint32_t* status;
  long long pool_blocks;  // num_blocks + 1
  long long tokens;
  int rows, heads, kv_heads, group, max_blocks;
  int max_tiles, tile_rows, tile_tokens, keys;  // keys: positions of one unit
  int grid;         // CTAs of the attention kernel
  int tile_cost;    // a tile's own cost, in runs
  int pair_units, half_units;  // units of a run of a tile that fills both halves, or one
  float qscale;     // scale * log2(e)
  float scale;
  float cap;        // 0: scores are not capped
};

// Over a 4-bit cache (kv4.cuh).  (Not among the parameters above, which every call over a
// bf16 or fp32 cache passes: there they cost a 2048-token prompt over a bf16 cache 56.0 us in
// place of 55.5 on one GPU, and nothing on another.)
struct Chunk4Params : ChunkParams {
  int n_min, n_max; // rows that bring fewer or more tokens have no tiles
  bool flag_above;  // more than n_max is an error (NSV_DEV_BAD_CHUNK)
  // its pools, and the fp32 scales of its KV heads or null
  const uint8_t* k4;
  const uint8_t* v4;
  const float* k_units;
  const float* v_units;
  const float* q_up;  // [tokens][heads]: what the converted query vectors are scaled down by
};
template <bool KV4>
using ChunkArgs = std::conditional_t<KV4, Chunk4Params, ChunkParams>;

// A tensor map of the query tokens for boxes of `rows` MMA rows (chunk_api.cu).
bool chunk_encode_q(const DeviceInfo& d, const nsv_shape* s, int64_t tokens, int rows,
                    const void* q, CUtensorMap* map);

// Launchers.
cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_plan(const Chunk4Params& p, cudaStream_t stream);
// The tile lists of two kernels that share a batch (a: null for one alone), and b's query
// vectors converted to fp16 on the way, in one launch.
struct ChunkQueries {
  const void* q;  // bf16 [vectors][head_dim]
  void* half;     // the same, each scaled by a power of two so that its largest element
                  // lies in [2^14, 2^15)
  float* up;      // [vectors] the inverse powers
  long long vectors;
};
cudaError_t launch_chunk_plans(const Chunk4Params* a, const Chunk4Params& b,
                               const ChunkQueries& q, int head_dim, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, cudaStream_t stream);
// The same over a 4-bit cache (k4, v4).
cudaError_t launch_chunk_kv4(const Chunk4Params& p, int head_dim, cudaStream_t stream);
cudaError_t launch_chunk_kv4_f32(const Chunk4Params& p, int head_dim, cudaStream_t stream);
cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t stream);
cudaError_t prepare_chunk_bf16();
cudaError_t prepare_chunk_f32();

#ifdef __CUDACC__
// Runs of `keys` positions of a tile; one for a tile that sees nothing (it
// writes its zeros).
__device__ __forceinline__ int chunk_runs(int kb, int ke, int keys) {
  return ke > kb ? (int)((unsigned)(ke - kb - 1) / (unsigned)keys) + 1 : 1;
}

// One tile of the list.
struct ChunkTile {
  int row, q0, n_tok, pos0;  // q0: global index of its first query token
  int kb, ke, ctx;           // key positions [kb, ke); the row's context length
  int cost;                  // units of one of its runs: 1, 3 or 4
};

// x / cost, rounded up, for x >= 0; 0 below.
__device__ __forceinline__ int chunk_ceil(int x, int cost) {
  const unsigned y = (unsigned)max(0, x + cost - 1);
  return (int)(cost == 3 ? y / 3u : y >> (cost >> 1));
}

// A CTA's run of units of one tile and KV head.
struct ChunkSegment {
  ChunkTile t;
  int head, tile;
  int j0, j1;        // its key runs: positions kb + keys * j
  bool first, last;  // whether it starts and ends the tile
};

// The CTAs whose pieces make up a segment's tile: the first one, and how many.
// A run belongs to the CTA whose share holds its first unit.  All lanes of a
// warp call together.
template <int KEYS>
__device__ __forceinline__ int2 chunk_pieces(const ChunkParams& p, const ChunkSegment& s,
                                             int lane) {
  const long long u0 =
      s.head * __ldcg(p.ws_head) + __ldcg(p.ws_prefix + s.tile) + p.tile_cost * s.t.cost;
  const long long u1 = u0 + (long long)(chunk_runs(s.t.kb, s.t.ke, KEYS) - 1) * s.t.cost;
  int before = 0, upto = 0;  // CTAs that start at or before the first run, the last one
#pragma unroll 1
  for (int c = 0; c < p.grid; c += 32) {
    const long long f = c + lane < p.grid ? __ldcg(p.ws_first + c + lane) : u1 + 1;
    before += __popc(__ballot_sync(sm::kFull, f <= u0));
    upto += __popc(__ballot_sync(sm::kFull, f <= u1));
  }
  return make_int2(before - 1, upto - before + 1);
}

// Walks the segments of CTA `c`.  (Kept to a few registers: what the attention
// kernel spills it reads back from L2, because shared memory leaves the L1 cache
// next to nothing.)
struct ChunkWalk {
  int left, head, tile, ntiles, skip;  // units left; where the next segment starts
  __device__ void init(const ChunkParams& p, int c) {
    const int4 at = __ldcg(p.ws_cta + c);
    ntiles = (int)__ldcg(p.ws_head + 1);
    left = at.x;
    head = at.y;
    tile = at.z;
    skip = at.w;
  }
  template <int KEYS>
  __device__ __forceinline__ bool next(const ChunkParams& p, ChunkSegment& s) {
    while (left > 0) {
      const int4 a = __ldcg(p.ws_tiles + 2 * (size_t)tile);
      const int4 b = __ldcg(p.ws_tiles + 2 * (size_t)tile + 1);
      const int own = p.tile_cost * b.w;
      const int runs = chunk_runs(b.x, b.y, KEYS);
      const int of_tile = own + runs * b.w - skip;
      const int take = min(left, of_tile);
      s.j0 = chunk_ceil(skip - own, b.w);
      s.j1 = chunk_ceil(skip + take - own, b.w);
      s.first = s.j0 == 0;
      s.last = s.j1 == runs;
      s.head = head;
      s.tile = tile;
      left -= take;
      skip = 0;
      if (take == of_tile && ++tile == ntiles) {
        tile = 0;
        ++head;
      }
      if (s.j0 == s.j1) continue;  // no run starts in the share
      s.t.row = a.x;
      s.t.q0 = a.y;
      s.t.n_tok = a.z;
      s.t.pos0 = a.w;
      s.t.kb = b.x;
      s.t.ke = b.y;
      s.t.ctx = b.z;
      s.t.cost = b.w;
      return true;
    }
    return false;
  }
};

// First position this row's query sees and one past the last, at most the context,
// and neither below 0 (the kernels subtract positions from them in 32 bits, which
// bounds near INT_MIN would wrap); g: global index of the query token, pos its
// position.
__device__ __forceinline__ int2 chunk_sees(const ChunkParams& p, long long g, int pos, int ctx) {
  const int b = p.see_begin ? max(0, __ldg(p.see_begin + g)) : 0;
  const int e = min(p.see_end ? __ldg(p.see_end + g) : pos + 1, ctx);
  return make_int2(b, max(e, 0));
}

// A row's new tokens and context length; none and 0 where they are bad.
struct RowChunk {
  int start, n, ctx;
};

template <typename P>
__device__ __forceinline__ RowChunk row_chunk(const P& p, int r, bool flag) {
  const int a = __ldg(p.chunk_starts + r), b = __ldg(p.chunk_starts + r + 1);
  RowChunk c{a, b - a, __ldg(p.context_lens + r)};
  if (a < 0 || b < a || b > p.tokens) {
    c.n = 0;
    if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_CHUNK);
  }
  if constexpr (std::is_same_v<P, Chunk4Params>) {
    if (c.n < p.n_min || c.n > p.n_max) {
      if (flag && p.flag_above && c.n > p.n_max) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_CHUNK);
      c.n = 0;
    }
  }
  if (c.ctx < 0 || (long long)c.ctx > (long long)p.max_blocks * kBlock) {
    c.ctx = 0;
    if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_CTX);
  }
  return c;
}

// The scales of a KV head's keys and values.
__device__ __forceinline__ float k_unit(const ChunkParams&, int) { return 1.f; }
__device__ __forceinline__ float v_unit(const ChunkParams&, int) { return 1.f; }
__device__ __forceinline__ float k_unit(const Chunk4Params& p, int head) {
  return p.k_units ? __ldg(p.k_units + head) : 1.f;
}
__device__ __forceinline__ float v_unit(const Chunk4Params& p, int head) {
  return p.v_units ? __ldg(p.v_units + head) : 1.f;
}

// Workspace slot of a cut tile's piece on CTA c: a CTA cuts at most the tile
// that its range starts inside of (slot 0) and the one it starts but does not
// finish (slot 1).
__device__ __forceinline__ int chunk_slot(int c, bool starts_tile) {
  return 2 * c + (starts_tile ? 1 : 0);
}

// A row's four output values at columns 4 v .. of one workspace slot.
__device__ __forceinline__ float4* chunk_acc(const ChunkParams& p, int slot, int head_dim, int v,
                                             int row) {
  return reinterpret_cast<float4*>(p.ws_acc) +
         ((size_t)slot * (head_dim / 4) + v) * p.tile_rows + row;
}

// Where a tile's row goes in `out`.
template <typename T>
__device__ __forceinline__ T* chunk_out(const ChunkParams& p, int q0, int head, int row,
                                        int head_dim) {
  const int tok = row / p.group, g = row - tok * p.group;
  return static_cast<T*>(p.out) + (((size_t)q0 + tok) * p.heads + head * p.group + g) * head_dim;
}

// Merge of a cut tile by the NT threads of the CTA whose piece arrived last:
// out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i over the n pieces i, of
// CTAs c0, c0 + 1, ..., in this order.  A row that saw nothing in any piece gives 0.
//
// A warp takes 8 rows and 4 column groups (of 4) at a time, so that both its loads
// (whole 128-byte lines of consecutive rows) and its stores (32 or 64 bytes of a
// row) are few lines; where there are few rows the warps share their columns.
// The pieces were just written by other SMs, a load is an L2 round trip (0.5 to
// 1 us), and a round has the states of NS pieces and NG x NS of their columns in
// flight: 8 loads of 16 bytes a thread, for as many columns of a piece as the warp has.
// With four columns of two pieces, or two of four, instead: a 509-token chunk among 32
// decodes 125 and 129 us (121), a 5000-token prompt 97 and 102 (95), 1000 tokens over
// 16000 positions 82 and 88 (80), fp32 336 and 326 (324), 100 single tokens in fp32 339 and
// 319 (321); short prompts the same.
template <typename T, int D, int NG, int NS>
__device__ __forceinline__ void chunk_merge_cols(const ChunkParams& p, int c0, int n, int row,
                                                 bool valid, int g0, int step, int quad, T* out) {
#pragma unroll 1
  for (int g = g0; g < D / 16; g += NG * step) {
    float M = -INFINITY, L = 0.f;
    float4 a[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int b = 0; b < n; b += NS) {
      float4 x[NG][NS];
      float2 ml[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int j = min(b + i, n - 1), slot = chunk_slot(c0 + j, j == 0);
        ml[i] = __ldcg(p.ws_ml + (size_t)slot * p.tile_rows + row);
#pragma unroll
        for (int k = 0; k < NG; ++k)
          x[k][i] =
              __ldcg(chunk_acc(p, slot, D, 4 * min(g + k * step, D / 16 - 1) + quad, row));
      }
      float mn = M;
#pragma unroll
      for (int i = 0; i < NS; ++i) mn = fmaxf(mn, ml[i].x);
      if (mn == -INFINITY) continue;  // nothing seen so far
      const float keep = exp2f(M - mn);
      M = mn;
      L *= keep;
#pragma unroll
      for (int k = 0; k < NG; ++k) a[k].x *= keep, a[k].y *= keep, a[k].z *= keep, a[k].w *= keep;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (b + i >= n || ml[i].x == -INFINITY) continue;  // such a state may hold anything
        const float w = exp2f(ml[i].x - M);
        L = fmaf(w, ml[i].y, L);
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          a[k].x = fmaf(w, x[k][i].x, a[k].x);
          a[k].y = fmaf(w, x[k][i].y, a[k].y);
          a[k].z = fmaf(w, x[k][i].z, a[k].z);
          a[k].w = fmaf(w, x[k][i].w, a[k].w);
        }
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      if (!valid || g + k * step >= D / 16) continue;
      T* o = out + 16 * (g + k * step) + 4 * quad;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(o) =
            make_float4(a[k].x * inv, a[k].y * inv, a[k].z * inv, a[k].w * inv);
      else
        *reinterpret_cast<uint2*>(o) = make_uint2(sm::pack_bf16(a[k].x * inv, a[k].y * inv),
                                                  sm::pack_bf16(a[k].z * inv, a[k].w * inv));
    }
  }
}

template <typename T, int D, int NT>
__device__ __forceinline__ void chunk_merge(const ChunkParams& p, int q0, int n_tok, int head,
                                            int c0, int n, int tid) {
  const int rows = n_tok * p.group, blocks = (rows + 7) / 8;
  const int lane = tid & 31, quad = lane >> 3;
  int share = 1;  // warps that share 8 rows
  while (2 * share <= D / 16 && 2 * share * blocks <= NT / 32) share *= 2;
#pragma unroll 1
  for (int rb = (tid >> 5) / share; rb < blocks; rb += NT / 32 / share) {
    const int row = min(8 * rb + (lane & 7), rows - 1);
    const bool valid = 8 * rb + (lane & 7) < rows;
    T* out = chunk_out<T>(p, q0, head, row, D);
    const int g0 = (tid >> 5) % share;
    if (D / 16 / share >= 8)
      chunk_merge_cols<T, D, 8, 1>(p, c0, n, row, valid, g0, share, quad, out);
    else if (D / 16 / share >= 4)
      chunk_merge_cols<T, D, 4, 2>(p, c0, n, row, valid, g0, share, quad, out);
    else
      chunk_merge_cols<T, D, 1, 8>(p, c0, n, row, valid, g0, share, quad, out);
  }
}
// What the two warps of a pair share: whose lanes must raise their maximum
// (two runs in turn), and whether one of them has given up.
struct PairWords {
  uint32_t raise[2][2];
  uint32_t failed;
};

// The two warps of a pair meet.  False when the other one has given up a wait
// (it came here on its way out).
__device__ __forceinline__ bool pair_sync(int bar, volatile PairWords* w) {
  asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
  return w->failed == 0;
}

// How a softmax warp ends.
enum : int { kDone = 0, kTimedOut = 1, kPartnerFailed = 2 };


// Once all softmax warps have written a cut tile's piece, counts it; the CTA
// that counts a tile's last piece will merge it (at most two: the tile that its
// range starts inside of and the one it ends inside of, which have a barrier each:
// piece0 and, if the tile starts here, piece1).
template <int KEYS>
__device__ __forceinline__ bool chunk_publish(const ChunkParams& p, uint32_t piece0,
                                              uint32_t piece1, uint32_t published, int4* s_todo,
                                              ChunkWalk wk, int lane) {
  long long runs = 0;  // since the wait before
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<KEYS>(p, s)) {
    runs += s.j1 - s.j0;
    if (s.first && s.last) continue;
    const int2 pc = chunk_pieces<KEYS>(p, s, lane);
    // (this wait lasts as long as all segments since the one before: a limit for
    // each of their runs)
    bool done = false;
#pragma unroll 1
    for (; runs >= 0 && !done; --runs) done = sm::warp_wait(s.first ? piece1 : piece0, 0);
    if (!done) return false;
    runs = 0;
    if (lane == 0) {
      __threadfence();  // (cumulative: what the warps wrote before they arrived)
      if (atomicAdd(p.ws_cnt + (size_t)s.tile * p.kv_heads + s.head, 1) == pc.y - 1) {
        s_todo[s.first ? 2 : 0] = make_int4(s.t.q0, s.t.n_tok, s.head, 0);
        s_todo[s.first ? 3 : 1] = make_int4(pc.x, pc.y, 0, 0);
      }
    }
  }
  __syncwarp();
  if (lane == 0) sm::mbar_arrive(published);
  return true;
}

// The tiles whose last piece was one of this CTA's, merged by its first NT threads
// once all its work is published: a merge within the loops would cost them registers.
template <typename T, int D, int NT>
__device__ __forceinline__ void chunk_merge_todo(const ChunkParams& p, const int4* s_todo) {
  __threadfence();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int4 t = s_todo[2 * k], c = s_todo[2 * k + 1];
    if (t.y) chunk_merge<T, D, NT>(p, t.x, t.y, t.z, c.x, c.y, threadIdx.x);
  }
}
#endif  // __CUDACC__

}  // namespace nsv
