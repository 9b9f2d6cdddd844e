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
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "nsv_common.cuh"
#include "sm103.cuh"

namespace nsv {

// bf16: a CTA works on two halves of 128 MMA rows (query tokens x query heads
// of one KV head); keys in runs of 128.  fp32: one set of 64 rows, runs of 64.
constexpr int kChunkHalfRows = 128;
constexpr int kChunkKeys = 128;
constexpr int kChunkRowsF32 = 64;
constexpr int kChunkKeysF32 = 64;

// Query tokens one tile holds.
__host__ __device__ constexpr int chunk_tile_tokens(int dtype, int group) {
  return dtype == NSV_F32 ? (kChunkRowsF32 / group > 0 ? kChunkRowsF32 / group : 1)
                          : 2 * (kChunkHalfRows / group);
}

// Workspace of one chunk attention (offsets are multiples of 256):
//   head    int64 units of one KV head, int64 tiles
//   prefix  int64 [max_tiles + 1]  units before each tile
//   tiles   int4 [max_tiles][2]    {row, first query token (global), tokens,
//           position of the first}, {first key, one past the last key, ctx, 0}
//   cnt     int32 [max_tiles][kv_heads]  pieces of a cut tile that finished
//   ml      float2 [grid][2][tile_rows]  running max (log2 units) and sum
//   acc     float [grid][2][tile_rows][head_dim]
struct ChunkWs {
  uint64_t off_prefix, off_tiles, off_cnt, off_ml, off_acc, total;
  int max_tiles, tile_rows;
};

inline ChunkWs make_chunk_ws(int rows, long long tokens, int kv_heads, int group, int head_dim,
                             int dtype, int grid) {
  ChunkWs W;
  const int tt = chunk_tile_tokens(dtype, group);
  // Every row's last tile may be partial.
  W.max_tiles = (int)(rows + tokens / tt);
  W.tile_rows = (int)(tokens < tt ? tokens : tt) * group;
  // bf16: a tile of few rows leaves up to four partial states per row, of at
  // most 128 rows together
  if (dtype == NSV_BF16) {
    const long long four = 4 * tokens * group;
    const int copies = four < kChunkHalfRows ? (int)four : kChunkHalfRows;
    if (copies > W.tile_rows) W.tile_rows = copies;
  }
  auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
  W.off_prefix = 256;
  W.off_tiles = W.off_prefix + up((uint64_t)(W.max_tiles + 1) * 8);
  W.off_cnt = W.off_tiles + up((uint64_t)W.max_tiles * 32);
  W.off_ml = W.off_cnt + up((uint64_t)W.max_tiles * kv_heads * 4);
  W.off_acc = W.off_ml + up((uint64_t)grid * 2 * W.tile_rows * 8);
  W.total = W.off_acc + (uint64_t)grid * 2 * W.tile_rows * head_dim * 4;
  return W;
}

struct ChunkParams {
  // bf16 only; tmap_q: boxes of 128, 64 and 32 MMA rows
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
  int32_t* ws_cnt;
  float2* ws_ml;
  float* ws_acc;
  uint32_t* status;
  long long pool_blocks;  // num_blocks + 1
  long long tokens;
  int rows, heads, kv_heads, group, max_blocks;
  int max_tiles, tile_rows, tile_tokens, keys;  // keys: positions of one unit
  float qscale;     // scale * log2(e)
  float scale;
  float cap;        // 0: scores are not capped
};

// Launchers.
cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, int grid, cudaStream_t stream);
cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, int grid, cudaStream_t stream);
cudaError_t prepare_chunk_bf16();
cudaError_t prepare_chunk_f32();

#ifdef __CUDACC__
// Units of a tile: runs of `keys` positions; one for a tile that sees nothing
// (it writes its zeros).
__device__ __forceinline__ int chunk_units(int kb, int ke, int keys) {
  return ke > kb ? (ke - kb - 1) / keys + 1 : 1;
}

// One tile of the list.
struct ChunkTile {
  int row, q0, n_tok, pos0;  // q0: global index of its first query token
  int kb, ke, ctx;           // key positions [kb, ke); the row's context length
};

// A CTA's run of units of one tile and KV head.
struct ChunkSegment {
  ChunkTile t;
  int head, tile;
  int j0, j1;        // its key runs: positions kb + keys * j
  bool first, last;  // whether it starts and ends the tile
};

// Walks the segments of CTA `c`.  All lanes of a warp call together.
struct ChunkWalk {
  long long u, end, per_head, U;
  int grid, head, tile, ntiles, skip;
  __device__ void init(const ChunkParams& p, int c, int lane) {
    per_head = __ldcg(p.ws_head);
    ntiles = (int)__ldcg(p.ws_head + 1);
    U = per_head * p.kv_heads;
    grid = U < (long long)gridDim.x ? (int)U : (int)gridDim.x;
    u = end = 0;
    head = tile = skip = 0;
    if (c >= grid) return;
    u = (long long)c * U / grid;
    end = (long long)(c + 1) * U / grid;
    head = (int)(u / per_head);
    const long long rem = u - head * per_head;
    // the last tile whose first unit is at most rem, 32 candidates at a time
    int lo = 0, hi = ntiles;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int i = lo + lane * step;
      const bool le = i < hi && __ldcg(p.ws_prefix + i) <= rem;
      const int n = __popc(__ballot_sync(sm::kFull, le));
      lo += (n - 1) * step;
      hi = min(hi, lo + step);
    }
    tile = lo;
    skip = (int)(rem - __ldcg(p.ws_prefix + tile));
  }
  __device__ bool next(const ChunkParams& p, ChunkSegment& s) {
    if (u >= end) return false;
    const int4 a = __ldcg(p.ws_tiles + 2 * (size_t)tile);
    const int4 b = __ldcg(p.ws_tiles + 2 * (size_t)tile + 1);
    s.t.row = a.x;
    s.t.q0 = a.y;
    s.t.n_tok = a.z;
    s.t.pos0 = a.w;
    s.t.kb = b.x;
    s.t.ke = b.y;
    s.t.ctx = b.z;
    s.head = head;
    s.tile = tile;
    const int n = chunk_units(s.t.kb, s.t.ke, p.keys);
    const int left = n - skip;
    const int take = end - u < left ? (int)(end - u) : left;
    s.j0 = skip;
    s.j1 = skip + take;
    s.first = skip == 0;
    s.last = take == left;
    u += take;
    skip = 0;
    if (s.last && ++tile == ntiles) {
      tile = 0;
      ++head;
    }
    return true;
  }
  // CTA that runs unit x (every CTA below `grid` has at least one unit).
  __device__ int cta_of(long long x) const {
    const long long c = ((x + 1) * grid + U - 1) / U - 1;
    return (int)(c < grid - 1 ? c : grid - 1);
  }
};

// First position this row's query sees and one past the last, clipped to the
// context; g: global index of the query token, pos its position.
__device__ __forceinline__ int2 chunk_sees(const ChunkParams& p, long long g, int pos, int ctx) {
  const int b = p.see_begin ? max(0, __ldg(p.see_begin + g)) : 0;
  const int e = min(p.see_end ? __ldg(p.see_end + g) : pos + 1, ctx);
  return make_int2(b, e);
}

// Workspace slot of a cut tile's piece on CTA c: a CTA cuts at most the tile
// that its range starts inside of (slot 0) and the one it starts but does not
// finish (slot 1).
__device__ __forceinline__ int chunk_slot(int c, bool starts_tile) {
  return 2 * c + (starts_tile ? 1 : 0);
}

// Merge of a cut tile by the warps of the CTA whose piece arrived last (nw
// warps, this one w): out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i over
// the pieces i, in their order.  A piece holds `copies` states per row, row after
// row within a copy.  A row that saw nothing in any piece gives 0.
//
// The states were just written by other SMs, so every load is an L2 round trip
// (about 0.4 us) and what counts is how many are in flight: a warp takes up to
// 32 consecutive rows, finds all their maxima and sums at once (a group of
// lanes per row, the states dealt out to the lanes), then sums NR rows x NS
// states per round, each row's head_dim values over the 32 lanes.  (One row at a
// time, as first written, took 40 us for a tile of 256 rows.)
struct ChunkMerge {
  const ChunkParams& p;
  const ChunkSegment& s;
  int c0, n, rows, shift;
  // workspace row of state i of tile row r
  __device__ __forceinline__ size_t at(int i, int r) const {
    const int c = c0 + (i >> shift);
    return (size_t)chunk_slot(c, c == c0) * p.tile_rows + (i & ((1 << shift) - 1)) * rows + r;
  }
};

// Rows r0 .. r0 + count - 1, whose maxima and inverse sums lane k * group holds
// for row r0 + k.
template <typename T, int D, int NR, int NS>
__device__ __forceinline__ void chunk_merge_rows(const ChunkMerge& m, int r0, int count, int group,
                                                 float M, float inv, int lane) {
  constexpr int kPer = D / 32;
  const ChunkParams& p = m.p;
  for (int k0 = 0; k0 < count; k0 += NR) {
    float a[NR][kPer], Mk[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      Mk[k] = __shfl_sync(sm::kFull, M, min(k0 + k, count - 1) * group);
#pragma unroll
      for (int e = 0; e < kPer; ++e) a[k][e] = 0.f;
    }
    for (int b = 0; b < m.n; b += NS) {
      float x[NR][NS][kPer], wt[NR][NS];
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const size_t at = m.at(min(b + i, m.n - 1), r0 + min(k0 + k, count - 1));
          wt[k][i] = __ldcg(p.ws_ml + at).x;
          const float* src = p.ws_acc + at * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            x[k][i][0] = v.x, x[k][i][1] = v.y, x[k][i][2] = v.z, x[k][i][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            x[k][i][0] = v.x, x[k][i][1] = v.y;
          }
        }
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          // (a state that saw nothing may hold anything)
          const float w =
              (b + i >= m.n || wt[k][i] == -INFINITY) ? 0.f : exp2f(wt[k][i] - Mk[k]);
          if (w != 0.f)
#pragma unroll
            for (int e = 0; e < kPer; ++e) a[k][e] = fmaf(w, x[k][i][e], a[k][e]);
        }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const float iv = __shfl_sync(sm::kFull, inv, min(k0 + k, count - 1) * group);
      if (k0 + k >= count) continue;
      const int r = r0 + k0 + k, tok = r / p.group, g = r - tok * p.group;
      T* o = static_cast<T*>(p.out) +
             (((size_t)m.s.t.q0 + tok) * p.heads + m.s.head * p.group + g) * D + lane * kPer;
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
          *reinterpret_cast<float2*>(o + e) = make_float2(a[k][e] * iv, a[k][e + 1] * iv);
      } else {
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
          *reinterpret_cast<uint32_t*>(o + e) = sm::pack_bf16(a[k][e] * iv, a[k][e + 1] * iv);
      }
    }
  }
}

template <typename T, int D>
__device__ __noinline__ void chunk_merge(const ChunkParams& p, const ChunkWalk& wk,
                                         const ChunkSegment& s, int copies, int w, int nw,
                                         int lane) {
  const long long u0 = s.head * wk.per_head + __ldcg(p.ws_prefix + s.tile);
  const long long u1 = s.head * wk.per_head + __ldcg(p.ws_prefix + s.tile + 1);
  const int c0 = wk.cta_of(u0), c1 = wk.cta_of(u1 - 1);
  const ChunkMerge m{p, s, c0, (c1 - c0 + 1) * copies, s.t.n_tok * p.group,
                     copies == 4 ? 2 : copies == 2 ? 1 : 0};
  const int per = min(32, (m.rows + nw - 1) / nw);  // rows of a warp at a time
  int group = 32;                                    // lanes per row
  while (group * per > 32) group >>= 1;
  for (int r0 = w * per; r0 < m.rows; r0 += nw * per) {
    const int count = min(per, m.rows - r0);
    const int r = r0 + min(lane / group, count - 1);
    float M = -INFINITY, L = 0.f;
    for (int i = lane % group; i < m.n; i += group) {
      const float2 ml = __ldcg(p.ws_ml + m.at(i, r));
      if (ml.x == -INFINITY) continue;
      const float mn = fmaxf(M, ml.x);
      L = L * exp2f(M - mn) + ml.y * exp2f(ml.x - mn);
      M = mn;
    }
    for (int o = 1; o < group; o <<= 1) {
      const float Mo = __shfl_xor_sync(sm::kFull, M, o), Lo = __shfl_xor_sync(sm::kFull, L, o);
      const float mn = fmaxf(M, Mo);
      if (mn != -INFINITY) {
        L = (M == -INFINITY ? 0.f : L * exp2f(M - mn)) + (Mo == -INFINITY ? 0.f : Lo * exp2f(Mo - mn));
        M = mn;
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    if (count >= 4)
      chunk_merge_rows<T, D, 8, 2>(m, r0, count, group, M, inv, lane);
    else
      chunk_merge_rows<T, D, 1, 8>(m, r0, count, group, M, inv, lane);
  }
}

// Pieces of a cut tile.
__device__ __forceinline__ int chunk_pieces(const ChunkParams& p, const ChunkWalk& wk,
                                            const ChunkSegment& s) {
  const long long u0 = s.head * wk.per_head + __ldcg(p.ws_prefix + s.tile);
  const long long u1 = s.head * wk.per_head + __ldcg(p.ws_prefix + s.tile + 1);
  return wk.cta_of(u1 - 1) - wk.cta_of(u0) + 1;
}
#endif  // __CUDACC__

}  // namespace nsv
