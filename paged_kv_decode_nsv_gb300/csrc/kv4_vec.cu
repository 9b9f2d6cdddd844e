// Attention over a paged 4-bit cache, for tiles of few query vectors (single
// tokens, a few guessed ones): the form that HBM bounds.
//
// For query vector i (a query token and head) of a tile and the positions t it sees:
//   x_t = scale * log2(e) * q_i . k_t   (capped and biased as in chunk_bf16.cu)
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m)
// folded 32 positions at a time with a running maximum m and sum (fp32, of the
// unrounded weights).
//
// A warp works alone: it takes its own share of the units (chunk.cuh; 32 positions,
// two blocks), copies their tiles into its own ring in shared memory by 16-byte
// asynchronous copies, and needs no other warp until the end.  (Four bulk copies a unit
// instead: 165 us against 160 for 256 single tokens: a warp stands still for longer to issue
// them than for nine copies a lane.)  heads_per_worker warps, one per KV head,
// share the same rows and positions, so that the tiles of a block, which lie one
// after the other, are read at about the same time.
//
// Both products run on mma.sync m16n8k16 in fp16 with the cache's side as the 16
// rows and up to 8 query vectors as the columns: the cache's numbers times their
// scales are exact in fp16, and widening them takes most of the instructions, so that
// each is widened once for all vectors.  (tcgen05 would want the widened operands in
// shared memory, written and read again; the vectors are far too few to fill its rows.)
//   scores: rows are tokens, a lane's k indices are dimensions that lie together in
//           its 16 bytes; the query vectors are laid out the same way.
//   output: rows are dimensions, k indices are tokens; the weights change from
//           accumulators to operands by movmatrix.
// MMA row r of the scores and k index r of the output stand for token
// r ^ ((r >> 1) & 1) of a block, which halves the bank conflicts of the values' loads.
//
// Rounding: query vectors are scaled by a power of two, so that their largest element lies in
// [2^14, 2^15).  bf16 ones are then exact in fp16 but for elements below 2^-28 of their
// vector's largest, which are off by 2^-39 of it at most.  Weights are held times 2^kUp, at
// most 2^15, and rounded to fp16: 2^-11 of themselves (the output's rounding to bf16 is 2^-8),
// or 2^-32 of the largest where that is more.
// fp32's queries and weights are the sum of two fp16 numbers, hi + 2^-12 lo, and the products
// with the lower parts are summed apart and scaled down: off by 2^-23 of themselves, below
// 2^-28 of the largest by up to 2^-51 of it.  (Without a power of two of their own the lower
// parts end at 2^-39 of the largest, and what lies below 2^-17 of it loses digits; 256 single
// tokens over 4096 positions take 303 us so, and 312 with it.)
//
// A tile cut between workers leaves partial states; kv4_merge_kernel joins them in the
// order of their positions.
//
// What bounds it: the latency of a warp's unit, widening and MMAs together, at 16 warps on an
// SM (128 registers a thread, of which 40 to 84 bytes are spilled at head_dim 128).  256 single tokens over 512 to 8192 positions, 32 heads, 8 KV heads, head_dim
// 128: 159 us, 5.0 TB/s of the cache's bytes.  The copies alone take 131, the work without them
// 144, each with the 12 us of the launches' start and the merge; a sub-partition issues 0.57
// instructions a cycle, the ALU pipe is 52 % busy and the tensor pipe 21 %.  Scores a unit
// ahead of the values: 173 instead of 167; 20 warps of 96 registers, which spill more: 196.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kv4.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kWarps = kVecWarps;
constexpr int kStages = 3;    // of a warp's ring
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum of a vector that has seen nothing: below all scores, but finite, so
// that its difference to a score has no special cases.
constexpr float kLeast = -3e38f;

template <typename T>
struct Round;
// The running maximum is raised when a score exceeds it by more than kSlack (log2
// units); weights are held times 2^kUp.
template <>
struct Round<__nv_bfloat16> {
  static constexpr int kParts = 1;
  static constexpr float kSlack = 8.f, kUp = 7.f;
};
template <>
struct Round<float> {
  static constexpr int kParts = 2;
  static constexpr float kSlack = 1.f, kUp = 14.f;
};
// The lower parts' own power of two: half a step of the largest upper part, 2^3, times it is
// still in fp16's range.
constexpr float kLowUp = 4096.f, kLowDown = 1.f / 4096.f;
// x - hi, the upper parts' rest, as lower parts.
__device__ __forceinline__ uint32_t lower_parts(float x, float y, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half((x - f.x) * kLowUp, (y - f.y) * kLowUp);
}

template <int D>
struct Ring {
  static constexpr uint32_t kTile = kv4_tile_bytes(D);
  static constexpr uint32_t kStage = 4 * kTile;  // keys of two blocks, values of two blocks
  static constexpr uint32_t kWarp = kStages * kStage;
};

// An asynchronous copy of 16 bytes; the thread's copies so far become a group; a wait for
// all of the thread's groups but the last N.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory by its 32-bit address, as ordinary loads (which barriers order).
template <typename V>
__device__ __forceinline__ V lds(uint32_t a) {
  return *static_cast<const V*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t both(uint32_t h, bool upper) {
  return __byte_perm(h, 0, upper ? 0x3232 : 0x1010);
}

// A warp's segments between the copies, which run ahead, and the work on them: a ring in
// shared memory, because their registers are worth more elsewhere.  A segment has at least
// one unit and copies are kStages units ahead at most, so that no more than kStages + 1
// are open.
constexpr int kSegments = 4;
static_assert(kSegments > kStages, "segments that are open at a time");
struct Segment {
  int q0, n_tok, pos0, ctx;
  int kb, j0, j1, head;
  int whole, first, valid;  // valid: 0 behind the share's last
  long long last;           // the tile's last unit, of all tiles' and groups'
};

constexpr uint32_t kSegmentBytes = kSegments * sizeof(Segment) + 32;  // and a Worker::Own

// A tile as a CTA works it out that has no list: number `tile` of rows times row_tiles.
struct OwnTile {
  int row, q0, n_tok, pos0, kb, ke, ctx, units;  // units 0: there is none
};
__device__ __forceinline__ OwnTile own_tile(const Kv4VecParams& p, int tile, bool flag) {
  OwnTile o;
  o.row = p.row_tiles == 1 ? tile : tile / p.row_tiles;
  const int i = tile - o.row * p.row_tiles, tok0 = i * p.c.tile_tokens;
  const RowChunk c = row_chunk(p.c, o.row, flag && i == 0);
  o.units = 0;
  if (tok0 >= c.n) return o;
  o.q0 = c.start + tok0;
  o.n_tok = min(p.c.tile_tokens, c.n - tok0);
  o.pos0 = c.ctx - c.n + tok0;
  o.ctx = c.ctx;
  o.kb = 0;
  o.ke = max(0, min(o.pos0 + o.n_tok, c.ctx));
  if (p.c.see_begin || p.c.see_end) {
    int kb = 0x7fffffff;
    o.ke = 0;
    for (int t = 0; t < o.n_tok; ++t) {
      const int2 v = chunk_sees(p.c, (long long)o.q0 + t, o.pos0 + t, c.ctx);
      if (v.x < v.y) {
        kb = min(kb, v.x);
        o.ke = max(o.ke, v.y);
      }
    }
    o.kb = kb < o.ke ? kb / kBlock * kBlock : 0;
  }
  o.units = p.c.tile_cost + chunk_runs(o.kb, o.ke, kVecKeys);
  return o;
}

// The units of a CTA's threads' tiles, before each thread's; all of one group of heads.
struct OwnPlan {
  long long units, shares;  // of one group of heads; workers that have any
  long long before[kWarps * 32 + 1];
  long long warp_sum[kWarps];
};
// All threads of the CTA together.
__device__ __forceinline__ void own_plan(const Kv4VecParams& p, OwnPlan* o) {
  const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
  const int tiles = p.c.rows * p.row_tiles;
  const int each = (tiles + blockDim.x - 1) / blockDim.x;
  long long mine = 0;
  for (int i = tid * each; i < min((tid + 1) * each, tiles); ++i)
    mine += own_tile(p, i, blockIdx.x == 0).units;
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long x = __shfl_up_sync(kFull, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) o->warp_sum[tid >> 5] = upto;
  __syncthreads();
  long long base = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < tid >> 5) base += o->warp_sum[w];
    total += o->warp_sum[w];
  }
  o->before[tid] = base + upto - mine;
  if (tid == 0) {
    // (a share is counted in 32 bits)
    if (total > 0x7fffffffll / p.c.kv_heads * p.c.grid) {
      if (blockIdx.x == 0) atomicOr(p.c.status, (uint32_t)NSV_DEV_BAD_CHUNK);
      total = 0;
    }
    o->units = total;
    o->shares = max(1ll, min(total * p.c.kv_heads / kVecLeastUnits, (long long)p.c.grid));
  }
  __syncthreads();
}

template <typename T, int D, int NT, bool CAP, bool BIAS>
struct Worker {
  static constexpr int kParts = Round<T>::kParts;
  static constexpr int kSteps = D / 16;  // k steps of the scores, row tiles of the output
  static constexpr int kVecs = 8 * NT;
  using R = Ring<D>;

  const Kv4VecParams& p;
  int lane, g, t;       // g: MMA row or column, t: its pair
  uint32_t ring;        // its shared-memory address
  Segment* segments;
  int head;             // within a group of heads
  // The copies' side: the walk, what its segment has left, and the ring's next stage.
  ChunkWalk wk;
  struct Own {
    long long unit, all, shares;  // without a list: the next unit; of how many; workers
  };
  volatile Own* own;
  const int32_t* table;
  const uint8_t* pool;  // this lane's part of the segment's KV head's tiles
  int block, block_end, units;  // next block, one past the last that any vector sees
  int ids, ids_from;    // the lane's block id of the 32 from ids_from on
  uint32_t fill, opened;
  uint32_t at;          // the stage that is next to be worked on
  uint32_t missing;     // two bits a stage: blocks that are not there though they should be

  __device__ __forceinline__ Worker(const Kv4VecParams& p_) : p(p_) {}

  // Where the share of worker `w` starts, without a list.
  __device__ __forceinline__ void start(const OwnPlan* o, int w) {
    const long long U = o->units * p.c.kv_heads, n = o->shares;
    wk.left = wk.head = wk.tile = wk.skip = 0;
    wk.ntiles = p.c.rows * p.row_tiles;
    const long long first = w < n ? w * U / n : U;
    if (lane == 0) {
      own->unit = first;
      own->all = U;
      own->shares = n;
    }
    __syncwarp();
    if (first >= U) return;
    wk.left = (int)((w + 1) * U / n - first);
    wk.head = (int)(first / o->units);
    const long long rem = first - wk.head * o->units;
    int lo = 0, hi = blockDim.x;  // the last thread whose first unit is at most rem
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (o->before[mid] <= rem) lo = mid; else hi = mid;
    }
    // of its tiles (at most 13: a CTA has 5 warps or more) the one that holds rem
    const int each = (wk.ntiles + blockDim.x - 1) / blockDim.x, i = lo * each + lane;
    const long long mine = lane < each && i < wk.ntiles ? own_tile(p, i, false).units : 0;
    long long upto = o->before[lo] + mine;
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
      const long long x = __shfl_up_sync(kFull, upto - o->before[lo], d);
      if (lane >= d) upto += x;
    }
    const int at = __ffs(__ballot_sync(kFull, rem < upto)) - 1;
    wk.tile = lo * each + at;
    wk.skip = (int)(rem - __shfl_sync(kFull, upto - mine, at));
  }
  // The next segment without a list.
  __device__ __forceinline__ bool own_next(ChunkSegment& s, long long& last) {
    __syncwarp();
    long long unit = own->unit;
    bool more = false;
    while (!more && wk.left > 0) {
      const OwnTile t = own_tile(p, wk.tile, false);
      const int of_tile = t.units - wk.skip, take = min(wk.left, of_tile);
      s.j0 = max(0, wk.skip - p.c.tile_cost);
      s.j1 = max(0, wk.skip + take - p.c.tile_cost);
      s.first = s.j0 == 0;
      s.last = take == of_tile;
      s.head = wk.head;
      last = unit + of_tile - 1;
      wk.left -= take;
      unit += take;
      wk.skip = 0;
      if (take == of_tile && ++wk.tile == wk.ntiles) {
        wk.tile = 0;
        ++wk.head;
      }
      more = s.j0 != s.j1;  // (else none of the tile, or not a run of it)
      s.t.row = t.row, s.t.q0 = t.q0, s.t.n_tok = t.n_tok, s.t.pos0 = t.pos0;
      s.t.kb = t.kb, s.t.ke = t.ke, s.t.ctx = t.ctx;
    }
    __syncwarp();
    if (lane == 0) own->unit = unit;
    return more;
  }

  // The next segment of the share.
  __device__ __forceinline__ void open() {
    ChunkSegment s;
    long long last = 0;
    bool more;
    if (p.row_tiles) {
      more = own_next(s, last);
    } else {
      more = wk.next<kVecKeys>(p.c, s);
      if (more) last = s.head * __ldcg(p.c.ws_head) + __ldcg(p.c.ws_prefix + s.tile + 1) - 1;
    }
    Segment* e = segments + opened % kSegments;
    ++opened;
    units = 0;
    if (lane == 0) {
      e->valid = more;
      if (more) {
        e->q0 = s.t.q0, e->n_tok = s.t.n_tok, e->pos0 = s.t.pos0, e->ctx = s.t.ctx;
        e->kb = s.t.kb, e->j0 = s.j0, e->j1 = s.j1, e->head = s.head;
        e->whole = s.first && s.last, e->first = s.first, e->last = last;
      }
    }
    if (!more) return;
    units = s.j1 - s.j0;
    block = s.t.kb / kBlock + 2 * s.j0;
    block_end = (int)((unsigned)(s.t.ke + kBlock - 1) / kBlock);
    table = p.c.block_tables + (size_t)s.t.row * p.c.max_blocks;
    pool = (lane < 16 ? p.k_pool : p.v_pool) + (lane & 7) * 16 +
           (size_t)((s.head / p.subs) * p.heads_per_worker + head) * R::kTile;
    ids_from = block - 32;
  }

  // Copies of the next unit into the ring, if there is one, as a group of their own: eight
  // lanes a tile (the first block's keys, the second's, their values), whole lines.
  __device__ __forceinline__ void issue() {
    if (units != 0) {
      if (block - ids_from >= 32) {
        ids = block + lane < block_end ? __ldg(table + block + lane) : -1;
        ids_from = block;
      }
      const int b = block + ((lane >> 3) & 1);
      const int id = __shfl_sync(kFull, ids, b - ids_from);
      const bool ok = b < block_end && id >= 0 && id < p.c.pool_blocks;
      if (ok) {
        const uint8_t* src = pool + (size_t)(unsigned)id * ((unsigned)p.kv_heads * R::kTile);
        const uint32_t dst = ring + fill * R::kStage + (lane >> 3) * R::kTile + (lane & 7) * 16;
#pragma unroll
        for (uint32_t i = 0; i < R::kTile / 128; ++i) copy16(dst + i * 128, src + i * 128);
        if (R::kTile % 128 && (lane & 7) * 16 < R::kTile % 128)
          copy16(dst + R::kTile / 128 * 128, src + R::kTile / 128 * 128);
      }
      if (!__all_sync(kFull, ok)) {  // past the last block, or a bad one
        const uint32_t there = __ballot_sync(kFull, ok);
        missing |= (((there & 1u) | ((there >> 7) & 2u)) ^ 3u) << (2 * fill);
        if (b < block_end && !ok && (lane == 0 || lane == 8))
          atomicOr(p.c.status, (uint32_t)NSV_DEV_BAD_BLOCK);
      }
      fill = fill + 1 == kStages ? 0 : fill + 1;
      block += 2;
      if (--units == 0) open();
    }
    copy_group();
  }

  // Scores of a block: c[nt], rows are tokens, columns query vectors.
  __device__ __forceinline__ void scores(uint32_t tile, const uint32_t (&q)[kParts][NT][kSteps][2],
                                         float (&c)[NT][4]) const {
    const int r0 = g ^ ((g >> 1) & 1), r1 = r0 + 8;
    const uint32_t sc = tile + kv4_number_bytes(D);
    uint32_t w[2][D / 32];  // a lane's numbers of its two tokens
    uint32_t s[2][D / 64];  // their scales, doubled
    if constexpr (D == 128) {
      const uint4 a = lds<uint4>(tile + r0 * 64 + t * 16), b = lds<uint4>(tile + r1 * 64 + t * 16);
      w[0][0] = a.x, w[0][1] = a.y, w[0][2] = a.z, w[0][3] = a.w;
      w[1][0] = b.x, w[1][1] = b.y, w[1][2] = b.z, w[1][3] = b.w;
      const uint32_t e = e4m3x2_to_half(lds<uint16_t>(sc + r0 * 8 + 2 * t));
      const uint32_t f = e4m3x2_to_half(lds<uint16_t>(sc + r1 * 8 + 2 * t));
      s[0][0] = both(e, false), s[0][1] = both(e, true);
      s[1][0] = both(f, false), s[1][1] = both(f, true);
    } else {
      const uint2 a = lds<uint2>(tile + r0 * 32 + t * 8), b = lds<uint2>(tile + r1 * 32 + t * 8);
      w[0][0] = a.x, w[0][1] = a.y;
      w[1][0] = b.x, w[1][1] = b.y;
      s[0][0] = both(e4m3x2_to_half(lds<uint8_t>(sc + r0 * 4 + t)), false);
      s[1][0] = both(e4m3x2_to_half(lds<uint8_t>(sc + r1 * 4 + t)), false);
    }
    float low[NT][4];  // of the lower parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[nt][i] = low[nt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {  // 8 dimensions of a lane: two k steps
      uint32_t a[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        e2m1x8_to_half(w[r][i], a[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[r][j] = hmul2(a[r][j], s[r][i / 2]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(part ? low[nt] : c[nt], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1],
                a[1][2 * j + 1], q[part][nt][2 * i + j][0], q[part][nt][2 * i + j][1]);
    }
    if constexpr (kParts == 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[nt][i] = fmaf(low[nt][i], kLowDown, c[nt][i]);
    }
  }

  // A block's values as operands: rows are dimensions (lane g holds D / 8 that lie
  // together), k indices tokens.  x[i][h]: a byte holds one dimension of two tokens, the k
  // pair of an operand (h: even dimensions of the first and odd ones of the first, then of
  // the second pair of tokens); e: the pairs' scales.  dead: a bit for each of a lane's four
  // tokens that holds nothing.
  static constexpr int kWords = D / 64;  // words of a lane's dimensions of one token
  __device__ __forceinline__ void load_values(uint32_t tile, uint32_t dead,
                                              uint32_t (&x)[kWords][4], uint32_t (&e2)[2]) const {
    const uint32_t sc = tile + kv4_number_bytes(D);
    uint32_t w[4][kWords], e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = ((2 * t + (j & 1)) ^ (t & 1)) + (j & 2) * 4;
      if constexpr (D == 128) {
        const uint2 v = lds<uint2>(tile + tok * 64 + g * 8);
        w[j][0] = v.x, w[j][1] = v.y;
        e[j] = lds<uint8_t>(sc + tok * 8 + g);
      } else {
        w[j][0] = lds<uint32_t>(tile + tok * 32 + g * 4);
        e[j] = lds<uint8_t>(sc + tok * 4 + g / 2);
      }
    }
    if (dead) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((dead >> j) & 1) e[j] = 0;
    }
    e2[0] = e4m3x2_to_half(e[0] | (e[1] << 8));
    e2[1] = e4m3x2_to_half(e[2] | (e[3] << 8));
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a = w[2 * h][i], c = w[2 * h + 1][i];
        x[i][2 * h] = (a & 0x0f0f0f0fu) | ((c << 4) & 0xf0f0f0f0u);
        x[i][2 * h + 1] = ((a >> 4) & 0x0f0f0f0fu) | (c & 0xf0f0f0f0u);
      }
  }
  static __device__ __forceinline__ void widen_values(const uint32_t (&x)[4],
                                                      const uint32_t (&e2)[2],
                                                      uint32_t (&a)[4][4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      e2m1x8_to_half(x[h], a[h]);
#pragma unroll
      for (int k = 0; k < 4; ++k) a[h][k] = hmul2(a[h][k], e2[h / 2]);
    }
  }

  // o += V^T P of two blocks, columns are query vectors; dead: four bits a block.
  __device__ __forceinline__ void values(uint32_t tile,
                                         const uint32_t (&pb)[2][kParts][NT][2], uint32_t dead,
                                         float (&o)[kSteps][NT][4]) const {
    if constexpr (kParts == 1) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t x[kWords][4], e2[2];
        load_values(tile + b * R::kTile, dead >> (4 * b), x, e2);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint32_t a[4][4];
          widen_values(x[i], e2, a);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma(o[4 * i + k][nt], a[0][k], a[1][k], a[2][k], a[3][k], pb[b][0][nt][0],
                  pb[b][0][nt][1]);
        }
      }
    } else {
      // The tensor core's accumulator drops what it does not hold, always towards zero:
      // each unit's sum starts at zero and is added up rounded.
      uint32_t x[2][kWords][4], e2[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
        load_values(tile + b * R::kTile, dead >> (4 * b), x[b], e2[b]);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float sum[4][NT][4], low[4][NT][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[k][nt][j] = low[k][nt][j] = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t a[4][4];
          widen_values(x[b][i], e2[b], a);
#pragma unroll
          for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(part ? low[k][nt] : sum[k][nt], a[0][k], a[1][k], a[2][k], a[3][k],
                    pb[b][part][nt][0], pb[b][part][nt][1]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[4 * i + k][nt][j] += fmaf(low[k][nt][j], kLowDown, sum[k][nt][j]);
      }
    }
  }

  // The whole share.
  __device__ __forceinline__ void run(int worker) {
    if (!p.row_tiles) wk.init(p.c, worker);
    opened = fill = missing = at = 0;
    open();
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue();

#pragma unroll 1
    for (uint32_t taken = 0;; ++taken) {
      __syncwarp();
      const volatile Segment* s = segments + taken % kSegments;
      if (!s->valid) return;
      const int sub = s->head % p.subs;
      const int kv_head = (s->head / p.subs) * p.heads_per_worker + head;
      const int per = p.subs > 1 ? min(kVecs, p.c.group - sub * kVecs) : p.c.group;
      const int vecs = s->n_tok * per;
      const int h0 = kv_head * p.c.group + sub * kVecs;  // first query head
      auto row_of = [&](int v) {  // of query vector v, in q and out
        const int tok = v / per;
        return ((size_t)s->q0 + tok) * p.c.heads + h0 + (v - tok * per);
      };
      // the query vectors as operands, and what brings their scores to log2 units (the
      // scale's sign goes with the vectors)
      uint32_t q[kParts][NT][kSteps][2];
      float mul[NT][2];
      const float k_unit =
          fabsf(CAP ? p.c.scale : p.c.qscale) * (p.k_scales ? __ldg(p.k_scales + kv_head) : 1.f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int v = 8 * nt + g;
        float x[D / 4];  // dimensions D / 4 * t ..
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
        if (v < vecs) {
          const T* src = static_cast<const T*>(p.c.q) + row_of(v) * D + t * (D / 4);
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < D / 4; i += 4) {
              const float4 f = __ldg(reinterpret_cast<const float4*>(src + i));
              x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 4; i += 8) {
              const uint4 f = __ldg(reinterpret_cast<const uint4*>(src + i));
              const uint32_t r[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x[i + 2 * k] = __uint_as_float(r[k] << 16);
                x[i + 2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
              }
            }
          }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // top * 2^e in [2^14, 2^15), as far as 2^e is in range
        const int e = min(126, 14 + 127 - (int)(__float_as_uint(top) >> 23));
        const float up = copysignf(__uint_as_float((uint32_t)(127 + e) << 23), p.c.scale);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 4; i += 2) {
          const float a = x[i] * up, b = x[i + 1] * up;
          const uint32_t h = pack_half(a, b);
          q[0][nt][i / 4][(i / 2) & 1] = h;
          if constexpr (kParts == 2)
            q[kParts - 1][nt][i / 4][(i / 2) & 1] = lower_parts(a, b, h);
        }
        // (never 0: what is not seen, -inf, has to stay that)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          mul[nt][c] =
              fmaxf(k_unit * __shfl_sync(kFull, down, 4 * (2 * t + c)), 1.17549435e-38f);
      }
      // of the two columns of each column tile that this lane's scores are in: token,
      // position, what it sees
      auto token_of = [&](int nt, int c) { return (8 * nt + 2 * t + c) / per; };
      auto sees = [&](int nt, int c) {
        const int tok = token_of(nt, c);
        return 8 * nt + 2 * t + c < vecs
                   ? chunk_sees(p.c, (long long)s->q0 + tok, s->pos0 + tok, s->ctx)
                   : make_int2(0, 0x7fffffff);
      };
      float m[NT][2], l[NT][2], comp[NT][2], slope[NT][2];
      int pos[NT][2];
      int lo_all = 0, hi_all = 0x7fffffff;  // positions that all vectors see
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          m[nt][c] = kLeast;
          l[nt][c] = comp[nt][c] = 0.f;
          if constexpr (BIAS) {
            const int v = 8 * nt + 2 * t + c, tok = token_of(nt, c);
            pos[nt][c] = s->pos0 + tok;
            slope[nt][c] = v < vecs ? __ldg(p.c.slopes + h0 + (v - tok * per)) * kLog2e : 0.f;
          }
          const int2 see = sees(nt, c);
          lo_all = max(lo_all, see.x);
          hi_all = min(hi_all, see.y);
        }
      lo_all = __reduce_max_sync(kFull, lo_all);
      hi_all = __reduce_min_sync(kFull, hi_all);
      float o[kSteps][NT][4];
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;

      int t0 = s->kb + s->j0 * kVecKeys;
#pragma unroll 1
      for (int n = s->j1 - s->j0; n > 0; --n, t0 += kVecKeys) {
        issue();  // into the stage that the unit before was in
        copy_wait<kStages - 1>();
        __syncwarp();  // every lane's copies of this unit are there
        const uint32_t stage = ring + at * R::kStage;
        float x[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) scores(stage + b * R::kTile, q, x[b]);
        const int row = g ^ ((g >> 1) & 1);  // this lane's first token within a block
        if constexpr (CAP || BIAS) {         // to log2 units
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int c = i & 1;
                float y = x[b][nt][i] * mul[nt][c];
                if (CAP) y = p.c.cap * kLog2e * tanhf(y / p.c.cap);
                if (BIAS) {
                  const int rel = b * kBlock + row + (i & 2) * 4;
                  y -= slope[nt][c] * fabsf((float)(pos[nt][c] - t0 - rel));
                }
                x[b][nt][i] = y;
              }
        }
        uint32_t dead = 0;
        if (missing || t0 < lo_all || hi_all - t0 < kVecKeys) {  // what is not seen
          const uint32_t gone = (missing >> (2 * at)) & 3u;
          missing &= ~(3u << (2 * at));
          const int ctx = s->ctx;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int2 see = sees(nt, c);
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int rel = b * kBlock + row + 8 * h;
                  if (((gone >> b) & 1) || rel < see.x - t0 || rel >= see.y - t0)
                    x[b][nt][2 * h + c] = -INFINITY;
                }
            }
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rel = b * kBlock + ((2 * t + (k & 1)) ^ (t & 1)) + (k & 2) * 4;
              if (((gone >> b) & 1) || rel >= ctx - t0) dead |= 1u << (4 * b + k);
            }
        }
        // the running maxima
        float mx[NT][2];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx[nt][c] =
                fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
            if (!CAP && !BIAS) mx[nt][c] *= mul[nt][c];
            raise |= mx[nt][c] > m[nt][c] + Round<T>::kSlack;
          }
        if (__any_sync(kFull, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float y = mx[nt][c];
#pragma unroll
              for (int d = 4; d < 32; d *= 2) y = fmaxf(y, __shfl_xor_sync(kFull, y, d));
              y = fmaxf(y, m[nt][c]);
              const float alpha = ex2_approx(m[nt][c] - y);
              m[nt][c] = y;
              l[nt][c] *= alpha;
              comp[nt][c] *= alpha;
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                o[i][nt][c] *= alpha;
                o[i][nt][c + 2] *= alpha;
              }
            }
        }
        // weights, and as operands
        uint32_t pb[2][kParts][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float neg[2], sum[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) neg[c] = Round<T>::kUp - m[nt][c];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = ex2_approx(CAP || BIAS ? x[b][nt][i] + neg[i & 1]
                                            : fmaf(x[b][nt][i], mul[nt][i & 1], neg[i & 1]));
#pragma unroll
            for (int c = 0; c < 2; ++c) sum[c] = b ? sum[c] + (w[c] + w[c + 2]) : w[c] + w[c + 2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t up2 = pack_half(w[2 * h], w[2 * h + 1]);
              pb[b][0][nt][h] = transpose8x8(up2);
              if constexpr (kParts == 2)
                pb[b][kParts - 1][nt][h] =
                    transpose8x8(lower_parts(w[2 * h], w[2 * h + 1], up2));
            }
          }
          // (fp32's is compensated: nearly equal weights round the same way each time)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if constexpr (kParts == 1) {
              l[nt][c] += sum[c];
            } else {
              const float y = sum[c] - comp[nt][c];
              const float z = l[nt][c] + y;
              comp[nt][c] = (z - l[nt][c]) - y;
              l[nt][c] = z;
            }
          }
        }
        values(stage + 2 * R::kTile, pb, dead, o);
        at = at + 1 == kStages ? 0 : at + 1;
        __syncwarp();  // all lanes have read the stage
      }

      // The sums over the lanes that share a column; then the result or the piece.
      const bool whole = s->whole;
      const float v_unit = p.v_scales ? __ldg(p.v_scales + kv_head) : 1.f;
      const int slot = 2 * worker + (s->first ? 1 : 0);
      const size_t state = ((size_t)slot * p.heads_per_worker + head) * kVecs;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nt][c];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(kFull, sum, d);
          const int v = 8 * nt + 2 * t + c;
          if (v >= vecs) continue;
          if (whole) {
            const float inv = sum > 0.f ? v_unit / sum : 0.f;
            T* out = static_cast<T*>(p.c.out) + row_of(v) * D + g * (D / 8);
            if constexpr (sizeof(T) == 4) {
#pragma unroll
              for (int i = 0; i < kSteps; i += 2)
                *reinterpret_cast<float4*>(out + 2 * i) =
                    make_float4(o[i][nt][c] * inv, o[i][nt][c + 2] * inv, o[i + 1][nt][c] * inv,
                                o[i + 1][nt][c + 2] * inv);
            } else {
#pragma unroll
              for (int i = 0; i < kSteps; i += 4)
                *reinterpret_cast<uint4*>(out + 2 * i) =
                    make_uint4(pack_bf16(o[i][nt][c] * inv, o[i][nt][c + 2] * inv),
                               pack_bf16(o[i + 1][nt][c] * inv, o[i + 1][nt][c + 2] * inv),
                               pack_bf16(o[i + 2][nt][c] * inv, o[i + 2][nt][c + 2] * inv),
                               pack_bf16(o[i + 3][nt][c] * inv, o[i + 3][nt][c + 2] * inv));
            }
          } else {
            if (g == 0) p.ml[state + v] = make_float2(m[nt][c], sum);
            float* acc = p.acc + (state + v) * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < kSteps; i += 2)
              *reinterpret_cast<float4*>(acc + 2 * i) = make_float4(
                  o[i][nt][c], o[i][nt][c + 2], o[i + 1][nt][c], o[i + 1][nt][c + 2]);
          }
        }
      if (!whole && s->first && head == 0) {
        // how many workers the tile's pieces are on: those that start at or before
        // its last unit's first
        const long long last = s->last;
        int n = 0;
        if (p.row_tiles) n = (int)(((last + 1) * own->shares - 1) / own->all) - worker + 1;
#pragma unroll 1
        for (int c = worker; !p.row_tiles && c < p.c.grid; c += 32) {
          const unsigned in = __ballot_sync(
              kFull, c + lane < p.c.grid && __ldcg(p.c.ws_first + c + lane) <= last);
          n += __popc(in);
          if (in != kFull) break;
        }
        if (lane == 0) p.todo[worker] = make_int4(s->q0, s->n_tok, s->head, n);
      }
    }
  }
};

template <typename T, int NT>
constexpr int ctas_per_sm() {
  return sizeof(T) == 2 && NT == 1 ? 2 : 1;
}

template <typename T, int D, int NT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32, (ctas_per_sm<T, NT>()))
    kv4_vec_kernel(const __grid_constant__ Kv4VecParams p) {
  using R = Ring<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const uint32_t base = smem_u32(smem);
  using W = Worker<T, D, NT, CAP, BIAS>;
  const uint32_t segments = warps * R::kWarp;
  W w(p);
  griddep_wait();  // the tile list, and whatever was written before it
  griddep_launch();
  const int worker = blockIdx.x * p.workers_per_cta + warp / p.heads_per_worker;
  w.lane = lane;
  w.g = lane >> 2;
  w.t = lane & 3;
  w.ring = base + warp * R::kWarp;
  w.segments = reinterpret_cast<Segment*>(smem + segments + warp * kSegmentBytes);
  w.own = reinterpret_cast<volatile typename W::Own*>(w.segments + kSegments);
  w.head = warp % p.heads_per_worker;
  if (p.row_tiles) {
    OwnPlan* o = reinterpret_cast<OwnPlan*>(smem);  // where the ring will be
    static_assert(sizeof(OwnPlan) <= R::kWarp, "the ring of one warp");
    own_plan(p, o);
    w.start(o, worker);
    __syncthreads();
  }
  if (worker >= p.c.grid) return;
  if (w.head == 0 && lane == 0) p.todo[worker] = make_int4(0, 0, 0, 0);
  w.run(worker);
  copy_wait<0>();
}

// Joins the pieces of cut tiles, for KV head blockIdx.y of their groups:
// out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.  A warp takes one query vector, a
// lane D / 32 of its columns; where there are many pieces 2, 4 or 8 warps share them.  CTA
// blockIdx.x stands for a worker: those whose workers have the first pieces of a tile share its
// vectors.  (Few CTAs of 16 warps, one for each worker: 5 to 10 us slower.)
constexpr int kMergeWarps = 8;
// Most CTAs that share a tile: one for each vector that 8 warps take at a time.  (Of 32, whose
// tiles' list each CTA has to read, the call after a chunk of 2048 tokens starts later: 900 us
// a call in place of 880; 4: one long row of 16 vectors 74 us in place of 60.)
constexpr int kMergeShared = 16;
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv4_merge_kernel(const __grid_constant__ Kv4VecParams p) {
  constexpr int kVecs = 8 * NT, kCols = D / 32, kAhead = D == 128 ? 4 : 8;
  __shared__ float s_state[kMergeWarps][D + 2];
  griddep_wait();
  griddep_launch();
  const int head = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the tile that this worker starts, and the one of which it has a later piece
  int4 near = make_int4(0, 0, 0, 0);
  if (lane < kMergeShared && (int)blockIdx.x >= lane)
    near = __ldcg(p.todo + blockIdx.x - lane);
  if (__ballot_sync(kFull, near.w > lane) == 0) return;
  const int before = __ffs(__ballot_sync(kFull, near.w != 0 && lane > 0)) - 1;
#pragma unroll 1
  for (int back = max(0, before); back >= 0; back = back > 0 ? 0 : -1) {
    const int4 todo = make_int4(__shfl_sync(kFull, near.x, back), __shfl_sync(kFull, near.y, back),
                                __shfl_sync(kFull, near.z, back), __shfl_sync(kFull, near.w, back));
    if (todo.w <= back) continue;
    const int worker = blockIdx.x - back;
    const int sub = todo.z % p.subs;
    const int per = p.subs > 1 ? min(kVecs, p.c.group - sub * kVecs) : p.c.group;
    const int vecs = todo.y * per;
    int parts = 1;
    while (parts < kMergeWarps && parts * kAhead < todo.w) parts *= 2;
    const int part = warp % parts;
    const int b0 = (int)((long long)todo.w * part / parts);
    const int b1 = (int)((long long)todo.w * (part + 1) / parts);
#pragma unroll 1
    for (int v0 = back * (kMergeWarps / parts); v0 < vecs;
         v0 += min(todo.w, kMergeShared) * (kMergeWarps / parts)) {
      const int item = v0 + warp / parts, v = min(item, vecs - 1);
      float M = kLeast, L = 0.f, a[kCols];
#pragma unroll
      for (int k = 0; k < kCols; ++k) a[k] = 0.f;
      // takes states `ml` and `x` of n pieces in
      auto take = [&](const float2* ml, float (*x)[kCols], int n) {
        float top = M;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) top = fmaxf(top, ml[i].x);
        const float keep = ex2_approx(M - top);
        M = top;
        L *= keep;
#pragma unroll
        for (int k = 0; k < kCols; ++k) a[k] *= keep;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (i >= n) continue;
          const float w = ex2_approx(ml[i].x - M);
          L = fmaf(w, ml[i].y, L);
#pragma unroll
          for (int k = 0; k < kCols; ++k) a[k] = fmaf(w, x[i][k], a[k]);
        }
      };
#pragma unroll 1
      for (int b = b0; b < b1 && item < vecs; b += kAhead) {
        float2 ml[kAhead];
        float x[kAhead][kCols];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int j = min(b + i, b1 - 1);
          const size_t slot = 2 * (size_t)(worker + j) + (j == 0 ? 1 : 0);
          const size_t at = (slot * p.heads_per_worker + head) * kVecs + v;
          ml[i] = __ldcg(p.ml + at);
          const float* src = p.acc + at * D + lane * kCols;
          if constexpr (D == 128) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
            x[i][0] = f.x, x[i][1] = f.y, x[i][2] = f.z, x[i][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
            x[i][0] = f.x, x[i][1] = f.y;
          }
        }
        take(ml, x, b1 - b);
      }
      if (parts > 1) {  // the first of the warps that share joins their states, in order
        __syncthreads();
        float* st = s_state[warp];
#pragma unroll
        for (int k = 0; k < kCols; ++k) st[lane * kCols + k] = a[k];
        if (lane == 0) st[D] = M, st[D + 1] = L;
        __syncthreads();
        if (part == 0) {
          M = kLeast, L = 0.f;
#pragma unroll
          for (int k = 0; k < kCols; ++k) a[k] = 0.f;
#pragma unroll 1
          for (int b = 0; b < parts; b += kAhead) {
            float2 ml[kAhead];
            float x[kAhead][kCols];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              const float* o = s_state[warp + min(b + i, parts - 1)];
              ml[i] = make_float2(o[D], o[D + 1]);
#pragma unroll
              for (int k = 0; k < kCols; ++k) x[i][k] = o[lane * kCols + k];
            }
            take(ml, x, parts - b);
          }
        }
      }
      if (part != 0 || item >= vecs) continue;
      const int kv_head = (todo.z / p.subs) * p.heads_per_worker + head;
      const float inv = L > 0.f ? (p.v_scales ? __ldg(p.v_scales + kv_head) : 1.f) / L : 0.f;
      const int tok = v / per;
      T* out = static_cast<T*>(p.c.out) +
               (((size_t)todo.x + tok) * p.c.heads + kv_head * p.c.group + sub * kVecs +
                (v - tok * per)) * D + lane * kCols;
#pragma unroll
      for (int k = 0; k < kCols; k += 2) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float2*>(out + k) = make_float2(a[k] * inv, a[k + 1] * inv);
        else
          *reinterpret_cast<uint32_t*>(out + k) = pack_bf16(a[k] * inv, a[k + 1] * inv);
      }
    }
  }
}

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int D>
constexpr int smem_bytes(int warps) {
  return warps * (int)(Ring<D>::kWarp + kSegmentBytes);
}

template <typename T, int D, int NT, bool CAP, bool BIAS>
cudaError_t launch_one(const Kv4VecParams& p, cudaStream_t stream) {
  const int warps = p.workers_per_cta * p.heads_per_worker;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg =
      config(dim3((unsigned)((p.c.grid + p.workers_per_cta - 1) / p.workers_per_cta)), warps * 32,
             smem_bytes<D>(warps), stream, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_vec_kernel<T, D, NT, CAP, BIAS>, p);
  if (e != cudaSuccess) return e;
  cfg = config(dim3((unsigned)p.c.grid, (unsigned)p.heads_per_worker), kMergeWarps * 32, 0,
               stream, &attr);
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T, D, NT>, p);
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const Kv4VecParams& p, cudaStream_t stream) {
  const bool cap = p.c.cap > 0.f, bias = p.c.slopes != nullptr;
  return cap ? (bias ? launch_one<T, D, NT, true, true>(p, stream)
                     : launch_one<T, D, NT, true, false>(p, stream))
             : (bias ? launch_one<T, D, NT, false, true>(p, stream)
                     : launch_one<T, D, NT, false, false>(p, stream));
}

template <typename T, int D, int NT>
cudaError_t set_attrs() {
  const int bytes = smem_bytes<D>(kWarps);
  cudaError_t e = cudaFuncSetAttribute(kv4_vec_kernel<T, D, NT, false, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv4_vec_kernel<T, D, NT, false, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv4_vec_kernel<T, D, NT, true, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv4_vec_kernel<T, D, NT, true, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

}  // namespace

int kv4_vec_ctas_per_sm(int dtype, int col_tiles) {
  return dtype == NSV_BF16 && col_tiles == 1 ? 2 : 1;
}

cudaError_t prepare_kv4_vec() {
  cudaError_t e = set_attrs<float, 64, 1>();
  if (e == cudaSuccess) e = set_attrs<float, 128, 1>();
  if (e == cudaSuccess) e = set_attrs<__nv_bfloat16, 64, 1>();
  if (e == cudaSuccess) e = set_attrs<__nv_bfloat16, 128, 1>();
  if (e == cudaSuccess) e = set_attrs<__nv_bfloat16, 64, 2>();
  if (e == cudaSuccess) e = set_attrs<__nv_bfloat16, 128, 2>();
  return e;
}

cudaError_t launch_kv4_vec(const Kv4VecParams& p, int dtype, int head_dim, int col_tiles,
                           cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (dtype == NSV_F32)
    return head_dim == 64 ? launch_nt<float, 64, 1>(p, stream) : launch_nt<float, 128, 1>(p, stream);
  if (col_tiles == 1)
    return head_dim == 64 ? launch_nt<B, 64, 1>(p, stream) : launch_nt<B, 128, 1>(p, stream);
  return head_dim == 64 ? launch_nt<B, 64, 2>(p, stream) : launch_nt<B, 128, 2>(p, stream);
}

}  // namespace nsv
