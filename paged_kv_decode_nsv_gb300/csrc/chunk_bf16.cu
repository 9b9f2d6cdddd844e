// Attention of a chunk of new tokens over a paged cache, bf16, on the
// 5th-generation tensor cores.
//
// For query token i of a row and query head h, with KV head h / group:
//   s_t = scale * q_i,h . k_t      (optionally capped: cap * tanh(s_t / cap),
//                                   and biased: - slope_h * |pos_i - t|)
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x = s * log2(e)
// over the positions t that the token sees, folded 128 positions at a time
// with a running maximum m and sum l (fp32, the sum of the unrounded
// probabilities).  The probabilities are rounded to bf16 for the second
// product, as its tensor-core operand: half a step each (2^-8 relative at most),
// which is what rounding the output costs anyway.  Outputs are off by 0.0017 to
// 0.0023 of their size against 64 bits, the rounded exact ones by 0.0016 to 0.0017.
//
// One CTA per SM, nineteen warps:
//   warps 0-7, 8-15 softmax of stream 0 and stream 1: MMA row r (TMEM lane r) of a
//                   stream belongs to two threads, one in each warp of a pair,
//                   which split its columns (scores and output)
//   warp 16         TMA producer: query rows, then K and V of each run, block by
//                   block through the block table, into a ring of stages
//   warp 17         MMA issue: S = Q.K^T (both operands in shared memory) and
//                   O += P.V (P in tensor memory), accumulators in tensor memory
//   warp 18         publishes the pieces of cut tiles
// The rows of an MMA are the tile's query tokens times the query heads that
// share the KV head, so K and V are read once for all of them.  A tile with
// more than 128 rows gives each stream its half of the rows and both the same
// keys; a smaller tile gives both streams the same rows and every other run of
// keys, and the two states are joined at the end.  Either way one stream's
// softmax runs while the tensor core works for the other.
// A tile of at most 64 or 32 rows is laid out 2 or 4 times over the 128 MMA
// rows, and each copy takes its part of every run's keys (the probabilities of
// the rest are zeros), so that all warps share the softmax of a few rows; the
// copies' states are joined through shared memory.
//
// Tensor memory (512 columns): S of stream x at 128 x, a column per key; the
// bf16 probabilities of each 16 keys over the first 8 columns of their scores; O
// of stream x at 256 + D x.
// Work is dealt out in equal numbers of units (chunk.cuh); a tile cut between
// CTAs leaves partial states in the workspace and the CTA whose piece arrives
// last merges them.  All waits are bounded; one that gives up sets
// NSV_DEV_TIMEOUT and the kernel ends.
//
// Over a 4-bit cache (KV4) all operands are fp16, which holds its numbers times their scales
// exactly: query vectors come converted, each times a power of two that makes its largest
// element nearly 2^15, and probabilities are rounded to fp16 (2^-11).  Twenty warps: 16 and 17
// widen tiles, which wait as they are in the pool in a ring of half runs, into the stages; 18
// issues; 19 fetches tiles by bulk copies and publishes at the end.  2048 tokens over 32768
// positions, 32 heads, 8 KV heads: 875 to 884 us, 1.2 PFLOP/s; 751 with the widening left out, which is
// what the bf16 cache takes.  The widening warps' instructions take the softmax warps' issue
// slots.  (bf16 operands, four widening warps: 1351, e2m1 converts only to fp16; eight widening
// warps 1076, four and a fetching warp 926; query rows by the bulk copies 909; two widening
// warps, and 96 registers a thread without a split, 878.  Tile rings of the widening warps' own:
// 965; registers split 96 / 56 / 40: 1204.)
//
// What bounds it: for many tokens the chain of one stream, softmax of a run (1900
// cycles) and its two products (1170), against which the other stream's runs are
// laid: 1700 cycles a turn, 1420 without the softmax.  4096 tokens over 32768
// positions, 32 heads, 8 KV heads: 1.55 ms, 1.33 PFLOP/s, the tensor pipe busy 60 %
// of the time.  For single tokens HBM: 256 rows of 512 to 8192 positions, capped and
// biased, 551 us, 5.6 TB/s; a run of 64 KiB takes 1.5 us, a tile's start and end 4 to
// 5.

#include "chunk.cuh"
#include "kv4.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kSoftWarps = 16;
// Over a 4-bit cache: warps 16 and 17 widen, 18 issues, 19 fetches and then publishes.  (At
// most 20 warps, five on a sub-partition, have 96 registers each.)
constexpr int kWidenWarps = 2;
// Tiles as they are in the pool wait in a ring of half runs (a run's keys or values).
constexpr int kTileRing = 3;
template <int D>
constexpr uint32_t kHalfRun = kChunkKeys / kBlock * kv4_tile_bytes(D);
template <bool KV4>
constexpr int kThreads = (KV4 ? kSoftWarps + kWidenWarps + 2 : kSoftWarps + 3) * 32;
template <bool KV4>
constexpr int kMmaWarp = KV4 ? kSoftWarps + kWidenWarps : kSoftWarps + 1;
constexpr int kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr int kMetaRing = 16;
// The running maximum is raised only when a run exceeds it by more than this
// (log2 units): probabilities stay <= 2^8, and most runs skip the rescale.
constexpr float kSlack = 8.f;
// fp16 ones are held times 2^7 (at most 2^15), so that small ones keep their digits.
constexpr float kUpHalf = 7.f;

// Over a 4-bit cache there is one stage less, which makes room for the tiles as they are
// in the pool (five: 970 us for 2048 tokens over 32768, with loads to registers in place
// of that room; four: 942).
template <int D, bool KV4>
struct Smem {
  static constexpr uint32_t kStage = kChunkKeys * D * 2;  // K or V of one run
  static constexpr int kStages = (KV4 ? 4 : 5) * (128 / D);
  static constexpr uint32_t kHalf = kChunkHalfRows * D * 2;  // query rows of one half
  static constexpr uint32_t kOffQ = kStages * kStage;
  // Exchange of the copies' outputs, [2 streams][2 halves][128 rows][16 columns]
  // floats: over the second half's query rows, which a tile with copies has
  // none of (head_dim 64 has room beside them).
  static constexpr uint32_t kQuarterX = kChunkHalfRows * 16 * 4;
  static constexpr uint32_t kOffX = D == 128 ? kOffQ + kHalf : kOffQ + 2 * kHalf;
  static constexpr uint32_t kOffMl = D == 128 ? kOffQ + 2 * kHalf : kOffX + 4 * kQuarterX;
  // kOffMl: float2 [2][128]
  // int4 [2][2]: tiles to merge
  static constexpr uint32_t kOffTodo = kOffMl + 2 * kChunkHalfRows * 8;
  static constexpr uint32_t kOffBars = kOffTodo + 64;
  static constexpr int kBars = 2 * kStages + 19;
  static constexpr uint32_t kOffMeta = kOffBars + kBars * 8;
  static constexpr uint32_t kOffPairs = kOffMeta + kMetaRing * 4;  // PairWords [8]
  static constexpr uint32_t kOffWord = kOffPairs + 8 * 20;  // the TMEM address, then kOffDone
  static constexpr uint32_t kOffDone = kOffWord + 4;        // softmax warps done, over all tiles
  static constexpr uint32_t kOffTiles = (kOffWord + 16 + 127) / 128 * 128;
  static constexpr uint32_t kOffTileBars = kOffTiles + kTileRing * kHalfRun<D>;  // full, free
  static constexpr uint32_t kTotal = KV4 ? kOffTileBars + 2 * kTileRing * 8 : kOffWord + 16;
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

template <int D, bool KV4>
struct Bars {
  uint32_t b;
  static constexpr int S = Smem<D, KV4>::kStages;
  __device__ uint32_t full(uint32_t i) const { return b + 8 * i; }
  __device__ uint32_t empty(uint32_t i) const { return b + 8 * (S + i); }
  __device__ uint32_t qfull() const { return b + 8 * (2 * S); }
  __device__ uint32_t qfree() const { return b + 8 * (2 * S + 1); }
  __device__ uint32_t scores(int x) const { return b + 8 * (2 * S + 2 + x); }
  __device__ uint32_t probs(int x) const { return b + 8 * (2 * S + 4 + x); }
  __device__ uint32_t out(int x) const { return b + 8 * (2 * S + 6 + x); }
  __device__ uint32_t ofree() const { return b + 8 * (2 * S + 8); }
  __device__ uint32_t join() const { return b + 8 * (2 * S + 9); }
  __device__ uint32_t drained() const { return b + 8 * (2 * S + 10); }
  __device__ uint32_t meet(int i) const { return b + 8 * (2 * S + 11 + i); }
  __device__ uint32_t piece(int first) const { return b + 8 * (2 * S + (first ? 18 : 15)); }
  __device__ uint32_t mlfree() const { return b + 8 * (2 * S + 17); }
  __device__ uint32_t published() const { return b + 8 * (2 * S + 16); }
};

// A bounded wait for a count that only grows.
__device__ __forceinline__ bool count_wait(const volatile uint32_t* count, uint32_t least) {
  const long long t0 = clock64();
  bool ok;
#pragma unroll 1
  while (!(ok = *count >= least) && clock64() - t0 <= kWaitLimitCycles) {
  }
  __threadfence_block();
  return __all_sync(kFull, ok);
}

// How a tile's rows lie: 0: over both halves; else how many copies of them one
// half holds.
__device__ __forceinline__ int copies_of(const ChunkParams& p, const ChunkSegment& s) {
  const int rows = s.t.n_tok * p.group;
  return s.t.n_tok * 2 > p.tile_tokens          ? 0
         : rows <= kChunkHalfRows / 4           ? 4
         : rows <= kChunkHalfRows / 2           ? 2
                                                : 1;
}

// ------------------------------------------------------------------ producer
// A segment's query rows.
template <int D, bool KV4>
__device__ __forceinline__ bool load_queries(const ChunkParams& p, const Bars<D, KV4>& B,
                                             uint32_t smem0,
                                             const volatile uint32_t* s_done,
                                             const ChunkSegment& s, int lane, uint32_t nseg,
                                             uint32_t& shared) {
  using L = Smem<D, KV4>;
  const int half_tok = p.tile_tokens / 2;
  // the query rows: one box of (tokens, group heads, 64 dims) per half or
  // copy and 64-dim slice; tokens past the tensor are filled with zeros
  if (nseg && !warp_wait(B.qfree(), (nseg - 1) & 1)) return false;
  const int copies = copies_of(p, s);
  // The second half may still serve an earlier tile's copies.  (A count, not a
  // barrier's parity: their epilogue can be two tiles behind.)
  if (copies == 0 && shared && !count_wait(s_done, shared * kSoftWarps)) return false;
  if (copies == 0) shared = 0;
  if (copies > 1) shared = nseg + 1;
  if (lane == 0) {
    const int boxes = copies == 0 ? 2 : copies;
    const int box_rows = copies == 0 ? kChunkHalfRows : kChunkHalfRows / copies;
    const int box_tok = box_rows / p.group;
    const CUtensorMap* map = &p.tmap_q[copies == 4 ? 2 : copies == 2 ? 1 : 0];
    mbar_arrive_tx(B.qfull(), (uint32_t)(boxes * box_tok * p.group * D * 2));
#pragma unroll 1
    for (int x = 0; x < boxes; ++x)
      for (int d = 0; d < D / 64; ++d)
        tma_load_3d(smem0 + L::kOffQ + (copies == 0 ? x * L::kHalf : x * box_rows * 128) +
                        d * (kChunkHalfRows * 128),
                    map, d * 64, s.head * p.group, s.t.q0 + (copies == 0 ? x * half_tok : 0),
                    B.qfull());
  }
  return true;
}

template <int D>
__device__ __forceinline__ bool produce(const ChunkParams& p, const Bars<D, false>& B,
                                        uint32_t smem0, volatile int* s_meta,
                                        const volatile uint32_t* s_done, ChunkWalk wk, int lane,
                                        uint32_t& i, uint32_t& nseg) {
  using L = Smem<D, false>;
  constexpr uint32_t kBlockBytes = kBlock * D * 2;
  uint32_t run = 0;
  uint32_t shared = 0;  // segments up to and with the last one whose copies were exchanged
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kChunkKeys>(p, s)) {
    if (!load_queries<D, false>(p, B, smem0, s_done, s, lane, nseg, shared)) return false;
    ++nseg;
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    auto block_id = [&](int j) -> int {  // lane's block of run j, -1 past the tile's keys
      const int b = (s.t.kb + j * kChunkKeys) / kBlock + lane;
      return lane < kChunkKeys / kBlock && (long long)b * kBlock < s.t.ke ? __ldg(table + b) : -1;
    };
    int id = block_id(s.j0);
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j) {
      const bool wanted = lane < kChunkKeys / kBlock &&
                          (long long)s.t.kb + j * kChunkKeys + lane * kBlock < s.t.ke;
      const bool ok = wanted && id >= 0 && id < p.pool_blocks;
      if (wanted && !ok) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_BLOCK);
      const unsigned mask = __ballot_sync(kFull, ok);
      const int coord = (int)(((long long)id * p.kv_heads + s.head) * 2);  // groups of 8 tokens
      id = j + 1 < s.j1 ? block_id(j + 1) : -1;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t slot = i % L::kStages, ph = (i / L::kStages) & 1;
        if (!warp_wait(B.empty(slot), ph ^ 1)) return false;
        if (lane == 0) {
          if (kv == 0) s_meta[run % kMetaRing] = (int)mask;
          mbar_arrive_tx(B.full(slot), __popc(mask) * kBlockBytes);
        }
        __syncwarp();
        if (ok)
          tma_load_4d(smem0 + slot * L::kStage + lane * kBlockBytes, kv ? &p.tmap_v : &p.tmap_k, 0,
                      0, 0, coord, B.full(slot));
        ++i;
      }
      ++run;
    }
  }
  return true;
}

// --------------------------------------------------------------------- widening
// Over a 4-bit cache operands are fp16: its numbers times their scales are exact, and a
// pair of them takes 11 instructions a word of 8 (bf16, which has no conversion from
// e2m1, 23).  The query rows have been scaled and converted when the tiles were listed
// (chunk_plan.cu; two of this kernel's warps took 7 us a tile for it).

// The query rows, and the tiles of a run's keys, then of its values, by one warp: tiles into
// a ring of half runs, a lane copies a block.
template <int D>
__device__ __forceinline__ bool fetch_tiles(const Chunk4Params& p, const Bars<D, true>& B,
                                            uint32_t smem0, volatile int* s_meta,
                                            const volatile uint32_t* s_done, ChunkWalk wk,
                                            int lane, uint32_t& issued, uint32_t& nseg) {
  using L = Smem<D, true>;
  constexpr uint32_t kTile = kv4_tile_bytes(D);
  uint32_t run = 0, in = 0, parity = 1, shared = 0;
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kChunkKeys>(p, s)) {
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    auto block_id = [&](int j) -> int {  // lane's block of run j, -1 past the tile's keys
      const int b = (s.t.kb + j * kChunkKeys) / kBlock + lane;
      return lane < kChunkKeys / kBlock && (long long)b * kBlock < s.t.ke ? __ldg(table + b) : -1;
    };
    int id = block_id(s.j0);
    if (!load_queries<D, true>(p, B, smem0, s_done, s, lane, nseg, shared)) return false;
    ++nseg;
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j) {
      const bool wanted = lane < kChunkKeys / kBlock &&
                          (long long)s.t.kb + j * kChunkKeys + lane * kBlock < s.t.ke;
      const bool ok = wanted && id >= 0 && id < p.pool_blocks;
      if (wanted && !ok) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_BLOCK);
      const unsigned mask = __ballot_sync(kFull, ok);
      const size_t at = ((size_t)(unsigned)id * p.kv_heads + s.head) * kTile;
      id = j + 1 < s.j1 ? block_id(j + 1) : -1;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!warp_wait(smem0 + L::kOffTileBars + 8 * (kTileRing + in), parity)) return false;
        const uint32_t full = smem0 + L::kOffTileBars + 8 * in;
        if (lane == 0) {
          // (the meta ring has room for more runs than the rings and stages hold)
          if (kv == 0) s_meta[run % kMetaRing] = (int)mask;
          mbar_arrive_tx(full, __popc(mask) * kTile);
        }
        __syncwarp();
        if (ok)
          bulk_load(smem0 + L::kOffTiles + in * kHalfRun<D> + lane * kTile,
                    (kv ? p.v4 : p.k4) + at, kTile, full);
        ++issued;
        if (++in == kTileRing) in = 0, parity ^= 1;
      }
      ++run;
    }
  }
  return true;
}

// Keys and values: a warp takes half of the blocks of a half run, 8 tokens at a time, a lane
// a quarter of one of them.  They go where the bulk copies of a bf16 cache would have put
// them, in the same swizzle.  (At head_dim 128 two of the 8 lanes that write together meet in
// each bank; words taken in another order, which avoids that, cost more than the meeting:
// what these warps issue, the softmax beside them waits for.)  Tokens that are not there
// become zeros.
template <int D>
__device__ __forceinline__ bool widen(const ChunkParams& p, const Bars<D, true>& B,
                                      unsigned char* smem, const volatile int* s_meta,
                                      ChunkWalk wk, int ww, int lane) {
  using L = Smem<D, true>;
  constexpr uint32_t kTile = kv4_tile_bytes(D);
  constexpr int kWords = D / 32;                         // words of a lane's quarter
  constexpr int kEights = kChunkKeys / 8 / kWidenWarps;  // of tokens a half run
  constexpr int kThere = (1 << (kEights / 2)) - 1;       // all of the warp's blocks
  const int row = lane >> 2, part = lane & 3;
  const uint32_t smem0 = smem_u32(smem);
  uint32_t i = 0, run = 0;
  uint32_t out = 0, parity = 0;  // the ring slot to read, and its turn
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kChunkKeys>(p, s)) {
#pragma unroll 1
    for (int h = 2 * s.j0; h < 2 * s.j1; ++h, ++i) {
      const uint32_t full = smem0 + L::kOffTileBars + 8 * out;
      const uint32_t slot = i % L::kStages, ph = (i / L::kStages) & 1;
      const bool here = mbar_wait(full, parity) && mbar_wait(B.empty(slot), ph ^ 1);
      if (!__all_sync(kFull, here)) return false;
      const int mask = s_meta[run % kMetaRing] >> (kEights / 2 * ww);
      // tokens that are there, of this warp's
      const int left = s.t.ctx - s.t.kb - (h >> 1) * kChunkKeys - 8 * kEights * ww;
      unsigned char* stage = smem + slot * L::kStage + kEights * ww * (D / 64) * 1024 + row * 128;
      const unsigned char* tiles =
          smem + L::kOffTiles + out * kHalfRun<D> + kEights / 2 * ww * kTile;
      uint32_t w[kEights][kWords], sc[kEights];
#pragma unroll
      for (int q = 0; q < kEights; ++q) {
        const unsigned char* t = tiles + (q >> 1) * kTile;
        const int off = 8 * (q & 1) + row;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(t + off * 64 + part * 16);
          w[q][0] = x.x, w[q][1] = x.y, w[q][2] = x.z, w[q][3] = x.w;
          sc[q] = *reinterpret_cast<const uint16_t*>(t + 8 * D + off * 8 + part * 2);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(t + off * 32 + part * 8);
          w[q][0] = x.x, w[q][1] = x.y;
          sc[q] = t[8 * D + off * 4 + part];
        }
      }
      if (left < 8 * kEights || (mask & kThere) != kThere) {
#pragma unroll
        for (int q = 0; q < kEights; ++q)
          if (8 * q + row >= left || !((mask >> (q >> 1)) & 1)) sc[q] = 0;
      }
#pragma unroll
      for (int q = 0; q < kEights; ++q) {
        const uint32_t e = e4m3x2_to_half(sc[q]);
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          const uint32_t s2 = __byte_perm(e, 0, k >= 2 ? 0x3232 : 0x1010);
          uint32_t g[4];
          e2m1x8_to_half(w[q][k], g);
#pragma unroll
          for (int n = 0; n < 4; ++n) g[n] = hmul2(g[n], s2);
          const int chunk = part * kWords + k;  // 8 dimensions
          *reinterpret_cast<uint4*>(stage + (q * (D / 64) + (chunk >> 3)) * 1024 +
                                    (((chunk & 7) ^ row) << 4)) =
              make_uint4(g[0], g[1], g[2], g[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();  // all lanes have read the tiles too
      if (lane == 0) {
        mbar_arrive(B.full(slot));
        mbar_arrive(full + 8 * kTileRing);
      }
      if (++out == kTileRing) out = 0, parity ^= 1;
      run += h & 1;
    }
  }
  return true;
}

// ------------------------------------------------------------------------ MMA
// One warp issues for both streams, in turn: products of one stream's
// probabilities and its next scores, then the other's.  (A warp per stream let
// both streams fall into step, their softmax at the same time and their MMAs at
// the same time: 2167 against 1753 us for 4096 tokens over 32768.)  The CTA holds
// all of tensor memory, which starts at column 0, so that all operands but the
// stage are compile-time constants.  One thread, elected, runs all of this: the
// votes that keep a whole warp together made a turn 1740 cycles long where its
// MMAs take 1000.
template <int D, bool KV4>
__device__ __forceinline__ bool issue_mma(const ChunkParams& p, const Bars<D, KV4>& B, uint32_t smem0,
                                          ChunkWalk wk) {
  using L = Smem<D, KV4>;
  // K and V stages: tokens in groups of 8, a group's 64-dim halves one
  // 1024-byte swizzle atom after the other
  constexpr uint32_t kGroup = (D / 64) * 1024u;
  constexpr uint32_t kTypes = KV4 ? kIdescHalf : 0;
  constexpr uint32_t idesc_s = umma_idesc_bf16(kChunkHalfRows, kChunkKeys, false) ^ kTypes;
  constexpr uint32_t idesc_o = umma_idesc_bf16(kChunkHalfRows, D, true) ^ kTypes;
  const uint64_t dq = umma_desc128(smem0 + L::kOffQ, 16, 1024);
  const uint64_t dk = umma_desc128(smem0, 16, kGroup);
  const uint64_t dv = umma_desc128(smem0, 1024, kGroup);
  // descriptors are linear in the start address: a base plus an offset
  auto stage_at = [](uint32_t i) { return (i % L::kStages) * (L::kStage >> 4); };
  auto scores = [&](uint32_t x, uint32_t half, uint32_t i) {
    tc_fence_after();
    const uint64_t a = dq + half * (L::kHalf >> 4), b = dk + stage_at(i);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      umma_ss(x * kChunkKeys, a + (((ks >> 2) * (kChunkHalfRows * 128) + (ks & 3) * 32) >> 4),
              b + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), idesc_s, ks > 0, true);
    umma_commit(B.scores(x), true);
  };
  auto values = [&](uint32_t x, uint32_t i, bool fresh) {
    const uint64_t b = dv + stage_at(i);
#pragma unroll
    for (int ks = 0; ks < kChunkKeys / 16; ++ks)
      umma_ts(kColO + x * D, x * kChunkKeys + ks * kBlock, b + ((ks * 2 * kGroup) >> 4), idesc_o,
              !fresh || ks > 0, true);
  };
  uint32_t base = 0, nseg = 0, np[2] = {0, 0};
  auto wait_full = [&](uint32_t i) {
    return mbar_wait(B.full(i % L::kStages), (i / L::kStages) & 1);
  };
  auto free_stage = [&](uint32_t i) { umma_commit(B.empty(i % L::kStages), true); };
  ChunkSegment s, next;
#pragma unroll 1
  for (bool more = wk.next<kChunkKeys>(p, s); more; s = next) {
    const int n = s.j1 - s.j0;
    const bool pair = copies_of(p, s) == 0;
    more = wk.next<kChunkKeys>(p, next);  // its loads overlap this segment's work
    if (!mbar_wait(B.qfull(), nseg & 1)) return false;
    // Turn k: stream x = k & 1 multiplies the probabilities of its run and starts
    // its next scores.  A pair's streams take every run each (turn 2 j + x), the
    // others run k.
    const int turns = pair ? 2 * n : n;
    const int ahead = pair ? 1 : 2;  // runs between a stream's runs
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!pair && x >= n) break;
      const uint32_t ik = base + (pair ? 0 : 2 * x);
      if (!wait_full(ik)) return false;
      scores(x, pair ? x : 0, ik);
      if (!pair || x == 1) free_stage(ik);
    }
    if (n <= ahead) umma_commit(B.qfree(), true);
    // before O is written again: the previous segment's has been read
    if (nseg && !mbar_wait(B.ofree(), (nseg - 1) & 1)) return false;
    auto turn = [&](uint32_t x, int j) {
      const uint32_t iv = base + 2 * j + 1, ik = base + 2 * (j + ahead);
      if (!wait_full(iv)) return false;
      if (!mbar_wait(B.probs(x), np[x]++ & 1)) return false;
      tc_fence_after();
      values(x, iv, j < ahead);
      const bool last_reader = !pair || x == 1;
      if (j + ahead < n) {
        if (!wait_full(ik)) return false;
        scores(x, pair ? x : 0, ik);
        if (last_reader) {
          free_stage(iv);
          free_stage(ik);
          if (j + ahead + 1 == n) umma_commit(B.qfree(), true);
        }
      } else {
        if (last_reader) free_stage(iv);
      }
      return true;
    };
#pragma unroll 1
    for (int k = 0; k < turns; k += 2) {
      if (!turn(0, pair ? k / 2 : k)) return false;
      if (k + 1 < turns && !turn(1, pair ? k / 2 : k + 1)) return false;
    }
    umma_commit(B.out(0), true);
    umma_commit(B.out(1), true);
    base += 2 * n;
    ++nseg;
  }
  return true;
}

// -------------------------------------------------------------------- softmax
// cap * tanh(s * scale / cap) in log2 units for caps so large that the scores
// stay near the tanh's linear part: z = s * scale / cap; below 1/4 the series
// z (1 - z^2/3 + 2 z^4/15 - 17 z^6/315) (relative error under 4e-7), above it
// 1 - 2 r, r = 1 / (1 + e^2z).  For smaller caps that second form alone will do: e^2z
// is off by 2^-22 of itself, the sum by 2^-24 and the reciprocal by 2^-23, so a score by
// at most cap * 3.7e-7 besides its own fp32 rounding.  At a cap of 256 that is 2^-13.4 of
// a weight, twice that where the other score of a ratio is off the other way: below
// 2^-12, and a probability's rounding to bf16 is up to 2^-8.  (256 single tokens over 512
// to 8192 positions: the second form alone 559 us, the choice of both 563.)
constexpr float kLargeCap = 256.f;
__device__ __forceinline__ float large_cap(float s, float cap_z, float cap_out) {
  const float z = s * cap_z;
  const float big = 1.f - 2.f * rcp_approx(1.f + ex2_approx(z * 2.8853900817779268f));
  const float z2 = z * z;
  const float small =
      z * fmaf(z2, fmaf(z2, fmaf(z2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return (z2 < 0.0625f ? small : big) * cap_out;
}

// The state of one row of a stream, as each of its two threads holds it.
struct RowState {
  bool valid, fresh;  // whether the row exists; whether O holds nothing yet
  int pos;            // the query token's position
  int2 see;           // what it sees
  float slope;        // slope * log2(e)
  float m, l;         // running maximum (log2 units); this thread's part of the sum
};

// Folds the NC keys of one run that are this thread's (columns col0 .. of the
// scores t_s) into its row: the maximum over both threads' columns, rescale of
// this thread's half of O (t_o) where it rises, probabilities (bf16) over the
// scores.
//
// Two passes over the scores in tensor memory, 16 columns at a time, instead of
// one with the row in registers: unrolled over 64 columns the loop's code, run by
// 16 warps each at its own place, did not fit the instruction cache, and warps
// waited for instructions more than for anything else.
template <int D, bool CAP, bool BIAS, bool KV4>
__device__ __forceinline__ bool fold_run(const ChunkParams& p, float unit, RowState& f, uint32_t t_s,
                                         uint32_t t_o, int t0, int col0, int NC, int hf, int copy,
                                         int mask, bool past, int bar, volatile PairWords* w,
                                         volatile float2* s_ml, uint32_t turn, int lane) {
  constexpr int kW = 16;
  float mul = p.qscale * unit;
  // positions that the row does not see; nothing to mask in most runs
  const int lo = f.see.x - t0 - col0, hi = f.see.y - t0 - col0;
  const int bm = mask >> (col0 / kBlock);
  const int all = (1 << (NC / kBlock)) - 1;
  const bool dense = (bm & all) == all && lo <= 0 && hi >= NC && mul > 0.f;
  float mx = -INFINITY;
  if (!CAP && !BIAS && __all_sync(kFull, dense)) {
    float m1 = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < NC; c += kW) {
      float s[kW];
      tmem_ld16(t_s + col0 + c, s);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < kW; k += 4) {
        mx = max3(mx, s[k], s[k + 1]);
        m1 = max3(m1, s[k + 2], s[k + 3]);
      }
    }
    mx = fmaxf(mx, m1) * mul;
  } else {
    // scale, cap, bias and mask, and put the result back
    const float d0 = (float)(f.pos - t0 - col0);
    const float cap_out = p.cap * 1.4426950408889634f;
    const float cap_z = CAP ? p.scale * unit / p.cap : 0.f, cap_in = cap_z * 2.8853900817779268f;
#pragma unroll 1
    for (int c = 0; c < NC; c += kW) {
      float s[kW];
      tmem_ld16(t_s + col0 + c, s);
      tmem_wait_ld();
      if (CAP) {
        if (p.cap > kLargeCap) {
#pragma unroll
          for (int k = 0; k < kW; ++k) s[k] = large_cap(s[k], cap_z, cap_out);
        } else {
#pragma unroll
          for (int k = 0; k < kW; ++k)
            s[k] = fmaf(rcp_approx(1.f + ex2_approx(s[k] * cap_in)), -2.f * cap_out, cap_out);
        }
      }
      const float m0 = CAP ? 1.f : mul;
      if (BIAS) {
        const float d = d0 - (float)c;
        if (past) {  // - slope * (d - k), in two multiply-adds for two columns
          const float b0 = -f.slope * d;
#pragma unroll
          for (int k = 0; k < kW; k += 2) {
            float x0, x1;
            fma2(x0, x1, f.slope, f.slope, (float)k, (float)(k + 1), b0, b0);
            fma2(s[k], s[k + 1], s[k], s[k + 1], m0, m0, x0, x1);
          }
        } else {  // positions on both sides of the token
#pragma unroll
          for (int k = 0; k < kW; ++k)
            s[k] = fmaf(-f.slope, fabsf(d - (float)k), s[k] * m0);
        }
      } else if (!CAP) {
#pragma unroll
        for (int k = 0; k < kW; ++k) s[k] *= m0;
      }
      const int a = min(max(lo - c, 0), kW), b = min(max(hi - c, 0), kW);
      const uint32_t bits = ((bm >> (c / kBlock)) & 1) ? ((1u << b) - 1u) & ~((1u << a) - 1u) : 0u;
      if (!__all_sync(kFull, bits == 0xffffu)) {
#pragma unroll
        for (int k = 0; k < kW; ++k) s[k] = (bits >> k) & 1u ? s[k] : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < kW; k += 2) mx = max3(mx, s[k], s[k + 1]);
      tmem_st16(t_s + col0 + c, s);
    }
    tmem_wait_st();
    mul = 1.f;
  }
  // Both warps learn which rows exceed the running maximum; in most runs none
  // does, and the maxima themselves need no exchange.
  const uint32_t mine = __ballot_sync(kFull, f.valid && mx > f.m + kSlack);
  if (lane == 0) w->raise[turn & 1][hf] = mine;
  if (!pair_sync(bar, w)) return false;
  if (mine | w->raise[turn & 1][hf ^ 1]) {
    (hf ? s_ml->y : s_ml->x) = mx;
    if (!pair_sync(bar, w)) return false;
    mx = fmaxf(mx, hf ? s_ml->x : s_ml->y);
    const bool raise = f.valid && mx > f.m + kSlack;  // also the first finite one
    float alpha = 1.f;
    if (raise) {
      alpha = ex2_approx(f.m - mx);
      f.m = mx;
      f.l *= alpha;
    }
    // The products that O holds are complete: the scores just waited for were
    // issued after them.
    if (!f.fresh && __any_sync(kFull, raise)) {
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        float o[16];
        tmem_ld16(t_o + hf * (D / 2) + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= alpha;
        tmem_st16(t_o + hf * (D / 2) + c, o);
      }
    }
  }
  const float neg = f.m == -INFINITY ? 0.f : KV4 ? kUpHalf - f.m : -f.m;
  float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
  for (int c = 0; c < NC; c += kW) {
    float s[kW];
    tmem_ld16(t_s + col0 + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < kW; k += 2) {
      float a, b;
      fma2(a, b, s[k], s[k + 1], mul, mul, neg, neg);
      a = ex2_approx(a);
      b = ex2_approx(b);
      add2(l0, l1, a, b);
      s[k / 2] = __uint_as_float(KV4 ? pack_half(a, b) : pack_bf16(a, b));
    }
    tmem_st8(t_s + col0 + c, s);
  }
  if (NC < 64) {  // the keys of the other copies: zeros, every other block each
    float zero[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) zero[k] = 0.f;
    const int first = 2 * copy * NC / kBlock, n = 2 * NC / kBlock;  // the copy's blocks
#pragma unroll 1
    for (int b = hf; b < kChunkKeys / kBlock; b += 2)
      if (b < first || b >= first + n) tmem_st8(t_s + b * kBlock, zero);
  }
  f.l += l0 + l1;
  tmem_wait_st();
  return true;
}

template <int D, bool CAP, bool BIAS, bool KV4>
__device__ __forceinline__ int softmax(const ChunkArgs<KV4>& p, const Bars<D, KV4>& B,
                                       unsigned char* smem, const volatile int* s_meta,
                                       int4* s_todo, uint32_t* s_done,
                                       volatile PairWords* words, ChunkWalk wk, int warp,
                                       int lane) {
  using L = Smem<D, KV4>;
  using T = __nv_bfloat16;
  const int x = warp >> 3;                     // stream
  const int hf = (warp >> 2) & 1;              // which of the pair: its half of the columns
  const int r = (warp & 3) * 32 + lane;        // MMA row, TMEM lane
  const int bar = 1 + x * 4 + (warp & 3);      // the pair's barrier
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t t_s = lane_base + x * kChunkKeys;
  const uint32_t t_o = lane_base + kColO;
  const int half_tok = p.tile_tokens / 2;
  float2* s_ml = reinterpret_cast<float2*>(smem + L::kOffMl);
  float* s_x = reinterpret_cast<float*>(smem + L::kOffX + (x * 2 + hf) * L::kQuarterX);
  uint32_t nscore = 0, nseg = 0, njoin = 0, nmeet = 0, run0 = 0, turn = 0;
  // the four warps with this stream and half meet
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(B.meet(x * 2 + hf));
    return warp_wait(B.meet(x * 2 + hf), nmeet++ & 1);
  };
  // all softmax warps meet
  auto join = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(B.join());
    return warp_wait(B.join(), njoin++ & 1);
  };
  ChunkSegment s, next;
#pragma unroll 1
  for (bool more = wk.next<kChunkKeys>(p, s); more; s = next) {
    const int copies = copies_of(p, s);
    const bool pair = copies == 0;
    const int n = s.j1 - s.j0;
    // this thread's row within its half or copy, and its part of a run's keys:
    // 64, 32 or 16 columns from col0 on
    const int shift = copies == 4 ? 2 : copies == 2 ? 1 : 0;
    const int copy_rows = kChunkHalfRows >> shift;
    const int copy = r >> (7 - shift), rc = r & (copy_rows - 1);
    const int col0 = (2 * copy + hf) * (64 >> shift);
    const int ti = (int)((unsigned)rc / (unsigned)p.group), g = rc - ti * p.group;
    const int tok = (pair && x ? half_tok : 0) + ti;  // query token within the tile
    const bool valid = (ti + 1) * p.group <= copy_rows && tok < s.t.n_tok;
    const bool any_valid = __any_sync(kFull, valid);
    RowState f;
    f.valid = valid;
    f.fresh = true;
    f.pos = s.t.pos0 + tok;
    f.see = make_int2(0, 0x7fffffff);  // rows that are not there mask nothing
    if (valid) f.see = chunk_sees(p, (long long)s.t.q0 + tok, f.pos, s.t.ctx);
    f.slope = BIAS && valid ? __ldg(p.slopes + s.head * p.group + g) * 1.4426950408889634f : 0.f;
    f.m = -INFINITY;
    f.l = 0.f;
    const bool past = !BIAS || __all_sync(kFull, !valid || f.see.y <= f.pos + 1);
    const int step = pair ? 1 : 2;
    // what brings a 4-bit cache's scores to their size
    float unit = k_unit(p, s.head);
    if constexpr (KV4) {
      if (valid)
        unit *= __ldg(p.q_up + ((size_t)s.t.q0 + tok) * p.heads + s.head * p.group + g);
    }
    // the states' exchange is free: every warp has read the previous tile's
    if (nseg && !warp_wait(B.mlfree(), (nseg - 1) & 1)) return kTimedOut;
#pragma unroll 1
    for (int j = s.j0 + (pair ? 0 : x); j < s.j1; j += step) {
      const uint32_t run = run0 + (uint32_t)(j - s.j0);
      const int t0 = s.t.kb + j * kChunkKeys;
      if (!warp_wait(B.scores(x), nscore++ & 1)) return kTimedOut;
      tc_fence_after();
      const int mask = s_meta[run % kMetaRing];
      // Values of positions that hold nothing (past the context, or in a
      // block that was not loaded) become zeros: their probability is 0, but
      // 0 * NaN is not.
      if (!KV4 && (mask != 0xff || s.t.ctx - t0 < kChunkKeys)) {
        const uint32_t i = 2 * run + 1, slot = i % L::kStages;
        if (!warp_wait(B.full(slot), (i / L::kStages) & 1)) return kTimedOut;
        if (!((mask >> (r >> 4)) & 1) || r >= s.t.ctx - t0) {
          unsigned char* v = smem + slot * L::kStage + (r >> 3) * (D / 64) * 1024 + (r & 7) * 128;
#pragma unroll 1
          for (int c = hf * (D / 16); c < (hf + 1) * (D / 16); ++c)
            *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (any_valid) {
        const bool ok = fold_run<D, CAP, BIAS, KV4>(p, unit, f, t_s, t_o + x * D, t0, col0,
                                                    64 >> shift, hf, copy, mask, past, bar, words,
                                                    s_ml + x * kChunkHalfRows + r, turn, lane);
        if (!ok) return kPartnerFailed;
        ++turn;
      }
      f.fresh = false;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(B.probs(x));
    }
    run0 += (uint32_t)n;

    more = wk.next<kChunkKeys>(p, next);  // its loads overlap the wait
    // The segment's end: O is complete once its last product is.
    if (!warp_wait(B.out(x), nseg & 1)) return kTimedOut;
    tc_fence_after();
    const bool whole = s.first && s.last;
    const int row = tok * p.group + g;  // within the tile
    const int slot = chunk_slot(blockIdx.x, s.first);
    // the row's maximum and sum over both threads
    float2* own = s_ml + x * kChunkHalfRows + r;
    if (hf) own->y = f.l;
    if (!pair_sync(bar, words)) return kPartnerFailed;
    if (!hf) *own = make_float2(f.m, f.l + own->y);
    // weights of the two streams' O (lane r of both holds the same row where the
    // tile is not a pair), and the row's maximum and sum over streams and copies
    float w0 = 1.f, w1 = 0.f, M, Lsum;
    if (pair) {
      if (!pair_sync(bar, words)) return kPartnerFailed;
      M = own->x;
      Lsum = own->y;
    } else {
      if (!join()) return kTimedOut;
      M = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < copies; ++c)
        M = fmaxf(M, fmaxf(s_ml[c * copy_rows + rc].x,
                           s_ml[kChunkHalfRows + c * copy_rows + rc].x));
      Lsum = 0.f;
      auto weight = [&](float mm) { return mm == -INFINITY ? 0.f : ex2_approx(mm - M); };
#pragma unroll 1
      for (int c = 0; c < copies; ++c) {
        const float2 a = s_ml[c * copy_rows + rc], b = s_ml[kChunkHalfRows + c * copy_rows + rc];
        Lsum += a.y * weight(a.x) + b.y * weight(b.x);
      }
      w0 = weight(s_ml[r].x);
      w1 = weight(s_ml[kChunkHalfRows + r].x);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(B.mlfree());  // read: the next tile's states may go there
    const float inv = (whole ? (Lsum > 0.f ? 1.f / Lsum : 0.f) : 1.f) * v_unit(p, s.head);
    w0 *= inv;
    w1 *= inv;
    // where the tile's rows go: row `off` of this KV head's
    T* out = static_cast<T*>(p.out) + ((size_t)s.t.q0 * p.heads + s.head * p.group) * D;
    const int off = valid ? tok * p.heads + g : -1;
    // A pair's stream writes all columns of its own rows, half by each warp;
    // otherwise each of a row's four warps takes a quarter of the columns.
    const int c_lo = pair ? hf * (D / 2) : (x * 2 + hf) * (D / 4);
    const int c_hi = c_lo + (pair ? D / 2 : D / 4);
    // Copies are added up through shared memory: all columns at once where the
    // rows fill at most half of a copy's, else 16 at a time.
    const bool few = 2 * s.t.n_tok * p.group <= copy_rows;
    const int round = copies > 1 ? (few ? D / 4 : 16) : c_hi - c_lo;
    const int x_rows = few ? copy_rows / 2 : copy_rows;  // its row stride
#pragma unroll 1
    for (int cr = c_lo; cr < c_hi; cr += round) {
      if (cr > c_lo && !meet()) return kTimedOut;  // the columns before have been read
#pragma unroll 1
      for (int c = cr; c < cr + round; c += 16) {
        float v[16];
        tmem_ld16(t_o + (pair ? x * D : 0) + c, v);
        if (!pair && n > 1) {
          float v1[16];
          tmem_ld16(t_o + D + c, v1);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = v[k] * w0 + v1[k] * w1;
        } else {
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] *= w0;
        }
        if (copies > 1) {
          float* e = s_x + (copy * round + c - cr) * x_rows + rc;
          if (valid) {
#pragma unroll
            for (int k = 0; k < 16; ++k) e[k * x_rows] = v[k];
          }
        } else if (whole) {
          // Two lanes trade halves, so that each writes 16 of the 32 bytes that the
          // two have of a row: a store then touches 16 lines and fills its sectors,
          // where each lane writing its own row would touch 32.
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
          const bool odd_lane = lane & 1;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t got = __shfl_xor_sync(kFull, odd_lane ? w[k] : w[4 + k], 1);
            if (odd_lane) w[k] = got; else w[4 + k] = got;
          }
          // now w[0..3]: the even lane's row, w[4..7]: the odd lane's
          const int peer = __shfl_xor_sync(kFull, off, 1);
          const int even = odd_lane ? peer : off, odd = odd_lane ? off : peer;
          T* o = out + c + (odd_lane ? 8 : 0);
          if (even >= 0)
            *reinterpret_cast<uint4*>(o + (size_t)even * D) = make_uint4(w[0], w[1], w[2], w[3]);
          if (odd >= 0)
            *reinterpret_cast<uint4*>(o + (size_t)odd * D) = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (valid) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *chunk_acc(p, slot, D, (c + k) / 4, row) =
                make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
      }
      if (copies > 1) {
        if (!meet()) return kTimedOut;
        // each copy sums its share of the columns
        const int share = round >> shift;
#pragma unroll 1
        for (int k0 = copy * share; valid && k0 < (copy + 1) * share; k0 += 4) {
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
          const float* e = s_x + k0 * x_rows + rc;
#pragma unroll 1
          for (int cp = 0; cp < copies; ++cp, e += round * x_rows) {
            t.x += e[0];
            t.y += e[x_rows];
            t.z += e[2 * x_rows];
            t.w += e[3 * x_rows];
          }
          if (whole)
            *reinterpret_cast<uint2*>(out + (size_t)off * D + cr + k0) =
                make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
          else
            *chunk_acc(p, slot, D, (cr + k0) / 4, row) = t;
        }
      }
    }
    if (!whole && valid && hf == 0 && (pair || (x == 0 && copy == 0)))
      p.ws_ml[(size_t)slot * p.tile_rows + row] = make_float2(M, Lsum);
    tc_fence_before();
    fence_proxy_async_smem();  // the exchange's bytes may become query rows again
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(B.ofree());
      __threadfence_block();
      atomicAdd(s_done, 1u);
      if (!whole) mbar_arrive(B.piece(s.first));
    }
    ++nseg;
  }
  if (!warp_wait(B.published(), 0)) return kTimedOut;
  chunk_merge_todo<T, D, kSoftWarps * 32>(p, s_todo);
  return kDone;
}

template <int D, bool CAP, bool BIAS, bool KV4>
__global__ void __launch_bounds__(kThreads<KV4>, 1) chunk_bf16_kernel(
    const __grid_constant__ ChunkArgs<KV4> p) {
  using L = Smem<D, KV4>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t smem0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars<D, KV4> B{smem0 + L::kOffBars};
  volatile int* s_meta = reinterpret_cast<volatile int*>(smem + L::kOffMeta);
  volatile PairWords* s_pairs = reinterpret_cast<volatile PairWords*>(smem + L::kOffPairs);
  volatile uint32_t* s_word = reinterpret_cast<volatile uint32_t*>(smem + L::kOffWord);
  int4* s_todo = reinterpret_cast<int4*>(smem + L::kOffTodo);
  uint32_t* s_done = reinterpret_cast<uint32_t*>(smem + L::kOffDone);
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2 * L::kStages + 2; ++i)
        mbar_init(smem0 + L::kOffBars + 8 * i,
                  KV4 && i < L::kStages ? kWidenWarps : 1);
      for (int i = 0; KV4 && i < 2 * kTileRing; ++i)
        mbar_init(smem0 + L::kOffTileBars + 8 * i, i < kTileRing ? 1 : kWidenWarps);
      mbar_init(B.drained(), 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(B.scores(x), 1);
        mbar_init(B.probs(x), kSoftWarps / 2);
        mbar_init(B.out(x), 1);
        mbar_init(B.meet(2 * x), kSoftWarps / 4);
        mbar_init(B.meet(2 * x + 1), kSoftWarps / 4);
      }
      mbar_init(B.ofree(), kSoftWarps);
      mbar_init(B.join(), kSoftWarps);
      mbar_init(B.piece(0), kSoftWarps);
      mbar_init(B.piece(1), kSoftWarps);
      mbar_init(B.published(), 1);
      mbar_init(B.mlfree(), kSoftWarps);
      fence_mbar_init();
      for (int i = 0; i < 8; ++i) s_pairs[i].failed = 0;
      for (int i = 0; i < 4; ++i) s_todo[i] = make_int4(0, 0, 0, 0);
      *s_done = 0;
    }
    __syncwarp();
    tmem_alloc(smem_u32(smem + L::kOffWord), kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // What the code takes for granted (never seen otherwise): the swizzled
  // operands' alignment, and that all of tensor memory starts at column 0.
  const uint32_t tmem = *s_word;
  const bool odd = (smem0 & 1023u) != 0 || tmem != 0;
  griddep_wait();  // the tile list, and whatever was written before it
  griddep_launch();
  ChunkWalk wk;
  wk.init(p, blockIdx.x);
  bool ok = !odd;
  if (odd) {
    // nothing runs; the end below flags it
  } else if (warp < kSoftWarps) {
    volatile PairWords* words = s_pairs + (warp >> 3) * 4 + (warp & 3);
    const int end = softmax<D, CAP, BIAS, KV4>(p, B, smem, s_meta, s_todo, s_done, words, wk, warp,
                                          lane);
    // Every warp but one whose partner failed meets its partner once more: so a
    // partner that still works learns of a timeout at its next meeting, and none
    // is left waiting.
    if (end != kPartnerFailed) {
      if (end == kTimedOut) words->failed = 1;
      __syncwarp();
      (void)pair_sync(1 + (warp >> 3) * 4 + (warp & 3), words);
    }
    ok = end == kDone;
  } else if (KV4 && warp < kSoftWarps + kWidenWarps) {
    if constexpr (KV4) {
      ok = widen<D>(p, B, smem, s_meta, wk, warp - kSoftWarps, lane);
    }
  } else if (!KV4 && warp == kSoftWarps) {
    if constexpr (!KV4) {
      uint32_t i = 0, nq = 0;
      ok = produce<D>(p, B, smem0, s_meta, s_done, wk, lane, i, nq);
      // every copy issued lands before the CTA can end, even after a timeout
      for (uint32_t k = i > (uint32_t)L::kStages ? i - L::kStages : 0; k < i; ++k)
        (void)mbar_wait(B.full(k % L::kStages), (k / L::kStages) & 1);
      if (nq) (void)mbar_wait(B.qfull(), (nq - 1) & 1);
    }
  } else {
    if (warp == kMmaWarp<KV4>) {
      if (elect_one()) {
        ok = issue_mma<D, KV4>(p, B, smem0, wk);
        if (!ok) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
        umma_commit(B.drained(), true);  // arrives once every MMA issued is done
        (void)mbar_wait(B.drained(), 0);
      }
      __syncwarp();
    } else {
      if constexpr (KV4) {
        uint32_t issued = 0, nq = 0;
        ok = fetch_tiles<D>(p, B, smem0, s_meta, s_done, wk, lane, issued, nq);
        if (nq) (void)mbar_wait(B.qfull(), (nq - 1) & 1);
        // every copy issued lands before the CTA can end, even after a timeout
        for (uint32_t k = issued > kTileRing ? issued - kTileRing : 0; k < issued; ++k)
          (void)mbar_wait(smem0 + L::kOffTileBars + 8 * (k % kTileRing), (k / kTileRing) & 1);
      }
      if (ok)
        ok = chunk_publish<kChunkKeys>(p, B.piece(0), B.piece(1), B.published(), s_todo, wk, lane);
    }
  }
  if (!ok && lane == 0) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool CAP, bool BIAS, bool KV4>
cudaError_t launch_one(const ChunkArgs<KV4>& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kThreads<KV4>);
  cfg.dynamicSmemBytes = Smem<D, KV4>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_bf16_kernel<D, CAP, BIAS, KV4>, p);
}

template <int D, bool KV4>
cudaError_t launch_dim(const ChunkArgs<KV4>& p, cudaStream_t stream) {
  const bool cap = p.cap > 0.f, bias = p.slopes != nullptr;
  return cap ? (bias ? launch_one<D, true, true, KV4>(p, stream)
                     : launch_one<D, true, false, KV4>(p, stream))
             : (bias ? launch_one<D, false, true, KV4>(p, stream)
                     : launch_one<D, false, false, KV4>(p, stream));
}

template <int D, bool CAP, bool BIAS>
cudaError_t set_attr() {
  const cudaError_t e =
      cudaFuncSetAttribute(chunk_bf16_kernel<D, CAP, BIAS, false>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, false>::kTotal);
  return e != cudaSuccess
             ? e
             : cudaFuncSetAttribute(chunk_bf16_kernel<D, CAP, BIAS, true>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Smem<D, true>::kTotal);
}

template <int D>
cudaError_t set_attrs() {
  cudaError_t e;
  if ((e = set_attr<D, false, false>()) != cudaSuccess) return e;
  if ((e = set_attr<D, false, true>()) != cudaSuccess) return e;
  if ((e = set_attr<D, true, false>()) != cudaSuccess) return e;
  return set_attr<D, true, true>();
}

}  // namespace

cudaError_t prepare_chunk_bf16() {
  const cudaError_t e = set_attrs<64>();
  return e != cudaSuccess ? e : set_attrs<128>();
}

cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64, false>(p, stream) : launch_dim<128, false>(p, stream);
}

cudaError_t launch_chunk_kv4(const Chunk4Params& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64, true>(p, stream) : launch_dim<128, true>(p, stream);
}

}  // namespace nsv
