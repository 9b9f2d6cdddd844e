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
// product, as its tensor-core operand: half an ulp each (2^-9 relative),
// which is what rounding the output costs anyway.
//
// One CTA per SM, twelve warps:
//   warps 0-3, 4-7  softmax of stream 0 and stream 1: thread r of a stream owns
//                   MMA row r (TMEM lane r): its scores, its state, its output
//   warp 8          TMA producer: query rows, then K and V of each run, block by
//                   block through the block table, into a ring of stages
//   warp 9          MMA issue: S = Q.K^T (both operands in shared memory) and
//                   O += P.V (P in tensor memory), accumulators in tensor memory
//   warps 10, 11    idle: they complete the warpgroup that gives registers away
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
// Tensor memory (512 columns): S of stream x at 128 x, its probabilities over
// the first 64 of them, O of stream x at 256 + D x.
// Work is dealt out in equal numbers of units (chunk.cuh); a tile cut between
// CTAs leaves partial states in the workspace and the CTA whose piece arrives
// last merges them.  All waits are bounded; one that gives up sets
// NSV_DEV_TIMEOUT and the kernel ends.

#include "chunk.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kThreads = 384;
// Registers per thread: 168 at launch (12 warps); the two softmax warpgroups
// (whose threads hold a row's 128 scores) take 208 from the third's share:
// 2 x 208 + 80 = 496 <= 3 x 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "more registers than the launch has");
constexpr int kStreamWarps = 4;
constexpr int kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr int kMetaRing = 16;
// The running maximum is raised only when a run exceeds it by more than this
// (log2 units): probabilities stay <= 2^8, and most runs skip the rescale.
constexpr float kSlack = 8.f;

template <int D>
struct Smem {
  static constexpr uint32_t kStage = kChunkKeys * D * 2;  // K or V of one run
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr uint32_t kHalf = kChunkHalfRows * D * 2;  // query rows of one half
  static constexpr uint32_t kOffQ = kStages * kStage;
  // Exchange of the copies' outputs, [2 streams][128 rows][32 columns] floats:
  // over the second half's query rows, which a tile with copies has none of
  // (head_dim 64 has room beside them).
  static constexpr uint32_t kStreamX = kChunkHalfRows * 32 * 4;
  static constexpr uint32_t kOffX = D == 128 ? kOffQ + kHalf : kOffQ + 2 * kHalf;
  static constexpr uint32_t kOffMl = D == 128 ? kOffQ + 2 * kHalf : kOffX + 2 * kStreamX;
  // kOffMl: float2 [2][128]
  static constexpr uint32_t kOffBars = kOffMl + 2 * kChunkHalfRows * 8;
  static constexpr int kBars = 2 * kStages + 13;
  static constexpr uint32_t kOffMeta = kOffBars + kBars * 8;
  static constexpr uint32_t kOffWords = kOffMeta + kMetaRing * 4;  // TMEM address, abort, merge
  static constexpr uint32_t kTotal = kOffWords + 16;
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

template <int D>
struct Bars {
  uint32_t b;
  static constexpr int S = Smem<D>::kStages;
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
  __device__ uint32_t meet(int x) const { return b + 8 * (2 * S + 11 + x); }
};

// A bounded wait with one answer for the whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait(bar, parity));
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
template <int D>
__device__ __forceinline__ bool produce(const ChunkParams& p, const Bars<D>& B, uint32_t smem0,
                                        volatile int* s_meta, ChunkWalk wk, int lane,
                                        uint32_t& i, uint32_t& nseg) {
  using L = Smem<D>;
  constexpr uint32_t kBlockBytes = kBlock * D * 2;
  const int half_tok = p.tile_tokens / 2;
  uint32_t run = 0;
  int before = 0;  // the previous segment's copies
  ChunkSegment s;
  while (wk.next(p, s)) {
    // the query rows: one box of (tokens, group heads, 64 dims) per half or
    // copy and 64-dim slice; tokens past the tensor are filled with zeros
    if (nseg && !warp_wait(B.qfree(), (nseg - 1) & 1)) return false;
    const int copies = copies_of(p, s);
    // (the second half may still serve the previous tile's copies)
    if (copies == 0 && before > 1 && !warp_wait(B.ofree(), (nseg - 1) & 1)) return false;
    before = copies;
    if (lane == 0) {
      const int boxes = copies == 0 ? 2 : copies;
      const int box_rows = copies == 0 ? kChunkHalfRows : kChunkHalfRows / copies;
      const int box_tok = box_rows / p.group;
      const CUtensorMap* map = &p.tmap_q[copies == 4 ? 2 : copies == 2 ? 1 : 0];
      mbar_arrive_tx(B.qfull(), (uint32_t)(boxes * box_tok * p.group * D * 2));
      for (int x = 0; x < boxes; ++x)
        for (int d = 0; d < D / 64; ++d)
          tma_load_3d(smem0 + L::kOffQ + (copies == 0 ? x * L::kHalf : x * box_rows * 128) +
                          d * (kChunkHalfRows * 128),
                      map, d * 64, s.head * p.group, s.t.q0 + (copies == 0 ? x * half_tok : 0),
                      B.qfull());
    }
    ++nseg;
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    auto block_id = [&](int j) -> int {  // lane's block of run j, -1 past the tile's keys
      const int b = (s.t.kb + j * kChunkKeys) / kBlock + lane;
      return lane < kChunkKeys / kBlock && (long long)b * kBlock < s.t.ke ? __ldg(table + b) : -1;
    };
    int id = block_id(s.j0);
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

// ------------------------------------------------------------------------ MMA
template <int D>
__device__ __forceinline__ bool issue_mma(const ChunkParams& p, const Bars<D>& B, uint32_t smem0,
                                          uint32_t tmem, ChunkWalk wk, bool lead) {
  using L = Smem<D>;
  // K and V stages: tokens in groups of 8, a group's 64-dim halves one
  // 1024-byte swizzle atom after the other
  constexpr uint32_t kGroup = (D / 64) * 1024u;
  constexpr uint32_t idesc_s = umma_idesc_bf16(kChunkHalfRows, kChunkKeys, false);
  constexpr uint32_t idesc_o = umma_idesc_bf16(kChunkHalfRows, D, true);
  const uint64_t dq = umma_desc128(smem0 + L::kOffQ, 16, 1024);
  const uint64_t dk = umma_desc128(smem0, 16, kGroup);
  const uint64_t dv = umma_desc128(smem0, 1024, kGroup);
  auto scores = [&](int x, int half, uint32_t slot) {
    tc_fence_after();
    const uint64_t a = dq + ((half * L::kHalf) >> 4), b = dk + ((slot * L::kStage) >> 4);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      umma_ss(tmem + x * kChunkKeys, a + (((ks >> 2) * (kChunkHalfRows * 128) + (ks & 3) * 32) >> 4),
              b + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), idesc_s, ks > 0, lead);
    umma_commit(B.scores(x), lead);
  };
  auto values = [&](int x, uint32_t slot, bool fresh) {
    const uint64_t b = dv + ((slot * L::kStage) >> 4);
#pragma unroll
    for (int ks = 0; ks < kChunkKeys / 16; ++ks)
      umma_ts(tmem + kColO + x * D, tmem + x * kChunkKeys + ks * 8, b + ((ks * 2 * kGroup) >> 4),
              idesc_o, !fresh || ks > 0, lead);
  };
  uint32_t base = 0, nseg = 0, np[2] = {0, 0};
  auto slot_of = [](uint32_t i) { return i % L::kStages; };
  auto wait_full = [&](uint32_t i) {
    return warp_wait(B.full(i % L::kStages), (i / L::kStages) & 1);
  };
  ChunkSegment s, next;
  for (bool more = wk.next(p, s); more; s = next) {
    const int n = s.j1 - s.j0;
    const bool pair = copies_of(p, s) == 0;
    more = wk.next(p, next);  // its loads overlap this segment's work
    if (!warp_wait(B.qfull(), nseg & 1)) return false;
    // before O is written again: the previous segment's has been read
    auto free_o = [&]() { return nseg == 0 || warp_wait(B.ofree(), (nseg - 1) & 1); };
    if (pair) {
      if (!wait_full(base)) return false;
      scores(0, 0, slot_of(base));
      scores(1, 1, slot_of(base));
      umma_commit(B.empty(slot_of(base)), lead);
      if (n == 1) umma_commit(B.qfree(), lead);
      for (int j = 0; j < n; ++j) {
        const uint32_t iv = base + 2 * j + 1, ik = iv + 1;
        const bool again = j + 1 < n;
        if (j == 0 && !free_o()) return false;
        if (!wait_full(iv)) return false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!warp_wait(B.probs(x), np[x]++ & 1)) return false;
          tc_fence_after();
          values(x, slot_of(iv), j == 0);
          if (x == 1) umma_commit(B.empty(slot_of(iv)), lead);
          if (again) {
            if (x == 0 && !wait_full(ik)) return false;
            scores(x, x, slot_of(ik));
            if (x == 1) {
              umma_commit(B.empty(slot_of(ik)), lead);
              if (j + 2 == n) umma_commit(B.qfree(), lead);
            }
          } else {
            umma_commit(B.out(x), lead);
          }
        }
      }
    } else {
      for (int j = 0; j < 2 && j < n; ++j) {
        const uint32_t ik = base + 2 * j;
        if (!wait_full(ik)) return false;
        scores(j, 0, slot_of(ik));
        umma_commit(B.empty(slot_of(ik)), lead);
      }
      if (n <= 2) umma_commit(B.qfree(), lead);
      for (int j = 0; j < n; ++j) {
        const uint32_t iv = base + 2 * j + 1, ik = base + 2 * j + 4;
        const int x = j & 1;
        if (j == 0 && !free_o()) return false;
        if (!wait_full(iv)) return false;
        if (!warp_wait(B.probs(x), np[x]++ & 1)) return false;
        tc_fence_after();
        values(x, slot_of(iv), j < 2);
        umma_commit(B.empty(slot_of(iv)), lead);
        if (j + 2 < n) {
          if (!wait_full(ik)) return false;
          scores(x, 0, slot_of(ik));
          umma_commit(B.empty(slot_of(ik)), lead);
          if (j + 3 == n) umma_commit(B.qfree(), lead);
        }
      }
      umma_commit(B.out(0), lead);
      umma_commit(B.out(1), lead);
    }
    base += 2 * n;
    ++nseg;
  }
  return true;
}

// -------------------------------------------------------------------- softmax
// cap * tanh(s * scale / cap) in log2 units.  z = s * scale / cap; below 1/4 the
// series z (1 - z^2/3 + 2 z^4/15 - 17 z^6/315) (relative error under 4e-7), above
// it 1 - 2 / (1 + e^2z), whose cancellation is harmless there.
__device__ __forceinline__ float capped(float s, float cap_z, float cap_out) {
  const float z = s * cap_z;
  const float e = ex2_approx(z * 2.8853900817779268f);  // 2 log2(e)
  const float big = 1.f - 2.f * rcp_approx(1.f + e);
  const float z2 = z * z;
  const float small =
      z * fmaf(z2, fmaf(z2, fmaf(z2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return (z2 < 0.0625f ? small : big) * cap_out;
}

// The state of one row of a stream, as its thread holds it.
struct RowState {
  bool valid, fresh;  // whether the row exists; whether O holds nothing yet
  int pos;            // the query token's position
  int2 see;           // what it sees
  float slope;        // slope * log2(e)
  float m, l;         // running maximum (log2 units) and sum
};

// Folds NCH x 32 keys of one run (columns col0 .. of the scores t_s) into a row:
// maximum, rescale of O (t_o) where it rises, probabilities over the scores.
template <int D, bool CAP, bool BIAS, int NCH>
__device__ __forceinline__ void fold_run(const ChunkParams& p, RowState& f, uint32_t t_s,
                                         uint32_t t_o, int t0, int col0, int mask) {
  uint32_t sr[NCH][32];
#pragma unroll
  for (int c = 0; c < NCH; ++c) tmem_ld32(t_s + col0 + c * 32, sr[c]);
  tmem_wait_ld();
  float mul = p.qscale;
  if constexpr (CAP || BIAS) {
    mul = 1.f;
    const float d0 = (float)(f.pos - t0 - col0);
    const float cap_z = CAP ? p.scale / p.cap : 0.f, cap_out = p.cap * 1.4426950408889634f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float v = __uint_as_float(sr[c][k]);
        v = CAP ? capped(v, cap_z, cap_out) : v * p.qscale;
        if (BIAS) v = fmaf(-f.slope, fabsf(d0 - (float)(c * 32 + k)), v);
        sr[c][k] = __float_as_uint(v);
      }
  }
  // positions that the row does not see; nothing to mask in most runs
  const int lo = f.see.x - t0, hi = f.see.y - t0;
  const bool dense = mask == 0xff && lo <= col0 && hi >= col0 + 32 * NCH && mul > 0.f;
  if (!__all_sync(kFull, dense)) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int cc = col0 + 32 * c;
      const int a = min(max(lo - cc, 0), 32), b = min(max(hi - cc, 0), 32);
      uint32_t bits = (b == 32 ? ~0u : (1u << b) - 1u) & ~(a == 32 ? ~0u : (1u << a) - 1u);
      const int bm = mask >> (cc / kBlock);
      bits &= ((bm & 1) ? 0xffffu : 0u) | ((bm & 2) ? 0xffff0000u : 0u);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float v = __uint_as_float(sr[c][k]) * mul;
        sr[c][k] = __float_as_uint((bits >> k) & 1u ? v : -INFINITY);
      }
    }
    mul = 1.f;
  }
  float mxs[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    mxs[c] = fmaxf(__uint_as_float(sr[c][0]), __uint_as_float(sr[c][1]));
#pragma unroll
    for (int k = 2; k < 32; k += 2)
      mxs[c] = fmaxf(mxs[c], fmaxf(__uint_as_float(sr[c][k]), __uint_as_float(sr[c][k + 1])));
  }
  float mx = mxs[0];
#pragma unroll
  for (int c = 1; c < NCH; ++c) mx = fmaxf(mx, mxs[c]);
  mx *= mul;
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
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t o[16];
      tmem_ld16(t_o + c * 16, o);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
      tmem_st16(t_o + c * 16, o);
    }
  }
  const float neg = f.m == -INFINITY ? 0.f : -f.m;
  float l0 = 0.f, l1 = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a, b;
      fma2(a, b, __uint_as_float(sr[c][2 * k]), __uint_as_float(sr[c][2 * k + 1]), mul, mul, neg,
           neg);
      a = ex2_approx(a);
      b = ex2_approx(b);
      add2(l0, l1, a, b);
      w[k] = pack_bf16(a, b);
    }
    tmem_st16(t_s + col0 / 2 + c * 16, w);
  }
  if constexpr (NCH < 4) {  // the keys of the other copies
    uint32_t zero[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) zero[k] = 0u;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c * 32 < col0 || c * 32 >= col0 + 32 * NCH) tmem_st16(t_s + c * 16, zero);
  }
  f.l += l0 + l1;
  tmem_wait_st();
}

template <int D, bool CAP, bool BIAS>
__device__ __forceinline__ bool softmax(const ChunkParams& p, const Bars<D>& B, uint32_t smem0,
                                        unsigned char* smem, uint32_t tmem,
                                        const volatile int* s_meta, volatile int* s_merge,
                                        ChunkWalk wk, int warp, int lane) {
  using L = Smem<D>;
  using T = __nv_bfloat16;
  const int x = warp >> 2;                     // stream
  const int r = (warp & 3) * 32 + lane;        // MMA row, TMEM lane
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t t_s = tmem + lane_base + x * kChunkKeys;
  const uint32_t t_o = tmem + lane_base + kColO;
  const int half_tok = p.tile_tokens / 2;
  float2* s_ml = reinterpret_cast<float2*>(smem + L::kOffMl);
  float* s_x = reinterpret_cast<float*>(smem + L::kOffX + x * L::kStreamX);
  uint32_t nscore = 0, nseg = 0, njoin = 0, nmeet = 0, run0 = 0;
  // the stream's four warps meet
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(B.meet(x));
    return warp_wait(B.meet(x), nmeet++ & 1);
  };
  // all eight softmax warps meet
  auto join = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(B.join());
    return warp_wait(B.join(), njoin++ & 1);
  };
  ChunkSegment s, next;
  for (bool more = wk.next(p, s); more; s = next) {
    const int copies = copies_of(p, s);
    const bool pair = copies == 0;
    const int n = s.j1 - s.j0;
    // this thread's row within its half or copy, and its part of a run's keys:
    // nch chunks of 32 columns from col0 on
    const int shift = copies == 4 ? 2 : copies == 2 ? 1 : 0;
    const int copy_rows = kChunkHalfRows >> shift;
    const int copy = r / copy_rows, rc = r - copy * copy_rows;
    const int nch = 4 >> shift, col0 = copy * 32 * nch;
    const int ti = rc / p.group, g = rc - ti * p.group;
    const int tok = (pair && x ? half_tok : 0) + ti;  // query token within the tile
    const bool valid = ti < copy_rows / p.group && tok < s.t.n_tok;
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
    const int step = pair ? 1 : 2;
    for (int j = s.j0 + (pair ? 0 : x); j < s.j1; j += step) {
      const uint32_t run = run0 + (uint32_t)(j - s.j0);
      const int t0 = s.t.kb + j * kChunkKeys;
      if (!warp_wait(B.scores(x), nscore++ & 1)) return false;
      tc_fence_after();
      const int mask = s_meta[run % kMetaRing];
      // Values of positions that hold nothing (past the context, or in a
      // block that was not loaded) become zeros: their probability is 0, but
      // 0 * NaN is not.
      if (mask != 0xff || s.t.ctx - t0 < kChunkKeys) {
        const uint32_t i = 2 * run + 1, slot = i % L::kStages;
        if (!warp_wait(B.full(slot), (i / L::kStages) & 1)) return false;
        if (!((mask >> (r >> 4)) & 1) || r >= s.t.ctx - t0) {
          unsigned char* v = smem + slot * L::kStage + (r >> 3) * (D / 64) * 1024 + (r & 7) * 128;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (any_valid) {
        if (nch == 4)
          fold_run<D, CAP, BIAS, 4>(p, f, t_s, t_o + x * D, t0, col0, mask);
        else if (nch == 2)
          fold_run<D, CAP, BIAS, 2>(p, f, t_s, t_o + x * D, t0, col0, mask);
        else
          fold_run<D, CAP, BIAS, 1>(p, f, t_s, t_o + x * D, t0, col0, mask);
      }
      f.fresh = false;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(B.probs(x));
    }
    run0 += (uint32_t)n;

    more = wk.next(p, next);  // its loads overlap the wait
    // The segment's end: O is complete once its last product is.
    if (!warp_wait(B.out(x), nseg & 1)) return false;
    tc_fence_after();
    const bool whole = s.first && s.last;
    const int row = tok * p.group + g;  // within the tile
    const int slot = chunk_slot(blockIdx.x, s.first);
    // weights of the two streams' O (lane r of both holds the same row where the
    // tile is not a pair), and the row's maximum and sum
    float w0 = 1.f, w1 = 0.f, M = f.m, Lsum = f.l;
    if (!pair) {
      s_ml[x * kChunkHalfRows + r] = make_float2(f.m, f.l);
      if (!join()) return false;
      M = -INFINITY;
      for (int c = 0; c < copies; ++c)
        M = fmaxf(M, fmaxf(s_ml[c * copy_rows + rc].x, s_ml[kChunkHalfRows + c * copy_rows + rc].x));
      Lsum = 0.f;
      auto weight = [&](float mm) { return mm == -INFINITY ? 0.f : ex2_approx(mm - M); };
      for (int c = 0; c < copies; ++c) {
        const float2 a = s_ml[c * copy_rows + rc], b = s_ml[kChunkHalfRows + c * copy_rows + rc];
        Lsum += a.y * weight(a.x) + b.y * weight(b.x);
      }
      w0 = weight(s_ml[r].x);
      w1 = weight(s_ml[kChunkHalfRows + r].x);
    }
    const float inv = whole ? (Lsum > 0.f ? 1.f / Lsum : 0.f) : 1.f;
    T* out = valid ? chunk_out<T>(p, s, row, D) : nullptr;
    // 8 consecutive columns of this thread's row
    auto store8 = [&](int col, const float* v) {
      if (whole) {
        *reinterpret_cast<uint4*>(out + col) =
            make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                       pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
      } else {
        *chunk_acc(p, slot, D, col / 4, row) = make_float4(v[0], v[1], v[2], v[3]);
        *chunk_acc(p, slot, D, col / 4 + 1, row) = make_float4(v[4], v[5], v[6], v[7]);
      }
    };
    // A pair's streams write all columns of their own rows; otherwise each
    // stream takes half of the columns.
    const int c_lo = pair ? 0 : x * (D / 2), c_hi = pair ? D : c_lo + D / 2;
    for (int c = c_lo; c < c_hi; c += 32) {
      uint32_t o[32];
      float v[32];
      tmem_ld32(t_o + (pair ? x * D : 0) + c, o);
      if (!pair && n > 1) {
        uint32_t o1[32];
        tmem_ld32(t_o + D + c, o1);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k)
          v[k] = __uint_as_float(o[k]) * w0 + __uint_as_float(o1[k]) * w1;
      } else {
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]) * w0;
      }
      if (copies <= 1) {
        if (valid) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) store8(c + k, v + k);
        }
        continue;
      }
      // the copies of a row add up; each sums its share of the columns
      if (c > c_lo && !meet()) return false;  // the columns before have been read
      if (valid) {
#pragma unroll
        for (int k = 0; k < 32; ++k) s_x[(copy * 32 + k) * copy_rows + rc] = v[k];
      }
      if (!meet()) return false;
      if (valid) {
        const int share = 32 / copies;
        for (int k0 = copy * share; k0 < (copy + 1) * share; k0 += 8) {
          float sum[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[k] = s_x[(k0 + k) * copy_rows + rc];
          for (int cp = 1; cp < copies; ++cp)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += s_x[(cp * 32 + k0 + k) * copy_rows + rc];
          store8(c + k0, sum);
        }
      }
    }
    if (!whole && valid && (pair || (x == 0 && copy == 0)))
      p.ws_ml[(size_t)slot * p.tile_rows + row] = make_float2(M, Lsum);
    tc_fence_before();
    fence_proxy_async_smem();  // the exchange's bytes may become query rows again
    __syncwarp();
    if (lane == 0) mbar_arrive(B.ofree());
    ++nseg;
    if (!whole) {
      // publish the piece; the CTA whose piece is the last merges them all
      if (!join()) return false;
      if (warp == 0 && lane == 0) {
        __threadfence();
        int* cnt = p.ws_cnt + (size_t)s.tile * p.kv_heads + s.head;
        *s_merge = atomicAdd(cnt, 1) == chunk_pieces(p, wk, s) - 1;
      }
      if (!join()) return false;
      if (*s_merge) {
        __threadfence();
        chunk_merge<T, D, 2 * kStreamWarps * 32>(p, wk, s, threadIdx.x);
      }
    }
  }
  return true;
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) chunk_bf16_kernel(
    const __grid_constant__ ChunkParams p) {
  using L = Smem<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t smem0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars<D> B{smem0 + L::kOffBars};
  volatile int* s_meta = reinterpret_cast<volatile int*>(smem + L::kOffMeta);
  volatile uint32_t* s_words = reinterpret_cast<volatile uint32_t*>(smem + L::kOffWords);
  if (smem0 & 1023u) {  // the swizzled operands need it; never seen
    if (threadIdx.x == 0) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
    return;
  }
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2 * L::kStages + 2; ++i) mbar_init(smem0 + L::kOffBars + 8 * i, 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(B.scores(x), 1);
        mbar_init(B.probs(x), kStreamWarps);
        mbar_init(B.out(x), 1);
        mbar_init(B.meet(x), kStreamWarps);
      }
      mbar_init(B.ofree(), 2 * kStreamWarps);
      mbar_init(B.join(), 2 * kStreamWarps);
      mbar_init(B.drained(), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(smem + L::kOffWords), kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_words[0];
  griddep_wait();  // the tile list, and whatever was written before it
  ChunkWalk wk;
  wk.init(p, blockIdx.x, lane);
  bool ok = true;
  if (warp < 8) {
    regs_raise<kRegsSoftmax>();
    ok = softmax<D, CAP, BIAS>(p, B, smem0, smem, tmem, s_meta,
                               reinterpret_cast<volatile int*>(smem + L::kOffWords) + 2, wk, warp,
                               lane);
  } else {
    regs_drop<kRegsOther>();
  }
  if (warp == 8) {
    uint32_t i = 0, nq = 0;
    ok = produce<D>(p, B, smem0, s_meta, wk, lane, i, nq);
    // every copy issued lands before the CTA can end, even after a timeout
    for (uint32_t k = i > (uint32_t)L::kStages ? i - L::kStages : 0; k < i; ++k)
      (void)mbar_wait(B.full(k % L::kStages), (k / L::kStages) & 1);
    if (nq) (void)mbar_wait(B.qfull(), (nq - 1) & 1);
  } else if (warp == 9) {
    ok = issue_mma<D>(p, B, smem0, tmem, wk, lane == 0);
    umma_commit(B.drained(), lane == 0);  // arrives once every MMA issued is done
    (void)mbar_wait(B.drained(), 0);
  }
  if (!ok && lane == 0) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch_one(const ChunkParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_bf16_kernel<D, CAP, BIAS>, p);
}

template <int D>
cudaError_t launch_dim(const ChunkParams& p, int grid, cudaStream_t stream) {
  const bool cap = p.cap > 0.f, bias = p.slopes != nullptr;
  return cap ? (bias ? launch_one<D, true, true>(p, grid, stream)
                     : launch_one<D, true, false>(p, grid, stream))
             : (bias ? launch_one<D, false, true>(p, grid, stream)
                     : launch_one<D, false, false>(p, grid, stream));
}

template <int D, bool CAP, bool BIAS>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(chunk_bf16_kernel<D, CAP, BIAS>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
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

cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, int grid, cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64>(p, grid, stream) : launch_dim<128>(p, grid, stream);
}

}  // namespace nsv
