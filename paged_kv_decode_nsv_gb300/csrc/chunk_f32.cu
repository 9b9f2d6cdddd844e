// Attention of a chunk of new tokens over a paged cache, fp32, on the
// 5th-generation tensor cores (see chunk_bf16.cu for the formulas).
//
// Both products run at fp32's precision with each factor as a sum of two tf32
// numbers: x = hi + lo, hi rounded to tf32's 11 bits, and of lo = x - hi, which is
// exact, the MMA takes the upper 11.  a b = a_hi b_hi + a_hi b_lo + a_lo b_hi: what
// is left out, a_lo b_lo, is at most 2^-22 of the product, and what the MMA drops of
// a lo 2^-21 of x.
//
// The tensor core's accumulator does not round: it drops what the sum does not hold.
// Left to it for a whole row, sums over 8192 positions came out 6e-6 to 2e-5 too small.
// So each run's products start from zero, and the softmax threads add them up in
// registers, rounded to nearest; the sum of the probabilities is compensated (it has more
// terms, and equal ones round the same way each time).  Against 64 bits
// the outputs are off by 2e-7 to 6e-7 (a plain fp32 computation: 1.3e-7 to 9e-7); means of
// values near 3 with nearly equal weights, in rows that one CTA holds whole, by at most
// 9e-7 over 8192 positions and 2.6e-6 over 131072.
//
// One CTA per SM, twenty warps (the last two idle):
//   warps 0-7   softmax: MMA row r (TMEM lane r) belongs to two threads, in warps
//               w and w + 4, which split its 64 scores and its output's columns
//   warps 8-15  loaders, four for the keys, four for the values, all for the query
//               rows: from global memory into registers (half of a run at head_dim 128
//               into shared memory), a run ahead; split, and stored as MMA operands
//   warp 16     MMA issue, one elected thread
//   warp 17     publishes the pieces of cut tiles
// The rows of an MMA are the tile's query tokens times the query heads that share
// the KV head.  All operands are K-major with a 128-byte swizzle, panels of 32
// elements (128 bytes) of K: query rows and keys by dims, values by keys, so the
// loaders transpose the values: a thread loads 4 dims of 4 keys and stores 4 keys
// of 4 dims.  Column n of O is dim 4 (n % (D/4)) + n / (D/4): with it, the stores
// of neighbouring lanes go to neighbouring rows, and hit all banks.
//
// Tensor memory (512 columns): scores of run j at 128 (j % 2), 64 columns, then the
// upper parts of its probabilities in their place; their lower parts in the next 64;
// O at 256; the lower parts of the query rows at 384.  (Their upper parts are in
// shared memory: 192 KiB hold them and one run's keys and values, at head_dim 64 two
// runs'.)  Scores of run j + 1 are issued before the products of run j's
// probabilities, so that each softmax runs while the tensor core works.
//
// A run of 64 positions takes 2.8 us at head_dim 128 and 1.5 to 1.6 at 64 whatever the
// rows; its MMAs alone would take 1.7 and 0.9, its bytes 1.5 and 0.7.  Nothing is far
// ahead: without the global loads or the softmax it takes 2.6 (head_dim 128), because a
// buffer of keys holds one run, which is stored after the scores before it are done and
// before the next can start.  638 tokens over up to 2048 positions, 12 heads: 65 us (56
// when the accumulator kept the sums).  The same split on mma.sync (64 rows, two CTAs per
// SM), where every warp splits the keys and values again, took 162, and multiply-adds on
// the CUDA cores 207.
//
// Over a 4-bit cache (KV4): a loader's registers hold four numbers and their scale, whose
// products are exact in tf32, so that keys and values have no lower parts: two products
// instead of three, and buffers of two runs.  The heads' scales go to the scores' scale and
// to the outputs' last factor.

#include "chunk.cuh"
#include "kv4.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kSoftWarps = 8, kLoadWarps = 8;
constexpr int kThreadsF32 = (kSoftWarps + kLoadWarps + 4) * 32;  // two warps are idle
// Registers of a thread: at launch (what 640 threads get), and as the roles share them
// (with 96 for all, what spilled in the loops cost half as much again).  At head_dim 128
// 112 and 88 or 104 and 96 are as fast as 120 and 80.
constexpr int kRegs = 96, kOtherRegs = 80;
template <int D>
struct Regs {
  static constexpr int kSoft = D == 128 ? 120 : 104, kLoad = D == 128 ? 80 : 96;
  static_assert(kSoftWarps * kSoft + kLoadWarps * kLoad + 4 * kOtherRegs <=
                    (kSoftWarps + kLoadWarps + 4) * kRegs,
                "more registers than the launch has would be waited for without end");
};
constexpr int kR = kChunkRowsF32, kC = kChunkKeysF32;
constexpr uint32_t kColO = 256, kColQ = 384;
constexpr int kTmemCols = 512;
constexpr int kMetaRing = 8;
// The running maximum is raised only when a run exceeds it by more than this (log2
// units): probabilities stay <= 2^8, and most runs skip the rescale.
constexpr float kSlack = 8.f;

// (What a 4-bit cache holds is exact in tf32 and has no lower parts.)
template <int D, bool KV4>
struct Smem {
  static constexpr uint32_t kQ = kR * D * 4;  // upper parts of the query rows
  static constexpr uint32_t kKV = kC * D * 4;  // upper or lower parts of a run's keys or values
  static constexpr uint32_t kRun = (KV4 ? 1 : 2) * kKV;
  // runs that the keys' and the values' buffers hold
  static constexpr uint32_t kStages = D == 64 || KV4 ? 2 : 1;
  static constexpr uint32_t kOffK = kQ;
  static constexpr uint32_t kOffV = kOffK + kStages * kRun;
  // Of a loader's 16 or 8 chunks of a run, on their way those it has no registers for
  // wait here: [loaders][chunks][128 threads] of 16 bytes.
  static constexpr int kHeld = D == 64 || KV4 ? 0 : 8;
  static constexpr uint32_t kOffHeld = kOffV + kStages * kRun;
  static constexpr uint32_t kOffMax = kOffHeld + kHeld * kLoadWarps * 32 * 16;  // float2 [128]
  static constexpr uint32_t kOffSum = kOffMax + kR * 8;   // float [2][128]
  static constexpr uint32_t kOffTodo = kOffSum + kR * 8;  // int4 [2][2]: tiles to merge
  static constexpr uint32_t kOffBars = kOffTodo + 64;
  static constexpr int kBars = 20;
  static constexpr uint32_t kOffMeta = kOffBars + kBars * 8 + 8;
  static constexpr uint32_t kOffPairs = kOffMeta + kMetaRing * 4;  // PairWords [4]
  static constexpr uint32_t kOffWord = kOffPairs + 4 * 20;         // the TMEM address
  // (at least half of an SM's, so that no two CTAs share its tensor memory)
  static constexpr uint32_t kUsed = kOffWord + 16;
  static constexpr uint32_t kTotal = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

struct Bars {
  uint32_t b;
  __device__ uint32_t at(uint32_t i) const { return b + 8 * i; }
  __device__ uint32_t kfull(uint32_t i) const { return at(i); }  // i: the run's stage
  __device__ uint32_t kempty(uint32_t i) const { return at(2 + i); }
  __device__ uint32_t vfull(uint32_t i) const { return at(4 + i); }
  __device__ uint32_t vempty(uint32_t i) const { return at(6 + i); }  // also: O holds its products
  __device__ uint32_t scores(uint32_t x) const { return at(8 + x); }
  __device__ uint32_t probs(uint32_t x) const { return at(10 + x); }
  __device__ uint32_t qfull() const { return at(12); }
  __device__ uint32_t qfree() const { return at(13); }
  __device__ uint32_t oread() const { return at(14); }
  __device__ uint32_t piece(int first) const { return at(first ? 19 : 16); }
  __device__ uint32_t published() const { return at(17); }
  __device__ uint32_t drained() const { return at(18); }
};

// x = hi + lo: hi rounded to tf32 (to nearest, ties away from zero), lo exact.  (Rounded
// too, lo leaves the outputs as far off and costs 4 us of 60.)
__device__ __forceinline__ float to_tf32(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
}
__device__ __forceinline__ float4 hi4(float4 x) {
  return make_float4(to_tf32(x.x), to_tf32(x.y), to_tf32(x.z), to_tf32(x.w));
}
__device__ __forceinline__ float4 lo4(float4 x, float4 h) {
  return make_float4(x.x - h.x, x.y - h.y, x.z - h.z, x.w - h.w);
}

// 16 bytes global -> shared, asynchronously; zeros where there is nothing.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N < 0 ? 0 : N) : "memory");
}

// Byte offset of 16-byte chunk v of row r of an operand with `rows` rows.
__device__ __forceinline__ uint32_t operand_at(int rows, int r, int v) {
  return (uint32_t)((v >> 3) * rows * 128 + r * 128 + (((v ^ r) & 7) << 4));
}

// -------------------------------------------------------------------- loaders
// Four warps load the keys (KEYS) and four the values, each for itself, so that the
// keys of a run are stored during products and its values during scores.  (Eight warps
// for both in turn: 5.7 us a run instead of 3.7.)
template <int D, bool KEYS, bool KV4>
__device__ __forceinline__ bool load(const ChunkArgs<KV4>& p, const Bars& B, unsigned char* smem,
                                     volatile int* s_meta, ChunkWalk wk, int warp, int lane) {
  using L = Smem<D, KV4>;
  constexpr int kV = D / 4;                   // 16-byte chunks of a key
  constexpr int kT = kLoadWarps * 32 / 2;     // threads that share a run
  constexpr int kN = kC * kV / kT;            // a thread's chunks of a run: 16 or 8
  constexpr int kStep = kT / kV;              // keys (or quads of them) between a thread's: 4 or 8
  constexpr int kSame = KEYS ? kBlock / kStep : 4;  // consecutive ones within a block
  constexpr int kHeld = L::kHeld;
  const int tid = (warp & 3) * 32 + lane;
  const int v = tid & (kV - 1), t1 = tid / kV;  // its chunk, and its first key or quad
  constexpr int kQueries = 8;                 // chunks of a query row at a time
  static_assert(KV4 || kN - kHeld == kQueries, "the registers of a run's chunks");
  const float* pool = static_cast<const float*>(KEYS ? p.k_pool : p.v_pool);
  uint32_t run = 0, nseg = 0;
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kC>(p, s)) {
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    // Lane l's block of run j (l < 4), -1 past the tile's keys.  Whether it is a good
    // one is looked at where it is used: here the warp would wait for it.
    auto wanted = [&](int j) {
      return j < s.j1 && lane < kC / kBlock &&
             (long long)s.t.kb + (long long)j * kC + lane * kBlock < s.t.ke;
    };
    auto block_ids = [&](int j) {
      return wanted(j) ? __ldg(table + (s.t.kb + j * kC) / kBlock + lane) : -1;
    };
    float4 x[kQueries];       // of a query row; of a run, chunks kHeld and on
    uint32_t raw[KV4 ? kN : 1];  // a 4-bit cache: four numbers, and their scale above them
    unsigned char* held = smem + L::kOffHeld + ((KEYS ? 0 : kHeld) * kT + tid) * 16;
    // This thread's chunks i .. i + kSame - 1 of run j, on their way.  (One group of
    // copies for each part that is held, whether it has any or not.)
    auto fetch = [&](int i, int ids, int j) {
      const int left = s.t.ke - (s.t.kb + j * kC);  // positions from the run's start on
      const int t = KEYS ? t1 + i * kStep : 4 * (t1 + (i >> 2) * kStep);
      const int id = __shfl_sync(kFull, ids, t / kBlock);
      const bool ok = id >= 0 && id < p.pool_blocks;
      if constexpr (KV4) {
        const uint8_t* tile = (KEYS ? p.k4 : p.v4) +
                              ((size_t)(ok ? id : 0) * p.kv_heads + s.head) * kv4_tile_bytes(D);
#pragma unroll
        for (int u = 0; u < kSame; ++u) {
          const int dt = KEYS ? u * kStep : u, off = t % kBlock + dt;
          raw[i + u] = 0;
          if (ok && t + dt < left)
            raw[i + u] = __ldg(reinterpret_cast<const uint16_t*>(tile + off * (D / 2)) + v) |
                         (uint32_t)__ldg(tile + 8 * D + off * (D / 16) + v / 4) << 16;
        }
        return;
      }
      const float4* at = reinterpret_cast<const float4*>(
          pool + (((size_t)(ok ? id : 0) * p.kv_heads + s.head) * kBlock + t % kBlock) * D) + v;
#pragma unroll
      for (int u = 0; u < kSame; ++u) {
        const int dt = KEYS ? u * kStep : u;
        const bool there = ok && t + dt < left;
        if (i < kHeld) {
          copy16(held + (i + u) * kT * 16, at + dt * kV, there);
        } else {
          x[i + u - kHeld] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (there) x[i + u - kHeld] = __ldg(at + dt * kV);
        }
      }
    };
    auto chunk = [&](int i) {
      if constexpr (KV4) {
        uint32_t h[4];
        e2m1x8_to_half(raw[i], h);  // (of which two are numbers)
        const uint32_t e = __byte_perm(e4m3x2_to_half(raw[i] >> 16), 0, 0x1010);
        h[0] = hmul2(h[0], e);
        h[1] = hmul2(h[1], e);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
        return make_float4(a.x, a.y, b.x, b.y);
      } else
      return i < kHeld ? *reinterpret_cast<const float4*>(held + i * kT * 16) : x[i - kHeld];
    };
    int ids = block_ids(s.j0), ids_next = block_ids(s.j0 + 1);

#pragma unroll
    for (int i = 0; i < kHeld; i += kSame) {
      fetch(i, ids, s.j0);
      copies_commit();
    }

    // The query rows: this thread's row, half of its dims, as many at a time as there
    // are registers; then the first run takes them.
    const int r = (warp & 3) * 32 + lane, half = warp >> 2;
    const int tok = (int)((unsigned)r / (unsigned)p.group), g = r - tok * p.group;
    const bool valid = tok < s.t.n_tok;
    const float4* q = static_cast<const float4*>(p.q) +
                      (((size_t)s.t.q0 + (valid ? tok : 0)) * p.heads + s.head * p.group + g) * kV +
                      half * kN;
    static_assert(kN == kV / 2, "a thread's part of a query row");
    const uint32_t t_q = ((uint32_t)((warp & 3) * 32) << 16) + kColQ + half * (D / 2);
#pragma unroll
    for (int b = 0; b < kN; b += kQueries) {
#pragma unroll
      for (int i = 0; i < kQueries; ++i) {
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid) x[i] = __ldg(q + b + i);
      }
      if (b == 0) {
        if (nseg && !warp_wait(B.qfree(), (nseg - 1) & 1)) return false;
        tc_fence_after();
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kQueries; i += 2) {
        float lo[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 h = hi4(x[i + k]), l = lo4(x[i + k], h);
          *reinterpret_cast<float4*>(smem + operand_at(kR, r, half * kN + b + i + k)) = h;
          lo[4 * k] = l.x, lo[4 * k + 1] = l.y, lo[4 * k + 2] = l.z, lo[4 * k + 3] = l.w;
        }
        tmem_st8(t_q + 4 * (b + i), lo);
      }
    }
#pragma unroll
    for (int i = kHeld; i < kN; i += kSame) fetch(i, ids, s.j0);
    tmem_wait_st();
    tc_fence_before();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(B.qfull());
    ++nseg;
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j, ++run) {
      const int ids_after = block_ids(j + 2);
      const uint32_t st = run % L::kStages;
      unsigned char* dst = smem + (KEYS ? L::kOffK : L::kOffV) + st * L::kRun;
      const uint32_t empty = KEYS ? B.kempty(st) : B.vempty(st);
      if (!warp_wait(empty, ((run / L::kStages) & 1) ^ 1)) return false;
      if (KEYS && warp == 0) {
        const bool good = ids >= 0 && ids < p.pool_blocks;
        const unsigned ok = __ballot_sync(kFull, good);
        if (!good && wanted(j)) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_BLOCK);
        if (lane == 0) s_meta[run % kMetaRing] = (int)ok;
      }
      // (each part's next load starts as soon as its registers are free)
      const bool more = j + 1 < s.j1;
#pragma unroll
      for (int i = 0; i < kN; i += kSame) {
        if (i < kHeld) copies_wait<kHeld / kSame - 1>();  // all groups but the later parts'
        if (KEYS) {
#pragma unroll
          for (int u = 0; u < kSame; ++u) {
            unsigned char* at = dst + operand_at(kC, t1 + (i + u) * kStep, v);
            const float4 y = chunk(i + u), h = KV4 ? y : hi4(y);
            *reinterpret_cast<float4*>(at) = h;
            if (!KV4) *reinterpret_cast<float4*>(at + L::kKV) = lo4(y, h);
          }
        } else {
          // 4 keys of dims 4 v .. 4 v + 3, rows v, v + D/4, ... of the operand
          const float4 a = chunk(i), b = chunk(i + 1), c = chunk(i + 2), d = chunk(i + 3);
          const float4 y[4] = {make_float4(a.x, b.x, c.x, d.x), make_float4(a.y, b.y, c.y, d.y),
                               make_float4(a.z, b.z, c.z, d.z), make_float4(a.w, b.w, c.w, d.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            unsigned char* at = dst + operand_at(D, e * kV + v, t1 + (i >> 2) * kStep);
            const float4 h = KV4 ? y[e] : hi4(y[e]);
            *reinterpret_cast<float4*>(at) = h;
            if (!KV4) *reinterpret_cast<float4*>(at + L::kKV) = lo4(y[e], h);
          }
        }
        if (more) fetch(i, ids_next, j + 1);
        if (i < kHeld) copies_commit();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(KEYS ? B.kfull(st) : B.vfull(st));
      ids = ids_next;
      ids_next = ids_after;
    }
  }
  return warp_wait(B.published(), 0);
}

// ------------------------------------------------------------------------ MMA
template <int D, bool KV4>
__device__ __forceinline__ bool issue_mma(const ChunkParams& p, const Bars& B, uint32_t smem0,
                                          ChunkWalk wk) {
  using L = Smem<D, KV4>;
  constexpr uint32_t idesc_s = umma_idesc_tf32(kR, kC), idesc_o = umma_idesc_tf32(kR, D);
  // (descriptors are linear in the start address: lower parts follow the upper ones)
  const uint64_t dq = umma_desc128(smem0, 16, 1024);
  const uint64_t dk0 = umma_desc128(smem0 + L::kOffK, 16, 1024);
  const uint64_t dv0 = umma_desc128(smem0 + L::kOffV, 16, 1024);
  constexpr uint64_t kLow = L::kKV >> 4;
  // offset of K step ks (8 elements) of an operand with `rows` rows
  auto step = [](int rows, int ks) {
    return (uint64_t)(((ks >> 2) * rows * 128 + (ks & 3) * 32) >> 4);
  };
  uint32_t run = 0, nseg = 0;
  auto scores = [&](uint32_t i) {
    const uint32_t st = i % L::kStages;
    if (!mbar_wait(B.kfull(st), (i / L::kStages) & 1)) return false;
    tc_fence_after();
    const uint32_t d = (i & 1) * 128;
    const uint64_t dk = dk0 + st * (L::kRun >> 4);
#pragma unroll
    for (int ks = 0; ks < D / 8; ++ks)
      umma_ts_tf32(d, kColQ + ks * 8, dk + step(kC, ks), idesc_s, ks > 0);
#pragma unroll
    for (int ks = 0; !KV4 && ks < D / 8; ++ks)
      umma_ss_tf32(d, dq + step(kR, ks), dk + kLow + step(kC, ks), idesc_s, true);
#pragma unroll
    for (int ks = 0; ks < D / 8; ++ks)
      umma_ss_tf32(d, dq + step(kR, ks), dk + step(kC, ks), idesc_s, true);
    umma_commit(B.kempty(st), true);
    umma_commit(B.scores(i & 1), true);
    return true;
  };
  auto values = [&](uint32_t i) {
    const uint32_t st = i % L::kStages;
    const uint64_t dv = dv0 + st * (L::kRun >> 4);
    if (!mbar_wait(B.vfull(st), (i / L::kStages) & 1)) return false;
    if (!mbar_wait(B.probs(i & 1), (i >> 1) & 1)) return false;
    if (i && !mbar_wait(B.oread(), (i - 1) & 1)) return false;
    tc_fence_after();
    const uint32_t a = (i & 1) * 128;
#pragma unroll
    for (int ks = 0; ks < kC / 8; ++ks)
      umma_ts_tf32(kColO, a + kC + ks * 8, dv + step(D, ks), idesc_o, ks > 0);
#pragma unroll
    for (int ks = 0; !KV4 && ks < kC / 8; ++ks)
      umma_ts_tf32(kColO, a + ks * 8, dv + kLow + step(D, ks), idesc_o, true);
#pragma unroll
    for (int ks = 0; ks < kC / 8; ++ks)
      umma_ts_tf32(kColO, a + ks * 8, dv + step(D, ks), idesc_o, true);
    umma_commit(B.vempty(st), true);
    return true;
  };
  ChunkSegment s, next;
#pragma unroll 1
  for (bool more = wk.next<kC>(p, s); more; s = next) {
    const int n = s.j1 - s.j0;
    more = wk.next<kC>(p, next);  // its loads overlap this segment's work
    if (!mbar_wait(B.qfull(), nseg & 1)) return false;
#pragma unroll 1
    for (int j = -1; j < n; ++j) {
      if (j + 1 < n) {
        if (!scores(run + j + 1)) return false;
        if (j + 2 == n) umma_commit(B.qfree(), true);
      }
      if (j >= 0 && !values(run + j)) return false;
    }
    run += n;
    ++nseg;
  }
  return true;
}

// -------------------------------------------------------------------- softmax
template <int D, bool CAP, bool KV4>
__device__ __forceinline__ int softmax(const ChunkArgs<KV4>& p, const Bars& B, unsigned char* smem,
                                       const volatile int* s_meta, int4* s_todo,
                                       volatile PairWords* words, ChunkWalk wk, int warp,
                                       int lane) {
  using L = Smem<D, KV4>;
  constexpr int kH = kC / 2;  // this thread's scores of a run
  constexpr float kLog2e = 1.4426950408889634f;
  const int hf = warp >> 2;                  // which of the pair
  const int r = (warp & 3) * 32 + lane;      // MMA row, TMEM lane
  const int bar = 1 + (warp & 3);            // the pair's barrier
  const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t t_o = t_lane + kColO;
  const int tok = (int)((unsigned)r / (unsigned)p.group), g = r - tok * p.group;
  volatile float2* s_max = reinterpret_cast<volatile float2*>(smem + L::kOffMax) + r;
  volatile float* s_sum = reinterpret_cast<volatile float*>(smem + L::kOffSum) + r;
  uint32_t run = 0, turn = 0;
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kC>(p, s)) {
    const bool valid = tok < s.t.n_tok;
    const bool any_valid = __any_sync(kFull, valid);
    const int pos = s.t.pos0 + tok;
    const int2 see = valid ? chunk_sees(p, (long long)s.t.q0 + tok, pos, s.t.ctx)
                           : make_int2(0, 0x7fffffff);  // rows that are not there mask nothing
    const float slope = valid && p.slopes ? __ldg(p.slopes + s.head * p.group + g) : 0.f;
    float m = -INFINITY, l = 0.f, lc = 0.f;  // lc: by how much l is too large
    float acc[4][D / 8];  // dims 4 v + e of this thread's half of the v
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < D / 8; ++k) acc[e][k] = 0.f;
    // Adds the products of run i, which O holds, once they are complete.
    auto add_products = [&](uint32_t i) {
      if (!warp_wait(B.vempty(i % L::kStages), (i / L::kStages) & 1)) return false;
      if (any_valid) {
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float o[D / 8];
#pragma unroll
          for (int k = 0; k < D / 8; k += 8)
            tmem_ld8(t_o + e * (D / 4) + hf * (D / 8) + k, o + k);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < D / 8; ++k) acc[e][k] += o[k];
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(B.oread());
      return true;
    };
    const float scale = p.scale * k_unit(p, s.head);
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j, ++run) {
      const uint32_t t_s = t_lane + (run & 1) * 128 + hf * kH;
      const int t0 = s.t.kb + j * kC;
      if (!warp_wait(B.scores(run & 1), (run >> 1) & 1)) return kTimedOut;
      tc_fence_after();
      float alpha = 1.f;
      if (any_valid) {
        float mul = scale;
        if (CAP) {
#pragma unroll 1
          for (int c = 0; c < kH; c += 8) {
            float x[8];
            tmem_ld8(t_s + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = p.cap * tanhf(x[k] * scale / p.cap);
            tmem_st8(t_s + c, x);
          }
          tmem_wait_st();
          mul = 1.f;
        }
        float x[kH];
        tmem_ld32(t_s, x);
        tmem_wait_ld();
        const int d = pos - t0 - hf * kH;
#pragma unroll
        for (int k = 0; k < kH; ++k) {
          x[k] *= mul;
          if (p.slopes) x[k] = fmaf(-slope, fabsf((float)(d - k)), x[k]);
          x[k] *= kLog2e;
        }
        // what the row does not see; nothing in most runs
        const int lo = min(max(see.x - t0 - hf * kH, 0), kH);
        const int hi = min(max(see.y - t0 - hf * kH, 0), kH);
        const int blocks = s_meta[run % kMetaRing] >> (hf * kH / kBlock);
        uint32_t bits = (hi == 32 ? kFull : (1u << hi) - 1u) & (lo == 32 ? 0u : kFull << lo);
        bits &= (blocks & 1 ? 0xffffu : 0u) | (blocks & 2 ? 0xffff0000u : 0u);
        if (!__all_sync(kFull, bits == kFull)) {
#pragma unroll
          for (int k = 0; k < kH; ++k) x[k] = (bits >> k) & 1u ? x[k] : -INFINITY;
        }
        float mx = x[0], m1 = x[1];
#pragma unroll
        for (int k = 2; k < kH; k += 2) {
          mx = fmaxf(mx, x[k]);
          m1 = fmaxf(m1, x[k + 1]);
        }
        mx = fmaxf(mx, m1);
        // Both warps learn which rows exceed the running maximum; in most runs none
        // does, and the maxima themselves need no exchange.
        const uint32_t mine = __ballot_sync(kFull, valid && mx > m + kSlack);
        if (lane == 0) words->raise[turn & 1][hf] = mine;
        if (!pair_sync(bar, words)) return kPartnerFailed;
        if (mine | words->raise[turn & 1][hf ^ 1]) {
          (hf ? s_max->y : s_max->x) = mx;
          if (!pair_sync(bar, words)) return kPartnerFailed;
          mx = fmaxf(mx, hf ? s_max->x : s_max->y);
          const bool raise = valid && mx > m + kSlack;  // also the first finite one
          if (raise) {
            alpha = ex2_approx(m - mx);
            m = mx;
            l *= alpha;
            lc *= alpha;
          }
        }
        ++turn;
        const float sub = m == -INFINITY ? 0.f : m;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < kH; c += 8) {
          float low[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float e = ex2_approx(x[c + k] - sub);
            (k & 1 ? l1 : l0) += e;
            x[c + k] = to_tf32(e);
            low[k] = e - x[c + k];
          }
          tmem_st8(t_s + c, x + c);
          tmem_st8(t_s + kC + c, low);
        }
        // (Kahan's summation.  One by one, without it, a sum over 32768 positions was up
        // to 1.7e-4 off; it costs single tokens at head_dim 128 1 %, chunks nothing.)
        const float add = l0 + l1 - lc, sum = l + add;
        lc = (sum - l) - add;
        l = sum;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(B.probs(run & 1));
      // While the tensor core goes on: the run before, still at the old maximum.
      if (j > s.j0 && !add_products(run - 1)) return kTimedOut;
      if (__any_sync(kFull, alpha != 1.f)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < D / 8; ++k) acc[e][k] *= alpha;
      }
    }
    if (!add_products(run - 1)) return kTimedOut;
    const bool whole = s.first && s.last;
    if (any_valid) {
      s_sum[hf * kR] = l;
      if (!pair_sync(bar, words)) return kPartnerFailed;
      l += s_sum[(hf ^ 1) * kR];
      const int slot = chunk_slot(blockIdx.x, s.first);
      const int row = tok * p.group + g;  // within the tile
      const float w = (whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f) *
                      v_unit(p, s.head);
      float* out = chunk_out<float>(p, s.t.q0, s.head, row, D);
      if (valid) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const int v = hf * (D / 8) + k;
          *(whole ? reinterpret_cast<float4*>(out) + v : chunk_acc(p, slot, D, v, row)) =
              make_float4(acc[0][k] * w, acc[1][k] * w, acc[2][k] * w, acc[3][k] * w);
        }
      }
      if (!whole && valid && hf == 0)
        p.ws_ml[(size_t)slot * p.tile_rows + row] = make_float2(m, l);
    }
    __syncwarp();
    if (lane == 0 && !whole) mbar_arrive(B.piece(s.first));
  }
  return warp_wait(B.published(), 0) ? kDone : kTimedOut;
}

template <int D, bool CAP, bool KV4>
__global__ void __launch_bounds__(kThreadsF32, 1) chunk_f32_kernel(
    const __grid_constant__ ChunkArgs<KV4> p) {
  using L = Smem<D, KV4>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t smem0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars B{smem0 + L::kOffBars};
  volatile int* s_meta = reinterpret_cast<volatile int*>(smem + L::kOffMeta);
  volatile PairWords* s_pairs = reinterpret_cast<volatile PairWords*>(smem + L::kOffPairs);
  volatile uint32_t* s_word = reinterpret_cast<volatile uint32_t*>(smem + L::kOffWord);
  int4* s_todo = reinterpret_cast<int4*>(smem + L::kOffTodo);
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(B.qfull(), kLoadWarps);
      mbar_init(B.qfree(), 1);
      for (uint32_t x = 0; x < 2; ++x) {
        mbar_init(B.kfull(x), kLoadWarps / 2);
        mbar_init(B.kempty(x), 1);
        mbar_init(B.vfull(x), kLoadWarps / 2);
        mbar_init(B.vempty(x), 1);
        mbar_init(B.scores(x), 1);
        mbar_init(B.probs(x), kSoftWarps);
      }
      mbar_init(B.oread(), kSoftWarps);
      mbar_init(B.piece(0), kSoftWarps);
      mbar_init(B.piece(1), kSoftWarps);
      mbar_init(B.published(), 1);
      mbar_init(B.drained(), 1);
      fence_mbar_init();
      for (int i = 0; i < 4; ++i) s_pairs[i].failed = 0;
      for (int i = 0; i < 4; ++i) s_todo[i] = make_int4(0, 0, 0, 0);
    }
    __syncwarp();
    tmem_alloc(smem_u32(smem + L::kOffWord), kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // What the code takes for granted (never seen otherwise): the swizzled operands'
  // alignment, and that all of tensor memory starts at column 0.
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
    reg_inc<Regs<D>::kSoft>();
    volatile PairWords* words = s_pairs + (warp & 3);
    const int end = softmax<D, CAP, KV4>(p, B, smem, s_meta, s_todo, words, wk, warp, lane);
    // Every warp but one whose partner failed meets its partner once more: so a
    // partner that still works learns of a timeout at its next meeting, and none
    // is left waiting.
    if (end != kPartnerFailed) {
      if (end == kTimedOut) words->failed = 1;
      __syncwarp();
      (void)pair_sync(1 + (warp & 3), words);
    }
    ok = end == kDone;
  } else if (warp < kSoftWarps + kLoadWarps) {
    reg_dec<Regs<D>::kLoad>();
    ok = warp < kSoftWarps + kLoadWarps / 2
             ? load<D, true, KV4>(p, B, smem, s_meta, wk, warp - kSoftWarps, lane)
             : load<D, false, KV4>(p, B, smem, s_meta, wk, warp - kSoftWarps, lane);
  } else {
    reg_dec<kOtherRegs>();
    if (warp == kSoftWarps + kLoadWarps) {
      if (elect_one()) {
        ok = issue_mma<D, KV4>(p, B, smem0, wk);
        if (!ok) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
        umma_commit(B.drained(), true);  // arrives once every MMA issued is done
        (void)mbar_wait(B.drained(), 0);
      }
      __syncwarp();
    } else if (warp == kSoftWarps + kLoadWarps + 1) {
      ok = chunk_publish<kC>(p, B.piece(0), B.piece(1), B.published(), s_todo, wk, lane);
    }
  }
  if (ok && warp < kSoftWarps + kLoadWarps)
    chunk_merge_todo<float, D, (kSoftWarps + kLoadWarps) * 32>(p, s_todo);
  if (!ok && lane == 0) atomicOr(p.status, (uint32_t)NSV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool CAP, bool KV4>
cudaError_t launch_one(const ChunkArgs<KV4>& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kThreadsF32);
  cfg.dynamicSmemBytes = Smem<D, KV4>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_f32_kernel<D, CAP, KV4>, p);
}

template <bool KV4>
cudaError_t launch_dim(const ChunkArgs<KV4>& p, int head_dim, cudaStream_t stream) {
  const bool cap = p.cap > 0.f;
  if (head_dim == 64)
    return cap ? launch_one<64, true, KV4>(p, stream) : launch_one<64, false, KV4>(p, stream);
  return cap ? launch_one<128, true, KV4>(p, stream) : launch_one<128, false, KV4>(p, stream);
}

template <int D, bool CAP, bool KV4>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(chunk_f32_kernel<D, CAP, KV4>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, KV4>::kTotal);
}

template <int D>
cudaError_t set_attrs() {
  cudaError_t e;
  if ((e = set_attr<D, false, false>()) != cudaSuccess) return e;
  if ((e = set_attr<D, true, false>()) != cudaSuccess) return e;
  if ((e = set_attr<D, false, true>()) != cudaSuccess) return e;
  return set_attr<D, true, true>();
}

}  // namespace

cudaError_t prepare_chunk_f32() {
  const cudaError_t e = set_attrs<64>();
  return e != cudaSuccess ? e : set_attrs<128>();
}

cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t stream) {
  return launch_dim<false>(p, head_dim, stream);
}

cudaError_t launch_chunk_kv4_f32(const Chunk4Params& p, int head_dim, cudaStream_t stream) {
  return launch_dim<true>(p, head_dim, stream);
}

}  // namespace nsv
