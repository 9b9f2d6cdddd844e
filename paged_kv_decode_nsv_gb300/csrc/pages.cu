// Page operators of the paged cache: copying blocks, forking, extending and
// freeing rows, compacting the pool.
//
// The allocator's whole state is one reference count per block (the number of
// block-table entries that name it; 0: free), in device memory beside the
// tables and lengths, so that every operator runs in stream order, is captured
// into graphs, and gives the same result every time: free blocks are always
// dealt out lowest id first, to the rows or forks in their order.
//
// fork, extend and compact need ranks of blocks over the whole pool (which is
// the k-th free one).  One cluster of 8 CTAs computes them: each of its 256
// warps counts its run of the reference counts, the counts are summed over the
// cluster, and each warp walks its run again with its offset.  A cluster
// barrier costs about a microsecond where another launch costs more.  Copies
// go to a second launch over all SMs, a warp per 4 KiB, with all of a unit's
// loads in flight before its first store.
//
// Measured: 2048 block pairs of 64 KiB (268 MB read and written) 45 us, 88 % of the
// copy bandwidth; the 2.6 GB of a compaction 415 us after 10 us of ranking, 90 %.  The
// rankings and the tables are latency: 64 forks of rows of up to 8192 positions 9 us
// and 4 for their blocks, 256 rows extended 10, 128 freed 4.
//
// Bad ids, lengths and rows are skipped and flagged; nothing is read or
// written out of bounds.

#include <cuda_runtime.h>
#include <stdint.h>

#include "pages.cuh"
#include "sm103.cuh"

namespace nsv {
namespace {

using sm::kFull;

constexpr int kCluster = 8;
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kAllWarps = kCluster * kScanWarps;
constexpr int kCopyThreads = 256;
constexpr int kUnitBytes = 4096;  // what one warp copies at a time
constexpr int kUnitVecs = kUnitBytes / 16;

__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

__device__ __forceinline__ void flag(const PageParams& p, uint32_t bit) { atomicOr(p.status, bit); }

// Where a thread stands in the cluster.
struct Place {
  int cta, warp, lane, tid, gw;  // gw: warp within the cluster
  __device__ Place()
      : cta(blockIdx.x), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), tid(threadIdx.x),
        gw(blockIdx.x * kScanWarps + (threadIdx.x >> 5)) {}
};

// A warp's run [lo, hi) of the blocks.
__device__ __forceinline__ void warp_run(long long n, int gw, long long* lo, long long* hi) {
  const long long per = ((n + kAllWarps - 1) / kAllWarps + 31) / 32 * 32;
  *lo = min(n, per * gw);
  *hi = min(n, per * (gw + 1));
}

// Counts the blocks of [lo, hi) whose reference count is (not) zero.
__device__ __forceinline__ int count_run(const int32_t* refs, long long lo, long long hi, int lane,
                                         bool want_free) {
  int n = 0;
  for (long long b = lo; b < hi; b += 32 * 8) {
    int r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const long long i = b + u * 32 + lane;
      r[u] = i < hi ? __ldcg(refs + i) : (want_free ? 1 : 0);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) n += __popc(__ballot_sync(kFull, (r[u] == 0) == want_free));
  }
  return n;
}

// Sum over the warps of the CTA before this one, plus the cluster's CTAs
// before this CTA; *total: over the cluster.  `slots`: kCluster ints of the
// workspace that nothing else uses.
__device__ __forceinline__ int cluster_before(int n, const Place& at, int* s_warp, int32_t* slots,
                                              int* total) {
  if (at.lane == 0) s_warp[at.warp] = n;
  __syncthreads();
  int v = at.lane < kScanWarps ? s_warp[at.lane] : 0, incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, incl, o);
    if (at.lane >= o) incl += x;
  }
  const int before = __shfl_sync(kFull, incl - v, at.warp);
  if (at.tid == 31) __stcg(slots + at.cta, incl);  // lane 31 of warp 0: the CTA's sum
  cluster_sync();
  int sum = at.lane < kCluster ? __ldcg(slots + at.lane) : 0, lower = at.lane < at.cta ? sum : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, o);
    lower += __shfl_xor_sync(kFull, lower, o);
  }
  *total = sum;
  return before + lower;
}

// Writes the ids of the free blocks of rank below `limit` to list[rank]; rank:
// of the run's first free block.
__device__ __forceinline__ void list_free(const int32_t* refs, long long lo, long long hi, int lane,
                                          int rank, int limit, int32_t* list) {
  for (long long b = lo; b < hi && rank < limit; b += 32) {
    const long long i = b + lane;
    const bool is_free = i < hi && __ldcg(refs + i) == 0;
    const unsigned m = __ballot_sync(kFull, is_free);
    const int k = rank + __popc(m & ((1u << lane) - 1u));
    if (is_free && k < limit) __stcg(list + k, (int)i);
    rank += __popc(m);
  }
}

// Inclusive sum over a CTA's threads; *total: the CTA's.  64 bits: rows whose
// chunk starts overlap can ask for more blocks together than 32 bits count.
__device__ __forceinline__ long long cta_scan(long long v, const Place& at, long long* s_warp,
                                              long long* total) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, v, o);
    if (at.lane >= o) v += x;
  }
  __syncthreads();
  if (at.lane == 31) s_warp[at.warp] = v;
  __syncthreads();
  const long long w = s_warp[at.lane];
  long long wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, wi, o);
    if (at.lane >= o) wi += x;
  }
  *total = __shfl_sync(kFull, wi, 31);
  return v + __shfl_sync(kFull, wi - w, at.warp);
}

// More blocks than any pool has stand for all larger counts.
__device__ __forceinline__ int clip(long long blocks) {
  return (int)min(blocks, 0x7fffffffll);
}

__device__ __forceinline__ int blocks_of(int ctx) { return ctx > 0 ? (ctx - 1) / kBlock + 1 : 0; }

__device__ __forceinline__ bool good_ctx(const PageParams& p, int c) {
  return c >= 0 && (long long)c <= (long long)p.max_blocks * kBlock;
}

// Workspace words: slots of the cluster sums, totals, then per-item arrays.
enum : int { kSlots0 = 0, kSlots1 = 8, kTotalNeed = 16, kMoves = 17, kLive = 18, kParts = 19 };

// ----------------------------------------------------------------------- fork
// items: {child's length or -1 (refused), see below}
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads)
    fork_kernel(const PageParams p) {
  __shared__ int s_warp[kScanWarps];
  __shared__ long long s_scan[kScanWarps];
  __shared__ int s_first[kMaxRows];
  const Place at;
  sm::griddep_launch();
  int2* items = reinterpret_cast<int2*>(p.ws + kPageWords);
  int2* pairs = items + p.rows;                             // what is to be copied
  int32_t* list = reinterpret_cast<int32_t*>(pairs + p.rows);  // free blocks
  // the free blocks of each run, and (first CTA) what each fork needs
  long long lo, hi;
  warp_run(p.num_blocks, at.gw, &lo, &hi);
  const int mine = count_run(p.refs, lo, hi, at.lane, true);
  if (at.cta == 0) {
    // a child that is named twice belongs to its first fork
    for (int r = at.tid; r < p.rows; r += kScanThreads) s_first[r] = 0x7fffffff;
    __syncthreads();
    for (int i = at.tid; i < p.count; i += kScanThreads) {
      const int c = __ldg(p.children + i);
      if (c >= 0 && c < p.rows) atomicMin(&s_first[c], i);
    }
    __syncthreads();
    long long taken = 0;
    for (int base = 0; base < p.count; base += kScanThreads) {
      const int i = base + at.tid;
      int len = -1, need = 0;
      if (i < p.count) {
        const int par = __ldg(p.parents + i), c = __ldg(p.children + i);
        if (par == -1 && c == -1) {
          // a filler of a captured list
        } else if (par < 0 || par >= p.rows || c < 0 || c >= p.rows || s_first[c] != i ||
                   __ldcg(p.context_lens + c) != 0) {
          flag(p, NSV_DEV_BAD_ROW);
        } else if (!good_ctx(p, __ldcg(p.context_lens + par))) {
          flag(p, NSV_DEV_BAD_CTX);
        } else {
          len = __ldcg(p.context_lens + par);
          need = len % kBlock != 0;
        }
      }
      long long total;
      const int upto = (int)(taken + cta_scan(need, at, s_scan, &total));  // at most `rows`
      // {length, blocks needed up to and with this fork, signed by need}
      if (i < p.count) __stcg(items + i, make_int2(len, need ? upto : -upto - 1));
      taken += total;
    }
    if (at.tid == 0) __stcg(p.ws + kTotalNeed, (int)taken);
    __syncthreads();
  }
  int nfree;
  const int rank = cluster_before(mine, at, s_warp, p.ws + kSlots0, &nfree);
  list_free(p.refs, lo, hi, at.lane, rank, __ldcg(p.ws + kTotalNeed), list);
  cluster_sync();
  // A warp per 128 table entries of a fork: the child's table and references (four
  // loads in flight before the first store); the first also the copied block and
  // the length.
  const int parts = (p.max_blocks + 127) / 128;
  const long long work = (long long)p.count * parts;
  for (long long k = at.gw; k < work; k += kAllWarps) {
    const int i = (int)(k / parts), part = (int)(k - (long long)i * parts);
    const int2 it = __ldcg(items + i);
    const bool need = it.y >= 0;
    const int upto = need ? it.y : -it.y - 1;
    const bool ok = it.x >= 0 && upto <= nfree;
    if (part == 0 && at.lane == 0) {
      if (it.x >= 0 && !ok) flag(p, NSV_DEV_NO_BLOCKS);
      if (!ok) pairs[i] = make_int2(-1, -1);
    }
    if (!ok) continue;
    const int par = __ldg(p.parents + i), c = __ldg(p.children + i);
    const int32_t* from = p.block_tables + (size_t)par * p.max_blocks;
    int32_t* to = p.block_tables + (size_t)c * p.max_blocks;
    const int full = it.x / kBlock;
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = part * 128 + u * 32 + at.lane;
      id[u] = e < full ? __ldcg(from + e) : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = part * 128 + u * 32 + at.lane;
      if (e >= full) continue;
      to[e] = id[u];
      if (id[u] >= 0 && id[u] < p.num_blocks)
        atomicAdd(p.refs + id[u], 1);
      else
        flag(p, NSV_DEV_BAD_BLOCK);
    }
    if (part == 0 && at.lane == 0) {
      int2 pair = make_int2(-1, -1);
      if (need) {
        const int fresh = __ldcg(list + upto - 1), src = __ldcg(from + full);
        to[full] = fresh;
        p.refs[fresh] = 1;
        if (src >= 0 && src <= p.num_blocks)
          pair = make_int2(src, fresh);
        else
          flag(p, NSV_DEV_BAD_BLOCK);
      }
      pairs[i] = pair;
      p.context_lens[c] = it.x;
    }
  }
}

// --------------------------------------------------------------------- extend
// items: {blocks needed up to and with this row or -1 (refused), tokens}; grown:
// {parts before this row, its length before}
//
// PARTS: a warp takes 128 tokens of a row, else a whole row.  A warp alone took
// 181 us for a row of 32768 new tokens, in parts they take 13; finding the parts
// costs time with the number of rows (1024 rows of one new token each: 15 and 17 us,
// 8192: 50 and 70).  The host knows how many tokens there are, not whose: rows stay whole
// up to one each and kManyTokens more.  Where a few of very many rows bring all of those,
// that is the wrong side (8192 rows, one with 8704 new tokens, the others none: 68 us, in
// parts 23; 1024 rows, one with 1500: 19 and 13); with up to 256 rows the two are within
// 2 us.
constexpr int kPartTokens = 128, kManyTokens = 512;
template <bool PARTS>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads)
    extend_kernel(const PageParams p) {
  __shared__ int s_warp[kScanWarps];
  __shared__ long long s_scan[kScanWarps];
  __shared__ int s_parts[PARTS ? kMaxRows : 1];
  const Place at;
  int2* items = reinterpret_cast<int2*>(p.ws + kPageWords);
  int2* grown = items + p.rows;
  int32_t* list = reinterpret_cast<int32_t*>(grown + p.rows);
  // tokens of no row, and of rows that cannot grow, write the sink
  for (long long i = (long long)at.cta * kScanThreads + at.tid; i < p.tokens;
       i += kCluster * kScanThreads)
    p.write_slots[i] = (long long)p.num_blocks * kBlock;
  long long lo, hi;
  warp_run(p.num_blocks, at.gw, &lo, &hi);
  const int mine = count_run(p.refs, lo, hi, at.lane, true);
  if (at.cta == 0) {
    // Rows whose tokens overlap (starts that go back between them, flagged there) could
    // have more parts than 32 bits count: those past what rows of their own tokens can
    // have are refused.
    const long long most = p.tokens / kPartTokens + p.rows;
    long long taken = 0, parts = 0;
    for (int base = 0; base < p.rows; base += kScanThreads) {
      const int r = base + at.tid;
      int n = 0, need = 0, old = 0;
      bool ok = false;
      if (r < p.rows) {
        const int a = __ldg(p.chunk_starts + r), b = __ldg(p.chunk_starts + r + 1);
        const int c = __ldcg(p.context_lens + r);
        n = b - a;
        old = c;
        if (a < 0 || b < a || b > p.tokens) {
          flag(p, NSV_DEV_BAD_CHUNK);
          n = 0;
        } else if (!good_ctx(p, c) || (long long)c + n > (long long)p.max_blocks * kBlock) {
          flag(p, NSV_DEV_BAD_CTX);
        } else if (n > 0) {
          ok = true;
          if (c % kBlock) {  // the row appends to its last block: its own alone
            const int id = p.block_tables[(size_t)r * p.max_blocks + c / kBlock];
            if (id < 0 || id >= p.num_blocks) {
              flag(p, NSV_DEV_BAD_BLOCK);
              ok = false;
            } else if (__ldcg(p.refs + id) != 1) {
              flag(p, NSV_DEV_BAD_ROW);
              ok = false;
            }
          }
          if (ok) need = blocks_of(c + n) - blocks_of(c);
        }
      }
      long long total;
      if (PARTS) {
        const int own = ok ? (n - 1) / kPartTokens + 1 : 0;
        const long long before = parts + cta_scan(own, at, s_scan, &total) - own;
        if (r < p.rows) __stcg(grown + r, make_int2(clip(before), old));
        parts += total;
        if (ok && before + own > most) {
          flag(p, NSV_DEV_BAD_CHUNK);
          ok = false;
          need = 0;
        }
      }
      const long long upto = taken + cta_scan(need, at, s_scan, &total);
      if (r < p.rows) __stcg(items + r, make_int2(ok ? clip(upto) : -1, n));
      taken += total;
    }
    if (at.tid == 0) {
      __stcg(p.ws + kTotalNeed, clip(taken));
      __stcg(p.ws + kParts, (int)min(parts, most));
    }
    __syncthreads();
  }
  int nfree;
  const int rank = cluster_before(mine, at, s_warp, p.ws + kSlots0, &nfree);
  list_free(p.refs, lo, hi, at.lane, rank, __ldcg(p.ws + kTotalNeed), list);
  if (PARTS)
    for (int r = at.tid; r < p.rows; r += kScanThreads) s_parts[r] = __ldcg(grown + r).x;
  cluster_sync();
  // new blocks and the tokens' slots; the row's first warp also its length
  const int work = PARTS ? __ldcg(p.ws + kParts) : p.rows;
  for (int k = at.gw; k < work; k += kAllWarps) {
    int r = k, i0 = 0;
    if (PARTS) {  // the last row with at most k parts before it
      int end = p.rows;
      r = 0;
      while (end - r > 1) {
        const int mid = (r + end) >> 1;
        if (s_parts[mid] <= k) r = mid; else end = mid;
      }
      i0 = (k - s_parts[r]) * kPartTokens;
    }
    const int2 it = __ldcg(items + r);
    if (it.x < 0) continue;
    if (it.x > nfree) {
      if (i0 == 0 && at.lane == 0) flag(p, NSV_DEV_NO_BLOCKS);
      continue;
    }
    const int old = PARTS ? __ldcg(grown + r).y : __ldcg(p.context_lens + r), n = it.y;
    const int had = blocks_of(old), will = blocks_of(old + n);
    int32_t* table = p.block_tables + (size_t)r * p.max_blocks;
    const int32_t* fresh = list + (it.x - (will - had)) - had;  // indexed by table column
    const int start = __ldg(p.chunk_starts + r);
    const int i1 = PARTS ? min(n, i0 + kPartTokens) : n;
#pragma unroll 4
    for (int i = i0 + at.lane; i < i1; i += 32) {
      const int pos = old + i, b = pos / kBlock, off = pos % kBlock;
      const int id = __ldcg(b < had ? table + b : fresh + b);
      if (b >= had && off == 0) {
        table[b] = id;
        p.refs[id] = 1;
      }
      p.write_slots[start + i] = (long long)id * kBlock + off;
    }
    __syncwarp();
    if (i0 == 0 && at.lane == 0) p.context_lens[r] = old + n;
  }
}

// ----------------------------------------------------------------------- free
constexpr int kFreeThreads = 256;
__global__ void __launch_bounds__(kFreeThreads) free_kernel(const PageParams p) {
  __shared__ int s_ctx;
  const int row = __ldg(p.parents + blockIdx.x);
  if (row == -1) return;  // a filler of a captured list
  if (row < 0 || row >= p.rows) {
    if (threadIdx.x == 0) flag(p, NSV_DEV_BAD_ROW);
    return;
  }
  // a row that is named twice is empty the second time
  if (threadIdx.x == 0) s_ctx = atomicExch(p.context_lens + row, 0);
  __syncthreads();
  const int c = s_ctx;
  if (!good_ctx(p, c)) {
    if (threadIdx.x == 0) flag(p, NSV_DEV_BAD_CTX);
    return;
  }
  int32_t* table = p.block_tables + (size_t)row * p.max_blocks;
#pragma unroll 4
  for (int b = threadIdx.x; b < blocks_of(c); b += blockDim.x) {
    const int id = __ldcg(table + b);
    table[b] = -1;
    if (id < 0 || id >= p.num_blocks) {
      flag(p, NSV_DEV_BAD_BLOCK);
    } else if (atomicSub(p.refs + id, 1) <= 0) {  // it was free already
      atomicAdd(p.refs + id, 1);
      flag(p, NSV_DEV_BAD_BLOCK);
    }
  }
}

// -------------------------------------------------------------------- compact
// With n live blocks: the live ones at and past n move, in order, into the free
// ones below n, in order.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads)
    compact_plan_kernel(const PageParams p) {
  __shared__ int s_warp[kScanWarps];
  const Place at;
  sm::griddep_launch();
  int32_t* map = p.ws + kPageWords;    // [num_blocks]: rank of a moving block, else -1
  int32_t* holes = map + p.num_blocks;  // [moves], then the moving blocks
  int32_t* movers = holes + p.num_blocks / 2 + 1;
  long long lo, hi;
  warp_run(p.num_blocks, at.gw, &lo, &hi);
  const int mine = count_run(p.refs, lo, hi, at.lane, false);
  int live;
  int before = cluster_before(mine, at, s_warp, p.ws + kSlots0, &live);
  // live blocks below `live`: this run's, and all
  const int low = hi <= live   ? mine
                  : lo >= live ? 0
                               : count_run(p.refs, lo, live, at.lane, false);
  int stay;
  (void)cluster_before(low, at, s_warp, p.ws + kSlots1, &stay);
  for (long long b = lo; b < hi; b += 32) {
    const long long i = b + at.lane;
    const bool is_live = i < hi && __ldcg(p.refs + i) != 0;
    const unsigned m = __ballot_sync(kFull, is_live);
    const int lb = before + __popc(m & ((1u << at.lane) - 1u));  // live ones before block i
    if (i < hi) {
      if (i >= live) {
        map[i] = is_live ? lb - stay : -1;
        if (is_live) movers[lb - stay] = (int)i;
      } else if (!is_live) {
        holes[i - lb] = (int)i;
      }
    }
    before += __popc(m);
  }
  if (at.gw == 0 && at.lane == 0) {
    p.ws[kMoves] = live - stay;
    p.ws[kLive] = live;
  }
}

// ----------------------------------------------------------------------- copy
// One unit: up to 4 KiB of one block of K or V, every load before the first
// store.
__device__ __forceinline__ void copy_unit(const PageParams& p, long long unit, int src, int dst,
                                          int lane) {
  const int per_pool = p.units_per_block;
  const int part = (int)(unit % (2 * per_pool));
  uint4* pool = static_cast<uint4*>(part < per_pool ? p.k_pool : p.v_pool);
  const int v0 = (part < per_pool ? part : part - per_pool) * kUnitVecs;
  const int n = min(kUnitVecs, p.block_vecs - v0);
  const uint4* from = pool + (size_t)src * p.block_vecs + v0;
  uint4* to = pool + (size_t)dst * p.block_vecs + v0;
  uint4 x[kUnitVecs / 32];
#pragma unroll
  for (int u = 0; u < kUnitVecs / 32; ++u)
    if (u * 32 + lane < n) x[u] = __ldcs(from + u * 32 + lane);
#pragma unroll
  for (int u = 0; u < kUnitVecs / 32; ++u)
    if (u * 32 + lane < n) __stcs(to + u * 32 + lane, x[u]);
}

// Block pairs: the caller's two lists, or (pairs not null) a fork's.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PageParams p, const int2* pairs) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
  const long long units = (long long)p.count * 2 * p.units_per_block;
  sm::griddep_wait();
  for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units;
       u += warps) {
    const int i = (int)(u / (2 * p.units_per_block));
    const int2 pr =
        pairs ? __ldcg(pairs + i) : make_int2(__ldg(p.parents + i), __ldg(p.children + i));
    if (pr.x == -1 && pr.y == -1) continue;  // a fork without a copy, a filler
    if (pr.x < 0 || pr.x > p.num_blocks || pr.y < 0 || pr.y > p.num_blocks) {
      if (lane == 0) flag(p, NSV_DEV_BAD_BLOCK);
      continue;
    }
    if (pr.x != pr.y) copy_unit(p, u, pr.x, pr.y, lane);
  }
}

// The moves of a compaction: blocks, reference counts and table entries.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const PageParams p) {
  const int lane = threadIdx.x & 31;
  const long long w0 = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
  const int32_t* map = p.ws + kPageWords;
  const int32_t* holes = map + p.num_blocks;
  const int32_t* movers = holes + p.num_blocks / 2 + 1;
  sm::griddep_wait();
  const int moves = __ldcg(p.ws + kMoves), live = __ldcg(p.ws + kLive);
  // table entries, a warp per row
  for (long long r = w0; r < p.rows; r += warps) {
    const int c = __ldg(p.context_lens + r);
    if (!good_ctx(p, c)) {
      if (lane == 0) flag(p, NSV_DEV_BAD_CTX);
      continue;
    }
    int32_t* table = p.block_tables + (size_t)r * p.max_blocks;
    for (int b = lane; b < blocks_of(c); b += 32) {
      const int id = table[b];
      if (id >= 0 && id < live) continue;
      const int k = id >= 0 && id < p.num_blocks ? __ldcg(map + id) : -1;
      if (k >= 0)
        table[b] = __ldcg(holes + k);
      else
        flag(p, NSV_DEV_BAD_BLOCK);  // an entry that names no live block
    }
  }
  for (long long k = w0 * 32 + lane; k < moves; k += warps * 32) {
    const int src = __ldcg(movers + k), dst = __ldcg(holes + k);
    p.refs[dst] = p.refs[src];
    p.refs[src] = 0;
  }
  const long long units = (long long)moves * 2 * p.units_per_block;
  for (long long u = w0; u < units; u += warps) {
    const int k = (int)(u / (2 * p.units_per_block));
    copy_unit(p, u, __ldcg(movers + k), __ldcg(holes + k), lane);
  }
}

cudaError_t launch_after(void (*kernel)(const PageParams), const PageParams& p, int grid,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// CTAs of a copy over `units` warp units: enough for every SM's warps, no more
// than there are units.
int copy_grid(const PageParams& p, long long units) {
  const long long want = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const long long most = (long long)p.num_sms * (2048 / kCopyThreads);
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace

int page_units(int block_vecs) { return (block_vecs + kUnitVecs - 1) / kUnitVecs; }

cudaError_t launch_blocks_copy(const PageParams& p, cudaStream_t stream) {
  copy_kernel<<<copy_grid(p, (long long)p.count * 2 * p.units_per_block), kCopyThreads, 0,
                stream>>>(p, nullptr);
  return cudaGetLastError();
}

cudaError_t launch_rows_fork(const PageParams& p, cudaStream_t stream) {
  fork_kernel<<<kCluster, kScanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int2* pairs = reinterpret_cast<const int2*>(p.ws + kPageWords) + p.rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)copy_grid(p, (long long)p.count * 2 * p.units_per_block));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_kernel, p, pairs);
}

cudaError_t launch_rows_extend(const PageParams& p, cudaStream_t stream) {
  if (p.tokens > (long long)p.rows + kManyTokens)
    extend_kernel<true><<<kCluster, kScanThreads, 0, stream>>>(p);
  else
    extend_kernel<false><<<kCluster, kScanThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rows_free(const PageParams& p, cudaStream_t stream) {
  free_kernel<<<p.count, kFreeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_blocks_compact(const PageParams& p, cudaStream_t stream) {
  compact_plan_kernel<<<kCluster, kScanThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // at most half of the blocks can move
  const long long most = (long long)(p.num_blocks / 2) * 2 * p.units_per_block;
  return launch_after(compact_move_kernel, p, copy_grid(p, most > p.rows ? most : p.rows), stream);
}

}  // namespace nsv
