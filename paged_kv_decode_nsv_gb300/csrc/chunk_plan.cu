// Planning kernel of the chunk attention: from the chunk starts, context
// lengths and visibility bounds in device memory to the list of tiles, each
// with the key range that its query tokens see, and the prefix sums of their
// units.  Lengths never reach the host, so a captured step replays with new
// ones.  One CTA: the list is short (rows + tokens / tile tokens).
//
// Bad values are caught here: a context length outside [0, max_blocks * 16] is
// taken as 0 (NSV_DEV_BAD_CTX) and a pair of chunk starts that is not an
// ascending pair within [0, tokens] as no tokens (NSV_DEV_BAD_CHUNK); a list
// that would outgrow its room (starts that overlap) is cut off and flagged.

#include "chunk.cuh"

namespace nsv {
namespace {

constexpr int kPlanThreads = 1024;
// Inclusive sum over the block's threads; *total is the block's.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp,
                                                long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(sm::kFull, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(sm::kFull, w, o);
      if (lane >= o) w += x;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  if (warp) v += s_warp[warp - 1];
  *total = s_warp[31];
  __syncthreads();
  return v;
}

template <typename P>
__device__ __forceinline__ void plan(const P& p) {
  __shared__ int s_first[kMaxRows + 1];  // tiles before each row
  __shared__ long long s_prefix[kPlanThreads];
  __shared__ long long s_warp[32];
  // a tile's key range, before its prefix takes its place
  int2* s_keys = reinterpret_cast<int2*>(s_prefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tt = p.tile_tokens;

  long long carry = 0;
  for (int base = 0; base < p.rows; base += kPlanThreads) {
    const int r = base + tid;
    long long n = 0;
    if (r < p.rows) n = (row_chunk(p, r, true).n + (long long)tt - 1) / tt;
    long long total;
    const long long upto = carry + block_scan(n, s_warp, &total);
    if (r < p.rows) s_first[r] = (int)min(upto - n, (long long)p.max_tiles);
    carry += total;
  }
  if (carry > p.max_tiles) {
    if (tid == 0) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_CHUNK);
    carry = p.max_tiles;
  }
  if (tid == 0) s_first[p.rows] = (int)carry;
  __syncthreads();
  const int ntiles = (int)carry;

  auto tile_of = [&](int i, int& row, RowChunk& c, int& tok0) {
    int lo = 0, hi = p.rows;  // the last row whose first tile is at most i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= i) lo = mid; else hi = mid;
    }
    row = lo;
    c = row_chunk(p, row, false);
    tok0 = (i - s_first[row]) * tt;
  };

  long long units = 0;
  int longest = 0;  // runs of the longest tile
  for (int base = 0; base < ntiles; base += kPlanThreads) {
    if (p.see_begin || p.see_end) {
      // a warp per tile: the range that its tokens see
      for (int i = warp; i < kPlanThreads && base + i < ntiles; i += kPlanThreads / 32) {
        int row, tok0;
        RowChunk c;
        tile_of(base + i, row, c, tok0);
        const int n = min(tt, c.n - tok0);
        int kb = 0x7fffffff, ke = 0;
        for (int t = lane; t < n; t += 32) {
          const int2 v =
              chunk_sees(p, (long long)c.start + tok0 + t, c.ctx - c.n + tok0 + t, c.ctx);
          if (v.x < v.y) {
            kb = min(kb, v.x);
            ke = max(ke, v.y);
          }
        }
        kb = __reduce_min_sync(sm::kFull, kb);
        ke = __reduce_max_sync(sm::kFull, ke);
        if (lane == 0) {
          s_keys[i] = make_int2(kb < ke ? kb / kBlock * kBlock : 0, ke);
        }
      }
      __syncthreads();
    }
    const int i = base + tid;
    long long n = 0;
    if (i < ntiles) {
      int row, tok0;
      RowChunk c;
      tile_of(i, row, c, tok0);
      const int nt = min(tt, c.n - tok0), pos0 = c.ctx - c.n + tok0;
      int kb = 0, ke = 0;
      if (p.see_begin || p.see_end) {
        kb = s_keys[tid].x;
        ke = s_keys[tid].y;
      } else {
        ke = max(0, min(pos0 + nt, c.ctx));
      }
      p.ws_tiles[2 * (size_t)i] = make_int4(row, c.start + tok0, nt, pos0);
      // (a tile with more than half of the tokens fills both halves)
      const int cost = 2 * nt > tt ? p.pair_units : p.half_units;
      p.ws_tiles[2 * (size_t)i + 1] = make_int4(kb, ke, c.ctx, cost);
      const int runs = chunk_runs(kb, ke, p.keys);
      n = (long long)(p.tile_cost + runs) * cost;
      longest = max(longest, runs);
    }
    long long total;
    const long long upto = block_scan(n, s_warp, &total);
    if (i < ntiles) {
      p.ws_prefix[i] = units + upto - n;
      s_prefix[tid] = units + upto - n;  // used where one pass covers all tiles
    }
    units += total;
    __syncthreads();
  }
  // (a CTA's share is counted in 32 bits: in bf16 2^29 runs of four units would take it
  // 17 minutes, in fp32 2^31 of one 55 or 100, at head_dim 64 or 128)
  if (units > 0x7fffffffll / p.kv_heads * p.grid) {
    if (tid == 0) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_CHUNK);
    units = 0;
  }
  if (tid == 0) {
    p.ws_prefix[ntiles] = units;
    p.ws_head[0] = units;
    p.ws_head[1] = ntiles;
  }
  if (!std::is_same_v<P, Chunk4Params> || p.ws_cnt)
    for (long long i = tid; i < (long long)ntiles * p.kv_heads; i += kPlanThreads) p.ws_cnt[i] = 0;
  // Where each CTA's share of the units starts: c * U / n for the first n CTAs, of
  // at least a run's units each, so that a run starts in every share that lies
  // within a tile; the others get none.  (Moving a boundary that leaves a run or less
  // on one side of a tile to the tile's edge saved pieces to merge, but the uneven
  // shares cost more: a 2048-token prompt 58 us instead of 56.)
  __syncthreads();
  const bool whole = !__syncthreads_or(longest > kChunkWholeRuns) &&
                     (long long)ntiles * p.kv_heads <= p.grid;
  const long long U = units * p.kv_heads;
  const int run = p.pair_units;
  const int n = whole ? ntiles * p.kv_heads : (int)max(1ll, min(U / run, (long long)p.grid));
  auto prefix = [&](int i) {
    return i == ntiles ? units : ntiles <= kPlanThreads ? s_prefix[i] : __ldcg(p.ws_prefix + i);
  };
  auto start = [&](int c, int& head, int& tile, int& skip) -> long long {
    head = tile = skip = 0;
    if (c >= n || U == 0) return U;
    if (whole) {
      head = c / ntiles;
      tile = c - head * ntiles;
      return head * units + prefix(tile);
    }
    const long long u = (long long)c * U / n;
    head = (int)(u / units);
    const long long rem = u - head * units;
    int lo = 0, hi = ntiles;  // the last tile whose first unit is at most rem
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix(mid) <= rem) lo = mid; else hi = mid;
    }
    tile = lo;
    skip = (int)(rem - prefix(lo));
    return u;
  };
  for (int c = tid; c < p.grid; c += kPlanThreads) {
    int4 at;
    int h, t, k;
    const long long u = start(c, at.y, at.z, at.w);
    at.x = (int)(start(c + 1, h, t, k) - u);
    p.ws_cta[c] = at;
    p.ws_first[c] = u;
  }
}

template <typename P>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const P p) {
  sm::griddep_wait();  // lengths and bounds may be the previous kernel's
  sm::griddep_launch();
  plan(p);
}

// Query vectors to fp16, scaled by a power of two each: exact but for elements below 2^-28
// of a vector's largest, which are off by 2^-39 of it at most.  A lane holds 8 dimensions.
template <int D>
__device__ __forceinline__ void convert_queries(const ChunkQueries& c, int cta, int ctas) {
  constexpr int kLanes = D / 8, kVecs = 32 / kLanes;  // lanes of a vector; vectors of a warp
  const int lane = threadIdx.x & 31;
  const long long step = (long long)ctas * (kPlanThreads / 32) * kVecs;
  const long long first = ((long long)cta * (kPlanThreads / 32) + (threadIdx.x >> 5)) * kVecs;
  for (long long v0 = first; v0 < c.vectors; v0 += step) {
    const long long v = v0 + lane / kLanes;
    const size_t at = (size_t)min(v, c.vectors - 1) * kLanes + lane % kLanes;
    const uint4 r = __ldg(static_cast<const uint4*>(c.q) + at);
    uint32_t w[4] = {r.x, r.y, r.z, r.w}, top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = max(top, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(sm::kFull, top, o));
    const int e = min(126, 14 + 127 - (int)(top >> 23));
    const float mul = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = sm::pack_half(__uint_as_float(w[i] << 16) * mul,
                           __uint_as_float(w[i] & 0xffff0000u) * mul);
    if (v >= c.vectors) continue;
    static_cast<uint4*>(c.half)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane % kLanes == 0) c.up[v] = __uint_as_float((uint32_t)(127 - e) << 23);
  }
}

// A CTA for each list (`both`: or for the second alone), the others for the query vectors.
template <int D>
__global__ void __launch_bounds__(kPlanThreads)
    chunk_plans_kernel(const __grid_constant__ Chunk4Params a,
                       const __grid_constant__ Chunk4Params b,
                       const __grid_constant__ ChunkQueries q, bool both) {
  sm::griddep_wait();
  sm::griddep_launch();
  if (blockIdx.x > 1) {
    convert_queries<D>(q, blockIdx.x - 2, gridDim.x - 2);
  } else if (blockIdx.x == 1 || both) {
    plan(blockIdx.x ? b : a);
  }
}

template <typename P>
cudaError_t launch_plan(const P& p, cudaStream_t stream) {
  // (programmatic: its launch overlaps the previous kernel's end, and it waits for
  // that kernel before it reads anything)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_plan_kernel<P>, p);
}

}  // namespace

cudaError_t launch_chunk_plans(const Chunk4Params* a, const Chunk4Params& b,
                               const ChunkQueries& q, int head_dim, int num_sms,
                               cudaStream_t stream) {
  // (a CTA takes 64 vectors a turn at head_dim 128)
  const long long ctas = (q.vectors + 63) / 64;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 + (ctas < num_sms ? ctas : num_sms)));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const Chunk4Params& first = a ? *a : b;
  return head_dim == 64
             ? cudaLaunchKernelEx(&cfg, chunk_plans_kernel<64>, first, b, q, a != nullptr)
             : cudaLaunchKernelEx(&cfg, chunk_plans_kernel<128>, first, b, q, a != nullptr);
}

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream) {
  return launch_plan(p, stream);
}
cudaError_t launch_chunk_plan(const Chunk4Params& p, cudaStream_t stream) {
  return launch_plan(p, stream);
}

}  // namespace nsv
