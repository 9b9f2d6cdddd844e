// Attention of a chunk of new tokens over a paged cache, fp32 (see
// chunk_bf16.cu for the formulas).  A CTA of 256 threads folds runs of 64
// positions into up to 64 rows (query tokens x query heads of one KV head).
//
// Both products run on the tensor cores at fp32's precision, each factor as a
// sum of two tf32 numbers (x = hi + lo, hi = x rounded to tf32's 11 bits, lo the
// rest): a b = a_hi b_hi + a_hi b_lo + a_lo b_hi, where what is left out, a_lo
// b_lo, is 2^-22 of the product, and lo's own truncation to tf32 as much.  With
// fp32 multiply-adds on the CUDA cores instead the kernel was bound by
// shared-memory loads (8 of 16 bytes for every 64 multiply-adds of a 4 x 4 tile a
// thread): 207 us for 638 tokens over up to 2048 positions at 12 heads.
//
// Warp (wm, wn) of 4 x 2: 16 rows; half of the keys in the scores, half of the
// dims in the output.  m16n8k8 fragments, lane = 4 g + t: A rows g and g + 8 at k
// = t and t + 4, B column g, C rows g and g + 8 at columns 2 t and 2 t + 1.  The
// probabilities go through shared memory.  The next run's keys are copied
// (cp.async) from the end of this run's scores on, its values from the end of
// its products on, and two CTAs share an SM.  Rows of 16-byte chunks are stored
// swizzled, so that the fragments' loads hit all banks: chunk v of row r at
// v ^ (r % 8), of the values' rows (which B reads down the columns) at
// v ^ 2 (r % 4).

#include "chunk.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kThreadsF32 = 256;
constexpr int kR = kChunkRowsF32, kC = kChunkKeysF32;

template <int D>
struct SmemF32 {
  static constexpr uint32_t kOffK = kR * D * 4;
  static constexpr uint32_t kOffV = kOffK + kC * D * 4;
  static constexpr uint32_t kOffP = kOffV + kC * D * 4;
  static constexpr uint32_t kOffX = kOffP + kR * kC * 4;   // float [2][64]: maxima, sums
  static constexpr uint32_t kOffOk = kOffX + 2 * kR * 4;   // blocks of two runs in turn
  static constexpr uint32_t kOffMerge = kOffOk + 16;
  static constexpr uint32_t kTotal = kOffMerge + 16;
  static_assert(2 * (kTotal + 1024) <= 228 * 1024, "two CTAs per SM");
};

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
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Float index of 16-byte chunk v of row r, W floats to a row; of the values'.
template <int W>
__device__ __forceinline__ int at_chunk(int r, int v) {
  return r * W + ((v ^ ((r & 1) << 2 | (r & 2))) << 2);
}
template <int W>
__device__ __forceinline__ int at_value(int r, int v) {
  const int x = r >> 2 & 3;
  return r * W + ((v ^ (W == 128 ? (x & 1) | (x & 2) << 1 : x << 1)) << 2);
}
__device__ __forceinline__ float4 load4(const float* s) {
  return *reinterpret_cast<const float4*>(s);
}

// x = hi + lo.
struct Split {
  uint32_t hi, lo;
  __device__ __forceinline__ explicit Split(float x) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // to nearest, ties away from zero
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
};
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d[n] += A B for four column tiles, the small products first; a product waits for
// the one before it of its tile, so the tiles take turns.
__device__ __forceinline__ void mma_f32(float (*d)[4], const Split (&a)[4], const Split (&b0)[4],
                                        const Split (&b1)[4]) {
#pragma unroll
  for (int n = 0; n < 4; ++n)
    mma_tf32(d[n], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b0[n].hi, b1[n].hi);
#pragma unroll
  for (int n = 0; n < 4; ++n)
    mma_tf32(d[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0[n].lo, b1[n].lo);
#pragma unroll
  for (int n = 0; n < 4; ++n)
    mma_tf32(d[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0[n].hi, b1[n].hi);
}

template <int D>
__global__ void __launch_bounds__(kThreadsF32, 2) chunk_f32_kernel(
    const __grid_constant__ ChunkParams p) {
  using L = SmemF32<D>;
  constexpr int kNt = D / 16;  // 8-column tiles of a warp's half of the dims
  extern __shared__ __align__(16) unsigned char smem[];
  float* sq = reinterpret_cast<float*>(smem);
  float* sk = reinterpret_cast<float*>(smem + L::kOffK);
  float* sv = reinterpret_cast<float*>(smem + L::kOffV);
  float* sp = reinterpret_cast<float*>(smem + L::kOffP);
  float* s_x = reinterpret_cast<float*>(smem + L::kOffX);
  int* s_ok = reinterpret_cast<int*>(smem + L::kOffOk);
  int* s_merge = reinterpret_cast<int*>(smem + L::kOffMerge);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp & 3, wn = warp >> 2, g = lane >> 2, t4 = lane & 3;
  const int r0 = wm * 16 + g;  // this thread's rows: r0 and r0 + 8
  const float* q = static_cast<const float*>(p.q);
  const float* kp = static_cast<const float*>(p.k_pool);
  const float* vp = static_cast<const float*>(p.v_pool);
  constexpr float kLog2e = 1.4426950408889634f;
  griddep_wait();
  griddep_launch();
  ChunkWalk wk;
  wk.init(p, blockIdx.x);
  ChunkSegment s;
#pragma unroll 1
  while (wk.next<kC>(p, s)) {
    const int rows = s.t.n_tok * p.group;
    __syncthreads();  // the previous segment's readers are done
    for (int c = tid; c < kR * (D / 4); c += kThreadsF32) {
      const int r = c / (D / 4), v = c - r * (D / 4);
      const int tok = (int)((unsigned)r / (unsigned)p.group), h = r - tok * p.group;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        x = __ldg(reinterpret_cast<const float4*>(
                      q + (((size_t)s.t.q0 + tok) * p.heads + s.head * p.group + h) * D) + v);
      *reinterpret_cast<float4*>(sq + at_chunk<D>(r, v)) = x;
    }
    int2 see[2];
    int pos[2];
    float slope[2], m[2], l[2], acc[kNt][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i, tok = (int)((unsigned)r / (unsigned)p.group);
      pos[i] = s.t.pos0 + tok;
      see[i] = r < rows ? chunk_sees(p, (long long)s.t.q0 + tok, pos[i], s.t.ctx) : make_int2(0, 0);
      slope[i] =
          r < rows && p.slopes ? __ldg(p.slopes + s.head * p.group + r - tok * p.group) : 0.f;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    // Copies one run's keys (or values); positions at and past `ke` (at most the
    // context) and in bad blocks become zeros.
    auto copy_run = [&](const float* pool, float* dst, int j, bool keys) {
      const int t0 = s.t.kb + j * kC;
#pragma unroll 4
      for (int c = tid; c < kC * (D / 4); c += kThreadsF32) {
        const int t = c / (D / 4), v = c - t * (D / 4);
        bool ok = (long long)t0 + t < s.t.ke;
        const int b = ok ? __ldg(table + (t0 + t) / kBlock) : 0;
        const bool bad = b < 0 || b >= p.pool_blocks;
        if (keys && bad && v == 0) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_BLOCK);
        ok = ok && !bad;
        const size_t at =
            ok ? (((size_t)b * p.kv_heads + s.head) * kBlock + (t0 + t) % kBlock) * D + v * 4 : 0;
        copy16(dst + (keys ? at_chunk<D>(t, v) : at_value<D>(t, v)), pool + at, ok);
      }
      copies_commit();
    };
    // which of a run's blocks hold something
    auto run_blocks = [&](int j) {
      if (tid < 32) {
        const long long t = (long long)s.t.kb + j * kC + tid * kBlock;
        const int b = tid < kC / kBlock && t < s.t.ke ? __ldg(table + t / kBlock) : -1;
        const unsigned ok = __ballot_sync(kFull, b >= 0 && b < p.pool_blocks);
        if (tid == 0) s_ok[j & 1] = (int)ok;
      }
    };
    copy_run(kp, sk, s.j0, true);
    copy_run(vp, sv, s.j0, false);
    run_blocks(s.j0);
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j) {
      const int t0 = s.t.kb + j * kC;
      copies_wait<1>();  // the keys
      __syncthreads();
      float sc[4][4];  // keys wn * 32 + n * 8 + 2 t4 + {0, 1}, rows r0 and r0 + 8
#pragma unroll
      for (int n = 0; n < 4; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll 2
      for (int ks = 0; ks < D / 16; ++ks) {
        const float4 x0 = load4(sq + at_chunk<D>(r0, 4 * ks + t4));
        const float4 x1 = load4(sq + at_chunk<D>(r0 + 8, 4 * ks + t4));
        float4 y[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          y[n] = load4(sk + at_chunk<D>(wn * 32 + n * 8 + g, 4 * ks + t4));
        {
          const Split a[4] = {Split(x0.x), Split(x1.x), Split(x0.y), Split(x1.y)};
          const Split b0[4] = {Split(y[0].x), Split(y[1].x), Split(y[2].x), Split(y[3].x)};
          const Split b1[4] = {Split(y[0].y), Split(y[1].y), Split(y[2].y), Split(y[3].y)};
          mma_f32(sc, a, b0, b1);
        }
        {
          const Split a[4] = {Split(x0.z), Split(x1.z), Split(x0.w), Split(x1.w)};
          const Split b0[4] = {Split(y[0].z), Split(y[1].z), Split(y[2].z), Split(y[3].z)};
          const Split b1[4] = {Split(y[0].w), Split(y[1].w), Split(y[2].w), Split(y[3].w)};
          mma_f32(sc, a, b0, b1);
        }
      }
      const int blocks = s_ok[j & 1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = wn * 32 + n * 8 + 2 * t4 + e;
            float x = sc[n][2 * i + e] * p.scale;
            if (p.cap > 0.f) x = p.cap * tanhf(x / p.cap);
            x = fmaf(-slope[i], fabsf((float)(pos[i] - t0 - t)), x) * kLog2e;
            const bool seen =
                t >= see[i].x - t0 && t < see[i].y - t0 && ((blocks >> (t / kBlock)) & 1);
            sc[n][2 * i + e] = seen ? x : -INFINITY;
            mx = fmaxf(mx, sc[n][2 * i + e]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        if (t4 == 0) s_x[wn * kR + r0 + 8 * i] = mx;
      }
      __syncthreads();  // the keys are free, the maxima of both halves there
      if (j + 1 < s.j1) {
        copy_run(kp, sk, j + 1, true);
        run_blocks(j + 1);
      } else {
        copies_commit();
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mx = fmaxf(s_x[r0 + 8 * i], s_x[kR + r0 + 8 * i]);
        if (mx > m[i]) {
          const float alpha = exp2f(m[i] - mx);
          m[i] = mx;
          l[i] *= alpha;
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            acc[n][2 * i] *= alpha;
            acc[n][2 * i + 1] *= alpha;
          }
        }
        const float sub = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float p0 = exp2f(sc[n][2 * i] - sub), p1 = exp2f(sc[n][2 * i + 1] - sub);
          l[i] += p0 + p1;  // this thread's keys
          const int t = wn * 32 + n * 8 + 2 * t4;
          *reinterpret_cast<float2*>(sp + at_chunk<kC>(r0 + 8 * i, t >> 2) + (t & 3)) =
              make_float2(p0, p1);
        }
      }
      copies_wait<1>();  // the values (the next run's keys may still be on their way)
      __syncthreads();
#pragma unroll 1
      for (int ks = 0; ks < kC / 16; ++ks) {
        const float4 x0 = load4(sp + at_chunk<kC>(r0, 4 * ks + t4));
        const float4 x1 = load4(sp + at_chunk<kC>(r0 + 8, 4 * ks + t4));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const Split a[4] = {Split(half ? x0.z : x0.x), Split(half ? x1.z : x1.x),
                              Split(half ? x0.w : x0.y), Split(half ? x1.w : x1.y)};
          const int key = 16 * ks + 4 * t4 + 2 * half;
#pragma unroll
          for (int c = 0; c < kNt / 4; ++c) {
            const int v = wn * (D / 8) + g * (kNt / 4) + c;
            const float4 y0 = load4(sv + at_value<D>(key, v));
            const float4 y1 = load4(sv + at_value<D>(key + 1, v));
            const Split b0[4] = {Split(y0.x), Split(y0.y), Split(y0.z), Split(y0.w)};
            const Split b1[4] = {Split(y1.x), Split(y1.y), Split(y1.z), Split(y1.w)};
            mma_f32(acc + 4 * c, a, b0, b1);
          }
        }
      }
      __syncthreads();  // the values and probabilities are free
      if (j + 1 < s.j1)
        copy_run(vp, sv, j + 1, false);
      else
        copies_commit();
    }
    // the rows' sums over the quad's and both halves' keys
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(kFull, l[i], 1);
      l[i] += __shfl_xor_sync(kFull, l[i], 2);
      if (t4 == 0) s_x[wn * kR + r0 + 8 * i] = l[i];
    }
    __syncthreads();
    const bool whole = s.first && s.last;
    const int slot = chunk_slot(blockIdx.x, s.first);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      if (r >= rows) continue;
      const float sum = s_x[r] + s_x[kR + r];
      float* o = chunk_out<float>(p, s.t.q0, s.head, r, D);
      const float inv = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < kNt; n += 4) {
          const int d = wn * (D / 2) + (2 * t4 + e) * kNt + n, k = 2 * i + e;
          *(whole ? reinterpret_cast<float4*>(o + d) : chunk_acc(p, slot, D, d >> 2, r)) =
              make_float4(acc[n][k] * inv, acc[n + 1][k] * inv, acc[n + 2][k] * inv,
                          acc[n + 3][k] * inv);
        }
      if (!whole && wn == 0 && t4 == 0)
        p.ws_ml[(size_t)slot * p.tile_rows + r] = make_float2(m[i], sum);
    }
    if (!whole) {
      // publish the piece; the CTA whose piece is the last merges them all
      __syncthreads();
      if (tid < 32) {
        const int2 pc = chunk_pieces<kC>(p, s, lane);
        if (lane == 0) {
          __threadfence();
          int* cnt = p.ws_cnt + (size_t)s.tile * p.kv_heads + s.head;
          s_merge[0] = atomicAdd(cnt, 1) == pc.y - 1;
          s_merge[1] = pc.x;
          s_merge[2] = pc.y;
        }
      }
      __syncthreads();
      if (s_merge[0]) {
        __threadfence();
        chunk_merge<float, D, kThreadsF32>(p, s.t.q0, s.t.n_tok, s.head, s_merge[1], s_merge[2],
                                           tid);
      }
    }
  }
}

template <int D>
cudaError_t launch_dim(const ChunkParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kThreadsF32);
  cfg.dynamicSmemBytes = SmemF32<D>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_f32_kernel<D>, p);
}

}  // namespace

cudaError_t prepare_chunk_f32() {
  const cudaError_t e =
      cudaFuncSetAttribute(chunk_f32_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SmemF32<64>::kTotal);
  return e != cudaSuccess
             ? e
             : cudaFuncSetAttribute(chunk_f32_kernel<128>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    SmemF32<128>::kTotal);
}

cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64>(p, stream) : launch_dim<128>(p, stream);
}

}  // namespace nsv
