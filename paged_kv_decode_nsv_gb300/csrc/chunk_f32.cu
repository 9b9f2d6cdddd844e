// Attention of a chunk of new tokens over a paged cache, fp32, on the CUDA
// cores (the tensor cores take no fp32 operand; see chunk_bf16.cu for the
// formulas).  A CTA of 256 threads folds runs of 64 positions into up to 64
// rows (query tokens x query heads of one KV head).  The scores of a run are a
// 64 x 64 product of which a thread computes 4 x 4 from shared memory; the
// probabilities go back through shared memory (over the keys, which are done)
// for the second product, of which a thread holds 4 rows x head_dim / 16 dims in
// registers.  Everything is fp32, the exponentials by exp2f.  Two CTAs per SM,
// so that one computes while the other loads.

#include "chunk.cuh"

namespace nsv {
namespace {

using namespace sm;

constexpr int kThreadsF32 = 256;
constexpr int kR = kChunkRowsF32, kC = kChunkKeysF32;

template <int D>
struct SmemF32 {
  static constexpr int kLd = D + 4;  // rows padded so that 16 lanes hit 16 bank groups
  static constexpr int kLdP = kC + 4;
  static constexpr uint32_t kOffK = kR * kLd * 4;
  static constexpr uint32_t kOffV = kOffK + kC * kLd * 4;
  static constexpr uint32_t kOffOk = kOffV + kC * D * 4;
  static constexpr uint32_t kOffMerge = kOffOk + kC * 4;
  static constexpr uint32_t kTotal = kOffMerge + 16;
  static_assert(kR * kLdP <= kC * kLd, "probabilities fit over the keys");
};

template <int D>
__global__ void __launch_bounds__(kThreadsF32, 2) chunk_f32_kernel(
    const __grid_constant__ ChunkParams p) {
  using L = SmemF32<D>;
  constexpr int kVec = D / 64;  // float4 of a row's dims that a thread owns
  extern __shared__ __align__(16) unsigned char smem[];
  float* sq = reinterpret_cast<float*>(smem);
  float* sk = reinterpret_cast<float*>(smem + L::kOffK);
  float* sp = sk;
  float* sv = reinterpret_cast<float*>(smem + L::kOffV);
  int* s_ok = reinterpret_cast<int*>(smem + L::kOffOk);
  int* s_merge = reinterpret_cast<int*>(smem + L::kOffMerge);
  const int tid = threadIdx.x, lane = tid & 31;
  const int ty = tid >> 4, tx = tid & 15;
  const float* q = static_cast<const float*>(p.q);
  const float* kp = static_cast<const float*>(p.k_pool);
  const float* vp = static_cast<const float*>(p.v_pool);
  constexpr float kLog2e = 1.4426950408889634f;
  griddep_wait();
  ChunkWalk wk;
  wk.init(p, blockIdx.x);
  ChunkSegment s;
  while (wk.next<kC>(p, s)) {
    const int rows = s.t.n_tok * p.group;
    __syncthreads();  // the previous segment's readers are done
    for (int c = tid; c < kR * (D / 4); c += kThreadsF32) {
      const int r = c / (D / 4), v = c - r * (D / 4);
      const int tok = r / p.group, g = r - tok * p.group;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        x = __ldg(reinterpret_cast<const float4*>(
                      q + (((size_t)s.t.q0 + tok) * p.heads + s.head * p.group + g) * D) + v);
      *reinterpret_cast<float4*>(sq + r * L::kLd + v * 4) = x;
    }
    int2 see[4];
    int pos[4];
    float slope[4], m[4], l[4], acc[4][4 * kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, tok = r / p.group, g = r - tok * p.group;
      pos[i] = s.t.pos0 + tok;
      see[i] = r < rows ? chunk_sees(p, (long long)s.t.q0 + tok, pos[i], s.t.ctx) : make_int2(0, 0);
      slope[i] = r < rows && p.slopes ? __ldg(p.slopes + s.head * p.group + g) : 0.f;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 4 * kVec; ++e) acc[i][e] = 0.f;
    }
    const int32_t* table = p.block_tables + (size_t)s.t.row * p.max_blocks;
    for (int j = s.j0; j < s.j1; ++j) {
      const int t0 = s.t.kb + j * kC;
      __syncthreads();  // the run before has been read
      for (int c = tid; c < kC * (D / 4); c += kThreadsF32) {
        const int t = c / (D / 4), v = c - t * (D / 4);
        float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
        bool ok = (long long)t0 + t < s.t.ke;  // ke is at most the context
        if (ok) {
          const int b = __ldg(table + (t0 + t) / kBlock);
          ok = b >= 0 && b < p.pool_blocks;
          if (ok) {
            const size_t at =
                (((size_t)b * p.kv_heads + s.head) * kBlock + (t0 + t) % kBlock) * D + v * 4;
            kx = __ldg(reinterpret_cast<const float4*>(kp + at));
            vx = __ldg(reinterpret_cast<const float4*>(vp + at));
          } else if (v == 0) {
            atomicOr(p.status, (uint32_t)NSV_DEV_BAD_BLOCK);
          }
        }
        if (v == 0) s_ok[t] = ok;
        *reinterpret_cast<float4*>(sk + t * L::kLd + v * 4) = kx;
        *reinterpret_cast<float4*>(sv + t * D + v * 4) = vx;
      }
      __syncthreads();
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * L::kLd + d);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          b[c] = *reinterpret_cast<const float4*>(sk + (tx + 16 * c) * L::kLd + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sc[i][c] = fmaf(a[i].x, b[c].x, sc[i][c]);
            sc[i][c] = fmaf(a[i].y, b[c].y, sc[i][c]);
            sc[i][c] = fmaf(a[i].z, b[c].z, sc[i][c]);
            sc[i][c] = fmaf(a[i].w, b[c].w, sc[i][c]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = tx + 16 * c;
          float x = sc[i][c] * p.scale;
          if (p.cap > 0.f) x = p.cap * tanhf(x / p.cap);
          x = fmaf(-slope[i], fabsf((float)(pos[i] - t0 - t)), x) * kLog2e;
          const bool seen = t0 + t >= see[i].x && t0 + t < see[i].y && s_ok[t];
          sc[i][c] = seen ? x : -INFINITY;
          mx = fmaxf(mx, sc[i][c]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        if (mx > m[i]) {  // the same for the row's 16 lanes
          const float alpha = exp2f(m[i] - mx);
          m[i] = mx;
          l[i] *= alpha;
#pragma unroll
          for (int e = 0; e < 4 * kVec; ++e) acc[i][e] *= alpha;
        }
        const float sub = m[i] == -INFINITY ? 0.f : m[i];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sc[i][c] = exp2f(sc[i][c] - sub);
          sum += sc[i][c];
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        l[i] += sum;
      }
      __syncthreads();  // every thread is done with the keys
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sp[(ty * 4 + i) * L::kLdP + tx + 16 * c] = sc[i][c];
      __syncwarp();  // a row's probabilities are written and read by one warp
#pragma unroll 2
      for (int t = 0; t < kC; t += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pr[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * L::kLdP + t);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            const float4 x = *reinterpret_cast<const float4*>(sv + (t + u) * D + v * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = u == 0 ? pr[i].x : u == 1 ? pr[i].y : u == 2 ? pr[i].z : pr[i].w;
              acc[i][4 * v] = fmaf(w, x.x, acc[i][4 * v]);
              acc[i][4 * v + 1] = fmaf(w, x.y, acc[i][4 * v + 1]);
              acc[i][4 * v + 2] = fmaf(w, x.z, acc[i][4 * v + 2]);
              acc[i][4 * v + 3] = fmaf(w, x.w, acc[i][4 * v + 3]);
            }
          }
      }
    }
    const bool whole = s.first && s.last;
    const int slot = chunk_slot(blockIdx.x, s.first);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      float* o = chunk_out<float>(p, s.t.q0, s.head, r, D);
      const float inv = whole ? (l[i] > 0.f ? 1.f / l[i] : 0.f) : 1.f;
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        *(whole ? reinterpret_cast<float4*>(o + v * 64 + tx * 4)
                : chunk_acc(p, slot, D, v * 16 + tx, r)) =
            make_float4(acc[i][4 * v] * inv, acc[i][4 * v + 1] * inv, acc[i][4 * v + 2] * inv,
                        acc[i][4 * v + 3] * inv);
      if (!whole && tx == 0) p.ws_ml[(size_t)slot * p.tile_rows + r] = make_float2(m[i], l[i]);
    }
    if (!whole) {
      // publish the piece; the CTA whose piece is the last merges them all
      __syncthreads();
      if (tid < 32) {
        const int2 pc = chunk_pieces(p, s.head, s.tile, lane);
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
