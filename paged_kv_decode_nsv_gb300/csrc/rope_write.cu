// Appends that rotate on the way, and the way into and out of a 4-bit cache.
//
// Rotation: a pair (a, b) of a query's or key's first rotary_dim dimensions, at
// position m with cosine c and sine s of its angle from the table, becomes
//   (a c - b s, b c + a s),
// in fp32 with every product and sum rounded on its own (no fused multiply-add), so
// that the same inputs give the same bits on any implementation; then it is rounded
// once to the element type.  Pairs are dimensions (i, i + rotary_dim / 2), or (2i,
// 2i + 1) when interleaved.
//
// 4-bit cache: 16 dimensions x of a token and KV head, y = x / head scale, share a
// scale s = e4m3(max |y| / 6), and are stored as e2m1(y / s) (zeros where s is 0);
// keys are quantised from the unrounded rotation.  Quotients are rounded to fp32 and
// conversions to nearest even.
//
// All three kernels move each byte once.  The launch bounds small calls of each, and HBM
// large ones of the append that keeps the type and of the read: 8192 tokens of 32 query and 8
// KV heads, head_dim 128, rotated 35 us in bf16 (88 % of the copy bandwidth) and 62 in fp32
// (98 %); 65536 tokens of 8 KV heads read back 64 us (81 %, mostly writes) and 126 (73 %).
// Quantising is bound by its chain of loads, divisions and conversions: 16381 tokens take 76
// us in bf16 where their bytes take 51, 8192 in fp32 58 where theirs take 52.  (72 registers a
// thread in bf16, of which 20 bytes are spilled; 64, which spill more, 78, and 80, with fewer
// warps, 81.  fp32 has 96 and spills 4 bytes.)

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"

namespace nsv {
namespace {

// Of an append (8192 tokens with their queries: 35.0 us, 128 threads 36.2; 32 threads 53),
// and of a read, whose threads wait less (65536 tokens: 63.7 us, 64 threads 69.6).
constexpr int kThreads = 64, kReadThreads = 256;
constexpr int kPasses = 2;  // heads of a lane whose loads go out together (1: 110 us against 98)

// 16 bytes of elements as fp32, and back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 r, float* x) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(sm::pack_bf16(x[0], x[1]), sm::pack_bf16(x[2], x[3]),
                      sm::pack_bf16(x[4], x[5]), sm::pack_bf16(x[6], x[7]));
  }
};

__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

template <int N>
__device__ __forceinline__ void load_f32(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// 8 elements of a head: what a lane holds of one.
template <typename T>
struct Eight {
  static constexpr int N = 8 / Vec<T>::N;
  uint4 r[N];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  __device__ __forceinline__ void store(T* x) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(x)[i] = r[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* y) const {
#pragma unroll
    for (int i = 0; i < N; ++i) Vec<T>::unpack(r[i], y + i * Vec<T>::N);
  }
  __device__ __forceinline__ void set(const float* y) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = Vec<T>::pack(y + i * Vec<T>::N);
  }
};

// What a lane holds of a head: dimensions 8 u .. and 8 v .., and what the rotation does to
// them.  kPairs: halves, v is u's partner.  kOwn: interleaved or not rotated, u and v lie
// together.  kApart: halves of which a scale's 16 dimensions do not lie in one; u and v lie
// together, and their partners are loaded besides.
enum : int { kPairs, kOwn, kApart };
template <typename T>
struct Turn {
  int u, v, mode;
  bool turn;
  float c[8], s[8];
  // The lane's place: `l` counts the head's lanes, of 16 dimensions each.
  __device__ __forceinline__ void place(const RopeParams& p, int l, bool four) {
    const int half = p.rotary_dim / 16;
    mode = p.interleaved || l >= half ? kOwn : kPairs;
    turn = p.positions && l < half;
    u = 2 * l, v = 2 * l + 1;
    if (four && !p.interleaved && (half & 1)) {
      mode = kApart;
      turn = p.positions != nullptr;
    } else if (mode == kPairs) {
      u = l, v = l + half;
    }
  }
  __device__ __forceinline__ void init(const RopeParams& p, const float* row) {
    if (!turn || mode == kApart) return;
    if (mode == kPairs) {
      load_f32<8>(row + 8 * u, c);
      load_f32<8>(row + p.rotary_dim / 2 + 8 * u, s);
    } else {  // interleaved: pairs 4 u ..
      load_f32<8>(row + 4 * u, c);
      load_f32<8>(row + p.rotary_dim / 2 + 4 * u, s);
    }
  }
  // x: the head.
  __device__ __forceinline__ void apply(const RopeParams& p, const T* x, const float* row,
                                        float* a, float* b) const {
    if (!turn) return;
    if (mode == kPairs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = a[i], f = b[i];
        a[i] = turn_a(e, f, c[i], s[i]);
        b[i] = turn_b(e, f, c[i], s[i]);
      }
    } else if (mode == kOwn) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float* y = i < 4 ? a + 2 * i : b + 2 * (i - 4);
        const float e = y[0], f = y[1];
        y[0] = turn_a(e, f, c[i], s[i]);
        y[1] = turn_b(e, f, c[i], s[i]);
      }
    } else {
      apart(p, x, row, 8 * u, a);
      apart(p, x, row, 8 * v, b);
    }
  }
  static __device__ __forceinline__ void apart(const RopeParams& p, const T* x, const float* row,
                                               int d, float* y) {
    if (d >= p.rotary_dim) return;
    const int half = p.rotary_dim / 2;
    const bool upper = d >= half;
    const int e = upper ? d - half : d;
    const float *c = row + e, *sn = row + half + e;
    const T* o = x + (upper ? e : d + half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = to_float(o[i]);
      const float ci = __ldg(c + i), si = __ldg(sn + i);
      y[i] = upper ? turn_b(z, y[i], ci, si) : turn_a(y[i], z, ci, si);
    }
  }
};

// The quotient x / d rounded to nearest, from r = 1 / d rounded to nearest: the residual of
// the first product is exact, and the correction by it rounds as the quotient does
// (P. Markstein, Computation of elementary functions on the IBM RISC System/6000, 1990).
// Where the residual underflows (|x| below 2^-101, d within 2^-60 .. 2^60) the quotient may
// be off, but so far below the smallest number that it is stored as 0 either way.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float y = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-y, d, x), r, y);
}

// 8 dimensions as numbers of scale s, whose reciprocal is r.
__device__ __forceinline__ uint32_t numbers8(const float* y, float s, float r) {
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = quotient(y[i], s, r);
  const uint32_t w = to_e2m1x8(z);
  return s == 0.f ? 0u : w;
}

// A unit is up to kPasses passes over one token's query heads, keys or values, by a warp: a
// lane holds 16 dimensions of a head in each, all loads go out together, and the token's
// cosines and sines serve them all.  The position's row of the table is the only load that
// has to wait for another.  Times of 8192 tokens appended, and 16381 into 4 bits (with
// their values read back, 16 us), before later steps: 8 dimensions a lane, partners by
// shuffles 44 and 105 us; a thread with four whole heads' pairs, 111 to 147 registers, 43
// and 127.
template <typename T, int D, bool FOUR>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 10 : FOUR ? 14 : 16)
    append_kernel(const RopeParams p, int q_units, int kv_units) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes of a head; heads of a pass
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int units = q_units + 2 * kv_units;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long token = unit >> 32 ? unit / units : (uint32_t)unit / (uint32_t)units;
  if (token >= p.tokens) return;
  int n = (int)(unit - token * units);
  const bool query = n < q_units, value = n >= q_units + kv_units;
  n -= query ? 0 : value ? q_units + kv_units : q_units;
  const int heads = query ? p.heads : p.kv_heads;
  const T* src = query   ? static_cast<const T*>(p.q) + token * p.q_stride
                 : value ? static_cast<const T*>(p.v) + token * p.v_stride
                         : static_cast<const T*>(p.k) + token * p.k_stride;
  const int h0 = n * kPasses * kHeads + lane / kLanes;
  const int pos = p.positions ? __ldg(p.positions + token) : 0;
  const long long slot = query ? 0 : __ldg(p.write_slots + token);
  Turn<T> t;
  t.place(p, l, FOUR && !query);
  Eight<T> x[kPasses][2];
#pragma unroll
  for (int j = 0; j < kPasses; ++j) {
    const int h = h0 + j * kHeads;
    if (h < heads) {
      x[j][0].load(src + (size_t)h * D + 8 * t.u);
      x[j][1].load(src + (size_t)h * D + 8 * t.v);
    } else {
      x[j][0].clear();
      x[j][1].clear();
    }
  }
  // (flagged by the token's first keys' unit)
  const bool flag = lane == 0 && n == 0 && !query && !value;
  const float* row = nullptr;
  if (p.positions) {
    if (pos < 0 || pos >= p.num_positions) {
      if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_POS);
      return;
    }
    row = p.rotary + (size_t)pos * p.rotary_dim;
  }
  if (slot < 0 || slot >= p.pool_slots) {
    if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_SLOT);
    return;
  }
  t.turn = t.turn && !value;
  t.init(p, row);
  const long long block = slot / kBlock;
  const int off = (int)(slot % kBlock);
  const float* units_of = value ? p.v_scales : p.k_scales;
#pragma unroll
  for (int j = 0; j < kPasses; ++j) {
    const int h = h0 + j * kHeads;
    if (!FOUR || query) {
      if (h >= heads) continue;
      if (t.turn) {
        float a[8], b[8];
        x[j][0].get(a);
        x[j][1].get(b);
        t.apply(p, src + (size_t)h * D, row, a, b);
        x[j][0].set(a);
        x[j][1].set(b);
      }
      T* out = query ? static_cast<T*>(p.q_out) + ((size_t)token * p.heads + h) * D
                     : static_cast<T*>(value ? p.v_pool : p.k_pool) +
                           ((size_t)(block * p.kv_heads + h) * kBlock + off) * D;
      x[j][0].store(out + 8 * t.u);
      x[j][1].store(out + 8 * t.v);
      continue;
    }
    const bool real = h < heads;
    float a[8], b[8];
    x[j][0].get(a);
    x[j][1].get(b);
    if (real) t.apply(p, src + (size_t)h * D, row, a, b);
    float top_a = 0.f, top_b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top_a = fmaxf(top_a, fabsf(a[i]));
      top_b = fmaxf(top_b, fabsf(b[i]));
    }
    if (units_of) {
      const float d = real ? __ldg(units_of + h) : 1.f, r = __frcp_rn(d);
      const float most = 4096.f * d;  // beyond 2688 all quotients end the same
      if (__any_sync(sm::kFull, fmaxf(top_a, top_b) > most)) {
        top_a = fminf(top_a, most);
        top_b = fminf(top_b, most);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = fminf(fmaxf(a[i], -most), most);
          b[i] = fminf(fmaxf(b[i], -most), most);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = quotient(a[i], d, r);
        b[i] = quotient(b[i], d, r);
      }
      // (rounding keeps the order: the largest quotient is the largest's)
      top_a = quotient(top_a, d, r);
      top_b = quotient(top_b, d, r);
    }
    // a scale's 16 dimensions: the lane's own, or 8 of its neighbour's
    const float next_a = __shfl_xor_sync(sm::kFull, top_a, 1);
    const float next_b = __shfl_xor_sync(sm::kFull, top_b, 1);
    const bool pairs = t.mode == kPairs;
    top_a = fmaxf(top_a, pairs ? next_a : top_b);
    top_b = pairs ? fmaxf(top_b, next_b) : top_a;
    const uint32_t code_a = to_e4m3(quotient(top_a, 6.f, 1.f / 6.f));
    const uint32_t code_b = to_e4m3(quotient(top_b, 6.f, 1.f / 6.f));
    const uint32_t wide = e4m3x2_to_half(code_a | (code_b << 8));
    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&wide));
    const uint32_t wa = numbers8(a, s.x, __frcp_rn(s.x)), wb = numbers8(b, s.y, __frcp_rn(s.y));
    const uint32_t other = __shfl_xor_sync(sm::kFull, lane & 1 ? wa : wb, 1);
    if (!real) continue;
    uint8_t* tile = static_cast<uint8_t*>(value ? p.v_pool : p.k_pool) +
                    (size_t)(block * p.kv_heads + h) * kv4_tile_bytes(D);
    // 16 dimensions that lie together: of partners, the even lane stores a's and the odd one b's
    const bool upper = pairs && (lane & 1);
    const int first = upper ? t.v - 1 : t.u;
    const uint2 num = make_uint2(upper ? other : wa, pairs && !upper ? other : wb);
    *reinterpret_cast<uint2*>(tile + off * (D / 2) + first * 4) = num;
    tile[kv4_number_bytes(D) + off * (D / 16) + first / 2] = (uint8_t)(upper ? code_b : code_a);
  }
}

// A thread widens 8 dimensions of the keys and values of kReads slots, whose loads go out
// together.
constexpr int kReads = 2;
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) kv4_read_kernel(const Kv4ReadParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kItems = D / 8;
  const long long i = (long long)blockIdx.x * kReadThreads + threadIdx.x;
  const int item = (int)(i % kItems);
  const long long th = i / kItems;
  const long long t0 = th / p.kv_heads;  // the thread's tokens are `step` apart
  const int g = (int)(th - t0 * p.kv_heads);
  const long long step = (p.tokens + kReads - 1) / kReads;
  if (t0 >= step) return;
  long long slot[kReads];
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    const long long t = t0 + k * step;
    slot[k] = t < p.tokens ? __ldg(p.slots + t) : -1;
    if (slot[k] < 0 || slot[k] >= p.pool_slots) {
      if (t < p.tokens && item == 0 && g == 0) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_SLOT);
      slot[k] = -1;
    }
  }
  uint32_t num[kReads][2], sb[kReads][2];
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    if (slot[k] < 0) continue;
    const size_t tile = (size_t)(slot[k] / kBlock * p.kv_heads + g) * kv4_tile_bytes(D);
    const int off = (int)(slot[k] % kBlock);
    const size_t at = tile + off * (D / 2) + item * 4;
    const size_t sc = tile + kv4_number_bytes(D) + off * (D / 16) + item / 2;
    num[k][0] = __ldg(reinterpret_cast<const uint32_t*>(p.k_pool + at));
    num[k][1] = __ldg(reinterpret_cast<const uint32_t*>(p.v_pool + at));
    sb[k][0] = __ldg(p.k_pool + sc);
    sb[k][1] = __ldg(p.v_pool + sc);
  }
  const float unit[2] = {p.k_scales ? __ldg(p.k_scales + g) : 1.f,
                         p.v_scales ? __ldg(p.v_scales + g) : 1.f};
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    if (slot[k] < 0) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t h[4];
      e2m1x8_to_half(num[k][kv], h);
      const uint32_t sh = e4m3x2_to_half(sb[k][kv]);
      const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        x[2 * j] = __fmul_rn(__fmul_rn(f.x, s), unit[kv]);
        x[2 * j + 1] = __fmul_rn(__fmul_rn(f.y, s), unit[kv]);
      }
      T* out = static_cast<T*>(kv ? p.v_out : p.k_out) +
               ((size_t)(t0 + k * step) * p.kv_heads + g) * D + item * 8;
#pragma unroll
      for (int j = 0; j < 8; j += Vec<T>::N)
        *reinterpret_cast<uint4*>(out + j) = Vec<T>::pack(x + j);
    }
  }
}

template <typename T, int D>
cudaError_t launch_append(const RopeParams& p, bool four, cudaStream_t stream) {
  const int heads = kPasses * 512 / D;  // of a unit
  const int q_units = p.q ? (p.heads + heads - 1) / heads : 0;
  const int kv_units = (p.kv_heads + heads - 1) / heads;
  const long long units = p.tokens * (q_units + 2 * kv_units);
  const unsigned grid = (unsigned)((units * 32 + kThreads - 1) / kThreads);
  if (four)
    append_kernel<T, D, true><<<grid, kThreads, 0, stream>>>(p, q_units, kv_units);
  else
    append_kernel<T, D, false><<<grid, kThreads, 0, stream>>>(p, q_units, kv_units);
  return cudaGetLastError();
}

cudaError_t launch_any(const RopeParams& p, int dtype, int head_dim, bool four,
                       cudaStream_t stream) {
  if (dtype == NSV_F32)
    return head_dim == 64 ? launch_append<float, 64>(p, four, stream)
                          : launch_append<float, 128>(p, four, stream);
  return head_dim == 64 ? launch_append<__nv_bfloat16, 64>(p, four, stream)
                        : launch_append<__nv_bfloat16, 128>(p, four, stream);
}

template <typename T, int D>
cudaError_t launch_read(const Kv4ReadParams& p, cudaStream_t stream) {
  const long long n = (p.tokens + kReads - 1) / kReads * p.kv_heads * (D / 8);
  kv4_read_kernel<T, D>
      <<<(unsigned)((n + kReadThreads - 1) / kReadThreads), kReadThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream) {
  return launch_any(p, dtype, head_dim, false, stream);
}

cudaError_t launch_kv4_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream) {
  return launch_any(p, dtype, head_dim, true, stream);
}

cudaError_t launch_kv4_read(const Kv4ReadParams& p, int dtype, int head_dim, cudaStream_t stream) {
  if (dtype == NSV_F32)
    return head_dim == 64 ? launch_read<float, 64>(p, stream) : launch_read<float, 128>(p, stream);
  return head_dim == 64 ? launch_read<__nv_bfloat16, 64>(p, stream)
                        : launch_read<__nv_bfloat16, 128>(p, stream);
}

}  // namespace nsv
