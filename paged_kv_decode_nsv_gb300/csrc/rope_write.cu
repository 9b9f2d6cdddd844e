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
// All three kernels move each byte once, and HBM or the launch bounds them.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"

namespace nsv {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerThread = 4;

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

// What a thread that moves one pair of 16-byte vectors of a head does to it: which
// vectors they are, and its cosines and sines.  Halves: vectors i and i + R/2 of
// the rotated dimensions; interleaved and unrotated ones: 2i and 2i + 1.
template <typename T>
struct Pair {
  static constexpr int N = Vec<T>::N;
  int v0, v1;
  bool turn;
  float c[N], s[N];
  __device__ __forceinline__ void init(const RopeParams& p, int item, const float* row) {
    const int half = p.rotary_dim / (2 * N);  // vectors of half the rotated dimensions
    turn = item < half;
    v0 = 2 * item, v1 = 2 * item + 1;
    if (turn) {
      if (!p.interleaved) v0 = item, v1 = item + half;
      load_f32<N>(row + item * N, c);
      load_f32<N>(row + p.rotary_dim / 2 + item * N, s);
    }
  }
  __device__ __forceinline__ void apply(const RopeParams& p, uint4& r0, uint4& r1) const {
    if (!turn) return;
    float x[N], y[N];
    Vec<T>::unpack(r0, x);
    Vec<T>::unpack(r1, y);
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float a = x[i], b = x[i + 1], d = y[i], e = y[i + 1];
        x[i] = turn_a(a, b, c[i / 2], s[i / 2]);
        x[i + 1] = turn_b(a, b, c[i / 2], s[i / 2]);
        y[i] = turn_a(d, e, c[N / 2 + i / 2], s[N / 2 + i / 2]);
        y[i + 1] = turn_b(d, e, c[N / 2 + i / 2], s[N / 2 + i / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float a = x[i], b = y[i];
        x[i] = turn_a(a, b, c[i], s[i]);
        y[i] = turn_b(a, b, c[i], s[i]);
      }
    }
    r0 = Vec<T>::pack(x);
    r1 = Vec<T>::pack(y);
  }
};

// The row of the table for a token: null without rotation; *ok false (and flagged
// by `flag`) for a position that has none.
__device__ __forceinline__ const float* table_row(const RopeParams& p, long long token, bool flag,
                                                  bool* ok) {
  *ok = true;
  if (!p.positions) return nullptr;
  const int pos = __ldg(p.positions + token);
  if (pos < 0 || pos >= p.num_positions) {
    if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_POS);
    *ok = false;
    return nullptr;
  }
  return p.rotary + (size_t)pos * p.rotary_dim;
}

// A token's write slot; -1 (and flagged) outside the pool.
__device__ __forceinline__ long long slot_of(const RopeParams& p, long long token, bool flag) {
  const long long slot = __ldg(p.write_slots + token);
  if (slot >= 0 && slot < p.pool_slots) return slot;
  if (flag) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_SLOT);
  return -1;
}

// Query heads h0 .. of one token: a thread takes one pair of vectors of up to
// four heads, whose loads go out together and share the cosines and sines.
template <typename T, int D>
__device__ __forceinline__ void turn_queries(const RopeParams& p, long long token, int h0,
                                             int item, const float* row) {
  constexpr int NV = D / Vec<T>::N;  // vectors of a head
  Pair<T> t;
  t.init(p, item, row);
  const uint4* in =
      reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + token * p.q_stride);
  uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out)) + (size_t)token * p.heads * NV;
  uint4 r[kHeadsPerThread][2];
#pragma unroll
  for (int j = 0; j < kHeadsPerThread; ++j)
    if (h0 + j < p.heads) {
      r[j][0] = in[(h0 + j) * NV + t.v0];
      r[j][1] = in[(h0 + j) * NV + t.v1];
    }
#pragma unroll
  for (int j = 0; j < kHeadsPerThread; ++j)
    if (h0 + j < p.heads) {
      t.apply(p, r[j][0], r[j][1]);
      out[(h0 + j) * NV + t.v0] = r[j][0];
      out[(h0 + j) * NV + t.v1] = r[j][1];
    }
}

// Units of a token: (four query heads, pair) and (KV head, pair), in this order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const RopeParams p, int per_cta) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int NV = D / Vec<T>::N, kItems = NV / 2;
  const int q_units = (p.q ? (p.heads + kHeadsPerThread - 1) / kHeadsPerThread : 0) * kItems;
  const int units = q_units + p.kv_heads * kItems;
  const long long first = (long long)blockIdx.x * per_cta;
#pragma unroll 1
  for (int u = threadIdx.x; u < per_cta * units; u += kThreads) {
    const int ti = u / units, w = u - ti * units;
    const long long token = first + ti;
    if (token >= p.tokens) break;
    bool ok;
    const float* row = table_row(p, token, w == 0, &ok);
    if (!ok) continue;
    const int item = w % kItems;
    if (w < q_units) {
      turn_queries<T, D>(p, token, w / kItems * kHeadsPerThread, item, row);
      continue;
    }
    const int g = (w - q_units) / kItems;
    const long long slot = slot_of(p, token, w == q_units);
    if (slot < 0) continue;
    Pair<T> t;
    t.init(p, item, row);
    const uint4* k =
        reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + token * p.k_stride) + g * NV;
    const uint4* v =
        reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + token * p.v_stride) + g * NV;
    uint4 k0 = k[t.v0], k1 = k[t.v1];
    const uint4 v0 = v[t.v0], v1 = v[t.v1];
    const size_t dst =
        ((size_t)(slot / kBlock * p.kv_heads + g) * kBlock + slot % kBlock) * NV;
    t.apply(p, k0, k1);
    static_cast<uint4*>(p.k_pool)[dst + t.v0] = k0;
    static_cast<uint4*>(p.k_pool)[dst + t.v1] = k1;
    static_cast<uint4*>(p.v_pool)[dst + t.v0] = v0;
    static_cast<uint4*>(p.v_pool)[dst + t.v1] = v1;
  }
}

// Elements d .. d + 7 of one head of one token, fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* x, int d, float* y) {
#pragma unroll
  for (int i = 0; i < 8; i += Vec<T>::N)
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(x + d + i), y + i);
}

// The same rotated.  (A half of the rotated dimensions is a whole number of eights.)
template <typename T>
__device__ __forceinline__ void load8_turned(const RopeParams& p, const T* x, int d,
                                             const float* row, float* y) {
  load8(x, d, y);
  if (!row || d >= p.rotary_dim) return;
  const int half = p.rotary_dim / 2;
  if (p.interleaved) {
    float c[4], s[4];
    load_f32<4>(row + d / 2, c);
    load_f32<4>(row + half + d / 2, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      y[2 * i] = turn_a(a, b, c[i], s[i]);
      y[2 * i + 1] = turn_b(a, b, c[i], s[i]);
    }
    return;
  }
  float c[8], s[8], z[8];
  const bool upper = d >= half;
  const int e = upper ? d - half : d;
  load_f32<8>(row + e, c);
  load_f32<8>(row + half + e, s);
  load8(x, upper ? e : d + half, z);  // the other of each pair
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = upper ? turn_b(z[i], y[i], c[i], s[i]) : turn_a(y[i], z[i], c[i], s[i]);
}

// 16 dimensions of a token and KV head to their numbers and scale.
__device__ __forceinline__ void store16(float* y, const float* head_scale, uint8_t* tile, int off,
                                        int group, int head_dim) {
  if (head_scale) {
    const float h = __ldg(head_scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(y[i], h);
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
  const uint32_t code = to_e4m3(__fdiv_rn(top, 6.f));
  const __half2 wide = __half2(__half2_raw{(unsigned short)(e4m3x2_to_half(code) & 0xffffu), 0});
  const float s = __low2float(wide);
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      w[i / 8] |= to_e2m1x2(__fdiv_rn(y[i], s), __fdiv_rn(y[i + 1], s)) << (4 * (i % 8));
  }
  *reinterpret_cast<uint2*>(tile + off * (head_dim / 2) + group * 8) = make_uint2(w[0], w[1]);
  tile[kv4_number_bytes(head_dim) + off * (head_dim / 16) + group] = (uint8_t)code;
}

// Units of a token: (four query heads, pair), then (keys or values, KV head, 16
// dimensions).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const RopeParams p, int per_cta) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kItems = D / Vec<T>::N / 2, kGroups = D / 16;
  const int q_units = (p.q ? (p.heads + kHeadsPerThread - 1) / kHeadsPerThread : 0) * kItems;
  const int units = q_units + 2 * p.kv_heads * kGroups;
  const long long first = (long long)blockIdx.x * per_cta;
#pragma unroll 1
  for (int u = threadIdx.x; u < per_cta * units; u += kThreads) {
    const int ti = u / units, w = u - ti * units;
    const long long token = first + ti;
    if (token >= p.tokens) break;
    bool ok;
    const float* row = table_row(p, token, w == 0, &ok);
    if (!ok) continue;
    if (w < q_units) {
      turn_queries<T, D>(p, token, w / kItems * kHeadsPerThread, w % kItems, row);
      continue;
    }
    int g = (w - q_units) / kGroups;
    const int group = (w - q_units) % kGroups;
    const long long slot = slot_of(p, token, w == q_units);
    if (slot < 0) continue;
    const bool value = g >= p.kv_heads;
    if (value) g -= p.kv_heads;
    const T* x = (value ? static_cast<const T*>(p.v) + token * p.v_stride
                        : static_cast<const T*>(p.k) + token * p.k_stride) + g * D;
    float y[16];
    load8_turned(p, x, group * 16, value ? nullptr : row, y);
    load8_turned(p, x, group * 16 + 8, value ? nullptr : row, y + 8);
    const float* scales = value ? p.v_scales : p.k_scales;
    uint8_t* tile = static_cast<uint8_t*>(value ? p.v_pool : p.k_pool) +
                    (size_t)(slot / kBlock * p.kv_heads + g) * kv4_tile_bytes(D);
    store16(y, scales ? scales + g : nullptr, tile, (int)(slot % kBlock), group, D);
  }
}

// A thread widens 8 dimensions of a slot's key and value.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4ReadParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kItems = D / 8;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int item = (int)(i % kItems);
  const long long th = i / kItems;
  const long long token = th / p.kv_heads;
  const int g = (int)(th - token * p.kv_heads);
  if (token >= p.tokens) return;
  const long long slot = __ldg(p.slots + token);
  if (slot < 0 || slot >= p.pool_slots) {
    if (item == 0 && g == 0) atomicOr(p.status, (uint32_t)NSV_DEV_BAD_SLOT);
    return;
  }
  const size_t tile = (size_t)(slot / kBlock * p.kv_heads + g) * kv4_tile_bytes(D);
  const int off = (int)(slot % kBlock);
  const size_t at = tile + off * (D / 2) + item * 4;
  const size_t sc = tile + kv4_number_bytes(D) + off * (D / 16) + item / 2;
  const uint32_t num[2] = {__ldg(reinterpret_cast<const uint32_t*>(p.k_pool + at)),
                           __ldg(reinterpret_cast<const uint32_t*>(p.v_pool + at))};
  const uint32_t sb[2] = {__ldg(p.k_pool + sc), __ldg(p.v_pool + sc)};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t h[4];
    e2m1x8_to_half(num[kv], h);
    const uint32_t sh = e4m3x2_to_half(sb[kv]);
    const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
    const float* scales = kv ? p.v_scales : p.k_scales;
    const float unit = scales ? __ldg(scales + g) : 1.f;
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      x[2 * j] = __fmul_rn(__fmul_rn(f.x, s), unit);
      x[2 * j + 1] = __fmul_rn(__fmul_rn(f.y, s), unit);
    }
    T* out = static_cast<T*>(kv ? p.v_out : p.k_out) + (size_t)th * D + item * 8;
#pragma unroll
    for (int j = 0; j < 8; j += Vec<T>::N)
      *reinterpret_cast<uint4*>(out + j) = Vec<T>::pack(x + j);
  }
}

// Tokens one CTA takes, so that its threads have a unit each.
int tokens_per_cta(int units) { return units >= kThreads ? 1 : kThreads / units; }

template <typename T, int D>
cudaError_t launch_append(const RopeParams& p, bool four, cudaStream_t stream) {
  const int items = D / Vec<T>::N / 2;
  const int q_units = (p.q ? (p.heads + kHeadsPerThread - 1) / kHeadsPerThread : 0) * items;
  const int units = q_units + p.kv_heads * (four ? 2 * (D / 16) : items);
  const int per_cta = tokens_per_cta(units);
  const unsigned grid = (unsigned)((p.tokens + per_cta - 1) / per_cta);
  if (four)
    kv4_write_kernel<T, D><<<grid, kThreads, 0, stream>>>(p, per_cta);
  else
    rope_write_kernel<T, D><<<grid, kThreads, 0, stream>>>(p, per_cta);
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
  const long long n = p.tokens * p.kv_heads * (D / 8);
  kv4_read_kernel<T, D><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
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
