// Internal declarations of the rotating appends and of the 4-bit cache
// (nsv_rope_write, nsv_kv4_write, nsv_kv4_read, nsv_kv4_chunk): the format of
// its pools, the conversions between it and fp16, and the kernels' parameters.
//
// A tile is 16 tokens of one KV head: 16 x head_dim / 2 bytes of e2m1 pairs (the
// even dimension in the low half), then 16 x head_dim / 16 e4m3 scales, one for 16
// dimensions.  A number times its scale has at most 6 significant bits and lies
// within 2^-10 .. 2688, so that it is exact in fp16 and in bf16: the attention
// multiplies what the cache holds, not a rounding of it.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chunk.cuh"
#include "nsv_common.cuh"

namespace nsv {

// Bytes of a tile, of its numbers, and of one token's numbers and scales.
__host__ __device__ constexpr int kv4_tile_bytes(int head_dim) { return kBlock * head_dim * 9 / 16; }
__host__ __device__ constexpr int kv4_number_bytes(int head_dim) { return kBlock * head_dim / 2; }

// A rotating append, into pools of the new tokens' type or into 4-bit ones.
struct RopeParams {
  const void* q;      // null: no queries
  const void* k;
  const void* v;
  const int32_t* positions;  // null: no rotation
  const float* rotary;       // [num_positions][rotary_dim]
  const int64_t* write_slots;
  const float* k_scales;  // [kv_heads] or null (4-bit pools only)
  const float* v_scales;
  void* q_out;
  void* k_pool;
  void* v_pool;
  uint32_t* status;
  long long tokens, q_stride, k_stride, v_stride;  // strides of a token, in elements
  long long pool_slots, num_positions;
  int heads, kv_heads, rotary_dim, interleaved;
};

struct Kv4ReadParams {
  const int64_t* slots;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scales;
  const float* v_scales;
  void* k_out;
  void* v_out;
  uint32_t* status;
  long long tokens, pool_slots;
  int kv_heads;
};

// The vector form of the attention: few query vectors per tile, on mma.sync.
struct Kv4VecParams {
  ChunkParams c;  // its plan: kv_heads counts the groups of heads that workers take
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scales;
  const float* v_scales;
  int4* todo;     // [workers] what each has to merge: {first query token, tokens, group, pieces}
  float2* ml;     // [workers][2][heads_per_worker][vectors]
  float* acc;     // [workers][2][heads_per_worker][vectors][head_dim]
  // Where it is not 0 there is no list: every CTA works its shares out itself, a row
  // having at most this many tiles.
  int row_tiles;
  int kv_heads, heads_per_worker, workers_per_cta;
  int subs;       // parts that a KV head's query heads are taken in
};

// Query vectors of a tile of the vector form: 8 a column tile of the MMA.
constexpr int kVecKeys = 32;  // positions of one unit: two blocks
constexpr int kVecMostVectors = 24, kVecMostVectorsF32 = 64;  // of a row and KV head
constexpr int kVecTileCost = 3;   // of a tile, in units
constexpr int kVecLeastUnits = 2; // of a share, where CTAs work them out themselves
// The most tiles (rows times row_tiles) that they do it for: eight a thread.
constexpr int kVecOwnTiles = 2048;
constexpr int kVecWholeRuns = 8;  // as kChunkWholeRuns

cudaError_t launch_rope_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4ReadParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_vec(const Kv4VecParams& p, int dtype, int head_dim, int col_tiles,
                           cudaStream_t stream);
cudaError_t prepare_kv4_vec();
// Warps of one CTA of the vector form, and its CTAs per SM.
int kv4_vec_warps(int dtype, int col_tiles);
int kv4_vec_ctas_per_sm(int dtype, int col_tiles);

#ifdef __CUDACC__
// Four pairs of e2m1 numbers (the low half of a byte first) to fp16.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t x, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(x));
}
// Two e4m3 numbers (the low byte first) to fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t x) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(x));
  return h;
}
// To nearest even, saturating: e4m3 of one value; e2m1 of eight, the first lowest.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
#endif

}  // namespace nsv
