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
  Chunk4Params c;  // its plan: kv_heads counts the groups of heads that workers take
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

constexpr int kVecWarps = 8;  // of a CTA of the vector form, at most
constexpr int kVecKeys = 32;  // positions of one unit of the vector form: two blocks
// Most query vectors of a row and KV head that it takes; rows that bring more go to the
// tcgen05 forms.  The rule looks at a row's vectors alone, not at the call's rows or contexts,
// nor at whether the caller names the most tokens of a row, which saves the planning launch
// and, in bf16, takes two column tiles.  In us here, named and not, and there, replayed from a
// graph, 32 heads, 8 KV heads, head_dim 128 (of a row; "-": not taken):
//                                 12 vectors       24              32              64
//   bf16  29 rows over 4000     50   72   97   82   96  100   83  117  101  150  209  102
//         1 row over 30000      26   33   37   33   39   41    -    -    -   49   67   44
//   fp32  29 rows over 4000      -    -    -    -    -    -  148  155  309  277  286  311
//         1 row over 30000      32   34   72    -    -    -    -    -    -   81   84   78
// (Named, 32 vectors of bf16 would gain as much as 24 do.)
constexpr int kVecMostVectors = 24, kVecMostVectorsF32 = 64;
// Cost of a tile, in units.  256 single tokens: 160 us at 1, 158.6 at 3; a few short rows do
// not care up to 3 (18.9 us; 19.5 at 5).
constexpr int kVecTileCost = 3;
// Least units of a share, where CTAs work them out themselves (a few short rows: 26 us at 1,
// 19.7 to 22 at 2, 20.5 at 4).
constexpr int kVecLeastUnits = 2;
// Workers for each tile and group of heads, at most: so the most pieces of a tile where all
// are alike.  It binds only where a call has few tiles; beside others a long tile is cut into
// what its share of the units gives.  One token over 131072 positions, 8 heads of 1 KV head: 128
// pieces 56 us, 256 42, 384 40, 2432 75; two over 32768, head_dim 64: 23, 21, 25.  (Replayed
// from a graph 35 us alone, and beside 1, 3, 10 and 30 rows of 200 to 600 positions 37, 41, 63
// and 64; with 32 heads over 8 51 to 54 in all of these.)
constexpr int kVecMostPieces = 256;
// The most tiles (rows times row_tiles) that CTAs work their shares out of themselves: eight
// a thread.  With a list instead, 256 single tokens take 165 us in place of 160, four 23.6 in
// place of 18.9.
constexpr int kVecOwnTiles = 2048;

cudaError_t launch_rope_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_write(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4ReadParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kv4_vec(const Kv4VecParams& p, int dtype, int head_dim, int col_tiles,
                           cudaStream_t stream);
cudaError_t prepare_kv4_vec();
// CTAs per SM of the vector form.
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
