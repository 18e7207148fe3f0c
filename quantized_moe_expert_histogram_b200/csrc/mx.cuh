// MXFP4 (OCP microscaling, 4-bit): 32 consecutive elements along K share one
// power-of-two scale.
//
//   a = max |v| of the block, S = floor(log2 a) - 2 clamped to [-127, 127]
//   code = e2m1(v / 2^S), round-half-even, saturating at 6
//   scale byte = S + 127 (255: the block stands for NaN)
//
// The exponent of the largest e2m1 value is 2 (6 = 1.5 * 2^2), hence the
// -2.  Both divisions are by powers of two, so the code is the correctly
// rounded one: one rounding per element, the format's own.
#pragma once

#include "common.cuh"

namespace moeq {

constexpr int kMxBlock = 32;  // elements per scale

// Scale byte of a block from the largest magnitude's fp32 bits (sign
// cleared).  Biased exponent b of the fp32 value: floor(log2 a) + 127, so
// the byte is b - 2 (0 where that would be negative: zeros, subnormals);
// Inf and NaN (b = 255) give 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int b = static_cast<int>(amax_bits >> 23);
  return b == 255 ? 255u : static_cast<uint32_t>(max(b - 2, 0));
}

// 2^-S of a scale byte below 255 (exponent bits 254 - byte, in [2, 254]).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^S of a scale byte (byte 0 is the subnormal 2^-127; 255 is NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : byte == 0u ? 0x00400000u : byte << 23);
}

// Eight scaled values -> eight e2m1 codes, element i in nibble i.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight e2m1 codes -> their values (exact in fp16).
__device__ __forceinline__ void mx_decode8(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// Byte of (row, 32-block) inside a weight matrix's scale section: tiles of
// 128 rows x 128 K (4 blocks), 512 bytes each, K inside a row of tiles;
// inside a tile row r, block b sits at (r % 32) * 16 + (r / 32) * 4 + b.
// That is the order in which the block-scaled MMA's scale operand lies in
// tensor memory (lane r % 32, column r / 32, byte b), so that a tile goes
// there with one copy.
__host__ __device__ __forceinline__ size_t mx_scale_at(size_t row, int blk, int K) {
  return ((row >> 7) * static_cast<size_t>(K / 128) + blk / 4) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (blk & 3);
}

// Bytes of an MXFP4 weight matrix [N][K]: codes [N][K/2], then the scales.
inline size_t mx_matrix_bytes(int N, int K) {
  return static_cast<size_t>(N) * (K / 2) + static_cast<size_t>(N) * (K / 32);
}

struct MxGemmArgs {
  const uint8_t* a_codes;   // [rows][K/2]
  const uint8_t* a_scales;  // [rows][K/32]
  const int32_t* offsets;   // [E + 1]
  const uint8_t* mats;      // matrix of expert e at mats + e * mat_stride
  size_t mat_stride;
  int rows, E, N, K;
  int out_kind;  // kMxOut*
  void* out;     // [rows][N]; kMxOutSwiglu: codes [rows][N/4] of h [rows][N/2]
  uint8_t* out_scales;  // kMxOutSwiglu: [rows][N/64]
  int32_t* status;
};
enum { kMxOutF16 = 0, kMxOutBf16 = 1, kMxOutF32 = 2, kMxOutSwiglu = 3 };
moe_status_t launch_mx_gemm(const MxGemmArgs& a, cudaStream_t s);
constexpr int kMxMaxExperts = 256;
extern int g_mx_stall;  // test hook moe_debug_mx_timeout

}  // namespace moeq
