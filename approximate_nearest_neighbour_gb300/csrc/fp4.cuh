// 4-bit block-scaled vectors: element and scale conversions and the packed
// layout shared by the fp4_* kernels.
//
// An element is E2M1 (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2,
// 3, 4, 6 in magnitude). MXFP4 gives 32 consecutive columns one power-of-two
// scale (E8M0, value 2^(byte - 127)); NVFP4 gives 16 columns one E4M3 scale
// and a matrix one fp32 scale besides.
//
// Packed layout of [rows, cols], kp = cols rounded up to 32:
//  codes   [rows, kp / 2] bytes, even column in the low half, zero past cols
//  scales  tiles of 128 rows x 4 blocks, 512 bytes, [ceil(rows / 128)]
//          [ceil(nblk / 4)]: row r, block c at byte
//          (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4 of its tile, zero on the
//          padding -- 32 lanes x 16 bytes, as the tensor core's scale operand
//          lies in TMEM, so that a tile is one copy from shared memory.
#pragma once

#include <cuda_fp8.h>

#include "rowvec.cuh"

namespace ivfpq {

inline int64_t fp4_padded_cols(int64_t cols) { return ceil_div(cols, 32) * 32; }
inline int fp4_block(int fmt) { return fmt == IVFPQ_MXFP4 ? 32 : 16; }
// 4-block scale tiles along the columns
inline int64_t fp4_scale_tiles(int64_t cols, int fmt) {
  return ceil_div(fp4_padded_cols(cols), 4 * fp4_block(fmt));
}
__host__ __device__ __forceinline__ int64_t fp4_scale_at(int64_t row, int64_t blk, int64_t ntile) {
  return ((row >> 7) * ntile + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (blk & 3);
}

// ---- conversions ------------------------------------------------------------------
// 8 values to 8 codes, value 0 in the lowest bits: nearest, ties to the even
// code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// 8 codes to 4 pairs of binary16 values (exact).
__device__ __forceinline__ void e2m1_unpack8(uint32_t c, __half2 (&h)[4]) {
  uint32_t r0, r1, r2, r3;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(c));
  h[0] = *reinterpret_cast<__half2*>(&r0);
  h[1] = *reinterpret_cast<__half2*>(&r1);
  h[2] = *reinterpret_cast<__half2*>(&r2);
  h[3] = *reinterpret_cast<__half2*>(&r3);
}
__device__ __forceinline__ float e4m3_value(uint8_t s) {
  __nv_fp8_e4m3 e;
  e.__x = s;
  return float(e);
}
// 2^(byte - 127); byte 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint8_t s) {
  return s == 255 ? __int_as_float(0x7fc00000)
                  : (s == 0 ? __int_as_float(0x00400000) : __int_as_float(uint32_t(s) << 23));
}

// Scale byte of a block and the factor its values are multiplied by before
// they are rounded, from the block's largest magnitude as raw bits (an
// integer maximum, so that an infinity or a NaN is never lost): such a block
// gets a NaN scale and zero codes, that is, it reads back as NaN.
//  MXFP4: the scale is 2^(floor(log2(amax)) - 2), so amax / scale lies in
//         [4, 8); the exponent is read off the bits, the factor is exact.
//  NVFP4: the scale is amax / (6 g) rounded to E4M3 (saturating at 448); the
//         factor is 1 / (scale * g), one IEEE division per block. With a g for which
//         scale * g may be subnormal (inexact, and its reciprocal may pass fp32) the
//         values are multiplied by lift = 2^64 and the factor is that of g * lift;
//         else lift is 1.
__device__ __forceinline__ float nvfp4_lift(float g) {
  return g < 0x1p-117f ? 0x1p64f : 1.f;  // the smallest scale is 2^-9
}
struct BlockScale {
  uint8_t byte;
  float factor;
};
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, float g, float lift) {
  BlockScale r;
  if (amax_bits >= 0x7f800000u) {
    r.byte = FMT == IVFPQ_MXFP4 ? 0xff : 0x7f;
    r.factor = 0.f;
    return r;
  }
  if (FMT == IVFPQ_MXFP4) {
    const int eb = int(amax_bits >> 23);
    r.byte = uint8_t(max(eb - 2, 0));
    r.factor = __int_as_float(uint32_t(254 - int(r.byte)) << 23);
  } else {
    // 6 g passes fp32 for the largest g: an eighth of both sides then (exact; a
    // magnitude it makes subnormal is far below the smallest scale)
    const float eighth = g > 0x1p125f ? 0.125f : 1.f;
    r.byte = __nv_cvt_float_to_fp8(
        __fdiv_rn(__uint_as_float(amax_bits) * eighth, 6.f * eighth * g), __NV_SATFINITE,
        __NV_E4M3);
    const float sv = e4m3_value(r.byte) * (g * lift);
    r.factor = sv > 0.f ? __fdiv_rn(1.f, sv) : 0.f;
  }
  return r;
}

}  // namespace ivfpq
