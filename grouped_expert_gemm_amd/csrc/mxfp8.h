// MXFP8 blocks (32 E4M3 codes and one E8M0 scale) made from float32 values and read back:
// helpers of the kernels that keep activations in 8 bits.
#pragma once

#include "common.h"

namespace moe {
namespace mx8 {

// The largest magnitude of two, NaN if either is NaN (v_maximum3_f32).
__device__ __forceinline__ float max_magnitude(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

// E8M0 byte of a block whose largest magnitude is top: s + 127 with s of mx_scale_exponent, 0
// for an all-zero block; 255 (E8M0's NaN) for a block that holds an infinity or a NaN.
// 448 = 1.75 * 2^8: the biased exponent less 8, one more where the significand is above 1.75,
// which the addition carries into the exponent.
__device__ __forceinline__ int scale_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  const int b = (int)((u + 0x1FFFFFu) >> 23) - 8;
  return u >= 0x7F800000u ? 255 : b < 0 ? 0 : b;
}

// 2^(byte - 127), NaN for 255 (byte 0 is the subnormal 2^-127): the scale operand of the
// conversions below
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte ? (uint32_t)byte << 23 : 0x00400000u);
}

// Four E4M3 codes (the first in the low byte) of values divided by scale = scale_value(byte), at
// most 448 in magnitude: gfx950's scaled conversion, which rounds the quotient by a power of two
// to nearest, ties to even, as e4m3_pack4 rounds it (checked for every byte over 2^20 float32
// patterns each). byte 255: 0.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float scale, int byte) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  i16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return byte == 255 ? 0u : __builtin_bit_cast(uint32_t, w);
}

// the four values of a word of codes, times scale = scale_value(byte): exact in float32, NaN for 255
__device__ __forceinline__ void unpack4(uint32_t w, float scale, float* v) {
  const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
  const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

// Reads of MXFP8 rows [src_rows, cols] as bf16 rows: out[r] = values of row src_row[r] (of row r
// where src_row is NULL), for r < rows and, with offsets [E + 1], the rows of E experts alone
// (routed_end). A row whose src_row is out of [0, src_rows) is left as it was, or zeros with
// zero_missing. cols % 32 == 0, codes and out 16-byte aligned.
moe_status launch_read(const uint8_t* codes, const uint8_t* scales, int64_t src_rows, int64_t cols,
                       const int32_t* src_row, int64_t rows, const int32_t* offsets, int E, bool zero_missing, bf16_t* out,
                       hipStream_t s);

}  // namespace mx8
}  // namespace moe
