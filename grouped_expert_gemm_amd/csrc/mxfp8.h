// MXFP8 blocks (32 E4M3 codes and one E8M0 scale) made from float32 values and read back:
// helpers of the kernels that keep activations in 8 bits.
#pragma once

#include "common.h"

namespace moe {
namespace mx8 {

// E8M0 byte of a block whose largest magnitude has the float32 bits u: s + 127 with s of
// mx_scale_exponent, 0 for an all-zero block; 255 (E8M0's NaN) for a block that holds an
// infinity or a NaN (as integers, their magnitude bits are the largest).
__device__ __forceinline__ int scale_byte(uint32_t u) {
  return u >= 0x7F800000u ? 255 : mx_scale_exponent(__uint_as_float(u)) + 127;
}

// 2^(byte - 127), NaN for 255 (byte 0 is the subnormal 2^-127)
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte ? (uint32_t)byte << 23 : 0x00400000u);
}

// 2^(127 - byte), what a block's values are multiplied with before they are rounded: exact but
// for results far below E4M3's smallest step (byte 254: the subnormal 2^-127)
__device__ __forceinline__ float inverse_scale(int byte) {
  return __uint_as_float(byte >= 254 ? 0x00400000u : (uint32_t)(254 - byte) << 23);
}

// the four values of a word of codes, times a power of two
__device__ __forceinline__ void unpack4(uint32_t w, float scale, float* v) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0] * scale;
  v[1] = lo[1] * scale;
  v[2] = hi[0] * scale;
  v[3] = hi[1] * scale;
}

// Reads of MXFP8 rows [src_rows, cols] as bf16 rows: out[r] = values of row src_row[r] (of row r
// where src_row is NULL), for r < rows and, with limit, r < *limit (a device word, clamped to
// [0, rows]). A row whose src_row is out of [0, src_rows) is left as it was, or zeros with
// zero_missing. cols % 32 == 0, codes and out 16-byte aligned.
moe_status launch_read(const uint8_t* codes, const uint8_t* scales, int64_t src_rows, int64_t cols,
                       const int32_t* src_row, int64_t rows, const int32_t* limit, bool zero_missing, bf16_t* out,
                       hipStream_t s);

}  // namespace mx8
}  // namespace moe
