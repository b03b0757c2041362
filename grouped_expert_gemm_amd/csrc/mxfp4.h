// MXFP4 (E2M1 codes, one E8M0 scale per 32 values): quantisation helpers shared by the
// quantiser and the GEMM epilogues, and the grouped MLP's host entry.
#pragma once

#include "common.h"

namespace moe {
namespace mx4 {

constexpr int kMaxE = 128;  // experts per call (two pointer tables in the kernel arguments)

enum { EP_STORE = 0, EP_SWIGLU = 1 };

// Operands of a grouped product. The row kernel reads the public row-major layouts; the tile
// kernel reads every scale in the MFMA's lane order (lane_scales) and the rows' codes in
// fragment order (frag_rows).
struct Params {
  const uint8_t* tab[kMaxE];    // per-expert weight codes [N][K / 2]
  const uint8_t* tab_s[kMaxE];  // per-expert weight scales
  const uint8_t* q;             // row codes [R][K / 2]
  const uint8_t* q_s;           // row scales
  void* c;                      // STORE: bf16 [R][N]; SWIGLU: h codes [R][I / 2] ...
  uint8_t* c_s;                 // ... and h's scales, both as the down product reads them
  const int32_t* offsets;
  const float* prob;
  int64_t R;
  int K, N, E, I, n_tiles;
};

constexpr uint32_t kNotFinite = 0x7F800000u;  // magnitude bits of infinity; above: NaN

// E8M0 byte of a block whose largest magnitude has the float32 bits u: s + 127 with s the
// smallest exponent that fits the maximum under 6 * 2^s, in [-127, 127]; 0 for an all-zero
// block; 255 (E8M0's NaN) for a block that holds an infinity or a NaN.
__device__ __forceinline__ int scale_byte(uint32_t u) {
  if (u >= kNotFinite) return 255;
  if (u == 0) return 0;
  int e = (int)(u >> 23);
  uint32_t m = u & 0x7FFFFFu;
  if (e == 0) {  // subnormal: normalise
    const int sh = __clz(m) - 8;
    m = (m << sh) & 0x7FFFFFu;
    e = 1 - sh;
  }
  // 6 = 1.5 * 2^2: the byte e - 2 if the significand is at most 1.5, else e - 1
  const int b = m <= 0x400000u ? e - 2 : e - 1;
  return b < 0 ? 0 : (b > 254 ? 254 : b);
}

// 2^(byte - 127), the scale operand of the conversions (byte 0: the subnormal 2^-127)
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte ? (uint32_t)byte << 23 : 0x00400000u);
}

// Eight E2M1 codes (value 0 in the low nibble) of f / 2^(byte - 127), |f| <= 6 * 2^(byte - 127):
// the conversion divides by its scale operand, a power of two, rounds to nearest, ties to the
// even code, and keeps the sign of zero.
__device__ __forceinline__ uint32_t pack8(const float* f, int byte) {
  const float s = scale_value(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
  return byte == 255 ? 0u : w;
}

// lanes: scales in lane order, word ((k / 256 * rows + r) * 2 + g) with byte s the scale of
// block 2s + g of the row's 256 values (cols % 256 == 0, scales 4-byte aligned)
moe_status quantize(const void* in_bf16, int64_t rows, int64_t cols, uint8_t* e2m1, uint8_t* e8m0, hipStream_t s,
                    bool lanes = false);
// public-layout scales [rows][cols / 32] of n tensors of one shape -> lane order
moe_status lane_scales(const uint8_t* const* src, uint8_t* const* dst, int n, int64_t rows, int64_t cols, hipStream_t s);

// Rows for the tile kernel. Fragment order: the 16 bytes of block 2s + g of row r's K values
// [64 s, 64 s + 64) stand at ((r / 32) * (cols / 64) + s) * 1024 + g * 512 + (r % 32) * 16, so
// the operand of an MFMA is 1 KiB in a row; the buffer has frag_bytes. Scales in lane order.
// From bf16 (quantised) or from public-layout codes and scales; cols % 256 == 0.
inline size_t frag_bytes(int64_t rows, int64_t cols) { return (size_t)((rows + 31) / 32 * 32) * cols / 2; }
moe_status quantize_frag(const void* in_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales, hipStream_t s);
moe_status frag_rows(const uint8_t* e2m1, const uint8_t* e8m0, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                     hipStream_t s);

moe_status launch_tile(int ep, const Params& p, hipStream_t s);

moe_status check_shape(int E, int K, int N, const char* what);
moe_status check_rows(int64_t R, int E, int K, moe_dtype act, const char* what);
size_t mlp_workspace_bytes(const moe_mlp_desc& d, int64_t R);
size_t linear_workspace_bytes(int E, int64_t R, int K, int N, moe_dtype act);
moe_status forward(const moe_mlp_desc& d, int64_t R, const void* x_perm, const uint8_t* x_perm_scale,
                   const void* const* w_gate_up, const void* const* w_down, const uint8_t* const* w_gate_up_scale,
                   const uint8_t* const* w_down_scale, const int32_t* offsets, const float* prob_perm, void* y_perm,
                   uint8_t* ws, hipStream_t s);

}  // namespace mx4
}  // namespace moe
