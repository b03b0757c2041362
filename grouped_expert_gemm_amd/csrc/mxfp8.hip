// Reading MXFP8 rows back: value = code * 2^(scale byte - 127), rounded once to bf16 (exact but
// below bf16's smallest step and past its range), optionally gathered by row.
//
// HBM-bound: 33/32 bytes in, 2 bytes out an element. A thread takes 16 codes (half a block) a load
// and writes 32 bytes, four loads in flight together: 8192 x 28672 in 117 to 121 us, 5.9 TB/s (between
// other work; one call after another 137, 5.2 TB/s, what a copy reaches, and 156 with one load at a
// time), 131072 rows of 2048 gathered from 16384 in 125, their codes from the cache.
#include "mxfp8.h"

#include "common.h"
#include "internal.h"
#include "lanes.h"

namespace moe {
namespace mx8 {

constexpr int kItems = 4;  // loads of a thread in flight together

template <bool GATHER>
__global__ __launch_bounds__(256) void read_kernel(const uint4* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   int64_t src_rows, uint32_t row16, const int32_t* __restrict__ src_row,
                                                   int64_t rows, const int32_t* __restrict__ offsets, int E,
                                                   bool zero_missing, uint4* __restrict__ out) {
  const int64_t n = offsets ? routed_end(offsets, E, rows) : rows;
  const int64_t total = n * row16;
  const int64_t q0 = (int64_t)blockIdx.x * (256 * kItems) + threadIdx.x;
  int64_t at[kItems];
  uint4 w[kItems];
  uint8_t sb[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int64_t q = q0 + i * 256;
    at[i] = q;
    if constexpr (GATHER) {
      const int64_t r = total <= 0xFFFFFFFFll ? (int64_t)((uint32_t)q / row16) : q / row16;
      const int64_t from = q < total ? src_row[r] : -1;
      at[i] = from < 0 || from >= src_rows ? -1 : from * row16 + (q - r * row16);
    }
    if (q < total && at[i] >= 0) {
      w[i] = codes[at[i]];
      sb[i] = scales[at[i] >> 1];  // two items a block (row16 is even)
    }
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int64_t q = q0 + i * 256;
    if (q >= total) break;
    if (GATHER && at[i] < 0) {
      if (zero_missing) out[2 * q] = out[2 * q + 1] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const float sc = scale_value(sb[i]);
    const uint32_t word[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
      unpack4(word[j], sc, v);
      o[2 * j] = pack_bf16x2(v[0], v[1]);
      o[2 * j + 1] = pack_bf16x2(v[2], v[3]);
    }
    out[2 * q] = make_uint4(o[0], o[1], o[2], o[3]);
    out[2 * q + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

moe_status launch_read(const uint8_t* codes, const uint8_t* scales, int64_t src_rows, int64_t cols,
                       const int32_t* src_row, int64_t rows, const int32_t* offsets, int E, bool zero_missing, bf16_t* out,
                       hipStream_t s) {
  const int64_t row16 = cols / 16;
  if (rows == 0 || cols == 0) return MOE_OK;
  const int64_t grid = (rows * row16 + 256 * kItems - 1) / (256 * kItems);
  if (grid > 0xFFFFFFFF / 256) return fail(MOE_ERR_UNSUPPORTED, "mxfp8_dequantize: more elements than one launch holds");
  const auto kernel = src_row ? read_kernel<true> : read_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, (const uint4*)codes, scales, src_rows, (uint32_t)row16,
                     src_row, rows, offsets, E, zero_missing, (uint4*)out);
  return check_launch("mxfp8_dequantize");
}

}  // namespace mx8
}  // namespace moe

using namespace moe;

static moe_status read_rows(const char* fn, const uint8_t* e4m3, const uint8_t* e8m0, int64_t src_rows, int64_t cols,
                            const int32_t* src_row, int64_t rows, bool zero_missing, void* out_bf16, void* stream) {
  auto bad = [&](const char* what) { return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": " + what); };
  if (src_rows < 0 || rows < 0 || cols < 0) return bad("negative size");
  if (cols % 32 != 0) return bad("cols % 32 != 0");
  if (!src_row && rows != src_rows) return bad("without src_row, rows and src_rows must be equal");
  if (cols > 0x7FFFFFFF || rows > 0x7FFFFFFF || src_rows > 0x7FFFFFFF)
    return fail(MOE_ERR_UNSUPPORTED, std::string(fn) + ": a size of 2^31 or more");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!out_bf16 || (zero_missing && !src_row) || (src_rows > 0 && (!e4m3 || !e8m0))) return bad("NULL pointer");
  if (!aligned(e4m3, 16) || !aligned(out_bf16, 16) || !aligned(src_row, 4))
    return bad("codes and out must be 16-byte, src_row 4-byte aligned");
  return mx8::launch_read(e4m3, e8m0, src_rows, cols, src_row, rows, nullptr, 0, zero_missing, (bf16_t*)out_bf16,
                          as_stream(stream));
}

extern "C" moe_status mxfp8_dequantize(const uint8_t* e4m3, const uint8_t* e8m0, int64_t src_rows, int64_t cols,
                                       const int32_t* src_row, int64_t rows, void* out_bf16, void* stream) {
  return read_rows("mxfp8_dequantize", e4m3, e8m0, src_rows, cols, src_row, rows, false, out_bf16, stream);
}

extern "C" moe_status mxfp8_dequantize_gather(const uint8_t* e4m3, const uint8_t* e8m0, int64_t src_rows, int64_t cols,
                                              const int32_t* src_row, int64_t rows, void* out_bf16, void* stream) {
  return read_rows("mxfp8_dequantize_gather", e4m3, e8m0, src_rows, cols, src_row, rows, true, out_bf16, stream);
}
