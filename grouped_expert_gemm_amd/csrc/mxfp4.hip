// MXFP4: quantisation, and the grouped GEMMs of experts whose weights are served in it.
//
// Elements are OCP E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two a byte, the
// even one in the low nibble; 32 consecutive values share one E8M0 scale 2^s, s the
// smallest with max|block| <= 6 * 2^s (the rule mxfp8_quantize uses with 448).
//
// GEMM operands: gfx950's scaled MFMA takes 16 bytes a lane, 32 consecutive values of one
// row and their block's scale. In v_mfma_scale_f32_16x16x128 lane l holds row l % 16 and
// block l / 16 of the 128 values.
//
// grouped_gemm_rows_kernel: y = x W^T for few rows an expert, bound by the weights' bytes.
// The weights go straight from memory to the MFMA, without LDS: a workgroup takes 32 or 64
// output columns (32 gate and 32 up rows with SwiGLU) of one expert, its four wavefronts every
// fourth 256-value unit of K, and their partial products are added through LDS in wavefront
// order. The next unit's weights are in flight while one is multiplied.
// (Many rows: mxfp4_tile.hip.)
#include <cstring>

#include "common.h"
#include "gemm_common.h"
#include "internal.h"
#include "lanes.h"
#include "mxfp4.h"

namespace moe {
namespace mx4 {

using gemm::silu_f;

constexpr int kUnit = 256;  // K values of one unit

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t wide(i32x4_t v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// ---------------------------------------------------------------------------
// quantisation: HBM-bound, 2 bytes in, 17/32 out a value. Four lanes own a block (16 bytes
// of bf16 each), whose largest magnitude two lane moves find.
// ---------------------------------------------------------------------------

// byte of block b of row r in lane order (mxfp4.h)
__device__ __forceinline__ int64_t lane_at(int64_t r, int64_t b, int64_t rows) {
  return (((b >> 3) * rows + r) * 2 + (b & 1)) * 4 + ((b >> 1) & 3);
}

// lane_rows: 0 for row-major scales, else the row count, for lane order
__global__ __launch_bounds__(256) void quantize_kernel(const uint4* __restrict__ in, int64_t nblocks,
                                                       uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       int64_t cols32, int64_t lane_rows) {
  const int64_t total = nblocks * 4, stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t padded = (total + 63) / 64 * 64;  // whole wavefronts: every lane reaches the lane moves
  for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < padded; q += stride) {
    const bool live = q < total;
    const uint4 v = live ? in[q] : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      top = max(top, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    }
    top = lanes_umax<4>(top);
    const int b = scale_byte(top);
    if (live) {
      codes[q] = pack8(f, b);
      if ((q & 3) == 0) {
        const int64_t n = q >> 2, r = lane_rows ? n / cols32 : 0;
        scales[lane_rows ? lane_at(r, n - r * cols32, lane_rows) : n] = (uint8_t)b;
      }
    }
  }
}

moe_status quantize(const void* in_bf16, int64_t rows, int64_t cols, uint8_t* e2m1, uint8_t* e8m0, hipStream_t s,
                    bool lanes) {
  const int64_t nblocks = rows * (cols / 32);
  if (nblocks == 0) return MOE_OK;
  int64_t grid = (nblocks * 4 + 255) / 256;
  const int64_t most = (int64_t)num_cus() * 16;
  if (grid > most) grid = most;
  hipLaunchKernelGGL(quantize_kernel, dim3((unsigned)grid), dim3(256), 0, s, (const uint4*)in_bf16, nblocks,
                     (uint32_t*)e2m1, e8m0, cols / 32, lanes ? rows : 0);
  return check_launch("mxfp4_quantize");
}

// Row-major scales to lane order: 64 rows x 8 steps a workgroup through LDS, 64 bytes of a
// row read together, 512 bytes of a step written together.
__device__ __forceinline__ uint2 lane_order(uint2 v) {  // the 8 scales of a row's 256 values
  return make_uint2(__builtin_amdgcn_perm(v.y, v.x, 0x06040200u), __builtin_amdgcn_perm(v.y, v.x, 0x07050301u));
}

struct ScaleTables {
  const uint2* src[kMaxE];
  uint2* dst[kMaxE];
};

__global__ __launch_bounds__(256) void lane_scales_kernel(const ScaleTables tabs, int64_t rows, int steps) {
  __shared__ uint2 tile[8][65];
  const uint2* src = tabs.src[blockIdx.z];
  uint2* dst = tabs.dst[blockIdx.z];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int s0 = blockIdx.y * 8, tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (i * 256 + tid) >> 3, st = tid & 7;
    if (r0 + r < rows && s0 + st < steps) {
      tile[st][r] = lane_order(src[(r0 + r) * steps + s0 + st]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int st = (i * 256 + tid) >> 6, r = tid & 63;
    if (r0 + r < rows && s0 + st < steps) dst[(int64_t)(s0 + st) * rows + r0 + r] = tile[st][r];
  }
}

moe_status lane_scales(const uint8_t* const* src, uint8_t* const* dst, int n, int64_t rows, int64_t cols, hipStream_t s) {
  ScaleTables t;
  for (int i = 0; i < n; ++i) {
    t.src[i] = reinterpret_cast<const uint2*>(src[i]);
    t.dst[i] = reinterpret_cast<uint2*>(dst[i]);
  }
  const int steps = (int)(cols / 256);
  const dim3 grid((unsigned)((rows + 63) / 64), (unsigned)((steps + 7) / 8), (unsigned)n);
  hipLaunchKernelGGL(lane_scales_kernel, grid, dim3(256), 0, s, t, rows, steps);
  return check_launch("MXFP4 scale conversion");
}

// Rows into fragment order (mxfp4.h): a wavefront takes 8 rows x 256 values, 8 lanes a row, and
// writes whole 128-byte lines (8 rows of one 16-byte block).
__global__ __launch_bounds__(256) void quantize_frag_kernel(const uint16_t* __restrict__ in, int64_t rows, int64_t cols,
                                                            uint8_t* __restrict__ codes, uint2* __restrict__ scales) {
  const int lane = threadIdx.x & 63, l8 = lane & 7;
  const int64_t steps = cols / 256;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t step = item % steps, r = item / steps * 8 + (lane >> 3);
  const bool live = r < rows;
  uint4 v[4];
  const uint16_t* src = in + r * cols + step * 256 + l8 * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = live ? *reinterpret_cast<const uint4*>(src + i * 64) : make_uint4(0, 0, 0, 0);
  uint8_t* dst = codes + ((r >> 5) * (cols / 64) + step * 4) * 1024 + (l8 >> 2) * 512 + (r & 31) * 16 + (l8 & 3) * 4;
  uint32_t word = 0;  // the scales of block l8 / 4 of the four slices
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float f[8];
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f[2 * h] = __uint_as_float(w[h] << 16);
      f[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
      top = max(top, max((w[h] << 16) & 0x7FFFFFFFu, w[h] & 0x7FFF0000u));
    }
    const int b = scale_byte(lanes_umax<4>(top));
    word |= (uint32_t)b << (8 * i);
    if (live) *reinterpret_cast<uint32_t*>(dst + i * 1024) = pack8(f, b);
  }
  if (live && (l8 & 3) == 0) reinterpret_cast<uint32_t*>(scales + step * rows + r)[l8 >> 2] = word;
}

__global__ __launch_bounds__(256) void frag_rows_kernel(const uint8_t* __restrict__ in, const uint2* __restrict__ in_s,
                                                        int64_t rows, int64_t cols, uint8_t* __restrict__ codes,
                                                        uint2* __restrict__ scales) {
  const int lane = threadIdx.x & 63, l8 = lane & 7;
  const int64_t steps = cols / 256;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t step = item % steps, r = item / steps * 8 + (lane >> 3);
  if (r >= rows) return;
  const uint4 v = *reinterpret_cast<const uint4*>(in + r * (cols / 2) + step * 128 + l8 * 16);
  *reinterpret_cast<uint4*>(codes + ((r >> 5) * (cols / 64) + step * 4 + (l8 >> 1)) * 1024 + (l8 & 1) * 512 + (r & 31) * 16) = v;
  if (l8 == 0) scales[step * rows + r] = lane_order(in_s[r * steps + step]);
}

// workgroups of the two kernels above; check_rows keeps them within a launch
static int64_t row_groups(int64_t rows, int64_t cols) { return ((rows + 7) / 8 * (cols / 256) + 3) / 4; }

moe_status quantize_frag(const void* in_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  hipLaunchKernelGGL(quantize_frag_kernel, dim3((unsigned)row_groups(rows, cols)), dim3(256), 0, s, (const uint16_t*)in_bf16,
                     rows, cols, codes, (uint2*)scales);
  return check_launch("MXFP4 row quantisation");
}

moe_status frag_rows(const uint8_t* e2m1, const uint8_t* e8m0, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                     hipStream_t s) {
  hipLaunchKernelGGL(frag_rows_kernel, dim3((unsigned)row_groups(rows, cols)), dim3(256), 0, s, e2m1, (const uint2*)e8m0, rows,
                     cols, codes, (uint2*)scales);
  return check_launch("MXFP4 row conversion");
}

__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t words,
                                                         uint4* __restrict__ out) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < words; q += stride) {
    const uint32_t w = codes[q];
    const int b = scales[q >> 2], s = b - 127;
    auto pair = [&](auto i) -> uint32_t {
      const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, decltype(i)::value);
      const float nan = __uint_as_float(0x7FC00000u);
      return b == 255 ? pack_bf16x2(nan, nan) : pack_bf16x2(ldexpf(v[0], s), ldexpf(v[1], s));
    };
    out[q] = make_uint4(pair(std::integral_constant<int, 0>{}), pair(std::integral_constant<int, 1>{}),
                        pair(std::integral_constant<int, 2>{}), pair(std::integral_constant<int, 3>{}));
  }
}

// ---------------------------------------------------------------------------
// grouped GEMM, few rows an expert
// ---------------------------------------------------------------------------

// the rank-th expert that has rows, or -1: its rows are [beg, end). Offsets are kept inside
// [0, R]; a wavefront looks at 64 experts at a time.
__device__ __forceinline__ int find_expert(const int32_t* offsets, int E, int R, int rank, int& beg, int& end) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int b = 0, n = 0;
    if (e < E) {
      b = min(max(offsets[e], 0), R);
      n = min(max(offsets[e + 1], b), R);
    }
    const uint64_t some = __ballot(n > b);
    const int cnt = __popcll(some);
    if (rank < cnt) {
      const uint64_t below = some & ((1ull << lane) - 1);
      const uint64_t hit = __ballot(n > b && __popcll(below) == rank);
      const int src = __ffsll((unsigned long long)hit) - 1;
      beg = __builtin_amdgcn_readfirstlane(__shfl(b, src));
      end = __builtin_amdgcn_readfirstlane(__shfl(n, src));
      return __builtin_amdgcn_readfirstlane(e0 + src);
    }
    rank -= cnt;
  }
  return -1;
}

// 32 bf16 values of one block -> its codes and scale byte
__device__ __forceinline__ i32x4_t quantize_block(const i32x4_t* x, int& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint32_t w = (uint32_t)x[i][h];
      top = max(top, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
    }
  byte = scale_byte(top);
  i32x4_t c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f[2 * h] = __uint_as_float((uint32_t)x[i][h] << 16);
      f[2 * h + 1] = __uint_as_float((uint32_t)x[i][h] & 0xFFFF0000u);
    }
    c[i] = (int)pack8(f, byte);
  }
  return c;
}

// How a workgroup takes its expert's rows: 16 at a time, each wavefront with one unit of weights
// and rows in flight and, by its registers, seven workgroups a CU (four with SwiGLU); the same
// with bf16 rows, whose blocks each lane quantises as it multiplies them (for calls of so few
// rows that doing it in every workgroup costs less than a launch of its own; four workgroups a
// CU, three with SwiGLU); or 64 at a time, so that the weights of an expert with
// more rows are read once, with two units of weights in flight, two workgroups a CU and 64
// columns a workgroup, as the rows are read once for every workgroup of columns.
// Eight experts of 4096 x 14336, 249 MB, 48 us at the rate of a copy: with 4, 8, 12, 24 and 64
// rows each 16 at a time take 51, 55, 60, 101 and 199 us, 64 at a time 54, 55, 57, 64 and 84 us
// (with 32 columns 109 us at 64 rows; with 128 the registers spill: 365). Those passes repeat
// over one set of weights, which the last-level cache holds in part; with six sets in turn 12, 24
// and 64 rows, 64 at a time and quantised in the call, take 61, 70 and 91 us in place of 47, 54
// and 83.
enum { ROWS_16 = 0, ROWS_16_BF16 = 1, ROWS_64 = 2 };

template <int EP, int MODE>
__global__ __launch_bounds__(256, MODE == ROWS_64 ? 2 : 3) void grouped_gemm_rows_kernel(const Params prm) {
  constexpr bool kBF16 = MODE == ROWS_16_BF16;
  constexpr int NA = EP == EP_SWIGLU || MODE == ROWS_64 ? 4 : 2;  // 16-row weight tiles
  constexpr int NC = EP == EP_SWIGLU ? 32 : NA * 16;              // output columns
  constexpr int NR = MODE == ROWS_64 ? 4 : 1;   // 16-row tiles of x at a time
  constexpr int D = MODE == ROWS_64 ? 2 : 1;    // units of weights in flight
  constexpr int LD = NA * 16 + 4;
  constexpr int XL = kBF16 ? 8 : 2;             // 16-byte loads of a row tile, a unit
  __shared__ __attribute__((aligned(16))) float part[4][16][LD];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int beg, end;
  const int e = find_expert(prm.offsets, prm.E, (int)prm.R, blockIdx.y, beg, end);
  if (e < 0) return;
  const int K = prm.K, units = K / kUnit;
  const int64_t ldc = K / 2, lds = K / 32;
  // a wavefront-uniform base and 32-bit lane offsets (a weight is under 2^30 bytes)
  const uint8_t* wbase = prm.tab[e];
  const uint8_t* sbase = prm.tab_s[e];
  uint32_t wc[NA], ws[NA];
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    const int n = EP == EP_SWIGLU ? (a >= 2 ? prm.I : 0) + blockIdx.x * 32 + (a & 1) * 16 + l16
                                  : blockIdx.x * NC + a * 16 + l16;
    wc[a] = (uint32_t)(n * ldc + g * 16);
    ws[a] = (uint32_t)(n * lds);
  }
  typedef float f4 __attribute__((ext_vector_type(4)));
  for (int r0 = beg; r0 < end; r0 += NR * 16) {
    const int nrt = min(NR, (end - r0 + 15) / 16);
    const uint8_t* xbase = prm.q + (int64_t)r0 * (kBF16 ? (int64_t)K * 2 : ldc);
    const uint8_t* xsbase = kBF16 ? nullptr : prm.q_s + (int64_t)r0 * lds;
    uint32_t xc[NR], xs[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = min(r * 16 + l16, end - 1 - r0);  // past the expert: any valid row, discarded
      xc[r] = kBF16 ? (uint32_t)((row * K + g * 32) * 2) : (uint32_t)(row * ldc + g * 16);
      xs[r] = (uint32_t)(row * lds);
    }
    f4 acc[NA][NR];
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[a][r] = f4{0.f, 0.f, 0.f, 0.f};
    i32x4_t w[D][NA][2];
    uint2 sw[D][NA];
    auto load = [&](int u, auto I) {
      constexpr int i = decltype(I)::value;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        w[i][a][0] = *reinterpret_cast<const i32x4_t*>(wbase + u * 128 + wc[a]);
        w[i][a][1] = *reinterpret_cast<const i32x4_t*>(wbase + u * 128 + 64 + wc[a]);
        sw[i][a] = *reinterpret_cast<const uint2*>(sbase + u * 8 + ws[a]);
      }
    };
    auto step = [&](int u, auto I) {
      constexpr int i = decltype(I)::value;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (r >= nrt) break;
        i32x4_t x[XL];
#pragma unroll
        for (int j = 0; j < XL; ++j)
          x[j] = kBF16 ? *reinterpret_cast<const i32x4_t*>(xbase + u * 512 + (j >> 2) * 256 + (j & 3) * 16 + xc[r])
                       : *reinterpret_cast<const i32x4_t*>(xbase + u * 128 + j * 64 + xc[r]);
        i32x4_t x0 = x[0], x1 = x[1];
        int sx0, sx1;
        if constexpr (kBF16) {
          x0 = quantize_block(x, sx0);
          x1 = quantize_block(x + 4, sx1);
        } else {
          const uint2 sx = *reinterpret_cast<const uint2*>(xsbase + u * 8 + xs[r]);
          sx0 = (int)(sx.x >> (8 * g));
          sx1 = (int)(sx.y >> (8 * g));
        }
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          acc[a][r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i][a][0]), wide(x0), acc[a][r], 4, 4, 0,
                                                                        (int)(sw[i][a].x >> (8 * g)), 0, sx0);
          acc[a][r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i][a][1]), wide(x1), acc[a][r], 4, 4, 0,
                                                                        (int)(sw[i][a].y >> (8 * g)), 0, sx1);
        }
      }
    };
    using U0 = std::integral_constant<int, 0>;
    using U1 = std::integral_constant<int, D - 1>;
    if constexpr (D == 1) {
      for (int u = wave; u < units; u += 4) {
        load(u, U0{});
        step(u, U0{});
      }
    } else {
      if (wave < units) load(wave, U0{});
      for (int u = wave; u < units; u += 8) {
        if (u + 4 < units) load(u + 4, U1{});
        step(u, U0{});
        if (u + 8 < units) load(u + 8, U0{});
        if (u + 4 < units) step(u + 4, U1{});
      }
    }
    // each 16-row tile: the four wavefronts' partial products, added in order
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r >= nrt) break;
#pragma unroll
      for (int a = 0; a < NA; ++a) *reinterpret_cast<f4*>(&part[wave][l16][a * 16 + 4 * g]) = acc[a][r];
      __syncthreads();
      const int row = tid >> 4, cp = (tid & 15) * 2;
      const int64_t mg = r0 + r * 16 + row;
      auto sum = [&](int col) {
        return (part[0][row][col] + part[1][row][col]) + (part[2][row][col] + part[3][row][col]);
      };
      if constexpr (EP == EP_STORE) {
        if (mg < end)
#pragma unroll
          for (int c = cp; c < NC; c += 32)
            *reinterpret_cast<uint32_t*>((bf16_t*)prm.c + mg * prm.N + blockIdx.x * NC + c) = pack_bf16x2(sum(c), sum(c + 1));
      } else {
        const float v0 = sum(cp), v1 = sum(cp + 1);
        const float p = prm.prob[mg < end ? mg : end - 1];
        const float h0 = silu_f(v0) * sum(32 + cp) * p, h1 = silu_f(v1) * sum(32 + cp + 1) * p;
        uint32_t top = max(__float_as_uint(h0) & 0x7FFFFFFFu, __float_as_uint(h1) & 0x7FFFFFFFu);
        top = lanes_umax<16>(top);
        const int b = scale_byte(top);
        if (mg < end) {
          const uint32_t code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h0, h1, scale_value(b), 0);
          ((uint8_t*)prm.c)[mg * (prm.I / 2) + blockIdx.x * 16 + (tid & 15)] = b == 255 ? 0 : (uint8_t)code;
          if ((tid & 15) == 0) prm.c_s[mg * (prm.I / 32) + blockIdx.x] = (uint8_t)b;
        }
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static size_t a256(size_t x) { return align_up(x, 256); }

moe_status check_shape(int E, int K, int N, const char* what) {
  if (E > kMaxE) return fail(MOE_ERR_UNSUPPORTED, std::string(what) + ": MXFP4 supports at most 128 experts");
  if (K % 256 != 0 || N % 256 != 0)
    return fail(MOE_ERR_UNSUPPORTED, std::string(what) + ": MXFP4 kernels need every GEMM size to be a multiple of 256");
  return MOE_OK;
}

// How a call reads its rows: few rows an expert are bound by the weights' bytes and go to the
// row kernel, otherwise to 256-row tiles (8 experts of 4096 x 14336: 64 rows each 83 us, 65 rows
// 108). At most 16 rows in all, given in bf16, are quantised by the row kernel itself. The offsets
// are on the device, so the rule sees the average alone: an expert with many more rows than that
// is walked 16 or 64 rows at a time by its columns' workgroups, its weights read again each time
// (128 experts of 2048 x 2048 and 8192 rows: 105 us with 64 rows each, 428 with half of all rows
// on one, 800 with all of them).
enum class Path { kRowsBF16, kRows, kTiles };
static Path choose(int64_t R, int E, moe_dtype act) {
  if (act == MOE_BF16 && R <= 16) return Path::kRowsBF16;
  return R <= (int64_t)64 * E ? Path::kRows : Path::kTiles;
}

moe_status check_rows(int64_t R, int E, int K, moe_dtype act, const char* what) {
  constexpr int64_t kMaxGroups = (1 << 24) - 1;  // a launch holds fewer than 2^32 threads: workgroups of 256
  if (choose(R, E, act) == Path::kTiles && (R > 0x7FFFFFFF || row_groups(R, K) > kMaxGroups))
    return fail(MOE_ERR_UNSUPPORTED, std::string(what) + ": too many MXFP4 row values for one launch");
  return MOE_OK;
}

static void fill(Params& p, int E, int64_t R, int K, int N, const uint8_t* x, const uint8_t* xs, const uint8_t* const* w,
                 const uint8_t* const* ws, const int32_t* offsets, void* c) {
  std::memset(&p, 0, sizeof(p));
  for (int e = 0; e < E; ++e) {
    p.tab[e] = w[e];
    p.tab_s[e] = ws[e];
  }
  p.q = x, p.q_s = xs, p.c = c, p.offsets = offsets, p.R = R, p.K = K, p.N = N, p.E = E, p.n_tiles = N / 256;
}

template <int EP>
static moe_status launch(const Params& p, Path path, hipStream_t s) {
  if (path == Path::kTiles) return launch_tile(EP, p, s);
  const int64_t experts = p.R < p.E ? p.R : p.E;
  const dim3 grid((unsigned)((EP == EP_SWIGLU ? p.I : p.N) / 32), (unsigned)experts);
  const dim3 wide_grid(EP == EP_SWIGLU ? grid.x : grid.x / 2, grid.y);
  if (path == Path::kRowsBF16) hipLaunchKernelGGL((grouped_gemm_rows_kernel<EP, ROWS_16_BF16>), grid, dim3(256), 0, s, p);
  else if (p.R <= 16 || p.R <= (int64_t)8 * p.E)  // 8 rows an expert on average: of near-even loads hardly any has more than 16
    hipLaunchKernelGGL((grouped_gemm_rows_kernel<EP, ROWS_16>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((grouped_gemm_rows_kernel<EP, ROWS_64>), wide_grid, dim3(256), 0, s, p);
  return check_launch(EP == EP_SWIGLU ? "MXFP4 gate_up + ScaledSwiGLU" : "MXFP4 grouped linear");
}

// The operands of one call: codes and scales as the chosen kernel reads them, from codes as
// they are (scales converted for the tile kernel) or quantised from bf16. `take` hands out
// workspace; the same walk with ws = nullptr counts it.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  uint8_t* take(size_t n) {
    uint8_t* p = base ? base + used : nullptr;
    used += a256(n);
    return p;
  }
};

static moe_status rows_in(Carver& ws, moe_dtype act, const void* x, const uint8_t* x_scale, int64_t R, int K, Path path,
                          const uint8_t*& q, const uint8_t*& qs, hipStream_t s) {
  q = (const uint8_t*)x, qs = x_scale;
  if (path == Path::kRowsBF16 || (path == Path::kRows && act != MOE_BF16)) return MOE_OK;
  uint8_t* c = ws.take(path == Path::kTiles ? frag_bytes(R, K) : (size_t)R * K / 2);
  uint8_t* b = ws.take((size_t)R * K / 32);
  q = c, qs = b;
  if (!ws.base) return MOE_OK;
  if (path == Path::kRows) return quantize(x, R, K, c, b, s);
  return act == MOE_BF16 ? quantize_frag(x, R, K, c, b, s) : frag_rows((const uint8_t*)x, x_scale, R, K, c, b, s);
}

static moe_status weights_in(Carver& ws, moe_dtype wt, const void* const* w, const uint8_t* const* scale, int E, int N,
                             int K, Path path, const uint8_t** c, const uint8_t** cs, hipStream_t s) {
  const size_t n = (size_t)N * K;
  uint8_t* dst[kMaxE];
  for (int e = 0; e < E; ++e) {
    if (wt == MOE_BF16) {
      uint8_t* a = ws.take(n / 2);
      uint8_t* b = ws.take(n / 32);
      c[e] = a, cs[e] = b;
      if (ws.base) {
        const moe_status st = quantize(w[e], N, K, a, b, s, path == Path::kTiles);
        if (st != MOE_OK) return st;
      }
    } else if (path != Path::kTiles) {
      c[e] = w ? (const uint8_t*)w[e] : nullptr, cs[e] = scale ? scale[e] : nullptr;
    } else {
      c[e] = w ? (const uint8_t*)w[e] : nullptr, cs[e] = dst[e] = ws.take(n / 32);
    }
  }
  return ws.base && wt != MOE_BF16 && path == Path::kTiles ? lane_scales(scale, dst, E, N, K, s) : MOE_OK;
}

// the whole MLP, or with ws.base NULL only its workspace
static moe_status mlp(Carver& ws, const moe_mlp_desc& d, int64_t R, const void* x_perm, const uint8_t* x_perm_scale,
                      const void* const* w_gate_up, const void* const* w_down, const uint8_t* const* w_gate_up_scale,
                      const uint8_t* const* w_down_scale, const int32_t* offsets, const float* prob_perm, void* y_perm,
                      hipStream_t s) {
  const int E = d.E, H = d.H, I = d.I;
  const Path path = choose(R, E, d.act);
  uint8_t* hq = ws.take(path == Path::kTiles ? frag_bytes(R, I) : (size_t)R * I / 2);
  uint8_t* hs = ws.take((size_t)R * I / 32);
  const uint8_t *xq, *xs;
  const uint8_t *w1[kMaxE], *s1[kMaxE], *w2[kMaxE], *s2[kMaxE];
  moe_status st;
  if ((st = rows_in(ws, d.act, x_perm, x_perm_scale, R, H, path, xq, xs, s)) != MOE_OK) return st;
  if ((st = weights_in(ws, d.wt, w_gate_up, w_gate_up_scale, E, 2 * I, H, path, w1, s1, s)) != MOE_OK) return st;
  if ((st = weights_in(ws, d.wt, w_down, w_down_scale, E, H, I, path, w2, s2, s)) != MOE_OK) return st;
  if (!ws.base) return MOE_OK;
  Params p;
  fill(p, E, R, H, 2 * I, xq, xs, w1, s1, offsets, hq);
  p.I = I, p.prob = prob_perm, p.c_s = hs, p.n_tiles = I / 128;
  if ((st = launch<EP_SWIGLU>(p, path, s)) != MOE_OK) return st;
  fill(p, E, R, I, H, hq, hs, w2, s2, offsets, y_perm);
  return launch<EP_STORE>(p, path == Path::kTiles ? path : Path::kRows, s);  // h is MXFP4 already
}

size_t mlp_workspace_bytes(const moe_mlp_desc& d, int64_t R) {
  Carver ws{nullptr};
  mlp(ws, d, R, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return ws.used;
}

moe_status forward(const moe_mlp_desc& d, int64_t R, const void* x_perm, const uint8_t* x_perm_scale,
                   const void* const* w_gate_up, const void* const* w_down, const uint8_t* const* w_gate_up_scale,
                   const uint8_t* const* w_down_scale, const int32_t* offsets, const float* prob_perm, void* y_perm,
                   uint8_t* workspace, hipStream_t s) {
  const moe_status st = check_rows(R, d.E, d.H, d.act, "moe_grouped_mlp_fwd");
  if (st != MOE_OK) return st;
  Carver ws{workspace};
  return mlp(ws, d, R, x_perm, x_perm_scale, w_gate_up, w_down, w_gate_up_scale, w_down_scale, offsets, prob_perm,
             y_perm, s);
}

static moe_status grouped_linear(Carver& ws, int E, int64_t R, int K, int N, moe_dtype act, const void* x,
                                 const uint8_t* x_scale, const uint8_t* const* w, const uint8_t* const* w_scale,
                                 const int32_t* offsets, void* y, hipStream_t s) {
  const Path path = choose(R, E, act);
  const uint8_t *xq, *xs;
  const uint8_t *wq[kMaxE], *wqs[kMaxE];
  moe_status st = rows_in(ws, act, x, x_scale, R, K, path, xq, xs, s);
  if (st != MOE_OK) return st;
  st = weights_in(ws, MOE_MXFP4, (const void* const*)w, w_scale, E, N, K, path, wq, wqs, s);
  if (st != MOE_OK || !ws.base) return st;
  Params p;
  fill(p, E, R, K, N, xq, xs, wq, wqs, offsets, y);
  return launch<EP_STORE>(p, path, s);
}

size_t linear_workspace_bytes(int E, int64_t R, int K, int N, moe_dtype act) {
  Carver ws{nullptr};
  grouped_linear(ws, E, R, K, N, act, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return ws.used;
}

}  // namespace mx4
}  // namespace moe

using namespace moe;

extern "C" moe_status mxfp4_quantize(const void* in_bf16, int64_t rows, int64_t cols, uint8_t* e2m1, uint8_t* e8m0,
                                     void* stream) {
  if (rows < 0 || cols < 0) return fail(MOE_ERR_INVALID_ARG, "mxfp4_quantize: negative size");
  if (cols % 32 != 0) return fail(MOE_ERR_INVALID_ARG, "mxfp4_quantize: cols % 32 != 0");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!in_bf16 || !e2m1 || !e8m0) return fail(MOE_ERR_INVALID_ARG, "mxfp4_quantize: NULL pointer");
  if (!aligned(in_bf16, 16) || !aligned(e2m1, 4))
    return fail(MOE_ERR_INVALID_ARG, "mxfp4_quantize: input must be 16-byte and codes 4-byte aligned");
  return mx4::quantize(in_bf16, rows, cols, e2m1, e8m0, as_stream(stream));
}

extern "C" moe_status mxfp4_dequantize(const uint8_t* e2m1, const uint8_t* e8m0, int64_t rows, int64_t cols,
                                       void* out_bf16, void* stream) {
  if (rows < 0 || cols < 0) return fail(MOE_ERR_INVALID_ARG, "mxfp4_dequantize: negative size");
  if (cols % 32 != 0) return fail(MOE_ERR_INVALID_ARG, "mxfp4_dequantize: cols % 32 != 0");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!e2m1 || !e8m0 || !out_bf16) return fail(MOE_ERR_INVALID_ARG, "mxfp4_dequantize: NULL pointer");
  if (!aligned(out_bf16, 16) || !aligned(e2m1, 4))
    return fail(MOE_ERR_INVALID_ARG, "mxfp4_dequantize: output must be 16-byte and codes 4-byte aligned");
  const int64_t words = rows * (cols / 8);
  int64_t grid = (words + 255) / 256;
  const int64_t most = (int64_t)num_cus() * 16;
  if (grid > most) grid = most;
  hipLaunchKernelGGL(mx4::dequantize_kernel, dim3((unsigned)grid), dim3(256), 0, as_stream(stream),
                     (const uint32_t*)e2m1, e8m0, words, (uint4*)out_bf16);
  return check_launch("mxfp4_dequantize");
}

extern "C" moe_status moe_grouped_linear_mxfp4(int E, int64_t R, int K, int N, moe_dtype act, const void* x,
                                               const uint8_t* x_scale, const uint8_t* const* w,
                                               const uint8_t* const* w_scale, const int32_t* offsets, void* y,
                                               void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_linear_mxfp4";
  const std::string f(fn);
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, f + ": E out of [1, 256]");
  if (R < 0 || R > 0x7FFFFFFF || K < 1 || N < 1) return fail(MOE_ERR_INVALID_ARG, f + ": bad R/K/N");
  if (act != MOE_BF16 && act != MOE_MXFP4) return fail(MOE_ERR_INVALID_ARG, f + ": act must be BF16 or MXFP4");
  moe_status st = mx4::check_shape(E, K, N, fn);
  if (st != MOE_OK) return st;
  if ((int64_t)N * K > 0x7FFFFFFFLL) return fail(MOE_ERR_UNSUPPORTED, f + ": weight exceeds 2^31 elements");
  if (R == 0) return MOE_OK;
  if (!x || !y || !offsets || !w || !w_scale) return fail(MOE_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(offsets, 4)) return fail(MOE_ERR_INVALID_ARG, f + ": misaligned tensor");
  if (act == MOE_MXFP4 && (!x_scale || !aligned(x_scale, 8)))
    return fail(MOE_ERR_INVALID_ARG, f + ": MXFP4 rows need an 8-byte aligned x_scale");
  for (int e = 0; e < E; ++e) {
    if (!w[e] || !w_scale[e]) return fail(MOE_ERR_INVALID_ARG, f + ": NULL pointer for expert " + std::to_string(e));
    if (!aligned(w[e], 16) || !aligned(w_scale[e], 8))
      return fail(MOE_ERR_INVALID_ARG, f + ": weights must be 16-byte and their scales 8-byte aligned");
  }
  if ((st = mx4::check_rows(R, E, K, act, fn)) != MOE_OK) return st;
  const size_t need = mx4::linear_workspace_bytes(E, R, K, N, act);
  if (workspace_bytes < need) return fail(MOE_ERR_WORKSPACE, f + ": workspace too small");
  if (need > 0 && (!workspace || !aligned(workspace, 256)))
    return fail(MOE_ERR_INVALID_ARG, f + ": workspace NULL or not 256-byte aligned");
  // a call that needs no workspace still walks the same way: any non-NULL base serves
  mx4::Carver ws{need > 0 ? (uint8_t*)workspace : (uint8_t*)y};
  return mx4::grouped_linear(ws, E, R, K, N, act, x, x_scale, w, w_scale, offsets, y, as_stream(stream));
}
