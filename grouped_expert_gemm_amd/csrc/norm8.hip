// The residual's addition, the RMS norm and MXFP8 rows of its result in one pass:
//
//   s[t] = residual[t] + sum_j x[row(t, j)]   (float32, rounded once to the stored dtype)
//   r[t] = 1 / sqrt(mean_h s^2 + eps),  n = s r w
//   per 32 columns: e the smallest with max|n| <= 448 2^e, codes E4M3(n 2^-e)
//
// HBM-bound: k + 1 rows in, the sum, the codes and (on request) n in the stored dtype out. A
// team of TPR threads holds one row in registers, NV groups of 8 columns a thread, so four
// neighbouring lanes hold a block; its maximum takes two lane moves. 16384 x 2048, 8 rows a token,
// residual, sum and y: 773 MB in 156 to 160 us (4.9 TB/s; a copy reaches 5.2); 8192 x 4096, one row:
// 303 MB in 55 to 60 us (5.1 TB/s). One wavefront a row of 2048 takes as long.
// The sums of 8 squares are added up in float64 and r is kept as two float32 words, so that n is the
// exact product rounded about once. Where that rounding lands on a border (the middle between two codes,
// or between two bf16 values), the side that it came from is put into its last bit (round_to_odd), so
// that the codes, their scales and a bf16 y are those of the product itself: of 33.5 M values about 20
// would land on the wrong side. One value in 2^15 to 2^19 needs it, so the others only look.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lanes.h"
#include "mxfp8.h"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxSlots = 16;
constexpr int V = 8;  // columns a thread holds side by side

struct Params {
  const void* x;        // [T, H], or [T * k, H] reached through rows
  const int32_t* rows;  // [T * k] or NULL
  const void* residual; // NULL or [T, H]
  const void* w;        // [H]
  void* sum;            // NULL or [T, H]
  void* y;              // NULL or [T, H]
  float* rstd;          // NULL or [T]
  uint2* codes;         // [T, H] bytes
  uint8_t* scales;      // [T, H / 32]
  int64_t T;
  int H, k;
  float eps;
};

template <bool BF16>
struct Raw {  // 8 columns as they are stored
  uint4 v[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void* p, int64_t group) {
  Raw<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = ((const uint4*)p)[group * (BF16 ? 1 : 2) + i];
  return r;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t group, const Raw<BF16>& r) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) ((uint4*)p)[group * (BF16 ? 1 : 2) + i] = r.v[i];
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw<BF16>& r, float* f) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        f[4 * i + j] = __uint_as_float(w[j]);
      }
    }
  }
}

template <bool BF16>
__device__ __forceinline__ Raw<BF16> pack8(const float* f) {
  Raw<BF16> r;
  if constexpr (BF16) {
    r.v[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
  }
  return r;
}

// n = x + d, |d| at most half a step of n, as n with an odd last bit where d is not 0: it lies on
// x + d's side of every value that has fewer bits, so rounding it further rounds x + d itself.
// Infinities and NaN (d no less than n, or NaN) stay as they are.
__device__ __forceinline__ float round_to_odd(float n, float d) {
  const int32_t u = __float_as_int(n);
  const bool even = (u & 1) == 0 && (d < 0.f || d > 0.f) && __builtin_fabsf(d) < __builtin_fabsf(n);
  return __int_as_float(even ? u + (((u ^ __float_as_int(d)) >> 31) | 1) : u);
}

template <bool BF16, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_norm_kernel(const Params p) {
  constexpr int kTeams = TPR < 256 ? 256 / TPR : 1;
  __shared__ double red[2][TPR > 64 ? TPR / 64 : 1];  // alternating: a thread is at most one row ahead
  const int tr = threadIdx.x % TPR;
  const int groups = p.H / V;
  const double inv_h = 1.0 / p.H;
  Raw<BF16> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = Raw<BF16>{};
    if (i * TPR + tr < groups) w[i] = load8<BF16>(p.w, i * TPR + tr);
  }
  const int64_t R = p.T * p.k;
  // bits that are all 0 (in normal numbers) in the middle between two codes and where a block's scale
  // changes, and, for a bf16 y, in the middle between two bf16 values
  const uint32_t border = BF16 && p.y ? 0x7FFFu : 0x7FFFFu;
  int par = 0;
  // every thread of a workgroup runs the same rows' loop where the workgroup is one team
  for (int64_t t = (int64_t)blockIdx.x * kTeams + threadIdx.x / TPR; t < p.T; t += (int64_t)gridDim.x * kTeams) {
    float acc[NV][V];
    Raw<BF16> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      res[i] = Raw<BF16>{};
      if (p.residual && i * TPR + tr < groups) res[i] = load8<BF16>(p.residual, t * groups + i * TPR + tr);
    }
    constexpr int kSlots = BF16 || NV <= 2 ? 4 : 2;  // rows whose loads are in flight together
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      Raw<BF16> q[kSlots][NV];
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        int64_t row = -1;
        if (j0 + u < p.k) row = p.rows ? (int64_t)p.rows[t * p.k + j0 + u] : t;
        const bool ok = row >= 0 && row < R;  // a dropped slot adds nothing
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          q[u][i] = Raw<BF16>{};
          if (ok && i * TPR + tr < groups) q[u][i] = load8<BF16>(p.x, row * groups + i * TPR + tr);
        }
      }
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (j0 + u >= p.k) break;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[V];
          unpack8<BF16>(q[u][i], f);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[i][v] += f[v];
        }
      }
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      unpack8<BF16>(res[i], f);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] = f[v] + acc[i][v];
      const Raw<BF16> o = pack8<BF16>(acc[i]);
      if (p.sum && i * TPR + tr < groups) store8<BF16>(p.sum, t * groups + i * TPR + tr, o);
      unpack8<BF16>(o, acc[i]);  // the norm reads the sum as it is stored
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = acc[i][v] * acc[i][v];  // exact for bf16
      ss += (double)(((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7])));
    }
    ss = wave_sum(ss);
    if constexpr (TPR > 64) {
      if ((threadIdx.x & 63) == 0) red[par][threadIdx.x >> 6] = ss;
      __syncthreads();
      ss = 0.0;
#pragma unroll
      for (int i = 0; i < TPR / 64; ++i) ss += red[par][i];
      par ^= 1;
    }
    // r to float64 by one Newton step from its float32 value (0 and NaN stay as they are)
    const double m = ss * inv_h + (double)p.eps, r0 = (double)(1.f / sqrtf((float)m));
    const double r = r0 > 0.0 ? r0 * (1.5 - 0.5 * m * r0 * r0) : r0;
    // in two words, for bf16 rows the first of 16 bits: s times it is exact
    const float rf = (float)r, rh = BF16 ? __uint_as_float(__float_as_uint(rf) & 0xFFFFFF00u) : rf;
    const float rl = (float)(r - (double)rh);
    if (p.rstd && tr == 0) p.rstd[t] = rf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = t * groups + i * TPR + tr;
      const bool in = i * TPR + tr < groups;  // groups % 4 == 0: the four lanes of a block agree
      float f[V], n[V], top = 0.f;
      unpack8<BF16>(w[i], f);
      auto product = [&](int v, float& q, float& t) {  // s r w = q w + t
        const float a = acc[i][v];
        q = a * rh;
        t = (BF16 ? a * rl : __builtin_fmaf(a, rl, __builtin_fmaf(a, rh, -q))) * f[v];
      };
      uint32_t low = ~0u;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float q, t;
        product(v, q, t);
        n[v] = __builtin_fmaf(q, f[v], t);
        low = min(low, __float_as_uint(n[v]) & border);
        top = mx8::max_magnitude(top, n[v]);
      }
      if (!BF16 && p.y && in) store8<BF16>(p.y, at, pack8<BF16>(n));
      if (__builtin_expect(__any(low == 0), 0)) {
        top = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float q, t;
          product(v, q, t);
          n[v] = round_to_odd(n[v], __builtin_fmaf(q, f[v], -n[v]) + t);
          top = mx8::max_magnitude(top, n[v]);
        }
      }
      if (BF16 && p.y && in) store8<BF16>(p.y, at, pack8<BF16>(n));
      top = __uint_as_float(lanes_reduce<4>(__float_as_uint(top), [](uint32_t a, uint32_t b) {
        return __float_as_uint(mx8::max_magnitude(__uint_as_float(a), __uint_as_float(b)));
      }));
      const int b = mx8::scale_byte(top);
      const float sc = mx8::scale_value(b);
      if (in) {
        p.codes[at] = make_uint2(mx8::pack4(n[0], n[1], n[2], n[3], sc, b),
                                 mx8::pack4(n[4], n[5], n[6], n[7], sc, b));
        if ((threadIdx.x & 3) == 0) p.scales[at >> 2] = (uint8_t)b;
      }
    }
  }
}

template <int N>
using Int = std::integral_constant<int, N>;

template <bool BF16>
void launch(const Params& p, hipStream_t s) {
  auto go = [&](auto Tc, auto Nc) {
    constexpr int TPR = decltype(Tc)::value;
    constexpr int teams = TPR < 256 ? 256 / TPR : 1;
    int64_t grid = (p.T + teams - 1) / teams;
    const int64_t most = (int64_t)num_cus() * 8;
    if (grid > most) grid = most;
    hipLaunchKernelGGL((add_norm_kernel<BF16, TPR, decltype(Nc)::value>), dim3((unsigned)grid), dim3(TPR < 256 ? 256 : TPR),
                       0, s, p);
  };
  const int u = p.H / V;  // groups of a row
  if (u <= 64) go(Int<64>{}, Int<1>{});
  else if (u <= 128) go(Int<64>{}, Int<2>{});
  else if (u <= 256) go(Int<256>{}, Int<1>{});
  else if (u <= 512) go(Int<256>{}, Int<2>{});
  else if (u <= 1024) go(Int<256>{}, Int<4>{});
  else go(Int<1024>{}, Int<2>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_add_norm_mxfp8(const void* x, const int32_t* row_id_map, int k, const void* residual,
                                         const void* weight, moe_dtype dt, int64_t T, int H, float eps, void* sum,
                                         void* y, float* rstd, uint8_t* codes, uint8_t* scales, void* stream) {
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "moe_add_norm_mxfp8: dtype must be F32 or BF16");
  if (T < 0 || H < 1) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: T < 0 or H < 1");
  if (H > kMaxH || H % 32 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "moe_add_norm_mxfp8: needs H % 32 == 0 and H <= 16384");
  if (k < 1) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: k < 1");
  if (k > kMaxSlots) return fail(MOE_ERR_UNSUPPORTED, "moe_add_norm_mxfp8: k > 16");
  if (!row_id_map && k != 1) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: k > 1 needs row_id_map");
  if (T > 0x7FFFFFFF / k) return fail(MOE_ERR_UNSUPPORTED, "moe_add_norm_mxfp8: T * k exceeds int32 rows");
  if (!(eps > 0.f)) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: eps must be positive");
  if (T == 0) return MOE_OK;
  if (!x || !weight || !codes || !scales) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: NULL pointer");
  for (const void* p : {x, residual, weight, (const void*)sum, (const void*)y})
    if (!aligned(p, 16)) return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: tensors must be 16-byte aligned");
  if (!aligned(codes, 8) || !aligned(row_id_map, 4) || !aligned(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: codes must be 8-byte, row_id_map and rstd 4-byte aligned");
  if (sum && sum == x && row_id_map)
    return fail(MOE_ERR_INVALID_ARG, "moe_add_norm_mxfp8: sum may be x only without row_id_map");
  Params p{};
  p.x = x, p.rows = row_id_map, p.residual = residual, p.w = weight, p.sum = sum, p.y = y, p.rstd = rstd;
  p.codes = (uint2*)codes, p.scales = scales, p.T = T, p.H = H, p.k = k, p.eps = eps;
  if (dt == MOE_BF16) launch<true>(p, as_stream(stream));
  else launch<false>(p, as_stream(stream));
  return check_launch("moe_add_norm_mxfp8");
}
