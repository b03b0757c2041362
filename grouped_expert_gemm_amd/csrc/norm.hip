// The RMS norms around the expert block: the norm before it, and the norm after it
// fused with the combine of each token's k rows, the block's gate, the scaled residual and,
// on request, the next block's norm. Their backward passes.
//
//   pre :  y = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//   post:  c = sum_j y_perm[row(t, j)],  out = s x + gate (c r w),  r from c
//   bwd :  with n = c r (the stored c), a = dout n:
//          dw = sum_t gate a,  d_gate = w a (summed over what shares the gate value),
//          dc = r (dout gate w - n mean(dout gate w n)), written to each of the token's rows
// The pre norm's backward is the same with gate 1, one row a token and dx = s dx_in + dc.
//
// HBM-bound: every tensor passes through once. A team of TPR threads holds one row in
// registers (NV vectors of 16 bytes a thread), so the sum of squares, the result and the
// next norm come from one read. A forward workgroup walks several rows with the weights
// held in registers; a backward team walks a run of consecutive tokens and keeps the column
// sums of a in registers, so that dw and d_gate cost one partial row per run.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxSlots = 16;
constexpr int64_t kTargetChunks = 512;

enum { GATE_NONE = 0, GATE_TOKEN = 1, GATE_CHANNEL = 2 };

// ---- vectors of V elements: 16 bytes, or one element where rows are not aligned ----
template <bool BF16, int V>
struct Raw;
template <>
struct Raw<true, 8> { typedef uint4 type; };
template <>
struct Raw<true, 1> { typedef uint16_t type; };
template <>
struct Raw<false, 4> { typedef float4 type; };
template <>
struct Raw<false, 1> { typedef float type; };

template <bool BF16, int V>
__device__ __forceinline__ void unpack(const typename Raw<BF16, V>::type& r, float* v) {
  if constexpr (BF16 && V == 8) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else if constexpr (BF16) {
    v[0] = bf16_to_f32(r);
  } else if constexpr (V == 4) {
    v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
  } else {
    v[0] = r;
  }
}

template <bool BF16, int V>
__device__ __forceinline__ typename Raw<BF16, V>::type pack(const float* v) {
  if constexpr (BF16 && V == 8)
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else if constexpr (BF16) return (uint16_t)f32_to_bf16(v[0]);
  else if constexpr (V == 4) return make_float4(v[0], v[1], v[2], v[3]);
  else return v[0];
}

// the team's sum of v, in every thread; buf: TPR / 64 floats, one of two alternating buffers
// (a thread may be one reduction ahead of another, never two)
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* buf) {
  v = lanes_sum<64>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += buf[i];
  }
  return v;
}

struct FwdParams {
  const void* y;        // rows to normalise: [T, H], or [T * k, H] reached through rows
  const int32_t* rows;  // [T * k] or NULL
  const void* x;        // residual [T, H] (post)
  const void* w;
  const void* gate;     // NULL, [T] or [ceil(T / group), H]
  const void* w_next;   // NULL: no next norm
  void* out;            // [T, H]
  void* c;              // NULL or [T, H]
  void* y_next;
  float* rstd;          // NULL or [T]
  float* rstd_next;
  int64_t T, group;
  int H, k, gate_kind;
  float eps, scale;
};

// kPost: combine, gate, residual, next norm; else the plain norm of y's rows
template <bool BF16, int V, int TPR, int NV, bool kPost>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(const FwdParams p) {
  typedef typename Raw<BF16, V>::type raw_t;
  typedef typename std::conditional<BF16, uint16_t, float>::type elem_t;
  constexpr int kTeams = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
  const int tr = threadIdx.x % TPR;
  const int H = p.H;
  const float inv_h = 1.f / (float)H;  // applied to each term: a sum of squares would overflow H times earlier
  raw_t w[NV], w2[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + tr) * V;
    in[i] = col < H;
    w[i] = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.w + col) : raw_t{};
    w2[i] = kPost && p.w_next && in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.w_next + col) : raw_t{};
  }
  // every thread of a workgroup runs the same rows' loop (team_sum has barriers only where
  // the workgroup is one team)
  for (int64_t t = (int64_t)blockIdx.x * kTeams + threadIdx.x / TPR; t < p.T; t += (int64_t)gridDim.x * kTeams) {
    float acc[NV][V];
    raw_t xr[NV];
    if constexpr (kPost) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        xr[i] = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.x + t * H + (i * TPR + tr) * V) : raw_t{};
    }
    if (kPost && p.rows) {
      const int64_t R = p.T * p.k;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
      constexpr int kSlots = NV * V <= 32 ? 4 : 2;  // rows whose loads are in flight together
      for (int j0 = 0; j0 < p.k; j0 += kSlots) {
        raw_t q[kSlots][NV];
        bool ok[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          const int32_t r = j0 + u < p.k ? p.rows[t * p.k + j0 + u] : -1;
          ok[u] = r >= 0 && r < R;  // a dropped slot adds nothing
          const elem_t* src = (const elem_t*)p.y + (int64_t)(ok[u] ? r : 0) * H;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            q[u][i] = in[i] && ok[u] ? *reinterpret_cast<const raw_t*>(src + (i * TPR + tr) * V) : raw_t{};
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (ok[u]) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              float f[V];
              unpack<BF16, V>(q[u][i], f);
#pragma unroll
              for (int v = 0; v < V; ++v) acc[i][v] += f[v];
            }
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const raw_t q = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.y + t * H + (i * TPR + tr) * V) : raw_t{};
        unpack<BF16, V>(q, acc[i]);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) ss += acc[i][v] * inv_h * acc[i][v];
    const float r = 1.f / sqrtf(team_sum<TPR>(ss, red[0]) + p.eps);
    if (p.rstd && tr == 0) p.rstd[t] = r;
    float gt = 1.f;
    if (kPost && p.gate_kind == GATE_TOKEN) gt = BF16 ? bf16_to_f32(((const uint16_t*)p.gate)[t]) : ((const float*)p.gate)[t];
    const elem_t* grow = (const elem_t*)p.gate + (kPost && p.gate_kind == GATE_CHANNEL ? t / p.group * H : 0);
    float ss2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = t * H + (i * TPR + tr) * V;
      if constexpr (kPost)
        if (p.c && in[i]) *reinterpret_cast<raw_t*>((elem_t*)p.c + at) = pack<BF16, V>(acc[i]);
      float f[V];
      unpack<BF16, V>(w[i], f);
      if constexpr (kPost) {
        float x[V], g[V];
        unpack<BF16, V>(xr[i], x);
        if (p.gate_kind == GATE_CHANNEL && in[i]) {
          unpack<BF16, V>(*reinterpret_cast<const raw_t*>(grow + (i * TPR + tr) * V), g);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) g[v] = gt;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) acc[i][v] = p.scale * x[v] + g[v] * (acc[i][v] * r * f[v]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[i][v] = acc[i][v] * r * f[v];
      }
      const raw_t o = pack<BF16, V>(acc[i]);
      if (in[i]) *reinterpret_cast<raw_t*>((elem_t*)p.out + at) = o;
      if constexpr (kPost) {  // the next norm reads the sum as it was stored
        unpack<BF16, V>(o, acc[i]);
        if (in[i])
#pragma unroll
          for (int v = 0; v < V; ++v) ss2 += acc[i][v] * inv_h * acc[i][v];
      }
    }
    if constexpr (kPost) {
      if (p.w_next) {
        const float r2 = 1.f / sqrtf(team_sum<TPR>(ss2, red[1]) + p.eps);
        if (p.rstd_next && tr == 0) p.rstd_next[t] = r2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[V];
          unpack<BF16, V>(w2[i], f);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[i][v] = acc[i][v] * r2 * f[v];
          if (in[i]) *reinterpret_cast<raw_t*>((elem_t*)p.y_next + t * H + (i * TPR + tr) * V) = pack<BF16, V>(acc[i]);
        }
      } else if (TPR > 64) {
        __syncthreads();  // red[0] is written again by the next row
      }
    } else if (TPR > 64) {
      __syncthreads();
    }
  }
}

// Runs of tokens of the backward: run c covers [c * chunk, + chunk), or, where a gate row is
// shared by more tokens than that (pieces > 1), piece c % pieces of group c / pieces.
struct ChunkPlan {
  int64_t chunks, chunk, pieces;
};

ChunkPlan plan_chunks(int64_t T, int gate_kind, int64_t group) {
  ChunkPlan p{0, 1, 1};
  if (T == 0) return p;
  int64_t c = (T + kTargetChunks - 1) / kTargetChunks;
  if (c < 4) c = T < 4 ? T : 4;
  if (gate_kind == GATE_CHANNEL && group < T) {
    if (group > c) {
      p.pieces = (group + c - 1) / c;
      p.chunk = (group + p.pieces - 1) / p.pieces;
      p.chunks = (T + group - 1) / group * p.pieces;
      return p;
    }
    c = c / group * group;
  } else if (gate_kind == GATE_CHANNEL) {  // one gate row for every token
    p.pieces = (T + c - 1) / c;
    p.chunk = c;
    p.chunks = p.pieces;
    return p;
  }
  p.chunk = c;
  p.chunks = (T + c - 1) / c;
  return p;
}

struct BwdParams {
  const void* dout;
  const void* c;        // what was normalised: the stored sum, or x
  const float* rstd;
  const void* w;
  const void* gate;
  const int32_t* rows;  // NULL, or where each token's gradient goes (k rows)
  const void* dx_in;    // NULL, or added to the result with dx_scale (one row a token)
  void* dy;             // [T, H] or [T * k, H]
  float* dgate;         // [T], [ceil(T / group), H] or NULL
  float* part;          // [chunks][H] partial column sums
  int64_t T, group;
  ChunkPlan plan;
  int H, k;
  float dx_scale;
};

// A partial row holds the sum of gate a (no gate, gate per token, or whole groups in the
// run, whose d_gate rows are then written here), or of a alone where the run is a piece of
// one group (the join then makes both dw and d_gate from it).
template <bool BF16, int V, int TPR, int NV, int GATE>
__global__ __launch_bounds__(TPR) void norm_bwd_kernel(const BwdParams p) {
  typedef typename Raw<BF16, V>::type raw_t;
  typedef typename std::conditional<BF16, uint16_t, float>::type elem_t;
  __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
  const int tr = threadIdx.x;
  const int H = p.H;
  const float inv_h = 1.f / (float)H;
  const int64_t ch = blockIdx.x;
  int64_t t0, t1;
  if (p.plan.pieces > 1) {
    const int64_t g = ch / p.plan.pieces, q = ch % p.plan.pieces;
    t0 = g * p.group + q * p.plan.chunk;
    t1 = t0 + p.plan.chunk;
    const int64_t end = (g + 1) * p.group;
    t1 = t1 < end ? t1 : end;
  } else {
    t0 = ch * p.plan.chunk;
    t1 = t0 + p.plan.chunk;
  }
  t1 = t1 < p.T ? t1 : p.T;
  raw_t w[NV], graw[NV];
  bool in[NV];
  float sum[NV][V], own[NV][V];  // own: sum of a over the current group (channel gates)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + tr) * V;
    in[i] = col < H;
    w[i] = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.w + col) : raw_t{};
    graw[i] = raw_t{};
#pragma unroll
    for (int v = 0; v < V; ++v) sum[i][v] = own[i][v] = 0.f;
  }
  const int64_t R = p.T * p.k;
  int par = 0;
  for (int64_t t = t0; t < t1; ++t) {
    raw_t dr[NV], cr[NV], xr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = t * H + (i * TPR + tr) * V;
      dr[i] = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.dout + at) : raw_t{};
      cr[i] = in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.c + at) : raw_t{};
      xr[i] = GATE == GATE_NONE && p.dx_in && in[i] ? *reinterpret_cast<const raw_t*>((const elem_t*)p.dx_in + at) : raw_t{};
    }
    const float r = p.rstd[t];
    float gt = 1.f;
    if (GATE == GATE_TOKEN) gt = BF16 ? bf16_to_f32(((const uint16_t*)p.gate)[t]) : ((const float*)p.gate)[t];
    if (GATE == GATE_CHANNEL && (t == t0 || t % p.group == 0)) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i])
          graw[i] = *reinterpret_cast<const raw_t*>((const elem_t*)p.gate + t / p.group * H + (i * TPR + tr) * V);
    }
    float n[NV][V], d[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V];
      unpack<BF16, V>(cr[i], n[i]);
      unpack<BF16, V>(dr[i], d[i]);
      unpack<BF16, V>(w[i], f);
      if (GATE == GATE_CHANNEL) unpack<BF16, V>(graw[i], g);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        n[i][v] *= r;
        const float a = d[i][v] * n[i][v];
        if (GATE == GATE_CHANNEL) own[i][v] += a;
        else sum[i][v] += gt * a;
        d[i][v] *= GATE == GATE_CHANNEL ? g[v] * f[v] : f[v];
        s += d[i][v] * n[i][v];
      }
    }
    s = team_sum<TPR>(s, red[par]);
    par ^= 1;
    if (GATE == GATE_TOKEN && p.dgate && tr == 0) p.dgate[t] = s;
    const float m = gt * r, q = s * inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float x[V];
      unpack<BF16, V>(xr[i], x);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        d[i][v] = m * (d[i][v] - n[i][v] * q);
        if (GATE == GATE_NONE && p.dx_in) d[i][v] += p.dx_scale * x[v];
      }
    }
    if (p.rows) {
      for (int j = 0; j < p.k; ++j) {
        const int32_t row = p.rows[t * p.k + j];
        if (row < 0 || row >= R) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (in[i])
            *reinterpret_cast<raw_t*>((elem_t*)p.dy + (int64_t)row * H + (i * TPR + tr) * V) = pack<BF16, V>(d[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) *reinterpret_cast<raw_t*>((elem_t*)p.dy + t * H + (i * TPR + tr) * V) = pack<BF16, V>(d[i]);
    }
    if (GATE == GATE_CHANNEL && p.plan.pieces == 1 && (t + 1 == t1 || (t + 1) % p.group == 0)) {  // the group ends here
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[V], g[V];
        unpack<BF16, V>(w[i], f);
        unpack<BF16, V>(graw[i], g);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (in[i] && p.dgate) p.dgate[t / p.group * H + (i * TPR + tr) * V + v] = f[v] * own[i][v];
          sum[i][v] += g[v] * own[i][v];
          own[i][v] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (in[i])
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.part[ch * H + (i * TPR + tr) * V + v] = GATE == GATE_CHANNEL && p.plan.pieces > 1 ? own[i][v] : sum[i][v];
}

// dw (and, for pieces, d_gate): 16 columns a workgroup and 64 threads a column (4 a
// wavefront), `par` <= 16 groups of them on different gate groups at a time and 64 / par on
// the pieces of each; sums in a fixed order. The partial rows come from other XCDs' caches,
// so what counts is that all of a column's loads are in flight at once (512 rows x 4096
// columns: 10.3 us with 16 threads a column).
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* __restrict__ part, int64_t groups, int64_t pieces,
                                                         int par, int H, const void* __restrict__ w,
                                                         const void* __restrict__ gate, float* __restrict__ dw,
                                                         float* __restrict__ dgate) {
  __shared__ float sums[16][17];
  const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 16 + cl;
  const int each = 64 / par, gq = q / each, sub = q % each;
  const int waves = each / 4;                            // wavefronts on one group
  const bool lead = wave % waves == 0 && (q & 3) == 0;   // the thread that finishes its group's column
  float total = 0.f;
  for (int64_t g0 = 0; g0 < groups; g0 += par) {
    const int64_t g = g0 + gq;
    float s = 0.f;
    if (col < H && g < groups) {
      const float* src = part + g * pieces * H + col;
#pragma unroll 8
      for (int64_t i = sub; i < pieces; i += each) s += src[i * H];
    }
    // the wavefront's 4 threads of a column, then the group's wavefronts in order
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    s = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    s = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    if (waves > 1) {
      if ((q & 3) == 0) sums[wave][cl] = s;
      __syncthreads();
      if (lead)
        for (int i = 1; i < waves; ++i) s += sums[wave + i][cl];
      __syncthreads();
    }
    if (lead && col < H && g < groups) {
      if (gate) {
        const float gv = BF16 ? bf16_to_f32(((const uint16_t*)gate)[g * H + col]) : ((const float*)gate)[g * H + col];
        const float wv = BF16 ? bf16_to_f32(((const uint16_t*)w)[col]) : ((const float*)w)[col];
        if (dgate) dgate[g * H + col] = wv * s;
        total += gv * s;
      } else {
        total = s;
      }
    }
  }
  if (lead) sums[wave][cl] = total;
  __syncthreads();
  if (q == 0 && col < H) {
    for (int i = 1; i < par; ++i) total += sums[i * waves][cl];
    dw[col] = total;
  }
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(BF16, V, TPR, NV): the narrowest team and fewest vectors a thread that hold the row.
// many: rows enough to fill the card with one wavefront each; a row of up to 64 x 4 vectors then
// goes to one wavefront, which reduces without barriers and keeps four times the rows of a
// 256-thread team in flight (16384 x 2048, 8 rows combined: 185 -> 153 us; a single row takes
// longer that way).
template <typename F>
void dispatch(bool bf16, bool vec, int H, bool many, F&& f) {
  const std::true_type B{};
  const std::false_type S{};
  if (many && vec && bf16 && H > 1024 && H <= 2048) return f(B, Int<8>{}, Int<64>{}, Int<4>{});
  if (many && vec && !bf16 && H > 512 && H <= 1024) return f(S, Int<4>{}, Int<64>{}, Int<4>{});
  if (bf16 && vec) {
    if (H <= 512) f(B, Int<8>{}, Int<64>{}, Int<1>{});
    else if (H <= 1024) f(B, Int<8>{}, Int<64>{}, Int<2>{});
    else if (H <= 2048) f(B, Int<8>{}, Int<256>{}, Int<1>{});
    else if (H <= 4096) f(B, Int<8>{}, Int<256>{}, Int<2>{});
    else if (H <= 8192) f(B, Int<8>{}, Int<256>{}, Int<4>{});
    else f(B, Int<8>{}, Int<1024>{}, Int<2>{});
  } else if (vec) {
    if (H <= 512) f(S, Int<4>{}, Int<64>{}, Int<2>{});
    else if (H <= 1024) f(S, Int<4>{}, Int<256>{}, Int<1>{});
    else if (H <= 2048) f(S, Int<4>{}, Int<256>{}, Int<2>{});
    else if (H <= 4096) f(S, Int<4>{}, Int<256>{}, Int<4>{});
    else if (H <= 8192) f(S, Int<4>{}, Int<1024>{}, Int<2>{});
    else f(S, Int<4>{}, Int<1024>{}, Int<4>{});
  } else {
    auto scalar = [&](auto b) {
      if (H <= 512) f(b, Int<1>{}, Int<64>{}, Int<8>{});
      else if (H <= 1024) f(b, Int<1>{}, Int<256>{}, Int<4>{});
      else if (H <= 4096) f(b, Int<1>{}, Int<256>{}, Int<16>{});
      else f(b, Int<1>{}, Int<1024>{}, Int<16>{});
    };
    if (bf16) scalar(B);
    else scalar(S);
  }
}

bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

moe_status check_common(const std::string& fn, moe_dtype dt, int64_t T, int H, int k, const void* rows) {
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, fn + ": dtype must be F32 or BF16");
  if (T < 0 || H < 1) return fail(MOE_ERR_INVALID_ARG, fn + ": T < 0 or H < 1");
  if (H > kMaxH) return fail(MOE_ERR_UNSUPPORTED, fn + ": H > 16384");
  if (k < 1) return fail(MOE_ERR_INVALID_ARG, fn + ": k < 1");
  if (k > kMaxSlots) return fail(MOE_ERR_UNSUPPORTED, fn + ": k > 16");
  if (!rows && k != 1) return fail(MOE_ERR_INVALID_ARG, fn + ": k > 1 needs row_id_map");
  if (T > 0x7FFFFFFF / k) return fail(MOE_ERR_UNSUPPORTED, fn + ": T * k exceeds int32 rows");
  return MOE_OK;
}

moe_status check_gate(const std::string& fn, int gate_kind, const void* gate, int64_t gate_group) {
  if (gate_kind != GATE_NONE && gate_kind != GATE_TOKEN && gate_kind != GATE_CHANNEL)
    return fail(MOE_ERR_INVALID_ARG, fn + ": bad gate kind");
  if (gate_kind == GATE_CHANNEL && gate_group < 1) return fail(MOE_ERR_INVALID_ARG, fn + ": gate_group < 1");
  if (gate_kind != GATE_NONE && !gate) return fail(MOE_ERR_INVALID_ARG, fn + ": gate is NULL");
  return MOE_OK;
}

template <bool kPost>
void launch_fwd(const FwdParams& p, bool bf16, bool vec, hipStream_t s) {
  dispatch(bf16, vec, p.H, p.T >= 4 * num_cus(), [&](auto B, auto Vc, auto Tc, auto Nc) {
    constexpr int TPR = decltype(Tc)::value;
    constexpr int teams = TPR < 256 ? 256 / TPR : 1;
    int64_t grid = (p.T + teams - 1) / teams;
    const int64_t most = (int64_t)num_cus() * 8;
    if (grid > most) grid = most;
    hipLaunchKernelGGL((norm_fwd_kernel<decltype(B)::value, decltype(Vc)::value, TPR, decltype(Nc)::value, kPost>),
                       dim3((unsigned)grid), dim3(TPR < 256 ? 256 : TPR), 0, s, p);
  });
}

void launch_bwd(const BwdParams& p, int gate_kind, bool bf16, bool vec, float* dw, hipStream_t s) {
  dispatch(bf16, vec, p.H, false, [&](auto B, auto Vc, auto Tc, auto Nc) {
    constexpr int TPR = decltype(Tc)::value;
    const dim3 grid((unsigned)p.plan.chunks), block(TPR);
    constexpr bool b = decltype(B)::value;
    constexpr int V = decltype(Vc)::value, NV = decltype(Nc)::value;
    if (gate_kind == GATE_TOKEN) hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_TOKEN>), grid, block, 0, s, p);
    else if (gate_kind == GATE_CHANNEL) hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_CHANNEL>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_NONE>), grid, block, 0, s, p);
  });
  const bool pieces = p.plan.pieces > 1;
  const dim3 grid((unsigned)((p.H + 15) / 16));
  const int64_t groups = pieces ? p.plan.chunks / p.plan.pieces : 1, each = pieces ? p.plan.pieces : p.plan.chunks;
  int par = 1;
  while (par < 16 && par < groups) par *= 2;
  auto kernel = bf16 ? norm_join_kernel<true> : norm_join_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(1024), 0, s, p.part, groups, each, par, p.H, p.w, pieces ? p.gate : nullptr, dw,
                     pieces ? p.dgate : nullptr);
}

__global__ void fill_zero_kernel(float* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

moe_status zero_dw(float* dw, int H, hipStream_t s, const char* what) {
  hipLaunchKernelGGL(fill_zero_kernel, dim3((H + 255) / 256), dim3(256), 0, s, dw, (int64_t)H);
  return check_launch(what);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t T, int H, int gate_kind, int64_t gate_group) {
  return align_up((size_t)plan_chunks(T, gate_kind, gate_group).chunks * H * 4, 256);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_pre_norm(const void* x, const void* weight, moe_dtype dt, int64_t T, int H, float eps,
                                   void* y, float* rstd, void* stream) {
  moe_status st = check_common("moe_pre_norm", dt, T, H, 1, nullptr);
  if (st != MOE_OK) return st;
  if (!(eps > 0.f)) return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm: eps must be positive");
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y) return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm: NULL pointer");
  const size_t esz = dt == MOE_BF16 ? 2 : 4;
  if (!all_aligned({x, weight, y}, esz) || !aligned(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm: misaligned pointer");
  FwdParams p{};
  p.y = x, p.w = weight, p.out = y, p.rstd = rstd, p.T = T, p.H = H, p.k = 1, p.eps = eps;
  launch_fwd<false>(p, dt == MOE_BF16, H * esz % 16 == 0 && all_aligned({x, weight, y}, 16), as_stream(stream));
  return check_launch("moe_pre_norm");
}

extern "C" moe_status moe_pre_norm_bwd(const void* dy, const void* x, const void* weight, const float* rstd,
                                       const void* dx_in, float dx_in_scale, moe_dtype dt, int64_t T, int H, void* dx,
                                       float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_common("moe_pre_norm_bwd", dt, T, H, 1, nullptr);
  if (st != MOE_OK) return st;
  if (!dweight || !aligned(dweight, 4)) return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm_bwd: dweight NULL or misaligned");
  const hipStream_t s = as_stream(stream);
  if (T == 0) return zero_dw(dweight, H, s, "moe_pre_norm_bwd");
  if (!dy || !x || !weight || !rstd || !dx) return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm_bwd: NULL pointer");
  const size_t esz = dt == MOE_BF16 ? 2 : 4;
  if (!all_aligned({dy, x, weight, dx_in, dx}, esz) || !aligned(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm_bwd: misaligned pointer");
  if (workspace_bytes < norm_bwd_workspace_bytes(T, H, GATE_NONE, 0))
    return fail(MOE_ERR_WORKSPACE, "moe_pre_norm_bwd: workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return fail(MOE_ERR_INVALID_ARG, "moe_pre_norm_bwd: workspace NULL or not 256-byte aligned");
  BwdParams p{};
  p.dout = dy, p.c = x, p.rstd = rstd, p.w = weight, p.dx_in = dx_in, p.dx_scale = dx_in_scale, p.dy = dx;
  p.part = (float*)workspace, p.T = T, p.H = H, p.k = 1, p.plan = plan_chunks(T, GATE_NONE, 0);
  launch_bwd(p, GATE_NONE, dt == MOE_BF16, H * esz % 16 == 0 && all_aligned({dy, x, weight, dx_in, dx}, 16), dweight, s);
  return check_launch("moe_pre_norm_bwd");
}

extern "C" moe_status moe_post_norm(const void* y, const int32_t* row_id_map, int k, const void* x, const void* weight,
                                    moe_gate gate_kind, const void* gate, int64_t gate_group, float residual_scale,
                                    const void* next_weight, moe_dtype dt, int64_t T, int H, float eps, void* out,
                                    void* c, float* rstd, void* y_next, float* rstd_next, void* stream) {
  moe_status st = check_common("moe_post_norm", dt, T, H, k, row_id_map);
  if (st != MOE_OK) return st;
  if (!(eps > 0.f)) return fail(MOE_ERR_INVALID_ARG, "moe_post_norm: eps must be positive");
  if (T == 0) return MOE_OK;
  if ((st = check_gate("moe_post_norm", gate_kind, gate, gate_group)) != MOE_OK) return st;
  if (!y || !x || !weight || !out) return fail(MOE_ERR_INVALID_ARG, "moe_post_norm: NULL pointer");
  if (!next_weight != !y_next) return fail(MOE_ERR_INVALID_ARG, "moe_post_norm: next_weight and y_next go together");
  const size_t esz = dt == MOE_BF16 ? 2 : 4;
  const bool channel = gate_kind == GATE_CHANNEL;
  if (!all_aligned({y, x, weight, gate, next_weight, out, c, y_next}, esz) || !all_aligned({row_id_map, rstd, rstd_next}, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_post_norm: misaligned pointer");
  FwdParams p{};
  p.y = y, p.rows = row_id_map, p.x = x, p.w = weight, p.gate = gate, p.w_next = next_weight, p.out = out, p.c = c;
  p.y_next = y_next, p.rstd = rstd, p.rstd_next = next_weight ? rstd_next : nullptr, p.T = T, p.group = gate_group;
  p.H = H, p.k = k, p.gate_kind = gate_kind, p.eps = eps, p.scale = residual_scale;
  const bool vec = H * esz % 16 == 0 && all_aligned({y, x, weight, channel ? gate : nullptr, next_weight, out, c, y_next}, 16);
  launch_fwd<true>(p, dt == MOE_BF16, vec, as_stream(stream));
  return check_launch("moe_post_norm");
}

extern "C" moe_status moe_post_norm_bwd(const void* dout, const void* c, const float* rstd, const void* weight,
                                        moe_gate gate_kind, const void* gate, int64_t gate_group,
                                        const int32_t* row_id_map, int k, moe_dtype dt, int64_t T, int H, void* dy,
                                        float* dweight, float* dgate, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  moe_status st = check_common("moe_post_norm_bwd", dt, T, H, k, row_id_map);
  if (st != MOE_OK) return st;
  if (!dweight || !aligned(dweight, 4)) return fail(MOE_ERR_INVALID_ARG, "moe_post_norm_bwd: dweight NULL or misaligned");
  const hipStream_t s = as_stream(stream);
  if (T == 0) return zero_dw(dweight, H, s, "moe_post_norm_bwd");
  if ((st = check_gate("moe_post_norm_bwd", gate_kind, gate, gate_group)) != MOE_OK) return st;
  if (!dout || !c || !rstd || !weight || !dy) return fail(MOE_ERR_INVALID_ARG, "moe_post_norm_bwd: NULL pointer");
  const size_t esz = dt == MOE_BF16 ? 2 : 4;
  const bool channel = gate_kind == GATE_CHANNEL;
  if (!all_aligned({dout, c, weight, gate, dy}, esz) || !all_aligned({rstd, row_id_map, dgate}, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_post_norm_bwd: misaligned pointer");
  if (workspace_bytes < norm_bwd_workspace_bytes(T, H, gate_kind, gate_group))
    return fail(MOE_ERR_WORKSPACE, "moe_post_norm_bwd: workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return fail(MOE_ERR_INVALID_ARG, "moe_post_norm_bwd: workspace NULL or not 256-byte aligned");
  BwdParams p{};
  p.dout = dout, p.c = c, p.rstd = rstd, p.w = weight, p.gate = gate, p.rows = row_id_map, p.dy = dy;
  p.dgate = dgate, p.part = (float*)workspace, p.T = T, p.group = channel ? gate_group : 1, p.H = H, p.k = k;
  p.plan = plan_chunks(T, gate_kind, gate_group);
  const bool vec = H * esz % 16 == 0 && all_aligned({dout, c, weight, channel ? gate : nullptr, dy}, 16);
  launch_bwd(p, gate_kind, dt == MOE_BF16, vec, dweight, s);
  return check_launch("moe_post_norm_bwd");
}
