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
// Teams of 1024 threads have 128 registers a thread, which the widest rows exceed: the channel-gate
// backward of more than 8192 elements spills 31 to 59 of them, the float32 post norm of more than
// 8192 elements 37 or 40, the float32 backward without a gate of unaligned such rows 11. Whole
// calls, 134 MB a tensor, against 8192 wide: channel-gate backward of bf16 4096 x 16384 121 us (67 MB
// at 4096 x 8192: 49), of float32 2048 x 16384 116 (4096 x 8192: 90); float32 post norm with
// c and the next norm 234 (141).
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxSlots = 16;

enum { GATE_NONE = 0, GATE_TOKEN = 1, GATE_CHANNEL = 2 };

// ---- vectors of 16 bytes: V = 8 bf16 or 4 float32 ----
template <bool BF16>
constexpr int kVec = BF16 ? 8 : 4;
typedef unsigned int raw_t __attribute__((ext_vector_type(4)));
typedef raw_t raw_any_t __attribute__((aligned(2)));  // at any element's address: the card reads those too

// One of a thread's vectors of a row of H elements: its first column, how many of the row's
// elements it holds, and where it is read. ALIGNED rows are whole 16-byte vectors. In other
// rows the last vector may be part-filled: it is read as the row's last 16 bytes, `skip`
// elements early, and shifted when it is used, so that no load waits for a branch; rows of
// less than one vector are read element by element.
struct Span {
  int col, cnt, at, skip;
};

template <int V>
__device__ __forceinline__ Span span(int H, int i) {
  Span c;
  c.col = i * V;
  c.cnt = min(max(H - c.col, 0), V);
  c.at = max(min(c.col, H - V), 0);
  c.skip = H < V ? 0 : min(c.col - c.at, V);
  return c;
}

// SHORT: the row may be shorter than a vector
template <bool BF16, bool ALIGNED, bool SHORT>
__device__ __forceinline__ raw_t load_vec(const void* base, int64_t row, const Span& c, int H) {
  typedef typename std::conditional<BF16, uint16_t, float>::type elem_t;
  const elem_t* p = (const elem_t*)base + row;
  raw_t r = {0, 0, 0, 0};
  if constexpr (ALIGNED) {
    if (c.cnt > 0) r = *reinterpret_cast<const raw_t*>(p + c.col);
  } else if (!SHORT || H >= kVec<BF16>) {
    r = *reinterpret_cast<const raw_any_t*>(p + c.at);
  } else {
#pragma unroll
    for (int i = 0; i < kVec<BF16> - 1; ++i)
      if (i < c.cnt) {
        if constexpr (BF16) r[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        else r[i] = __float_as_uint(p[i]);
      }
  }
  return r;
}

// a loaded vector without the elements before its first column, zeros behind the row's end
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ raw_t settle(raw_t r, const Span& c) {
  if constexpr (!ALIGNED)
    if (c.skip > 0) {
      int s = c.skip;
      if constexpr (BF16) {
        if (s & 1) r = raw_t{r[0] >> 16 | r[1] << 16, r[1] >> 16 | r[2] << 16, r[2] >> 16 | r[3] << 16, r[3] >> 16};
        s >>= 1;
      }
      if (s & 1) r = raw_t{r[1], r[2], r[3], 0};
      if (s & 2) r = raw_t{r[2], r[3], 0, 0};
      if (s & 4) r = raw_t{0, 0, 0, 0};
    }
  return r;
}

template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void store_vec(void* base, int64_t at, int n, raw_t r) {
  typedef typename std::conditional<BF16, uint16_t, float>::type elem_t;
  elem_t* p = (elem_t*)base + at;
  if constexpr (ALIGNED) {
    if (n > 0) *reinterpret_cast<raw_t*>(p) = r;
  } else if (n == kVec<BF16>) {
    *reinterpret_cast<raw_any_t*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < kVec<BF16> - 1; ++i)
      if (i < n) {
        if constexpr (BF16) p[i] = (uint16_t)(r[i / 2] >> (16 * (i & 1)));
        else p[i] = __uint_as_float(r[i]);
      }
  }
}

// the first n of V sums
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void store_sums(float* p, int n, const float* v) {
  constexpr int V = kVec<BF16>;
  if constexpr (ALIGNED) {
    if (n > 0)
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = v[i];
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack(raw_t r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    } else {
      v[i] = __uint_as_float(r[i]);
    }
  }
}

template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void unpack(raw_t r, const Span& c, float* v) {
  unpack<BF16>(settle<BF16, ALIGNED>(r, c), v);
}

template <bool BF16>
__device__ __forceinline__ raw_t pack(const float* v) {
  if constexpr (BF16)
    return raw_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  else return raw_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
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
template <bool BF16, bool AL, int TPR, int NV, bool kPost>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(const FwdParams p) {
  constexpr int V = kVec<BF16>;
  constexpr bool kShort = TPR * NV == 64;
  constexpr int kTeams = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
  const int tr = threadIdx.x % TPR;
  const int H = p.H;
  const float inv_h = 1.f / (float)H;  // applied to each term: a sum of squares would overflow H times earlier
  raw_t w[NV], w2[NV];
  Span c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i] = span<V>(H, i * TPR + tr);
    w[i] = settle<BF16, AL>(load_vec<BF16, AL, kShort>(p.w, 0, c[i], H), c[i]);
    w2[i] = kPost && p.w_next ? settle<BF16, AL>(load_vec<BF16, AL, kShort>(p.w_next, 0, c[i], H), c[i]) : raw_t{};
  }
  // every thread of a workgroup runs the same rows' loop (team_sum has barriers only where
  // the workgroup is one team)
  for (int64_t t = (int64_t)blockIdx.x * kTeams + threadIdx.x / TPR; t < p.T; t += (int64_t)gridDim.x * kTeams) {
    float acc[NV][V];
    raw_t xr[NV];
    if constexpr (kPost) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        xr[i] = load_vec<BF16, AL, kShort>(p.x, t * H, c[i], H);
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
#pragma unroll
          for (int i = 0; i < NV; ++i)
            q[u][i] = j0 + u < p.k ? load_vec<BF16, AL, kShort>(p.y, ok[u] ? (int64_t)r * H : 0, c[i], H) : raw_t{};
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (ok[u]) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              float f[V];
              unpack<BF16, AL>(q[u][i], c[i], f);
#pragma unroll
              for (int v = 0; v < V; ++v) acc[i][v] += f[v];
            }
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<BF16, AL>(load_vec<BF16, AL, kShort>(p.y, t * H, c[i], H), c[i], acc[i]);
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
    const int64_t grow = kPost && p.gate_kind == GATE_CHANNEL ? t / p.group * H : 0;
    float ss2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = t * H + c[i].col;
      if constexpr (kPost)
        if (p.c) store_vec<BF16, AL>(p.c, at, c[i].cnt, pack<BF16>(acc[i]));
      float f[V];
      unpack<BF16>(w[i], f);
      if constexpr (kPost) {
        float x[V], g[V];
        unpack<BF16, AL>(xr[i], c[i], x);
        if (p.gate_kind == GATE_CHANNEL) {
          unpack<BF16, AL>(load_vec<BF16, AL, kShort>(p.gate, grow, c[i], H), c[i], g);
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
      const raw_t o = pack<BF16>(acc[i]);
      store_vec<BF16, AL>(p.out, at, c[i].cnt, o);
      if constexpr (kPost) {  // the next norm reads the sum as it was stored (0 past the row's end)
        unpack<BF16>(o, acc[i]);
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
          unpack<BF16>(w2[i], f);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[i][v] = acc[i][v] * r2 * f[v];
          store_vec<BF16, AL>(p.y_next, t * H + c[i].col, c[i].cnt, pack<BF16>(acc[i]));
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
// The partial rows of all runs come to about 2^21 floats, which the caches hold: 512 runs of
// wide rows, up to 2048 of narrow ones, whose teams of one wavefront need that many to fill
// the card (131072 x 128 in bf16: 151 us with 512 runs, 49 with 2048; 16384 x 2048 to 8 rows
// a token: 169 with 512, 147 with 1024; 32768 x 4096: 165 with 512, 173 with 1024). A run has
// at least 4 rows, down to one for few tokens, where the rows that follow one another take
// longer than more partial rows to join (64 x 4096: 10.6 us with 4 rows a run, 8.1 with one;
// 512 x 8192: 20.6 and 23.4).
struct ChunkPlan {
  int64_t chunks, chunk, pieces;
};

ChunkPlan plan_chunks(int64_t T, int H, int gate_kind, int64_t group) {
  ChunkPlan p{0, 1, 1};
  if (T == 0) return p;
  const int64_t fit = (1 << 21) / H, target = fit < 512 ? 512 : fit > 2048 ? 2048 : fit;
  const int64_t least = T <= 128 ? 1 : T <= 384 ? (T + 127) / 128 : 4;
  int64_t c = (T + target - 1) / target;
  if (c < least) c = least;
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
template <bool BF16, bool AL, int TPR, int NV, int GATE>
__global__ __launch_bounds__(TPR) void norm_bwd_kernel(const BwdParams p) {
  constexpr int V = kVec<BF16>;
  constexpr bool kShort = TPR * NV == 64;
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
  Span c[NV];
  float sum[NV][V], own[NV][V];  // own: sum of a over the current group (channel gates)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i] = span<V>(H, i * TPR + tr);
    w[i] = settle<BF16, AL>(load_vec<BF16, AL, kShort>(p.w, 0, c[i], H), c[i]);
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
      dr[i] = load_vec<BF16, AL, kShort>(p.dout, t * H, c[i], H);
      cr[i] = load_vec<BF16, AL, kShort>(p.c, t * H, c[i], H);
      xr[i] = GATE == GATE_NONE && p.dx_in ? load_vec<BF16, AL, kShort>(p.dx_in, t * H, c[i], H) : raw_t{};
    }
    const float r = p.rstd[t];
    float gt = 1.f;
    if (GATE == GATE_TOKEN) gt = BF16 ? bf16_to_f32(((const uint16_t*)p.gate)[t]) : ((const float*)p.gate)[t];
    if (GATE == GATE_CHANNEL && (t == t0 || t % p.group == 0)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) graw[i] = settle<BF16, AL>(load_vec<BF16, AL, kShort>(p.gate, t / p.group * H, c[i], H), c[i]);
    }
    float n[NV][V], d[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V];
      unpack<BF16, AL>(cr[i], c[i], n[i]);
      unpack<BF16, AL>(dr[i], c[i], d[i]);
      unpack<BF16>(w[i], f);
      if (GATE == GATE_CHANNEL) unpack<BF16>(graw[i], g);
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
      unpack<BF16, AL>(xr[i], c[i], x);
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
        for (int i = 0; i < NV; ++i) store_vec<BF16, AL>(p.dy, (int64_t)row * H + c[i].col, c[i].cnt, pack<BF16>(d[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) store_vec<BF16, AL>(p.dy, t * H + c[i].col, c[i].cnt, pack<BF16>(d[i]));
    }
    if (GATE == GATE_CHANNEL && p.plan.pieces == 1 && (t + 1 == t1 || (t + 1) % p.group == 0)) {  // the group ends here
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[V], g[V];
        unpack<BF16>(w[i], f);
        unpack<BF16>(graw[i], g);
        float dg[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dg[v] = f[v] * own[i][v];
          sum[i][v] += g[v] * own[i][v];
          own[i][v] = 0.f;
        }
        if (p.dgate) store_sums<BF16, AL>(p.dgate + t / p.group * H + c[i].col, c[i].cnt, dg);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    store_sums<BF16, AL>(p.part + ch * H + c[i].col, c[i].cnt, GATE == GATE_CHANNEL && p.plan.pieces > 1 ? own[i] : sum[i]);
}

__device__ __forceinline__ float fold4(float s) {  // the sum of a column's 4 threads of the wavefront
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  s = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// dw (and, for pieces, d_gate): 16 columns a workgroup and 64 threads a column (4 a
// wavefront), `par` <= 16 groups of them on different gate groups at a time and 64 / par on
// the pieces of each; sums in a fixed order. The partial rows come from other XCDs' caches,
// so what counts is that all of a column's loads are in flight at once (512 rows x 4096
// columns: 10.3 us with 16 threads a column). More than 64 groups (then of few pieces each):
// par = 64, one thread a group, as 16 at a time would wait for memory once for every 16 (131072
// x 128 in groups of 65 tokens, the whole backward: 169 -> 62 us).
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* __restrict__ part, int64_t groups, int64_t pieces,
                                                         int par, int H, const void* __restrict__ w,
                                                         const void* __restrict__ gate, float* __restrict__ dw,
                                                         float* __restrict__ dgate) {
  __shared__ float sums[16][17];
  const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 16 + cl;
  float total = 0.f;
  if (par == 64) {
    if (col < H) {
      const float wv = BF16 ? bf16_to_f32(((const uint16_t*)w)[col]) : ((const float*)w)[col];
#pragma unroll 4
      for (int64_t g = q; g < groups; g += 64) {
        const float* src = part + g * pieces * H + col;
        float s = 0.f;
        for (int64_t i = 0; i < pieces; ++i) s += src[i * H];
        if (dgate) dgate[g * H + col] = wv * s;
        total += (BF16 ? bf16_to_f32(((const uint16_t*)gate)[g * H + col]) : ((const float*)gate)[g * H + col]) * s;
      }
    }
    total = fold4(total);
    if ((q & 3) == 0) sums[wave][cl] = total;
    __syncthreads();
    if (q == 0 && col < H) {
      for (int i = 1; i < 16; ++i) total += sums[i][cl];
      dw[col] = total;
    }
    return;
  }
  const int each = 64 / par, gq = q / each, sub = q % each;
  const int waves = each / 4;                            // wavefronts on one group
  const bool lead = wave % waves == 0 && (q & 3) == 0;   // the thread that finishes its group's column
  for (int64_t g0 = 0; g0 < groups; g0 += par) {
    const int64_t g = g0 + gq;
    float s = 0.f;
    if (col < H && g < groups) {
      const float* src = part + g * pieces * H + col;
#pragma unroll 8
      for (int64_t i = sub; i < pieces; i += each) s += src[i * H];
    }
    s = fold4(s);  // then the group's wavefronts in order
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

// f(BF16, ALIGNED, TPR, NV): the narrowest team and fewest vectors a thread that hold the row.
// MANY: rows enough to fill the card with one wavefront each; a row of up to 64 x 4 vectors then
// goes to one wavefront, which reduces without barriers and keeps four times the rows of a
// 256-thread team in flight (16384 x 2048, 8 rows combined: 185 -> 153 us; a single row takes
// longer that way).
template <bool MANY, typename F>
void dispatch(bool bf16, bool al, int H, F&& f) {
  auto by_width = [&](auto B, auto A) {
    const int u = (H + kVec<decltype(B)::value> - 1) / kVec<decltype(B)::value>;  // vectors of a row
    if (u <= 64) f(B, A, Int<64>{}, Int<1>{});
    else if (u <= 128) f(B, A, Int<64>{}, Int<2>{});
    else if (u <= 256) f(B, A, Int<MANY ? 64 : 256>{}, Int<MANY ? 4 : 1>{});
    else if (u <= 512) f(B, A, Int<256>{}, Int<2>{});
    else if (u <= 1024) f(B, A, Int<256>{}, Int<4>{});
    else if (u <= 2048) f(B, A, Int<1024>{}, Int<2>{});
    else if constexpr (!decltype(B)::value) f(B, A, Int<1024>{}, Int<4>{});  // float32 up to 16384
  };
  auto by_rows = [&](auto B) {
    if (al) by_width(B, std::true_type{});
    else by_width(B, std::false_type{});
  };
  if (bf16) by_rows(std::true_type{});
  else by_rows(std::false_type{});
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
  auto go = [&](auto B, auto Vc, auto Tc, auto Nc) {
    constexpr int TPR = decltype(Tc)::value;
    constexpr int teams = TPR < 256 ? 256 / TPR : 1;
    int64_t grid = (p.T + teams - 1) / teams;
    const int64_t most = (int64_t)num_cus() * 8;
    if (grid > most) grid = most;
    hipLaunchKernelGGL((norm_fwd_kernel<decltype(B)::value, decltype(Vc)::value, TPR, decltype(Nc)::value, kPost>),
                       dim3((unsigned)grid), dim3(TPR < 256 ? 256 : TPR), 0, s, p);
  };
  if (p.T >= 4 * num_cus()) dispatch<true>(bf16, vec, p.H, go);
  else dispatch<false>(bf16, vec, p.H, go);
}

void launch_bwd(const BwdParams& p, int gate_kind, bool bf16, bool vec, float* dw, hipStream_t s) {
  dispatch<false>(bf16, vec, p.H, [&](auto B, auto Vc, auto Tc, auto Nc) {
    constexpr int TPR = decltype(Tc)::value;
    const dim3 grid((unsigned)p.plan.chunks), block(TPR);
    constexpr bool b = decltype(B)::value;
    constexpr bool V = decltype(Vc)::value;
    constexpr int NV = decltype(Nc)::value;
    if (gate_kind == GATE_TOKEN) hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_TOKEN>), grid, block, 0, s, p);
    else if (gate_kind == GATE_CHANNEL) hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_CHANNEL>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((norm_bwd_kernel<b, V, TPR, NV, GATE_NONE>), grid, block, 0, s, p);
  });
  const bool pieces = p.plan.pieces > 1;
  const dim3 grid((unsigned)((p.H + 15) / 16));
  const int64_t groups = pieces ? p.plan.chunks / p.plan.pieces : 1, each = pieces ? p.plan.pieces : p.plan.chunks;
  int par = 1;
  while (par < 16 && par < groups) par *= 2;
  if (groups > 64) par = 64;
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
  return align_up((size_t)plan_chunks(T, H, gate_kind, gate_group).chunks * H * 4, 256);
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
  p.part = (float*)workspace, p.T = T, p.H = H, p.k = 1, p.plan = plan_chunks(T, H, GATE_NONE, 0);
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
  p.plan = plan_chunks(T, H, gate_kind, gate_group);
  const bool vec = H * esz % 16 == 0 && all_aligned({dout, c, weight, channel ? gate : nullptr, channel ? dgate : nullptr, dy}, 16);
  launch_bwd(p, gate_kind, dt == MOE_BF16, vec, dweight, s);
  return check_launch("moe_post_norm_bwd");
}
