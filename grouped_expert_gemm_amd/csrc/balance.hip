// Load-balance loss of the router with its z-loss term, the tokens each expert was
// given, and the gradient in the logits.
//
// Per sequence of L tokens, N of them counted, with p = softmax of a token's logits:
//   f_e = c_e / (k N),  P_e = mean_t p[t, e],  B = E sum_e f_e P_e,  Z = mean_t lse[t]^2
//   loss = mean over the sequences with N > 0 of (a B + b Z)
// f is piecewise constant, so only P and lse carry a gradient:
//   d_logits[t, e] = g / (S' N) p[t, e] (a E (f_e - sum_e' f_e' p[t, e']) + 2 b lse[t])
// Both use over_e = E f_e - 1 = (E c_e - k N) / (k N), whose numerator is an exact integer:
// since p sums to 1, B = 1 + sum over_e P_e and E (f_e - sum f p) = over_e - sum over p,
// without the cancellation of two nearly equal shares.
//
// A group of L lanes holds one token's row, 4 logits a lane (L = ceil(E / 4) rounded up to
// a power of two): 16-byte loads when E % 4 == 0 and the rows are aligned, else logits
// j, j + L, ... one at a time. A workgroup takes a run of tokens of one sequence and keeps
// the sums of p in registers; partial sums leave through the workspace and are added in a
// fixed order (counts are integers, whose LDS atomics commute), so results repeat bit for bit.
//
// 131072 tokens x 256 experts: the forward kernel takes 44 us for 138 MB, 27 us at the rate of a
// copy. What bounds it is the vector ALU (157 instructions of a wavefront a token, busy 75 to
// 81% of the time): two reductions over 64 lanes and the exponentials for four logits a lane.
// The backward, 403 MB with d_in, takes 67 us right after it.
#include <cmath>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMinTokens = 2;       // tokens of a group that are worth a workgroup and a partial sum of their own
constexpr int64_t kTargetWgs = 1024;
constexpr int64_t kMaxSeqs = 1 << 23;  // a launch holds 2^24 - 1 workgroups of 256 threads

struct BalancePlan {
  int64_t S, L, nch, chunk;  // sequences, tokens of each, workgroups per sequence, tokens per workgroup
};

inline int group_lanes(int E) {
  int L = 1;
  while (L * 4 < E) L *= 2;
  return L;
}

BalancePlan make_plan(int64_t T, int64_t seq_len, int E) {
  BalancePlan p{T / seq_len, seq_len, 1, 0};
  const int64_t step = (int64_t)(kThreads / group_lanes(E)) * kMinTokens;
  const int64_t most = (seq_len + step - 1) / step;
  int64_t want = p.S > 0 ? (kTargetWgs + p.S - 1) / p.S : 1;
  if (want > most) want = most;
  if (want < 1) want = 1;
  p.chunk = ((seq_len + want - 1) / want + step - 1) / step * step;
  p.nch = (seq_len + p.chunk - 1) / p.chunk;
  return p;
}

// workspace: [S * nch][E] sums of p, [S * nch] sums of lse^2, [S * nch][E] counts,
// [S * nch] token counts, then per sequence [S] balance and [S] z (one workgroup a sequence),
// or [S][E] sums of p and [S] of lse^2
struct BalanceWs {
  float* p;
  float* z;
  int32_t* c;
  int32_t* n;
  float* seq;
};

BalanceWs carve(void* ws, const BalancePlan& p, int E) {
  BalanceWs w;
  const int64_t parts = p.S * p.nch;
  w.p = (float*)ws;
  w.z = w.p + parts * E;
  w.c = (int32_t*)(w.z + parts);
  w.n = w.c + parts * E;
  w.seq = (float*)(w.n + parts);
  return w;
}

// expert of this lane's value q
template <int L, bool VEC>
__device__ __forceinline__ int expert_of(int j, int q) {
  return VEC ? 4 * j + q : j + q * L;
}

template <int L, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int j, int E, float* v) {
  if constexpr (VEC) {
    if (4 * j < E) {
      const float4 f = *reinterpret_cast<const float4*>(row + 4 * j);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      v[0] = v[1] = v[2] = v[3] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = j + q * L < E ? row[j + q * L] : -INFINITY;
  }
}

// the row's softmax in place of its logits, and its log-sum-exp; false for a row of
// nothing but -infinity, which has no softmax. A NaN counts as the maximum, so it reaches
// every value of the row (as does +infinity).
template <int L>
__device__ __forceinline__ bool softmax_row(float* v, float& lse) {
  float mx = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) mx = fmaxf(mx, isnan(v[q]) ? INFINITY : v[q]);
  mx = lanes_max<L>(mx);
  float den = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = expf(v[q] - mx);
    den += v[q];
  }
  den = lanes_sum<L>(den);
  const float inv = 1.f / den;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] *= inv;
  lse = mx + logf(den);
  return mx != -INFINITY;
}

// The sequence's balance and z from its sums (E <= 256 threads' worth in LDS), by the
// whole workgroup; counts and the token count written out.
struct SeqOut {
  int32_t* counts;   // [S][E]
  int32_t* tokens;   // [S + 1], the last: sequences with tokens
  float* loss;       // [3], written here only for one sequence
  float* seq;        // [2][S]
  float a, b;
  int64_t S;
  int E, k;
};

// without a z-loss its mean, which overflows at logits near the type's limits, stays out
__device__ __forceinline__ float total_loss(float a, float bal, float b, float z) {
  return b != 0.f ? a * bal + b * z : a * bal;
}

__device__ __forceinline__ void finish_sequence(const SeqOut& o, int64_t s, const float* sp, const int32_t* sc, float zsum,
                                                int n, float* red) {
  const int tid = threadIdx.x;
  float term = 0.f, mass = 0.f;
  if (tid < o.E) {
    const int c = sc[tid];
    o.counts[s * o.E + tid] = c;
    const int64_t kn = (int64_t)o.k * n;
    if (n > 0) {
      mass = sp[tid] / (float)n;
      term = (float)((int64_t)o.E * c - kn) / (float)kn * mass;
    }
  }
  // 256 values, pairwise in a fixed order; mass (1 but for rounding) keeps a NaN row visible
  float v = term + mass;
  v = lanes_sum<64>(v);
  if ((tid & 63) == 0) red[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    const float bal = n > 0 ? (red[0] + red[1]) + (red[2] + red[3]) : 0.f;
    const float z = n > 0 ? zsum / (float)n : 0.f;
    o.tokens[s] = n;
    if (o.S == 1) {
      o.tokens[1] = n > 0;
      o.loss[0] = total_loss(o.a, bal, o.b, z);
      o.loss[1] = bal;
      o.loss[2] = z;
    } else {
      o.seq[s] = bal;
      o.seq[o.S + s] = z;
    }
  }
}

// kDirect: one workgroup a sequence, which finishes it itself
template <int L, bool VEC, bool kDirect, int U>
__global__ __launch_bounds__(kThreads) void balance_fwd_kernel(const float* __restrict__ logits,
                                                               const int32_t* __restrict__ idx,
                                                               const uint8_t* __restrict__ mask, int64_t seq_len,
                                                               int64_t nch, int64_t chunk, BalanceWs ws, SeqOut o) {
  constexpr int G = kThreads / L;  // tokens of the workgroup at a time
  __shared__ float sp[4][256];     // per wavefront: sums of p
  __shared__ int32_t sc[256];
  __shared__ float sz[4], red[4];
  __shared__ int32_t sn[4];
  const int E = o.E, k = o.k;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = tid % L, g = tid / L;
  const int64_t s = blockIdx.x / nch, c = blockIdx.x % nch;
  const int64_t beg = s * seq_len + c * chunk;
  const int64_t len = seq_len - c * chunk < chunk ? seq_len - c * chunk : chunk;
  sc[tid] = 0;
  __syncthreads();
  float ps[4] = {0.f, 0.f, 0.f, 0.f};
  float zs = 0.f;
  int n = 0;
  for (int64_t i0 = 0; i0 < len; i0 += (int64_t)G * U) {  // the same trip count in every lane
    float v[U][4];
    int32_t id[U][4];  // this lane's slots j, j + L, ... (k <= E <= 4 L); -1: none
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * G + g;
      live[u] = i < len && (!mask || mask[beg + i] != 0);
      if (live[u]) load_row<L, VEC>(logits + (beg + i) * E, j, E, v[u]);
      else v[u][0] = v[u][1] = v[u][2] = v[u][3] = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) id[u][q] = live[u] && j + q * L < k ? idx[(beg + i) * k + j + q * L] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lse;
      const bool ok = softmax_row<L>(v[u], lse) && live[u];
      if (ok) {
#pragma unroll
        for (int q = 0; q < 4; ++q) ps[q] += v[u][q];
        if (j == 0) {
          zs += lse * lse;
          ++n;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if ((unsigned)id[u][q] < (unsigned)E) atomicAdd(&sc[id[u][q]], 1);
      }
    }
  }
  // over the wavefront's groups (lanes of one j), then over the wavefronts
#pragma unroll
  for (int m = L; m < 64; m <<= 1) {
#pragma unroll
    for (int q = 0; q < 4; ++q) ps[q] += __shfl_xor(ps[q], m, 64);
    zs += __shfl_xor(zs, m, 64);
    n += __shfl_xor(n, m, 64);
  }
  if (lane < L) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = expert_of<L, VEC>(j, q);
      if (e < E) sp[wave][e] = ps[q];
    }
  }
  if (lane == 0) {
    sz[wave] = zs;
    sn[wave] = n;
  }
  __syncthreads();
  const float pe = tid < E ? (sp[0][tid] + sp[1][tid]) + (sp[2][tid] + sp[3][tid]) : 0.f;
  const float z = (sz[0] + sz[1]) + (sz[2] + sz[3]);
  const int nn = sn[0] + sn[1] + sn[2] + sn[3];
  if constexpr (kDirect) {
    __syncthreads();
    sp[0][tid] = pe;
    __syncthreads();
    finish_sequence(o, s, sp[0], sc, z, nn, red);
  } else {
    if (tid < E) {
      ws.p[(int64_t)blockIdx.x * E + tid] = pe;
      ws.c[(int64_t)blockIdx.x * E + tid] = sc[tid];
    }
    if (tid == 0) {
      ws.z[blockIdx.x] = z;
      ws.n[blockIdx.x] = nn;
    }
  }
}

// A sequence's nch partial sums: 8 experts a workgroup, 32 threads an expert each adding
// every 32nd, eight loads in flight, then the 32 in order. The first workgroup of a sequence
// also adds its nch sums of lse^2 and token counts.
__global__ __launch_bounds__(kThreads) void balance_join_kernel(int64_t nch, BalanceWs ws, SeqOut o) {
  __shared__ float fp[32][9];
  __shared__ int32_t fc[32][9];
  __shared__ float fz[4];
  __shared__ int32_t fn[4];
  const int tid = threadIdx.x, E = o.E;
  const int64_t s = blockIdx.y, first = s * nch;
  const int e = blockIdx.x * 8 + (tid & 7), r0 = tid >> 3;
  float p = 0.f;
  int32_t c = 0;
  if (e < E) {
#pragma unroll 8
    for (int64_t r = r0; r < nch; r += 32) {
      p += ws.p[(first + r) * E + e];
      c += ws.c[(first + r) * E + e];
    }
  }
  fp[r0][tid & 7] = p;
  fc[r0][tid & 7] = c;
  if (blockIdx.x == 0) {
    float z = 0.f;
    int32_t n = 0;
    for (int64_t r = tid; r < nch; r += kThreads) {
      z += ws.z[first + r];
      n += ws.n[first + r];
    }
    z = lanes_sum<64>(z);
    n = (int32_t)lanes_reduce<64>((uint32_t)n, [](uint32_t a, uint32_t b) { return a + b; });
    if ((tid & 63) == 0) {
      fz[tid >> 6] = z;
      fn[tid >> 6] = n;
    }
  }
  __syncthreads();
  if (tid < 8 && e < E) {
    p = 0.f;
    c = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      p += fp[r][tid];
      c += fc[r][tid];
    }
    ws.seq[s * E + e] = p;
    o.counts[s * E + e] = c;
  }
  if (blockIdx.x == 0 && tid == 0) {
    ws.seq[o.S * E + s] = (fz[0] + fz[1]) + (fz[2] + fz[3]);
    o.tokens[s] = fn[0] + fn[1] + fn[2] + fn[3];
  }
}

// The loss from the joined sums: a wavefront a sequence at a time, then the 16 wavefronts in order.
__global__ __launch_bounds__(1024) void balance_loss_kernel(BalanceWs ws, SeqOut o) {
  __shared__ float fb[16], fz[16];
  __shared__ int32_t fn[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = o.E;
  float bal = 0.f, z = 0.f;
  int32_t seqs = 0;
  for (int64_t s = wave; s < o.S; s += 16) {
    const int32_t n = o.tokens[s];
    if (n == 0) continue;
    const int64_t kn = (int64_t)o.k * n;
    float v = 0.f;
    for (int e = lane; e < E; e += 64) {
      const float mass = ws.seq[s * E + e] / (float)n;
      v += (float)((int64_t)E * o.counts[s * E + e] - kn) / (float)kn * mass + mass;
    }
    bal += lanes_sum<64>(v);
    z += ws.seq[o.S * E + s] / (float)n;
    ++seqs;
  }
  if (lane == 0) {
    fb[wave] = bal;
    fz[wave] = z;
    fn[wave] = seqs;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) {
      bal += fb[w];
      z += fz[w];
      seqs += fn[w];
    }
    const float d = seqs > 0 ? (float)seqs : 1.f;
    bal /= d;
    z /= d;
    o.loss[0] = total_loss(o.a, bal, o.b, z);
    o.loss[1] = bal;
    o.loss[2] = z;
    o.tokens[o.S] = seqs;
  }
}

// the mean over the sequences with tokens, where each was finished by its one workgroup
__global__ __launch_bounds__(kThreads) void balance_mean_kernel(SeqOut o) {
  __shared__ float fb[256], fz[256];
  __shared__ int32_t fn[256];
  const int tid = threadIdx.x;
  float b = 0.f, z = 0.f;
  int32_t n = 0;
  for (int64_t s = tid; s < o.S; s += 256) {
    b += o.seq[s];
    z += o.seq[o.S + s];
    n += o.tokens[s] > 0;
  }
  fb[tid] = b, fz[tid] = z, fn[tid] = n;
  __syncthreads();
  for (int m = 128; m >= 1; m >>= 1) {
    if (tid < m) {
      fb[tid] += fb[tid + m];
      fz[tid] += fz[tid + m];
      fn[tid] += fn[tid + m];
    }
    __syncthreads();
  }
  if (tid == 0) {
    const float d = fn[0] > 0 ? (float)fn[0] : 1.f;
    const float bal = fb[0] / d, zz = fz[0] / d;
    o.loss[0] = total_loss(o.a, bal, o.b, zz);
    o.loss[1] = bal;
    o.loss[2] = zz;
    o.tokens[o.S] = fn[0];
  }
}

// d_in may be d_logits itself: each value is read and written by the same lane
template <int L, bool VEC, int U>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(const float* __restrict__ logits,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ tokens,
                                                               const uint8_t* __restrict__ mask,
                                                               const float* __restrict__ d_loss, const float* d_in,
                                                               float* d_logits, int64_t S, int64_t seq_len, int64_t nch,
                                                               int64_t chunk, int E, int k, float a, float b) {
  constexpr int G = kThreads / L;
  const int tid = threadIdx.x;
  const int j = tid % L, g = tid / L;
  const int64_t s = blockIdx.x / nch, c = blockIdx.x % nch;
  const int64_t beg = s * seq_len + c * chunk;
  const int64_t len = seq_len - c * chunk < chunk ? seq_len - c * chunk : chunk;
  const int n = tokens[s], seqs = tokens[S];
  const int64_t kn = (int64_t)k * n;
  float over[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = expert_of<L, VEC>(j, q);
    over[q] = e < E && n > 0 ? a * ((float)((int64_t)E * counts[s * E + e] - kn) / (float)kn) : 0.f;
  }
  const float scale = n > 0 ? (d_loss ? *d_loss : 1.f) / ((float)seqs * (float)n) : 0.f;
  const float b2 = 2.f * b;
  for (int64_t i0 = 0; i0 < len; i0 += (int64_t)G * U) {
    float v[U][4], w[U][4];
    bool in[U], live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * G + g;
      in[u] = i < len;
      live[u] = in[u] && n > 0 && (!mask || mask[beg + i] != 0);
      if (live[u]) load_row<L, VEC>(logits + (beg + i) * E, j, E, v[u]);
      else v[u][0] = v[u][1] = v[u][2] = v[u][3] = -INFINITY;
      if (in[u] && d_in) load_row<L, VEC>(d_in + (beg + i) * E, j, E, w[u]);
      else w[u][0] = w[u][1] = w[u][2] = w[u][3] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lse, share = 0.f;
      const bool ok = softmax_row<L>(v[u], lse) && live[u];
#pragma unroll
      for (int q = 0; q < 4; ++q) share += v[u][q] * over[q];
      share = lanes_sum<L>(share);
      const float base = b2 * lse - share;
      float r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = w[u][q] + (ok ? scale * (v[u][q] * (over[q] + base)) : 0.f);
      if (in[u]) {
        float* dst = d_logits + (beg + i0 + u * G + g) * E;
        if constexpr (VEC) {
          if (4 * j < E) *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(r[0], r[1], r[2], r[3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (j + q * L < E) dst[j + q * L] = r[q];
        }
      }
    }
  }
}

__global__ void balance_empty_kernel(float* loss, int32_t* tokens) {
  if (threadIdx.x < 3) loss[threadIdx.x] = 0.f;
  if (threadIdx.x == 3) tokens[0] = 0;
}

// f(lanes of a group, 16-byte rows, tokens of a group in flight) as compile-time constants. Four
// tokens in flight pay off where a workgroup's run is long enough to repeat them (131072 x 256:
// forward 50 -> 43 us), and only cost registers in runs of two to seven tokens a group (16384 x
// 128: forward 6.0 us with two, 8.1 with four).
template <typename F>
void dispatch(int E, bool vec, int64_t chunk, F&& f) {
  const bool long_run = chunk * group_lanes(E) >= 8 * kThreads;
  auto with = [&](auto Lc) {
    auto then = [&](auto Vc) {
      if (long_run) f(Lc, Vc, std::integral_constant<int, 4>{});
      else f(Lc, Vc, std::integral_constant<int, 2>{});
    };
    if (vec) then(std::true_type{});
    else then(std::false_type{});
  };
  switch (group_lanes(E)) {
    case 1: with(std::integral_constant<int, 1>{}); break;
    case 2: with(std::integral_constant<int, 2>{}); break;
    case 4: with(std::integral_constant<int, 4>{}); break;
    case 8: with(std::integral_constant<int, 8>{}); break;
    case 16: with(std::integral_constant<int, 16>{}); break;
    case 32: with(std::integral_constant<int, 32>{}); break;
    default: with(std::integral_constant<int, 64>{}); break;
  }
}

moe_status check_sizes(const char* fn, int64_t T, int E, int k, int64_t seq_len) {
  const std::string f(fn);
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, f + ": T < 0");
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, f + ": E out of [1, 256]");
  if (k < 1 || k > E) return fail(MOE_ERR_INVALID_ARG, f + ": k out of [1, E]");
  if (seq_len < 1 || T % seq_len != 0) return fail(MOE_ERR_INVALID_ARG, f + ": seq_len must divide T");
  if (T > 0x7FFFFFFF / k) return fail(MOE_ERR_UNSUPPORTED, f + ": T * k exceeds int32 counts");
  if (T / seq_len > kMaxSeqs) return fail(MOE_ERR_UNSUPPORTED, f + ": more than 2^23 sequences");
  return MOE_OK;
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t seq_len, int E) {
  const BalancePlan p = make_plan(T, seq_len, E);
  if (p.S * p.nch <= 1) return 0;  // one workgroup does it all
  return align_up((size_t)(p.S * p.nch) * (8 * (size_t)E + 8) + (size_t)p.S * (4 * (size_t)E + 8), 256);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* mask, int64_t T,
                                       int E, int k, int64_t seq_len, float balance_coef, float z_coef,
                                       int32_t* counts, int32_t* tokens, float* loss, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  moe_status st = check_sizes("moe_balance_loss", T, E, k, seq_len);
  if (st != MOE_OK) return st;
  if (!tokens || !loss) return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss: NULL pointer");
  if (!aligned(tokens, 4) || !aligned(loss, 4)) return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss: misaligned pointer");
  const hipStream_t s = as_stream(stream);
  if (T == 0) {
    hipLaunchKernelGGL(balance_empty_kernel, dim3(1), dim3(64), 0, s, loss, tokens);
    return check_launch("moe_balance_loss");
  }
  if (!logits || !topk_idx || !counts) return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss: NULL pointer");
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(counts, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss: misaligned pointer");
  const size_t need = balance_workspace_bytes(T, seq_len, E);
  if (workspace_bytes < need) return fail(MOE_ERR_WORKSPACE, "moe_balance_loss: workspace too small");
  if (need > 0 && (!workspace || !aligned(workspace, 256)))
    return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss: workspace NULL or not 256-byte aligned");
  const BalancePlan p = make_plan(T, seq_len, E);
  const BalanceWs ws = carve(workspace, p, E);
  const SeqOut o{counts, tokens, loss, ws.seq, balance_coef, z_coef, p.S, E, k};
  dispatch(E, E % 4 == 0 && aligned(logits, 16), p.chunk, [&](auto Lc, auto Vc, auto Uc) {
    constexpr int L = decltype(Lc)::value, U = decltype(Uc)::value;
    constexpr bool V = decltype(Vc)::value;
    const dim3 grid((unsigned)(p.S * p.nch)), block(kThreads);
    if (p.nch == 1)
      hipLaunchKernelGGL((balance_fwd_kernel<L, V, true, U>), grid, block, 0, s, logits, topk_idx, mask, seq_len, p.nch,
                         p.chunk, ws, o);
    else
      hipLaunchKernelGGL((balance_fwd_kernel<L, V, false, U>), grid, block, 0, s, logits, topk_idx, mask, seq_len, p.nch,
                         p.chunk, ws, o);
  });
  if (p.nch > 1) {  // fewer than kTargetWgs sequences
    hipLaunchKernelGGL(balance_join_kernel, dim3((E + 7) / 8, (unsigned)p.S), dim3(kThreads), 0, s, p.nch, ws, o);
    hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(1024), 0, s, ws, o);
  } else if (p.S > 1) {
    hipLaunchKernelGGL(balance_mean_kernel, dim3(1), dim3(kThreads), 0, s, o);
  }
  return check_launch("moe_balance_loss");
}

extern "C" moe_status moe_balance_loss_bwd(const float* logits, const int32_t* counts, const int32_t* tokens,
                                           const uint8_t* mask, int64_t T, int E, int k, int64_t seq_len,
                                           float balance_coef, float z_coef, const float* d_loss,
                                           const float* d_logits_in, float* d_logits, void* stream) {
  moe_status st = check_sizes("moe_balance_loss_bwd", T, E, k, seq_len);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !tokens || !d_logits) return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss_bwd: NULL pointer");
  if (!aligned(logits, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(d_logits, 4) ||
      !aligned(d_loss, 4) || !aligned(d_logits_in, 4))
    return fail(MOE_ERR_INVALID_ARG, "moe_balance_loss_bwd: misaligned pointer");
  const BalancePlan p = make_plan(T, seq_len, E);
  const bool vec = E % 4 == 0 && aligned(logits, 16) && aligned(d_logits, 16) && aligned(d_logits_in, 16);
  dispatch(E, vec, p.chunk, [&](auto Lc, auto Vc, auto Uc) {
    hipLaunchKernelGGL((balance_bwd_kernel<decltype(Lc)::value, decltype(Vc)::value, decltype(Uc)::value>), dim3((unsigned)(p.S * p.nch)),
                       dim3(kThreads), 0, as_stream(stream), logits, counts, tokens, mask, d_loss, d_logits_in,
                       d_logits, p.S, seq_len, p.nch, p.chunk, E, k, balance_coef, z_coef);
  });
  return check_launch("moe_balance_loss_bwd");
}
