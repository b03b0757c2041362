// Grouped MLP entry points: GroupedLinear(gate_up) -> ScaledSwiGLU -> GroupedLinear(down)
// and its backward, per "Efficient MoE Training for Biological Foundation Models",
// Challenge 3. Host code: argument checks, workspace carving, kernel sequencing on
// the caller's stream.
#include <cstring>
#include <string>

#include "common.h"
#include "gemm_bf16.h"
#include "gemm_f32.h"
#include "gemm_mx.h"
#include "internal.h"
#include "lanes.h"
#include "mxfp4.h"
#include "mxfp8.h"

namespace moe {

static bool is_act_ok(const moe_mlp_desc& d) {
  switch (d.compute) {
    case MOE_F32: return d.act == MOE_F32 && d.wt == MOE_F32;
    case MOE_BF16: return d.act == MOE_BF16 && d.wt == MOE_BF16;
    case MOE_MXFP8: return (d.act == MOE_BF16 || d.act == MOE_MXFP8) && (d.wt == MOE_BF16 || d.wt == MOE_MXFP8);
    case MOE_FP8: return (d.act == MOE_BF16 || d.act == MOE_FP8) && (d.wt == MOE_BF16 || d.wt == MOE_FP8);
    case MOE_MXFP4: return (d.act == MOE_BF16 || d.act == MOE_MXFP4) && (d.wt == MOE_BF16 || d.wt == MOE_MXFP4);
  }
  return false;
}

moe_status validate_desc(const moe_mlp_desc& d, bool backward) {
  if (d.E < 1 || d.E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, "grouped MLP: E out of [1, 256]");
  if (d.H < 1 || d.I < 1) return fail(MOE_ERR_INVALID_ARG, "grouped MLP: H and I must be positive");
  if (d.compute != MOE_F32 && d.compute != MOE_BF16 && d.compute != MOE_MXFP8 && d.compute != MOE_FP8 &&
      d.compute != MOE_MXFP4)
    return fail(MOE_ERR_INVALID_ARG, "grouped MLP: bad compute dtype");
  if (!is_act_ok(d)) return fail(MOE_ERR_INVALID_ARG, "grouped MLP: act/wt storage does not match compute dtype");
  if ((int64_t)d.H * d.I * 2 > 0x7FFFFFFFLL)
    return fail(MOE_ERR_UNSUPPORTED, "grouped MLP: one expert's weight exceeds 2^31 bytes");
  if (d.compute == MOE_BF16 || d.compute == MOE_MXFP8 || d.compute == MOE_FP8) {
    if (d.H % 256 != 0 || d.I % 128 != 0)
      return fail(MOE_ERR_UNSUPPORTED, "grouped MLP: bf16/fp8 kernels need H % 256 == 0 and I % 128 == 0");
    if (backward && d.I % 256 != 0)
      return fail(MOE_ERR_UNSUPPORTED, "grouped MLP backward: bf16 kernels need I % 256 == 0");
  }
  if (d.compute == MOE_MXFP4) {
    if (backward || d.save_for_bwd)
      return fail(MOE_ERR_UNSUPPORTED, "grouped MLP: MXFP4 has a forward only (save_for_bwd must be 0)");
    const moe_status st = mx4::check_shape(d.E, d.H, d.I, "grouped MLP");
    if (st != MOE_OK) return st;
  }
  if (backward && d.compute == MOE_FP8 && d.act != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "grouped MLP backward: per-tensor FP8 takes bf16 activations (and bf16 master "
                                     "weights or weights packed by fp8_tensor_pack_weight_bwd)");
  if (backward && d.compute == MOE_MXFP8 && d.act != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "grouped MLP backward: MXFP8 takes bf16 activations (and bf16 master weights or "
                                     "weights packed by mxfp8_pack_weight_bwd)");
  return MOE_OK;
}

static size_t a256(size_t x) { return align_up(x, 256); }

size_t mlp_fwd_workspace_bytes(const moe_mlp_desc& d, int64_t R) {
  const size_t I = d.I, H = d.H, E = d.E;
  switch (d.compute) {
    case MOE_F32: return d.save_for_bwd ? 0 : a256(R * I * 4);
    case MOE_BF16: return (d.save_for_bwd ? 0 : a256(R * I * 2)) + grouped_gemm_workspace_bytes();
    case MOE_MXFP8: {
      size_t b = 0;
      // codes and step-major scales of what is given in bf16; converted scales otherwise
      b += (d.act == MOE_BF16 ? a256(R * H) : 0) + a256(R * H / 32);
      b += E * ((d.wt == MOE_BF16 ? a256(2 * I * H) + a256(H * I) : 0) + a256(2 * I * H / 32) + a256(H * I / 32));
      b += a256(R * I) + a256(R * I / 32);  // h as MXFP8
      return b;
    }
    case MOE_FP8: return mx::fp8_tensor_workspace_bytes(d, R);
    case MOE_MXFP4: return mx4::mlp_workspace_bytes(d, R);
  }
  return 0;
}

size_t grouped_gemm_workspace_bytes() { return a256(gemm::tail_ws_bytes(num_cus())); }

size_t mlp_bwd_workspace_bytes(const moe_mlp_desc& d, int64_t R) {
  const size_t I = d.I;
  if (d.compute == MOE_F32) return a256(4 * R * I * 4);
  if (d.compute == MOE_MXFP8) return mx::bwd_workspace_bytes(d, R);
  if (d.compute == MOE_FP8) return mx::fp8_bwd_workspace_bytes(d, R);
  return a256(R * 2 * I * 2) + a256((size_t)2 * (I / 256) * R * 4) + grouped_gemm_workspace_bytes();
}

moe_status validate_ckpt8(const moe_mlp_desc& d, bool backward, const char* what) {
  const std::string fn(what);
  if (d.E < 1 || d.E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, fn + ": E out of [1, 256]");
  if (d.H < 1 || d.I < 1) return fail(MOE_ERR_INVALID_ARG, fn + ": H and I must be positive");
  if (d.compute != MOE_BF16 || d.wt != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, fn + ": 8-bit checkpoints are built for bf16 products (compute and wt MOE_BF16)");
  if (d.act != MOE_BF16 && !(backward && d.act == MOE_MXFP8))
    return fail(MOE_ERR_UNSUPPORTED, fn + (backward ? ": act must be MOE_BF16 or MOE_MXFP8" : ": act must be MOE_BF16"));
  if (d.H % 256 != 0 || d.I % 256 != 0) return fail(MOE_ERR_UNSUPPORTED, fn + ": needs H % 256 == 0 and I % 256 == 0");
  if ((int64_t)d.H * d.I * 2 > 0x7FFFFFFFLL) return fail(MOE_ERR_UNSUPPORTED, fn + ": one expert's weight exceeds 2^31 bytes");
  return MOE_OK;
}

// [dZ] [h, then x] [dprob partials] [split-K tail]
static size_t ckpt8_rows_bytes(const moe_mlp_desc& d, int64_t R) {
  const int64_t wide = d.act == MOE_MXFP8 && d.H > d.I ? d.H : d.I;
  return a256((size_t)R * wide * 2);
}

size_t mlp_bwd_ckpt8_workspace_bytes(const moe_mlp_desc& d, int64_t R) {
  return a256((size_t)R * 2 * d.I * 2) + ckpt8_rows_bytes(d, R) + a256((size_t)2 * (d.I / 256) * R * 4) +
         grouped_gemm_workspace_bytes();
}

static moe_status check_table(const void* const* t, int E, size_t align, const char* what) {
  if (!t) return fail(MOE_ERR_INVALID_ARG, std::string(what) + ": pointer table is NULL");
  for (int e = 0; e < E; ++e) {
    if (!t[e]) return fail(MOE_ERR_INVALID_ARG, std::string(what) + ": NULL pointer for expert " + std::to_string(e));
    if (!aligned(t[e], align))
      return fail(MOE_ERR_INVALID_ARG, std::string(what) + ": expert pointer not " + std::to_string(align) +
                                           "-byte aligned");
  }
  return MOE_OK;
}

static PtrTab make_tab(const void* const* t, int E) {
  PtrTab tab;
  std::memset(&tab, 0, sizeof(tab));
  for (int e = 0; e < E; ++e) tab.p[e] = t[e];
  return tab;
}

// dprob[r] = sum over j of part[j][r] in a fixed order (deterministic): 8 threads per
// row each add the partials j = q, q + 8, ... in increasing j, then the 8 sums are added
// in q order. 32 rows per workgroup, consecutive threads on consecutive rows.
// With offsets, rows past the last expert's are not written.
__global__ __launch_bounds__(256) void reduce_partials(const float* __restrict__ part, int nparts, int64_t R,
                                                       float* __restrict__ out, const int32_t* __restrict__ offsets, int E) {
  __shared__ float sums[8][32];
  const int64_t end = offsets ? routed_end(offsets, E, R) : R;
  const int rl = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t r = (int64_t)blockIdx.x * 32 + rl;
  float s = 0.f;
  if (r < R)
    for (int j = q; j < nparts; j += 8) s += part[(int64_t)j * R + r];
  sums[q][rl] = s;
  __syncthreads();
  if (q == 0 && r < R) {
    float t = sums[0][rl];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sums[i][rl];
    if (r < end) out[r] = t;
  }
}

// split-K tail area carved from a workspace (nullptr: the kernels never split)
struct TailArea {
  float* part = nullptr;
  int32_t* meta = nullptr;
  int cap = 0;
  bool spread = false;
};
static TailArea tail_area(uint8_t* base) {
  TailArea t;
  if (!base) return t;
  t.meta = reinterpret_cast<int32_t*>(base);
  t.part = reinterpret_cast<float*>(base + gemm::kTailMetaSpace);
  t.cap = num_cus();
  return t;
}
// row tiles of E experts that share R rows, at most (an expert without rows has none)
static int64_t most_row_tiles(int E, int64_t R, const TailArea& t) {
  if (t.spread && R < E) E = (int)R;
  return (t.spread ? R : R + gemm::kBM - 1) / gemm::kBM + E;
}
// The tail of a product of R rows by n_tiles column tiles in the 8-bit checkpoint calls: tiles
// fewer than the CUs are cut along K as well (16 tiles of K = 4096: 82 us with one workgroup a tile),
// but not for K <= 512 (forwards whose down product has K = 512: 12 to 129 rows 32 to 43 us, at most 2 less
// when it is cut, 600 rows 53.6 and 62.0, 1500 rows 52.6 and 64.8) unless its epilogue is long and no
// launch of whole tiles has to come first: then the join, which spreads the epilogue over the card, pays
// for itself.
static TailArea tail_for(const TailArea& t, int E, int64_t R, int K, int n_tiles, bool long_epilogue) {
  TailArea r = t;
  r.spread = true;
  if (K <= 512 && !(long_epilogue && most_row_tiles(E, R, r) * n_tiles * 2 <= r.cap))
    r.cap = 0, r.part = nullptr, r.meta = nullptr;
  return r;
}
static void set_tail(gemm::Params& p, const TailArea& t) {
  p.tail = t.part;
  p.tail_meta = t.meta;
  p.tail_cap = t.cap;
  p.spread = t.spread;
}

// bf16 GroupedLinear(gate_up) + ScaledSwiGLU: h [R, I] (and z [R, 2I] when z != NULL, or its MXFP8
// codes and scales when z8 != NULL)
static moe_status bf16_gate_up(int E, int64_t R, int H, int I, const bf16_t* x, const PtrTab& w,
                               const int32_t* offsets, const float* prob, bf16_t* h, bf16_t* z, hipStream_t s,
                               const TailArea& tail = TailArea(), uint8_t* z8 = nullptr, uint8_t* z8s = nullptr) {
  gemm::Params p;
  std::memset(&p, 0, sizeof(p));
  set_tail(p, tail);
  std::memcpy(p.tab, w.p, sizeof(p.tab));
  p.q = x;
  p.q_ld = H;
  p.p_ld = H;
  p.c = h;
  p.c_ld = I;
  p.offsets = offsets;
  p.prob = prob;
  p.zout = z;
  p.z8 = z8;
  p.z8s = z8s;
  p.R = R;
  p.N = 2 * I;
  p.K = H;
  p.E = E;
  p.I = I;
  p.n_tiles = I / 128;
  const int64_t mtiles = most_row_tiles(E, R, tail);
  return gemm::run(p, gemm::KCONTIG, gemm::KCONTIG, gemm::GROUP_M, z8 ? gemm::EPI_SWIGLU_MX8 : gemm::EPI_SWIGLU,
                   mtiles * p.n_tiles, s, "grouped gate_up + ScaledSwiGLU");
}

// bf16 GroupedLinear: y [R, N] = x [R, K] W_e^T
static moe_status bf16_linear(int E, int64_t R, int K, int N, const bf16_t* x, const PtrTab& w,
                              const int32_t* offsets, bf16_t* y, hipStream_t s, const TailArea& tail = TailArea()) {
  gemm::Params q;
  std::memset(&q, 0, sizeof(q));
  set_tail(q, tail);
  std::memcpy(q.tab, w.p, sizeof(q.tab));
  q.q = x;
  q.q_ld = K;
  q.p_ld = K;
  q.c = y;
  q.c_ld = N;
  q.offsets = offsets;
  q.R = R;
  q.N = N;
  q.K = K;
  q.E = E;
  q.n_tiles = N / gemm::kBN;
  const int64_t mtiles = most_row_tiles(E, R, tail);
  return gemm::run(q, gemm::KCONTIG, gemm::KCONTIG, gemm::GROUP_M, gemm::EPI_STORE, mtiles * q.n_tiles, s,
                   "grouped linear");
}

// The products of the bf16 backward. dH = dY W2_e (W2_e is [H][I]: K rows, I contiguous) with the
// dSwiGLU epilogue: dz [R, 2I] and dprob from z [R, 2I] in bf16, or (z NULL) from its MXFP8 codes
// and scales, then with h [R, I] too and without dprob's rows past the last expert's.
static moe_status bf16_down_dgrad(const moe_mlp_desc& d, int64_t R, const bf16_t* dy, const PtrTab& w2,
                                  const int32_t* offsets, const float* prob, const bf16_t* z, bf16_t* dz, float* part,
                                  float* dprob, hipStream_t s, const uint8_t* z8 = nullptr,
                                  const uint8_t* z8s = nullptr, bf16_t* h = nullptr,
                                  const TailArea& tail = TailArea()) {
  gemm::Params p;
  std::memset(&p, 0, sizeof(p));
  std::memcpy(p.tab, w2.p, sizeof(p.tab));
  p.q = dy;
  p.q_ld = d.H;
  p.p_ld = d.I;
  p.c = dz;
  p.c_ld = 2 * (int64_t)d.I;
  p.offsets = offsets;
  p.prob = prob;
  p.zin = z;
  p.z8 = const_cast<uint8_t*>(z8);
  p.z8s = const_cast<uint8_t*>(z8s);
  p.hout = h;
  p.part = part;
  p.R = R;
  p.N = d.I;
  p.K = d.H;
  p.E = d.E;
  p.I = d.I;
  p.n_tiles = d.I / gemm::kBN;
  set_tail(p, tail);
  const int64_t mtiles = most_row_tiles(d.E, R, tail);
  moe_status st = gemm::run(p, gemm::MNCONTIG, gemm::KCONTIG, gemm::GROUP_M, z ? gemm::EPI_DSWIGLU : gemm::EPI_DSWIGLU_MX8,
                            mtiles * p.n_tiles, s, "moe_grouped_mlp_bwd(down dgrad)");
  if (st != MOE_OK) return st;
  hipLaunchKernelGGL(reduce_partials, dim3((unsigned)((R + 31) / 32)), dim3(256), 0, s, (const float*)part,
                     2 * p.n_tiles, R, dprob, z ? nullptr : offsets, d.E);
  return check_launch("moe_grouped_mlp_bwd(dprob)");
}

// dX = dZ W1_e (W1_e is [2I][H]: K rows, H contiguous)
static moe_status bf16_gate_up_dgrad(const moe_mlp_desc& d, int64_t R, const bf16_t* dz, const PtrTab& w1,
                                     const int32_t* offsets, bf16_t* dx, const TailArea& tail, hipStream_t s) {
  gemm::Params q;
  std::memset(&q, 0, sizeof(q));
  std::memcpy(q.tab, w1.p, sizeof(q.tab));
  q.q = dz;
  q.q_ld = 2 * (int64_t)d.I;
  q.p_ld = d.H;
  q.c = dx;
  q.c_ld = d.H;
  q.offsets = offsets;
  q.R = R;
  q.N = d.H;
  q.K = 2 * d.I;
  q.E = d.E;
  q.I = d.I;
  q.n_tiles = d.H / gemm::kBN;
  set_tail(q, tail);
  const int64_t mtiles = most_row_tiles(d.E, R, tail);
  return gemm::run(q, gemm::MNCONTIG, gemm::KCONTIG, gemm::GROUP_M, gemm::EPI_STORE, mtiles * q.n_tiles, s,
                   "moe_grouped_mlp_bwd(gate_up dgrad)");
}

// dW_e[m][n] = sum_r a[r][m] b[r][n] over expert e's rows, a [R, M] and b [R, N]
static moe_status bf16_wgrad(const moe_mlp_desc& d, int64_t R, const bf16_t* a, int M, const bf16_t* b, int N,
                             const PtrTab& dw, const int32_t* offsets, hipStream_t s, const char* what) {
  gemm::Params w;
  std::memset(&w, 0, sizeof(w));
  std::memcpy(w.tab, dw.p, sizeof(w.tab));
  w.p = b;
  w.p_ld = N;
  w.q = a;
  w.q_ld = M;
  w.c_ld = N;
  w.offsets = offsets;
  w.R = R;
  w.M = M;
  w.N = N;
  w.E = d.E;
  w.I = d.I;
  w.n_tiles = N / gemm::kBN;
  return gemm::run(w, gemm::MNCONTIG, gemm::MNCONTIG, gemm::GROUP_K, gemm::EPI_STORE,
                   (int64_t)d.E * (M / gemm::kBM) * w.n_tiles, s, what);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_mlp_fwd(const moe_mlp_desc* desc, int64_t R, const void* x_perm,
                                          const uint8_t* x_perm_scale, const void* const* w_gate_up,
                                          const void* const* w_down, const uint8_t* const* w_gate_up_scale,
                                          const uint8_t* const* w_down_scale, const int32_t* offsets,
                                          const float* prob_perm, void* y_perm, void* z_save, void* h_save,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: desc is NULL");
  const moe_mlp_desc d = *desc;
  moe_status st = validate_desc(d, false);
  if (st != MOE_OK) return st;
  if (R < 0 || R > 0x7FFFFFFF) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: R out of [0, 2^31)");
  if (R == 0) return MOE_OK;
  const size_t align = d.compute == MOE_F32 ? 4 : 16;
  if (!x_perm || !offsets || !prob_perm || !y_perm) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: NULL pointer");
  if (!aligned(x_perm, align) || !aligned(y_perm, align))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: x_perm / y_perm misaligned");
  if (d.save_for_bwd) {
    if (!z_save || !h_save) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: save_for_bwd needs z_save and h_save");
    if (!aligned(z_save, align) || !aligned(h_save, align))
      return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: z_save / h_save misaligned");
  }
  if ((st = check_table(w_gate_up, d.E, align, "moe_grouped_mlp_fwd(w_gate_up)")) != MOE_OK) return st;
  if ((st = check_table(w_down, d.E, align, "moe_grouped_mlp_fwd(w_down)")) != MOE_OK) return st;
  if (d.compute == MOE_MXFP8 && d.wt == MOE_MXFP8) {
    if ((st = check_table((const void* const*)w_gate_up_scale, d.E, 4, "moe_grouped_mlp_fwd(w_gate_up_scale)")) != MOE_OK) return st;
    if ((st = check_table((const void* const*)w_down_scale, d.E, 4, "moe_grouped_mlp_fwd(w_down_scale)")) != MOE_OK) return st;
  }
  if (d.compute == MOE_MXFP8 && d.act == MOE_MXFP8 && (!x_perm_scale || !aligned(x_perm_scale, 4)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: MXFP8 activations need a 4-byte aligned x_perm_scale");
  if (d.compute == MOE_FP8 && d.wt == MOE_FP8) {
    if ((st = check_table((const void* const*)w_gate_up_scale, d.E, 4, "moe_grouped_mlp_fwd(w_gate_up_scale)")) != MOE_OK) return st;
    if ((st = check_table((const void* const*)w_down_scale, d.E, 4, "moe_grouped_mlp_fwd(w_down_scale)")) != MOE_OK) return st;
  }
  if (d.compute == MOE_FP8 && d.act == MOE_FP8 && (!x_perm_scale || !aligned(x_perm_scale, 4)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: FP8 activations need a 4-byte aligned x_perm_scale");
  if (d.compute == MOE_MXFP4 && d.wt == MOE_MXFP4) {
    if ((st = check_table((const void* const*)w_gate_up_scale, d.E, 8, "moe_grouped_mlp_fwd(w_gate_up_scale)")) != MOE_OK) return st;
    if ((st = check_table((const void* const*)w_down_scale, d.E, 8, "moe_grouped_mlp_fwd(w_down_scale)")) != MOE_OK) return st;
  }
  if (d.compute == MOE_MXFP4 && d.act == MOE_MXFP4 && (!x_perm_scale || !aligned(x_perm_scale, 8)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: MXFP4 activations need an 8-byte aligned x_perm_scale");
  const size_t need = mlp_fwd_workspace_bytes(d, R);
  if (workspace_bytes < need) return fail(MOE_ERR_WORKSPACE, "moe_grouped_mlp_fwd: workspace too small");
  if (need > 0 && (!workspace || !aligned(workspace, 256)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_fwd: workspace NULL or not 256-byte aligned");
  const hipStream_t s = as_stream(stream);
  const PtrTab w1 = make_tab(w_gate_up, d.E), w2 = make_tab(w_down, d.E);

  if (d.compute == MOE_F32) {
    float* h = d.save_for_bwd ? (float*)h_save : (float*)workspace;
    return f32::forward(d, R, (const float*)x_perm, w1, w2, offsets, prob_perm, (float*)y_perm,
                        d.save_for_bwd ? (float*)z_save : nullptr, h, s);
  }
  if (d.compute == MOE_FP8) {
    return mx::forward_fp8_tensor(d, R, x_perm, reinterpret_cast<const float*>(x_perm_scale), w_gate_up, w_down,
                                  reinterpret_cast<const float* const*>(w_gate_up_scale),
                                  reinterpret_cast<const float* const*>(w_down_scale), offsets, prob_perm, y_perm,
                                  (uint8_t*)workspace, s, d.save_for_bwd ? z_save : nullptr,
                                  d.save_for_bwd ? h_save : nullptr);
  }
  if (d.compute == MOE_MXFP4)
    return mx4::forward(d, R, x_perm, x_perm_scale, w_gate_up, w_down, w_gate_up_scale, w_down_scale, offsets, prob_perm,
                        y_perm, (uint8_t*)workspace, s);
  if (d.compute == MOE_MXFP8) {
    return mx::forward(d, R, x_perm, x_perm_scale, w_gate_up, w_down, w_gate_up_scale, w_down_scale, offsets,
                       prob_perm, y_perm, (uint8_t*)workspace, s, d.save_for_bwd ? z_save : nullptr,
                       d.save_for_bwd ? h_save : nullptr);
  }

  // bf16: gate_up + ScaledSwiGLU (h, optionally z), then down; workspace: [h] [tail area]
  bf16_t* h = d.save_for_bwd ? (bf16_t*)h_save : (bf16_t*)workspace;
  const TailArea tail = tail_area((uint8_t*)workspace + (d.save_for_bwd ? 0 : a256((size_t)R * d.I * 2)));
  st = bf16_gate_up(d.E, R, d.H, d.I, (const bf16_t*)x_perm, w1, offsets, prob_perm, h,
                    d.save_for_bwd ? (bf16_t*)z_save : nullptr, s, tail);
  if (st != MOE_OK) return st;
  return bf16_linear(d.E, R, d.I, d.H, h, w2, offsets, (bf16_t*)y_perm, s, tail);
}

// the tail area of a caller's grouped-GEMM workspace (none if it is NULL); validated
static moe_status gemm_workspace(void* ws, size_t bytes, const char* what, TailArea* out) {
  *out = TailArea();
  if (!ws) return MOE_OK;
  if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, std::string(what) + ": workspace not 256-byte aligned");
  if (bytes < grouped_gemm_workspace_bytes()) return fail(MOE_ERR_WORKSPACE, std::string(what) + ": workspace too small");
  *out = tail_area((uint8_t*)ws);
  return MOE_OK;
}

extern "C" moe_status moe_grouped_linear(int E, int64_t R, int K, int N, moe_dtype dt, const void* x,
                                         const void* const* w, const int32_t* offsets, void* y, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_linear: E out of [1, 256]");
  if (R < 0 || R > 0x7FFFFFFF || K < 1 || N < 1) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_linear: bad R/K/N");
  if (dt != MOE_BF16 && dt != MOE_F32) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_linear: dtype must be BF16 or F32");
  if (dt == MOE_BF16 && (N % 256 != 0 || K % 64 != 0))
    return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_linear: bf16 needs N % 256 == 0 and K % 64 == 0");
  if ((int64_t)N * K * 2 > 0x7FFFFFFFLL) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_linear: weight exceeds 2^31 bytes");
  if (R == 0) return MOE_OK;
  const size_t align = dt == MOE_F32 ? 4 : 16;
  if (!x || !y || !offsets) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_linear: NULL pointer");
  if (!aligned(x, align) || !aligned(y, align)) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_linear: misaligned tensor");
  moe_status st = check_table(w, E, align, "moe_grouped_linear(w)");
  if (st != MOE_OK) return st;
  const PtrTab tab = make_tab(w, E);
  const hipStream_t s = as_stream(stream);
  if (dt == MOE_F32) return f32::linear(E, R, K, N, (const float*)x, tab, offsets, (float*)y, s);
  TailArea tail;
  if ((st = gemm_workspace(workspace, workspace_bytes, "moe_grouped_linear", &tail)) != MOE_OK) return st;
  return bf16_linear(E, R, K, N, (const bf16_t*)x, tab, offsets, (bf16_t*)y, s, tail);
}

extern "C" moe_status moe_grouped_gate_up_swiglu(int E, int64_t R, int H, int I, moe_dtype dt, const void* x,
                                                 const uint8_t* x_scale, const void* const* w,
                                                 const uint8_t* const* w_scale, const int32_t* offsets,
                                                 const float* prob, void* h, uint8_t* h_scale, void* z_save,
                                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: E out of [1, 256]");
  if (R < 0 || R > 0x7FFFFFFF || H < 1 || I < 1) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: bad R/H/I");
  if (dt != MOE_BF16 && dt != MOE_F32 && dt != MOE_MXFP8)
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: bad dtype");
  if (dt != MOE_F32 && (H % 256 != 0 || I % 128 != 0))
    return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gate_up_swiglu: needs H % 256 == 0 and I % 128 == 0");
  if ((int64_t)2 * I * H * 2 > 0x7FFFFFFFLL) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gate_up_swiglu: weight exceeds 2^31 bytes");
  if (dt == MOE_MXFP8 && z_save) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: z_save needs BF16 or F32");
  if (R == 0) return MOE_OK;
  const size_t align = dt == MOE_F32 ? 4 : 16;
  if (!x || !h || !offsets || !prob) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: NULL pointer");
  if (!aligned(x, align) || !aligned(h, align) || (z_save && !aligned(z_save, align)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: misaligned tensor");
  moe_status st = check_table(w, E, align, "moe_grouped_gate_up_swiglu(w)");
  if (st != MOE_OK) return st;
  const hipStream_t s = as_stream(stream);
  const PtrTab tab = make_tab(w, E);
  if (dt == MOE_MXFP8) {
    if (!x_scale || !h_scale) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_gate_up_swiglu: MXFP8 needs x_scale and h_scale");
    if ((st = check_table((const void* const*)w_scale, E, 4, "moe_grouped_gate_up_swiglu(w_scale)")) != MOE_OK) return st;
    return mx::gate_up(E, R, H, I, (const uint8_t*)x, x_scale, w, w_scale, offsets, prob, (uint8_t*)h, h_scale, s);
  }
  if (dt == MOE_F32)
    return f32::gate_up(E, R, H, I, (const float*)x, tab, offsets, prob, (float*)h, (float*)z_save, s);
  TailArea tail;
  if ((st = gemm_workspace(workspace, workspace_bytes, "moe_grouped_gate_up_swiglu", &tail)) != MOE_OK) return st;
  return bf16_gate_up(E, R, H, I, (const bf16_t*)x, tab, offsets, prob, (bf16_t*)h, (bf16_t*)z_save, s, tail);
}

extern "C" moe_status moe_grouped_mlp_bwd(const moe_mlp_desc* desc, int64_t R, const void* dy_perm,
                                          const void* x_perm, const void* z_save, const void* h_save,
                                          const float* prob_perm, const void* const* w_gate_up,
                                          const void* const* w_down, const int32_t* offsets, void* dx_perm,
                                          void* const* dw_gate_up, void* const* dw_down, float* dprob_perm,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: desc is NULL");
  const moe_mlp_desc d = *desc;
  moe_status st = validate_desc(d, true);
  if (st != MOE_OK) return st;
  if (R < 0 || R > 0x7FFFFFFF) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: R out of [0, 2^31)");
  const size_t align = d.compute == MOE_F32 ? 4 : 16;
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: offsets is NULL");
  if (R > 0) {
    if (!dy_perm || !x_perm || !z_save || !h_save || !prob_perm || !dx_perm || !dprob_perm)
      return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: NULL pointer");
    for (const void* ptr : {dy_perm, x_perm, z_save, h_save, (const void*)dx_perm})
      if (!aligned(ptr, align)) return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: misaligned tensor");
  }
  if ((st = check_table(w_gate_up, d.E, align, "moe_grouped_mlp_bwd(w_gate_up)")) != MOE_OK) return st;
  if ((st = check_table(w_down, d.E, align, "moe_grouped_mlp_bwd(w_down)")) != MOE_OK) return st;
  if ((st = check_table((const void* const*)dw_gate_up, d.E, align, "moe_grouped_mlp_bwd(dw_gate_up)")) != MOE_OK) return st;
  if ((st = check_table((const void* const*)dw_down, d.E, align, "moe_grouped_mlp_bwd(dw_down)")) != MOE_OK) return st;
  const size_t need = mlp_bwd_workspace_bytes(d, R);
  if (workspace_bytes < need) return fail(MOE_ERR_WORKSPACE, "moe_grouped_mlp_bwd: workspace too small");
  if (need > 0 && (!workspace || !aligned(workspace, 256)))
    return fail(MOE_ERR_INVALID_ARG, "moe_grouped_mlp_bwd: workspace NULL or not 256-byte aligned");
  const hipStream_t s = as_stream(stream);
  const PtrTab w1 = make_tab(w_gate_up, d.E), w2 = make_tab(w_down, d.E);
  const PtrTab dw1 = make_tab((const void* const*)dw_gate_up, d.E), dw2 = make_tab((const void* const*)dw_down, d.E);

  if (d.compute == MOE_F32) {
    return f32::backward(d, R, (const float*)dy_perm, (const float*)x_perm, (const float*)z_save,
                         (const float*)h_save, prob_perm, w1, w2, offsets, (float*)dx_perm, dw1, dw2, dprob_perm,
                         (float*)workspace, s);
  }

  if (d.compute == MOE_MXFP8) {
    return mx::backward(d, R, (const bf16_t*)dy_perm, (const bf16_t*)x_perm, (const bf16_t*)z_save,
                        (const bf16_t*)h_save, prob_perm, w_gate_up, w_down, offsets, (bf16_t*)dx_perm, dw_gate_up,
                        dw_down, dprob_perm, (uint8_t*)workspace, s);
  }
  if (d.compute == MOE_FP8) {
    return mx::backward_fp8_tensor(d, R, (const bf16_t*)dy_perm, (const bf16_t*)x_perm, (const bf16_t*)z_save,
                                   (const bf16_t*)h_save, prob_perm, w_gate_up, w_down, offsets, (bf16_t*)dx_perm,
                                   dw_gate_up, dw_down, dprob_perm, (uint8_t*)workspace, s);
  }

  uint8_t* ws = (uint8_t*)workspace;
  bf16_t* dz = (bf16_t*)ws;
  ws += a256((size_t)R * 2 * d.I * 2);
  float* part = (float*)ws;
  ws += a256((size_t)2 * (d.I / 256) * R * 4);
  const TailArea tail = tail_area(ws);  // split-K tail of the gate_up dgrad
  if (R > 0) {
    if ((st = bf16_down_dgrad(d, R, (const bf16_t*)dy_perm, w2, offsets, prob_perm, (const bf16_t*)z_save, dz, part,
                              dprob_perm, s)) != MOE_OK)
      return st;
    if ((st = bf16_gate_up_dgrad(d, R, dz, w1, offsets, (bf16_t*)dx_perm, tail, s)) != MOE_OK) return st;
  }
  st = bf16_wgrad(d, R, (const bf16_t*)dy_perm, d.H, (const bf16_t*)h_save, d.I, dw2, offsets, s,
                  "moe_grouped_mlp_bwd(down wgrad)");
  if (st != MOE_OK) return st;
  return bf16_wgrad(d, R, dz, 2 * d.I, (const bf16_t*)x_perm, d.H, dw1, offsets, s, "moe_grouped_mlp_bwd(gate_up wgrad)");
}

extern "C" moe_status moe_grouped_mlp_fwd_ckpt8(const moe_mlp_desc* desc, int64_t R, const void* x_perm,
                                                const void* const* w_gate_up, const void* const* w_down,
                                                const int32_t* offsets, const float* prob_perm, void* y_perm,
                                                uint8_t* z_codes, uint8_t* z_scales, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_mlp_fwd_ckpt8";
  if (!desc) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": desc is NULL");
  moe_mlp_desc d = *desc;
  d.save_for_bwd = 0;
  moe_status st = validate_ckpt8(d, false, fn);
  if (st != MOE_OK) return st;
  if (R < 0 || R > 0x7FFFFFFF) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": R out of [0, 2^31)");
  if (R == 0) return MOE_OK;
  if (!x_perm || !offsets || !prob_perm || !y_perm || !z_codes || !z_scales)
    return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
  if (!aligned(x_perm, 16) || !aligned(y_perm, 16) || !aligned(z_codes, 16) || !aligned(z_scales, 4) ||
      !aligned(offsets, 4) || !aligned(prob_perm, 4))
    return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": misaligned tensor");
  if ((st = check_table(w_gate_up, d.E, 16, "moe_grouped_mlp_fwd_ckpt8(w_gate_up)")) != MOE_OK) return st;
  if ((st = check_table(w_down, d.E, 16, "moe_grouped_mlp_fwd_ckpt8(w_down)")) != MOE_OK) return st;
  if (workspace_bytes < mlp_fwd_workspace_bytes(d, R))
    return fail(MOE_ERR_WORKSPACE, std::string(fn) + ": workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": workspace NULL or not 256-byte aligned");
  const hipStream_t s = as_stream(stream);
  bf16_t* h = (bf16_t*)workspace;
  const TailArea tail = tail_area((uint8_t*)workspace + a256((size_t)R * d.I * 2));
  st = bf16_gate_up(d.E, R, d.H, d.I, (const bf16_t*)x_perm, make_tab(w_gate_up, d.E), offsets, prob_perm, h, nullptr, s,
                    tail_for(tail, d.E, R, d.H, d.I / 128, true), z_codes, z_scales);
  if (st != MOE_OK) return st;
  return bf16_linear(d.E, R, d.I, d.H, h, make_tab(w_down, d.E), offsets, (bf16_t*)y_perm, s,
                     tail_for(tail, d.E, R, d.I, d.H / gemm::kBN, false));
}

extern "C" moe_status moe_grouped_mlp_bwd_ckpt8(const moe_mlp_desc* desc, int64_t R, const void* dy_perm, const void* x,
                                                const uint8_t* x_scale, int64_t T, const int32_t* src_token,
                                                const uint8_t* z_codes, const uint8_t* z_scales, const float* prob_perm,
                                                const void* const* w_gate_up, const void* const* w_down,
                                                const int32_t* offsets, void* dx_perm, void* const* dw_gate_up,
                                                void* const* dw_down, float* dprob_perm, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_mlp_bwd_ckpt8";
  if (!desc) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": desc is NULL");
  const moe_mlp_desc d = *desc;
  moe_status st = validate_ckpt8(d, true, fn);
  if (st != MOE_OK) return st;
  if (R < 0 || R > 0x7FFFFFFF) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": R out of [0, 2^31)");
  const bool kept8 = d.act == MOE_MXFP8;
  if (!offsets || !aligned(offsets, 4)) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": offsets NULL or misaligned");
  if (R > 0) {
    const bool has_x = x && (!kept8 || x_scale);
    if (!dy_perm || !z_codes || !z_scales || !prob_perm || !dx_perm || !dprob_perm || (!has_x && (!kept8 || T > 0)))
      return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    for (const void* p : {dy_perm, x, (const void*)z_codes, (const void*)dx_perm})
      if (!aligned(p, 16)) return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": misaligned tensor");
    if (!aligned(z_scales, 8) || !aligned(prob_perm, 4) || !aligned(dprob_perm, 4) || !aligned(src_token, 4))
      return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": z_scales must be 8-byte, prob, dprob and src_token 4-byte aligned");
    if (kept8 && (T < 0 || T > 0x7FFFFFFF || (!src_token && T != R)))
      return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": T out of [0, 2^31), or T != R without src_token");
    if (!kept8 && (x_scale || src_token))
      return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": x_scale and src_token belong to act = MOE_MXFP8");
  }
  if ((st = check_table(w_gate_up, d.E, 16, "moe_grouped_mlp_bwd_ckpt8(w_gate_up)")) != MOE_OK) return st;
  if ((st = check_table(w_down, d.E, 16, "moe_grouped_mlp_bwd_ckpt8(w_down)")) != MOE_OK) return st;
  if ((st = check_table((const void* const*)dw_gate_up, d.E, 16, "moe_grouped_mlp_bwd_ckpt8(dw_gate_up)")) != MOE_OK) return st;
  if ((st = check_table((const void* const*)dw_down, d.E, 16, "moe_grouped_mlp_bwd_ckpt8(dw_down)")) != MOE_OK) return st;
  if (workspace_bytes < mlp_bwd_ckpt8_workspace_bytes(d, R))
    return fail(MOE_ERR_WORKSPACE, std::string(fn) + ": workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return fail(MOE_ERR_INVALID_ARG, std::string(fn) + ": workspace NULL or not 256-byte aligned");
  const hipStream_t s = as_stream(stream);
  const PtrTab w1 = make_tab(w_gate_up, d.E), w2 = make_tab(w_down, d.E);
  const PtrTab dw1 = make_tab((const void* const*)dw_gate_up, d.E), dw2 = make_tab((const void* const*)dw_down, d.E);

  uint8_t* ws = (uint8_t*)workspace;
  bf16_t* dz = (bf16_t*)ws;
  ws += a256((size_t)R * 2 * d.I * 2);
  bf16_t* rows = (bf16_t*)ws;  // h until its weight gradient is done, then x in expert order
  ws += ckpt8_rows_bytes(d, R);
  float* part = (float*)ws;
  ws += a256((size_t)2 * (d.I / 256) * R * 4);
  const TailArea tail = tail_area(ws);
  if (R > 0) {
    st = bf16_down_dgrad(d, R, (const bf16_t*)dy_perm, w2, offsets, prob_perm, nullptr, dz, part, dprob_perm, s, z_codes,
                         z_scales, rows, tail_for(tail, d.E, R, d.H, d.I / gemm::kBN, true));
    if (st != MOE_OK) return st;
    st = bf16_gate_up_dgrad(d, R, dz, w1, offsets, (bf16_t*)dx_perm, tail_for(tail, d.E, R, 2 * d.I, d.H / gemm::kBN, false), s);
    if (st != MOE_OK) return st;
  }
  st = bf16_wgrad(d, R, (const bf16_t*)dy_perm, d.H, rows, d.I, dw2, offsets, s, "moe_grouped_mlp_bwd_ckpt8(down wgrad)");
  if (st != MOE_OK) return st;
  const bf16_t* xp = (const bf16_t*)x;
  if (kept8) {
    if (R > 0) {
      st = mx8::launch_read((const uint8_t*)x, x_scale, T, d.H, src_token, R, offsets, d.E, true, rows, s);
      if (st != MOE_OK) return st;
    }
    xp = rows;
  }
  return bf16_wgrad(d, R, dz, 2 * d.I, xp, d.H, dw1, offsets, s, "moe_grouped_mlp_bwd_ckpt8(gate_up wgrad)");
}
