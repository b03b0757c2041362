// Parameters of the persistent grouped GEMM kernels (bf16 MFMA).
#pragma once

#include <string>

#include "common.h"

namespace moe {
namespace gemm {

constexpr int kBM = 256, kBN = 256, kBK = 32;
constexpr int kStages = 4;                    // LDS ring depth
constexpr int kTileBytes = 256 * kBK * 2;     // one operand, one stage (16 KiB)
constexpr int kStageBytes = 2 * kTileBytes;   // P and Q
constexpr int kLdsBytes = kStages * kStageBytes;

enum { KCONTIG = 0, MNCONTIG = 1 };
enum { GROUP_M = 0, GROUP_K = 1 };
enum {
  EPI_STORE = 0,
  EPI_SWIGLU = 1,
  EPI_DSWIGLU = 2,
  EPI_SWIGLU_MX8 = 3,  // SWIGLU that also writes the gate_up output in MXFP8
  EPI_DSWIGLU_MX8 = 4  // DSWIGLU from a gate_up output in MXFP8, which also writes h
};
constexpr bool is_swiglu(int ep) { return ep == EPI_SWIGLU || ep == EPI_SWIGLU_MX8; }
// epilogues of the general kernel (rows grouped by expert) whose last tiles may be split along K
constexpr bool can_split(int ep) { return ep == EPI_STORE || ep == EPI_DSWIGLU_MX8; }

struct Params {
  // GROUP_M: per-expert P operand (weights). GROUP_K: per-expert output C.
  const void* tab[MOE_MAX_EXPERTS];
  const bf16_t* p;        // P operand when it is a token tensor (GROUP_K)
  const bf16_t* q;        // Q operand (token rows)
  bf16_t* c;              // output (GROUP_M)
  const int32_t* offsets; // [E+1] expert row offsets
  const float* prob;      // SWIGLU / DSWIGLU (and their MX8 forms): routing weight per row
  const bf16_t* zin;      // DSWIGLU: saved gate_up output [R, 2I]
  bf16_t* zout;           // SWIGLU: gate_up output to save [R, 2I] (or NULL)
  float* part;            // DSWIGLU, DSWIGLU_MX8: dprob partial sums [2 * n_tiles][R]
  int64_t p_ld, q_ld, c_ld;
  int64_t R;
  int M, N, K;            // GROUP_M uses N, K; GROUP_K uses M, N
  int E, I;
  int n_tiles;            // output column tiles (SWIGLU, SWIGLU_MX8: I / 128, else N / 256)
  // split-K tail (forward kernel): when the last round of tiles would leave at least
  // half the CUs idle, its tiles are cut into K chunks whose float32 partial tiles go
  // to `tail` (tail_cap of them at most; 0 = never split) and are finished by
  // run_tail_reduce; tail_meta holds [n_tail, split, first_tail, 0] then per tail
  // tile [first_row, row_end, column_tile, 0].
  float* tail;
  int32_t* tail_meta;
  int tail_cap;
  int spread;    // 1, with a tail: one workgroup per CU also where there are fewer tiles, so that those are
                 // split; 2 (set by the launch): so few that all are tail tiles, which the tail launch lists
  uint8_t* z8;   // E4M3 codes of the gate_up output [R, 2I] (SWIGLU_MX8: out, DSWIGLU_MX8: in)
  uint8_t* z8s;  // ... and its E8M0 scales [R, 2I / 32]
  bf16_t* hout;  // DSWIGLU_MX8: h [R, I]
};

constexpr size_t kTailTileBytes = (size_t)kBM * kBN * 4;  // one float32 partial tile
constexpr size_t kTailMetaSpace = 8192;                   // header + up to 511 tail tiles
// bytes of a split-K tail area (meta, then `units` partial tiles)
inline size_t tail_ws_bytes(int units) { return kTailMetaSpace + (size_t)units * kTailTileBytes; }

// workgroups of a launch over at most max_tiles tiles
inline int64_t grid_size(const Params& p, int64_t max_tiles, int cus) {
  return (p.spread && p.tail_cap > 0) || max_tiles > cus ? cus : max_tiles;
}

// whether a spread launch's tiles are all tail tiles, whatever the offsets: at most half a round of them,
// cut into two chunks or more
inline bool all_tail(const Params& p, int64_t max_tiles, int cus) {
  return p.spread && p.tail_cap >= cus && max_tiles * 2 <= cus && p.K >= 128;
}

moe_status run(const Params& p, int pl, int ql, int g, int ep, int64_t max_tiles, hipStream_t s,
               const char* what);
// forward kernel (gemm_fwd.hip): GROUP_M, both operands KCONTIG, EPI_STORE, EPI_SWIGLU or
// EPI_SWIGLU_MX8, K a multiple of 64
moe_status run_fwd(const Params& p, int ep, int64_t max_tiles, hipStream_t s, const char* what);
// sums the split-K partial tiles that run_fwd left in p.tail and applies the epilogue
moe_status run_tail_reduce(const Params& p, int ep, int64_t max_tiles, hipStream_t s, const char* what);

}  // namespace gemm
}  // namespace moe
