// MXFP4 grouped GEMM for many rows an expert: 256 x 256 tiles on v_mfma_scale_f32_32x32x64
// (E2M1 operands), bound by the MFMA.
//
// Lane l of that MFMA holds 32 consecutive K values (16 bytes) of row l % 32, K half l / 32
// of 64, and their block's scale. A K step is 256 values in four slices of 64. A wavefront
// takes 64 rows x 256 columns of the tile (2 x 8 MFMAs a slice), so each row's codes are
// needed by one wavefront only and each weight's by all four:
//   weights (P): one 128-byte line of each of the 256 weight rows a step, by range-checked
//     buffer copies into a ring of four 32 KiB LDS slots, three steps ahead;
//   rows (Q): straight from memory into registers, two steps ahead, from codes laid out in
//     the MFMA's own order (frag_rows below: a fragment is 1 KiB in a row), so that half of
//     the operand bytes need neither LDS nor a barrier.
// What bounds it is the card's power. A step is 64 MFMAs a SIMD; with random operands the card
// lowers its clock, and the MFMAs alone take 1.34 us a step with every operand in registers
// (6.4 PFLOP/s) and 1.48 with half of them read from LDS (5.8; all zeros: 8.9). The loop here
// runs at 1.65 us a step, its clock at 1.8 to 1.9 GHz. 16384 rows, 8 experts of 4096 x 14336:
// 950 us gate_up with SwiGLU, 485 down; both operands in LDS: 1045 and 500; 128 x 256 tiles, two
// workgroups a CU: 1273 and 834 (half-line copies, more traffic); workgroups started apart in
// time: within 2%.
// Besides: the epilogue, in which no MFMA runs (one workgroup a CU, one wavefront a SIMD), about a
// fifth of that gate_up's time and most of a product of three steps'; and the last round of tiles
// (1088 tiles of that down product are 4.25 rounds of 256 CUs and take five).
// The next tile's first loads are issued within a tile's epilogue, ahead of its stores or, with
// SwiGLU, between the blocks of its arithmetic. (STORE: the compiler, which cannot tell sOut from
// the slots being copied to, waits for the copies before the epilogue's first LDS store.)
//
// The K loop runs all but the last three steps in groups of four and RES more, so every ring
// slot is a constant; the last three issue no copies (an expert's product of fewer than three
// steps runs empty ones: zero weights). Waits count this wavefront's memory operations, which
// complete in order; the counts are those of the steps' fixed numbers of loads.
//
// Scales come in the lane order of the MFMA: word ((step * rows + row) * 2 + g) holds, in
// byte s, the scale of block 2s + g of the row's step, so a lane's one word serves its four
// slices, the byte picked by the instruction.
#include <cstring>
#include <type_traits>

#include "common.h"
#include "gemm_common.h"
#include "internal.h"
#include "lanes.h"
#include "mxfp4.h"

namespace moe {
namespace mx4 {

using namespace gemm;

namespace {

constexpr int kBM = 256, kBN = 256, kStep = 256;
constexpr int kRowBytes = kStep / 2;     // of a row, a step
constexpr int kSlot = kBN * kRowBytes;   // the weights of one step
constexpr int kRing = 4;
constexpr int kDrain = 3;                // steps at the end without copies

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t wide(i32x4_t v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The lane, computed where it is used: values made from it are not kept (or spilled: a reload
// would wait for every load and store before it) across the K loop.
__device__ __forceinline__ int fresh_lane() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

template <int EP, int RES>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
void grouped_gemm_tile_kernel(const Params prm) {
  __shared__ __attribute__((aligned(1024))) uint8_t sP0[kSlot], sP1[kSlot], sP2[kSlot], sP3[kSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t sOut[kSlot];  // STORE: 8 KiB of output a wavefront
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, lhi = lane >> 5;
  const int E = prm.E, R = (int)prm.R;
  const int ld = prm.K / 2;          // bytes of a code row
  const int nk = prm.K / kStep;
  const int n_run = nk < kDrain ? kDrain : nk;
  const int n_tiles = prm.n_tiles;
  const int nwg = gridDim.x;

  auto slot = [&](auto V) -> uint8_t* {
    if constexpr (V.value % kRing == 0) return sP0;
    else if constexpr (V.value % kRing == 1) return sP1;
    else if constexpr (V.value % kRing == 2) return sP2;
    else return sP3;
  };

  // ---------------- tiles ----------------
  // expert-major, row tiles in groups of at most 16 (tile_in_expert). Lane l holds experts l and
  // l + 64: their rows (offsets made a nondecreasing sequence inside [0, R]) and first tile, so
  // a tile is found without a memory access.
  struct Span {
    int beg, end, first;
  } span[2];
  int total = 0;
  for (int h = 0, rows_before = min(max(prm.offsets[0], 0), R); h < 2; ++h) {
    const int e = h * 64 + lane;
    int end = min(max(e < E ? prm.offsets[e + 1] : 0, rows_before), R);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(end, d, 64);
      if (lane >= d) end = max(end, o);
    }
    int beg = __shfl_up(end, 1, 64);
    if (lane == 0) beg = rows_before;
    const int tiles = e < E ? (end - beg + kBM - 1) / kBM * n_tiles : 0;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    span[h] = Span{beg, end, total + upto - tiles};
    rows_before = __builtin_amdgcn_readlane(end, 63);
    total += __builtin_amdgcn_readlane(upto, 63);
  }
  struct Tile {
    int e, nt, row, row_end;
  };
  auto find_tile = [&](int t, Tile& tile) -> bool {
    if (t >= total) return false;
    // of experts that start at one tile only the last has any
    const int e = __popcll(__ballot(lane < E && span[0].first <= t)) + __popcll(__ballot(lane + 64 < E && span[1].first <= t)) - 1;
    const bool up = e >= 64;
    const int beg = __builtin_amdgcn_readlane(up ? span[1].beg : span[0].beg, e & 63);
    const int end = __builtin_amdgcn_readlane(up ? span[1].end : span[0].end, e & 63);
    const int first = __builtin_amdgcn_readlane(up ? span[1].first : span[0].first, e & 63);
    int mt, nt;
    tile_in_expert(t - first, (end - beg + kBM - 1) / kBM, n_tiles, mt, nt);
    tile = Tile{e, __builtin_amdgcn_readfirstlane(nt), __builtin_amdgcn_readfirstlane(beg + mt * kBM), end};
    return true;
  };

  // ---------------- operands of a tile ----------------
  // first weight row (SWIGLU: 128 gate rows, then, p_up rows further, the up rows of the same columns)
  constexpr int kTileCols = EP == EP_SWIGLU ? 128 : kBN;
  const int p_up = EP == EP_SWIGLU ? prm.I - 128 : 0;
  const int kc_row0 = wave * 8 + (lane >> 3);  // copies: round i fills rows 32 i + kc_row0 of a slot
  const uint32_t p_off = (uint32_t)(kc_row0 * ld + ((lane & 7) ^ swz8(kc_row0)) * 16);
  const uint32_t ps_off = (uint32_t)((l32 * 2 + lhi) * 4);
  const int slices = prm.K / 64;
  const uint8_t *p_tile, *ps_tile, *q_tile, *qs_tile;
  uint32_t q_off[2], qs_off[2];
  auto set_tile = [&](const Tile& t) {
    p_tile = prm.tab[t.e] + (int64_t)t.nt * kTileCols * ld;
    ps_tile = prm.tab_s[t.e] + (int64_t)t.nt * kTileCols * 8;
    q_tile = prm.q + (int64_t)(t.row >> 5) * slices * 1024;
    qs_tile = prm.q_s + (int64_t)t.row * 8;
    const int ln = fresh_lane(), n32 = ln & 31, nhi = ln >> 5;
#pragma unroll
    for (int sm = 0; sm < 2; ++sm) {  // rows past the expert: another's, their products are discarded
      const int row = min(t.row + wave * 64 + sm * 32 + n32, R - 1);
      q_off[sm] = (uint32_t)(((row >> 5) - (t.row >> 5)) * slices * 1024 + nhi * 512 + (row & 31) * 16);
      qs_off[sm] = (uint32_t)(((row - t.row) * 2 + nhi) * 4);
    }
  };
  // rounds [I0, I0 + N) of step kt's weights; nrec: the range, 0 (zeros) past the last step
  auto copy_P = [&](int kt, auto V, auto I0, auto N, uint32_t nrec = 0xFFFFFFFFu) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p_tile + (int64_t)kt * kRowBytes), (short)0, (int)nrec, kBufferFlags);
#pragma unroll
    for (int i = decltype(I0)::value; i < decltype(I0)::value + decltype(N)::value; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(slot(V) + wave * 1024 + i * 4096), 16, p_off,
                                               (int)((uint32_t)(i * 32 + (i >= 4 ? p_up : 0)) * (uint32_t)ld), 0, 0);
  };
  i32x4_t q[2][4][2];  // [step parity][slice][row sub-tile]
  auto load_Q = [&](int kt, auto PAR, auto S) {
    constexpr int par = decltype(PAR)::value & 1, s = decltype(S)::value;
    kt = kt < nk ? kt : nk - 1;
    const uint8_t* base = q_tile + (int64_t)kt * 4096 + s * 1024;
#pragma unroll
    for (int sm = 0; sm < 2; ++sm) q[par][s][sm] = *reinterpret_cast<const i32x4_t*>(base + q_off[sm]);
  };
  struct Scales {
    uint32_t p[8], q[2];
  };
  auto load_scales = [&](int kt, Scales& w) {
    kt = kt < nk ? kt : nk - 1;
    const uint8_t* ps = ps_tile + (int64_t)kt * prm.N * 8;
    const uint8_t* qs = qs_tile + (int64_t)kt * R * 8;
    uint32_t po = ps_off;
    asm volatile("" : "+v"(po));  // one 32-bit offset, not a 64-bit one kept for every call
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w.p[j] = *reinterpret_cast<const uint32_t*>(ps + (j * 32 + (j >= 4 ? p_up : 0)) * 8 + po);
#pragma unroll
    for (int j = 0; j < 2; ++j) w.q[j] = *reinterpret_cast<const uint32_t*>(qs + qs_off[j]);
  };

  // ---------------- multiplication ----------------
  const uint32_t frag = (uint32_t)(l32 * kRowBytes);
  uint32_t ck[4];  // chunk 2s + lhi of a weight row for slice s, at its swizzled place
#pragma unroll
  for (int c = 0; c < 4; ++c) ck[c] = (uint32_t)(((2 * c + lhi) ^ swz8(l32)) << 4);
  f32x16 acc[8][2];
  i32x4_t fa[8];
  auto read_p = [&](auto V, int s, int sn) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(slot(V) + frag + sn * 32 * kRowBytes + ck[s]);
  };
  // slice S; fa[sn] is refilled from slice s_next of slot Vn as soon as its MFMAs are issued
  auto mfma_slice = [&](const i32x4_t* fb, const Scales& sc, auto S, auto Vn, int s_next) {
    constexpr int s = decltype(S)::value;
#pragma unroll
    for (int sn = 0; sn < 8; ++sn) {
#pragma unroll
      for (int sm = 0; sm < 2; ++sm)
        acc[sn][sm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fa[sn]), wide(fb[sm]), acc[sn][sm], 4, 4, s,
                                                                        (int)sc.p[sn], s, (int)sc.q[sm]);
      fa[sn] = read_p(Vn, s_next, sn);
    }
  };
  // 16 MFMAs with the 8 fragment reads and NL memory loads between them
  auto interleave = [&](auto NL) {
    constexpr int nl = decltype(NL)::value;
    static_for<8>([&](auto I) {
      constexpr int i = decltype(I)::value;
      __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if constexpr (i < nl) __builtin_amdgcn_sched_group_barrier(0x020, i + 8 < nl ? 2 : 1, 0);
    });
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  using C4 = std::integral_constant<int, 4>;
  using C6 = std::integral_constant<int, 6>;
  using C5 = std::integral_constant<int, 5>;
  using C7 = std::integral_constant<int, 7>;
  using C8 = std::integral_constant<int, 8>;
  using C12 = std::integral_constant<int, 12>;
  Scales r0, r1, r2;  // of steps kt, kt + 1, kt + 2
  // Step kt in slot V; MODE 0: copies of P three steps and loads of Q and scales two steps
  // ahead; 1, 2, 3: the last three steps, which have only the loads that are still to come.
  // The barrier ahead of the last slice publishes the next step's weights: copied two steps
  // ago, before at least `after` younger operations of this wavefront.
  auto kstep = [&](int kt, auto V, auto MODE) {
    constexpr int mode = decltype(MODE)::value;
    constexpr int v = decltype(V)::value, par = v & 1;
    using Vn = std::integral_constant<int, v + 1>;
    using Vc = std::integral_constant<int, v + 3>;
    if constexpr (mode == 0) copy_P(kt + 3, Vc{}, C0{}, C4{});
    if constexpr (mode <= 2) load_Q(kt + 1, Vn{}, C3{});
    mfma_slice(q[par][0], r0, C0{}, V, 1);
    interleave(std::integral_constant<int, mode == 0 ? 6 : (mode <= 2 ? 2 : 0)>{});
    if constexpr (mode == 0) copy_P(kt + 3, Vc{}, C4{}, C4{});
    if constexpr (mode <= 1) load_Q(kt + 2, V, C0{});
    mfma_slice(q[par][1], r0, C1{}, V, 2);
    interleave(std::integral_constant<int, mode == 0 ? 6 : (mode == 1 ? 2 : 0)>{});
    if constexpr (mode <= 1) {
      load_scales(kt + 2, r2);
      load_Q(kt + 2, V, C1{});
    }
    mfma_slice(q[par][2], r0, C2{}, V, 3);
    interleave(std::integral_constant<int, mode <= 1 ? 12 : 0>{});
    if constexpr (mode <= 2) {
      wait_vm<mode == 0 ? 52 : (mode == 1 ? 44 : 20)>();
      lds_barrier();
    }
    if constexpr (mode <= 1) load_Q(kt + 2, V, C2{});
    mfma_slice(q[par][3], r0, C3{}, Vn{}, 0);  // (the last step: a stale fragment, never used)
    interleave(std::integral_constant<int, mode <= 1 ? 2 : 0>{});
    r0 = r1;
    r1 = r2;
  };
  // a tile's first loads, in seven parts (a product may have fewer than three steps)
  auto range = [&](int kt) {
    asm volatile("" : "+s"(kt));  // compared here: made ahead of the tiles' loop, the result was spilled
    return (uint32_t)__builtin_amdgcn_readfirstlane(kt < nk ? -1 : 0);
  };
  auto first_loads = [&](auto I) {
    constexpr int i = decltype(I)::value;
    if constexpr (i == 0) load_scales(0, r0);
    if constexpr (i == 1) copy_P(0, C0{}, C0{}, C8{}, range(0));
    if constexpr (i == 2) static_for<4>([&](auto S) { load_Q(0, C0{}, S); });
    if constexpr (i == 3) copy_P(1, C1{}, C0{}, C8{}, range(1));
    if constexpr (i == 4) load_scales(1, r1);
    if constexpr (i == 5) copy_P(2, C2{}, C0{}, C8{}, range(2));
    if constexpr (i == 6) static_for<3>([&](auto S) { load_Q(1, C1{}, S); });
  };
  // parts [A, B), in that order among the operations around them
  auto parts = [&](auto A, auto B) {
    static_for<decltype(B)::value - decltype(A)::value>([&](auto I) {
      first_loads(std::integral_constant<int, decltype(A)::value + decltype(I)::value>{});
    });
    __builtin_amdgcn_sched_barrier(0);
  };

  Tile cur;
  const int first = (nwg % 8 == 0) ? (blockIdx.x % 8) * (nwg / 8) + blockIdx.x / 8 : blockIdx.x;
  int t = first;
  if (!find_tile(t, cur)) return;
  set_tile(cur);
  parts(C0{}, C7{});
  wait_vm<0>();
  bool more = true;
  while (more) {
    lds_barrier();  // every wavefront's first copies have landed
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
#pragma unroll
    for (int sn = 0; sn < 8; ++sn) fa[sn] = read_p(C0{}, 0, sn);
    int kt = 0;
    for (; kt + kRing <= n_run - kDrain; kt += kRing)
      static_for<kRing>([&](auto V) { kstep(kt + decltype(V)::value, V, C0{}); });
    static_for<RES>([&](auto V) { kstep(kt + decltype(V)::value, V, C0{}); });
    kt += RES;
    kstep(kt, std::integral_constant<int, RES>{}, C1{});
    kstep(kt + 1, std::integral_constant<int, RES + 1>{}, C2{});
    kstep(kt + 2, std::integral_constant<int, RES + 2>{}, C3{});
    // the sums are complete here: without this the compiler moves the last steps' MFMAs, with
    // their operands held or spilled, into the epilogue
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) asm volatile("" : "+a"(acc[a][b]));
    float p[2];
    if constexpr (EP == EP_SWIGLU) {  // ahead of the next tile's loads, which would be waited for too
#pragma unroll
      for (int sm = 0; sm < 2; ++sm) p[sm] = prm.prob[min(cur.row + wave * 64 + sm * 32 + l32, R - 1)];
    }
    lds_barrier();  // no wavefront reads a slot any more
    Tile next = cur;
    t += nwg;
    more = find_tile(t, next);
    set_tile(next);  // past the last tile: this one's first loads again, unused
    __builtin_amdgcn_sched_barrier(0);

    // ---------------- epilogue ----------------
    const int ln = fresh_lane();
    const int e32 = ln & 31, ehi = ln >> 5;
    const int row0 = wave * 64;   // this wavefront's first row of the tile
    if constexpr (EP == EP_STORE) {
      // bf16 through the wavefront's own 8 KiB: four blocks of 32 rows x 128 columns, 256-byte
      // rows with chunk c of row r at c ^ (r & 15); 4 whole row segments leave per store, rows
      // past the expert dropped by the range check. Non-temporal: the output, larger than the
      // caches where it matters, then leaves the operands in them (131072 rows x 768 x 2048:
      // 270 -> 240 us; the card writes such tiles at 6 TB/s when it does nothing else, 90 us).
      uint8_t* out = sOut + wave * 8192;
      const int64_t ldb = (int64_t)prm.N * 2;
      const int valid = min(cur.row_end - cur.row, kBM);
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((bf16_t*)prm.c + (int64_t)cur.row * prm.N + (int64_t)cur.nt * kBN), (short)0,
          (int)(uint32_t)((valid - 1) * ldb + kBN * 2), kBufferFlags);
      const int pc = ln & 15;
#pragma unroll
      for (int sm = 0; sm < 2; ++sm)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (sm == 0 && b == 0) {  // the copies of step 0 ahead of the rest, which the last wait counts on
            parts(C0{}, C2{});
            parts(C2{}, C7{});
          }
#pragma unroll
          for (int sq = 0; sq < 4; ++sq)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x16& a = acc[b * 4 + sq][sm];
              const int ch = sq * 4 + j;
              *reinterpret_cast<uint2*>(out + e32 * 256 + ((ch ^ (e32 & 15)) << 4) + ehi * 8) =
                  make_uint2(pack_bf16x2(a[j * 4], a[j * 4 + 1]), pack_bf16x2(a[j * 4 + 2], a[j * 4 + 3]));
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rl = 4 * i + (ln >> 4);
            const v4u32 val = *reinterpret_cast<const v4u32*>(out + rl * 256 + ((pc ^ (rl & 15)) << 4));
            __builtin_amdgcn_raw_buffer_store_b128(val, rs, (uint32_t)((row0 + sm * 32 + rl) * ldb + b * 256 + pc * 16), 0, 2);
          }
          __builtin_amdgcn_sched_barrier(0);  // one block's values in registers at a time
        }
    } else {
      // h in fragment order and its scales in lane order, as the down product reads them; a dead
      // row's stores get an offset past the range
      const int hslices = prm.I / 64, blk0 = cur.row >> 5;
      const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((uint8_t*)prm.c + ((int64_t)blk0 * hslices + cur.nt * 2) * 1024), (short)0, 0x7FFFFFFF, kBufferFlags);
      const __amdgpu_buffer_rsrc_t rsc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(prm.c_s + ((int64_t)(cur.nt >> 1) * R + cur.row) * 8), (short)0, 0x7FFFFFFF, kBufferFlags);
#pragma unroll
      for (int sm = 0; sm < 2; ++sm) {
        const int mg = cur.row + row0 + sm * 32 + e32;
        const bool live = mg < cur.row_end;
        const uint32_t at = (uint32_t)(((mg >> 5) - blk0) * hslices * 1024 + (mg & 31) * 16 + ehi * 8);
        uint32_t bytes[4];
#pragma unroll
        for (int sn = 0; sn < 4; ++sn) {
          if (sm == 0 && sn == 0) parts(C0{}, C2{});
          if (sm == 0 && sn == 1) parts(C2{}, C3{});
          if (sm == 0 && sn == 2) parts(C3{}, C4{});
          if (sm == 0 && sn == 3) parts(C4{}, C6{});
          if (sm == 1 && sn == 0) parts(C6{}, C7{});
          // a 32-value block of h: columns 8j + 4 ehi + (0..3) here, the others in lane ^ 32
          float h[16];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            h[i] = silu_f(acc[sn][sm][i]) * acc[sn + 4][sm][i] * p[sm];
            top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
          }
          const auto other = __builtin_amdgcn_permlane32_swap(top, top, false, false);
          const int b = scale_byte(max((uint32_t)other[0], (uint32_t)other[1]));
          bytes[sn] = (uint32_t)b;
          // 16-bit groups j = 0, 1 and 2, 3 of both halves -> 8 consecutive bytes a lane
          const auto sw = __builtin_amdgcn_permlane32_swap(pack8(h, b), pack8(h + 8, b), false, false);
          const uint32_t lo = (uint32_t)sw[0], hi = (uint32_t)sw[1];  // the lower and the upper lane's pair
          typedef unsigned int v2u32 __attribute__((ext_vector_type(2)));
          const v2u32 val = {(lo & 0xFFFFu) | (hi << 16), (lo >> 16) | (hi & 0xFFFF0000u)};
          __builtin_amdgcn_raw_buffer_store_b64(val, rc, live ? at + (uint32_t)((sn >> 1) * 1024 + (sn & 1) * 512) : 0xFFFFFFF0u,
                                                0, 0);
          __builtin_amdgcn_sched_barrier(0);  // one block's values in registers at a time
        }
        // blocks 4 (nt & 1) + sn of the down product's step nt / 2: bytes 2 (nt & 1) and + 1 of
        // word g = sn & 1, which lane half g writes
        const uint32_t half = ehi ? bytes[1] | (bytes[3] << 8) : bytes[0] | (bytes[2] << 8);
        __builtin_amdgcn_raw_buffer_store_b16((short)half, rsc,
                                              live ? (uint32_t)((mg - cur.row) * 8 + ehi * 4 + (cur.nt & 1) * 2) : 0xFFFFFFF0u, 0, 0);
      }
    }
    cur = next;
    // the next tile's first weights have landed. STORE: 40 more loads and all 32 stores are younger,
    // and no store is waited for here (the MLP of 131072 rows, 128 experts of 2048 x 768: 665 us
    // with the loads between the blocks of stores, 645 with them ahead). SWIGLU: four stores of
    // the last block and the scales' are younger
    wait_vm<EP == EP_STORE ? 63 : 5>();
  }
  wait_vm<0>();
}

}  // namespace

moe_status launch_tile(int ep, const Params& p, hipStream_t s) {
  const int64_t tiles = ((p.R + kBM - 1) / kBM + p.E) * p.n_tiles;
  const int64_t grid = tiles < num_cus() ? tiles : num_cus();
  const int nk = p.K / kStep;
  auto go = [&](auto RES) {
    constexpr int r = decltype(RES)::value;
    if (ep == EP_SWIGLU)
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<EP_SWIGLU, r>), dim3((unsigned)grid), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<EP_STORE, r>), dim3((unsigned)grid), dim3(256), 0, s, p);
  };
  switch (nk < kDrain ? 0 : (nk - kDrain) % kRing) {
    case 0: go(std::integral_constant<int, 0>{}); break;
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    default: go(std::integral_constant<int, 3>{}); break;
  }
  return check_launch(ep == EP_SWIGLU ? "MXFP4 gate_up + ScaledSwiGLU" : "MXFP4 grouped linear");
}

}  // namespace mx4
}  // namespace moe
