// MXFP4 grouped GEMM for many rows an expert: 256 x 256 tiles on v_mfma_scale_f32_32x32x64
// (E2M1 operands), bound by the MFMA.
//
// Lane l of that MFMA holds 32 consecutive K values (16 bytes) of row l % 32, K half l / 32
// of 64, and their block's scale. A K step is 256 values, one 128-byte line of every row of
// both operands, multiplied in four slices of 64. Four wavefronts of 128 x 128 (16 MFMAs a
// slice) share the tile through a ring of five 32 KiB LDS half-slots, P (weights) of step v
// in half-slot 2v mod 5 and Q (rows) in 2v + 1, filled by range-checked buffer copies:
//   slices 0, 1: copies of P of step v + 2 (into the half-slot Q of step v - 1 left)
//   slice 2    : then wait for step v + 1's copies, barrier
//   slice 3    : scales and copies of Q of step v + 2 (into P of step v's half-slot);
//                fragments of step v + 1's first slice
// so the copies are spread over the step and each has at least three slices to land. Every
// slice's fragments are read while the one before it is multiplied.
// The number of steps modulo 5 is a template parameter: the half-slots of a step are then
// constants without zero steps in front (at K = 2048 those would be 2 of 10).
//
// Scales come in the lane order of the MFMA: word ((step * rows + row) * 2 + g) holds, in
// byte s, the scale of block 2s + g of the row's step, so a lane's one word serves its four
// slices, the byte picked by the instruction.
#include <cstring>
#include <type_traits>

#include "common.h"
#include "gemm_common.h"
#include "internal.h"
#include "mxfp4.h"

namespace moe {
namespace mx4 {

using namespace gemm;

namespace {

constexpr int kBM = 256, kBN = 256, kStep = 256;
constexpr int kRowBytes = kStep / 2;       // of a row, a step
constexpr int kHalf = kBM * kRowBytes;     // an LDS half-slot: one operand of one step
constexpr int kRing = 5;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t wide(i32x4_t v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int EP, int RES>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
void grouped_gemm_tile_kernel(const Params prm) {
  __shared__ __attribute__((aligned(1024))) uint8_t sH0[kHalf], sH1[kHalf], sH2[kHalf], sH3[kHalf], sH4[kHalf];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, lhi = lane >> 5;
  const int E = prm.E, R = (int)prm.R;
  const int ld = prm.K / 2;          // bytes of a code row
  const int nk = prm.K / kStep;
  const int n_tiles = prm.n_tiles;
  const int nwg = gridDim.x;
  const int logical = (nwg % 8 == 0) ? (blockIdx.x % 8) * (nwg / 8) + blockIdx.x / 8 : blockIdx.x;

  auto half = [&](auto H) -> uint8_t* {
    if constexpr (H.value == 0) return sH0;
    else if constexpr (H.value == 1) return sH1;
    else if constexpr (H.value == 2) return sH2;
    else if constexpr (H.value == 3) return sH3;
    else return sH4;
  };

  // tiles: expert-major, row tiles in groups of at most 16 (tile_in_expert); the offsets are
  // walked once, made a nondecreasing sequence inside [0, R] on the way
  auto clamp_off = [&](int v, int prev) -> int {
    v = v < prev ? prev : v;
    return v > R ? R : v;
  };
  auto tiles_of = [&](int rows) -> int { return ((rows + kBM - 1) / kBM) * n_tiles; };
  int total = 0;
  for (int x = 0, prev = 0; x < E; ++x) {
    const int en = clamp_off(load_const(prm.offsets, x + 1), prev);
    total += tiles_of(en - prev);
    prev = en;
  }
  int e_w = 0, ob = 0, oe = clamp_off(load_const(prm.offsets, 1), 0), ts_w = 0;
  int nt_w = tiles_of(oe);

  // fragment addresses: chunk 2s + lhi of a row for slice s, at its swizzled place
  const uint32_t fragP = (uint32_t)((wn * 64 + l32) * kRowBytes);
  const uint32_t fragQ = (uint32_t)((wm * 128 + l32) * kRowBytes);
  uint32_t ck[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) ck[c] = (uint32_t)(((2 * c + lhi) ^ swz8(l32)) << 4);
  // copies: round i of a wavefront fills rows (4i + wave) * 8 + (lane >> 3) of a half-slot
  const int kc_row0 = wave * 8 + (lane >> 3);
  const int kc_chunk = (lane & 7) ^ swz8(kc_row0);
  const uint32_t off0 = (uint32_t)(kc_row0 * ld + kc_chunk * 16);
  constexpr int64_t kAll = 0xFFFFFFFFll;

  for (int t = logical; t < total; t += nwg) {
    while (e_w < E && t >= ts_w + nt_w) {
      ts_w += nt_w;
      ++e_w;
      ob = oe;
      if (e_w < E) {
        oe = clamp_off(load_const(prm.offsets, e_w + 1), ob);
        nt_w = tiles_of(oe - ob);
      }
    }
    if (e_w >= E) break;
    int mt, nt;
    tile_in_expert(t - ts_w, (oe - ob + kBM - 1) / kBM, n_tiles, mt, nt);
    const int e = __builtin_amdgcn_readfirstlane(e_w);
    mt = __builtin_amdgcn_readfirstlane(mt);
    nt = __builtin_amdgcn_readfirstlane(nt);
    const int row_end = __builtin_amdgcn_readfirstlane(oe);
    const int tile_row = __builtin_amdgcn_readfirstlane(ob) + mt * kBM;

    // weight row of local row r (SWIGLU: 128 gate rows, then the up rows of the same columns)
    auto p_row = [&](int r) -> int {
      if constexpr (EP == EP_SWIGLU) return (r < 128) ? nt * 128 + r : prm.I + nt * 128 + (r - 128);
      else return nt * kBN + r;
    };
    const uint8_t* p_tile = prm.tab[e] + (int64_t)p_row(0) * ld;
    const uint8_t* q_tile = prm.q + (int64_t)tile_row * ld;
    const int64_t q_extent = (int64_t)(row_end - tile_row) * ld;  // rows past the expert land as zeros
    const int p_up = EP == EP_SWIGLU ? prm.I - 128 : 0;
    // rounds [I0, I0 + N) of the copy of step kt's operand; an empty range past the last step
    auto copy_op = [&](const uint8_t* tile, int up, int64_t extent, int kt, uint8_t* dst, auto I0, auto N) {
      const int64_t at = (int64_t)kt * kRowBytes;
      int64_t lim = extent - at;
      lim = lim < 0 ? 0 : (lim > kAll ? kAll : lim);
      const uint32_t nrec = (uint32_t)__builtin_amdgcn_readfirstlane(kt < nk ? (int)(uint32_t)lim : 0);
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(tile + at), (short)0, (int)nrec, kBufferFlags);
#pragma unroll
      for (int i = decltype(I0)::value; i < decltype(I0)::value + decltype(N)::value; ++i) {
        const uint32_t rows = (uint32_t)(i * 32 + (i >= 4 ? up : 0));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(dst + wave * 1024 + i * 4096), 16, off0,
                                                 (int)(rows * (uint32_t)ld), 0, 0);
      }
    };
    using I0 = std::integral_constant<int, 0>;
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    auto copy_P = [&](int kt, auto H, auto First, auto N) { copy_op(p_tile, p_up, kAll, kt, half(H), First, N); };
    auto copy_Q = [&](int kt, auto H) { copy_op(q_tile, 0, q_extent, kt, half(H), I0{}, I8{}); };

    // this lane's scale words: 4 P sub-tiles, then 4 Q sub-tiles (rows past the expert: its last)
    const uint8_t* ps_tile = prm.tab_s[e];
    const uint8_t* qs_tile = prm.q_s + (int64_t)tile_row * 8;
    uint32_t ps_off[4], qs_off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ps_off[j] = (uint32_t)((p_row(sub_n(j, wn) + l32) * 2 + lhi) * 4);
      const int qr = wm * 128 + j * 32 + l32;
      qs_off[j] = (uint32_t)(((qr < row_end - tile_row ? qr : row_end - tile_row - 1) * 2 + lhi) * 4);
    }
    auto load_scales = [&](int kt, uint32_t* w) {
      kt = kt < nk ? kt : nk - 1;
      const uint8_t* ps = ps_tile + (int64_t)kt * prm.N * 8;
      const uint8_t* qs = qs_tile + (int64_t)kt * R * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = *reinterpret_cast<const uint32_t*>(ps + ps_off[j]);
        w[4 + j] = *reinterpret_cast<const uint32_t*>(qs + qs_off[j]);
      }
    };

    f32x16 acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

    i32x4_t fa[4], fb0[4], fb1[4];
    auto read_q = [&](auto H, int s, i32x4_t* fb) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        fb[u] = *reinterpret_cast<const i32x4_t*>(half(H) + fragQ + u * 32 * kRowBytes + ck[s]);
    };
    auto read_p = [&](auto H, int s, int sn) -> i32x4_t {
      return *reinterpret_cast<const i32x4_t*>(half(H) + fragP + ((sn >> 1) * 128 + (sn & 1) * 32) * kRowBytes + ck[s]);
    };
    // slice S with Q fragments fb and scale words sc; fa[sn] refilled from slice s_next of HPn
    // as soon as its four MFMAs are issued
    auto mfma_slice = [&](const i32x4_t* fb, const uint32_t* sc, auto S, auto HPn, int s_next) {
      constexpr int s = decltype(S)::value;
#pragma unroll
      for (int sn = 0; sn < 4; ++sn) {
#pragma unroll
        for (int sm = 0; sm < 4; ++sm)
          acc[sn][sm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fa[sn]), wide(fb[sm]), acc[sn][sm], 4, 4, s,
                                                                          (int)sc[sn], s, (int)sc[4 + sm]);
        fa[sn] = read_p(HPn, s_next, sn);
      }
    };
    // 16 MFMAs with 8 fragment reads between them, and CP copies
    auto interleave = [&](auto CP) {
      constexpr int cp = decltype(CP)::value;
      static_for<8>([&](auto I) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if constexpr (cp == 8 || (cp == 4 && decltype(I)::value % 2 == 0)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      });
    };

    uint32_t r0[8], r1[8], r2[8];  // scale words of steps kt, kt + 1, kt + 2
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
    using S3 = std::integral_constant<int, 3>;
    auto kstep = [&](int kt, auto V) {
      constexpr int v = decltype(V)::value;
      using HP = std::integral_constant<int, (2 * v) % kRing>;
      using HQ = std::integral_constant<int, (2 * v + 1) % kRing>;
      using HPn = std::integral_constant<int, (2 * v + 2) % kRing>;
      using HQn = std::integral_constant<int, (2 * v + 3) % kRing>;
      using HPnn = std::integral_constant<int, (2 * v + 4) % kRing>;
      copy_P(kt + 2, HPnn{}, I0{}, I4{});
      read_q(HQ{}, 1, fb1);
      mfma_slice(fb0, r0, S0{}, HP{}, 1);
      interleave(I4{});
      copy_P(kt + 2, HPnn{}, I4{}, I4{});
      read_q(HQ{}, 2, fb0);
      mfma_slice(fb1, r0, S1{}, HP{}, 2);
      interleave(I4{});
      read_q(HQ{}, 3, fb1);
      mfma_slice(fb0, r0, S2{}, HP{}, 3);
      interleave(I0{});
      wait_vm<8>();  // all but P of step kt + 2 has landed
      lds_barrier();
      load_scales(kt + 2, r2);
      __builtin_amdgcn_sched_barrier(0);  // ahead of the copies, which the wait above counts
      copy_Q(kt + 2, HP{});
      read_q(HQn{}, 0, fb0);  // past the last step: never used
      mfma_slice(fb1, r0, S3{}, HPn{}, 0);
      interleave(I8{});
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r0[i] = r1[i];
        r1[i] = r2[i];
      }
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    using H2 = std::integral_constant<int, 2>;
    using H3 = std::integral_constant<int, 3>;
    load_scales(0, r0);
    load_scales(1, r1);
    __builtin_amdgcn_sched_barrier(0);
    copy_P(0, H0{}, I0{}, I8{});
    copy_Q(0, H1{});
    copy_P(1, H2{}, I0{}, I8{});
    copy_Q(1, H3{});
    wait_vm<16>();  // the scale words and step 0
    lds_barrier();
    read_q(H1{}, 0, fb0);
#pragma unroll
    for (int sn = 0; sn < 4; ++sn) fa[sn] = read_p(H0{}, 0, sn);
    int kt = 0;
    for (; kt + kRing <= nk; kt += kRing) static_for<kRing>([&](auto V) { kstep(kt + decltype(V)::value, V); });
    static_for<RES>([&](auto V) { kstep(kt + decltype(V)::value, V); });
    wait_vm<0>();  // the empty copies past the last step land before LDS is reused
    lds_barrier();
    // the sums are complete here: without this the compiler moves the last steps' MFMAs, with
    // their operands held or spilled, into the epilogue's branches
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) asm volatile("" : "+a"(acc[a][b]));

    // ---------------- epilogue ----------------
    int ln = lane;
    asm volatile("" : "+v"(ln));  // keep the lane offsets inside the epilogue
    const int e32 = ln & 31, ehi = ln >> 5;
    if constexpr (EP == EP_STORE) {
      // bf16 through LDS as blocks of 256 rows x 128 columns: 256-byte rows, chunk c of row r at
      // c ^ (r & 15), rows 0-127 in the first array of a pair; 4 whole rows leave per store,
      // rows past the expert dropped by the range check
      const int valid = min(row_end - tile_row, kBM);
      auto put = [&](int b, uint8_t* arr0, uint8_t* arr1) __attribute__((always_inline)) {
        uint8_t* arr = wm ? arr1 : arr0;
#pragma unroll
        for (int sm = 0; sm < 4; ++sm)
#pragma unroll
          for (int sq = 0; sq < 2; ++sq)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const f32x16& a = acc[2 * b + sq][sm];
              const int rr = sm * 32 + e32, ch = wn * 8 + sq * 4 + i4;
              *reinterpret_cast<uint2*>(arr + rr * 256 + ((ch ^ (rr & 15)) << 4) + ehi * 8) =
                  make_uint2(pack_bf16x2(a[i4 * 4], a[i4 * 4 + 1]), pack_bf16x2(a[i4 * 4 + 2], a[i4 * 4 + 3]));
            }
      };
      auto drain = [&](const uint8_t* arr, bf16_t* dst) __attribute__((always_inline)) {
        const int64_t ldb = (int64_t)prm.N * 2;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(dst + (int64_t)tile_row * prm.N), (short)0, (int)(uint32_t)(valid * ldb), kBufferFlags);
        const int pc = ln & 15;
        const uint32_t vo = (uint32_t)((ln >> 4) * ldb + pc * 16);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rl = (wave & 1) * 64 + 4 * i + (ln >> 4);
          const v4u32 val = *reinterpret_cast<const v4u32*>(arr + rl * 256 + ((pc ^ (rl & 15)) << 4));
          __builtin_amdgcn_raw_buffer_store_b128(val, rs, vo, (int)((wave * 64 + 4 * i) * ldb), 0);
        }
      };
      put(0, sH0, sH1);
      put(1, sH2, sH3);
      lds_barrier();
      bf16_t* c0 = reinterpret_cast<bf16_t*>(prm.c) + (int64_t)nt * kBN;
      drain(wave < 2 ? sH0 : sH1, c0);
      drain(wave < 2 ? sH2 : sH3, c0 + 128);
      lds_barrier();  // read out before the next tile's copies land
    } else {
#pragma unroll
      for (int sm = 0; sm < 4; ++sm) {
        const int64_t mg = (int64_t)tile_row + wm * 128 + sm * 32 + e32;
        const bool live = mg < row_end;
        const float p = prm.prob[live ? mg : row_end - 1];
#pragma unroll
        for (int sn = 0; sn < 2; ++sn) {
          // a 32-value block of h: columns 8j + 4 ehi + (0..3) here, the others in lane ^ 32
          float h[16];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            h[i] = silu_f(acc[sn][sm][i]) * acc[sn + 2][sm][i] * p;
            top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
          }
          top = max(top, (uint32_t)__shfl_xor((int)top, 32));
          const int b = scale_byte(top);
          // 16-bit groups j = 0, 1 and 2, 3 of both halves -> 8 consecutive bytes a lane
          const uint32_t w0 = pack8(h, b), w1 = pack8(h + 8, b);
          const auto sw = __builtin_amdgcn_permlane32_swap(w0, w1, false, false);
          const uint32_t lo = (uint32_t)sw[0], hi = (uint32_t)sw[1];  // the lower and the upper lane's pair
          if (live) {
            const int col0 = nt * 128 + wn * 64 + sn * 32;
            uint8_t* C = reinterpret_cast<uint8_t*>(prm.c) + mg * (prm.I / 2) + col0 / 2 + ehi * 8;
            *reinterpret_cast<uint2*>(C) = make_uint2((lo & 0xFFFFu) | (hi << 16), (lo >> 16) | (hi & 0xFFFF0000u));
            // block 4 (nt & 1) + 2 wn + sn of the down product's step nt / 2
            if (ehi == 0) prm.c_s[(((int64_t)(nt >> 1) * R + mg) * 2 + sn) * 4 + (nt & 1) * 2 + wn] = (uint8_t)b;
          }
          __builtin_amdgcn_sched_barrier(0);  // one block's values in registers at a time
        }
      }
    }
  }
}

}  // namespace

moe_status launch_tile(int ep, const Params& p, hipStream_t s) {
  const int64_t tiles = ((p.R + kBM - 1) / kBM + p.E) * p.n_tiles;
  const int64_t grid = tiles < num_cus() ? tiles : num_cus();
  auto go = [&](auto RES) {
    constexpr int r = decltype(RES)::value;
    if (ep == EP_SWIGLU)
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<EP_SWIGLU, r>), dim3((unsigned)grid), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<EP_STORE, r>), dim3((unsigned)grid), dim3(256), 0, s, p);
  };
  switch (p.K / kStep % kRing) {
    case 0: go(std::integral_constant<int, 0>{}); break;
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    default: go(std::integral_constant<int, 4>{}); break;
  }
  return check_launch(ep == EP_SWIGLU ? "MXFP4 gate_up + ScaledSwiGLU" : "MXFP4 grouped linear");
}

}  // namespace mx4
}  // namespace moe
