// Host-side check of the entry points that hold activations in 8 bits, under AddressSanitizer: every call
// ends before any launch (argument, size, alignment, table and workspace checks, workspace sizes), and its
// status is checked. The pointer tables have exactly the entries that the checks may read.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "moe.h"

static int g_failures = 0;

static void expect(const char* what, moe_status got, moe_status want) {
  const char* msg = moe_last_error();
  const size_t len = msg ? std::strlen(msg) : 0;  // the sanitizer checks this read
  if (got != want || (want != MOE_OK && len == 0)) {
    std::printf("FAIL %s: status %d (%s), expected %d; last error '%s'\n", what, (int)got, moe_status_str(got),
                (int)want, msg ? msg : "(null)");
    ++g_failures;
  }
}

int main() {
  const moe_status OK = MOE_OK, INV = MOE_ERR_INVALID_ARG, UNS = MOE_ERR_UNSUPPORTED, WS = MOE_ERR_WORKSPACE;
  alignas(256) static uint8_t buf[4096];
  uint8_t* b = buf;
  int32_t* m = (int32_t*)buf;
  float* f = (float*)buf;

  auto norm = [&](const void* x, const int32_t* rows, int k, moe_dtype dt, int64_t T, int H, float eps, void* sum) {
    return moe_add_norm_mxfp8(x, rows, k, nullptr, b, dt, T, H, eps, sum, nullptr, f, b, b, nullptr);
  };
  expect("norm NULL", norm(nullptr, nullptr, 1, MOE_BF16, 4, 64, 1e-6f, nullptr), INV);
  expect("norm k", norm(b, nullptr, 2, MOE_BF16, 4, 64, 1e-6f, nullptr), INV);
  expect("norm k > 16", norm(b, m, 17, MOE_BF16, 4, 64, 1e-6f, nullptr), UNS);
  expect("norm H", norm(b, nullptr, 1, MOE_BF16, 4, 80, 1e-6f, nullptr), UNS);
  expect("norm eps", norm(b, nullptr, 1, MOE_BF16, 4, 64, 0.f, nullptr), INV);
  expect("norm dtype", norm(b, nullptr, 1, MOE_MXFP8, 4, 64, 1e-6f, nullptr), UNS);
  expect("norm rows", norm(b, m, 2, MOE_BF16, (int64_t)1 << 62, 64, 1e-6f, nullptr), UNS);
  expect("norm sum over gathered rows", norm(b, m, 1, MOE_BF16, 4, 64, 1e-6f, b), INV);
  expect("norm misaligned", norm(b + 8, nullptr, 1, MOE_BF16, 4, 64, 1e-6f, nullptr), INV);
  expect("norm T = 0", norm(nullptr, nullptr, 1, MOE_BF16, 0, 64, 1e-6f, nullptr), OK);

  expect("read cols", mxfp8_dequantize(b, b, 4, 33, nullptr, 4, b, nullptr), INV);
  expect("read rows", mxfp8_dequantize(b, b, 4, 64, nullptr, 5, b, nullptr), INV);
  expect("read huge", mxfp8_dequantize(b, b, (int64_t)1 << 40, 64, m, 4, b, nullptr), UNS);
  expect("read NULL", mxfp8_dequantize(nullptr, b, 4, 64, nullptr, 4, b, nullptr), INV);
  expect("read misaligned", mxfp8_dequantize(b + 4, b, 4, 64, nullptr, 4, b, nullptr), INV);
  expect("read none", mxfp8_dequantize(nullptr, nullptr, 0, 64, nullptr, 0, nullptr, nullptr), OK);

  for (int E : {1, 3, MOE_MAX_EXPERTS}) {
    moe_mlp_desc d{};
    d.E = E; d.H = 256; d.I = 512; d.compute = MOE_BF16; d.act = MOE_BF16; d.wt = MOE_BF16;
    std::vector<const void*> w(E, b);
    std::vector<void*> o(E, b);
    size_t fwd = 0, bwd = 0;
    expect("ws forward", moe_workspace_size(MOE_OP_MLP_FWD, &d, 100, 0, 0, 0, &fwd), OK);
    expect("ws backward", moe_workspace_size(MOE_OP_MLP_BWD_CKPT8, &d, 100, 0, 0, 0, &bwd), OK);
    expect("ws rows", moe_workspace_size(MOE_OP_MLP_BWD_CKPT8, &d, -1, 0, 0, 0, &bwd), INV);
    expect("ws desc", moe_workspace_size(MOE_OP_MLP_BWD_CKPT8, nullptr, 4, 0, 0, 0, &bwd), INV);
    auto forward = [&](const moe_mlp_desc& dd, const void* const* w1, const void* const* w2, size_t bytes) {
      return moe_grouped_mlp_fwd_ckpt8(&dd, 100, b, w1, w2, m, f, b, b, b, b, bytes, nullptr);
    };
    auto backward = [&](const moe_mlp_desc& dd, const void* const* w1, void* const* g2, size_t bytes) {
      return moe_grouped_mlp_bwd_ckpt8(&dd, 100, b, b, dd.act == MOE_MXFP8 ? b : nullptr, 100, nullptr, b, b, f, w1, w.data(),
                                       m, b, o.data(), g2, f, b, bytes, nullptr);
    };
    expect("forward workspace", forward(d, w.data(), w.data(), fwd - 1), WS);
    expect("backward workspace", backward(d, w.data(), o.data(), 0), WS);
    moe_mlp_desc e8 = d;
    e8.act = MOE_MXFP8;
    expect("forward in codes", forward(e8, w.data(), w.data(), fwd), UNS);
    expect("backward in codes, workspace", backward(e8, w.data(), o.data(), 0), WS);
    expect("forward NULL table", forward(d, nullptr, w.data(), fwd), INV);
    w[E - 1] = nullptr;
    expect("forward NULL weight", forward(d, w.data(), w.data(), fwd), INV);
    expect("backward NULL weight", backward(d, w.data(), o.data(), 0), INV);
    w[E - 1] = b + 8;
    expect("forward misaligned weight", forward(d, w.data(), w.data(), fwd), INV);
    w[E - 1] = b;
    o[E - 1] = nullptr;
    expect("backward NULL gradient", backward(d, w.data(), o.data(), 0), INV);
    for (int bad = 0; bad < 5; ++bad) {
      moe_mlp_desc x = d;
      if (bad == 0) x.E = 0;
      if (bad == 1) x.H = 255;
      if (bad == 2) x.I = 384;
      if (bad == 3) x.compute = MOE_MXFP8;
      if (bad == 4) x.wt = MOE_FP8;
      const moe_status want = bad == 0 ? INV : UNS;
      expect("forward desc", forward(x, w.data(), w.data(), fwd), want);
      expect("backward desc", backward(x, w.data(), o.data(), 0), want);
    }
  }
  expect("forward NULL desc",
         moe_grouped_mlp_fwd_ckpt8(nullptr, 4, b, nullptr, nullptr, m, f, b, b, b, b, 0, nullptr), INV);
  expect("backward NULL desc", moe_grouped_mlp_bwd_ckpt8(nullptr, 4, b, b, b, 4, m, b, b, f, nullptr, nullptr, m, b,
                                                         nullptr, nullptr, f, b, 0, nullptr), INV);
  std::printf("%s: %d failure(s)\n", g_failures ? "FAILED" : "ok", g_failures);
  return g_failures ? 1 : 0;
}
