// Host-side argument validation and size arithmetic of the running calls, run
// under AddressSanitizer and UndefinedBehaviorSanitizer (host code only).  Every
// call below is rejected, or has nothing to do, before any launch, so the fake
// address it passes is never used.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "gptq_run.h"

static int failures = 0;

static void expect(bool ok, const char *what) {
  if (!ok) {
    std::printf("FAIL: %s (last error: %s)\n", what, gptq_last_error());
    ++failures;
  }
}
static bool refused(gptq_status st, const char *word) {
  return st == GPTQ_ERR_INVALID_ARG && std::strstr(gptq_last_error(), word) != nullptr;
}

int main() {
  void *fake = reinterpret_cast<void *>(uintptr_t(0x10000));
  float *ff = static_cast<float *>(fake);
  int32_t *fi = static_cast<int32_t *>(fake);
  int8_t *fc = static_cast<int8_t *>(fake);
  uint8_t *fu = static_cast<uint8_t *>(fake);
  const int64_t extremes[] = {std::numeric_limits<int64_t>::min(), -1, 0,
                              std::numeric_limits<int64_t>::max()};
  const float nan = std::nanf("");

  // sizes
  expect(gptq_tokens_ld(65536) == 65536 && gptq_tokens_ld(1) == 128, "tokens_ld");
  for (int64_t e : extremes) {
    expect(gptq_tokens_ld(e) == 0, "tokens_ld extreme");
    expect(gptq_w8a8_layer_bytes(e, 64) == 0 && gptq_w8a8_layer_bytes(64, e) == 0, "layer bytes");
    expect(gptq_token_logprobs_ws_bytes(e, 1000, 5) == 0, "logprobs ws rows");
    expect(gptq_token_logprobs_ws_bytes(4, e, 0) == 0, "logprobs ws vocab");
  }
  expect(gptq_w8a8_layer_bytes(int64_t(1) << 24, 65536) == 0, "layer of 2^40 codes");
  expect(gptq_w8a8_layer_bytes(int64_t(1) << 19, 65536) > size_t(1) << 35, "largest layer");
  expect(gptq_token_logprobs_ws_bytes(1, int64_t(1) << 24, 64) > 0, "largest vocabulary");

  gptq_w8a8_layer layer{64, 300, 64, 384, fake, gptq_w8a8_layer_bytes(64, 300)};
  gptq_w8a8_layer up{600, 64, 608, 128, fake, gptq_w8a8_layer_bytes(600, 64)};
  for (int64_t e : extremes) {
    expect(gptq_w8a8_gemm_ws_bytes(&layer, e) == 0, "gemm ws");
    expect(gptq_w8a8_linear_ws_bytes(&layer, e) == 0, "linear ws");
  }
  expect(gptq_w8a8_linear_ws_bytes(&layer, int64_t(1) << 20) >= size_t(384) << 20, "linear ws 2^20");
  expect(gptq_w8a8_linear_ws_bytes(nullptr, 4) == 0, "linear ws NULL");

  // token codes
  for (int64_t e : extremes) {
    if (e != 0)
      expect(refused(gptq_quantize_tokens(fake, 0, e, 300, 300, fc, 384, ff, fi, nullptr), "tokens"),
             "quantize tokens");
    expect(refused(gptq_quantize_tokens(fake, 0, 4, e, 300, fc, 384, ff, fi, nullptr), "cols"),
           "quantize cols");
  }
  expect(gptq_quantize_tokens(nullptr, 0, 0, 300, 300, nullptr, 0, nullptr, nullptr, nullptr) ==
             GPTQ_OK, "quantize nothing");
  expect(refused(gptq_quantize_tokens(fake, 0, 4, 300, extremes[0], fc, 384, ff, fi, nullptr),
                 "stride"), "quantize stride");
  expect(refused(gptq_quantize_tokens(fake, 0, 4, 300, 300, fc, extremes[0], ff, fi, nullptr),
                 "ld_codes"), "quantize ld_codes");
  expect(refused(gptq_silu_mul_quantize(fake, nullptr, 0, 4, 300, 300, fc, 384, ff, fi, nullptr),
                 "u must"), "silu u");

  // product
  gptq_w8a8_layer out{};
  expect(refused(gptq_w8a8_prepare(fu, ff, fu, 64, 300, fake, 100, &out, nullptr), "too small"),
         "prepare mem");
  expect(refused(gptq_w8a8_prepare(fu, ff, fu, extremes[3], 300, fake, 100, &out, nullptr), "rows"),
         "prepare rows");
  expect(out.rows == 0 && out.mem == nullptr, "prepare leaves the layer");
  for (int64_t e : extremes) {
    if (e == 0) continue;
    expect(refused(gptq_w8a8_gemm(&layer, fc, 384, ff, fi, e, fake, 0, 64, fake, 0, nullptr),
                   "tokens"), "gemm tokens");
    expect(refused(gptq_w8a8_gemm(&layer, fc, e, ff, fi, 4, fake, 0, 64, fake, 0, nullptr),
                   "ld_codes"), "gemm ld_codes");
  }
  expect(refused(gptq_w8a8_linear(&layer, fake, 0, 300, 4, fake, 0, extremes[0], fake, 0, nullptr),
                 "ld_y"), "linear ld_y");
  expect(gptq_w8a8_linear(&layer, fake, 0, 300, 4, fake, 0, 64, fake, 16, nullptr) ==
             GPTQ_ERR_WORKSPACE, "linear workspace");

  // norm block
  gptq_norm_params norm{GPTQ_NORM_RMS, GPTQ_NORM_RMS, 0, 1e-6f, 0.f, 1.f, 1.f,
                        nullptr, nullptr, nullptr, nullptr};
  auto block = [&](const gptq_norm_params *p, int64_t t, int64_t d, int64_t ld, int64_t gt) {
    return gptq_norm_block(p, 0, t, d, fake, ld, fake, ld, fake, ld, gt, fake, ld, fake, ld, fc, 128,
                           ff, fi, nullptr);
  };
  expect(refused(block(nullptr, 4, 64, 64, 1), "params"), "norm params");
  for (int64_t e : extremes) {
    expect(refused(block(&norm, 4, e, 64, 1), "d must"), "norm d");
    if (e < 0) expect(refused(block(&norm, 4, 64, e, 1), "stride"), "norm ld");
    if (e <= 0) expect(refused(block(&norm, 4, 64, 64, e), "gate_tokens"), "norm gate_tokens");
    if (e != 0) expect(refused(block(&norm, e, 64, 64, 1), "tokens"), "norm tokens");
  }
  gptq_norm_params bad = norm;
  bad.eps = nan;
  expect(refused(block(&bad, 4, 64, 64, 1), "eps"), "norm eps");
  expect(block(&norm, 0, 64, 64, 1) == GPTQ_OK, "norm nothing");

  // gated MLP
  gptq_gated_mlp mlp{norm, norm, up, layer};
  expect(gptq_gated_mlp_ws_bytes(&mlp, 0, 4) >= 4 * (128 + 384) + 4 * 4 * 664, "mlp ws");
  expect(gptq_gated_mlp_ws_bytes(&mlp, 0, int64_t(1) << 20) > size_t(664) << 22, "mlp ws 2^20");
  for (int64_t e : extremes) {
    expect(gptq_gated_mlp_ws_bytes(&mlp, 0, e) == 0, "mlp ws extreme");
    if (e != 0)
      expect(refused(gptq_gated_mlp_forward(&mlp, 0, e, fake, 64, nullptr, 0, 1, fake, 64, fake, 64,
                                            fake, 0, nullptr), "tokens"), "mlp tokens");
  }
  expect(gptq_gated_mlp_forward(&mlp, 0, 4, fake, 64, nullptr, 0, 1, fake, 64, fake, 64, fake, 256,
                                nullptr) == GPTQ_ERR_WORKSPACE, "mlp workspace");

  // scoring
  auto score = [&](int64_t rows, int64_t vocab, int64_t ld, float scale, int32_t k) {
    return gptq_token_logprobs(fake, 0, rows, vocab, ld, static_cast<const int64_t *>(fake), scale,
                               k, ff, fi, ff, fi, ff, fake, 0, nullptr);
  };
  for (int64_t e : extremes) {
    if (e != 0) expect(refused(score(e, 1000, 1000, 1.f, 5), "rows"), "score rows");
    expect(refused(score(4, e, 1000, 1.f, 0), "vocab"), "score vocab");
    if (e <= 0) expect(refused(score(4, 1000, e, 1.f, 5), "ld must"), "score ld");
  }
  for (float s : {0.f, -1.f, nan, std::numeric_limits<float>::infinity(), 1e-40f})
    expect(refused(score(4, 1000, 1000, s, 5), "scale"), "score scale");
  for (int32_t k : {std::numeric_limits<int32_t>::min(), -1, 65, std::numeric_limits<int32_t>::max()})
    expect(refused(score(4, 1000, 1000, 1.f, k), "top_k"), "score top_k");
  expect(score(0, 1000, 1000, 1.f, 5) == GPTQ_OK, "score nothing");
  expect(score(1, int64_t(1) << 24, int64_t(1) << 24, 1.f, 64) == GPTQ_ERR_WORKSPACE, "score ws");

  std::printf("ok: %d failure(s)\n", failures);
  return failures ? 1 : 0;
}
