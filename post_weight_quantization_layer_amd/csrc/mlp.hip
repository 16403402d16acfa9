// A gated MLP block on per-row 8-bit layers as one call: the five launches of
// its operators, one after the other on the stream.  Issued from one place
// because for few tokens the host's work between them is the block's time (2
// tokens, 1024 x 1651: 36 us as five calls from Python, 24 us as one, 21 us with
// outputs of the caller's).
#include <algorithm>
#include <string>

#include "rows.h"

namespace gptq {
namespace {

// Scratch: each operator's output, in order, and the products' own scratch.
struct Codes {
  int8_t *codes;
  float *scale;
  int32_t *sum;
  int64_t ld;
};
struct BlockWs {
  Codes x, a;
  char *gu, *b, *product;
  size_t product_bytes, bytes;
};

BlockWs block_ws(const gptq_gated_mlp *m, int32_t dtype, int64_t tokens, void *mem) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(mem);   // 0 where only the size is asked
  size_t at = 0;
  auto take = [&](size_t n) {
    char *p = reinterpret_cast<char *>(base + at);
    at += align256(n);
    return p;
  };
  auto codes = [&](int64_t cols) {
    Codes c;
    c.ld = gptq_tokens_ld(cols);
    c.codes = reinterpret_cast<int8_t *>(take(size_t(tokens) * c.ld));
    c.scale = reinterpret_cast<float *>(take(size_t(tokens) * 4));
    c.sum = reinterpret_cast<int32_t *>(take(size_t(tokens) * 4));
    return c;
  };
  BlockWs w;
  w.x = codes(m->gate_up.cols);
  w.gu = take(size_t(tokens) * m->gate_up.rows * type_bytes(dtype));
  w.a = codes(m->down.cols);
  w.b = take(size_t(tokens) * m->down.rows * type_bytes(dtype));
  w.product_bytes = std::max(gptq_w8a8_gemm_ws_bytes(&m->gate_up, tokens),
                             gptq_w8a8_gemm_ws_bytes(&m->down, tokens));
  w.product = take(w.product_bytes);
  w.bytes = at;
  return w;
}

bool fits(const gptq_gated_mlp *m) {
  return m && m->gate_up.mem && m->down.mem && m->gate_up.cols == m->down.rows &&
         m->gate_up.rows == 2 * m->down.cols && m->down.rows >= 1 && m->down.rows <= 32768;
}
constexpr int64_t kMaxTokens = int64_t(1) << 20;

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

size_t gptq_gated_mlp_ws_bytes(const gptq_gated_mlp *mlp, int32_t dtype, int64_t tokens) {
  if (!fits(mlp) || !is_float_type(dtype) || tokens < 1 || tokens > kMaxTokens) return 0;
  return block_ws(mlp, dtype, tokens, nullptr).bytes;
}

gptq_status gptq_gated_mlp_forward(const gptq_gated_mlp *mlp, int32_t dtype, int64_t tokens,
                                   const void *r, int64_t ld_r, const void *gate, int64_t ld_gate,
                                   int64_t gate_tokens, void *r_out, int64_t ld_r_out, void *h,
                                   int64_t ld_h, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    if (!fits(mlp))
      return fail(GPTQ_ERR_INVALID_ARG,
                  "gate_up and down must be prepared, gate_up.cols = down.rows <= 32768, "
                  "gate_up.rows = 2 down.cols");
    if (!is_float_type(dtype))
      return fail(GPTQ_ERR_INVALID_ARG, "dtype must be F32, BF16 or F16");
    if (tokens < 0 || tokens > kMaxTokens)
      return fail(GPTQ_ERR_INVALID_ARG, "tokens must be in [0, 2^20]");
    if (tokens == 0) return GPTQ_OK;
    if (!r_out && !h) return fail(GPTQ_ERR_INVALID_ARG, "one of r_out and h must be given");
    if (!ws) return fail(GPTQ_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned_to(ws, 256))
      return fail(GPTQ_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    const int64_t d = mlp->down.rows, inner = mlp->down.cols, two = mlp->gate_up.rows;
    const BlockWs w = block_ws(mlp, dtype, tokens, ws);
    if (ws_bytes < w.bytes)
      return fail(GPTQ_ERR_WORKSPACE, "workspace too small: need " + std::to_string(w.bytes) +
                                          " bytes, got " + std::to_string(ws_bytes));
    GPTQ_TRY(gptq_norm_block(&mlp->enter, dtype, tokens, d, r, ld_r, nullptr, 0, nullptr, 0, 1,
                             nullptr, 0, nullptr, 0, w.x.codes, w.x.ld, w.x.scale, w.x.sum,
                             stream));
    GPTQ_TRY(gptq_w8a8_gemm(&mlp->gate_up, w.x.codes, w.x.ld, w.x.scale, w.x.sum, tokens, w.gu,
                            dtype, two, w.product, w.product_bytes, stream));
    GPTQ_TRY(gptq_silu_mul_quantize(w.gu, w.gu + inner * int64_t(type_bytes(dtype)), dtype, tokens,
                                    inner, two, w.a.codes, w.a.ld, w.a.scale, w.a.sum, stream));
    GPTQ_TRY(gptq_w8a8_gemm(&mlp->down, w.a.codes, w.a.ld, w.a.scale, w.a.sum, tokens, w.b, dtype,
                            d, w.product, w.product_bytes, stream));
    return gptq_norm_block(&mlp->leave, dtype, tokens, d, r, ld_r, w.b, d, gate, ld_gate,
                           gate_tokens, r_out, ld_r_out, h, ld_h, nullptr, 0, nullptr, nullptr,
                           stream);
  });
}

}  // extern "C"
