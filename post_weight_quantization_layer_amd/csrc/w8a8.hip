// y = x W^T of a per-row 8-bit layer in 8-bit integers: token codes times
// weight codes on v_mfma_i32_16x16x64_i8, exact in int32, scaled per token
// and row in the epilogue.
//
// With weights s_r (c - z_r), c and z in 0..255, held as c - 128 (one sign
// bit flip), sum_k q_k (c - z) = sum_k q_k (c - 128) - (z - 128) sum_k q_k:
// the zero point costs one product per output with the token's code sum.
// Sums wrap modulo 2^32, so only the result has to fit: |result| <=
// 127 * 255 * cols < 2^31 for cols <= 65536.
//
// Prepared layout: tiles of 16 rows x 128 k as the MFMA takes them, two
// 1 KiB halves of 64 k; lane l holds row l % 16, k = 16 (l / 16) .. + 15.
#include <algorithm>
#include <string>

#include "rows.h"

namespace gptq {

gptq_status quantize_impl(const void *x, const void *u, int32_t dtype, int64_t tokens,
                          int64_t cols, int64_t ld, int8_t *codes, int64_t ld_codes, float *scale,
                          int32_t *sum, hipStream_t s, const char *name);
gptq_status check_activations(const void *x, int32_t dtype, int64_t tokens, int64_t cols,
                              int64_t ld, const char *what);

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;       // k per prepared tile

// ----------------------------------------------------------------- prepare
struct Geometry {
  int64_t rows, cols, rows_pad, k_pad;
};
Geometry geometry(int64_t rows, int64_t cols) {
  return {rows, cols, (rows + 15) / 16 * 16, (cols + kStep - 1) / kStep * kStep};
}
// Codes, then scales, then z - 128, rows_pad each.
struct LayerMap {
  int8_t *w;
  float *scale;
  int32_t *shift;
  size_t bytes;
};
LayerMap layer_map(void *mem, const Geometry &g) {
  char *p = static_cast<char *>(mem);
  const size_t codes = align256(size_t(g.rows_pad) * g.k_pad);
  const size_t vec = align256(size_t(g.rows_pad) * 4);
  return {reinterpret_cast<int8_t *>(p), reinterpret_cast<float *>(p + codes),
          reinterpret_cast<int32_t *>(p + codes + vec), codes + 2 * vec};
}

// One 16-byte piece per thread: row r = 16 rt + l % 16, k from 128 step +
// 64 half + 16 (l / 16).  Rows and columns past the layer are 0.
__global__ void __launch_bounds__(256)
    w8a8_repack_kernel(const uint8_t *__restrict__ q, int64_t rows, int64_t cols, int64_t pieces,
                       int64_t steps, u32x4r_t *__restrict__ w) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int l = int(i & 63), half = int((i >> 6) & 1);
  const int64_t tile = i >> 7, step = tile % steps, rt = tile / steps;
  const int64_t r = rt * 16 + (l & 15), k = step * kStep + half * 64 + (l >> 4) * 16;
  u32x4r_t v = {0, 0, 0, 0};
  if (r < rows && k < cols) {
    const uint8_t *p = q + r * cols + k;
    if (k + 16 <= cols) {
      __builtin_memcpy(&v, p, 16);
      v ^= 0x80808080u;
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (k + b < cols) v[b >> 2] |= (uint32_t(p[b]) ^ 0x80u) << (8 * (b & 3));
    }
  }
  w[i] = v;
}
__global__ void __launch_bounds__(256)
    w8a8_row_scales_kernel(const float *__restrict__ scale, const uint8_t *__restrict__ zero,
                     int64_t rows, int64_t rows_pad, float *__restrict__ s,
                     int32_t *__restrict__ shift) {
  const int64_t r = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (r >= rows_pad) return;
  s[r] = r < rows ? scale[r] : 0.f;
  shift[r] = r < rows ? int(zero[r]) - 128 : 0;
}

// ----------------------------------------------------------------- product
struct GemmArgs {
  const int8_t *w;
  const float *w_scale;
  const int32_t *w_shift;
  const int8_t *x;
  const float *x_scale;
  const int32_t *x_sum;
  void *y;
  int64_t ld_x, ld_y;
  int tokens, rows, row_tiles, steps, y_type;
};

// Outputs of one 16 x 16 result block: the lane's token t (column l % 16) and
// four rows r .. r + 3 (4 (l / 16)).
__device__ __forceinline__ void store_block(const GemmArgs &a, const i32x4_t &acc, int t, int r) {
  if (t >= a.tokens || r >= a.rows) return;
  const float st = a.x_scale[t];
  const int sum = a.x_sum[t];
  float v[4];
  uint32_t n = a.rows - r;
#pragma unroll
  for (int j = 0; j < 4; ++j)       // rows_pad is a multiple of 16: in bounds
    v[j] = float(int(uint32_t(acc[j]) - uint32_t(a.w_shift[r + j]) * uint32_t(sum))) *
           (st * a.w_scale[r + j]);
  const int64_t at = int64_t(t) * a.ld_y + r;
  auto put = [&](auto tag) {
    using T = decltype(tag);
    T *p = static_cast<T *>(a.y) + at;
    T o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = narrow<T>(v[j]);
    if (n >= 4) __builtin_memcpy(p, o, sizeof(o));
    else
      for (uint32_t j = 0; j < n; ++j) p[j] = o[j];
  };
  if (a.y_type == GPTQ_DT_F32) put(float{});
  else if (a.y_type == GPTQ_DT_BF16) put(bf16_t{});
  else put(f16_t{});
}

// One wave per 16 rows x 64 tokens, operands straight from memory.
__global__ void __launch_bounds__(256) w8a8_plain_kernel(GemmArgs a) {
  const int lane = threadIdx.x & 63;
  const int rt = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * 64;
  if (rt >= a.row_tiles) return;
  i32x4_t acc[4] = {};
  const int8_t *w = a.w + int64_t(rt) * a.steps * 2048 + lane * 16;
  for (int s = 0; s < 2 * a.steps; ++s) {
    const i32x4_t wf = *reinterpret_cast<const i32x4_t *>(w + int64_t(s) * 1024);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = min(t0 + 16 * j + (lane & 15), a.tokens - 1);
      const i32x4_t xf = *reinterpret_cast<const i32x4_t *>(a.x + int64_t(t) * a.ld_x + s * 64 +
                                                            (lane >> 4) * 16);
      acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, xf, acc[j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    store_block(a, acc[j], t0 + 16 * j + (lane & 15), rt * 16 + 4 * (lane >> 4));
}

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxTokens = int64_t(1) << 20;

size_t codes_bytes(const gptq_w8a8_layer *l, int64_t tokens) {
  return align256(size_t(tokens) * l->k_pad);
}

gptq_status check_layer(const gptq_w8a8_layer *l) {
  if (!l || !l->mem || gptq_w8a8_layer_bytes(l->rows, l->cols) == 0 ||
      l->mem_bytes < gptq_w8a8_layer_bytes(l->rows, l->cols))
    return fail(GPTQ_ERR_INVALID_ARG, "layer is not prepared");
  return GPTQ_OK;
}
gptq_status check_output(const gptq_w8a8_layer *l, const void *y, int32_t y_dtype, int64_t ld_y) {
  if (!y) return fail(GPTQ_ERR_INVALID_ARG, "y must not be NULL");
  if (!is_float_type(y_dtype))
    return fail(GPTQ_ERR_INVALID_ARG, "y's type must be F32, BF16 or F16");
  if (!aligned_to(y, type_bytes(y_dtype)))
    return fail(GPTQ_ERR_INVALID_ARG, "y must be aligned to its elements");
  if (ld_y < l->rows) return fail(GPTQ_ERR_INVALID_ARG, "ld_y must be >= rows");
  return GPTQ_OK;
}
gptq_status check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens must be in [0, 2^20]");
  return GPTQ_OK;
}
gptq_status check_scratch(const void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return GPTQ_OK;
  if (!ws) return fail(GPTQ_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned_to(ws, 256)) return fail(GPTQ_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need)
    return fail(GPTQ_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) +
                                        " bytes, got " + std::to_string(ws_bytes));
  return GPTQ_OK;
}

gptq_status gemm_launch(const gptq_w8a8_layer *l, const int8_t *codes, int64_t ld_codes,
                        const float *scale, const int32_t *sum, int64_t tokens, void *y,
                        int32_t y_dtype, int64_t ld_y, void *ws, hipStream_t s) {
  const Geometry g = geometry(l->rows, l->cols);
  const LayerMap m = layer_map(l->mem, g);
  GemmArgs a;
  a.w = m.w;
  a.w_scale = m.scale;
  a.w_shift = m.shift;
  a.x = codes;
  a.x_scale = scale;
  a.x_sum = sum;
  a.y = y;
  a.ld_x = ld_codes;
  a.ld_y = ld_y;
  a.tokens = int(tokens);
  a.rows = int(g.rows);
  a.row_tiles = int(g.rows_pad / 16);
  a.steps = int(g.k_pad / kStep);
  a.y_type = y_dtype;
  return launch("w8a8_gemm", w8a8_plain_kernel,
                dim3(uint32_t(cdiv(a.row_tiles, 4)), uint32_t(cdiv(tokens, 64))), dim3(256), 0, s,
                a);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

size_t gptq_w8a8_layer_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || rows > kMaxRows || gptq_tokens_ld(cols) == 0) return 0;
  return layer_map(nullptr, geometry(rows, cols)).bytes;
}

gptq_status gptq_w8a8_prepare(const uint8_t *q, const float *scale, const uint8_t *zero,
                              int64_t rows, int64_t cols, void *mem, size_t mem_bytes,
                              gptq_w8a8_layer *layer, void *stream) {
  return guarded([&]() -> gptq_status {
    const size_t need = gptq_w8a8_layer_bytes(rows, cols);
    if (need == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "rows and cols must be in [1, 2^24] x [1, 65536]");
    if (!q || !scale || !zero || !mem || !layer)
      return fail(GPTQ_ERR_INVALID_ARG, "q, scale, zero, mem and layer must not be NULL");
    if (!aligned_to(scale, 4)) return fail(GPTQ_ERR_INVALID_ARG, "scale must be 4-byte aligned");
    if (!aligned_to(mem, 256)) return fail(GPTQ_ERR_INVALID_ARG, "mem must be 256-byte aligned");
    if (mem_bytes < need)
      return fail(GPTQ_ERR_INVALID_ARG, "mem too small: need " + std::to_string(need) +
                                            " bytes, got " + std::to_string(mem_bytes));
    const Geometry g = geometry(rows, cols);
    const LayerMap m = layer_map(mem, g);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t pieces = g.rows_pad * g.k_pad / 16;
    GPTQ_TRY(launch("w8a8_repack", w8a8_repack_kernel, dim3(uint32_t(cdiv(pieces, 256))),
                    dim3(256), 0, s, q, rows, cols, pieces, g.k_pad / kStep,
                    reinterpret_cast<u32x4r_t *>(m.w)));
    GPTQ_TRY(launch("w8a8_row_scales", w8a8_row_scales_kernel, dim3(uint32_t(cdiv(g.rows_pad, 256))),
                    dim3(256), 0, s, scale, zero, rows, g.rows_pad, m.scale, m.shift));
    *layer = gptq_w8a8_layer{rows, cols, g.rows_pad, g.k_pad, mem, mem_bytes};
    return GPTQ_OK;
  });
}

size_t gptq_w8a8_gemm_ws_bytes(const gptq_w8a8_layer *layer, int64_t tokens) {
  return 0;
}

// The token codes, their scales and their sums come before the product's own
// scratch.
size_t gptq_w8a8_linear_ws_bytes(const gptq_w8a8_layer *layer, int64_t tokens) {
  if (!layer || tokens < 1 || tokens > kMaxTokens) return 0;
  return codes_bytes(layer, tokens) + 2 * align256(size_t(tokens) * 4) +
         gptq_w8a8_gemm_ws_bytes(layer, tokens);
}

gptq_status gptq_w8a8_gemm(const gptq_w8a8_layer *layer, const int8_t *codes, int64_t ld_codes,
                           const float *scale, const int32_t *sum, int64_t tokens, void *y,
                           int32_t y_dtype, int64_t ld_y, void *ws, size_t ws_bytes,
                           void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_layer(layer));
    GPTQ_TRY(check_tokens(tokens));
    if (tokens == 0) return GPTQ_OK;
    if (!codes || !scale || !sum)
      return fail(GPTQ_ERR_INVALID_ARG, "codes, scale and sum must not be NULL");
    if (!aligned_to(codes, 16) || ld_codes % 16 || ld_codes < layer->k_pad)
      return fail(GPTQ_ERR_INVALID_ARG,
                  "codes must be 16-byte aligned, ld_codes a multiple of 16 and >= "
                  "gptq_tokens_ld(cols)");
    if (!aligned_to(scale, 4) || !aligned_to(sum, 4))
      return fail(GPTQ_ERR_INVALID_ARG, "scale and sum must be 4-byte aligned");
    GPTQ_TRY(check_output(layer, y, y_dtype, ld_y));
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_w8a8_gemm_ws_bytes(layer, tokens)));
    return gemm_launch(layer, codes, ld_codes, scale, sum, tokens, y, y_dtype, ld_y, ws,
                       static_cast<hipStream_t>(stream));
  });
}

gptq_status gptq_w8a8_linear(const gptq_w8a8_layer *layer, const void *x, int32_t x_dtype,
                             int64_t ld_x, int64_t tokens, void *y, int32_t y_dtype, int64_t ld_y,
                             void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_layer(layer));
    GPTQ_TRY(check_tokens(tokens));
    GPTQ_TRY(check_activations(x, x_dtype, tokens, layer->cols, ld_x, "x"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_output(layer, y, y_dtype, ld_y));
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_w8a8_linear_ws_bytes(layer, tokens)));
    char *p = static_cast<char *>(ws);
    int8_t *codes = reinterpret_cast<int8_t *>(p);
    float *scale = reinterpret_cast<float *>(p + codes_bytes(layer, tokens));
    int32_t *sum = reinterpret_cast<int32_t *>(p + codes_bytes(layer, tokens) +
                                               align256(size_t(tokens) * 4));
    void *rest = p + codes_bytes(layer, tokens) + 2 * align256(size_t(tokens) * 4);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    GPTQ_TRY(quantize_impl(x, nullptr, x_dtype, tokens, layer->cols, ld_x, codes, layer->k_pad,
                           scale, sum, s, "quantize_tokens"));
    return gemm_launch(layer, codes, layer->k_pad, scale, sum, tokens, y, y_dtype, ld_y, rest, s);
  });
}

}  // extern "C"
