// The residual stream's norms and the token codes an 8-bit product takes.
//
// All three kernels give a row (token) to 1, 4, 8 or 16 waves, hold it in
// registers as float32 from its one load to its one store, and reduce over
// the row's waves: mean and centred sum of squares (two passes over
// registers, so no cancellation), and the largest magnitude.  They move each
// byte once, so memory bounds them for many tokens and the chain of
// reductions for one.  Measured (a copy of 1 GiB moves 5.0 TB/s here): norm
// block 16384 x 8192 bf16 with a gate 195 us, 5.5 TB/s; 1 x 4096 f16 3.8 us;
// codes of 8192 x 8192 bf16 40 us, 5.0 TB/s; silu(g) u of 2048 x 11008 bf16
// 26 us, 4.3 TB/s.
#include <algorithm>
#include <string>
#include <utility>

#include "rows.h"

namespace gptq {
namespace {

// ------------------------------------------------------------- token codes
// codes, scale and sum of a row held as v[NCH][8] (lane's chunk c at element
// 8 (c * 64 WPR + lane)); chunks past the row hold zeros and fill the pad.
template <int WPR, int NCH>
__device__ __forceinline__ void store_codes(const float v[NCH][8], int lane, int64_t ld_pad,
                                            int8_t *codes, float *scale, int32_t *sum,
                                            uint32_t *slot_max, int *slot_sum) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = MaxU::op(m, __float_as_uint(v[c][j]) & 0x7fffffffu);
  m = row_all<MaxU, WPR>(m, slot_max);
  const float s = row_scale(m);
  const bool usable = s > 0.f;   // false for 0 and NaN
  const float inv = 1.f / s;
  int total = 0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int e0 = 8 * (c * 64 * WPR + lane);
    if (e0 >= ld_pad) continue;
    int q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (usable) codes8(v[c], s, inv, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) total += q[j];
    *reinterpret_cast<u32x2_t *>(codes + e0) = pack_codes8(q);
  }
  total = row_all<SumI, WPR>(total, slot_sum);
  if (lane == 0) {
    *scale = s;
    *sum = total;
  }
}

// g / (1 + e^-g) within 7 u (u = 2^-24): e^-g as a power of two (2 u) whose
// argument's rounding error is put back (u; it would be |g| ulp), the sum (u), and
// a reciprocal (2 u) and a product (u) instead of a division.  From |g| = 83 on the 1
// or the exponential no longer counts; g e^g is formed with e^(g/2) twice, since
// e^-g overflows and e^g loses bits before g e^g does.  +infinity stays, -infinity
// gives the quotient's NaN.
__device__ __forceinline__ float silu(float g) {
  const float t = g * -1.4426950408889634f;
  const float lo = __builtin_fmaf(g, -1.4426950408889634f, -t) - g * 1.9259629911266175e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  const float r = g * __builtin_amdgcn_rcpf(1.f + __builtin_fmaf(e, lo * 0.6931471805599453f, e));
  if (fabsf(t) < 120.f) return r;
  if (g > 0.f) return g;
  const float h = expf(0.5f * g);
  return g * h * h;
}

struct CodesOut {
  int8_t *codes;
  int64_t ld;      // bytes between rows
  int64_t pad;     // bytes written per row
  float *scale;
  int32_t *sum;
};

// One row's values: x, or silu(g) u.
template <typename T, Ends E, int WPR, int NCH, bool GATED>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR)
    quantize_kernel(const T *__restrict__ x, const T *__restrict__ u, int64_t tokens, int cols,
                    int64_t ld, CodesOut out) {
  __shared__ uint32_t slot_max[WPR];
  __shared__ int slot_sum[WPR];
  constexpr int kRows = WPR == 1 ? 4 : 1;
  const int lane = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t t = int64_t(blockIdx.x) * kRows + (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (t >= tokens) return;       // whole waves; no barrier when WPR == 1
  const T *xr = x + t * ld, *ur = GATED ? u + t * ld : nullptr;
  Pack8<T> kx[NCH], ku[GATED ? NCH : 1];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    kx[c] = fetch8<E>(xr, 8 * (c * 64 * WPR + lane), cols);
    if (GATED) ku[GATED ? c : 0] = fetch8<E>(ur, 8 * (c * 64 * WPR + lane), cols);
  }
  float v[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int e0 = 8 * (c * 64 * WPR + lane);
    widen8<E>(kx[c], e0, cols, 0.f, v[c]);
    if (GATED && e0 < cols) {
      float w[8];
      widen8<E>(ku[GATED ? c : 0], e0, cols, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = silu(v[c][j]) * w[j];
    }
  }
  store_codes<WPR, NCH>(v, lane, out.pad, out.codes + t * out.ld, out.scale + t, out.sum + t,
                        slot_max, slot_sum);
}

// Rows wider than 64 * 16 * 4 * 8 = 32768: two passes over the row.
template <typename T, Ends E, bool GATED>
__global__ void __launch_bounds__(1024)
    quantize_wide_kernel(const T *__restrict__ x, const T *__restrict__ u, int64_t tokens,
                         int cols, int64_t ld, CodesOut out) {
  __shared__ uint32_t slot_max[16];
  __shared__ int slot_sum[16];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  auto value = [&](int e0, float v[8]) {
    const T *xr = x + t * ld;
    const Pack8<T> k = fetch8<E>(xr, e0, cols);
    if (GATED) {
      const T *ur = u + t * ld;
      const Pack8<T> ku = fetch8<E>(ur, e0, cols);
      float w[8];
      widen8<E>(k, e0, cols, 0.f, v);
      widen8<E>(ku, e0, cols, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * w[j];
    } else {
      widen8<E>(k, e0, cols, 0.f, v);
    }
  };
  uint32_t m = 0;
  for (int e0 = 8 * tid; e0 < cols; e0 += 8192) {
    float v[8];
    value(e0, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = MaxU::op(m, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  m = row_all<MaxU, 16>(m, slot_max);
  const float s = row_scale(m), inv = 1.f / s;
  int total = 0;
  for (int e0 = 8 * tid; e0 < out.pad; e0 += 8192) {
    float v[8];
    int q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    value(e0, v);
    if (s > 0.f) codes8(v, s, inv, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) total += q[j];
    *reinterpret_cast<u32x2_t *>(out.codes + t * out.ld + e0) = pack_codes8(q);
  }
  total = row_all<SumI, 16>(total, slot_sum);
  if (tid == 0) {
    out.scale[t] = s;
    out.sum[t] = total;
  }
}

// --------------------------------------------------------------- norm block
struct NormArgs {
  const void *r, *b, *gate;
  void *r_out, *h;
  int64_t ld_r, ld_b, ld_gate, ld_r_out, ld_h, gate_tokens, tokens;
  const void *post_w, *post_b, *pre_w, *pre_b;
  int d, w_type, post, pre;
  float eps, offset, alpha, beta;
  CodesOut out;    // codes NULL: none
};

// The weights of one norm, fetched ahead of their use (four chunks per lane
// have no registers for that: they are fetched where they are used).
template <Ends E, int WB, int WPR, int NCH>
struct NormWeights {
  RawW<WB> w[NCH], b[NCH];
  __device__ __forceinline__ void fetch(const void *weight, const void *bias, int d, int lane) {
    if (NCH == 4) return;
    if (weight)
#pragma unroll
      for (int c = 0; c < NCH; ++c) w[c] = fetch_w<E, WB>(weight, 8 * (c * 64 * WPR + lane), d);
    if (bias)
#pragma unroll
      for (int c = 0; c < NCH; ++c) b[c] = fetch_w<E, WB>(bias, 8 * (c * 64 * WPR + lane), d);
  }
};

// v := N(v) with the sums over the row's d elements; chunks past the row
// stay 0.
template <Ends E, int WB, int WPR, int NCH>
__device__ __forceinline__ void normalize(float v[NCH][8], int kind,
                                          const NormWeights<E, WB, WPR, NCH> &nw, const void *w,
                                          const void *bias, int w_type, float offset, float eps,
                                          int d, int lane, float *slot_mean, float *slot_sq) {
  if (kind == GPTQ_NORM_NONE) return;
  if (kind == GPTQ_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[c][j];
    const float mean = row_all<SumF, WPR>(s, slot_mean) / float(d);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int n = d - 8 * (c * 64 * WPR + lane);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = j < n ? v[c][j] - mean : 0.f;
    }
  }
  float sq = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq += v[c][j] * v[c][j];
  const float rstd = 1.f / sqrtf(row_all<SumF, WPR>(sq, slot_sq) / float(d) + eps);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int e0 = 8 * (c * 64 * WPR + lane);
    float f[8];
    if (w) {
      widen_w<E, WB>(NCH == 4 ? fetch_w<E, WB>(w, e0, d) : nw.w[c], w_type, e0, d, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= rstd * (offset + f[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= rstd;
    }
    if (bias) {
      widen_w<E, WB>(NCH == 4 ? fetch_w<E, WB>(bias, e0, d) : nw.b[c], w_type, e0, d, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] += f[j];
    }
  }
}

// One launch for the four passes over the row that the formula names (mean and
// square of b, of r'): the row stays in registers.  Every vector is fetched
// before the reduction that its use waits for; with one chunk per lane (few
// rows) all of them at the start.
template <typename T, Ends E, int WB, int WPR, int NCH>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) norm_block_kernel(NormArgs a) {
  __shared__ float slots[4][WPR];
  __shared__ uint32_t slot_max[WPR];
  __shared__ int slot_sum[WPR];
  constexpr int kRows = WPR == 1 ? 4 : 1;
  const int lane = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t t = int64_t(blockIdx.x) * kRows + (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (t >= a.tokens) return;     // whole waves; no barrier when WPR == 1
  const int d = a.d;
  const bool out = a.h || a.out.codes;
  const T *r = static_cast<const T *>(a.r) + t * a.ld_r;
  Pack8<T> kr[NCH];
  NormWeights<E, WB, WPR, NCH> pre;
  float v[NCH][8];               // r, then r', then h
  if (a.b) {
    const T *b = static_cast<const T *>(a.b) + t * a.ld_b;
    const T *g = static_cast<const T *>(a.gate) +
                 (a.gate ? int64_t(uint32_t(t) / uint32_t(a.gate_tokens)) * a.ld_gate : 0);
    Pack8<T> kb[NCH], kg[NCH];
    NormWeights<E, WB, WPR, NCH> post;
    float p[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) kb[c] = fetch8<E>(b, 8 * (c * 64 * WPR + lane), d);
#pragma unroll
    for (int c = 0; c < NCH; ++c) kr[c] = fetch8<E>(r, 8 * (c * 64 * WPR + lane), d);
    post.fetch(a.post_w, a.post_b, d, lane);
    if (NCH == 1 && a.gate) kg[0] = fetch8<E>(g, 8 * lane, d);
    if (NCH == 1 && out) pre.fetch(a.pre_w, a.pre_b, d, lane);
#pragma unroll
    for (int c = 0; c < NCH; ++c) widen8<E>(kb[c], 8 * (c * 64 * WPR + lane), d, 0.f, p[c]);
    normalize<E, WB, WPR, NCH>(p, a.post, post, a.post_w, a.post_b, a.w_type, a.offset, a.eps, d,
                            lane, slots[0], slots[1]);
    if (a.gate) {
      if (NCH > 1)
#pragma unroll
        for (int c = 0; c < NCH; ++c) kg[c] = fetch8<E>(g, 8 * (c * 64 * WPR + lane), d);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float f[8];
        widen8<E>(kg[c], 8 * (c * 64 * WPR + lane), d, 0.f, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[c][j] *= f[j];
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      widen8<E>(kr[c], 8 * (c * 64 * WPR + lane), d, 0.f, v[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = a.alpha * v[c][j] + a.beta * p[c][j];
    }
    if (NCH > 1 && out) pre.fetch(a.pre_w, a.pre_b, d, lane);
  } else {
#pragma unroll
    for (int c = 0; c < NCH; ++c) kr[c] = fetch8<E>(r, 8 * (c * 64 * WPR + lane), d);
    if (out) pre.fetch(a.pre_w, a.pre_b, d, lane);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      widen8<E>(kr[c], 8 * (c * 64 * WPR + lane), d, 0.f, v[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= a.alpha;
    }
  }
  if (a.r_out) {
    T *o = static_cast<T *>(a.r_out) + t * a.ld_r_out;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = 8 * (c * 64 * WPR + lane);
      if (e0 < d) store8(o + e0, d - e0, v[c]);
    }
  }
  if (!out) return;
  normalize<E, WB, WPR, NCH>(v, a.pre, pre, a.pre_w, a.pre_b, a.w_type, a.offset, a.eps, d, lane,
                          slots[2], slots[3]);
  if (a.h) {
    T *o = static_cast<T *>(a.h) + t * a.ld_h;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = 8 * (c * 64 * WPR + lane);
      if (e0 < d) store8(o + e0, d - e0, v[c]);
    }
  }
  if (a.out.codes)
    store_codes<WPR, NCH>(v, lane, a.out.pad, a.out.codes + t * a.out.ld, a.out.scale + t,
                          a.out.sum + t, slot_max, slot_sum);
}

// ------------------------------------------------------------- launch rules
// Waves per row and 8-element chunks per lane for rows of `n` elements.  Few
// rows take more waves and fewer chunks, which shortens the chain of loads and
// reductions; many rows fewer waves and up to four chunks, a row of up to 2048
// a single wave, without barriers.  Measured, norm block in bf16 (us): 8192 x
// 1300 35 on {4, 1}, 25 on {1, 3}; 8192 x 2048 38 on {4, 1}, 33 on {1, 4}, but
// 1024 x 2048 8.3 and 9.4; 8192 x 5120 76 on {8, 2}, 68 on {4, 3}; 4096 x 12000
// 130 on {16, 2}, 87 on {8, 3}; 8000 x 16384 274 on {16, 2}, 228 on {8, 4}.
struct RowShape {
  int wpr, nch;
};
RowShape row_shape(int64_t n, int64_t rows, int cus) {
  const int64_t lanes = cdiv(n, 8);
  const bool many = rows >= 4 * cus;
  if (lanes <= 64) return {1, 1};
  if (many && lanes <= 128) return {1, 2};
  if (many && lanes <= 192) return {1, 3};
  if (rows >= 16 * cus && lanes <= 256) return {1, 4};
  if (lanes <= 256) return {4, 1};
  if (lanes <= 512) return many ? RowShape{4, 2} : RowShape{8, 1};
  if (many && lanes <= 768) return {4, 3};
  if (lanes <= 1024) return {8, 2};
  if (many && lanes <= 1536) return {8, 3};
  if (many && lanes <= 2048) return {8, 4};
  return {16, lanes <= 2048 ? 2 : 4};
}

template <Ends E, typename F>
gptq_status with_shape(RowShape s, F &&f) {
  switch (s.wpr * 8 + s.nch) {
    case 1 * 8 + 1: return f.template operator()<E, 1, 1>();
    case 1 * 8 + 2: return f.template operator()<E, 1, 2>();
    case 1 * 8 + 3: return f.template operator()<E, 1, 3>();
    case 1 * 8 + 4: return f.template operator()<E, 1, 4>();
    case 4 * 8 + 3: return f.template operator()<E, 4, 3>();
    case 4 * 8 + 1: return f.template operator()<E, 4, 1>();
    case 4 * 8 + 2: return f.template operator()<E, 4, 2>();
    case 8 * 8 + 1: return f.template operator()<E, 8, 1>();
    case 8 * 8 + 2: return f.template operator()<E, 8, 2>();
    case 8 * 8 + 3: return f.template operator()<E, 8, 3>();
    case 8 * 8 + 4: return f.template operator()<E, 8, 4>();
    case 16 * 8 + 2: return f.template operator()<E, 16, 2>();
    default: return f.template operator()<E, 16, 4>();
  }
}
// `d`: the row's width; `n`: the elements its lanes have to cover.
template <typename F>
gptq_status with_row(int64_t d, int64_t n, int64_t rows, F &&f) {
  const RowShape s = row_shape(n, rows, device_cu_count());
  if (ends_of(d) == kShort) return f.template operator()<kShort, 1, 1>();
  return ends_of(d) == kRagged ? with_shape<kRagged>(s, f) : with_shape<kWhole>(s, f);
}

template <typename T>
struct LaunchQuantize {
  const T *x, *u;
  int64_t tokens, cols, ld;
  CodesOut out;
  hipStream_t s;
  const char *name;
  template <Ends E, int WPR, int NCH>
  gptq_status operator()() {
    const dim3 grid(uint32_t(cdiv(tokens, WPR == 1 ? 4 : 1))), block(WPR == 1 ? 256 : 64 * WPR);
    return u ? launch(name, quantize_kernel<T, E, WPR, NCH, true>, grid, block, 0, s, x, u, tokens,
                      int(cols), ld, out)
             : launch(name, quantize_kernel<T, E, WPR, NCH, false>, grid, block, 0, s, x, u,
                      tokens, int(cols), ld, out);
  }
  template <Ends E>
  gptq_status wide() {
    const dim3 grid{uint32_t(tokens)};
    return u ? launch(name, quantize_wide_kernel<T, E, true>, grid, dim3(1024), 0, s, x, u, tokens,
                      int(cols), ld, out)
             : launch(name, quantize_wide_kernel<T, E, false>, grid, dim3(1024), 0, s, x, u,
                      tokens, int(cols), ld, out);
  }
};

template <typename T>
gptq_status quantize_typed(const void *x, const void *u, int64_t tokens, int64_t cols, int64_t ld,
                           const CodesOut &out, hipStream_t s, const char *name) {
  LaunchQuantize<T> l{static_cast<const T *>(x), static_cast<const T *>(u), tokens, cols, ld, out,
                      s, name};
  if (out.pad <= 32768) return with_row(cols, out.pad, tokens, l);
  return ends_of(cols) == kRagged ? l.template wide<kRagged>() : l.template wide<kWhole>();
}

template <typename T>
struct LaunchNorm {
  const NormArgs &a;
  hipStream_t s;
  template <Ends E, int WPR, int NCH>
  gptq_status operator()() {
    const dim3 grid(uint32_t(cdiv(a.tokens, WPR == 1 ? 4 : 1))), block(WPR == 1 ? 256 : 64 * WPR);
    return a.w_type == GPTQ_DT_F32
               ? launch("norm_block", norm_block_kernel<T, E, 4, WPR, NCH>, grid, block, 0, s, a)
               : launch("norm_block", norm_block_kernel<T, E, 2, WPR, NCH>, grid, block, 0, s, a);
  }
};

template <typename T>
gptq_status norm_typed(const NormArgs &a, hipStream_t s) {
  const int64_t n = a.out.codes ? std::max<int64_t>(a.d, a.out.pad) : a.d;
  return with_row(a.d, n, a.tokens, LaunchNorm<T>{a, s});
}

gptq_status check_codes(const int8_t *codes, int64_t ld_codes, int64_t cols, const float *scale,
                        const int32_t *sum) {
  if (!codes || !scale || !sum)
    return fail(GPTQ_ERR_INVALID_ARG, "codes, scale and sum must not be NULL");
  if (!aligned_to(codes, 16)) return fail(GPTQ_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (!aligned_to(scale, 4) || !aligned_to(sum, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "scale and sum must be 4-byte aligned");
  if (ld_codes < gptq_tokens_ld(cols) || ld_codes % 16)
    return fail(GPTQ_ERR_INVALID_ARG,
                "ld_codes must be a multiple of 16 and >= gptq_tokens_ld(cols)");
  return GPTQ_OK;
}

// Whether rows of `width` bytes, n of them `a_pitch` bytes apart from a on and m
// `b_pitch` apart from b on, share a byte.  (Columns of one matrix do not.)
bool rows_overlap(const void *a, uint64_t n, uint64_t a_pitch, const void *b, uint64_t m,
                  uint64_t b_pitch, uint64_t width) {
  if (reinterpret_cast<uintptr_t>(a) > reinterpret_cast<uintptr_t>(b))
    return rows_overlap(b, m, b_pitch, a, n, a_pitch, width);
  const uint64_t gap = reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a);
  if (gap >= (n - 1) * a_pitch + width) return false;     // b begins after a's last row
  uint64_t i = gap / a_pitch, j = 0;                      // the row of a that b begins in
  if (a_pitch == b_pitch) {
    const uint64_t at = gap % a_pitch;
    return at < width || (at + width > a_pitch && i + 1 < n);
  }
  while (i < n && j < m) {                                // along both, row by row
    const uint64_t x = i * a_pitch, y = gap + j * b_pitch;
    if (x < y + width && y < x + width) return true;
    if (x < y) ++i;
    else ++j;
  }
  return false;
}
// An output's rows may be an input's (each is read before it is written) or share
// nothing with it: rows that overlap others would be read and written by different
// workgroups.
bool clash(const void *out, int64_t ld_out, const void *in, int64_t ld_in, int64_t in_rows,
           int64_t tokens, int64_t d, size_t e) {
  if (!out || !in) return false;
  if (out == in && in_rows == tokens && (ld_out == ld_in || tokens == 1)) return false;
  return rows_overlap(out, tokens, ld_out * e, in, in_rows, ld_in * e, d * e);
}

// A launch has at most 2^32 threads, 1024 of them per row here.
constexpr int64_t kMaxTokens = int64_t(1) << 21;

}  // namespace

gptq_status quantize_impl(const void *x, const void *u, int32_t dtype, int64_t tokens,
                          int64_t cols, int64_t ld, int8_t *codes, int64_t ld_codes, float *scale,
                          int32_t *sum, hipStream_t s, const char *name) {
  const CodesOut out{codes, ld_codes, gptq_tokens_ld(cols), scale, sum};
  if (dtype == GPTQ_DT_F32) return quantize_typed<float>(x, u, tokens, cols, ld, out, s, name);
  if (dtype == GPTQ_DT_BF16) return quantize_typed<bf16_t>(x, u, tokens, cols, ld, out, s, name);
  return quantize_typed<f16_t>(x, u, tokens, cols, ld, out, s, name);
}

gptq_status check_activations(const void *x, int32_t dtype, int64_t tokens, int64_t cols,
                              int64_t ld, const char *what) {
  const std::string w(what);
  if (!is_float_type(dtype))
    return fail(GPTQ_ERR_INVALID_ARG, w + "'s type must be F32, BF16 or F16");
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens must be in [0, 2^21]");
  if (tokens == 0) return GPTQ_OK;
  if (!x) return fail(GPTQ_ERR_INVALID_ARG, w + " must not be NULL");
  if (!aligned_to(x, type_bytes(dtype)))
    return fail(GPTQ_ERR_INVALID_ARG, w + " must be aligned to its elements");
  if (ld < cols)
    return fail(GPTQ_ERR_INVALID_ARG, "the row stride of " + w + " is below its width");
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" {

int64_t gptq_tokens_ld(int64_t cols) {
  return cols < 1 || cols > 65536 ? 0 : (cols + 127) / 128 * 128;
}

gptq_status gptq_quantize_tokens(const void *x, int32_t x_dtype, int64_t tokens, int64_t cols,
                                 int64_t ld_x, int8_t *codes, int64_t ld_codes, float *scale,
                                 int32_t *sum, void *stream) {
  return guarded([&]() -> gptq_status {
    if (gptq_tokens_ld(cols) == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "cols must be in [1, 65536]");
    GPTQ_TRY(check_activations(x, x_dtype, tokens, cols, ld_x, "x"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_codes(codes, ld_codes, cols, scale, sum));
    return quantize_impl(x, nullptr, x_dtype, tokens, cols, ld_x, codes, ld_codes, scale, sum,
                         static_cast<hipStream_t>(stream), "quantize_tokens");
  });
}

gptq_status gptq_silu_mul_quantize(const void *g, const void *u, int32_t dtype, int64_t tokens,
                                   int64_t cols, int64_t ld, int8_t *codes, int64_t ld_codes,
                                   float *scale, int32_t *sum, void *stream) {
  return guarded([&]() -> gptq_status {
    if (gptq_tokens_ld(cols) == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "cols must be in [1, 65536]");
    GPTQ_TRY(check_activations(g, dtype, tokens, cols, ld, "g"));
    GPTQ_TRY(check_activations(u, dtype, tokens, cols, ld, "u"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_codes(codes, ld_codes, cols, scale, sum));
    return quantize_impl(g, u, dtype, tokens, cols, ld, codes, ld_codes, scale, sum,
                         static_cast<hipStream_t>(stream), "silu_mul_quantize");
  });
}

gptq_status gptq_norm_block(const gptq_norm_params *p, int32_t dtype, int64_t tokens, int64_t d,
                            const void *r, int64_t ld_r, const void *b, int64_t ld_b,
                            const void *gate, int64_t ld_gate, int64_t gate_tokens, void *r_out,
                            int64_t ld_r_out, void *h, int64_t ld_h, int8_t *codes,
                            int64_t ld_codes, float *scale, int32_t *sum, void *stream) {
  return guarded([&]() -> gptq_status {
    if (!p) return fail(GPTQ_ERR_INVALID_ARG, "params is NULL");
    if (p->post < GPTQ_NORM_NONE || p->post > GPTQ_NORM_LAYER || p->pre < GPTQ_NORM_NONE ||
        p->pre > GPTQ_NORM_LAYER)
      return fail(GPTQ_ERR_INVALID_ARG, "post and pre must be GPTQ_NORM_NONE, _RMS or _LAYER");
    if (!(p->eps >= 0.f) || !(p->eps < HUGE_VALF))
      return fail(GPTQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (d < 1 || d > 32768) return fail(GPTQ_ERR_INVALID_ARG, "d must be in [1, 32768]");
    const bool vectors = p->post_weight || p->post_bias || p->pre_weight || p->pre_bias;
    if (vectors && !is_float_type(p->w_dtype))
      return fail(GPTQ_ERR_INVALID_ARG, "w_dtype must be F32, BF16 or F16");
    for (const void *w : {p->post_weight, p->post_bias, p->pre_weight, p->pre_bias})
      if (w && !aligned_to(w, type_bytes(p->w_dtype)))
        return fail(GPTQ_ERR_INVALID_ARG, "weights and biases must be aligned to their elements");
    GPTQ_TRY(check_activations(r, dtype, tokens, d, ld_r, "r"));
    if (tokens == 0) return GPTQ_OK;
    if (b) GPTQ_TRY(check_activations(b, dtype, tokens, d, ld_b, "b"));
    if (b && gate) {
      if (gate_tokens < 1) return fail(GPTQ_ERR_INVALID_ARG, "gate_tokens must be >= 1");
      GPTQ_TRY(check_activations(gate, dtype, tokens, d, gate_tokens >= tokens ? d : ld_gate,
                                 "gate"));
    }
    if (!r_out && !h && !codes)
      return fail(GPTQ_ERR_INVALID_ARG, "one of r_out, h and codes must be given");
    if (r_out) GPTQ_TRY(check_activations(r_out, dtype, tokens, d, ld_r_out, "r_out"));
    if (h) GPTQ_TRY(check_activations(h, dtype, tokens, d, ld_h, "h"));
    if (codes) GPTQ_TRY(check_codes(codes, ld_codes, d, scale, sum));
    const size_t e = type_bytes(dtype);
    const int64_t gates = b && gate ? cdiv(tokens, std::min(gate_tokens, tokens)) : 0;
    for (const auto &[out, ld_out] : {std::pair{r_out, ld_r_out}, std::pair{h, ld_h}})
      if (clash(out, ld_out, r, ld_r, tokens, tokens, d, e) ||
          clash(out, ld_out, b, ld_b, tokens, tokens, d, e) ||
          (gates > 0 &&
           clash(out, ld_out, gate, gates > 1 ? ld_gate : d, gates, tokens, d, e)))
        return fail(GPTQ_ERR_INVALID_ARG, "r_out and h must be r, b or gate, row for row, or "
                                          "overlap nothing of them");
    if (r_out && h && rows_overlap(r_out, tokens, ld_r_out * e, h, tokens, ld_h * e, d * e))
      return fail(GPTQ_ERR_INVALID_ARG, "r_out and h must not overlap");
    NormArgs a;
    a.r = r;
    a.b = b;
    a.gate = b ? gate : nullptr;
    a.r_out = r_out;
    a.h = h;
    a.ld_r = ld_r;
    a.ld_b = ld_b;
    a.ld_gate = ld_gate;
    a.ld_r_out = ld_r_out;
    a.ld_h = ld_h;
    a.gate_tokens = std::min<int64_t>(std::max<int64_t>(gate_tokens, 1), tokens);   // 32 bits
    a.tokens = tokens;
    a.post_w = p->post_weight;
    a.post_b = p->post_bias;
    a.pre_w = p->pre_weight;
    a.pre_b = p->pre_bias;
    a.d = int(d);
    a.w_type = p->w_dtype;
    a.post = p->post;
    a.pre = p->pre;
    a.eps = p->eps;
    a.offset = p->weight_offset;
    a.alpha = p->residual_scale;
    a.beta = p->block_scale;
    a.out = CodesOut{codes, ld_codes, codes ? gptq_tokens_ld(d) : 0, scale, sum};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == GPTQ_DT_F32) return norm_typed<float>(a, s);
    if (dtype == GPTQ_DT_BF16) return norm_typed<bf16_t>(a, s);
    return norm_typed<f16_t>(a, s);
  });
}

}  // extern "C"
