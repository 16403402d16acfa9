// Row helpers of the token-major kernels (internal): 8-element loads and
// stores in the activation types, wave and row reductions, and the rounding
// of a row to 8-bit codes.
#pragma once

#include <exception>

#include "common.h"
#include "gptq_run.h"

namespace gptq {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4r_t __attribute__((ext_vector_type(4)));

// C++ exceptions (a host allocation that fails) end at the C entry.
template <typename F>
inline gptq_status guarded(F &&f) {
  try {
    return f();
  } catch (const std::exception &) {
    return GPTQ_ERR_DEVICE;
  }
}

inline bool is_float_type(int32_t t) {
  return t == GPTQ_DT_F32 || t == GPTQ_DT_BF16 || t == GPTQ_DT_F16;
}
inline size_t type_bytes(int32_t t) { return t == GPTQ_DT_F32 ? 4 : 2; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct f16_t {
  uint16_t bits;
};
struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16_t v) { return __uint_as_float(uint32_t(v.bits) << 16); }
__device__ __forceinline__ float widen(f16_t v) {
  return float(__builtin_bit_cast(_Float16, v.bits));
}
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float v) {
  return bf16_t{__builtin_bit_cast(uint16_t, __bf16(v))};
}
template <>
__device__ __forceinline__ f16_t narrow<f16_t>(float v) {
  return f16_t{__builtin_bit_cast(uint16_t, _Float16(v))};
}

// Eight consecutive elements at p, of which the first n exist (n >= 8: all).
// The full case is one 16-byte access (two in float32) at the element's own
// alignment: gfx950 takes global accesses of any alignment, and an aligned
// row costs nothing for it, so odd widths and strides need no second path.
template <typename T>
struct Pack8 {
  T v[8];
};
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float out[8]) {
  if (n >= 8) {
    Pack8<T> k;
    __builtin_memcpy(&k, p, sizeof(k));
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = widen(k.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = j < n ? widen(p[j]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float v[8]) {
  if (n >= 8) {
    Pack8<T> k;
#pragma unroll
    for (int j = 0; j < 8; ++j) k.v[j] = narrow<T>(v[j]);
    __builtin_memcpy(p, &k, sizeof(k));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = narrow<T>(v[j]);
  }
}
// The same with the type known only at run time (weight vectors).
__device__ __forceinline__ void load8_any(const void *p, int type, int64_t at, int n, float out[8]) {
  if (type == GPTQ_DT_F32) load8(static_cast<const float *>(p) + at, n, out);
  else if (type == GPTQ_DT_BF16) load8(static_cast<const bf16_t *>(p) + at, n, out);
  else load8(static_cast<const f16_t *>(p) + at, n, out);
}

// ------------------------------------------------------------- reductions
struct SumF {
  __device__ static float op(float a, float b) { return a + b; }
};
struct SumI {
  __device__ static int op(int a, int b) { return a + b; }
};
struct MaxU {
  __device__ static uint32_t op(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
template <typename Op, typename V>
__device__ __forceinline__ V wave_all(V v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = Op::op(v, __shfl_xor(v, m));
  return v;
}
// Over the row's WPR waves (the whole workgroup when WPR > 1): every thread
// gets the value, combined in wave order.  `slot` is WPR words of LDS used
// by this call only, so one barrier is enough.
template <typename Op, int WPR, typename V>
__device__ __forceinline__ V row_all(V v, V *slot) {
  v = wave_all<Op>(v);
  if (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  V r = slot[0];
#pragma unroll
  for (int w = 1; w < WPR; ++w) r = Op::op(r, slot[w]);
  return r;
}

// ------------------------------------------------------------ token codes
// clamp(rint(x / s), -127, 127) for eight values, the quotient correctly
// rounded as in the definition.  x * (1/s) is off by less than 127 * 2^-22;
// only where that could cross a half is the quotient itself formed (a
// division costs about ten instructions, a near tie is rarer than 1 in
// 1000).  Scales so small that 1/s overflows always divide.
__device__ __forceinline__ void codes8(const float x[8], float s, float inv, int q[8]) {
  bool redo = s < 1e-36f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r = x[j] * inv, i = rintf(r);
    q[j] = int(i);
    redo |= fabsf(fabsf(r - i) - 0.5f) < 1e-4f;
  }
  if (redo) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = int(fminf(fmaxf(rintf(x[j] / s), -127.f), 127.f));
  }
}
__device__ __forceinline__ u32x2_t pack_codes8(const int q[8]) {
  u32x2_t w;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = (uint32_t(q[4 * h]) & 0xffu) | ((uint32_t(q[4 * h + 1]) & 0xffu) << 8) |
           ((uint32_t(q[4 * h + 2]) & 0xffu) << 16) | (uint32_t(q[4 * h + 3]) << 24);
  return w;
}
// A row's scale from the largest magnitude's bits; NaN for a row that holds
// a NaN or an infinity (their bits exceed every finite value's).
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  return amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                  : __uint_as_float(amax_bits) / 127.f;
}

}  // namespace gptq
