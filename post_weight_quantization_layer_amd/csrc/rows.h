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

// How a row's width d ends, known at launch: in whole groups of 8 elements, in
// a ragged one, or before the first is full.
enum Ends { kWhole = 0, kRagged = 1, kShort = 2 };
inline Ends ends_of(int64_t d) { return d < 8 ? kShort : d % 8 ? kRagged : kWhole; }

// Eight consecutive elements e0 .. e0 + 7 of a row of d, in two steps, so that
// a lane's loads are all in flight before the first is waited for: fetch8
// loads without a branch (the row's last eight where e0 + 8 > d), widen8 turns
// the elements into float32, moves those of a ragged end into place and puts
// `fill` where there are none.  A fetch is one 16-byte access (two in float32)
// at the element's own alignment: gfx950 takes global accesses of any
// alignment, and an aligned row costs nothing for it.
template <typename T>
struct Pack8 {
  uint32_t w[2 * sizeof(T)];     // whole words: the load stays one access
  __device__ __forceinline__ float at(int j) const;
};
template <>
__device__ __forceinline__ float Pack8<float>::at(int j) const { return __uint_as_float(w[j]); }
template <>
__device__ __forceinline__ float Pack8<bf16_t>::at(int j) const {
  return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
}
template <>
__device__ __forceinline__ float Pack8<f16_t>::at(int j) const {
  return float(__builtin_bit_cast(_Float16, uint16_t(w[j >> 1] >> (16 * (j & 1)))));
}
template <Ends E, typename T>
__device__ __forceinline__ Pack8<T> fetch8(const T *row, int e0, int d) {
  Pack8<T> k = {};
  if (E != kShort) {
    __builtin_memcpy(&k, row + min(e0, d - 8), sizeof(k));
  } else {
    constexpr int kPerWord = 4 / sizeof(T);
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < d) {
        uint32_t bits = 0;
        __builtin_memcpy(&bits, row + j, sizeof(T));
        k.w[j / kPerWord] |= bits << (32 / kPerWord * (j % kPerWord));
      }
  }
  return k;
}
// The elements moved down by s places (0..8), zeros following.
template <typename T>
__device__ __forceinline__ Pack8<T> move_down(Pack8<T> k, int s) {
  constexpr int W = 2 * sizeof(T);
  int words = s;
  if (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      k.w[i] = __builtin_amdgcn_alignbit(i + 1 < W ? k.w[i + 1] : 0u, k.w[i], (s & 1) * 16);
    words = s >> 1;
  }
#pragma unroll
  for (int step = 1; step <= W; step *= 2)
#pragma unroll
    for (int i = 0; i < W; ++i)
      k.w[i] = words & step ? (i + step < W ? k.w[i + step] : 0u) : k.w[i];
  return k;
}
template <Ends E, typename T>
__device__ __forceinline__ void widen8(const Pack8<T> &k, int e0, int d, float fill,
                                       float out[8]) {
  const int n = d - e0;
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = k.at(j);
  if (E == kWhole) {                   // all eight or none
    if (__ballot(n <= 0)) {            // a branch of the whole wave, rarely taken
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = n <= 0 ? fill : out[j];
    }
    return;
  }
  if (__ballot(n < 8)) {               // a branch of the whole wave, rarely taken
    if (E == kRagged) {
      const Pack8<T> m = move_down(k, n < 8 ? min(8 - n, 8) : 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = m.at(j);
    }
    if (fill != 0.f) {                 // move_down and fetch8 leave zeros
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) out[j] = fill;
    } else if (E == kShort && n <= 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = 0.f;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float v[8]) {
  if (n >= 8) {
    T k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = narrow<T>(v[j]);
    __builtin_memcpy(p, k, sizeof(k));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = narrow<T>(v[j]);
  }
}
// Eight values of a weight vector, whose type (of WB bytes) is known only at
// run time: the load first, without a branch on the type, then the widening.
template <int WB>
struct WordOf {
  using type = f16_t;
};
template <>
struct WordOf<4> {
  using type = float;
};
template <int WB>
struct RawW {
  uint32_t k[2 * WB];
};
template <Ends E, int WB>
__device__ __forceinline__ RawW<WB> fetch_w(const void *p, int e0, int d) {
  using T = typename WordOf<WB>::type;
  const Pack8<T> k = fetch8<E>(static_cast<const T *>(p), e0, d);
  RawW<WB> r;
  __builtin_memcpy(r.k, &k, sizeof(r.k));
  return r;
}
template <Ends E, int WB>
__device__ __forceinline__ void widen_w(const RawW<WB> &r, int type, int e0, int d, float out[8]) {
  auto go = [&](auto tag) {
    Pack8<decltype(tag)> k;
    __builtin_memcpy(&k, r.k, sizeof(k));
    widen8<E>(k, e0, d, 0.f, out);
  };
  if constexpr (WB == 4) go(float{});
  else if (type == GPTQ_DT_BF16) go(bf16_t{});
  else go(f16_t{});
}

// ------------------------------------------------------------- reductions
struct SumF {
  __device__ static float op(float a, float b) { return a + b; }
};
struct MaxF {
  __device__ static float op(float a, float b) { return fmaxf(a, b); }
};
struct SumI {
  __device__ static int op(int a, int b) { return a + b; }
};
struct MaxU {
  __device__ static uint32_t op(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
struct MinU {
  __device__ static uint32_t op(uint32_t a, uint32_t b) { return a < b ? a : b; }
};
struct OrU {
  __device__ static uint32_t op(uint32_t a, uint32_t b) { return a | b; }
};
struct AndU {
  __device__ static uint32_t op(uint32_t a, uint32_t b) { return a & b; }
};
template <int CTRL, typename V>
__device__ __forceinline__ V dpp(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf,
                                                        true));
}
template <typename V>
__device__ __forceinline__ V lane_value(V v, int lane) {
  return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// Over a wave, every lane active, in a fixed order; the result is uniform.
// Within rows of 16 lanes by register moves between lanes (pairs, fours,
// mirrored eights and sixteens), a few cycles each where an exchange through
// LDS takes about a hundred; then the four rows' values as scalars.
template <typename Op, typename V>
__device__ __forceinline__ V wave_all(V v) {
  v = Op::op(v, dpp<0xb1>(v));    // lanes 1 0 3 2
  v = Op::op(v, dpp<0x4e>(v));    // lanes 2 3 0 1
  v = Op::op(v, dpp<0x141>(v));   // mirrored in 8
  v = Op::op(v, dpp<0x140>(v));   // mirrored in 16
  return Op::op(Op::op(lane_value(v, 0), lane_value(v, 16)),
                Op::op(lane_value(v, 32), lane_value(v, 48)));
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
