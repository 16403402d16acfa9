// What the tile products share (internal): the barrier of their pipelines, the
// order of their tiles, the check of their scratch.
#pragma once

#include <string>

#include "rows.h"

namespace gptq {

// A workgroup barrier that orders LDS accesses only: loads from memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Orders a wave's LDS accesses before and after it among its lanes.  (The hardware
// takes them in order; without this the compiler may move one lane's past another's.)
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Workgroups are dealt round-robin to the 8 XCDs; each XCD takes a contiguous run of
// the n units of work.  (Where a product is split, whole splits come one after the
// other: an XCD then reads a part of k of both operands, not all of it.)
__device__ __forceinline__ int xcd_run(int bid, int n) {
  const int x = bid & 7;
  return x * (n / 8) + min(x, n % 8) + (bid >> 3);
}
// Tiles in bands of kBand token tiles, tokens fastest, so that an XCD's 32 concurrent
// tiles share 4 token and 8 row panels in its L2.
constexpr int kBand = 4;
__device__ __forceinline__ void band_tile(int at, int tt, int rt, int &t, int &r) {
  const int band = at / (kBand * rt), b0 = band * kBand, h = min(kBand, tt - b0);
  const int u = at - b0 * rt;
  r = __builtin_amdgcn_readfirstlane(u / h);    // wave-uniform, kept scalar
  t = __builtin_amdgcn_readfirstlane(b0 + u % h);
}
__device__ __forceinline__ void tile_at(int bid, int tt, int rt, int &t, int &r) {
  band_tile(xcd_run(bid, tt * rt), tt, rt, t, r);
}

// 16 (or 4) bytes per lane from `base` + the lane's offset to consecutive LDS from byte
// `lds` on, past the registers.  Inline assembly because the compiler, which cannot
// tell one buffer in LDS from another, would wait for all such copies before every read.
// It does not count them, so it must not have to wait for a load of its own while some are
// on their way: that would be a wait for every copy asked for before the load.
// A load that writes LDS needs a wait state after a scalar write of M0; the compiler, which
// puts it before its own, does not look into assembly.
__device__ __forceinline__ void copy16_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(off), "s"(base) : "m0", "memory");
}
__device__ __forceinline__ void copy4_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :: "s"(lds), "v"(off), "s"(base) : "m0", "memory");
}
// The same from each lane's own address.
__device__ __forceinline__ void copy16_to_lds(const void *from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(lds), "v"(from) : "m0", "memory");
}
// All but this wave's last N copies have landed.
template <int N>
__device__ __forceinline__ void copies_done() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "i"(N) : "memory");
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// A wave's NI x FB result blocks (value(i, j): four rows 16 i + 4 (lane / 16) ..  of
// column 16 j + lane % 16), turned in the wave's own LDS so that what follows
// handles eight consecutive rows of a column: each(c, piece, read) is called for
// every column c < 16 FB and piece < PIECES; read(p, v) gives rows 8 p .. 8 p + 7
// of that column.  Half of the columns at a time, as rows of 16 NI floats whose
// 16-byte pieces are XOR-swizzled against bank conflicts.  The loop over pieces is
// not unrolled: what follows is code once per kernel, not once per block (unrolled,
// a 256 x 256 tile of gate and up took 26 us where it now takes 13).  What each()
// needs from memory, first(c, piece) loads for AHEAD pieces at a time.
// lds: 64 NI * 16 ceil(FB / 2) bytes.
template <int NI, int FB, int PIECES, int AHEAD, typename V, typename G, typename F>
__device__ __forceinline__ void turned(V value, int lane, uint8_t *lds, G first, F each) {
  constexpr int kRow = 64 * NI, kIn = 4 * NI, kHalf = (FB + 1) / 2;
  auto place = [&](int t, int piece) {
    const int x = kIn >= 16 ? t & 15 : kIn == 8 ? (t >> 1) & 7 : (t >> 2) & (kIn - 1);
    return reinterpret_cast<f32x4_t *>(lds + t * kRow + ((piece ^ x) << 4));
  };
#pragma unroll
  for (int j0 = 0; j0 < FB; j0 += kHalf) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < kHalf; ++j)
        if (j0 + j < FB) *place(16 * j + (lane & 15), 4 * i + (lane >> 4)) = value(i, j0 + j);
    wave_lds_fence();
    constexpr int kAll = kHalf * 16 * PIECES;
#pragma unroll 1
    for (int it = 0; it < (kAll + 63) / 64; it += AHEAD) {
      decltype(first(0, 0)) kept[AHEAD];
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) {
        const int at = min((it + n) * 64 + lane, kAll - 1);
        kept[n] = first(min(j0 * 16 + at / PIECES, 16 * FB - 1), at % PIECES);
      }
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) {
        const int at = (it + n) * 64 + lane, t = at / PIECES, piece = at % PIECES;
        if (at >= kAll || j0 * 16 + t >= 16 * FB) continue;
        each(j0 * 16 + t, piece, kept[n], [&](int p, float v[8]) {
          const f32x4_t a = *place(t, 2 * p), b = *place(t, 2 * p + 1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
          }
        });
      }
    }
    wave_lds_fence();
  }
}

// A wave's blocks as they are, to rows r0 .. and columns t0 .. of `out`: rounded to
// T before they are turned, half the LDS traffic of turned().
// lds: 16 NI sizeof(T) * 16 ceil(FB / 2) bytes.
template <typename T, int NI, int FB, typename V>
__device__ __forceinline__ void store_turned(V value, T *out, int64_t ld, int rows, int cols,
                                             int r0, int t0, int lane, uint8_t *lds) {
  constexpr int kRow = 16 * NI * sizeof(T), kPieces = kRow / 16, kHalf = (FB + 1) / 2;
  constexpr int kVals = 16 / sizeof(T), kAll = kHalf * 16 * kPieces;
  auto place = [&](int t, int piece) {
    const int x = kPieces >= 16 ? t & 15 : kPieces == 8 ? (t >> 1) & 7 : (t >> 2) & (kPieces - 1);
    return lds + t * kRow + ((piece ^ x) << 4);
  };
  const int g = lane >> 4;
#pragma unroll
  for (int j0 = 0; j0 < FB; j0 += kHalf) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        if (j0 + j >= FB) break;
        const f32x4_t f = value(i, j0 + j);
        T o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = narrow<T>(f[v]);
        const int byte = (16 * i + 4 * g) * int(sizeof(T));
        __builtin_memcpy(__builtin_assume_aligned(place(16 * j + (lane & 15), byte >> 4) + (byte & 15),
                                                  sizeof(o)), o, sizeof(o));
      }
    wave_lds_fence();
#pragma unroll 4
    for (int it = 0; it < (kAll + 63) / 64; ++it) {
      const int at = it * 64 + lane, t = at / kPieces, piece = at % kPieces;
      if (at >= kAll) continue;
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(place(t, piece));
      const int c = t0 + 16 * j0 + t, r = r0 + piece * kVals, left = rows - r;
      if (c >= cols || left <= 0) continue;
      T *p = out + int64_t(c) * ld + r;
      if (left >= kVals) {
        __builtin_memcpy(p, &v, 16);
      } else {
        T o[kVals];
        __builtin_memcpy(o, &v, 16);
#pragma unroll
        for (int e = 0; e < kVals - 1; ++e)
          if (e < left) p[e] = o[e];
      }
    }
    wave_lds_fence();
  }
}

// Whether two matrices (rows x cols of elements of `size` bytes, ld >= cols between rows) share
// memory; false for a matrix that is not there.  A stride that reaches past the address
// space counts as all that is on the way.
inline bool matrices_meet(const void *a, int64_t rows_a, int64_t cols_a, int64_t ld_a, size_t size_a,
                          const void *b, int64_t rows_b, int64_t cols_b, int64_t ld_b,
                          size_t size_b) {
  if (!a || !b || rows_a < 1 || rows_b < 1) return false;
  // in 128 bits: any stride
  const auto end = [](const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size) {
    return (unsigned __int128)(reinterpret_cast<uintptr_t>(p)) +
           ((unsigned __int128)(rows - 1) * uint64_t(rows > 1 ? ld : 0) + uint64_t(cols)) * size;
  };
  const unsigned __int128 end_a = end(a, rows_a, cols_a, ld_a, size_a);
  const unsigned __int128 end_b = end(b, rows_b, cols_b, ld_b, size_b);
  if (reinterpret_cast<uintptr_t>(a) >= end_b || reinterpret_cast<uintptr_t>(b) >= end_a) return false;
  if (end_a > UINTPTR_MAX || end_b > UINTPTR_MAX) return true;
  return rows_overlap(a, rows_a, (rows_a > 1 ? ld_a : cols_a) * size_a, cols_a * size_a, b, rows_b,
                      (rows_b > 1 ? ld_b : cols_b) * size_b, cols_b * size_b);
}

inline gptq_status check_scratch(const void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return GPTQ_OK;
  if (!ws) return fail(GPTQ_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned_to(ws, 256)) return fail(GPTQ_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need)
    return fail(GPTQ_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) +
                                        " bytes, got " + std::to_string(ws_bytes));
  return GPTQ_OK;
}

}  // namespace gptq
