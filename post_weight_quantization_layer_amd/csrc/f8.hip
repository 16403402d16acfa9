// Layers of 8-bit floats (e4m3) with a scale per 128 x 128 block, on activations
// quantized per token and 128 features: v_mfma_f32_16x16x128_f8f6f4, whose k is one
// block, so each instruction's result is scaled by the two blocks' scales as it is
// added to the float32 sum.  Gate and up of a block go through float16 instructions,
// which keep every product whole.
//
// Prepared layout: tiles of 16 rows x 128 k as the instruction takes them, two
// 1 KiB halves of 64 k; lane l holds row l % 16, k = 16 (l / 16) .. + 15 of
// either half.  (Which k a lane holds does not matter as long as both operands agree.)
#include <algorithm>
#include <iterator>
#include <string>

#include "gptq_ff.h"
#include "silu.h"
#include "tiles.h"

namespace gptq {

gptq_status check_activations(const void *x, int32_t dtype, int64_t tokens, int64_t cols,
                              int64_t ld, const char *what);

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int kStep = 128;       // k per block, tile and instruction
constexpr float kTop = 448.f;    // largest e4m3 value
constexpr uint32_t kFloorBits = 0x0d800000u;    // 2^-100

// ------------------------------------------------------------------- codes
// A block's scale and the factor its values are multiplied by; NaN and 0 for
// a block that holds a NaN or an infinity (their bits exceed every finite
// value's).
struct BlockScale {
  float scale, inv;
  bool usable;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.f, false};
  const float a = __uint_as_float(amax_bits > kFloorBits ? amax_bits : kFloorBits);
  return {a / kTop, kTop / a, true};
}
// |v * inv| <= 448 (1 + 2^-23), which still rounds to 448.
__device__ __forceinline__ u32x2_t codes8(const float v[8], const BlockScale &s) {
  u32x2_t w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * s.inv, v[4 * h + 1] * s.inv, 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * s.inv, v[4 * h + 3] * s.inv, q, true);
    w[h] = s.usable ? uint32_t(q) : 0u;
  }
  return w;
}
__device__ __forceinline__ uint32_t max_bits8(const float v[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = MaxU::op(m, __float_as_uint(v[j]) & 0x7fffffffu);
  return m;
}
// Over 16 consecutive lanes, every one of which gets the value.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = MaxU::op(m, dpp<0xb1>(m));
  m = MaxU::op(m, dpp<0x4e>(m));
  m = MaxU::op(m, dpp<0x141>(m));
  return MaxU::op(m, dpp<0x140>(m));
}

// A wave's turn is 512 features of a token, eight per lane: a block is 16 lanes, whose
// maximum goes round by register moves.  Memory bounds it: 8192 x 8192 bfloat16 42 us (4.8
// TB/s); one token is a launch, 2.5 us.  GATED: of silu(x) u.
template <typename T, Ends E, bool GATED>
__global__ void __launch_bounds__(256)
    f8_quantize_kernel(const T *__restrict__ x, const T *__restrict__ u, int64_t ld, int64_t turns,
                       int chunks, int cols, uint8_t *__restrict__ codes, int64_t ld_codes,
                       float *__restrict__ scale, int64_t ld_scale) {
  const int lane = threadIdx.x & 63;
  for (int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); at < turns;
       at += int64_t(gridDim.x) * 4) {
    const int64_t t = at / chunks;
    const int e0 = (int(at - t * chunks) * 64 + lane) * 8;
    const Pack8<T> kx = fetch8<E>(x + t * ld, e0, cols);
    float v[8];
    if constexpr (GATED) {
      const Pack8<T> ku = fetch8<E>(u + t * ld, e0, cols);
      float w[8];
      widen8<E>(kx, e0, cols, 0.f, v);
      widen8<E>(ku, e0, cols, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * w[j];
    } else {
      widen8<E>(kx, e0, cols, 0.f, v);
    }
    const BlockScale s = block_scale(max16(max_bits8(v, 0u)));
    if (e0 / kStep * kStep >= cols) continue;      // a block past the row
    *reinterpret_cast<u32x2_t *>(codes + t * ld_codes + e0) = codes8(v, s);
    if ((lane & 15) == 0) scale[e0 / kStep * ld_scale + t] = s.scale;
  }
}

// A workgroup per block: a thread eight values of every 16th row, so that the block stays
// in registers between its maximum and its codes and 16 lanes read a row of it.  28672 x
// 8192 bfloat16: 133 us, 5.3 TB/s (two lanes a row 292).
template <typename T, Ends E>
__global__ void __launch_bounds__(256)
    f8_quantize_weight_kernel(const T *__restrict__ w, int64_t ld, int64_t rows, int cols,
                              int col_blocks, uint8_t *__restrict__ codes,
                              float *__restrict__ scale) {
  __shared__ uint32_t slot[4];
  const int64_t block = blockIdx.x, rb = block / col_blocks;
  const int c = int(block - rb * col_blocks) * kStep + (threadIdx.x & 15) * 8, n = cols - c;
  const int64_t r0 = rb * kStep + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    const Pack8<T> k = fetch8<E>(w + (r < rows ? r : rows - 1) * ld, c, cols);
    widen8<E>(k, c, cols, 0.f, v[i]);
    if (r < rows) m = max_bits8(v[i], m);
  }
  const BlockScale s = block_scale(row_all<MaxU, 4>(m, slot));
  if (threadIdx.x == 0) scale[block] = s.scale;
  if (n <= 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r >= rows) break;
    const u32x2_t q = codes8(v[i], s);
    uint8_t *p = codes + r * cols + c;
    if (n >= 8) {
      __builtin_memcpy(p, &q, 8);
    } else {
      for (int e = 0; e < n; ++e) p[e] = uint8_t(q[e >> 2] >> (8 * (e & 3)));
    }
  }
}

// ----------------------------------------------------------------- prepare
struct Geometry {
  int64_t rows, cols, rows_pad, k_pad;
};
Geometry geometry(int64_t rows, int64_t cols) {
  return {rows, cols, (rows + 15) / 16 * 16, (cols + kStep - 1) / kStep * kStep};
}
// Codes, then the scales, a row of blocks after the other.
struct LayerMap {
  uint8_t *w;
  float *scale;
  size_t bytes;
};
LayerMap layer_map(void *mem, const Geometry &g) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(mem);    // 0 where only the size is asked
  const size_t codes = align256(size_t(g.rows_pad) * g.k_pad);
  const size_t scales = align256(size_t(cdiv(g.rows, kStep)) * (g.k_pad / kStep) * 4);
  return {reinterpret_cast<uint8_t *>(p), reinterpret_cast<float *>(p + codes), codes + scales};
}

// One 16-byte piece per thread: row 16 rt + l % 16, k from 128 step + 64 half +
// 16 (l / 16).  Rows and columns past the layer are 0.  28672 x 8192: 75 us, 6.3 TB/s.
__global__ void __launch_bounds__(256)
    f8_repack_kernel(const uint8_t *__restrict__ q, int64_t rows, int64_t cols, int64_t pieces,
                     int64_t steps, u32x4_t *__restrict__ w) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int l = int(i & 63), half = int((i >> 6) & 1);
  const int64_t tile = i >> 7, step = tile % steps, rt = tile / steps;
  const int64_t r = rt * 16 + (l & 15), k = step * kStep + half * 64 + (l >> 4) * 16;
  u32x4_t v = {0, 0, 0, 0};
  if (r < rows && k < cols) {
    const uint8_t *p = q + r * cols + k;
    if (k + 16 <= cols) {
      __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (k + b < cols) v[b >> 2] |= uint32_t(p[b]) << (8 * (b & 3));
    }
  }
  w[i] = v;
}
__global__ void __launch_bounds__(256)
    f8_scales_kernel(const float *__restrict__ from, int64_t n, float *__restrict__ to) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) to[i] = from[i];
}

// ----------------------------------------------------------------- product
// kExact: gate's and up's products, to float32.  kGated: both and v's codes.  Either with sums
// to 32 bits.
enum Mode { kPlain, kExact, kGated };

struct GemmArgs {
  const uint8_t *w, *w2;           // kGated: gate and up
  const float *w_scale, *w2_scale;
  const uint8_t *x;                // codes, or floats (rows kernel)
  const float *x_scale;
  void *y, *y2;                    // kPlain, kExact; y2 of w2 where there are two problems
  uint8_t *v;                      // kGated: codes of v and their scales
  float *v_scale;
  int64_t ld_x, ld_xs, ld_y, ld_v, ld_vs;
  int tokens, rows, cols, row_tiles, steps, y_type, problems;
  f32x4_t *part;                   // split products: the blocks of each (tile, split)
  int splits;
};

__device__ __forceinline__ f32x4_t block_product(i32x4_t a0, i32x4_t a1, i32x4_t b0, i32x4_t b1) {
  const i32x8_t a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
  const i32x8_t b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
}
// The same with sums to 32 bits: the codes as float16, which holds them, so that every
// product is kept whole.  The 8-bit instruction keeps, of each eight products, 13 bits below
// the largest one's leading bit: 1.3e-5 of a sum's size, which is nothing next to a
// 16-bit result's rounding, but what becomes a code of v (gate and up) may be one step
// of 2^-3 off then: with it 2e-4 of them were, 1.5e-3 of y.  So gate and up take this form at
// every size.  Four instructions of half the work, and conversions that an operand's other
// blocks share: 5 tokens x 4096 x 11008 take 15.2 us in place of 14.5, 301 x 1001 x 2731 15.5
// in place of 12, 2048 x 4096 x 11008 297 in place of 183.
struct Wide {
  f16x8_t h[4];
};
__device__ __forceinline__ Wide widen_codes(i32x4_t a0, i32x4_t a1) {
  Wide w;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = (q < 2 ? a0 : a1)[2 * (q & 1) + e];
      const f16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.f, false);
      const f16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.f, true);
      w.h[q][4 * e] = lo[0];
      w.h[q][4 * e + 1] = lo[1];
      w.h[q][4 * e + 2] = hi[0];
      w.h[q][4 * e + 3] = hi[1];
    }
  return w;
}
__device__ __forceinline__ f32x4_t block_product(const Wide &a, const Wide &b) {
  f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[q], b.h[q], p, 0, 0, 0);
  return p;
}
__device__ __forceinline__ void add_scaled(f32x4_t &acc, f32x4_t p, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
  asm volatile("" : "+v"(acc));     // here, not where the sum is next used
}

template <int FA, int FB, Mode M>
__device__ __forceinline__ void store_blocks(const GemmArgs &a, const f32x4_t (&acc)[FA][FB],
                                             void *y, int t0, int r0, int lane, uint8_t *lds) {
  auto value = [&](int i, int j) { return acc[i][j]; };
  auto go = [&](auto *y) {
    store_turned<std::remove_pointer_t<decltype(y)>, FA, FB>(value, y, a.ld_y, a.rows, a.tokens,
                                                             r0, t0, lane, lds);
  };
  if constexpr (M == kExact) go(static_cast<float *>(y));
  else if (a.y_type == GPTQ_DT_BF16) go(static_cast<bf16_t *>(y));
  else go(static_cast<f16_t *>(y));
}

__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// v = silu(g) u of a tile of gate and up, as codes.  A wave holds 8 FA rows of v (its
// first half of FA blocks is of gate, the second of up) of 16 FB tokens; WM waves
// make the 128 rows of a block of v, so a token's largest magnitude is found within the
// workgroup: over a lane's values, four lanes, and the WM waves through LDS.
template <int WM, int WN, int FA, int FB>
__device__ __forceinline__ void finish_gated(const GemmArgs &a, f32x4_t (&acc)[FA][FB], int r0,
                                             int t0, int wm, int wn, int lane, uint8_t *smem) {
  constexpr int H = FA / 2, kTokens = 16 * FB * WN;
  static_assert(16 * H * WM == kStep, "a tile is one block of v");
  uint32_t *tops = reinterpret_cast<uint32_t *>(smem + kTokens * kStep);
  const int g = lane >> 4, mine = wm * 16 * H + 4 * g;      // rows within the block
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = silu(acc[i][j][e]) * acc[H + i][j][e];
        acc[i][j][e] = r0 + mine + 16 * i + e < a.rows ? v : 0.f;    // zeros fill the pad
        top = MaxU::op(top, __float_as_uint(acc[i][j][e]) & 0x7fffffffu);
      }
    top = MaxU::op(top, uint32_t(__shfl_xor(int(top), 16)));
    top = MaxU::op(top, uint32_t(__shfl_xor(int(top), 32)));
    if (g == 0) tops[wm * kTokens + (wn * FB + j) * 16 + lane] = top;
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    const int t = (wn * FB + j) * 16 + (lane & 15);
    uint32_t top = tops[t];
#pragma unroll
    for (int m = 1; m < WM; ++m) top = MaxU::op(top, tops[m * kTokens + t]);
    const BlockScale s = block_scale(top);
    if (wm == 0 && g == 0 && t0 + t < a.tokens)
      a.v_scale[int64_t(r0 / kStep) * a.ld_vs + t0 + t] = s.scale;
    // four rows of a token are a word; 16-byte pieces of a token's 128 bytes are swizzled
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const f32x4_t v = acc[i][j];
      int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * s.inv, v[1] * s.inv, 0, false);
      q = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * s.inv, v[3] * s.inv, q, true);
      const int at = mine + 16 * i;
      *reinterpret_cast<int *>(smem + t * kStep + (((at >> 4) ^ (t & 7)) << 4) + (at & 15)) =
          s.usable ? q : 0;
    }
  }
  lds_barrier();
  const int tid = threadIdx.x;
#pragma unroll 1
  for (int at = tid; at < kTokens * 8; at += 64 * WM * WN) {
    const int t = at >> 3, piece = at & 7;
    if (t0 + t < a.tokens)
      *reinterpret_cast<u32x4_t *>(a.v + int64_t(t0 + t) * a.ld_v + r0 + piece * 16) =
          *reinterpret_cast<const u32x4_t *>(smem + t * kStep + ((piece ^ (t & 7)) << 4));
  }
}

// ---- Tiles through LDS.  WM x WN waves make a tile of 16 FA WM rows x 16 FB WN
// tokens, each FA x FB blocks of 16 x 16.  Every product of two blocks of 128 k
// comes out of the matrix unit on its own and is added to the sums with its scales
// by vector instructions, so the sums lie in vector registers: 128 of a wave's 256 for
// FA FB = 32, eight waves per compute unit, of which two share a SIMD and overlap
// one's matrix instructions with the other's additions.
//
// Stages of 128 k lie in a ring of NBUF buffers in LDS, copied there by loads that
// write LDS directly (no registers): weights in the prepared order, tokens as 128-byte
// rows whose 16-byte pieces are XOR-swizzled on the way, the tokens' scales.  The
// weights' scales of the whole range of k are read first.  A wave holds the stage's
// token fragments and a ring of four weight fragments, two ahead of use.  Once the last
// two are read, two fragments before the stage's end, a barrier tells that every
// wave has read stage u and that stage u + 1 is there: while the last products of u are
// made, stage u + NBUF is asked for, into u's buffer, and u + 1's first fragments are
// read, a copy or two per product (all of them in a row after the barrier, where every
// wave is at once, took 8192 x 28672 x 8192 from 1650 us to 1726).  A product is added
// three products later, across the stage's end.  256 x 256 tiles have room for two buffers;
// 128 x 64 tiles, whose stages are shorter than a memory access, take four.
// (With scales loaded in the loop 8192 x 28672 x 8192 took 1881 us, without waits for
// them 1753.)  In 62 % of its cycles the matrix units are busy, at 1.88 GHz.
constexpr int kMaxSteps = 65536 / kStep;
// Bytes of a stage, and of LDS in all.
constexpr int stage_bytes(int wm, int wn, int fa, int fb) {
  return 2048 * fa * wm + 16 * fb * wn * (kStep + 4);
}
constexpr int scale_rows(int wm, int fa, Mode m) { return m == kGated ? 2 : (16 * fa * wm + 127) / 128; }
constexpr int tile_lds(int wm, int wn, int fa, int fb, int nbuf, Mode m) {
  return nbuf * stage_bytes(wm, wn, fa, fb) + scale_rows(wm, fa, m) * kMaxSteps * 4;
}

template <int WM, int WN, int FA, int FB, int NBUF, Mode M>
__global__ void __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(1, FA * FB >= 16 ? 2 : 3)))
    f8_tile_kernel(GemmArgs a, int token_tiles, int row_tiles) {
  constexpr int kWaves = WM * WN, kTiles = FA * WM;       // 16-row tiles of weights per stage
  constexpr int kTokens = 16 * FB * WN;
  constexpr int kWBytes = 2048 * kTiles, kXBytes = kTokens * kStep;
  constexpr int kStageBytes = stage_bytes(WM, WN, FA, FB);
  constexpr int kWCopies = 2 * kTiles / kWaves;           // KiB of weights per wave and stage
  constexpr int kXCopies = kXBytes / 1024 / kWaves;       // eight tokens' rows each
  constexpr int kCopies = kWCopies + kXCopies + 1;        // one of scales
  constexpr int kOut = M == kGated ? kTiles / 2 : kTiles; // tiles of rows of the result
  extern __shared__ __align__(16) uint8_t smem[];
  float *const w_scales = reinterpret_cast<float *>(smem + NBUF * kStageBytes);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = token_tiles * row_tiles;
  const int at = xcd_run(int(blockIdx.x), tiles * a.splits * a.problems);
  const int unit = __builtin_amdgcn_readfirstlane(at / tiles), tile = at - unit * tiles;
  const bool second = unit >= a.splits;    // the second problem: w2 -> y2
  const int split = second ? unit - a.splits : unit;
  const uint8_t *const w_of = second ? a.w2 : a.w;
  const float *const w_scale_of = second ? a.w2_scale : a.w_scale;
  int tt, tr;
  band_tile(tile, token_tiles, row_tiles, tt, tr);
  const int rt0 = tr * kOut, t0 = tt * kTokens;
  const int s0 = int(int64_t(a.steps) * split / a.splits);
  const int U = int(int64_t(a.steps) * (split + 1) / a.splits) - s0;

  // Tile i of wave row m: of gate for the first half of FA, then of up.  Rows past
  // the layer or the tokens are clamped; they only feed outputs that are not stored.
  auto tile_row = [&](int m, int i) {
    return min(rt0 + (M == kGated ? m * (FA / 2) + i % (FA / 2) : m * FA + i), a.row_tiles - 1);
  };
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t *)smem));
  const uint8_t *wsrc[kWCopies];
#pragma unroll
  for (int q = 0; q < kWCopies; ++q) {
    const int kib = wave * kWCopies + q, t = kib >> 1, m = t / FA, i = t % FA;
    const uint8_t *w = M == kGated && i >= FA / 2 ? a.w2 : w_of;
    wsrc[q] = w + (int64_t(tile_row(m, i)) * a.steps + s0) * 2048 + (kib & 1) * 1024;
  }
  const uint8_t *xsrc = a.x + int64_t(t0) * a.ld_x + int64_t(s0) * kStep;
  const uint8_t *ssrc = reinterpret_cast<const uint8_t *>(a.x_scale + int64_t(s0) * a.ld_xs + t0);
  uint32_t xoff[kXCopies];
#pragma unroll
  for (int q = 0; q < kXCopies; ++q) {
    const int row = (wave * kXCopies + q) * 8 + (lane >> 3);
    xoff[q] = uint32_t(min(row, a.tokens - 1 - t0)) * uint32_t(a.ld_x) +
              (((lane & 7) ^ swz(row)) << 4);
  }
  // 64 tokens' scales; where there are more waves, two write the same
  const int sblock = wave % (kTokens / 64);
  const uint32_t soff = 4 * uint32_t(min(64 * sblock + lane, a.tokens - 1 - t0)), woff = lane * 16;
  // Copies from .. to - 1 of a stage; past the last stage: of that one again, not read.
  auto copy_part = [&](int u, int buf, int from, int to) {
    const int64_t at = min(u, U - 1);
    const uint32_t lds = lds0 + buf * kStageBytes;
#pragma unroll
    for (int c = from; c < to; ++c) {
      if (c < kWCopies)
        copy16_to_lds(wsrc[c] + at * 2048, woff, lds + (wave * kWCopies + c) * 1024);
      else if (c < kWCopies + kXCopies)
        copy16_to_lds(xsrc + at * kStep, xoff[c - kWCopies],
                      lds + kWBytes + (wave * kXCopies + c - kWCopies) * 1024);
      else
        copy4_to_lds(ssrc + at * a.ld_xs * 4, soff, lds + kWBytes + kXBytes + 256 * sblock);
    }
  };

  struct Frag {
    i32x4_t h[2];
  };
  auto frag_w = [&](int buf, int i) {
    const uint8_t *p = smem + buf * kStageBytes + (wm * FA + i) * 2048 + lane * 16;
    return Frag{{*reinterpret_cast<const i32x4_t *>(p),
                 *reinterpret_cast<const i32x4_t *>(p + 1024)}};
  };
  auto frag_x = [&](int buf, int j) {
    const int row = (wn * FB + j) * 16 + (lane & 15), c = lane >> 4;
    const uint8_t *p = smem + buf * kStageBytes + kWBytes + row * kStep;
    return Frag{{*reinterpret_cast<const i32x4_t *>(p + ((c ^ swz(row)) << 4)),
                 *reinterpret_cast<const i32x4_t *>(p + (((c + 4) ^ swz(row)) << 4))}};
  };
  auto token_scale = [&](int buf, int j) {
    return *reinterpret_cast<const float *>(smem + buf * kStageBytes + kWBytes + kXBytes +
                                            ((wn * FB + j) * 16 + (lane & 15)) * 4);
  };
  const float *const my_scales =
      w_scales + (M == kGated ? 0 : (wm * FA * 16 / kStep) * kMaxSteps);

  // The weights' scales first: these loads are waited for before any copy.
  for (int n = tid; n < scale_rows(WM, FA, M) * U; n += 64 * kWaves) {
    const int row = n / U, u = n - row * U;
    const int rb = min(rt0 / 8 + (M == kGated ? 0 : row), (a.row_tiles - 1) / 8);
    w_scales[row * kMaxSteps + u] =
        (M == kGated && row ? a.w2_scale : w_scale_of)[int64_t(rb) * a.steps + s0 + u];
  }
  f32x4_t acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  copies_done<0>();
#pragma unroll
  for (int u = 0; u < NBUF; ++u) copy_part(u, u, 0, kCopies);
  copies_done<(NBUF - 1) * kCopies>();
  lds_barrier();
  Frag fw[4], fx[FB];
  // The factors of the stage's blocks (M == kGated: of gate's and of up's), which the last
  // three products' additions still need in the next stage, and the scales they are made of.
  constexpr int kSides = M == kGated ? 2 : 1;
  float m[kSides][FB] = {}, next[FB], next_w[kSides];
  auto weight_scales = [&](int u) {
#pragma unroll
    for (int i = 0; i < kSides; ++i) next_w[i] = my_scales[i * kMaxSteps + min(u, U - 1)];
  };
  // Sums to 32 bits on more than two columns fill the registers with widened tokens: rows then
  // go in order to the last, so that one row's widened weights are held at a time; weights are
  // read one row ahead, not two, and scales when the stage starts.  (2048 tokens, 4096 x
  // 11008: 297 us; columns in groups of two, which widens the weights twice, 345.)
  constexpr bool kWide = M != kPlain, kFull = kWide && FB > 2;
  weight_scales(0);
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    fx[j] = frag_x(0, j);
    next[j] = token_scale(0, j);
  }
  fw[0] = frag_w(0, 0);
  fw[1] = frag_w(0, 1);

  // Product n of a stage: the blocks in the rows' order, but (kFull: to the end) the last two
  // rows' in pairs, so that the tokens' fragments become free one after the other.
  constexpr int kProducts = FA * FB, kTail = 2 * FB, kMain = kProducts - kTail;
  auto row = [](int n) { return kFull || n < kMain ? n / FB : FA - 2 + (n - kMain) % 2; };
  auto col = [](int n) { return kFull || n < kMain ? n % FB : (n - kMain) / 2; };
  f32x4_t p[4] = {};
  Wide wide_x[kWide ? FB : 1];             // of the stage
  Wide wide_w[kFull ? 1 : 2];              // of the row, and the one before it
  int buf = 0;                             // u % NBUF
  for (int u = 0; u < U; ++u) {
    const int after = buf + 1 == NBUF ? 0 : buf + 1;
    auto multiply = [&](int n) {
      const Frag &w = fw[row(n) % 4], &x = fx[col(n)];
      if constexpr (kWide) {
        const int of = kFull ? 0 : row(n) % 2;
        if (row(n) == 0) wide_x[col(n)] = widen_codes(x.h[0], x.h[1]);
        if (col(n) == 0) wide_w[of] = widen_codes(w.h[0], w.h[1]);
        p[n % 4] = block_product(wide_w[of], wide_x[col(n)]);
      } else {
        p[n % 4] = block_product(w.h[0], w.h[1], x.h[0], x.h[1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // The product three before n; of the first three, of the stage before.
    auto add_before = [&](int n) {
      const int b = (n + kProducts - 3) % kProducts;
      add_scaled(acc[row(b)][col(b)], p[b % 4], m[row(b) >= FA / 2 ? kSides - 1 : 0][col(b)]);
      __builtin_amdgcn_sched_barrier(0);
      if (n == 2) {
#pragma unroll
        for (int i = 0; i < kSides; ++i)
#pragma unroll
          for (int j = 0; j < FB; ++j) m[i][j] = next[j] * next_w[i];
      }
    };
    static_assert(kProducts % 4 == 0 && FA % 4 == 0, "the products' places go round");
#pragma unroll
    for (int n = 0; n < kMain; ++n) {
      if (kFull && n == 0) {
#pragma unroll
        for (int j = 0; j < FB; ++j) next[j] = token_scale(buf, j);
        weight_scales(u);
      }
      if (!kFull && n % FB == 0) fw[(n / FB + 2) % 4] = frag_w(buf, n / FB + 2);
      multiply(n);
      if (kFull && n % FB == 0) fw[(n / FB + 1) % 4] = frag_w(buf, n / FB + 1);
      add_before(n);
    }
    if (kFull) fw[(FA - 1) % 4] = frag_w(buf, FA - 1);
    copies_done<(NBUF - 2) * kCopies>();
    lds_barrier();
    if (!kFull) {
      fw[0] = frag_w(after, 0);            // past the last stage: read, not used
      fw[1] = frag_w(after, 1);
    }
#pragma unroll
    for (int t = 0; t < kTail; ++t) {
      multiply(kMain + t);
      copy_part(u + NBUF, buf, t * kCopies / kTail, (t + 1) * kCopies / kTail);
      add_before(kMain + t);
      if (kFull) {
        if (t >= FB) fx[t - FB] = frag_x(after, t - FB);
        if (t == FB) fw[0] = frag_w(after, 0);
      } else {
        if (t % 2) fx[t / 2] = frag_x(after, t / 2);
        else next[t / 2] = token_scale(after, t / 2);
        if (t == 0) weight_scales(u + 1);
      }
    }
    buf = after;
  }
#pragma unroll
  for (int n = kProducts - 3; n < kProducts; ++n)
    add_scaled(acc[row(n)][col(n)], p[n % 4], m[kSides - 1][col(n)]);
  copies_done<0>();                        // none may land in what follows
  if (a.splits > 1) {
    // A wave's blocks as they lie in its registers: 1 KiB per store.
    f32x4_t *to = a.part + int64_t(second ? tiles + tile : tile) * a.splits *
                               (kWaves * FA * FB * 64) +
                  (split * kWaves + wave) * (FA * FB * 64) + lane;
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) to[(i * FB + j) * 64] = acc[i][j];
    return;
  }
  lds_barrier();                           // every wave is done with the stages
  if constexpr (M == kGated) {
    finish_gated<WM, WN, FA, FB>(a, acc, rt0 * 16, t0, wm, wn, lane, smem);
  } else {
    store_blocks<FA, FB, M>(a, acc, second ? a.y2 : a.y, t0 + wn * 16 * FB, (rt0 + wm * FA) * 16, lane,
                         smem + wave * (64 * FA * 16 * ((FB + 1) / 2)));
  }
}

// Adds a split product's parts, in their order: a wave per block of rows of a tile's
// wave, in the tile kernel's register order.  A launch and the parts' way through the caches:
// 64 x 4096 k 11008 in parts 4.5 us.
template <int WM, int WN, int FA, int FB, Mode M>
__global__ void __launch_bounds__(256) f8_join_kernel(GemmArgs a, int token_tiles, int row_tiles) {
  constexpr int kWaves = WM * WN, kPiece = 64 * 16 * ((FB + 1) / 2);
  __shared__ __align__(16) uint8_t lds[4 * kPiece];
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int i = unit % FA, wave = unit / FA % kWaves, tile = unit / (kWaves * FA);
  const int tiles = token_tiles * row_tiles;
  const bool second = tile >= tiles;
  int tt, tr;
  band_tile(second ? tile - tiles : tile, token_tiles, row_tiles, tt, tr);
  const int r0 = ((tr * WM + wave / WN) * FA + i) * 16;
  const int t0 = (tt * WN + wave % WN) * FB * 16;
  if (r0 >= a.rows || t0 >= a.tokens) return;
  const f32x4_t *p = a.part + int64_t(tile) * a.splits * (kWaves * FA * FB * 64) +
                     (wave * FA + i) * (FB * 64) + lane;
  f32x4_t acc[1][FB];
#pragma unroll
  for (int j = 0; j < FB; ++j) acc[0][j] = p[j * 64];
  for (int s = 1; s < a.splits; ++s) {
    p += kWaves * FA * FB * 64;
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[0][j] += p[j * 64];
  }
  store_blocks<1, FB, M>(a, acc, second ? a.y2 : a.y, t0, r0, lane, lds + (threadIdx.x >> 6) * kPiece);
}

// ---- Few tokens: a workgroup per 16 rows, its waves splitting k.  A wave takes
// every WAVES-th 128-k step; its weights come straight from memory as contiguous
// KiB, several steps ahead, and each is used for all tokens at once.  The waves' sums
// meet in LDS.  W weights of one shape (gate and up) share the activations.  Memory bounds
// it: 1 token x 4096 x 11008 9.1 us, 5 tokens through two weights of 11008 x 4096 15.6 us (4.9
// and 5.8 TB/s of codes).
//
// T = uint8_t: the activations are codes.  Otherwise they are floats, and every
// workgroup makes all their codes first, in LDS, while its first weights are on their
// way: a launch less.
constexpr int kRowsWaves = 4;
constexpr int64_t kRowsTokens = 16;

// A token's codes in LDS start 64 bytes further round the banks than the one's before.
constexpr int kRowsPad = 64;
__host__ __device__ constexpr int rows_stride(int steps) { return steps * kStep + kRowsPad; }

template <int W, typename T>
__global__ void __launch_bounds__(64 * kRowsWaves) __attribute__((amdgpu_waves_per_eu(W == 2 ? 2 : 3)))
    f8_rows_kernel(GemmArgs a) {
  constexpr bool kCodes = __is_same(T, uint8_t);
  constexpr int WAVES = kRowsWaves, kThreads = 64 * WAVES;
  constexpr int kAhead = W == 1 ? 4 : 2;    // steps loaded at a time, two such sets in flight
  __shared__ f32x4_t sums[W * WAVES * 64];
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rt = blockIdx.x;
  // This wave's steps: wave, wave + WAVES, ...  Loads past the last repeat it.
  const int n = (a.steps - wave + WAVES - 1) / WAVES;
  const uint8_t *w[W];
  const float *ws[W];
#pragma unroll
  for (int m = 0; m < W; ++m) {
    w[m] = (m ? a.w2 : a.w) + int64_t(rt) * a.steps * 2048 + lane * 16;
    ws[m] = (m ? a.w2_scale : a.w_scale) + int64_t(rt / 8) * a.steps;
  }
  const int token = min(lane & 15, a.tokens - 1), stride = rows_stride(a.steps);
  float *const scales = reinterpret_cast<float *>(smem + a.tokens * stride);
  const uint8_t *xrow;
  const float *xs;
  if constexpr (kCodes) {
    xrow = a.x + int64_t(token) * a.ld_x + (lane >> 4) * 16;
    xs = a.x_scale + token;
  } else {
    xrow = smem + token * stride + (lane >> 4) * 16;
    xs = scales + token * a.steps;
  }
  struct Set {
    i32x4_t w[kAhead][W][2], x[kAhead][2];
    float s[kAhead], ws[kAhead][W];
  };
  auto step_of = [&](int at) { return wave + min(at, n - 1) * WAVES; };
  auto load_w = [&](Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t s = step_of(at + i);
#pragma unroll
      for (int m = 0; m < W; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b.w[i][m][h] = *reinterpret_cast<const i32x4_t *>(w[m] + s * 2048 + h * 1024);
        b.ws[i][m] = ws[m][s];
      }
    }
  };
  auto load_x = [&](Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t s = step_of(at + i);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b.x[i][h] = *reinterpret_cast<const i32x4_t *>(xrow + s * kStep + h * 64);
      b.s[i] = xs[kCodes ? s * a.ld_xs : s];
    }
  };
  f32x4_t acc[W];
#pragma unroll
  for (int m = 0; m < W; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](Set &b, int at) {
    if constexpr (!kCodes) load_x(b, at);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (at + i >= n) break;
      if constexpr (W == 2) {
        const Wide x = widen_codes(b.x[i][0], b.x[i][1]);
#pragma unroll
        for (int m = 0; m < W; ++m)
          add_scaled(acc[m], block_product(widen_codes(b.w[i][m][0], b.w[i][m][1]), x),
                     b.s[i] * b.ws[i][m]);
      } else {
        add_scaled(acc[0], block_product(b.w[i][0][0], b.w[i][0][1], b.x[i][0], b.x[i][1]),
                   b.s[i] * b.ws[i][0]);
      }
    }
  };
  auto load = [&](Set &b, int at) {
    load_w(b, at);
    if constexpr (kCodes) load_x(b, at);
  };
  Set s0, s1;
  if constexpr (!kCodes) {
    // Eight values per lane and turn: a block is 16 lanes.  The first batch of turns is
    // asked for before the weights, so that it can be waited for without them.
    constexpr int kBatch = 8;
    const int chunks = a.steps * (kStep / 8), all = a.tokens * chunks;
    Pack8<T> k[kBatch];
    auto fetch = [&](int first) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = min(first + i * kThreads + tid, all - 1), t = at / chunks;
        const int e0 = (at - t * chunks) * 8;
        const T *p = reinterpret_cast<const T *>(a.x) + int64_t(t) * a.ld_x;
        k[i] = Pack8<T>{};
        if (e0 + 8 <= a.cols) {
          __builtin_memcpy(&k[i], p + e0, sizeof(k[i]));
        } else {
          T v[8] = {};
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e0 + e < a.cols) v[e] = p[e0 + e];
          __builtin_memcpy(&k[i], v, sizeof(v));
        }
      }
    };
    fetch(0);
    if (n > 0) {
      load_w(s0, 0);
      load_w(s1, kAhead);
    }
    for (int first = 0;;) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = first + i * kThreads + tid;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k[i].at(e);
        const BlockScale s = block_scale(max16(max_bits8(v, 0u)));
        if (at >= all) continue;
        const int t = at / chunks, c = at - t * chunks;
        *reinterpret_cast<u32x2_t *>(smem + t * stride + c * 8) = codes8(v, s);
        if ((c & 15) == 0) scales[t * a.steps + c / 16] = s.scale;
      }
      first += kBatch * kThreads;
      if (first >= all) break;
      fetch(first);
    }
    lds_barrier();
  } else if (n > 0) {
    load(s0, 0);
    load(s1, kAhead);
  }
  for (int at = 0; at < n; at += 2 * kAhead) {
    multiply(s0, at);
    if (at + 2 * kAhead < n) load(s0, at + 2 * kAhead);
    multiply(s1, at + kAhead);
    if (at + 3 * kAhead < n) load(s1, at + 3 * kAhead);
  }
#pragma unroll
  for (int m = 0; m < W; ++m) sums[(m * WAVES + wave) * 64 + lane] = acc[m];
  lds_barrier();
  // Output (token, row) of thread: 16 consecutive rows per token.  Lane
  // 16 (r / 4) + t of a block holds rows 4 (r / 4) .. + 3 of token t.
  const float *flat = reinterpret_cast<const float *>(sums);
  const int t = tid >> 4, r = tid & 15, row = rt * 16 + r;
  const int from = (16 * (r >> 2) + t) * 4 + (r & 3);
  if (t >= a.tokens || row >= a.rows) return;
  float y[W];
#pragma unroll
  for (int m = 0; m < W; ++m) {
    y[m] = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) y[m] += flat[(m * WAVES + i) * 256 + from];
  }
  if constexpr (W == 2) y[0] = silu(y[0]) * y[W - 1];
  const int64_t to = int64_t(t) * a.ld_y + row;
  if (W == 2) static_cast<float *>(a.y)[to] = y[0];
  else if (a.y_type == GPTQ_DT_BF16) static_cast<bf16_t *>(a.y)[to] = narrow<bf16_t>(y[0]);
  else static_cast<f16_t *>(a.y)[to] = narrow<f16_t>(y[0]);
}

// -------------------------------------------------------------------- host
constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxTokens = int64_t(1) << 20;
// A launch has at most 2^32 threads; a thread repacks 16 codes.
constexpr int64_t kMaxCodes = int64_t(1) << 35;

gptq_status check_layer(const gptq_f8_layer *l) {
  if (!l || !l->mem || gptq_f8_layer_bytes(l->rows, l->cols) == 0 ||
      l->mem_bytes < gptq_f8_layer_bytes(l->rows, l->cols))
    return fail(GPTQ_ERR_INVALID_ARG, "layer is not prepared");
  return GPTQ_OK;
}
gptq_status check_output(const void *y, int32_t y_dtype, int64_t ld_y, int64_t rows) {
  if (!y) return fail(GPTQ_ERR_INVALID_ARG, "y must not be NULL");
  if (y_dtype != GPTQ_DT_BF16 && y_dtype != GPTQ_DT_F16)
    return fail(GPTQ_ERR_INVALID_ARG, "y's type must be BF16 or F16");
  if (!aligned_to(y, 2)) return fail(GPTQ_ERR_INVALID_ARG, "y must be aligned to its elements");
  if (ld_y < rows) return fail(GPTQ_ERR_INVALID_ARG, "ld_y must be >= rows");
  return GPTQ_OK;
}
gptq_status check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens must be in [0, 2^20]");
  return GPTQ_OK;
}
gptq_status check_codes(const uint8_t *codes, int64_t ld_codes, const float *scale,
                        int64_t ld_scale, int64_t tokens, int64_t cols) {
  if (!codes || !scale)
    return fail(GPTQ_ERR_INVALID_ARG, "codes and scale must not be NULL");
  if (!aligned_to(codes, 16) || ld_codes % 16 || ld_codes < gptq_tokens_ld(cols) ||
      ld_codes > (int64_t(1) << 22))
    return fail(GPTQ_ERR_INVALID_ARG,
                "codes must be 16-byte aligned, ld_codes a multiple of 16 in "
                "[gptq_tokens_ld(cols), 2^22]");
  if (!aligned_to(scale, 4)) return fail(GPTQ_ERR_INVALID_ARG, "scale must be 4-byte aligned");
  if (ld_scale < tokens) return fail(GPTQ_ERR_INVALID_ARG, "ld_scale must be >= tokens");
  return GPTQ_OK;
}

template <typename T, bool GATED>
gptq_status quantize_typed(const void *x, const void *u, int64_t tokens, int64_t cols, int64_t ld,
                           uint8_t *codes, int64_t ld_codes, float *scale, int64_t ld_scale,
                           hipStream_t s) {
  const int chunks = int(cdiv(cols, 512));
  const int64_t turns = tokens * chunks;
  const Ends e = ends_of(cols);
  auto kern = e == kWhole ? f8_quantize_kernel<T, kWhole, GATED>
              : e == kRagged ? f8_quantize_kernel<T, kRagged, GATED>
                             : f8_quantize_kernel<T, kShort, GATED>;
  return launch(GATED ? "f8_silu_mul_quantize" : "f8_quantize_tokens", kern,
                dim3(uint32_t(std::min<int64_t>(cdiv(turns, 4), 1 << 22))), dim3(256), 0, s,
                static_cast<const T *>(x), static_cast<const T *>(u), ld, turns, chunks, int(cols), codes, ld_codes, scale,
                ld_scale);
}
gptq_status quantize(const void *x, int32_t dtype, int64_t tokens, int64_t cols, int64_t ld,
                     uint8_t *codes, int64_t ld_codes, float *scale, int64_t ld_scale,
                     hipStream_t s) {
  if (dtype == GPTQ_DT_F32)
    return quantize_typed<float, false>(x, nullptr, tokens, cols, ld, codes, ld_codes, scale,
                                        ld_scale, s);
  if (dtype == GPTQ_DT_BF16)
    return quantize_typed<bf16_t, false>(x, nullptr, tokens, cols, ld, codes, ld_codes, scale,
                                         ld_scale, s);
  return quantize_typed<f16_t, false>(x, nullptr, tokens, cols, ld, codes, ld_codes, scale,
                                      ld_scale, s);
}

template <typename T>
gptq_status quantize_weight_typed(const void *w, int64_t ld, int64_t rows, int64_t cols,
                                  uint8_t *codes, float *scale, hipStream_t s) {
  const int64_t cb = cdiv(cols, kStep), blocks = cdiv(rows, kStep) * cb;
  const Ends e = ends_of(cols);
  auto kern = e == kWhole ? f8_quantize_weight_kernel<T, kWhole>
              : e == kRagged ? f8_quantize_weight_kernel<T, kRagged>
                             : f8_quantize_weight_kernel<T, kShort>;
  return launch("f8_quantize_weight", kern, dim3(uint32_t(blocks)), dim3(256), 0, s,
                static_cast<const T *>(w), ld, rows, int(cols), int(cb), codes, scale);
}

// A token's codes and scales as a call keeps them in scratch.
struct Codes {
  uint8_t *codes;
  float *scale;
  int64_t ld;
  size_t bytes;
};
Codes codes_at(void *mem, int64_t tokens, int64_t cols) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(mem);
  const int64_t ld = gptq_tokens_ld(cols);
  const size_t n = align256(size_t(tokens) * ld);
  return {reinterpret_cast<uint8_t *>(p), reinterpret_cast<float *>(p + n), ld,
          n + align256(size_t(tokens) * (ld / kStep) * 4)};
}

// ------------------------------------------------------------- launch rules
// Whether the rows kernel makes the codes of `tokens` floats itself.  Each workgroup
// does, so it pays where the launch it saves is long against the work (us, in the
// kernel / with a launch before it): 4096 x 4096 1 token 7.9 / 11.4, 4 tokens 9.1 / 11.4,
// 5 tokens 12.0 / 11.3; 4096 x 11008 1 token 15.6 / 14.5; 14336 x 4096 1 token 16.2 / 14.4.
bool rows_floats(const Geometry &g, int64_t tokens) {
  return tokens <= kRowsTokens && g.k_pad <= 4096 && tokens * g.k_pad <= 16384 &&
         g.rows_pad <= 16 * device_cu_count();
}

// How `problems` products of `tokens` tokens run: on the rows kernel, or on tiles of
// `rows` x `cols`, k in `splits` parts.
struct Plan {
  int rows, cols, splits;      // rows 16: the rows kernel
  double us;                   // modelled
};
Plan plan_for(const Geometry &g, int64_t tokens, int problems) {
  const int steps = int(g.k_pad / kStep), cus = device_cu_count();
  // The rows kernel reads every token once per 16 rows, 128 x 64 tiles once per 128 but
  // with idle compute units below a tile per unit.  Measured (us, rows kernel / tiles): 16
  // tokens 4096 x 4096 11 / 14, 4096 x 11008 18 / 21, 14336 x 4096 18 / 20, 28672 x 8192
  // 58 / 45; 3 tokens 28672 x 8192 45.5 / 45.
  if (tokens <= 3 || (tokens <= kRowsTokens && 10 * cdiv(g.rows, 128) < 8 * cus))
    return {16, 0, 1, 0};
  // The shape and the split of the least modelled time.  A compute unit runs n =
  // ceil(tiles splits / CUs) workgroups of steps / splits stages; a stage of a
  // shape costs it `stage` us and a workgroup `fixed` us (first loads, epilogue;
  // shared by `fit` resident workgroups); a split adds the join.  The figures are fits
  // to measured products (us): 4096 x 4096 x 4096 62 on 256 x 256, 75 on 128 x 128; 2048
  // x 11008 x 4096 116 and 107; 1024 x 4096 x 4096 24 on 128 x 128, 31 on 128 x 64; 512
  // x 4096 x 4096 22 and 17; 128 x 4096 x 11008 on 128 x 64 21 with k in four, 29 in one.
  // Two problems are gate and up, with sums to 32 bits: 400 x 8192 x 3584 65 on 128 x 128, 512
  // x 4096 x 2048 28 on 128 x 64.
  struct Shape {
    int rows, cols, fit, most;
    double stage, fixed;
  };
  constexpr Shape kPlainShapes[] = {{256, 256, 1, 1, 1.65, 8}, {128, 128, 2, 8, 0.5, 6},
                                    {128, 64, 1, 8, 0.4, 4}};
  constexpr Shape kExactShapes[] = {{128, 128, 1, 8, 0.94, 6}, {128, 64, 1, 8, 0.72, 4}};
  Plan best{128, 64, 1, 1e30};
  const bool exact = problems == 2;
  for (const Shape *at = exact ? kExactShapes : kPlainShapes,
                   *end = exact ? std::end(kExactShapes) : std::end(kPlainShapes);
       at != end; ++at) {
    const Shape &sh = *at;
    const int64_t tiles = cdiv(g.rows, sh.rows) * cdiv(tokens, sh.cols) * problems;
    for (int splits = 1; splits <= sh.most && splits * 4 <= std::max(steps, 4); ++splits) {
      const int64_t n = cdiv(tiles * splits, cus);
      double us = double(n * cdiv(steps, splits)) * sh.stage + double(cdiv(n, sh.fit)) * sh.fixed;
      if (splits > 1) us += 4.5 + double(tiles * splits) * (sh.rows * sh.cols) * 8e-6 / 4;
      if (us < best.us) best = {sh.rows, sh.cols, splits, us};
    }
  }
  return best;
}
size_t part_bytes(const Geometry &g, int64_t tokens, int problems) {
  const Plan p = plan_for(g, tokens, problems);
  if (p.rows == 16 || p.splits == 1) return 0;
  return align256(size_t(cdiv(g.rows, p.rows) * cdiv(tokens, p.cols)) * p.splits * problems *
                  (size_t(p.rows) * p.cols * sizeof(float)));
}

// Launch names tell the tile: rows x tokens.
template <int WM, int WN, int FA, int FB, int NBUF, Mode M = kPlain>
gptq_status launch_tiles(const char *name, const GemmArgs &a, hipStream_t s) {
  auto kern = f8_tile_kernel<WM, WN, FA, FB, NBUF, M>;
  constexpr size_t lds = tile_lds(WM, WN, FA, FB, NBUF, M);
  // what follows the stages: results turned, as float32 at most, half of the columns at
  // a time, or codes and a word per token and wave row
  static_assert(lds >= WM * WN * 64 * FA * 16 * ((FB + 1) / 2) || M == kGated, "");
  static_assert(lds >= 16 * FB * WN * (kStep + 4 * WM), "");
  GPTQ_TRY(allow_dynamic_lds(reinterpret_cast<const void *>(kern), lds));
  const int rt = int(cdiv(a.rows, 16 * FA * WM / (M == kGated ? 2 : 1)));
  const int tt = int(cdiv(a.tokens, 16 * FB * WN));
  const uint32_t tiles = uint32_t(rt) * uint32_t(tt) * a.problems;
  GPTQ_TRY(launch(name, kern, dim3(tiles * a.splits), dim3(64 * WM * WN), lds, s, a, tt, rt));
  if constexpr (M != kGated && FA * FB <= 16)     // the shapes that are split
    if (a.splits > 1)
      return launch("f8_join", f8_join_kernel<WM, WN, FA, FB, M>, dim3(tiles * FA * WM * WN / 4),
                    dim3(256), 0, s, a, tt, rt);
  return GPTQ_OK;
}

GemmArgs gemm_args(const gptq_f8_layer *l, const uint8_t *codes, int64_t ld_codes,
                   const float *scale, int64_t ld_scale, int64_t tokens) {
  const Geometry g = geometry(l->rows, l->cols);
  const LayerMap m = layer_map(l->mem, g);
  GemmArgs a{};
  a.w = a.w2 = m.w;
  a.w_scale = a.w2_scale = m.scale;
  a.x = codes;
  a.x_scale = scale;
  a.ld_x = ld_codes;
  a.ld_xs = ld_scale;
  a.tokens = int(tokens);
  a.rows = int(g.rows);
  a.cols = int(g.cols);
  a.row_tiles = int(g.rows_pad / 16);
  a.steps = int(g.k_pad / kStep);
  a.splits = a.problems = 1;
  return a;
}
// Products on codes; `a` says which and whereto.
gptq_status gemm_launch(const Geometry &g, GemmArgs a, void *ws, hipStream_t s) {
  const Plan p = plan_for(g, a.tokens, a.problems);
  if (p.rows == 16)
    return launch("f8_rows", f8_rows_kernel<1, uint8_t>, dim3(uint32_t(a.row_tiles)),
                  dim3(64 * kRowsWaves), 0, s, a);
  a.part = static_cast<f32x4_t *>(ws);
  a.splits = p.splits;
  if (a.problems == 2)
    return p.cols == 64 ? launch_tiles<2, 4, 4, 1, 4, kExact>("f8_gate_up_128x64", a, s)
                        : launch_tiles<2, 4, 4, 2, 4, kExact>("f8_gate_up_128x128", a, s);
  if (p.rows == 256) return launch_tiles<2, 4, 8, 4, 2>("f8_gemm_256x256", a, s);
  if (p.cols == 64) return launch_tiles<2, 4, 4, 1, 4>("f8_gemm_128x64", a, s);
  // a single workgroup on a compute unit has room for four buffers
  const int64_t units = cdiv(g.rows, 128) * cdiv(a.tokens, 128) * a.splits * a.problems;
  return units <= device_cu_count() ? launch_tiles<2, 4, 4, 2, 4>("f8_gemm_128x128_deep", a, s)
                                    : launch_tiles<2, 4, 4, 2, 2>("f8_gemm_128x128", a, s);
}
gptq_status gemm_launch(const gptq_f8_layer *l, const Codes &c, int64_t ld_scale, int64_t tokens,
                        void *y, int32_t y_dtype, int64_t ld_y, void *ws, hipStream_t s) {
  GemmArgs a = gemm_args(l, c.codes, c.ld, c.scale, ld_scale, tokens);
  a.y = y;
  a.ld_y = ld_y;
  a.y_type = y_dtype;
  return gemm_launch(geometry(l->rows, l->cols), a, ws, s);
}
// The rows kernel on floats.
gptq_status rows_on_floats(const gptq_f8_layer *l, const void *x, int32_t x_dtype, int64_t ld_x,
                           int64_t tokens, void *y, int32_t y_dtype, int64_t ld_y, hipStream_t s) {
  GemmArgs a = gemm_args(l, static_cast<const uint8_t *>(x), ld_x, nullptr, 0, tokens);
  a.y = y;
  a.ld_y = ld_y;
  a.y_type = y_dtype;
  auto kern = x_dtype == GPTQ_DT_F32    ? f8_rows_kernel<1, float>
              : x_dtype == GPTQ_DT_BF16 ? f8_rows_kernel<1, bf16_t>
                                        : f8_rows_kernel<1, f16_t>;
  const size_t lds = size_t(tokens) * (rows_stride(a.steps) + 4 * a.steps);
  GPTQ_TRY(allow_dynamic_lds(reinterpret_cast<const void *>(kern), 32768));
  return launch("f8_rows_floats", kern, dim3(uint32_t(a.row_tiles)), dim3(64 * kRowsWaves), lds, s, a);
}

bool fits(const gptq_f8_ff *f) {
  return f && check_layer(&f->gate) == GPTQ_OK && check_layer(&f->up) == GPTQ_OK &&
         check_layer(&f->down) == GPTQ_OK && f->gate.rows == f->up.rows &&
         f->gate.cols == f->up.cols && f->down.cols == f->gate.rows &&
         f->down.rows == f->gate.cols;
}
// How the block's first half runs.
//   kFew      on the rows kernel, to float32
//   kApart    both products to float32, which may be split, and a pass that makes the codes
//   kFused    gate, up and the codes of v in one kernel, on tiles of 128 rows of v x 64
//             tokens, or x 256
enum Half { kFew, kApart, kFused64, kFused256 };
Half half_for(const gptq_f8_ff *f, int64_t tokens) {
  if (tokens <= kRowsTokens) return kFew;
  const Geometry g = geometry(f->gate.rows, f->gate.cols);
  const int64_t steps = g.k_pad / kStep, rt = cdiv(g.rows, kStep);
  const int cus = device_cu_count();
  // As in plan_for; the pass between costs a launch and 8 bytes per value each way.
  const double apart = plan_for(g, tokens, 2).us + 4.5 + double(tokens) * g.rows * 16 / 4e6;
  // Measured (us, 64 / 256 tokens wide): 300 x 4096 x 11008 79 / 101, 512 x 118 / 97; 1024
  // x 4096 x 4096 79 / 96, 2048 x 152 / 108; 1024 x 1024 x 4096 30 / 34, 2048 x 57 / 38.
  const double wide = double(cdiv(rt * cdiv(tokens, 256), cus)) * (steps * 2.5 + 12);
  const double narrow = double(cdiv(rt * cdiv(tokens, 64), cus)) * (steps * 1.03 + 6);
  if (std::min(wide, narrow) < apart)
    return wide < narrow ? kFused256 : kFused64;
  return kApart;
}
struct BlockWs {
  Codes x, v;
  float *g, *u;
  void *parts;
  size_t bytes;
};
BlockWs block_ws(const gptq_f8_ff *f, int64_t tokens, void *mem) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(mem);
  const Half half = half_for(f, tokens);
  const size_t one = align256(size_t(tokens) * f->gate.rows * 4);
  BlockWs w{};
  w.x = codes_at(mem, tokens, f->gate.cols);
  size_t at = w.x.bytes;
  w.v = codes_at(reinterpret_cast<void *>(base + at), tokens, f->gate.rows);
  at += w.v.bytes;
  if (half <= kApart) {
    w.g = reinterpret_cast<float *>(base + at);
    w.u = reinterpret_cast<float *>(base + at + one);
    at += half == kFew ? one : 2 * one;
  }
  w.parts = reinterpret_cast<void *>(base + at);
  // The down product is planned on its own: wide ones of few tokens are split too.
  at += std::max(half == kApart ? part_bytes(geometry(f->gate.rows, f->gate.cols), tokens, 2) : 0,
                 part_bytes(geometry(f->down.rows, f->down.cols), tokens, 1));
  w.bytes = at;
  return w;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

gptq_status gptq_f8_quantize_tokens(const void *x, int32_t x_dtype, int64_t tokens, int64_t cols,
                                    int64_t ld_x, uint8_t *codes, int64_t ld_codes, float *scale,
                                    int64_t ld_scale, void *stream) {
  return guarded([&]() -> gptq_status {
    if (gptq_tokens_ld(cols) == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "cols must be in [1, 65536]");
    GPTQ_TRY(check_activations(x, x_dtype, tokens, cols, ld_x, "x"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_codes(codes, ld_codes, scale, ld_scale, tokens, cols));
    return quantize(x, x_dtype, tokens, cols, ld_x, codes, ld_codes, scale, ld_scale,
                    static_cast<hipStream_t>(stream));
  });
}

gptq_status gptq_f8_quantize_weight(const void *w, int32_t w_dtype, int64_t rows, int64_t cols,
                                    int64_t ld_w, uint8_t *codes, float *scale, void *stream) {
  return guarded([&]() -> gptq_status {
    if (gptq_f8_layer_bytes(rows, cols) == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "rows and cols must be in [1, 2^24] x [1, 65536]");
    GPTQ_TRY(check_activations(w, w_dtype, 1, cols, ld_w, "w"));
    if (!codes || !scale) return fail(GPTQ_ERR_INVALID_ARG, "codes and scale must not be NULL");
    if (!aligned_to(scale, 4)) return fail(GPTQ_ERR_INVALID_ARG, "scale must be 4-byte aligned");
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (w_dtype == GPTQ_DT_F32)
      return quantize_weight_typed<float>(w, ld_w, rows, cols, codes, scale, s);
    if (w_dtype == GPTQ_DT_BF16)
      return quantize_weight_typed<bf16_t>(w, ld_w, rows, cols, codes, scale, s);
    return quantize_weight_typed<f16_t>(w, ld_w, rows, cols, codes, scale, s);
  });
}

size_t gptq_f8_layer_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || rows > kMaxRows || gptq_tokens_ld(cols) == 0) return 0;
  const Geometry g = geometry(rows, cols);
  return g.rows_pad * g.k_pad > kMaxCodes ? 0 : layer_map(nullptr, g).bytes;
}

gptq_status gptq_f8_prepare(const uint8_t *codes, const float *scale, int64_t rows, int64_t cols,
                            void *mem, size_t mem_bytes, gptq_f8_layer *layer, void *stream) {
  return guarded([&]() -> gptq_status {
    const size_t need = gptq_f8_layer_bytes(rows, cols);
    if (need == 0)
      return fail(GPTQ_ERR_INVALID_ARG, "rows and cols must be in [1, 2^24] x [1, 65536]");
    if (!codes || !scale || !mem || !layer)
      return fail(GPTQ_ERR_INVALID_ARG, "codes, scale, mem and layer must not be NULL");
    if (!aligned_to(scale, 4)) return fail(GPTQ_ERR_INVALID_ARG, "scale must be 4-byte aligned");
    if (!aligned_to(mem, 256)) return fail(GPTQ_ERR_INVALID_ARG, "mem must be 256-byte aligned");
    if (mem_bytes < need)
      return fail(GPTQ_ERR_INVALID_ARG, "mem too small: need " + std::to_string(need) +
                                            " bytes, got " + std::to_string(mem_bytes));
    const Geometry g = geometry(rows, cols);
    const LayerMap m = layer_map(mem, g);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t pieces = g.rows_pad * g.k_pad / 16;
    const int64_t scales = cdiv(rows, kStep) * (g.k_pad / kStep);
    GPTQ_TRY(launch("f8_repack", f8_repack_kernel, dim3(uint32_t(cdiv(pieces, 256))), dim3(256), 0,
                    s, codes, rows, cols, pieces, g.k_pad / kStep,
                    reinterpret_cast<u32x4_t *>(m.w)));
    GPTQ_TRY(launch("f8_scales", f8_scales_kernel, dim3(uint32_t(cdiv(scales, 256))), dim3(256), 0,
                    s, scale, scales, m.scale));
    *layer = gptq_f8_layer{rows, cols, g.rows_pad, g.k_pad, mem, mem_bytes};
    return GPTQ_OK;
  });
}

size_t gptq_f8_gemm_ws_bytes(const gptq_f8_layer *layer, int64_t tokens) {
  return guarded_bytes([&]() -> size_t {
    if (!layer || tokens < 1 || tokens > kMaxTokens || gptq_f8_layer_bytes(layer->rows, layer->cols) == 0)
      return 0;
    return part_bytes(geometry(layer->rows, layer->cols), tokens, 1);
  });
}

size_t gptq_f8_linear_ws_bytes(const gptq_f8_layer *layer, int64_t tokens) {
  return guarded_bytes([&]() -> size_t {
    if (!layer || tokens < 1 || tokens > kMaxTokens || gptq_f8_layer_bytes(layer->rows, layer->cols) == 0)
      return 0;
    if (rows_floats(geometry(layer->rows, layer->cols), tokens)) return 0;
    return codes_at(nullptr, tokens, layer->cols).bytes + gptq_f8_gemm_ws_bytes(layer, tokens);
  });
}

gptq_status gptq_f8_gemm(const gptq_f8_layer *layer, const uint8_t *codes, int64_t ld_codes,
                         const float *scale, int64_t ld_scale, int64_t tokens, void *y,
                         int32_t y_dtype, int64_t ld_y, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_layer(layer));
    GPTQ_TRY(check_tokens(tokens));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_codes(codes, ld_codes, scale, ld_scale, tokens, layer->cols));
    GPTQ_TRY(check_output(y, y_dtype, ld_y, layer->rows));
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_f8_gemm_ws_bytes(layer, tokens)));
    const Codes c{const_cast<uint8_t *>(codes), const_cast<float *>(scale), ld_codes, 0};
    return gemm_launch(layer, c, ld_scale, tokens, y, y_dtype, ld_y, ws,
                       static_cast<hipStream_t>(stream));
  });
}

gptq_status gptq_f8_linear(const gptq_f8_layer *layer, const void *x, int32_t x_dtype, int64_t ld_x,
                           int64_t tokens, void *y, int32_t y_dtype, int64_t ld_y, void *ws,
                           size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_layer(layer));
    GPTQ_TRY(check_tokens(tokens));
    GPTQ_TRY(check_activations(x, x_dtype, tokens, layer->cols, ld_x, "x"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_output(y, y_dtype, ld_y, layer->rows));
    if (matrices_meet(x, tokens, layer->cols, ld_x, type_bytes(x_dtype), y, tokens, layer->rows, ld_y,
                     2))
      return fail(GPTQ_ERR_INVALID_ARG, "y must not overlap x");
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_f8_linear_ws_bytes(layer, tokens)));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows_floats(geometry(layer->rows, layer->cols), tokens))
      return rows_on_floats(layer, x, x_dtype, ld_x, tokens, y, y_dtype, ld_y, s);
    const Codes c = codes_at(ws, tokens, layer->cols);
    GPTQ_TRY(quantize(x, x_dtype, tokens, layer->cols, ld_x, c.codes, c.ld, c.scale, tokens, s));
    return gemm_launch(layer, c, tokens, tokens, y, y_dtype, ld_y,
                       static_cast<char *>(ws) + c.bytes, s);
  });
}

size_t gptq_f8_ff_ws_bytes(const gptq_f8_ff *ff, int64_t tokens) {
  return guarded_bytes([&]() -> size_t {
    if (!fits(ff) || tokens < 1 || tokens > kMaxTokens) return 0;
    return block_ws(ff, tokens, nullptr).bytes;
  });
}

gptq_status gptq_f8_ff_forward(const gptq_f8_ff *ff, const void *x, int32_t x_dtype, int64_t ld_x,
                               int64_t tokens, void *y, int32_t y_dtype, int64_t ld_y, void *ws,
                               size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    if (!fits(ff))
      return fail(GPTQ_ERR_INVALID_ARG,
                  "gate, up and down must be prepared, gate and up inner x d, down d x inner");
    GPTQ_TRY(check_tokens(tokens));
    const int64_t d = ff->gate.cols, inner = ff->gate.rows;
    GPTQ_TRY(check_activations(x, x_dtype, tokens, d, ld_x, "x"));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_output(y, y_dtype, ld_y, d));
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_f8_ff_ws_bytes(ff, tokens)));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const BlockWs w = block_ws(ff, tokens, ws);
    const Half half = half_for(ff, tokens);
    GPTQ_TRY(quantize(x, x_dtype, tokens, d, ld_x, w.x.codes, w.x.ld, w.x.scale, tokens, s));
    GemmArgs a = gemm_args(&ff->gate, w.x.codes, w.x.ld, w.x.scale, tokens, tokens);
    const LayerMap up = layer_map(ff->up.mem, geometry(inner, d));
    a.w2 = up.w;
    a.w2_scale = up.scale;
    if (half <= kApart) {
      a.y = w.g;
      a.y2 = w.u;
      a.ld_y = inner;
      if (half == kFew) {                  // v itself comes out of the rows kernel
        GPTQ_TRY(launch("f8_rows_gate_up", f8_rows_kernel<2, uint8_t>,
                        dim3(uint32_t(a.row_tiles)), dim3(64 * kRowsWaves), 0, s, a));
        if (rows_floats(geometry(d, inner), tokens))
          return rows_on_floats(&ff->down, w.g, GPTQ_DT_F32, inner, tokens, y, y_dtype, ld_y, s);
        GPTQ_TRY(quantize(w.g, GPTQ_DT_F32, tokens, inner, inner, w.v.codes, w.v.ld, w.v.scale,
                          tokens, s));
      } else {
        a.problems = 2;
        GPTQ_TRY(gemm_launch(geometry(inner, d), a, w.parts, s));
        GPTQ_TRY((quantize_typed<float, true>(w.g, w.u, tokens, inner, inner, w.v.codes, w.v.ld,
                                              w.v.scale, tokens, s)));
      }
    } else {
      a.v = w.v.codes;
      a.ld_v = w.v.ld;
      a.v_scale = w.v.scale;
      a.ld_vs = tokens;
      if (half == kFused256)
        GPTQ_TRY((launch_tiles<2, 4, 8, 4, 2, kGated>("f8_gate_up_256x256", a, s)));
      else
        GPTQ_TRY((launch_tiles<4, 2, 4, 2, 3, kGated>("f8_gate_up_256x64", a, s)));
    }
    return gemm_launch(&ff->down, w.v, tokens, tokens, y, y_dtype, ld_y, w.parts, s);
  });
}

}  // extern "C"
