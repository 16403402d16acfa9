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
// Laying a layer out moves it once each way (28672 x 8192: 75 us).
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
typedef float f32x4r_t __attribute__((ext_vector_type(4)));

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
  const uintptr_t p = reinterpret_cast<uintptr_t>(mem);    // 0 where only the size is asked
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
  i32x4_t *part;    // split products: the blocks of each (tile, split)
};

// Result blocks of a wave: acc[i][j] holds rows r0 + 16 i + 4 (l / 16) .. + 3
// (registers) of token t0 + 16 j + l % 16 (l the lane).
//
// Stored as they lie, a wave's store would touch 16 tokens' rows for 32 bytes
// each.  They are turned in the wave's own piece of LDS instead, half the
// token blocks at a time: token-major rows of 16 FA values, whose 16-byte
// pieces are XOR-swizzled so that neither side meets bank conflicts; a store
// then writes 16 FA consecutive values per token.  (Direct stores took 25 us
// per 256 x 256 tile, as long as 17 of its 128-k stages.)
template <typename T, int FA, int FB>
__device__ __forceinline__ void store_typed(const GemmArgs &a, const i32x4_t (&acc)[FA][FB],
                                            int t0, int r0, int lane, uint8_t *lds) {
  constexpr int kRow = 16 * FA * sizeof(T), kPieces = kRow / 16, kHalf = (FB + 1) / 2;
  constexpr int kVals = 16 / sizeof(T);
  auto place = [&](int t, int piece) {
    const int x = kPieces >= 16 ? t & 15 : kPieces == 8 ? (t >> 1) & 7 : (t >> 2) & (kPieces - 1);
    return lds + t * kRow + ((piece ^ x) << 4);
  };
  const int g = lane >> 4;
#pragma unroll
  for (int j0 = 0; j0 < FB; j0 += kHalf) {
    float st[kHalf];
    int sum[kHalf];
#pragma unroll
    for (int j = 0; j < kHalf; ++j) {
      const int t = min(t0 + 16 * (j0 + j) + (lane & 15), a.tokens - 1);
      st[j] = a.x_scale[t];
      sum[j] = a.x_sum[t];
    }
#pragma unroll
    for (int i = 0; i < FA; ++i) {
      const int r = min(r0 + 16 * i, a.row_tiles * 16 - 16) + 4 * g;   // past the layer: unused
      const f32x4r_t ws = *reinterpret_cast<const f32x4r_t *>(a.w_scale + r);
      const i32x4_t sh = *reinterpret_cast<const i32x4_t *>(a.w_shift + r);
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        if (j0 + j >= FB) break;
        T o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          // z - 128 and the code sum both fit in 24 bits
          float f = float(acc[i][j0 + j][v] - __mul24(sh[v], sum[j])) * (st[j] * ws[v]);
          // rounded to float32 before it is narrowed (not in one
          // mixed-precision multiply)
          asm("" : "+v"(f));
          o[v] = narrow<T>(f);
        }
        const int byte = (16 * i + 4 * g) * int(sizeof(T));
        __builtin_memcpy(__builtin_assume_aligned(place(16 * j + (lane & 15), byte >> 4) + (byte & 15),
                                                  sizeof(o)), o, sizeof(o));
      }
    }
#pragma unroll
    for (int it = 0; it < (kHalf * 16 * kPieces + 63) / 64; ++it) {
      const int at = it * 64 + lane, t = at / kPieces, piece = at % kPieces;
      if (t >= kHalf * 16) continue;
      const u32x4r_t v = *reinterpret_cast<const u32x4r_t *>(place(t, piece));
      const int tok = t0 + 16 * j0 + t, r = r0 + piece * kVals, left = a.rows - r;
      if (tok >= a.tokens || left <= 0) continue;
      T *p = static_cast<T *>(a.y) + int64_t(tok) * a.ld_y + r;
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
  }
}
// `lds`: the wave's own 16 FA * 16 ceil(FB / 2) * 4 bytes.
template <int FA, int FB>
__device__ __forceinline__ void store_blocks(const GemmArgs &a, const i32x4_t (&acc)[FA][FB],
                                             int t0, int r0, int lane, uint8_t *lds) {
  if (a.y_type == GPTQ_DT_F32) store_typed<float>(a, acc, t0, r0, lane, lds);
  else if (a.y_type == GPTQ_DT_BF16) store_typed<bf16_t>(a, acc, t0, r0, lane, lds);
  else store_typed<f16_t>(a, acc, t0, r0, lane, lds);
}

// A workgroup barrier that orders LDS accesses only: loads from memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---- Tiles through LDS.  A workgroup of 4 waves (2 x 2) makes a tile of
// 32 FA rows x 32 FB tokens; a wave FA x FB blocks of 16 x 16.  Stages of
// 128 k are double-buffered in LDS: weights in the prepared order (a
// fragment is 1 KiB of consecutive LDS), tokens as 128-byte rows whose
// 16-byte pieces are XOR-swizzled; both read without bank conflicts.
//
// Iteration u: step 0 multiplies the first 64 k of stage u (set X) while the
// second 64 k (set Y) are read; a barrier makes stage u + 1 visible; step 1
// multiplies set Y while set X is read from stage u + 1.  Each of a stage's
// copies waits in registers from its load to its store DEPTH stages later,
// into the ring slot whose last reads came before the previous barrier.
// Small tiles, whose stages are shorter than a memory access, take DEPTH 2
// or 3; 256 x 256 tiles have registers for 1.
//
// 8192 x 28672 x 8192: 1.43-1.55 ms, 2.5-2.7 POP/s (a library product of the
// same sizes 1.90 ms).  It takes 2.98 M cycles, in 62 % of which the matrix units
// are busy; with every load from memory left out it gained 11 %.  The clock under
// it was 1.64 to 1.91 GHz of 2.4, and the time goes with it.  16 x 28672 x 8192: 44
// us, its 236 MB at 5.4 TB/s.  333 x 4091 x 4100: 16 us, by latency: 192 workgroups
// leave 64 compute units idle, and in the others, with a wave per SIMD, the matrix
// units are busy 24 % of the time; a wave waits for data or a barrier in 26 % of
// its cycles and to issue in 25 %.  (L2 gives 159 MB, 49 bytes per ns and unit.)
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// Tiles in bands of kBand token tiles, tokens fastest: workgroups are dealt
// round-robin to the 8 XCDs, each XCD takes a contiguous run of this order,
// so its 32 concurrent tiles share 4 token and 8 row panels in its L2.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_at(int bid, int tt, int rt, int &t, int &r) {
  const int n = tt * rt, x = bid & 7;
  const int at = x * (n / 8) + min(x, n % 8) + (bid >> 3);
  const int band = at / (kBand * rt), b0 = band * kBand, h = min(kBand, tt - b0);
  const int u = at - b0 * rt;
  r = __builtin_amdgcn_readfirstlane(u / h);    // wave-uniform, kept scalar
  t = __builtin_amdgcn_readfirstlane(b0 + u % h);
}

// acc += w x^T on the matrix core, in place in accumulation registers.  (The
// builtin leaves the result's register free; with every accumulation register
// taken, the compiler then moved whole accumulators between files in the
// loop.)  The operands come from LDS reads, never straight from vector ALU
// instructions.  An acc is next touched FA FB of these later (8 in the smallest
// tiles, at 16 cycles each), and then only as the accumulator of the same
// instruction, which the matrix unit orders by itself.  After the last one, and
// before the first, settle() waits the pipeline out.
__device__ __forceinline__ void mfma_acc(i32x4_t &acc, i32x4_t w, i32x4_t x) {
  asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(w), "v"(x));
}
template <int FA, int FB>
__device__ __forceinline__ void settle(i32x4_t (&acc)[FA][FB]) {
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) asm volatile("" : "+a"(acc[i][j]));
}

template <int FA, int FB, int DEPTH, bool SPLIT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, FA * FB > 16 ? 1 : 2)))
    w8a8_tile_kernel(GemmArgs a, int token_tiles, int row_tiles, int splits) {
  constexpr int kWBytes = 32 * FA * kStep, kXBytes = 32 * FB * kStep;
  constexpr int kStageBytes = kWBytes + kXBytes;
  constexpr int kWLoads = FA, kLoads = FA + FB;     // 16-byte copies per lane and stage
  constexpr int kHalf = kLoads / 2;
  constexpr int kSlots = FA * FB;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int tt, tr;
  const int tiles = token_tiles * row_tiles;
  const int split = SPLIT ? int(blockIdx.x) / tiles : 0;
  const int tile = int(blockIdx.x) - split * tiles;
  tile_at(tile, token_tiles, row_tiles, tt, tr);
  const int rt0 = tr * 2 * FA, t0 = tt * 32 * FB;   // first 16-row tile, first token
  const int s0 = SPLIT ? a.steps * split / splits : 0;
  const int U = SPLIT ? a.steps * (split + 1) / splits - s0 : a.steps;

  // Copy q of a lane: 4 KiB of weights (two 16-row tiles) or 32 token rows.
  // Rows past the layer or the tokens are clamped; they only feed outputs
  // that are never stored.
  const int8_t *wbase = a.w + (int64_t(rt0) * a.steps + s0) * 2048;
  const int8_t *xbase = a.x + int64_t(t0) * a.ld_x + s0 * kStep;
  uint32_t voff[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    if (q < kWLoads)
      voff[q] = uint32_t(min(2 * q + (tid >> 7), a.row_tiles - 1 - rt0)) * uint32_t(a.steps * 2048) +
                (tid & 127) * 16;
    else
      voff[q] = uint32_t(min(32 * (q - kWLoads) + (tid >> 3), a.tokens - 1 - t0)) *
                    uint32_t(a.ld_x) + (tid & 7) * 16;
  }
  const int xrow = tid >> 3;
  const int lds_x = kWBytes + xrow * kStep + (((tid & 7) ^ swz(xrow)) << 4);
  u32x4r_t stg[DEPTH][kLoads];   // copies of stage t wait in set t % DEPTH
  auto load_one = [&](int q, int t, int set) {
    t = min(t, U - 1);
    auto base = (const __attribute__((address_space(1))) int8_t *)(
        q < kWLoads ? wbase + int64_t(t) * 2048 : xbase + int64_t(t) * kStep);
    uint32_t off = voff[q];
    asm("" : "+s"(base), "+v"(off));   // scalar base, the lane's fixed 32-bit offset
    stg[set][q] = *(const __attribute__((address_space(1))) u32x4r_t *)(base + off);
  };
  auto store_one = [&](int q, int t, int set) {
    uint8_t *p = smem + (t & 1) * kStageBytes +
                 (q < kWLoads ? q * 4096 + tid * 16 : lds_x + (q - kWLoads) * 32 * kStep);
    *reinterpret_cast<u32x4r_t *>(p) = stg[set][q];
  };
  auto frag_a = [&](int u, int h, int i) {
    return *reinterpret_cast<const i32x4_t *>(smem + (u & 1) * kStageBytes +
                                              (wm * FA + i) * 2048 + h * 1024 + lane * 16);
  };
  auto frag_b = [&](int u, int h, int j) {
    const int row = wn * 16 * FB + 16 * j + (lane & 15), c = 4 * h + (lane >> 4);
    return *reinterpret_cast<const i32x4_t *>(smem + (u & 1) * kStageBytes + kWBytes +
                                              row * kStep + ((c ^ swz(row)) << 4));
  };

  i32x4_t acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  i32x4_t xa[4], xb[FB], ya[FA], yb[FB];   // xa: block row i in slot i % 4
  // Copies below kHalf run one stage ahead of the others: stages 0 and 1 of
  // them are stored here, stage 0 of the others; then each has DEPTH stages
  // in flight.
#pragma unroll
  for (int t = 0; t < DEPTH; ++t)
#pragma unroll
    for (int q = 0; q < kLoads; ++q) load_one(q, t, t);
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    store_one(q, 0, 0);
    load_one(q, DEPTH, 0);
  }
#pragma unroll
  for (int q = 0; q < kHalf; ++q) {
    store_one(q, 1, 1 % DEPTH);
    load_one(q, 1 + DEPTH, 1 % DEPTH);
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < FB; ++j) xb[j] = frag_b(0, 0, j);
#pragma unroll
  for (int i = 0; i < 3; ++i) xa[i] = frag_a(0, 0, i);

  settle<FA, FB>(acc);   // the zeros are written well before the first MFMA reads them

  constexpr int kY = FA + FB, kYEvery = kSlots / kY;       // reads of set Y in step 0
  constexpr int kX = FB + 3, kXEvery = kSlots / kX;        // reads of set X in step 1
  constexpr int kCEvery = kSlots / kHalf;                  // copies in either step
  auto stage = [&](int u, int ph) {    // ph = u % DEPTH
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        mfma_acc(acc[i][j], xa[i % 4], xb[j]);
        const int q = FB * i + j;
        if (j == 1 && i + 3 < FA) xa[(i + 3) % 4] = frag_a(u, 0, i + 3);
        if (q % kYEvery == kYEvery / 2 && q / kYEvery < kY) {
          const int f = q / kYEvery;
          if (f == 0) ya[0] = frag_a(u, 1, 0);
          else if (f <= FB) yb[f - 1] = frag_b(u, 1, f - 1);
          else ya[f - FB] = frag_a(u, 1, f - FB);
        }
        if (q % kCEvery == kCEvery - 1 && q / kCEvery < kHalf) {
          store_one(kHalf + q / kCEvery, u + 1, (ph + 1) % DEPTH);
          load_one(kHalf + q / kCEvery, u + 1 + DEPTH, (ph + 1) % DEPTH);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    lds_barrier();                         // stores of u + 1, reads of u done
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        mfma_acc(acc[i][j], ya[i], yb[j]);
        const int q = FB * i + j;
        if (q % kXEvery == kXEvery / 2 && q / kXEvery < kX) {
          const int f = q / kXEvery;
          if (f < FB) xb[f] = frag_b(u + 1, 0, f);
          else xa[f - FB] = frag_a(u + 1, 0, f - FB);
        }
        if (q % kCEvery == kCEvery - 1 && q / kCEvery < kHalf) {
          store_one(q / kCEvery, u + 2, (ph + 2) % DEPTH);
          load_one(q / kCEvery, u + 2 + DEPTH, (ph + 2) % DEPTH);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  int u = 0;
  for (; u + DEPTH <= U; u += DEPTH) {
#pragma unroll
    for (int ph = 0; ph < DEPTH; ++ph) stage(u + ph, ph);
  }
#pragma unroll
  for (int ph = 0; ph < DEPTH - 1; ++ph)
    if (u + ph < U) stage(u + ph, ph);
  settle<FA, FB>(acc);
  if (SPLIT) {
    // A wave's blocks as they lie in its registers: 1 KiB per store.
    i32x4_t *p = a.part + (int64_t(tile) * splits + split) * (4 * FA * FB * 64) +
                 wave * (FA * FB * 64) + lane;
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) p[(i * FB + j) * 64] = acc[i][j];
    return;
  }
  lds_barrier();                           // every wave is done with the stages
  store_blocks<FA, FB>(a, acc, t0 + wn * 16 * FB, (rt0 + wm * FA) * 16, lane,
                       smem + wave * (kStageBytes / 2));
}

// Adds a split product's parts: a wave per block row (FB blocks) of a tile's
// wave, in the tile kernel's register order.
template <int FA, int FB>
__global__ void __launch_bounds__(256)
    w8a8_join_kernel(GemmArgs a, int token_tiles, int row_tiles, int splits) {
  constexpr int kPiece = 16 * 16 * ((FB + 1) / 2) * 4;
  __shared__ __align__(16) uint8_t lds[4 * kPiece];
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int i = unit % FA, wave = unit / FA % 4, tile = unit / (4 * FA);
  int tt, tr;
  tile_at(tile, token_tiles, row_tiles, tt, tr);
  const int r0 = (tr * 2 * FA + (wave >> 1) * FA + i) * 16;
  const int t0 = tt * 32 * FB + (wave & 1) * 16 * FB;
  if (r0 >= a.rows || t0 >= a.tokens) return;
  const i32x4_t *p = a.part + int64_t(tile) * splits * (4 * FA * FB * 64) +
                     (wave * FA + i) * (FB * 64) + lane;
  i32x4_t acc[1][FB];
#pragma unroll
  for (int j = 0; j < FB; ++j) acc[0][j] = p[j * 64];
  for (int s = 1; s < splits; ++s) {
    p += 4 * FA * FB * 64;
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[0][j] += p[j * 64];
  }
  store_blocks<1, FB>(a, acc, t0, r0, lane, lds + (threadIdx.x >> 6) * kPiece);
}

// ---- Few tokens: a workgroup per 16 rows, its waves splitting k.  A wave
// takes every WAVES-th 128-k step: its weights come straight from memory as
// contiguous KiB, several steps ahead, and each is used for all tokens at
// once, so the product runs at the rate the weights arrive: 5 x 22016 x 4096
// 18 us, 90 MB at 5.0 TB/s; 1 x 4096 x 11008 9.3 us, 45 MB at 4.8 TB/s.  The
// waves' sums meet in LDS.
//
// (Quantizing the activations in each workgroup, to save a launch, was slower:
// 1 x 28672 x 8192 took 54 us against 47 with the separate launch, 1 x 14336 x
// 4096 21.8 against 15.2.)
// Four waves: with 8 or 16 fewer workgroups fit a compute unit, and the tail
// of one is not covered by others (16 x 14336 x 4096: 12, 22 and 22 us).
constexpr int kRowsWaves = 4;

template <int NB>
__global__ void __launch_bounds__(64 * kRowsWaves) w8a8_rows_kernel(GemmArgs a) {
  constexpr int WAVES = kRowsWaves, kThreads = 64 * WAVES;
  __shared__ i32x4_t sums[WAVES * NB * 64];
  constexpr int kAhead = NB == 1 ? 4 : 2;   // steps loaded at a time, two such sets in flight
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rt = blockIdx.x;

  // This wave's steps: wave, wave + WAVES, ...  Loads past the last repeat it.
  const int n = (a.steps - wave + WAVES - 1) / WAVES;
  const int8_t *w = a.w + int64_t(rt) * a.steps * 2048 + lane * 16;
  const int8_t *xrow[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int t = min(16 * j + (lane & 15), a.tokens - 1);
    xrow[j] = a.x + int64_t(t) * a.ld_x + (lane >> 4) * 16;
  }
  struct Set {
    i32x4_t w[kAhead][2], x[kAhead][2][NB];
  };
  auto load = [&](Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t s = wave + int64_t(min(at + i, n - 1)) * WAVES;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b.w[i][h] = *reinterpret_cast<const i32x4_t *>(w + s * 2048 + h * 1024);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          b.x[i][h][j] = *reinterpret_cast<const i32x4_t *>(xrow[j] + s * kStep + h * 64);
      }
    }
  };
  i32x4_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = i32x4_t{0, 0, 0, 0};
  auto multiply = [&](const Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (at + i >= n) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[i][h], b.x[i][h][j], acc[j], 0, 0, 0);
    }
  };
  Set s0, s1;
  if (n > 0) {
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
  for (int j = 0; j < NB; ++j) sums[(wave * NB + j) * 64 + lane] = acc[j];
  lds_barrier();
  // Output (token, row) of thread: 16 consecutive rows per token.
  const int *flat = reinterpret_cast<const int *>(sums);
  for (int o = tid; o < 16 * a.tokens; o += kThreads) {
    const int t = o >> 4, r = o & 15, row = rt * 16 + r;
    // block t / 16: lane 16 (r / 4) + t % 16 holds rows 4 (r / 4) ..
    const int at = (t >> 4) * 256 + (16 * (r >> 2) + (t & 15)) * 4 + (r & 3);
    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) total += uint32_t(flat[i * NB * 256 + at]);
    if (row >= a.rows) continue;
    float y = float(int(total - uint32_t(a.w_shift[row]) * uint32_t(a.x_sum[t]))) *
              (a.x_scale[t] * a.w_scale[row]);
    asm("" : "+v"(y));    // rounded to float32 before it is narrowed
    const int64_t to = int64_t(t) * a.ld_y + row;
    if (a.y_type == GPTQ_DT_F32) static_cast<float *>(a.y)[to] = y;
    else if (a.y_type == GPTQ_DT_BF16) static_cast<bf16_t *>(a.y)[to] = narrow<bf16_t>(y);
    else static_cast<f16_t *>(a.y)[to] = narrow<f16_t>(y);
  }
}

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxTokens = int64_t(1) << 20;
// A launch has at most 2^32 threads; a thread repacks 16 codes.
constexpr int64_t kMaxCodes = int64_t(1) << 35;

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

// ------------------------------------------------------------- launch rules
// How a product of `tokens` tokens runs: on the rows kernel, or on tiles of
// 32 fa rows x 32 fb tokens, k in `splits` parts.
struct Plan {
  bool rows;
  int fa, fb, splits;
};

Plan plan_for(const Geometry &g, int64_t tokens, int cus) {
  const int steps = int(g.k_pad / kStep);
  // The rows kernel reads every token once per 16 rows, the 128 x 64 tiles
  // once per 128 but with idle compute units below a tile per unit.  Measured
  // (us, rows kernel / tiles): 8 x 28672 x 8192 42 / 43, 16 tokens 50 / 43,
  // 32 tokens 67 / 43; 14336 x 4096: 16 tokens 12 / 15, 32 tokens 19 / 15;
  // 8192 x 8192: 24 tokens 17 / 18.5; 4096 x 11008: 32 tokens 14 / 15.
  const int64_t wide = cdiv(g.rows, 128);
  if (tokens <= 8 || (tokens <= 16 && 10 * wide < 7 * cus) || (tokens <= 32 && 10 * wide < 4 * cus))
    return {true, 0, 0, 1};
  // Tiles: the shape and the split of the least modelled time.  A compute
  // unit runs n = ceil(tiles splits / CUs) workgroups of steps / splits
  // stages; a stage of a shape costs it `stage` us and a workgroup `fixed` us
  // (first loads, epilogue; shared by `fit` resident workgroups); a split adds
  // the join.  Larger tiles read less per product, smaller ones leave fewer
  // compute units idle.  The figures are fits to measured products (us):
  // 2048 x 22016 x 4096 took 177 on 256 x 256 tiles, 209 on 128 x 256; 2048 x
  // 4096 x 11008 119 against 85 (90 on 128 x 128); 1024 x 4096 x 4096 33 on
  // 128 x 256, 23 on 128 x 128; 512 x 4096 x 4096 21 on 128 x 128, 16 on
  // 128 x 64; 128 x 4096 x 11008 29 on 128 x 64, 17 with k in four.
  struct Shape {
    int fa, fb, fit, most;
    double stage, fixed;
  };
  constexpr Shape kShapes[] = {
      {8, 8, 1, 1, 1.47, 12.8}, {4, 8, 1, 1, 0.92, 6}, {4, 4, 2, 8, 0.53, 5}, {4, 2, 3, 8, 0.33, 5}};
  Plan best{false, 4, 2, 1};
  double least = 1e30;
  for (const Shape &sh : kShapes) {
    const int64_t tiles = cdiv(g.rows, 32 * sh.fa) * cdiv(tokens, 32 * sh.fb);
    for (int splits = 1; splits <= sh.most && splits * 4 <= std::max(steps, 4); ++splits) {
      const int64_t n = cdiv(tiles * splits, cus);
      double us = double(n * cdiv(steps, splits)) * sh.stage + double(cdiv(n, sh.fit)) * sh.fixed;
      if (splits > 1) us += 4.5 + double(tiles * splits) * (32 * sh.fa * 32 * sh.fb) * 8e-6 / 4;
      if (us < least) {
        least = us;
        best = {false, sh.fa, sh.fb, splits};
      }
    }
  }
  return best;
}

size_t part_bytes(const Geometry &g, int64_t tokens, const Plan &p) {
  if (p.rows || p.splits == 1) return 0;
  return align256(size_t(cdiv(g.rows, 32 * p.fa) * cdiv(tokens, 32 * p.fb)) * p.splits *
                  (32 * p.fa * 32 * p.fb * sizeof(int32_t)));
}

// Launch names tell the tile: rows x tokens.
template <int FA, int FB, int DEPTH, bool SPLIT>
gptq_status launch_tiles(const char *name, const GemmArgs &a, int splits, hipStream_t s) {
  auto kern = w8a8_tile_kernel<FA, FB, DEPTH, SPLIT>;
  const size_t lds = size_t(2) * 32 * (FA + FB) * kStep;
  GPTQ_TRY(allow_dynamic_lds(reinterpret_cast<const void *>(kern), lds));
  const int rt = int(cdiv(a.rows, 32 * FA)), tt = int(cdiv(a.tokens, 32 * FB));
  const uint32_t tiles = uint32_t(rt) * uint32_t(tt);
  GPTQ_TRY(launch(name, kern, dim3(tiles * splits), dim3(256), lds, s, a, tt, rt, splits));
  if constexpr (SPLIT)
    GPTQ_TRY(launch("w8a8_join", w8a8_join_kernel<FA, FB>, dim3(tiles * FA), dim3(256), 0, s, a, tt,
                    rt, splits));
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
  a.part = static_cast<i32x4_t *>(ws);
  const Plan p = plan_for(g, tokens, device_cu_count());
  if (p.rows)
    return launch("w8a8_rows", tokens <= 16 ? w8a8_rows_kernel<1> : w8a8_rows_kernel<2>,
                  dim3(uint32_t(a.row_tiles)), dim3(64 * kRowsWaves), 0, s, a);
  if (p.fa == 8) return launch_tiles<8, 8, 1, false>("w8a8_gemm_256x256", a, 1, s);
  if (p.fb == 8) return launch_tiles<4, 8, 1, false>("w8a8_gemm_128x256", a, 1, s);
  if (p.fb == 2)
    return p.splits > 1 ? launch_tiles<4, 2, 3, true>("w8a8_gemm_128x64_split", a, p.splits, s)
                        : launch_tiles<4, 2, 3, false>("w8a8_gemm_128x64", a, 1, s);
  return p.splits > 1 ? launch_tiles<4, 4, 2, true>("w8a8_gemm_128x128_split", a, p.splits, s)
                      : launch_tiles<4, 4, 2, false>("w8a8_gemm_128x128", a, 1, s);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

size_t gptq_w8a8_layer_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || rows > kMaxRows || gptq_tokens_ld(cols) == 0) return 0;
  const Geometry g = geometry(rows, cols);
  return g.rows_pad * g.k_pad > kMaxCodes ? 0 : layer_map(nullptr, g).bytes;
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
  if (!layer || tokens < 1 || tokens > kMaxTokens) return 0;
  const Geometry g = geometry(layer->rows, layer->cols);
  return part_bytes(g, tokens, plan_for(g, tokens, device_cu_count()));
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
    if (!aligned_to(codes, 16) || ld_codes % 16 || ld_codes < layer->k_pad ||
        ld_codes > (int64_t(1) << 22))
      return fail(GPTQ_ERR_INVALID_ARG,
                  "codes must be 16-byte aligned, ld_codes a multiple of 16 in "
                  "[gptq_tokens_ld(cols), 2^22]");
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
    const hipStream_t s = static_cast<hipStream_t>(stream);
    char *p = static_cast<char *>(ws);
    int8_t *codes = reinterpret_cast<int8_t *>(p);
    float *scale = reinterpret_cast<float *>(p + codes_bytes(layer, tokens));
    int32_t *sum = reinterpret_cast<int32_t *>(p + codes_bytes(layer, tokens) +
                                               align256(size_t(tokens) * 4));
    void *rest = p + codes_bytes(layer, tokens) + 2 * align256(size_t(tokens) * 4);
    GPTQ_TRY(quantize_impl(x, nullptr, x_dtype, tokens, layer->cols, ld_x, codes, layer->k_pad,
                           scale, sum, s, "quantize_tokens"));
    return gemm_launch(layer, codes, layer->k_pad, scale, sum, tokens, y, y_dtype, ld_y, rest, s);
  });
}

}  // extern "C"
