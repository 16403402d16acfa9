// The gated feed-forward block in 16 bits and its gradients: products on
// v_mfma_f32_16x16x32_{bf16,f16} with what belongs to them in the epilogue.
//
//   gate and up, v = silu(g) u     one product of both weights' rows, kGated
//   y = v W_down^T                 kPlain
//   dv = dy W_down, dg, du         kDGate: dv stays in registers
//   dW_down = dy^T v               kPlain
//   dW_gate, dW_up                 kPlain, two problems in one launch
//   dx = dg W_gate + du W_up       kPlain, both sums in one accumulator
//
// An operand is a matrix with contiguous rows.  Either its rows run along the
// contraction (k-major: x and the weights in the forward products) or the
// contraction runs across rows (m-major: the weights in products with
// gradients, everything in weight gradients); both are read from LDS as
// the matrix instruction takes them, so nothing is transposed in memory.
#include <algorithm>
#include <string>

#include "gptq_ff.h"
#include "silu.h"
#include "tiles.h"

namespace gptq {
namespace {

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));

enum Mode { kPlain, kGated, kDGate };

constexpr int kStep = 64;        // k per stage: 128 bytes of a k-major row

// C[c][r] = sum_k A[r][k] B[c][k], r along C's rows in memory.
struct Args {
  const uint16_t *a[2], *b[2];
  int64_t ld_a[2], ld_b[2];
  int rows, cols, k;       // r, c and k of one segment
  int segments;            // 2: the sums over a[0] b[0] and a[1] b[1] are one
  int problems;            // 2: a[0] b[0] -> out[0], a[0] b[1] -> out[1]
  uint16_t *out[3];        // kPlain C; kGated v, g, u (g NULL: v only); kDGate dg, du
  int64_t ld_out;
  int store_rows;          // kGated, kDGate: r up to which is written, zeros past `rows`
  const uint16_t *g, *u;   // kDGate
  f32x4_t *part;           // split sums
  int splits;
};

__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }
// m-major rows of 64 F bytes hold 2 F chunks of 16 values, permuted by k: the
// eight rows that half a wave reads at a time lie in different banks.
template <int F>
__device__ __forceinline__ int chunk_swz(int k) {
  return F >= 4 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
}

template <typename T>
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (__is_same(T, bf16_t)) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  } else {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
}
// In place, in accumulation registers (the builtin leaves the result's register
// free, which costs moves where all are taken).  Operands come from LDS reads.
// An accumulator is next touched at least 8 instructions later, as the
// accumulator of the same instruction; settle() waits the pipeline out.
template <typename T>
__device__ __forceinline__ void mfma_acc(f32x4_t &acc, u32x4_t a, u32x4_t b) {
  if constexpr (sizeof(T) == 2 && __is_same(T, bf16_t))
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  else
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
template <int FA, int FB>
__device__ __forceinline__ void settle(f32x4_t (&acc)[FA][FB]) {
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

// What a wave's sums become.  acc holds FA blocks of rows (kGated: half of them of
// gate, then as many of up, for the same rows of v).
template <typename T, Mode M, int FA, int FB>
__device__ __forceinline__ void finish(const Args &a, const f32x4_t (&acc)[FA][FB], int problem,
                                       int r0, int t0, int lane, uint8_t *lds) {
  auto value = [&](int i, int j) { return acc[i][j]; };
  if constexpr (M == kPlain) {
    store_turned<T, FA, FB>(value, reinterpret_cast<T *>(a.out[problem]), a.ld_out, a.rows,
                            a.cols, r0, t0, lane, lds);
    return;
  }
  constexpr int kPieces = M == kGated ? FA : 2 * FA;
  struct Pair {
    Pack8<T> g, u;
  };
  auto first = [&](int c, int piece) {
    Pair k{};
    if constexpr (M == kDGate) {
      // a.store_rows is a multiple of 8: eight rows of g and u are there
      const int64_t at = int64_t(min(t0 + c, a.cols - 1)) * a.ld_out +
                         min(r0 + 8 * piece, a.store_rows - 8);
      k.g = fetch8<kWhole>(reinterpret_cast<const T *>(a.g) + at, 0, 8);
      k.u = fetch8<kWhole>(reinterpret_cast<const T *>(a.u) + at, 0, 8);
    }
    return k;
  };
  turned<FA, FB, kPieces, M == kDGate ? 4 : 2>(value, lane, lds, first, [&](int c, int piece,
                                                                          const Pair &k,
                                                                          auto read) {
    const int r = r0 + 8 * piece;
    if (t0 + c >= a.cols || r >= a.store_rows) return;
    const int64_t at = int64_t(t0 + c) * a.ld_out + r;
    T *out0 = reinterpret_cast<T *>(a.out[0]) + at;
    const int n = a.rows - r;       // zeros from there to the padded row's end
    if constexpr (M == kGated) {
      float g[8], u[8];
      read(piece, g);
      read(piece + FA, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= n) g[e] = u[e] = 0.f;
      }
      if (a.out[1]) {
        store8(reinterpret_cast<T *>(a.out[1]) + at, 8, g);
        store8(reinterpret_cast<T *>(a.out[2]) + at, 8, u);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = silu(g[e]) * u[e];
      store8(out0, 8, g);
    } else {
      float dg[8], du[8];
      read(piece, dg);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = k.g.at(e), dv = dg[e];
        // s = 1 / (1 + e^-|g|): p and 1 - p without cancellation or overflow
        const float x = expf(-fabsf(g)), s = 1.f / (1.f + x), xs = x * s;
        const float p = g < 0.f ? xs : s, rest = g < 0.f ? s : xs;
        dg[e] = e < n ? dv * k.u.at(e) * (p * __builtin_fmaf(g, rest, 1.f)) : 0.f;
        du[e] = e < n ? dv * (g * p) : 0.f;
      }
      store8(out0, 8, dg);
      store8(reinterpret_cast<T *>(a.out[1]) + at, 8, du);
    }
  });
}

// ---- A workgroup of 4 waves (2 x 2) makes a tile of 32 FA rows x 32 FB
// columns; a wave FA x FB blocks of 16 x 16.  Stages of 64 k are
// double-buffered in LDS, copied there by loads that write LDS directly, and read into
// registers a step before they are multiplied.  Step 0 of stage u multiplies the first
// half of a wave's rows with all of its columns while the other half is read, step 1
// that one while the first half and the columns of stage u + 1 are read.  What a step has
// read is asked for in the next one, of stage u + 2: a copy has a whole stage and more to
// arrive, and a barrier waits for copies that were asked for two steps ago.  Halves of the
// rows, not of k, so that a copy takes whole 128-byte lines: with halves of k 4096 x
// 4096 x 11008 took 314 us.  Reads and copies are spread over the matrix instructions: more
// of them in a row than fit in the shadow of one leave the matrix unit idle, as this is
// the only wave of its SIMD.  A stage that k does not fill comes last, on its own, with
// zeros.  Bound by the matrix instructions, and the clock under them: bfloat16 4096 x
// 4096 x 11008 247 us (1.50 PFLOP/s, 73 % of the cycles at 1.92 GHz), k 22016 478 us (1.55,
// 80 % at 1.84); a round of tiles adds 20 us of first loads and epilogue, with dg and du 59.
__device__ const uint32_t kZeros[4] = {0, 0, 0, 0};

template <typename T, bool AM, bool BM, int FA, int FB, Mode M>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
    ff_tile_kernel(Args a, int col_tiles, int row_tiles) {
  constexpr int H = FA / 2;                // blocks of rows in a half
  constexpr int kHalfBytes = 32 * H * 128, kABytes = 2 * kHalfBytes, kBBytes = 32 * FB * 128;
  constexpr int kStageBytes = kABytes + kBBytes;
  constexpr int kCopies = FA + FB;         // KiB per wave and stage: A's halves, B
  constexpr int kSlots = 2 * H * FB;       // matrix instructions of a step
  constexpr int kOutRows = M == kGated ? 16 * FA : 32 * FA;    // rows of C in a tile
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles = col_tiles * row_tiles;
  const int at = xcd_run(int(blockIdx.x), tiles * a.problems);
  const int problem = __builtin_amdgcn_readfirstlane(at / tiles);
  int tt, tr;
  band_tile(at - problem * tiles, col_tiles, row_tiles, tt, tr);
  const int m0 = tr * kOutRows, n0 = tt * 32 * FB;
  const int full = a.k / kStep, U = full * a.segments;

  // Copy q of a wave and stage.  k-major: eight rows of 128 bytes; m-major: rows of k.
  // voff: bytes from the stage's start.  Rows past the operand are clamped; they only
  // feed outputs that are not stored, or stored as zeros.
  auto of_a = [](int q) { return q < FA; };
  auto source = [](int q) { return M == kGated && q >= H && q < FA; };   // gate's half, then up's
  auto kib_of = [&](int q) { return 4 * (q < FA ? q % H : q - FA) + wave; };
  // Row R of the LDS rows of A's half -> row of the tile.
  auto tile_row = [&](int q, int R) {
    return M == kGated ? R : R / (16 * H) * (16 * FA) + q / H * (16 * H) + R % (16 * H);
  };
  auto m_width = [](int q) { return q < FA ? H : FB; };        // m-major: 32 of them are a row
  auto m_row = [&](int q) { return 16 / m_width(q) * kib_of(q) + lane / (4 * m_width(q)); };
  auto k_piece = [&](int q) { return (lane & 7) ^ swz(8 * kib_of(q) + (lane >> 3)); };
  uint32_t voff[kCopies];
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int64_t ld = of_a(q) ? (source(q) ? a.ld_a[1] : a.ld_a[0]) : a.ld_b[0];
    const int first = of_a(q) ? min(m0, a.rows - 1) : n0, last = (of_a(q) ? a.rows : a.cols) - 1;
    if (of_a(q) ? AM : BM) {
      const int F = m_width(q), k = m_row(q), pos = lane % (4 * F);
      const int swzd = F == 8 ? chunk_swz<8>(k) : F == 4 ? chunk_swz<4>(k) : chunk_swz<2>(k);
      const int c = 16 * ((pos >> 1) ^ swzd) + 8 * (pos & 1);
      voff[q] = uint32_t(k) * uint32_t(2 * ld) +
                2 * min((of_a(q) ? m0 + tile_row(q, c) : n0 + c), last & ~7);
    } else {
      const int R = 8 * kib_of(q) + (lane >> 3);
      voff[q] = uint32_t(min(of_a(q) ? tile_row(q, R) : R, last - first)) * uint32_t(2 * ld) +
                (k_piece(q) << 4);
    }
  }
  // Of the two sources, segments or problems (selected by ?:, so that they stay scalar).
  const int64_t am0 = AM ? 0 : min(m0, a.rows - 1), bn0 = BM ? 0 : n0;
  const uint16_t *abase0 = a.a[0] + am0 * a.ld_a[0], *abase1 = a.a[1] + am0 * a.ld_a[1];
  const uint16_t *bfirst = a.b[0] + bn0 * a.ld_b[0], *bbase1 = a.b[1] + bn0 * a.ld_b[1];
  const uint16_t *bbase0 = problem ? bbase1 : bfirst;
  const int64_t step_a = AM ? kStep * a.ld_a[0] : kStep, step_b = BM ? kStep * a.ld_b[0] : kStep;
  auto stage_base = [&](int q, int t) {    // t counts stages over both segments
    const bool second = M == kPlain && AM && !BM && t >= full;
    const int64_t at = second ? t - full : t;
    if (of_a(q)) return ((M == kGated ? source(q) : second) ? abase1 : abase0) + at * step_a;
    return (second ? bbase1 : bbase0) + at * step_b;
  };
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t *)smem));
  auto lds_of = [&](int q) {
    return (of_a(q) ? q / H * kHalfBytes : kABytes) + kib_of(q) * 1024;
  };
  auto copy_one = [&](int q, int t) {      // past the last stage: that one again, not read
    copy16_to_lds(reinterpret_cast<const uint8_t *>(stage_base(q, min(t, U - 1))), voff[q],
                  lds0 + (t & 1) * kStageBytes + lds_of(q));
  };
  // Block `blk` of 16 rows, k = 32 h + 8 (lane / 16) .. + 7.
  auto read_k = [&](const uint8_t *at, int blk, int h) {
    const int row = 16 * blk + (lane & 15), c = 4 * h + (lane >> 4);
    return *reinterpret_cast<const u32x4_t *>(at + row * 128 + ((c ^ swz(row)) << 4));
  };
  auto read_m = [&](const uint8_t *at, int blk, int h, auto f) {
    // Four rows of 16 values per 16 lanes and read, turned: a lane gets one
    // column's four.
    constexpr int F = decltype(f)::value;
    i32x2_t w[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int k = 32 * h + 8 * (lane >> 4) + 4 * p + ((lane >> 2) & 3);
      auto src = (__attribute__((address_space(3))) s16x4_t *)(at + k * (64 * F) +
                                                               ((blk ^ chunk_swz<F>(k)) << 5) +
                                                               8 * (lane & 3));
      w[p] = __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(src));
    }
    return u32x4_t{uint32_t(w[0][0]), uint32_t(w[0][1]), uint32_t(w[1][0]), uint32_t(w[1][1])};
  };
  u32x4_t fa[2][FA], fb[2][2 * FB];        // A's halves; B's stages by turns; k's halves in either
  auto read_a = [&](int u, int half, int f) {
    const uint8_t *at = smem + (u & 1) * kStageBytes + half * kHalfBytes;
    if constexpr (AM)
      fa[half][f] = read_m(at, wm * H + f % H, f / H, std::integral_constant<int, H>{});
    else
      fa[half][f] = read_k(at, wm * H + f % H, f / H);
  };
  auto read_b = [&](int u, int to, int f) {
    const uint8_t *at = smem + (u & 1) * kStageBytes + kABytes;
    if constexpr (BM)
      fb[to][f] = read_m(at, wn * FB + f % FB, f / FB, std::integral_constant<int, FB>{});
    else
      fb[to][f] = read_k(at, wn * FB + f % FB, f / FB);
  };

  f32x4_t acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  settle<FA, FB>(acc);     // the zeros are written well before the first MFMA reads them
  auto multiply = [&](int half, int of, int n) {
    const int h = n / (H * FB), i = n / FB % H, j = n % FB;
    mfma_acc<T>(acc[half * H + i][j], fa[half][h * H + i], fb[of][h * FB + j]);
  };

  if (U > 0) {
    // In the order of the loop: A's first half and B, A's second half.
    auto first_copy = [](int n) { return n < H ? n : n - H + FA; };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < H + FB; ++n) copy_one(first_copy(n), t);
#pragma unroll
      for (int q = H; q < FA; ++q) copy_one(q, t);
    }
    copies_done<kCopies>();
    lds_barrier();
#pragma unroll
    for (int f = 0; f < FA; ++f) read_a(0, 0, f);
#pragma unroll
    for (int f = 0; f < 2 * FB; ++f) read_b(0, 0, f);
    lds_barrier();                           // before anything is asked for in their place
    for (int u0 = 0; u0 < U; u0 += 2) {
#pragma unroll
      for (int turn = 0; turn < 2; ++turn) {
        const int u = u0 + turn;
        if (turn && u >= U) break;
        constexpr int kRead0 = (kSlots - 8) / FA, kCopy0 = kSlots / (H + FB);
        constexpr int kRead1 = (kSlots - 8) / (FA + 2 * FB), kCopy1 = kSlots / H;
#pragma unroll
        for (int n = 0; n < kSlots; ++n) {
          multiply(0, turn, n);
          if (n % kRead0 == 0 && n / kRead0 < FA) read_a(u, 1, n / kRead0);
          if (n % kCopy0 == kCopy0 / 2 && n / kCopy0 < H + FB) copy_one(first_copy(n / kCopy0), u + 2);
          __builtin_amdgcn_sched_barrier(0);
        }
        copies_done<kCopies>();              // but for those of the last two steps
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kSlots; ++n) {
          multiply(1, turn, n);
          if (n % kRead1 == 0 && n / kRead1 < FA + 2 * FB) {   // past the last stage: not used
            const int f = n / kRead1;
            if (f < FA) read_a(u + 1, 0, f);
            else read_b(u + 1, 1 - turn, f - FA);
          }
          if (n % kCopy1 == kCopy1 / 2) copy_one(H + n / kCopy1, u + 2);
          __builtin_amdgcn_sched_barrier(0);
        }
        copies_done<kCopies>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    copies_done<0>();                        // none may land in what follows
  }
  const int rest = a.k - full * kStep;
  if (rest > 0) {
    for (int seg = 0; seg < a.segments; ++seg) {
      lds_barrier();                         // every wave is done with the stages
#pragma unroll
      for (int q = 0; q < kCopies; ++q) {
        const bool m = of_a(q) ? AM : BM;
        const int64_t ld = of_a(q) ? a.ld_a[0] : a.ld_b[0];
        const int k = m ? m_row(q) : 8 * k_piece(q);   // this lane's row of k, or first k
        const uint16_t *src =
            (of_a(q) ? (M == kGated ? source(q) : seg) ? abase1 : abase0 : seg ? bbase1 : bbase0) +
            (m ? ld : 1) * int64_t(full) * kStep;
        const void *mine = reinterpret_cast<const uint8_t *>(src) + voff[q];
        copy16_to_lds(k < rest ? mine : kZeros, lds0 + lds_of(q));
      }
      copies_done<0>();
      lds_barrier();
#pragma unroll
      for (int f = 0; f < 2 * FB; ++f) read_b(0, 0, f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int f = 0; f < FA; ++f) read_a(0, half, f);
#pragma unroll
        for (int n = 0; n < kSlots; ++n) multiply(half, 0, n);
      }
    }
  }
  settle<FA, FB>(acc);
  lds_barrier();                           // every wave is done with the stages
  finish<T, M>(a, acc, problem, m0 + wm * (kOutRows / 2), n0 + wn * 16 * FB, lane,
               smem + wave * (kStageBytes / 2));
}

// ---- Smaller tiles: eight waves (2 x 4) make a tile of 128 rows x 64 FB columns, a
// wave 4 x FB blocks.  Two waves per SIMD hide each other's waits, where tiles of four
// waves as above left the matrix units idle for lack of tiles.  Stages lie in a ring of
// NBUF buffers in LDS, copied there by loads that write LDS directly.  A stage is
// SUB parts of 64 k; each half of a part is multiplied while the next is read.  Once
// a stage's last half is read, a barrier tells that every wave has read stage u and
// that stage u + 1 is there: stage u + NBUF is asked for, into u's buffer, and the last
// half is multiplied while u + 1's first is read.  (128 x 64 tiles have 8 matrix
// instructions per wave in 64 k, few for a barrier: they take 128.)  Where k does not
// fill a stage, lanes past it copy zeros.  What bounds it is a stage's way from the caches,
// not its rate: 777 x 1001 x 2731 float16 13 to 22 us a product (0.2 to 0.4 PFLOP/s).
constexpr int ring_lds(int fb, int sub, int nbuf) { return nbuf * sub * (128 + 64 * fb) * 128; }

template <typename T, bool AM, bool BM, int FB, int SUB, int NBUF, Mode M>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
    ff_ring_kernel(Args a, int col_tiles, int row_tiles) {
  constexpr int FA = 4, WN = 4, kCols = 16 * FB * WN;
  constexpr int kABytes = 128 * 128, kBBytes = kCols * 128, kPartBytes = kABytes + kBBytes;
  constexpr int kStageBytes = SUB * kPartBytes, kStageK = SUB * kStep;
  constexpr int kACopies = kABytes / 8192, kBCopies = kBBytes / 8192;   // KiB per wave
  constexpr int kCopies = kACopies + kBCopies;                          // of a part
  constexpr int kOutRows = M == kGated ? 64 : 128;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = col_tiles * row_tiles;
  const int at = xcd_run(int(blockIdx.x), tiles * a.problems * a.splits);
  const int unit = __builtin_amdgcn_readfirstlane(at / tiles);
  const int problem = unit / a.splits, split = unit % a.splits, tile = at - unit * tiles;
  int tt, tr;
  band_tile(tile, col_tiles, row_tiles, tt, tr);
  const int m0 = tr * kOutRows, n0 = tt * kCols;
  const int whole = a.k / kStageK, rest = a.k - whole * kStageK;   // of a segment
  const int each = whole + (rest > 0), all = each * a.segments;
  const int s0 = int(int64_t(all) * split / a.splits);
  const int s1 = int(int64_t(all) * (split + 1) / a.splits), U = s1 - s0;

  // Copy q of a wave and part: a KiB of A, then of B.  k-major: eight rows of 128
  // bytes; m-major: rows of k.  voff: bytes from the part's start; kof: the lane's row of
  // k, or first k.  Rows past the operand are clamped; they only feed outputs that are not
  // stored, or stored as zeros.
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t *)smem));
  uint32_t voff[kCopies];
  int kof[kCopies];
  auto source = [&](int q) {               // kGated: whether copy q is of up
    return M == kGated && q < kACopies && ((wave * kACopies + q) >> 1) % FA >= FA / 2;
  };
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const bool of_a = q < kACopies, m = of_a ? AM : BM;
    const int kib = of_a ? wave * kACopies + q : wave * kBCopies + q - kACopies;
    const int64_t ld = of_a ? (source(q) ? a.ld_a[1] : a.ld_a[0]) : a.ld_b[0];
    const int width = of_a ? 128 : kCols;
    if (m) {
      const int per = width / 8, k = 64 / per * kib + lane / per, pos = lane % per;
      const int swzd = width == 128 ? chunk_swz<4>(k) : width == 256 ? chunk_swz<8>(k)
                                                                     : chunk_swz<2>(k);
      const int c = 16 * ((pos >> 1) ^ swzd) + 8 * (pos & 1);
      kof[q] = k;
      voff[q] = uint32_t(k) * uint32_t(2 * ld) +
                2 * min((of_a ? m0 : n0) + c, ((of_a ? a.rows : a.cols) - 1) & ~7);
    } else {
      const int R = 8 * kib + (lane >> 3), piece = (lane & 7) ^ swz(R);
      int r = R;
      if (M == kGated && of_a) {           // blocks of 16: two of gate, two of up per wave
        const int blk = R >> 4, i = blk % FA;
        r = 16 * (blk / FA * (FA / 2) + i % (FA / 2)) + (R & 15);
      }
      const int left = of_a ? a.rows - 1 - m0 : a.cols - 1 - n0;
      kof[q] = 8 * piece;
      voff[q] = uint32_t(min(r, left)) * uint32_t(2 * ld) + 16 * piece;
    }
  }
  const int64_t am0 = AM ? 0 : m0, bn0 = BM ? 0 : n0;
  const uint16_t *a0 = a.a[0] + am0 * a.ld_a[0], *a1 = a.a[1] + am0 * a.ld_a[1];
  const uint16_t *bfirst = a.b[0] + bn0 * a.ld_b[0], *b1 = a.b[1] + bn0 * a.ld_b[1];
  const uint16_t *b0 = problem ? b1 : bfirst;
  // Bytes from one part to the next.
  const int64_t step_a = 2 * (AM ? kStep * a.ld_a[0] : kStep);
  const int64_t step_a1 = 2 * (AM ? kStep * a.ld_a[1] : kStep);
  const int64_t step_b = 2 * (BM ? kStep * a.ld_b[0] : kStep);
  // The next stage to be copied, and how many stages from it on are whole.
  int g = s0, run;
  const uint8_t *pa, *pa1, *pb;
  auto seek = [&]() {
    const bool second = g >= each;         // the second segment
    const int kk = second ? g - each : g;
    pa = reinterpret_cast<const uint8_t *>(second ? a1 : a0) + kk * (SUB * step_a);
    pa1 = reinterpret_cast<const uint8_t *>(a1) + kk * (SUB * step_a1);
    pb = reinterpret_cast<const uint8_t *>(second ? b1 : b0) + kk * (SUB * step_b);
    run = min(whole - kk, s1 - g);
  };
  seek();
  auto lds_of = [&](int q) {
    return q < kACopies ? (wave * kACopies + q) * 1024
                        : kABytes + (wave * kBCopies + q - kACopies) * 1024;
  };
  auto copy_next = [&](int buf) {          // past the last stage: zeros, not read
    const uint32_t to = lds0 + buf * kStageBytes;
    if (run > 0) {
#pragma unroll
      for (int p = 0; p < SUB; ++p) {
#pragma unroll
        for (int q = 0; q < kCopies; ++q)
          copy16_to_lds(q < kACopies ? source(q) ? pa1 : pa : pb, voff[q],
                        to + p * kPartBytes + lds_of(q));
        pa += step_a;
        if (M == kGated) pa1 += step_a1;
        pb += step_b;
      }
      --run;
    } else {
      const int left = g < s1 ? rest : 0;
#pragma unroll
      for (int p = 0; p < SUB; ++p)
#pragma unroll
        for (int q = 0; q < kCopies; ++q) {
          const void *mine = (q < kACopies ? (source(q) ? pa1 + p * step_a1 : pa + p * step_a)
                                           : pb + p * step_b) + voff[q];
          copy16_to_lds(kof[q] + p * kStep < left ? mine : kZeros, to + p * kPartBytes + lds_of(q));
        }
    }
    ++g;
    if (run == 0 && g == each && g < s1) seek();
  };
  auto read_k = [&](const uint8_t *at, int blk, int h) {
    const int row = 16 * blk + (lane & 15), c = 4 * h + (lane >> 4);
    return *reinterpret_cast<const u32x4_t *>(at + row * 128 + ((c ^ swz(row)) << 4));
  };
  auto read_m = [&](const uint8_t *at, int blk, int h, auto f) {
    constexpr int F = decltype(f)::value;
    i32x2_t w[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int k = 32 * h + 8 * (lane >> 4) + 4 * p + ((lane >> 2) & 3);
      auto src = (__attribute__((address_space(3))) s16x4_t *)(at + k * (64 * F) +
                                                               ((blk ^ chunk_swz<F>(k)) << 5) +
                                                               8 * (lane & 3));
      w[p] = __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(src));
    }
    return u32x4_t{uint32_t(w[0][0]), uint32_t(w[0][1]), uint32_t(w[1][0]), uint32_t(w[1][1])};
  };
  struct Half {
    u32x4_t a[FA], b[FB];
  };
  auto read = [&](Half &x, int buf, int half) {   // half: of the stage's 2 SUB
    const uint8_t *at = smem + buf * kStageBytes + (half >> 1) * kPartBytes;
    const int h = half & 1;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      if constexpr (BM)
        x.b[j] = read_m(at + kABytes, wn * FB + j, h, std::integral_constant<int, kCols / 32>{});
      else
        x.b[j] = read_k(at + kABytes, wn * FB + j, h);
    }
#pragma unroll
    for (int i = 0; i < FA; ++i) {
      if constexpr (AM) x.a[i] = read_m(at, wm * FA + i, h, std::integral_constant<int, 4>{});
      else x.a[i] = read_k(at, wm * FA + i, h);
    }
  };
  f32x4_t acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Half &x) {
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[i][j] = mfma<T>(x.a[i], x.b[j], acc[i][j]);
  };
  for (int u = 0; u < NBUF; ++u) copy_next(u);
  copies_done<(NBUF - 1) * SUB * kCopies>();
  lds_barrier();
  Half x[2];
  read(x[0], 0, 0);
  int buf = 0;                             // u % NBUF
  for (int u = 0; u < U; ++u) {
    const int after = buf + 1 == NBUF ? 0 : buf + 1;
#pragma unroll
    for (int half = 0; half < 2 * SUB - 1; ++half) {
      read(x[(half + 1) & 1], buf, half + 1);
      multiply(x[half & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    copies_done<(NBUF - 2) * SUB * kCopies>();
    lds_barrier();
    copy_next(buf);
    __builtin_amdgcn_sched_barrier(0);
    read(x[0], after, 0);                  // past the last stage: zeros, not used
    multiply(x[1]);
    __builtin_amdgcn_sched_barrier(0);
    buf = after;
  }
  copies_done<0>();                        // none may land in what follows
  if (a.splits > 1) {
    // A wave's blocks as they lie in its registers: 1 KiB per store.
    f32x4_t *p = a.part + int64_t(problem * tiles + tile) * a.splits * (8 * FA * FB * 64) +
                 (split * 8 + wave) * (FA * FB * 64) + lane;
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) p[(i * FB + j) * 64] = acc[i][j];
    return;
  }
  lds_barrier();                           // every wave is done with the stages
  finish<T, M>(a, acc, problem, m0 + wm * (kOutRows / 2), n0 + wn * 16 * FB, lane,
               smem + wave * (64 * FA * 16 * ((FB + 1) / 2)));
}

// Adds a split product's parts, in their order: a wave per block of rows (kGated: of
// gate and of up) of a tile's wave, in the tile kernel's register order.  777 x 1001 in two
// parts: 4.9 us.
template <typename T, int FB, Mode M>
__global__ void __launch_bounds__(256) ff_join_kernel(Args a, int col_tiles, int row_tiles) {
  constexpr int FA = 4, kOutRows = M == kGated ? 64 : 128, H = kOutRows / 32;
  constexpr int NI = M == kGated ? 2 : 1, kPiece = 64 * NI * 16 * ((FB + 1) / 2);
  __shared__ __align__(16) uint8_t lds[4 * kPiece];
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int i = unit % H, wave = unit / H % 8, tile = unit / (8 * H);
  const int tiles = col_tiles * row_tiles, problem = tile / tiles;
  int tt, tr;
  band_tile(tile - problem * tiles, col_tiles, row_tiles, tt, tr);
  const int r0 = tr * kOutRows + (wave / 4) * (kOutRows / 2) + 16 * i;
  const int t0 = (tt * 4 + wave % 4) * 16 * FB;
  if (r0 >= a.store_rows || t0 >= a.cols) return;
  const f32x4_t *p = a.part + int64_t(tile) * a.splits * (8 * FA * FB * 64) +
                     wave * (FA * FB * 64) + lane;
  f32x4_t acc[NI][FB];
#pragma unroll
  for (int n = 0; n < NI; ++n)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[n][j] = p[((n * H + i) * FB + j) * 64];
  for (int s = 1; s < a.splits; ++s) {
    p += 8 * FA * FB * 64;
#pragma unroll
    for (int n = 0; n < NI; ++n)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[n][j] += p[((n * H + i) * FB + j) * 64];
  }
  finish<T, M>(a, acc, problem, r0, t0, lane, lds + (threadIdx.x >> 6) * kPiece);
}

// ---- Few tokens: a workgroup per 16 rows of the weights, its waves splitting k.  A
// wave takes every WAVES-th step of 64 k; its weights come straight from memory, two
// sets of steps ahead, and each is used for all tokens at once.  The waves' sums
// meet in LDS.  Rows may start anywhere: nothing is copied for alignment.  Memory bounds
// it: 1 token bfloat16, two weights of 11008 x 4096 32 us (5.6 TB/s), 4096 x 11008 17.7 us.
constexpr int kRowsWaves = 4;
constexpr int64_t kRowsTokens = 16;

struct RowsArgs {
  const uint16_t *w[2];    // gate and up, or one weight
  int64_t ld_w[2];
  const uint16_t *x;
  int64_t ld_x;
  int rows, tokens, k;
  uint16_t *y, *g, *u;     // g, u: NULL, or the gated product's factors
  int64_t ld_y;
};

template <typename T, bool GATED>
__global__ void __launch_bounds__(64 * kRowsWaves) ff_rows_kernel(RowsArgs a) {
  constexpr int WAVES = kRowsWaves, W = GATED ? 2 : 1;
  constexpr int kAhead = GATED ? 2 : 4;   // steps loaded at a time, two such sets in flight
  __shared__ f32x4_t sums[W * WAVES * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = blockIdx.x * 16, full = a.k / kStep;
  const int row = min(r0 + (lane & 15), a.rows - 1), token = min(lane & 15, a.tokens - 1);
  const uint16_t *src[W + 1];             // the weights' rows, then the token's
#pragma unroll
  for (int m = 0; m < W; ++m) src[m] = a.w[m] + int64_t(row) * a.ld_w[m] + 8 * (lane >> 4);
  src[W] = a.x + int64_t(token) * a.ld_x + 8 * (lane >> 4);
  struct Set {
    u32x4_t v[kAhead][2][W + 1];
  };
  const int n = (full - wave + WAVES - 1) / WAVES;      // loads past the last step repeat it
  auto load = [&](Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t k = (wave + int64_t(min(at + i, n - 1)) * WAVES) * kStep;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m <= W; ++m) __builtin_memcpy(&b.v[i][h][m], src[m] + k + 32 * h, 16);
    }
  };
  f32x4_t acc[W];
#pragma unroll
  for (int m = 0; m < W; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply_one = [&](const u32x4_t (&v)[W + 1]) {
#pragma unroll
    for (int m = 0; m < W; ++m) acc[m] = mfma<T>(v[m], v[W], acc[m]);
  };
  auto multiply = [&](const Set &b, int at) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (at + i >= n) break;
      multiply_one(b.v[i][0]);
      multiply_one(b.v[i][1]);
    }
  };
  if (n > 0) {
    Set s0, s1;
    load(s0, 0);
    load(s1, kAhead);
    for (int at = 0; at < n; at += 2 * kAhead) {
      multiply(s0, at);
      if (at + 2 * kAhead < n) load(s0, at + 2 * kAhead);
      multiply(s1, at + kAhead);
      if (at + 3 * kAhead < n) load(s1, at + 3 * kAhead);
    }
  }
  if (wave == full % WAVES && a.k > full * kStep) {     // a step that k does not fill
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t v[W + 1];
      const int k = full * kStep + 32 * h, left = a.k - k - 8 * (lane >> 4);
#pragma unroll
      for (int m = 0; m <= W; ++m) {
        v[m] = u32x4_t{0, 0, 0, 0};
        if (left >= 8) {
          __builtin_memcpy(&v[m], src[m] + k, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e < left) v[m][e >> 1] |= uint32_t(src[m][k + e]) << (16 * (e & 1));
        }
      }
      multiply_one(v);
    }
  }
#pragma unroll
  for (int m = 0; m < W; ++m) sums[(m * WAVES + wave) * 64 + lane] = acc[m];
  lds_barrier();
  // Output (token, row) of thread: 16 consecutive rows per token.  Lane
  // 16 (r / 4) + t of a block holds rows 4 (r / 4) .. + 3 of token t.
  const float *flat = reinterpret_cast<const float *>(sums);
  if (tid >= 16 * a.tokens) return;
  const int t = tid >> 4, r = tid & 15, at = (16 * (r >> 2) + t) * 4 + (r & 3);
  if (r0 + r >= a.rows) return;
  float y[W];
#pragma unroll
  for (int m = 0; m < W; ++m) {
    y[m] = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) y[m] += flat[(m * WAVES + i) * 256 + at];
  }
  const int64_t to = int64_t(t) * a.ld_y + r0 + r;
  if constexpr (GATED) {
    if (a.g) {
      a.g[to] = narrow<T>(y[0]).bits;
      a.u[to] = narrow<T>(y[1]).bits;
    }
    y[0] = silu(y[0]) * y[1];
  }
  a.y[to] = narrow<T>(y[0]).bits;
}

// ------------------------------------------------------------------ copies
// Rows copied to multiples of 8 values, zeros following: for operands whose
// 16-byte pieces are not aligned.  All of a call's in one launch: the weights and tokens of
// 777 x 1001 x 2731 9 us (4 TB/s, read and written).
struct Pad {
  const uint16_t *src;
  uint16_t *dst;
  int64_t ld, end;         // pieces of this matrix and those before it
  int cols, pieces;        // per row
};
constexpr int kMaxPads = 5;
struct Pads {
  Pad p[kMaxPads];
  int n;
};
__global__ void __launch_bounds__(256) ff_pad_kernel(Pads a) {
  const int64_t n = a.p[a.n - 1].end;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    Pad m = a.p[0];
    int64_t at = i;
#pragma unroll
    for (int k = 1; k < kMaxPads; ++k)
      if (k < a.n && i >= a.p[k - 1].end) {
        m = a.p[k];
        at = i - a.p[k - 1].end;
      }
    const int64_t r = at / m.pieces;
    const int c = int(at - r * m.pieces) * 8;
    const uint16_t *p = m.src + r * m.ld + c;
    u32x4_t v = {0, 0, 0, 0};
    if (c + 8 <= m.cols) {
      __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (c + e < m.cols) v[e >> 1] |= uint32_t(p[e]) << (16 * (e & 1));
    }
    *reinterpret_cast<u32x4_t *>(m.dst + at * 8) = v;
  }
}
// The weights' gradients where there is no token.
__global__ void __launch_bounds__(256)
    ff_zero_kernel(uint16_t *__restrict__ p, int64_t ld, int64_t rows, int cols) {
  const int64_t n = rows * cols;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
    p[i / cols * ld + i % cols] = 0;
}

// -------------------------------------------------------------------- host
constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxSide = 65536;
// A tile's rows are reached with 32-bit offsets of bytes.
constexpr int64_t kMaxLd = int64_t(1) << 22;

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
bool direct(const void *p, int64_t rows, int64_t cols, int64_t ld) {
  return cols % 8 == 0 && aligned_to(p, 16) && (rows == 1 || (ld % 8 == 0 && ld <= kMaxLd));
}
size_t padded_bytes(int64_t rows, int64_t cols) { return align256(size_t(rows) * up8(cols) * 2); }

struct Operand {
  const uint16_t *p;
  int64_t ld;
};
// Scratch in the order it is taken.
struct Arena {
  uintptr_t base;
  size_t at = 0;
  uint16_t *take(size_t bytes) {
    uint16_t *p = reinterpret_cast<uint16_t *>(base + at);
    at += align256(bytes);
    return p;
  }
};
// The operands themselves, or where their padded copies go.
struct Padder {
  Arena &ws;
  Pads pads{};
  Operand operator()(const void *p, int64_t rows, int64_t cols, int64_t ld, bool copy) {
    const uint16_t *src = static_cast<const uint16_t *>(p);
    if (!copy) return {src, rows == 1 ? up8(cols) : ld};
    uint16_t *dst = ws.take(padded_bytes(rows, cols));
    const int64_t pieces = up8(cols) / 8, before = pads.n ? pads.p[pads.n - 1].end : 0;
    pads.p[pads.n++] = {src, dst, ld, before + rows * pieces, int(cols), int(pieces)};
    return {dst, up8(cols)};
  }
  gptq_status launch_all(hipStream_t s) const {
    if (pads.n == 0) return GPTQ_OK;
    const int64_t blocks = std::min<int64_t>(cdiv(pads.p[pads.n - 1].end, 256), 1 << 14);
    return launch("ff_pad", ff_pad_kernel, dim3(uint32_t(blocks)), dim3(256), 0, s, pads);
  }
};

bool overlap(const void *a, int64_t rows_a, int64_t cols_a, int64_t ld_a, const void *b,
             int64_t rows_b, int64_t cols_b, int64_t ld_b) {
  return matrices_meet(a, rows_a, cols_a, ld_a, 2, b, rows_b, cols_b, ld_b, 2);
}

gptq_status check_ff(const gptq_ff *f) {
  if (!f) return fail(GPTQ_ERR_INVALID_ARG, "ff is NULL");
  if (f->d < 1 || f->d > kMaxSide || f->inner < 1 || f->inner > kMaxSide)
    return fail(GPTQ_ERR_INVALID_ARG, "d and inner must be in [1, 65536]");
  if (f->dtype != GPTQ_DT_BF16 && f->dtype != GPTQ_DT_F16)
    return fail(GPTQ_ERR_INVALID_ARG, "dtype must be BF16 or F16");
  if (!f->gate || !f->up || !f->down)
    return fail(GPTQ_ERR_INVALID_ARG, "gate, up and down must not be NULL");
  if (!aligned_to(f->gate, 2) || !aligned_to(f->up, 2) || !aligned_to(f->down, 2))
    return fail(GPTQ_ERR_INVALID_ARG, "gate, up and down must be aligned to their elements");
  if (f->ld_gate < f->d || f->ld_up < f->d || f->ld_down < f->inner)
    return fail(GPTQ_ERR_INVALID_ARG, "the row stride of a weight is below its width");
  return GPTQ_OK;
}
gptq_status check_matrix(const void *p, int64_t ld, int64_t cols, const char *what) {
  const std::string w(what);
  if (!p) return fail(GPTQ_ERR_INVALID_ARG, w + " must not be NULL");
  if (!aligned_to(p, 2)) return fail(GPTQ_ERR_INVALID_ARG, w + " must be aligned to its elements");
  if (ld < cols)
    return fail(GPTQ_ERR_INVALID_ARG, "the row stride of " + w + " is below its width");
  return GPTQ_OK;
}
gptq_status check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens must be in [0, 2^20]");
  return GPTQ_OK;
}
gptq_status check_saved(const gptq_ff *f, int64_t tokens, const void *saved, size_t bytes) {
  if (!aligned_to(saved, 256))
    return fail(GPTQ_ERR_INVALID_ARG, "saved must be 256-byte aligned");
  const size_t need = gptq_ff_saved_bytes(f, tokens);
  if (bytes < need)
    return fail(GPTQ_ERR_INVALID_ARG, "saved too small: need " + std::to_string(need) +
                                          " bytes, got " + std::to_string(bytes));
  return GPTQ_OK;
}

// ------------------------------------------------------------- launch rules
// What a product runs on: tiles of 32 fa x 32 fb (of 16 fa rows of v for gate and
// up), k in `splits` parts; the shape of the least modelled time.  A compute unit runs n
// workgroups of a shape one after the other, each `stage` us per 64 k and `fixed` us
// for its first loads and its epilogue.  A round that leaves units idle clocks higher and
// shares its loads among fewer: half a round's stage takes 84 % of a full one's.  Two 128 x
// 128 workgroups share a unit and cover each other's epilogues; where there is at most one
// per unit it takes four buffers (4096 x 4096 k 8192: 76 us against 118).  A split adds the
// join.  The figures are fits to measured products (us; rows x columns x k):
//   256 x 256  4096 x 4096 x 11008 242, 11008 x 4096 x 4096 278 plain, 382 with dg and du
//   128 x 256  302, 359, 472      128 x 128  376, 367, 430      128 x 64  525, 604, 688
//   1000 x 777 x 2728: 61, 41, 35 (28 with four buffers), 22
struct Plan {
  int fa, fb, splits;
  double us;
};
Plan plan_for(int64_t rows, int64_t cols, int64_t k, int segments, int problems, Mode m) {
  struct Shape {
    int fa, fb, most;
    double stage, fixed, dgate;
  };
  constexpr Shape kShapes[] = {{8, 8, 1, 1.4, 9, 30}, {4, 8, 1, 0.84, 5, 18},
                               {4, 4, 8, 0.485, 2.5, 7.5}, {4, 2, 8, 0.32, 4, 5}};
  const int cus = device_cu_count();
  const int64_t stages = segments * std::max<int64_t>(cdiv(k, kStep), 1);
  Plan best{4, 2, 1, 1e30};
  for (const Shape &sh : kShapes) {
    const int64_t tiles =
        cdiv(rows, (m == kGated ? 16 : 32) * sh.fa) * cdiv(cols, 32 * sh.fb) * problems;
    const double fixed = sh.fixed + (m == kDGate ? sh.dgate : 0);
    for (int splits = 1; splits <= sh.most && splits * 4 <= std::max<int64_t>(stages, 4); ++splits) {
      const int64_t units = tiles * splits;
      const double each = double(cdiv(stages, splits)) * sh.stage + fixed;
      // two workgroups per unit: few of them end together, many smooth out
      const int64_t pairs = cdiv(units, 2 * cus);
      const bool shared = sh.fa == 4 && sh.fb == 4 && units > cus;
      const double part = double(units % cus) / cus, idle = part > 0 ? 0.32 * (1 - part) : 0;
      double us = !shared     ? double(cdiv(units, cus)) * each + 2 -
                                idle * (each - fixed) * (sh.fb == 8)
                  : pairs < 5 ? 2 * double(pairs) * each + 2
                              : double(units) / cus * each + 6;
      if (splits > 1) us += 4.5 + double(units) * (32 * sh.fa * 32 * sh.fb) * 8e-6 / 4;
      if (us < best.us) best = {sh.fa, sh.fb, splits, us};
    }
  }
  return best;
}
// A product on 256 x 256 tiles whose last round would leave compute units idle may end
// in a part of its own plan: rows from r0 on, or columns from c0 on.  Its launch waits for
// the last of the whole rounds' tiles, about 8 us in all (gate and up of 4096 tokens x 4096 x
// 11008: 505 us + 58 against 583 in one).
struct Cut {
  int64_t r0, c0;          // 0: none
  Plan first, rest;
};
Cut cut_for(int64_t rows, int64_t cols, int64_t k, int segments, int problems, Mode m) {
  Cut cut{0, 0, plan_for(rows, cols, k, segments, problems, m), {}};
  if (cut.first.fa != 8) return cut;
  const int64_t th = m == kGated ? 128 : 256;
  const int64_t rt = cdiv(rows, th), ct = cdiv(cols, 256), cus = device_cu_count();
  const int64_t rounds = rt * ct * problems / cus;
  if (rounds == 0 || rt * ct * problems % cus == 0) return cut;
  double least = cut.first.us;
  const Plan whole = cut.first;
  for (int along = 0; along < 2; ++along) {
    // the most tiles along one side that fill no more than the whole rounds
    const int64_t other = (along ? rt : ct) * problems, n = rounds * cus / other;
    if (n == 0) continue;
    const int64_t at = n * (along ? 256 : th);
    const Plan first = plan_for(along ? rows : at, along ? at : cols, k, segments, problems, m);
    const Plan rest = plan_for(along ? rows : rows - at, along ? cols - at : cols, k, segments,
                               problems, m);
    if (first.fa == 8 && first.us + rest.us + 8 < least) {
      least = first.us + rest.us + 8;
      cut = {along ? 0 : at, along ? at : 0, whole, rest};
      cut.first = first;
    }
  }
  return cut;
}

template <typename T, bool AM, bool BM, int FA, int FB, Mode M>
gptq_status launch_tiles(const std::string &name, const Args &a, hipStream_t s) {
  auto kern = ff_tile_kernel<T, AM, BM, FA, FB, M>;
  const size_t lds = size_t(2) * 32 * (FA + FB) * 128;
  GPTQ_TRY(allow_dynamic_lds(reinterpret_cast<const void *>(kern), lds));
  const int rt = int(cdiv(a.rows, M == kGated ? 16 * FA : 32 * FA));
  const int ct = int(cdiv(a.cols, 32 * FB));
  return launch(name.c_str(), kern, dim3(uint32_t(rt) * uint32_t(ct) * a.problems), dim3(256), lds,
                s, a, ct, rt);
}
template <typename T, bool AM, bool BM, int FB, int SUB, int NBUF, Mode M>
gptq_status launch_ring(const std::string &name, const Args &a, hipStream_t s) {
  auto kern = ff_ring_kernel<T, AM, BM, FB, SUB, NBUF, M>;
  constexpr size_t lds = ring_lds(FB, SUB, NBUF);
  static_assert(lds >= 8 * 64 * 4 * 16 * ((FB + 1) / 2), "the epilogue's");
  GPTQ_TRY(allow_dynamic_lds(reinterpret_cast<const void *>(kern), lds));
  const int rt = int(cdiv(a.rows, M == kGated ? 64 : 128)), ct = int(cdiv(a.cols, 64 * FB));
  const uint32_t tiles = uint32_t(rt) * uint32_t(ct) * a.problems;
  GPTQ_TRY(launch(name.c_str(), kern, dim3(tiles * a.splits), dim3(512), lds, s, a, ct, rt));
  if (a.splits == 1) return GPTQ_OK;
  return launch("ff_join", ff_join_kernel<T, FB, M>, dim3(tiles * (M == kGated ? 4 : 8)), dim3(256),
                0, s, a, ct, rt);
}
template <typename T, bool AM, bool BM, Mode M>
gptq_status product_typed(const std::string &name, const Plan &p, const Args &a, hipStream_t s) {
  if (p.fa == 8) return launch_tiles<T, AM, BM, 8, 8, M>(name + "_256x256", a, s);
  if (p.fb == 8) return launch_tiles<T, AM, BM, 4, 8, M>(name + "_128x256", a, s);
  if (p.fb == 2) return launch_ring<T, AM, BM, 1, 2, 3, M>(name + "_128x64", a, s);
  const int64_t units = cdiv(a.rows, M == kGated ? 64 : 128) * cdiv(a.cols, 128) * a.problems *
                        a.splits;
  return units <= device_cu_count() ? launch_ring<T, AM, BM, 2, 1, 4, M>(name + "_128x128_deep", a, s)
                                    : launch_ring<T, AM, BM, 2, 1, 2, M>(name + "_128x128", a, s);
}
// Scratch for the parts of a split product; one after the other use the same.
struct Parts {
  size_t bytes = 0;
  f32x4_t *at = nullptr;
};
template <bool AM, bool BM, Mode M>
gptq_status product_on(const char *name, int32_t dtype, Args a, const Plan &p, Parts &parts,
                       bool run, hipStream_t s) {
  a.splits = p.splits;
  if (!run) {
    if (p.splits > 1)
      parts.bytes = std::max(parts.bytes,
                             size_t(cdiv(a.rows, (M == kGated ? 16 : 32) * p.fa)) *
                                 cdiv(a.cols, 32 * p.fb) * a.problems * p.splits *
                                 (32 * p.fa * 32 * p.fb * sizeof(float)));
    return GPTQ_OK;
  }
  a.part = parts.at;
  return dtype == GPTQ_DT_BF16 ? product_typed<bf16_t, AM, BM, M>(name, p, a, s)
                               : product_typed<f16_t, AM, BM, M>(name, p, a, s);
}
template <bool AM, bool BM, Mode M>
gptq_status product(const char *name, int32_t dtype, const Args &a, Parts &parts, bool run,
                    hipStream_t s) {
  const Cut cut = cut_for(a.rows, a.cols, a.k, a.segments, a.problems, M);
  if (cut.r0 == 0 && cut.c0 == 0)
    return product_on<AM, BM, M>(name, dtype, a, cut.first, parts, run, s);
  Args first = a, rest = a;
  if (cut.r0) {
    first.rows = first.store_rows = int(cut.r0);
    rest.rows -= int(cut.r0);
    rest.store_rows -= int(cut.r0);
  } else {
    first.cols = int(cut.c0);
    rest.cols -= int(cut.c0);
  }
  for (int i = 0; run && i < 2; ++i) {
    rest.a[i] += cut.r0 * (AM ? 1 : a.ld_a[i]);
    rest.b[i] += cut.c0 * (BM ? 1 : a.ld_b[0]);
  }
  for (uint16_t *&o : rest.out)
    if (o) o += cut.r0 + cut.c0 * a.ld_out;
  for (const uint16_t **o : {&rest.g, &rest.u})
    if (*o) *o += cut.r0 + cut.c0 * a.ld_out;
  GPTQ_TRY((product_on<AM, BM, M>(name, dtype, first, cut.first, parts, run, s)));
  return product_on<AM, BM, M>(name, dtype, rest, cut.rest, parts, run, s);
}

template <bool GATED>
gptq_status rows_product(const char *name, int32_t dtype, const RowsArgs &a, hipStream_t s) {
  return launch(name, dtype == GPTQ_DT_BF16 ? ff_rows_kernel<bf16_t, GATED>
                                            : ff_rows_kernel<f16_t, GATED>,
                dim3(uint32_t(cdiv(a.rows, 16))), dim3(64 * kRowsWaves), 0, s, a);
}

// g, u and v of a pass, rows of inner rounded up to 8.
struct Saved {
  uint16_t *v, *g, *u;
  int64_t ld;
  size_t bytes;
};
Saved saved_map(const gptq_ff *f, int64_t tokens, const void *mem, bool all) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(mem);
  const size_t n = padded_bytes(tokens, f->inner);
  return {reinterpret_cast<uint16_t *>(p), all ? reinterpret_cast<uint16_t *>(p + n) : nullptr,
          all ? reinterpret_cast<uint16_t *>(p + 2 * n) : nullptr, up8(f->inner),
          all ? 3 * n : n};
}

Args empty_args() {
  Args a{};
  a.segments = a.problems = a.splits = 1;
  return a;
}

// Walks a forward pass: with `run` false only its scratch is added up.
gptq_status forward(const gptq_ff *f, const void *x, int64_t ld_x, int64_t tokens, void *y,
                    int64_t ld_y, void *saved, Arena &ws, bool run, hipStream_t s) {
  const int64_t d = f->d, n = f->inner;
  const Saved sv = saved_map(f, tokens, saved, saved != nullptr);
  if (tokens <= kRowsTokens) {
    uint16_t *v = saved ? sv.v : ws.take(padded_bytes(tokens, n));
    if (!run) return GPTQ_OK;
    RowsArgs a{};
    a.w[0] = static_cast<const uint16_t *>(f->gate);
    a.w[1] = static_cast<const uint16_t *>(f->up);
    a.ld_w[0] = f->ld_gate;
    a.ld_w[1] = f->ld_up;
    a.x = static_cast<const uint16_t *>(x);
    a.ld_x = ld_x;
    a.rows = int(n);
    a.tokens = int(tokens);
    a.k = int(d);
    a.y = v;
    a.g = sv.g;
    a.u = sv.u;
    a.ld_y = sv.ld;
    GPTQ_TRY(rows_product<true>("ff_rows_gate_up", f->dtype, a, s));
    a = RowsArgs{};
    a.w[0] = static_cast<const uint16_t *>(f->down);
    a.ld_w[0] = f->ld_down;
    a.x = v;
    a.ld_x = sv.ld;
    a.rows = int(d);
    a.tokens = int(tokens);
    a.k = int(n);
    a.y = static_cast<uint16_t *>(y);
    a.ld_y = ld_y;
    return rows_product<false>("ff_rows_down", f->dtype, a, s);
  }
  Padder pad{ws};
  // x is copied where it has to be; its room is always there, since the
  // scratch's size is asked before x is known
  const bool x_direct = run && direct(x, tokens, d, ld_x);
  if (x_direct) ws.take(padded_bytes(tokens, d));
  const Operand xo = pad(x, tokens, d, ld_x, !x_direct);
  const Operand go = pad(f->gate, n, d, f->ld_gate, !direct(f->gate, n, d, f->ld_gate));
  const Operand uo = pad(f->up, n, d, f->ld_up, !direct(f->up, n, d, f->ld_up));
  const Operand wo = pad(f->down, d, n, f->ld_down, !direct(f->down, d, n, f->ld_down));
  if (run) GPTQ_TRY(pad.launch_all(s));
  uint16_t *v = saved ? sv.v : ws.take(padded_bytes(tokens, n));
  Parts parts{0, reinterpret_cast<f32x4_t *>(ws.base + ws.at)};     // the rest of the scratch
  Args a = empty_args();
  a.a[0] = go.p;
  a.a[1] = uo.p;
  a.ld_a[0] = go.ld;
  a.ld_a[1] = uo.ld;
  a.b[0] = a.b[1] = xo.p;
  a.ld_b[0] = a.ld_b[1] = xo.ld;
  a.rows = int(n);
  a.cols = int(tokens);
  a.k = int(d);
  a.out[0] = v;
  a.out[1] = sv.g;
  a.out[2] = sv.u;
  a.ld_out = sv.ld;
  a.store_rows = int(sv.ld);
  GPTQ_TRY((product<false, false, kGated>("ff_gate_up", f->dtype, a, parts, run, s)));
  a = empty_args();
  a.a[0] = a.a[1] = wo.p;
  a.ld_a[0] = a.ld_a[1] = wo.ld;
  a.b[0] = a.b[1] = v;
  a.ld_b[0] = a.ld_b[1] = sv.ld;
  a.rows = a.store_rows = int(d);
  a.cols = int(tokens);
  a.k = int(n);
  a.out[0] = static_cast<uint16_t *>(y);
  a.ld_out = ld_y;
  GPTQ_TRY((product<false, false, kPlain>("ff_down", f->dtype, a, parts, run, s)));
  if (!run) ws.at += align256(parts.bytes);
  return GPTQ_OK;
}

gptq_status backward(const gptq_ff *f, const void *x, int64_t ld_x, int64_t tokens,
                     const void *saved, const void *dy, int64_t ld_dy, void *dx, int64_t ld_dx,
                     void *dgate, int64_t ld_dgate, void *dup, int64_t ld_dup, void *ddown,
                     int64_t ld_ddown, Arena &ws, bool run, hipStream_t s) {
  Padder pad{ws};
  const int64_t d = f->d, n = f->inner;
  const bool x_direct = run && direct(x, tokens, d, ld_x);
  const bool dy_direct = run && direct(dy, tokens, d, ld_dy);
  if (x_direct) ws.take(padded_bytes(tokens, d));
  const Operand xo = pad(x, tokens, d, ld_x, !x_direct);
  if (dy_direct) ws.take(padded_bytes(tokens, d));
  const Operand dyo = pad(dy, tokens, d, ld_dy, !dy_direct);
  const Operand wo = pad(f->down, d, n, f->ld_down, !direct(f->down, d, n, f->ld_down));
  // one stride for both weights: one offset serves both segments
  const bool copies = f->ld_gate != f->ld_up || !direct(f->gate, n, d, f->ld_gate) ||
                      !direct(f->up, n, d, f->ld_up);
  Operand go{}, uo{};
  if (dx || !run) {
    go = pad(f->gate, n, d, f->ld_gate, copies);
    uo = pad(f->up, n, d, f->ld_up, copies);
  }
  if (run) GPTQ_TRY(pad.launch_all(s));
  const Saved sv = saved_map(f, tokens, saved, true);
  uint16_t *dg = ws.take(padded_bytes(tokens, n)), *du = ws.take(padded_bytes(tokens, n));
  Parts parts{0, reinterpret_cast<f32x4_t *>(ws.base + ws.at)};     // the rest of the scratch
  Args a;
  if (dx || dgate || dup || !run) {
    a = empty_args();                       // dv = dy W_down -> dg, du
    a.a[0] = a.a[1] = wo.p;
    a.ld_a[0] = a.ld_a[1] = wo.ld;
    a.b[0] = a.b[1] = dyo.p;
    a.ld_b[0] = a.ld_b[1] = dyo.ld;
    a.rows = int(n);
    a.cols = int(tokens);
    a.k = int(d);
    a.g = sv.g;
    a.u = sv.u;
    a.out[0] = dg;
    a.out[1] = du;
    a.ld_out = sv.ld;
    a.store_rows = int(sv.ld);
    GPTQ_TRY((product<true, false, kDGate>("ff_dgate_up", f->dtype, a, parts, run, s)));
  }
  if (dx || !run) {
    a = empty_args();
    a.segments = 2;
    a.a[0] = go.p;
    a.a[1] = uo.p;
    a.ld_a[0] = a.ld_a[1] = go.ld;
    a.b[0] = dg;
    a.b[1] = du;
    a.ld_b[0] = a.ld_b[1] = sv.ld;
    a.rows = a.store_rows = int(d);
    a.cols = int(tokens);
    a.k = int(n);
    a.out[0] = static_cast<uint16_t *>(dx);
    a.ld_out = ld_dx;
    GPTQ_TRY((product<true, false, kPlain>("ff_dx", f->dtype, a, parts, run, s)));
  }
  a = empty_args();
  a.a[0] = a.a[1] = xo.p;
  a.ld_a[0] = a.ld_a[1] = xo.ld;
  a.ld_b[0] = a.ld_b[1] = sv.ld;
  a.rows = a.store_rows = int(d);
  a.cols = int(n);
  a.k = int(tokens);
  if (!run || (dgate && dup && ld_dgate == ld_dup)) {
    a.problems = 2;
    a.b[0] = dg;
    a.b[1] = du;
    a.out[0] = static_cast<uint16_t *>(dgate);
    a.out[1] = static_cast<uint16_t *>(dup);
    a.ld_out = ld_dgate;
    GPTQ_TRY((product<true, true, kPlain>("ff_dweights", f->dtype, a, parts, run, s)));
  }
  if (!run || !(dgate && dup && ld_dgate == ld_dup)) {
    a.problems = 1;
    for (auto [o, ld, b] : {std::tuple{dgate, ld_dgate, dg}, std::tuple{dup, ld_dup, du}}) {
      if (run && !o) continue;
      a.b[0] = a.b[1] = b;
      a.out[0] = static_cast<uint16_t *>(o);
      a.ld_out = ld;
      GPTQ_TRY((product<true, true, kPlain>("ff_dweight", f->dtype, a, parts, run, s)));
    }
  }
  if (ddown || !run) {
    a = empty_args();
    a.a[0] = a.a[1] = sv.v;
    a.ld_a[0] = a.ld_a[1] = sv.ld;
    a.b[0] = a.b[1] = dyo.p;
    a.ld_b[0] = a.ld_b[1] = dyo.ld;
    a.rows = a.store_rows = int(n);
    a.cols = int(d);
    a.k = int(tokens);
    a.out[0] = static_cast<uint16_t *>(ddown);
    a.ld_out = ld_ddown;
    GPTQ_TRY((product<true, true, kPlain>("ff_ddown", f->dtype, a, parts, run, s)));
  }
  if (!run) ws.at += align256(parts.bytes);
  return GPTQ_OK;
}

gptq_status zero(void *p, int64_t ld, int64_t rows, int64_t cols, hipStream_t s) {
  if (!p) return GPTQ_OK;
  return launch("ff_zero", ff_zero_kernel,
                dim3(uint32_t(std::min<int64_t>(cdiv(rows * cols, 256), 1 << 16))), dim3(256), 0, s,
                static_cast<uint16_t *>(p), ld, rows, int(cols));
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

size_t gptq_ff_saved_bytes(const gptq_ff *ff, int64_t tokens) {
  if (!ff || ff->inner < 1 || ff->inner > kMaxSide || tokens < 1 || tokens > kMaxTokens) return 0;
  return 3 * padded_bytes(tokens, ff->inner);
}

size_t gptq_ff_forward_ws_bytes(const gptq_ff *ff, int64_t tokens) {
  return guarded_bytes([&]() -> size_t {
    if (check_ff(ff) != GPTQ_OK || tokens < 1 || tokens > kMaxTokens) return 0;
    Arena ws{0};
    (void)forward(ff, nullptr, 0, tokens, nullptr, 0, nullptr, ws, false, nullptr);
    return ws.at;
  });
}

size_t gptq_ff_backward_ws_bytes(const gptq_ff *ff, int64_t tokens) {
  return guarded_bytes([&]() -> size_t {
    if (check_ff(ff) != GPTQ_OK || tokens < 1 || tokens > kMaxTokens) return 0;
    Arena ws{0};
    (void)backward(ff, nullptr, 0, tokens, nullptr, nullptr, 0, nullptr, 0, nullptr, 0, nullptr, 0,
                   nullptr, 0, ws, false, nullptr);
    return ws.at;
  });
}

gptq_status gptq_ff_forward(const gptq_ff *ff, const void *x, int64_t ld_x, int64_t tokens, void *y,
                            int64_t ld_y, void *saved, size_t saved_bytes, void *ws,
                            size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_ff(ff));
    GPTQ_TRY(check_tokens(tokens));
    if (tokens == 0) return GPTQ_OK;
    GPTQ_TRY(check_matrix(x, ld_x, ff->d, "x"));
    GPTQ_TRY(check_matrix(y, ld_y, ff->d, "y"));
    const int64_t d = ff->d, n = ff->inner;
    if (overlap(x, tokens, d, ld_x, y, tokens, d, ld_y) ||
        overlap(ff->gate, n, d, ff->ld_gate, y, tokens, d, ld_y) ||
        overlap(ff->up, n, d, ff->ld_up, y, tokens, d, ld_y) ||
        overlap(ff->down, d, n, ff->ld_down, y, tokens, d, ld_y))
      return fail(GPTQ_ERR_INVALID_ARG, "y must not overlap x or a weight");
    if (saved) GPTQ_TRY(check_saved(ff, tokens, saved, saved_bytes));
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_ff_forward_ws_bytes(ff, tokens)));
    Arena at{reinterpret_cast<uintptr_t>(ws)};
    return forward(ff, x, ld_x, tokens, y, ld_y, saved, at, true, static_cast<hipStream_t>(stream));
  });
}

gptq_status gptq_ff_backward(const gptq_ff *ff, const void *x, int64_t ld_x, int64_t tokens,
                             const void *saved, size_t saved_bytes, const void *dy, int64_t ld_dy,
                             void *dx, int64_t ld_dx, void *dgate, int64_t ld_dgate, void *dup,
                             int64_t ld_dup, void *ddown, int64_t ld_ddown, void *ws,
                             size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    GPTQ_TRY(check_ff(ff));
    GPTQ_TRY(check_tokens(tokens));
    const int64_t d = ff->d, n = ff->inner;
    if (dgate) GPTQ_TRY(check_matrix(dgate, ld_dgate, d, "dgate"));
    if (dup) GPTQ_TRY(check_matrix(dup, ld_dup, d, "dup"));
    if (ddown) GPTQ_TRY(check_matrix(ddown, ld_ddown, n, "ddown"));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (tokens == 0) {
      GPTQ_TRY(zero(dgate, ld_dgate, n, d, s));
      GPTQ_TRY(zero(dup, ld_dup, n, d, s));
      return zero(ddown, ld_ddown, d, n, s);
    }
    GPTQ_TRY(check_matrix(x, ld_x, d, "x"));
    GPTQ_TRY(check_matrix(dy, ld_dy, d, "dy"));
    if (dx) GPTQ_TRY(check_matrix(dx, ld_dx, d, "dx"));
    if (!saved) return fail(GPTQ_ERR_INVALID_ARG, "saved must not be NULL");
    GPTQ_TRY(check_saved(ff, tokens, saved, saved_bytes));
    struct M {
      const void *p;
      int64_t rows, cols, ld;
    };
    const M outs[] = {{dx, tokens, d, ld_dx}, {dgate, n, d, ld_dgate}, {dup, n, d, ld_dup},
                      {ddown, d, n, ld_ddown}};
    const int64_t half = int64_t(gptq_ff_saved_bytes(ff, tokens) / 2);
    const M ins[] = {{x, tokens, d, ld_x}, {dy, tokens, d, ld_dy}, {ff->gate, n, d, ff->ld_gate},
                     {ff->up, n, d, ff->ld_up}, {ff->down, d, n, ff->ld_down},
                     {saved, 1, half, half}};
    for (int i = 0; i < 4; ++i) {
      for (const M &m : ins)
        if (overlap(outs[i].p, outs[i].rows, outs[i].cols, outs[i].ld, m.p, m.rows, m.cols, m.ld))
          return fail(GPTQ_ERR_INVALID_ARG, "gradients must not overlap the inputs");
      for (int j = 0; j < i; ++j)
        if (overlap(outs[i].p, outs[i].rows, outs[i].cols, outs[i].ld, outs[j].p, outs[j].rows,
                    outs[j].cols, outs[j].ld))
          return fail(GPTQ_ERR_INVALID_ARG, "gradients must not overlap each other");
    }
    GPTQ_TRY(check_scratch(ws, ws_bytes, gptq_ff_backward_ws_bytes(ff, tokens)));
    Arena at{reinterpret_cast<uintptr_t>(ws)};
    return backward(ff, x, ld_x, tokens, saved, dy, ld_dy, dx, ld_dx, dgate, ld_dgate, dup, ld_dup,
                    ddown, ld_ddown, at, true, s);
  });
}

}  // extern "C"
