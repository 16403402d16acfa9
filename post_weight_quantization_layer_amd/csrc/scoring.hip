// Log probabilities of given tokens, entropy and top alternatives from rows
// of logits, in one pass over the logits.
//
// With c = scale log2 e, every lane keeps a running maximum m of its logits,
// s = sum 2^(c l - M) and t = sum (c l - M) 2^(c l - M), M being the float
// nearest c m (c m itself from 2^22 up); lanes, waves and, when a row is split
// over workgroups, parts are joined by rescaling to the common maximum.  Then
// ln p = ln 2 (c l - M) - ln s and the entropy is ln s - ln 2 t / s.  c l - M is
// one fused operation, exact up to its last rounding because M, not c m, is the
// reference.
//
// Alternatives: the pass keeps each lane's maximum over groups of tiles, in
// LDS.  After it, the k-th largest of the 256 lanes' own maxima is a threshold
// that k logits reach and few others, and only the tiles whose group reaches it
// are read again (from cache, about k of them), into a short list per wave;
// where a list grows past a few k it is cut to its k best, whose smallest is
// the new threshold.  Candidates listed during the pass instead, each wave
// against its own rising threshold, cost as much as the pass itself.  All
// selections go by (value, lower index), so the result does not depend on the
// order of the work.
//
// 4096 x 128000 bf16: 190 us without alternatives, 5.5 TB/s, bound by memory;
// 222 us with 20, 266 us with 64.  1 x 32000: 6.7 us and 2.8 us for the join, a
// chain of dependent steps.
#include <algorithm>

#include "rows.h"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunkElems = 8 * kThreads;   // elements a workgroup takes per chunk
// Chunks per tile, whose loads are in flight together (with four, a wave's
// registers leave room for fewer waves: 4096 x 128000 399 us against 308).
constexpr int kUnroll = 2;
constexpr int kTile = kUnroll * kChunkElems;
constexpr int kMaxTop = 64;
constexpr int kGroups = 32;                 // groups of tiles with a maximum of their own
typedef uint16_t __attribute__((may_alias)) group_max_t;   // shares LDS with the lists' keys
constexpr int kUncut = 64;                  // shorter lists are not cut before the last step
// A wave's list is cut to k once it is longer than 2 k + 32, before the next
// entry is added; so it takes a chunk (512) on top of that.
constexpr int kListSlack = 32;
constexpr int kListCap = 512 + 2 * kMaxTop + kListSlack + 16;   // 16: zeros after the last

struct ScoreArgs {
  const void *logits;
  const int64_t *ids;
  int64_t ld;
  int vocab, k, splits, seg;    // seg: elements per split (a multiple of 16)
  float scale;
  float *logprob;
  int *rank;
  float *entropy;
  int *top_ids;
  float *top_logprobs;
  float *part;                  // splits > 1: per (row, split) kPartWords words
  uint64_t *part_keys;          //             and k keys
};
constexpr int kPartWords = 8;   // m, s, t, rank count, the given token's logit

constexpr float kLog2e = 1.4426950408889634f;

// Floats as integers of the same order; -0 and +0 are equal.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ (uint32_t(int32_t(~o) >> 31) | 0x80000000u));
}
// Largest float below v (v > -inf): "x > below(v)" is "x >= v".
__device__ __forceinline__ float below(float v) {
  if (v == 0.f) return __uint_as_float(0x80000001u);
  return from_ordered(ordered(v) - 1);
}
// Sorts by value, then by lower index.
__device__ __forceinline__ uint64_t make_key(float v, int index) {
  return (uint64_t(ordered(v)) << 32) | uint32_t(~index);
}
__device__ __forceinline__ float key_value(uint64_t key) { return from_ordered(uint32_t(key >> 32)); }
__device__ __forceinline__ int key_index(uint64_t key) { return int(~uint32_t(key)); }

// c l - M for a row maximum m.  M is off c m by up to half a unit in its last
// place, and the sums are off by 2 to that power until they are joined: nothing
// below kLarge, where it is 1/8 at most, but past float32 for a lane that has seen
// only masks of -1e10, where it is hundreds.  From kLarge up the sums are relative
// to c m itself: c (l - m), halved against overflow.
constexpr float kLarge = 4194304.f;
// M: the product rounded, never fused into what uses it.
__device__ __forceinline__ float reference(float m, float c) {
  float M = m * c;
  asm("" : "+v"(M));
  return M;
}
__device__ __forceinline__ float exponent(float l, float m, float c) {
  const float M = reference(m, c);
  return fabsf(M) < kLarge ? __builtin_fmaf(l, c, -M) : (0.5f * l - 0.5f * m) * c * 2.f;
}

// Running softmax statistics of part of a row; empty: s = 0.
struct Stat {
  float m, s, t;
};
// What takes sums at the maximum `from` to the maximum m: the difference of their
// references, each M or c m by its own size.  (With exponent()'s the sums would keep a
// part of the rounding of c m each time; this is 0 where they are equal.)
__device__ __forceinline__ float shift(float from, float m, float c) {
  const float F = reference(from, c), M = reference(m, c);
  if (fabsf(M) < kLarge) return fabsf(F) < kLarge ? F - M : __builtin_fmaf(from, c, -M);
  return fabsf(F) < kLarge ? -__builtin_fmaf(m, c, -F) : exponent(from, m, c);
}
// The part at its own maximum, rescaled to the maximum m.
__device__ __forceinline__ Stat rescaled(const Stat &a, float m, float c) {
  const float d = shift(a.m, m, c);
  const float f = exp2f(d);
  // a part scaled to nothing adds nothing (its t would be 0 * infinity); a NaN
  // in s stays
  return Stat{m, f * a.s, f > 0.f ? f * (a.t + d * a.s) : 0.f};
}
// Joins the lanes' statistics (uniform result).
__device__ __forceinline__ Stat join_wave(const Stat &st, float c) {
  const float m = wave_all<MaxF>(st.m);
  const Stat r = rescaled(st, m, c);
  return Stat{m, wave_all<SumF>(r.s), wave_all<SumF>(r.t)};
}

// Highest bit that differs among values with this or and this and (-1: none),
// and the bits above it, which all of them share.
__device__ __forceinline__ int first_differing(uint32_t any, uint32_t all) {
  return any == all ? -1 : 31 - __builtin_clz(any ^ all);
}
__device__ __forceinline__ uint32_t common_prefix(uint32_t all, int first) {
  return first < 0 ? all : all & ~((2u << first) - 1);
}

// The largest value that k of a wave's entries v (kListLane to a lane) reach, or,
// where several entries are equal, the value from which more than k do; `reach`
// is the number that reach it (at first: all entries that count).  Searched bit
// by bit, counting with ballots, over the bits in which the entries differ
// (`any`, `all`: their or and and); entries that do not count are 0.
constexpr int kListLane = (kListCap + 63) / 64;   // 11
__device__ __forceinline__ uint32_t kth_of(const uint32_t (&v)[kListLane], int k, uint32_t any,
                                           uint32_t all, int &reach) {
  const int first = first_differing(any, all);
  uint32_t value = common_prefix(all, first);
  for (int bit = first; bit >= 0 && reach > k; --bit) {
    const uint32_t probe = value | (1u << bit);
    if (!((any ^ all) >> bit & 1)) {
      value |= all & (1u << bit);
      continue;
    }
    int c = 0;
#pragma unroll
    for (int i = 0; i < kListLane; ++i) c += __popcll(__ballot(v[i] >= probe));
    if (c >= k) value = probe, reach = c;
  }
  return value;
}

// Cuts the list of n keys to its k best, exactly (k < n <= kListCap), and
// returns the smallest kept value: the k-th largest value and, if more than k
// entries reach it, the lowest of the indices to keep among equals.  One wave;
// the list is in its LDS, read again at each step so that only one word per
// entry stays in registers (80 per lane in all, six workgroups per compute unit;
// with 95 and five, 6276 x 16586 with 64 alternatives took 105 us against 93).
// No branch per 64 entries in the search, and none of the bits that all entries
// share: 300 x 500 with 64 alternatives 19 us, 36 with both.
__device__ __forceinline__ float cut_list(uint64_t *list, int n, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t v[kListLane];                 // an entry's value; then its index
  uint32_t any = 0, all = ~0u;
#pragma unroll
  for (int i = 0; i < kListLane; ++i) {
    const bool entry = lane + 64 * i < n;
    v[i] = entry ? uint32_t(list[lane + 64 * i] >> 32) : 0;   // above 0 in every entry
    any |= v[i];
    if (entry) all &= v[i];
  }
  int reach = n;
  const uint32_t value = kth_of(v, k, wave_all<OrU>(any), wave_all<AndU>(all), reach);
  // Entries above the value count always, those equal to it by index.
  any = 0, all = ~0u;
#pragma unroll
  for (int i = 0; i < kListLane; ++i) {
    const uint32_t at = v[i];
    v[i] = at > value ? ~0u : at == value ? uint32_t(list[lane + 64 * i]) : 0u;
    if (at == value) any |= v[i], all &= v[i];
  }
  uint32_t from = 1;
  if (reach > k) from = kth_of(v, k, wave_all<OrU>(any), wave_all<AndU>(all), reach);
  int at = 0;
  uint32_t least = ~0u;
#pragma unroll
  for (int i = 0; i < kListLane; ++i) {
    const bool keep = v[i] >= from;
    const uint64_t mask = __ballot(keep);
    if (keep) {                          // to a place below the entries not read yet
      const uint64_t e = list[lane + 64 * i];
      list[at + __popcll(mask & ((uint64_t(1) << lane) - 1))] = e;
      least = min(least, uint32_t(e >> 32));
    }
    at += __popcll(mask);
  }
  return from_ordered(wave_all<MinU>(least));
}

// How many of kBatch keys in LDS are above `key`; the reads are in flight
// together.
constexpr int kBatch = 16;
__device__ __forceinline__ int count_above(const uint64_t *keys, uint64_t key) {
  uint64_t e[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) e[i] = keys[i];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) n += e[i] > key;
  return n;
}

// A value that at least k elements of the row's part reach: the k-th largest of
// the 256 lanes' maxima (four to a lane here) or a little below; -inf if fewer
// than k are above that.
__device__ __forceinline__ float reached_by(const float most[kWaves], int k) {
  uint32_t o[kWaves];
#pragma unroll
  for (int c = 0; c < kWaves; ++c) o[c] = ordered(most[c]);
  uint32_t any = o[0], all = o[0];
#pragma unroll
  for (int c = 1; c < kWaves; ++c) any |= o[c], all &= o[c];
  any = wave_all<OrU>(any);
  all = wave_all<AndU>(all);
  const int first = first_differing(any, all);
  uint32_t v = common_prefix(all, first);
  for (int bit = first; bit >= 0; --bit) {
    const uint32_t probe = v | (1u << bit);
    int n = 0;
#pragma unroll
    for (int c = 0; c < kWaves; ++c) n += __popcll(__ballot(o[c] >= probe));
    if (n >= k) v = probe;
    if (n >= k && n <= k + k / 4 + 1) break;
  }
  const float f = from_ordered(v);
  return f > -INFINITY ? f : -INFINITY;    // also for patterns below -inf
}

// The final outputs of a row from its joined statistics.
constexpr float kLn2 = 0.6931471805599453f;
struct RowOut {
  float m, c, log_s, entropy, logprob;
  int rank;
  bool bad, empty;
};
// ln p of an entry of value l (not of an empty row).
__device__ __forceinline__ float log_prob(const ScoreArgs &a, const RowOut &o, float l) {
  const float M = reference(o.m, o.c), z = __builtin_fmaf(l, o.c, -M);
  // c l may overflow where scale (l - m) does not
  const bool plain = fabsf(M) < kLarge && z > -3e38f;
  const float d = plain ? kLn2 * z : (0.5f * l - 0.5f * o.m) * a.scale * 2.f;
  return d - o.log_s;
}
__device__ __forceinline__ RowOut finish_row(const ScoreArgs &a, const Stat &st, int rank_count,
                                             int64_t id, float given) {
  RowOut o;
  const float nan = __uint_as_float(0x7fc00000u);
  o.bad = !(st.s >= 0.f) || st.m == INFINITY;     // NaN or +inf somewhere
  o.empty = st.s == 0.f;
  o.m = st.m;
  o.c = a.scale * kLog2e;
  o.log_s = logf(st.s);
  o.entropy = o.bad ? nan : o.empty ? 0.f : o.log_s - kLn2 * (st.t / st.s);
  o.rank = rank_count;
  o.logprob = o.empty ? -INFINITY : log_prob(a, o, given);
  if (o.bad) o.logprob = nan, o.rank = -1;
  if (id >= a.vocab) o.logprob = nan, o.rank = -1;
  if (id < 0) o.logprob = o.bad ? nan : 0.f, o.rank = -1;
  return o;
}
__device__ __forceinline__ void write_scalars(const ScoreArgs &a, int64_t row, const RowOut &o) {
  if (a.ids) {
    if (a.logprob) a.logprob[row] = o.logprob;
    if (a.rank) a.rank[row] = o.rank;
  }
  if (a.entropy) a.entropy[row] = o.entropy;
}
// Place p of the row's alternatives.
__device__ __forceinline__ void write_top(const ScoreArgs &a, int64_t row, int p, const RowOut &o,
                                          bool present, uint64_t key) {
  const float nan = __uint_as_float(0x7fc00000u);
  a.top_ids[row * a.k + p] = o.bad || !present ? -1 : key_index(key);
  a.top_logprobs[row * a.k + p] =
      o.bad ? nan : present ? log_prob(a, o, key_value(key)) : -INFINITY;
}

__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float load_one(const bf16_t *p) { return widen(*p); }
__device__ __forceinline__ float load_one(const f16_t *p) { return widen(*p); }

// Workgroup (row, split): the row's elements [split seg, split seg + seg).
template <typename T, Ends E, bool TOP>
__global__ void __launch_bounds__(kThreads) score_kernel(ScoreArgs a) {
  __shared__ uint64_t lists[TOP ? kWaves * kListCap : 1];
  __shared__ float lane_max[TOP ? kThreads : 1];
  __shared__ Stat slot[kWaves];
  __shared__ int slot_rank[kWaves], slot_n[kWaves];
  const int64_t row = blockIdx.x / a.splits;
  const int split = blockIdx.x % a.splits;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const T *l = static_cast<const T *>(a.logits) + row * a.ld;
  const int v0 = split * a.seg, v1 = min(v0 + a.seg, a.vocab);
  const float c = a.scale * kLog2e;

  // The first tile is on its way before the given token's logit is asked for.
  Pack8<T> raw[kUnroll];
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) raw[q] = fetch8<E>(l, v0 + q * kChunkElems + 8 * tid, v1);
  const int64_t id = a.ids ? a.ids[row] : -1;
  const bool given = id >= 0 && id < a.vocab;
  const int at = given ? int(id) : 0;
  const float lt = given ? load_one(l + at) : 0.f;
  const float lt_below = lt > -INFINITY ? below(lt) : INFINITY;

  Stat st{-3.402823466e38f, 0.f, 0.f};
  int ahead = 0;                   // the wave's count
  bool masked = false;             // whether -infinity has been seen (by the wave)
  uint64_t *list = lists + (TOP ? wave * kListCap : 0);
  // The group maxima of a wave lie where its list will be.
  static_assert(kGroups * 64 * 2 <= kListCap * 8, "");
  group_max_t *group_max = reinterpret_cast<group_max_t *>(list) + lane;
  int n = 0;                       // list length (wave-uniform)
  float thr = -INFINITY;           // candidates are > thr
  const int limit = 2 * a.k + kListSlack;

  // A tile's values and the maximum of each 8.
  float x[kUnroll][8], cmax[kUnroll];
  auto widen_tile = [&](int tile) {
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      widen8<E>(raw[q], tile + q * kChunkElems + 8 * tid, v1, -INFINITY, x[q]);
      // three at a time
      const float h = fmaxf(fmaxf(x[q][0], x[q][1]), x[q][2]);
      const float i = fmaxf(fmaxf(h, x[q][3]), x[q][4]);
      cmax[q] = fmaxf(fmaxf(fmaxf(i, x[q][5]), x[q][6]), x[q][7]);
    }
  };
  auto fetch_tile = [&](int tile) {
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) raw[q] = fetch8<E>(l, tile + q * kChunkElems + 8 * tid, v1);
  };
  // Adds a tile's entries above the threshold to the list.  Tiles come in
  // index order, so after a cut entries that only equal the threshold lose
  // against the k that reach it.
  auto list_tile = [&](int tile) {
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      if (!__ballot(cmax[q] > thr)) continue;
      if (n > limit) {                 // then a whole chunk fits
        thr = fmaxf(thr, cut_list(list, n, a.k));
        n = a.k;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool take = x[q][j] > thr;
        const uint64_t mask = __ballot(take);
        if (!mask) continue;           // most of the eight: nothing to add
        if (take)
          list[n + __popcll(mask & ((uint64_t(1) << lane) - 1))] =
              make_key(x[q][j], tile + q * kChunkElems + 8 * tid + j);
        n += __popcll(mask);
      }
    }
  };
  const int per_group = ((v1 - v0 + kTile - 1) / kTile + kGroups - 1) / kGroups;   // tiles
  float group = -INFINITY;             // the lane's maximum over the current group
  int in_group = 0, groups = 0;

  for (int tile = v0; tile < v1; tile += kTile) {
    widen_tile(tile);
    if (tile + kTile < v1) fetch_tile(tile + kTile);
    float m = st.m;
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) m = fmaxf(m, cmax[q]);
    const float M = reference(m, c), from = reference(st.m, c);
    // (a lane whose elements were all -infinity so far has s = t = 0)
    if (!__ballot(!(fabsf(M) < kLarge) || (!(fabsf(from) < kLarge) && st.s != 0.f))) {
      const float dm = fmaxf(from - M, -200.f), f = __builtin_amdgcn_exp2f(dm);
      st.t = f * (st.t + dm * st.s);
      st.s *= f;
      if (!masked) {
        const float t = st.t;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = __builtin_fmaf(x[i][j], c, -M);
            const float e = __builtin_amdgcn_exp2f(d);
            st.s += e;
            st.t = __builtin_fmaf(d, e, st.t);
          }
        // -infinity times 0: such a row takes the other form from here on
        masked = __ballot(!(st.t == st.t)) != 0;
        if (masked) {
          st.t = t;
#pragma unroll
          for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float d = __builtin_fmaf(x[i][j], c, -M);
              st.t = __builtin_fmaf(fmaxf(d, -3e38f), __builtin_amdgcn_exp2f(d), st.t);
            }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = __builtin_fmaf(x[i][j], c, -M);
            const float e = __builtin_amdgcn_exp2f(d);
            st.s += e;
            st.t = __builtin_fmaf(fmaxf(d, -3e38f), e, st.t);   // -inf: 0
          }
      }
    } else {
      // Some lane has only -infinity or huge values so far, or had until now.
      const float dm = shift(st.m, m, c), f = exp2f(dm);
      st.t = f > 0.f ? f * (st.t + dm * st.s) : 0.f;
      st.s *= f;
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = exponent(x[i][j], m, c), e = exp2f(d);
          st.s += e;
          st.t += fmaxf(d, -3e38f) * e;
        }
    }
    st.m = m;
    if (given) {
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        // Entries before the given token count from its value up, entries
        // after it from above its value.
        const int e0 = tile + q * kChunkElems + 8 * tid;
        const bool before = e0 + 7 < at;
        const float from = before ? lt_below : lt;
#pragma unroll
        for (int j = 0; j < 8; ++j) ahead += __popcll(__ballot(x[q][j] > from));
        const bool has_given = !before && e0 < at && e0 < v1;
        const bool below_given = before && e0 < v1 && lt == -INFINITY;   // all eight are >= -inf
        if (__ballot(has_given || below_given)) {
          ahead += 8 * __popcll(__ballot(below_given));
#pragma unroll
          for (int j = 0; j < 8; ++j)
            ahead += __popcll(__ballot(has_given && e0 + j < at && x[q][j] == lt));
        }
      }
    }
    if (TOP) {
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) group = fmaxf(group, cmax[q]);
      if (++in_group == per_group || tile + kTile >= v1) {
        // the upper half of the ordered form, rounded up
        const uint32_t o = ordered(group);
        group_max[groups * 64] = uint16_t(min((o >> 16) + ((o & 0xffffu) != 0), 0xffffu));
        ++groups;
        in_group = 0;
        group = -INFINITY;
      }
    }
  }
  if (TOP) {
    // The k-th largest of the 256 lanes' maxima is reached by k elements of the
    // row, and few others: only groups that reach it are read again.
    lane_max[tid] = st.s == 0.f ? -INFINITY : st.m;
    __syncthreads();
    float most[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) most[w] = lane_max[w * 64 + lane];
    const float reached = reached_by(most, a.k);
    if (reached > -INFINITY) thr = below(reached);
    const uint32_t bar = ordered(thr) >> 16;
    uint32_t todo = 0;                 // groups, a bit each
    for (int g = 0; g < groups; ++g)
      if (__ballot(group_max[g * 64] >= bar)) todo |= 1u << g;
    // Tiles of those groups, the next one's loads in flight; a part's only tile
    // is still there.
    const bool single = v1 - v0 <= kTile;
    int left = 0, tile = v1;
    auto advance = [&]() {
      if (left > 0) {
        --left;
        tile += kTile;
      } else if (todo) {
        tile = v0 + __builtin_ctz(todo) * per_group * kTile;
        todo &= todo - 1;
        left = per_group - 1;
      } else {
        tile = v1;
      }
      return tile < v1;                // only the last group can end past v1
    };
    bool more = advance();
    if (more && !single) fetch_tile(tile);
    while (more) {
      const int now = tile;
      if (!single) widen_tile(now);
      more = advance();
      if (more) fetch_tile(tile);
      list_tile(now);
    }
  }

  st = join_wave(st, c);
  if (TOP && n > kUncut) {
    cut_list(list, n, a.k);
    n = a.k;
  }
  if (TOP && lane < kBatch) list[n + lane] = 0;
  if (lane == 0) {
    slot[wave] = st;
    slot_rank[wave] = ahead;
    slot_n[wave] = n;
  }
  __syncthreads();
  float m_all = slot[0].m;
  ahead = slot_rank[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    m_all = fmaxf(m_all, slot[w].m);
    ahead += slot_rank[w];
  }
  st = rescaled(slot[0], m_all, c);
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    const Stat r = rescaled(slot[w], m_all, c);
    st.s += r.s;
    st.t += r.t;
  }
  const bool whole = a.splits == 1;
  RowOut o;
  if (whole) {
    o = finish_row(a, st, ahead, id, lt);
    if (tid == 0) write_scalars(a, row, o);
  } else if (tid == 0) {
    float *p = a.part + int64_t(blockIdx.x) * kPartWords;
    p[0] = st.m;
    p[1] = st.s;
    p[2] = st.t;
    p[3] = __int_as_float(ahead);
    p[4] = lt;
  }
  if (TOP) {
    // The waves' lists (at most 64 keys each, zeros up to a multiple of
    // kBatch): a key's place is the number of larger ones, counted a batch of
    // LDS reads at a time.  Thread w * 64 + i holds entry i of wave w's list.
    const bool mine = lane < slot_n[wave];
    const uint64_t key = mine ? list[lane] : 0;
    int place = 0, total = 0;
    for (int w = 0; w < kWaves; ++w) {
      const int nw = slot_n[w];
      total += nw;
      for (int i = 0; i < nw; i += kBatch) place += count_above(lists + w * kListCap + i, key);
    }
    if (whole) {
      if (mine && place < a.k) write_top(a, row, place, o, true, key);
      if (tid >= total && tid < a.k) write_top(a, row, tid, o, false, 0);
    } else {
      uint64_t *out = a.part_keys + int64_t(blockIdx.x) * a.k;
      if (mine && place < a.k) out[place] = key;
      if (tid >= total && tid < a.k) out[tid] = 0;    // no key is 0
    }
  }
}

// Joins a row's splits: one workgroup per row.  The splits' lists are sorted,
// so with p = ceil(k / splits) the least of their p-th keys is one that k keys
// reach; only keys from there on are ranked against each other.
constexpr int kMaxJoin = 1024;   // splits * k
constexpr int kMaxSplits = 64;
__global__ void __launch_bounds__(kThreads) score_join_kernel(ScoreArgs a) {
  __shared__ uint64_t keys[kMaxJoin + kBatch];
  __shared__ uint64_t bound;
  __shared__ int kept;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const float c = a.scale * kLog2e;
  const int n = a.splits * a.k;
  const uint64_t *src = a.part_keys + row * n;
  uint64_t mine[kMaxJoin / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxJoin / kThreads; ++i)
    mine[i] = tid + kThreads * i < n ? src[tid + kThreads * i] : 0;
  // the splits' statistics, one lane each, joined over the wave
  const float *p = a.part + row * a.splits * kPartWords + min(lane, a.splits - 1) * kPartWords;
  const int64_t id = a.ids ? a.ids[row] : -1;
  Stat st{p[0], p[1], p[2]};
  int ahead = __float_as_int(p[3]);
  const float lt = p[4];
  if (lane >= a.splits) st = Stat{-3.402823466e38f, 0.f, 0.f}, ahead = 0;
  st = join_wave(st, c);
  ahead = wave_all<SumI>(ahead);
  const RowOut o = finish_row(a, st, ahead, id, lt);
  if (tid == 0) write_scalars(a, row, o);
  if (a.k == 0) return;
  if (tid < 64) {
    uint64_t key = lane < a.splits ? src[lane * a.k + (a.k + a.splits - 1) / a.splits - 1]
                                   : ~uint64_t(0);
    // the least key: its high words first, then the low ones among those
    const uint32_t hi = wave_all<MinU>(uint32_t(key >> 32));
    const uint32_t lo = wave_all<MinU>(uint32_t(key >> 32) == hi ? uint32_t(key) : ~0u);
    if (tid == 0) bound = (uint64_t(hi) << 32) | lo, kept = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMaxJoin / kThreads; ++i)
    if (mine[i] != 0 && mine[i] >= bound) keys[atomicAdd(&kept, 1)] = mine[i];   // in any order
  __syncthreads();
  const int total = kept;
  if (tid < kBatch) keys[total + tid] = 0;
  __syncthreads();
  for (int at = tid; at < total; at += kThreads) {
    const uint64_t key = keys[at];
    int place = 0;
    for (int i = 0; i < total; i += kBatch) place += count_above(keys + i, key);
    if (place < a.k) write_top(a, row, place, o, true, key);
  }
  if (tid >= total && tid < a.k) write_top(a, row, tid, o, false, 0);
}

// A row is split over workgroups until there is about one of them per compute
// unit (16 x 128000 with 20 alternatives: 13.4 us, 17.1 with four per unit, whose
// join has more to rank).  The parts have no more tiles than whole ones would
// and about equal lengths: one of fewer than 8 k elements has no threshold and
// lists all it has (96 x 24799 with 64 alternatives in parts of 12288, 12288 and
// 223: 28 us, 16 in equal ones).
struct ScorePlan {
  int splits, seg;
};
ScorePlan score_plan(int64_t rows, int64_t vocab, int32_t k, int cus) {
  const int64_t tiles = cdiv(vocab, kTile);
  const int64_t most = std::min<int64_t>(kMaxSplits, kMaxJoin / std::max(k, 1));
  const int64_t want = std::min<int64_t>({tiles, cdiv(cus, rows), most});
  const int64_t splits = cdiv(tiles, cdiv(tiles, want));
  return {int(splits), int(cdiv(cdiv(vocab, splits), 16) * 16)};
}

constexpr size_t kPartBytes = kPartWords * sizeof(float);

size_t score_ws(int64_t rows, int64_t vocab, int32_t k, int cus) {
  const ScorePlan p = score_plan(rows, vocab, k, cus);
  if (p.splits == 1) return 0;
  return align256(size_t(rows) * p.splits * kPartBytes) +
         align256(size_t(rows) * p.splits * size_t(k) * sizeof(uint64_t));
}

template <typename T, Ends E>
gptq_status score_ends(const ScoreArgs &a, int64_t rows, hipStream_t s) {
  const dim3 grid(uint32_t(rows * a.splits)), block(kThreads);
  return a.k ? launch("token_logprobs", score_kernel<T, E, true>, grid, block, 0, s, a)
             : launch("token_logprobs", score_kernel<T, E, false>, grid, block, 0, s, a);
}
template <typename T>
gptq_status score_typed(const ScoreArgs &a, int64_t rows, hipStream_t s) {
  switch (ends_of(a.vocab)) {
    case kWhole: GPTQ_TRY((score_ends<T, kWhole>(a, rows, s))); break;
    case kRagged: GPTQ_TRY((score_ends<T, kRagged>(a, rows, s))); break;
    default: GPTQ_TRY((score_ends<T, kShort>(a, rows, s)));
  }
  if (a.splits == 1) return GPTQ_OK;
  return launch("token_logprobs_join", score_join_kernel, dim3(uint32_t(rows)), dim3(kThreads), 0,
                s, a);
}

// A launch has at most 2^32 threads, 256 of them per row here.
constexpr int64_t kMaxVocab = int64_t(1) << 24, kMaxScoreRows = int64_t(1) << 23;
bool valid_score(int64_t rows, int64_t vocab, int32_t k) {
  return rows >= 0 && rows <= kMaxScoreRows && vocab >= 1 && vocab <= kMaxVocab && k >= 0 &&
         k <= kMaxTop && k <= vocab;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" {

size_t gptq_token_logprobs_ws_bytes(int64_t rows, int64_t vocab, int32_t top_k) {
  if (!valid_score(rows, vocab, top_k) || rows == 0) return 0;
  return score_ws(rows, vocab, top_k, device_cu_count());
}

gptq_status gptq_token_logprobs(const void *logits, int32_t dtype, int64_t rows, int64_t vocab,
                                int64_t ld, const int64_t *ids, float scale, int32_t top_k,
                                float *logprob, int32_t *rank, float *entropy, int32_t *top_ids,
                                float *top_logprobs, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> gptq_status {
    if (!valid_score(rows, vocab, top_k))
      return fail(GPTQ_ERR_INVALID_ARG,
                  "rows and vocab must be in [0, 2^23] x [1, 2^24], top_k in [0, min(64, vocab)]");
    if (!is_float_type(dtype))
      return fail(GPTQ_ERR_INVALID_ARG, "the logits' type must be F32, BF16 or F16");
    if (!(scale >= 1e-30f) || !(scale <= 1e30f))
      return fail(GPTQ_ERR_INVALID_ARG, "scale must be in [1e-30, 1e30]");
    if (rows == 0) return GPTQ_OK;
    if (!logits) return fail(GPTQ_ERR_INVALID_ARG, "logits must not be NULL");
    if (!aligned_to(logits, type_bytes(dtype)) || !aligned_to(ids, 8))
      return fail(GPTQ_ERR_INVALID_ARG, "logits and ids must be aligned to their elements");
    if (ld < vocab) return fail(GPTQ_ERR_INVALID_ARG, "ld must be >= vocab");
    if (top_k > 0 && (!top_ids || !top_logprobs))
      return fail(GPTQ_ERR_INVALID_ARG, "top_ids and top_logprobs must not be NULL");
    if ((logprob || rank) && !ids)
      return fail(GPTQ_ERR_INVALID_ARG, "logprob and rank need ids");
    for (const void *p : {(const void *)logprob, (const void *)rank, (const void *)entropy,
                          (const void *)top_ids, (const void *)top_logprobs})
      if (!aligned_to(p, 4)) return fail(GPTQ_ERR_INVALID_ARG, "outputs must be 4-byte aligned");
    const int cus = device_cu_count();
    const ScorePlan plan = score_plan(rows, vocab, top_k, cus);
    const size_t need = score_ws(rows, vocab, top_k, cus);
    if (need) {
      if (!ws) return fail(GPTQ_ERR_WORKSPACE, "workspace is NULL");
      if (!aligned_to(ws, 256))
        return fail(GPTQ_ERR_WORKSPACE, "workspace must be 256-byte aligned");
      if (ws_bytes < need)
        return fail(GPTQ_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) +
                                            " bytes, got " + std::to_string(ws_bytes));
    }
    ScoreArgs a;
    a.logits = logits;
    a.ids = ids;
    a.ld = ld;
    a.vocab = int(vocab);
    a.k = top_k;
    a.splits = plan.splits;
    a.seg = plan.seg;
    a.scale = scale;
    a.logprob = logprob;
    a.rank = rank;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.part = static_cast<float *>(ws);
    a.part_keys = reinterpret_cast<uint64_t *>(
        static_cast<char *>(ws) + (need ? align256(size_t(rows) * plan.splits * kPartBytes) : 0));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == GPTQ_DT_F32) return score_typed<float>(a, rows, s);
    if (dtype == GPTQ_DT_BF16) return score_typed<bf16_t>(a, rows, s);
    return score_typed<f16_t>(a, rows, s);
  });
}

}  // extern "C"
