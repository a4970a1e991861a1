// beam.hip -- one step of beam search over materialized logits: the n_out best
// (beam, token) pairs of every sequence, and the reordering of per-beam states.
//
// total(k, v) = score_k + x_kv - lse_k over the allowed tokens v of beam k;
// a finished beam offers (eos, score_k) alone.  Within a beam the order of
// totals is the order of the logits, so one pass over a row gives both what
// the normaliser needs (max, sum of exponentials) and the row's n_out largest
// logits; only those meet across beams, in fp64.
//
// Selection, bound by the read of the logits: every block of 256 threads holds
// one piece of a row in registers (8 VECS values a thread, so the loads of a
// piece are all in flight together and nothing is read twice), takes the
// piece's maximum and sum of exponentials, and finds its n_out largest values
// by a threshold: with the 256 threads in 64 groups of four, the n_out-th
// largest group maximum T has at least n_out values at or above it, all held
// by a few threads, so the values >= T (typically a few more than n_out) go to
// a list in LDS and the list is ranked by counting.  T is found by bisecting
// on the bits of the ordered value with one ballot a step, a group maximum a
// lane.  A piece in which more values than the list holds reach T (long ties)
// finds the exact cut by bisection on (value, token) keys, which are all
// different.
// A second kernel, one block per sequence, folds the pieces' sums in fp64 and
// ranks the candidates of all beams by the same kind of threshold.
//
// Measured: 512 x 151936 bf16: 37 us for the pieces (4.2 TB/s: the read, and
// vector work that an earlier form's counters put at about 25 us), 8.7 for the
// 64 sequences' merge, too little work to be more than latency.  64 logits a
// thread as they lie in memory leave room for eight waves a SIMD (50
// registers); held as fp32 they took 200 registers and 75 us.
// Masked by value (the type's lowest number): 44 us in all with 99 % of the
// tokens at random, 42 with the last 293, but 1735 with all behind the first
// 1000, where most pieces are one long tie and every step of the bisection reads
// them again; 99 % masked by `allowed` 52.
#include <math.h>

#include <algorithm>

#include "ops_common.h"

namespace lce {

constexpr int kBeamThreads = 256;
constexpr int kBeamGroups = 64;                                  // threshold groups per block
constexpr int kBeamList = 1024;                                  // candidates a block can list
constexpr int64_t kMaxBeams = 32, kMaxBeamOut = 64;
static_assert(kMaxBeamOut <= kBeamGroups, "the threshold needs n_out groups");
static_assert(LCE_MAX_VOCAB <= (1 << 24) && kMaxBeams <= 128, "a place is beam << 24 | token");

// fp32 in an unsigned order (-0 counts as +0); 0 is below every number.
__device__ inline uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ inline float unorder32(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ inline uint64_t order64(double x) {
  const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));
  return u ^ (u >> 63 ? ~uint64_t(0) : uint64_t(1) << 63);
}
__device__ inline double unorder64(uint64_t k) {
  return __longlong_as_double(int64_t(k ^ (k >> 63 ? uint64_t(1) << 63 : ~uint64_t(0))));
}

// What a piece of a row leaves for the second kernel.
struct PieceStats {
  double sum;       // of exp(x - top)
  float top;        // largest value, -inf when the piece offers none
  int32_t pad;
};

// Eight logits as they lie in memory, and as fp32.
template <class T> struct Logit;
template <bool F16> struct Half8 {};
template <bool F16> struct Logit<Half8<F16>> {
  typedef uint16_t E;
  struct Vec { u32x4 a; };
  __device__ static inline Vec load8(const E *p) { return Vec{load16(p)}; }
  __device__ static inline float load1(const E *p) { return widen<F16>(*p); }
  __device__ static inline void values(const Vec &v, float (&f)[8]) { widen8<F16>(v.a, f); }
  __device__ static inline Vec nothing() {
    const uint32_t none = F16 ? 0xfc00fc00u : 0xff80ff80u;
    return Vec{u32x4{none, none, none, none}};
  }
  // -inf in place i
  __device__ static inline void blank(Vec &v, int i) {
    const uint32_t none = F16 ? 0xfc00u : 0xff80u;
    v.a[i >> 1] = i & 1 ? (v.a[i >> 1] & 0xffffu) | (none << 16) : (v.a[i >> 1] & 0xffff0000u) | none;
  }
  __device__ static inline void put(Vec &v, int i, E x) {
    v.a[i >> 1] = i & 1 ? (v.a[i >> 1] & 0xffffu) | (uint32_t(x) << 16)
                        : (v.a[i >> 1] & 0xffff0000u) | x;
  }
  // makes the values opaque: they are widened again where they are used again
  // (kept as fp32 they would take twice the registers)
  __device__ static inline void hold(Vec &v) { asm volatile("" : "+v"(v.a)); }
};
template <> struct Logit<float> {
  typedef float E;
  struct Vec { u32x4 a, b; };
  __device__ static inline Vec load8(const E *p) { return Vec{load16(p), load16(p + 4)}; }
  __device__ static inline float load1(const E *p) { return *p; }
  __device__ static inline void values(const Vec &v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(v.a[i]);
      f[4 + i] = __uint_as_float(v.b[i]);
    }
  }
  __device__ static inline Vec nothing() {
    const uint32_t none = 0xff800000u;
    return Vec{u32x4{none, none, none, none}, u32x4{none, none, none, none}};
  }
  __device__ static inline void put(Vec &v, int i, E x) {
    (i < 4 ? v.a : v.b)[i & 3] = __float_as_uint(x);
  }
  __device__ static inline void blank(Vec &v, int i) { put(v, i, -INFINITY); }
  __device__ static inline void hold(Vec &v) { asm volatile("" : "+v"(v.a), "+v"(v.b)); }
};

// Lane swaps within a row of 16 lanes (DPP: no LDS), then one lane of each of
// the wave's four rows: the result is uniform.
#define LCE_ROW16(x, op)                                                                \
  x = op(x, __builtin_bit_cast(decltype(x), __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, true)));  /* 1 0 3 2 */       \
  x = op(x, __builtin_bit_cast(decltype(x), __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x4E, 0xF, 0xF, true)));  /* 2 3 0 1 */       \
  x = op(x, __builtin_bit_cast(decltype(x), __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x141, 0xF, 0xF, true))); /* half mirror */   \
  x = op(x, __builtin_bit_cast(decltype(x), __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x140, 0xF, 0xF, true)))  /* mirror */
__device__ inline float row_lane(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ inline float add_f(float a, float b) { return a + b; }
__device__ inline int add_i(int a, int b) { return a + b; }
__device__ inline float wave_max(float x) {
  LCE_ROW16(x, fmaxf);
  return fmaxf(fmaxf(row_lane(x, 0), row_lane(x, 16)), fmaxf(row_lane(x, 32), row_lane(x, 48)));
}
// 16 fp32 terms at a time, the rest in fp64.
__device__ inline double wave_sum_rows(float x) {
  LCE_ROW16(x, add_f);
  return (double(row_lane(x, 0)) + row_lane(x, 16)) + (double(row_lane(x, 32)) + row_lane(x, 48));
}
__device__ inline int wave_sum(int x) {
  LCE_ROW16(x, add_i);
  return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) +
         __builtin_amdgcn_readlane(x, 32) + __builtin_amdgcn_readlane(x, 48);
}
__device__ inline double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// The largest value with BITS leading bits that at least `want` of the wave's
// keys reach (0 when fewer are above 0).
template <int BITS>
__device__ inline uint32_t wave_cut(uint32_t key, int want) {
  uint32_t cut = 0;
#pragma unroll
  for (int bit = 31; bit > 31 - BITS; --bit) {
    const uint32_t next = cut | (1u << bit);
    if (__popcll(__builtin_amdgcn_ballot_w64(key >= next)) >= want) cut = next;
  }
  return cut;
}

// Candidates of one piece, best first: (order32(value) << 32) | ~token.
__device__ inline uint64_t piece_key(float x, uint32_t token) {
  return (uint64_t(order32(x)) << 32) | uint32_t(~token);
}

// Block (row, piece): cand[row][piece][n_out] and stats[row][piece].
// (16-bit logits: at most 80 registers, so that six waves a SIMD keep the
// memory busy while others compute)
template <class T, int VECS, bool MASK>
__global__ void __launch_bounds__(kBeamThreads, sizeof(typename Logit<T>::E) == 2 ? 6 : 3)
    beam_piece_kernel(
    const typename Logit<T>::E *logits, const uint8_t *allowed, const uint8_t *finished,
    int64_t vocab, int pieces, int n_out, uint64_t *cand, PieceStats *stats) {
  constexpr int PIECE = kBeamThreads * VECS * 8;
  const uint32_t row = blockIdx.x / uint32_t(pieces);
  const int piece = int(blockIdx.x - row * uint32_t(pieces));
  if (finished && finished[row]) return;     // nothing of the row is read
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t base = int64_t(piece) * PIECE;
  const int64_t left = vocab - base;         // values of the row from here on
  const typename Logit<T>::E *p = logits + row * vocab + base;
  const uint8_t *ok = MASK ? allowed + row * vocab + base : nullptr;

  __shared__ float s_top[4];
  __shared__ double s_sum[4];
  __shared__ float s_group[kBeamGroups];
  __shared__ float s_cut;
  __shared__ int s_count;
  __shared__ uint64_t s_list[kBeamList];

  typedef typename Logit<T>::Vec Vec;
  Vec x[VECS];
  if (left >= PIECE) {          // block-uniform: all of the piece in flight at once
#pragma unroll
    for (int v = 0; v < VECS; ++v) x[v] = Logit<T>::load8(p + (v * kBeamThreads + tid) * 8);
    if constexpr (MASK) {
      AnyVec8 m[VECS];
#pragma unroll
      for (int v = 0; v < VECS; ++v)
        m[v] = *reinterpret_cast<const AnyVec8 *>(ok + (v * kBeamThreads + tid) * 8);
#pragma unroll
      for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (((m[v].v[i >> 2] >> (8 * (i & 3))) & 0xff) == 0) Logit<T>::blank(x[v], i);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int at = (v * kBeamThreads + tid) * 8;
      x[v] = Logit<T>::nothing();
      if (at + 8 <= left) {
        x[v] = Logit<T>::load8(p + at);
        if constexpr (MASK) {
          const AnyVec8 m = *reinterpret_cast<const AnyVec8 *>(ok + at);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (((m.v[i >> 2] >> (8 * (i & 3))) & 0xff) == 0) Logit<T>::blank(x[v], i);
        }
      } else if (at < left) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < left && (!MASK || ok[at + i])) Logit<T>::put(x[v], i, p[at + i]);
      }
    }
  }
  // NaN is passed over by fmaxf and shows in the sum.
  float mine = -INFINITY;
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    float f[8];
    Logit<T>::values(x[v], f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) mine = fmaxf(mine, fmaxf(f[i], f[i + 1]));
    __builtin_amdgcn_sched_barrier(0);
  }
  float group = fmaxf(mine, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(mine), 0xB1, 0xF, 0xF, true)));
  group = fmaxf(group, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(group), 0x4E, 0xF, 0xF, true)));
  if ((lane & 3) == 0) s_group[tid >> 2] = group;
  float top = wave_max(group);
  if (lane == 0) s_top[wave] = top;
  if (tid == 0) s_count = 0;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  const float m = top == -INFINITY ? 0.0f : top;
  // exp(x - m) = 2^((x - m) log2 e): the difference first, so that it is 0 at
  // the maximum and at most 0 elsewhere however large the logits are (m log2 e
  // subtracted from x log2 e by an fma leaves m's own rounding, which passes
  // 2^7 from |m| of about 3e9 on)
  const float L2E = 1.4426950408889634f;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    float f[8];
    Logit<T>::hold(x[v]);
    Logit<T>::values(x[v], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i & 3] += __builtin_amdgcn_exp2f((f[i] - m) * L2E);
    __builtin_amdgcn_sched_barrier(0);      // (widened values of one vector at a time)
  }
  const double wsum = wave_sum_rows((sum[0] + sum[1]) + (sum[2] + sum[3]));
  if (lane == 0) s_sum[wave] = wsum;
  // one wave finds the cut; 16 bits tell all bf16 values apart
  if (wave == 0) {
    const uint32_t group_key = order32(s_group[lane]);
    const uint32_t none = order32(-INFINITY);
    const uint32_t key = wave_cut<16>(group_key > none ? group_key : 0, n_out);
    if (lane == 0) s_cut = unorder32(key > none ? key : none + 1);   // -inf is no candidate
  }
  __syncthreads();
  const float cut = s_cut;
  // which of the thread's values reach the cut; the few that do are read again
  uint32_t reach[(VECS + 3) / 4];
#pragma unroll
  for (int w = 0; w < (VECS + 3) / 4; ++w) reach[w] = 0;
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    float f[8];
    Logit<T>::hold(x[v]);
    Logit<T>::values(x[v], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) reach[v / 4] |= f[i] >= cut ? 1u << (8 * (v & 3) + i) : 0u;
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int w = 0; w < (VECS + 3) / 4; ++w)
    while (reach[w] != 0) {
      const int bit = __builtin_ctz(reach[w]);
      reach[w] &= reach[w] - 1;
      const int idx = ((w * 4 + bit / 8) * kBeamThreads + tid) * 8 + (bit & 7);
      const int at = atomicAdd(&s_count, 1);
      if (at < kBeamList) s_list[at] = piece_key(Logit<T>::load1(p + idx), uint32_t(base) + idx);
    }
  __syncthreads();
  if (tid == 0) {
    PieceStats st;
    st.sum = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    st.top = top;
    st.pad = 0;
    stats[int64_t(row) * pieces + piece] = st;
  }
  int count = s_count;
  if (count > kBeamList) {
    // Bisection: the largest key that n_out keys reach, a key being the value's
    // order and the place in the piece, lower places first: all different, and
    // at least n_out of them exist.  The values are read again in every step.
    constexpr int PLACE = 16;
    static_assert(PIECE <= 1 << PLACE, "places in a piece");
    __shared__ int s_n[4];
    auto key_at = [&](int idx) {
      if (idx >= left || (MASK && !ok[idx])) return uint64_t(0);
      const float value = Logit<T>::load1(p + idx);
      return value >= cut ? (uint64_t(order32(value)) << PLACE) | uint32_t((1 << PLACE) - 1 - idx)
                          : uint64_t(0);
    };
    uint64_t lo_key = uint64_t(order32(cut)) << PLACE;                    // reached by >= n_out
    uint64_t hi_key = (uint64_t(order32(top)) << PLACE) + (1 << PLACE);   // by none
    while (hi_key - lo_key > 1) {
      const uint64_t mid = lo_key + (hi_key - lo_key) / 2;
      int c = 0;
      for (int idx = tid; idx < PIECE; idx += kBeamThreads) c += key_at(idx) >= mid ? 1 : 0;
      c = wave_sum(c);
      if (lane == 0) s_n[wave] = c;
      __syncthreads();
      c = s_n[0] + s_n[1] + s_n[2] + s_n[3];
      __syncthreads();
      if (c >= n_out) lo_key = mid;
      else hi_key = mid;
      if (c == n_out) break;
    }
    if (tid == 0) s_count = 0;
    __syncthreads();
    for (int idx = tid; idx < PIECE; idx += kBeamThreads) {
      const uint64_t key = key_at(idx);
      if (key >= lo_key) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kBeamList)
          s_list[at] = piece_key(unorder32(uint32_t(key >> PLACE)), uint32_t(base) + idx);
      }
    }
    __syncthreads();
    count = s_count;
  }
  uint64_t *out = cand + (int64_t(row) * pieces + piece) * n_out;
  for (int i = tid; i < count; i += kBeamThreads) {
    const uint64_t key = s_list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s_list[j] > key ? 1 : 0;
    if (rank < n_out) out[rank] = key;
  }
  for (int i = count + tid; i < n_out; i += kBeamThreads) out[i] = 0;
}

// A candidate of a sequence: larger total first, then the lower place
// (beam << 24 | token).
struct BeamKey {
  uint64_t total;    // order64(total), 0: none
  uint32_t place;
};
__device__ inline bool before(const BeamKey &a, const BeamKey &b) {
  return a.total > b.total || (a.total == b.total && a.place < b.place);
}

// One block per sequence.
__global__ void __launch_bounds__(kBeamThreads) beam_merge_kernel(
    const uint64_t *cand, const PieceStats *stats, const float *scores, const uint8_t *finished,
    int beams, int pieces, int n_out, int64_t eos, float *out_scores, int64_t *out_parents,
    int64_t *out_tokens, uint8_t *out_finished) {
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // A total is score + ((x - top) - log_sum): the maximum goes first, so that
  // a large one does not swallow the logarithm.
  __shared__ double s_score[kMaxBeams], s_top[kMaxBeams], s_log_sum[kMaxBeams];
  __shared__ int s_state[kMaxBeams];        // 0: offers nothing, 1: open, 2: finished
  __shared__ uint64_t s_total[kBeamList];
  __shared__ uint32_t s_place[kBeamList];
  __shared__ uint32_t s_group[kBeamGroups];
  __shared__ int s_count;

  // the thread's first eight candidates, on their way while the rest begins
  const int per_beam = pieces * n_out, total = beams * per_beam;
  const uint64_t *keys = cand + seq * total;
  uint64_t held[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = tid + u * kBeamThreads;
    held[u] = i < total ? keys[i] : 0;
  }
  // normalisers: 32 lanes a beam, each folding the pieces it meets
  for (int k = tid >> 5; k < beams; k += kBeamThreads / 32) {
    const int64_t row = seq * beams + k;
    const float score = scores[row];
    const bool done = finished && finished[row];
    float top = -INFINITY;
    double sum = 0.0;
    if (!done) {
      // the first 32 pieces are held, further ones (a vocabulary beyond 2^19)
      // are read again
      const int c0 = tid & 31;
      PieceStats st = {0.0, -INFINITY, 0};
      if (c0 < pieces) st = stats[row * pieces + c0];
      top = st.top;
      for (int c = c0 + 32; c < pieces; c += 32) top = fmaxf(top, stats[row * pieces + c].top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
      const double m = top == -INFINITY ? 0.0 : double(top);
      // (a maximum of -inf comes with a sum of 0, or of NaN, which stays)
      sum = st.sum == 0.0 ? 0.0 : st.sum * exp(double(st.top) - m);
      for (int c = c0 + 32; c < pieces; c += 32) {
        st = stats[row * pieces + c];
        if (st.sum != 0.0) sum += st.sum * exp(double(st.top) - m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    }
    if ((tid & 31) == 0) {
      const double log_sum = log(sum);
      s_score[k] = score;
      s_top[k] = top;
      s_log_sum[k] = log_sum;
      // NaN, +inf (whose sum is NaN) or nothing allowed: the beam offers nothing
      s_state[k] = !isfinite(score) ? 0 : done ? 2 : isfinite(log_sum) ? 1 : 0;
    }
  }
  if (tid == 0) s_count = 0;
  __syncthreads();

  // every candidate of the sequence that this thread looks at
  auto each = [&](auto &&use) {
    auto look = [&](const uint64_t (&key)[8], int i0) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t k = uint32_t(i0 + u * kBeamThreads) / uint32_t(per_beam);
        if (key[u] != 0 && k < uint32_t(beams) && s_state[k] == 1)
          use(BeamKey{order64(s_score[k] + ((double(unorder32(uint32_t(key[u] >> 32))) - s_top[k]) -
                                            s_log_sum[k])),
                      (k << 24) | ~uint32_t(key[u])});
      }
    };
    look(held, tid);
    for (int i0 = tid + 8 * kBeamThreads; i0 < total; i0 += 8 * kBeamThreads) {
      uint64_t key[8];                       // eight loads in flight
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kBeamThreads;
        key[u] = i < total ? keys[i] : 0;
      }
      look(key, i0);
    }
    if (tid < beams && s_state[tid] == 2)
      use(BeamKey{order64(s_score[tid]), (uint32_t(tid) << 24) | uint32_t(eos)});
  };
  uint32_t best = 0;      // the leading half of the largest total
  each([&](const BeamKey &c) {
    const uint32_t h = uint32_t(c.total >> 32);
    best = h > best ? h : best;
  });
  uint32_t o = __builtin_amdgcn_mov_dpp(int(best), 0xB1, 0xF, 0xF, true);
  best = o > best ? o : best;
  o = __builtin_amdgcn_mov_dpp(int(best), 0x4E, 0xF, 0xF, true);
  best = o > best ? o : best;
  if ((lane & 3) == 0) s_group[tid >> 2] = best;
  __syncthreads();
  // at least n_out candidates reach the cut (all, where there are fewer groups)
  const uint32_t cut = wave_cut<32>(s_group[lane], n_out);
  each([&](const BeamKey &c) {
    if (uint32_t(c.total >> 32) >= cut) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kBeamList) {
        s_total[at] = c.total;
        s_place[at] = c.place;
      }
    }
  });
  __syncthreads();
  const int count = s_count;
  const int64_t first = seq * n_out;
  auto emit = [&](int at, const BeamKey &c) {
    const bool real = c.total != 0;
    const int64_t token = real ? int64_t(c.place & 0xffffffu) : -1;
    out_scores[first + at] = real ? float(unorder64(c.total)) : -INFINITY;
    out_parents[first + at] = real ? int64_t(c.place >> 24) : -1;
    out_tokens[first + at] = token;
    if (out_finished) out_finished[first + at] = real && token == eos ? 1 : 0;
  };
  if (count <= kBeamList) {
    for (int i = tid; i < count; i += kBeamThreads) {
      const BeamKey c{s_total[i], s_place[i]};
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += before(BeamKey{s_total[j], s_place[j]}, c) ? 1 : 0;
      if (rank < n_out) emit(rank, c);
    }
    for (int i = count + tid; i < n_out; i += kBeamThreads) emit(i, BeamKey{0, 0});
    return;
  }
  // More than the list holds (totals whose leading halves are equal): take the
  // best one n_out times, each after the one before it.
  BeamKey last{~uint64_t(0), 0};
  for (int r = 0; r < n_out; ++r) {
    BeamKey b{0, ~0u};
    each([&](const BeamKey &c) {
      if (before(last, c) && before(c, b)) b = c;
    });
    __syncthreads();
    s_total[tid] = b.total;
    s_place[tid] = b.place;
    __syncthreads();
    for (int half = kBeamThreads / 2; half > 0; half >>= 1) {
      if (tid < half) {
        const BeamKey x{s_total[tid], s_place[tid]}, y{s_total[tid + half], s_place[tid + half]};
        if (before(y, x)) {
          s_total[tid] = y.total;
          s_place[tid] = y.place;
        }
      }
      __syncthreads();
    }
    last = BeamKey{s_total[0], s_place[0]};
    if (tid == 0) emit(r, last);
  }
}

// ------------------------------------------------------------- reordering --

constexpr int kMaxStates = 64;     // states per launch
constexpr int kMostStates = 1024;  // states per call
struct Span {
  uintptr_t begin, end;
};
struct StateList {
  const char *src[kMaxStates];
  char *dst[kMaxStates];
};

// Rows of `segs` segments, the first `bytes` of each `stride` bytes carried
// over: dst row (q, j) = src row (q, parents[q][j]), zeros where the parent is
// no beam.  A thread owns one 16-byte column of a sequence's rows and loads
// it for every destination before it stores any, so src may be dst; there a
// row that stays is neither read nor written.  Bound by memory: each source
// row that has a child is read once (its other children find it in cache);
// 64 rows of 16 caches [8][777 of 1024][128] bf16, 2.7 GB: 498 us, 5.4 TB/s.
template <int B>
__global__ void __launch_bounds__(256) beam_reorder_kernel(
    StateList list, const int64_t *parents, int64_t n_seq, int beams, int n_out, int64_t segs,
    int64_t bytes, int64_t stride, int in_place) {
  const int64_t cols = (bytes + 15) / 16, total = segs * cols;
  const int64_t row_bytes = segs * stride;
  const char *src = list.src[blockIdx.z];
  char *dst = list.dst[blockIdx.z];
  for (int64_t q = blockIdx.y; q < n_seq; q += gridDim.y) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += int64_t(gridDim.x) * 256) {
      const int64_t seg = i / cols, col = i - seg * cols;
      const int64_t at = seg * stride + col * 16;
      const int n = bytes - col * 16 >= 16 ? 16 : int(bytes - col * 16);
      const char *s = src + q * beams * row_bytes + at;
      char *d = dst + q * n_out * row_bytes + at;
      u32x4 v[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        v[j] = u32x4{0, 0, 0, 0};
        if (j < n_out) {
          const int64_t k = parents[q * n_out + j];
          if (k >= 0 && k < beams && !(in_place && k == j)) {
            const char *a = s + k * row_bytes;
            if (n == 16) {
              v[j] = load16(a);
            } else {
              uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
              for (int b = 0; b < 15; ++b)
                if (b < n) w[b >> 2] |= uint32_t(uint8_t(a[b])) << (8 * (b & 3));
              v[j] = u32x4{w[0], w[1], w[2], w[3]};
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (j < n_out && !(in_place && parents[q * n_out + j] == j)) {
          char *a = d + j * row_bytes;
          if (n == 16) {
            store16(a, v[j]);
          } else {
#pragma unroll
            for (int b = 0; b < 15; ++b)
              if (b < n) a[b] = char(v[j][b >> 2] >> (8 * (b & 3)));
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------- host --

struct BeamPlan {
  int64_t rows = 0, pieces = 0;
  int vecs = 0;             // 8-value vectors a thread of the first kernel holds
  size_t off_stats = 0, off_cand = 0, total = 0;
};

static int32_t plan_beam(int64_t n_seq, int64_t beams, int64_t vocab, int64_t n_out, BeamPlan *p) {
  if (n_seq < 1 || beams < 1 || vocab < 1 || n_out < 1) return LCE_EMPTY_DIMENSION;
  if (n_seq > LCE_MAX_N_TOK || beams > kMaxBeams || vocab > LCE_MAX_VOCAB || n_out > kMaxBeamOut)
    return LCE_DIMENSION_TOO_LARGE;
  p->rows = n_seq * beams;
  // Long pieces leave fewer candidates to merge, short ones spread a small
  // call over the chip.
  p->vecs = p->rows * vocab >= int64_t(1024) * kBeamThreads * 64 ? 8 : 2;
  p->pieces = ceil_div(vocab, kBeamThreads * 8 * p->vecs);
  // (a launch holds fewer than 2^32 threads)
  if (p->rows * p->pieces >= (int64_t(1) << 32) / kBeamThreads) return LCE_WORK_BUDGET_EXCEEDED;
  p->off_stats = 0;
  p->off_cand = size_t(round_to(p->rows * p->pieces * int64_t(sizeof(PieceStats)), 256));
  p->total = p->off_cand + size_t(p->rows * p->pieces * n_out) * 8 + 256;
  return LCE_OK;
}

}  // namespace lce

using namespace lce;

extern "C" {

int64_t lce_beam_workspace_bytes(int64_t n_seq, int64_t beams, int64_t vocab, int64_t n_out) {
  BeamPlan p;
  const int32_t st = plan_beam(n_seq, beams, vocab, n_out, &p);
  return st == LCE_OK ? int64_t(p.total) : -int64_t(st);
}

int32_t lce_beam_select(const lce_tensor *logits, const lce_tensor *scores,
                        const lce_tensor *finished, const lce_tensor *allowed, int64_t n_seq,
                        int64_t beams, int64_t vocab, int64_t n_out, int64_t eos,
                        lce_tensor *out_scores, lce_tensor *out_parents, lce_tensor *out_tokens,
                        lce_tensor *out_finished, lce_tensor *workspace, void *stream) {
  BeamPlan p;
  if (const int32_t st = plan_beam(n_seq, beams, vocab, n_out, &p); st != LCE_OK) return st;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace)
    return LCE_LENGTH_MISMATCH;
  if ((!half_type(logits->dtype) && logits->dtype != LCE_F32) || scores->dtype != LCE_F32 ||
      out_scores->dtype != LCE_F32 || out_parents->dtype != LCE_I64 ||
      out_tokens->dtype != LCE_I64 || workspace->dtype != LCE_U8 ||
      (given(finished) && finished->dtype != LCE_U8) ||
      (given(allowed) && allowed->dtype != LCE_U8) ||
      (given(out_finished) && out_finished->dtype != LCE_U8))
    return LCE_DTYPE_MISMATCH;
  const int64_t outs = n_seq * n_out;
  if (!holds(logits, p.rows * vocab) || !holds(scores, p.rows) || !holds(out_scores, outs) ||
      !holds(out_parents, outs) || !holds(out_tokens, outs) ||
      !holds(workspace, int64_t(p.total)) || (given(finished) && finished->numel < p.rows) ||
      (given(allowed) && allowed->numel < p.rows * vocab) ||
      (given(out_finished) && out_finished->numel < outs))
    return LCE_LENGTH_MISMATCH;
  if (eos < -1 || eos >= vocab || (eos < 0 && given(finished))) return LCE_TARGET_OUT_OF_RANGE;

  (void)hipGetLastError();
  const hipStream_t st = hipStream_t(stream);
  char *ws = aligned_base(workspace);
  PieceStats *stats = reinterpret_cast<PieceStats *>(ws + p.off_stats);
  uint64_t *cand = reinterpret_cast<uint64_t *>(ws + p.off_cand);
  const uint8_t *fin = given(finished) ? static_cast<const uint8_t *>(finished->data) : nullptr;
  const uint8_t *ok = given(allowed) ? static_cast<const uint8_t *>(allowed->data) : nullptr;
  auto run = [&](auto type, auto *x) {
    typedef decltype(type) T;
    auto go = [&](auto kernel) {
      kernel<<<uint32_t(p.rows * p.pieces), kBeamThreads, 0, st>>>(
          x, ok, fin, vocab, int(p.pieces), int(n_out), cand, stats);
    };
    if (p.vecs == 8) ok ? go(beam_piece_kernel<T, 8, true>) : go(beam_piece_kernel<T, 8, false>);
    else ok ? go(beam_piece_kernel<T, 2, true>) : go(beam_piece_kernel<T, 2, false>);
  };
  if (logits->dtype == LCE_F32) run(float(), static_cast<const float *>(logits->data));
  else if (logits->dtype == LCE_F16)
    run(Half8<true>(), static_cast<const uint16_t *>(logits->data));
  else run(Half8<false>(), static_cast<const uint16_t *>(logits->data));
  beam_merge_kernel<<<uint32_t(n_seq), kBeamThreads, 0, st>>>(
      cand, stats, static_cast<const float *>(scores->data), fin, int(beams), int(p.pieces),
      int(n_out), eos, static_cast<float *>(out_scores->data),
      static_cast<int64_t *>(out_parents->data), static_cast<int64_t *>(out_tokens->data),
      given(out_finished) ? static_cast<uint8_t *>(out_finished->data) : nullptr);
  return enqueued_status();
}

int32_t lce_beam_reorder(const lce_tensor *src, lce_tensor *dst, int32_t n_states,
                         const lce_tensor *parents, int64_t n_seq, int64_t beams, int64_t n_out,
                         int64_t segs, int64_t seg_elems, int64_t seg_stride, void *stream) {
  if (n_states < 1 || n_seq < 1 || beams < 1 || n_out < 1 || segs < 1 || seg_elems < 0 ||
      seg_stride < 1)
    return LCE_EMPTY_DIMENSION;
  if (n_seq > LCE_MAX_N_TOK || beams > kMaxBeams || n_out > kMaxBeams || n_states > kMostStates)
    return LCE_DIMENSION_TOO_LARGE;
  // the elements of one state: within 2^46
  const int64_t most = beams > n_out ? beams : n_out;
  if (!lce_work_fits(segs, seg_stride, n_seq * most, LCE_MAX_WORK_CELLS))
    return LCE_WORK_BUDGET_EXCEEDED;
  if (!src || !dst || !parents) return LCE_LENGTH_MISMATCH;
  if (parents->dtype != LCE_I64) return LCE_DTYPE_MISMATCH;
  const size_t size = dtype_size(src[0].dtype);
  bool same = true;
  for (int32_t i = 0; i < n_states; ++i)
    if (dtype_size(src[i].dtype) == 0 || src[i].dtype != dst[i].dtype || dtype_size(src[i].dtype) != size)
      return LCE_DTYPE_MISMATCH;
  if (seg_elems > seg_stride || !holds(parents, n_seq * n_out)) return LCE_LENGTH_MISMATCH;
  const int64_t row = segs * seg_stride;
  // every destination by itself, and no source in one but its own
  Span to[kMostStates];
  const uintptr_t from_bytes = uintptr_t(n_seq * beams * row) * size;
  const uintptr_t to_bytes = uintptr_t(n_seq * n_out * row) * size;
  for (int32_t i = 0; i < n_states; ++i) {
    if (!holds(&src[i], n_seq * beams * row) || !holds(&dst[i], n_seq * n_out * row))
      return LCE_LENGTH_MISMATCH;
    const bool here = src[i].data == dst[i].data;
    if (i == 0) same = here;
    if (same != here || (same && n_out != beams)) return LCE_LENGTH_MISMATCH;
    const uintptr_t at = reinterpret_cast<uintptr_t>(dst[i].data);
    to[i] = {at, at + to_bytes};
  }
  std::sort(to, to + n_states, [](const Span &a, const Span &b) { return a.begin < b.begin; });
  for (int32_t i = 1; i < n_states; ++i)
    if (to[i].begin < to[i - 1].end) return LCE_LENGTH_MISMATCH;
  auto meets = [&](uintptr_t begin, uintptr_t end) {
    const Span *s = std::upper_bound(to, to + n_states, begin,
                                     [](uintptr_t x, const Span &t) { return x < t.end; });
    return s != to + n_states && s->begin < end;
  };
  for (int32_t i = 0; !same && i < n_states; ++i) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(src[i].data);
    if (meets(at, at + from_bytes)) return LCE_LENGTH_MISMATCH;
  }
  const uintptr_t order = reinterpret_cast<uintptr_t>(parents->data);
  if (meets(order, order + uintptr_t(n_seq * n_out) * 8)) return LCE_LENGTH_MISMATCH;
  if (seg_elems == 0) return LCE_OK;

  (void)hipGetLastError();
  const int64_t bytes = seg_elems * int64_t(size), stride = seg_stride * int64_t(size);
  const int64_t cols = segs * ceil_div(bytes, 16);
  const int64_t gx = ceil_div(cols, 256) < 65536 ? ceil_div(cols, 256) : 65536;
  const int64_t gy = n_seq < 32768 ? n_seq : 32768;
  for (int32_t first = 0; first < n_states; first += kMaxStates) {
    const int count = n_states - first < kMaxStates ? n_states - first : kMaxStates;
    StateList list = {};
    for (int i = 0; i < count; ++i) {
      list.src[i] = static_cast<const char *>(src[first + i].data);
      list.dst[i] = static_cast<char *>(dst[first + i].data);
    }
    auto run = [&](auto kernel) {
      kernel<<<dim3(uint32_t(gx), uint32_t(gy), uint32_t(count)), 256, 0, hipStream_t(stream)>>>(
          list, static_cast<const int64_t *>(parents->data), n_seq, int(beams), int(n_out), segs,
          bytes, stride, same ? 1 : 0);
    };
    if (n_out <= 4) run(beam_reorder_kernel<4>);
    else if (n_out <= 8) run(beam_reorder_kernel<8>);
    else if (n_out <= 16) run(beam_reorder_kernel<16>);
    else run(beam_reorder_kernel<32>);
  }
  return enqueued_status();
}

}  // extern "C"
