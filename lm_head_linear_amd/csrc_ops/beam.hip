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
// one piece of a row in registers (32 values a thread, so the loads of a
// piece are all in flight together and nothing is read twice), takes the
// piece's maximum and sum of exponentials, and finds its n_out largest values
// by a threshold: with the 256 threads in 64 groups, the n_out-th largest
// group maximum T has at least n_out values at or above it, all held by a few
// threads, so the values >= T (typically a few more than n_out) go to a list
// in LDS and the list is ranked by counting.  A piece in which more values
// than the list holds reach T (long ties) finds the exact cut by bisection on
// (value, token) keys, which are all different.
// A second kernel, one block per sequence, folds the pieces' sums in fp64 and
// ranks the candidates of all beams by the same threshold.
#include <math.h>

#include "ops_common.h"

namespace lce {

constexpr int kBeamThreads = 256;
constexpr int kBeamVecs = 4;                                     // 8-value vectors per thread
constexpr int kBeamPiece = kBeamThreads * kBeamVecs * 8;         // values of a row per block
constexpr int kBeamGroups = 64;                                  // threshold groups per block
constexpr int kBeamList = 1024;                                  // candidates a block can list
constexpr int64_t kMaxBeams = 32, kMaxBeamOut = 64;
static_assert(kMaxBeamOut <= kBeamGroups, "the threshold needs n_out groups");

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

template <class T> struct Logit;   // eight values at p as fp32
template <bool F16> struct Half8 {};
template <bool F16> struct Logit<Half8<F16>> {
  typedef uint16_t E;
  __device__ static inline void load8(const E *p, float (&f)[8]) { widen8<F16>(load16(p), f); }
  __device__ static inline float load1(const E *p) { return widen<F16>(*p); }
};
template <> struct Logit<float> {
  typedef float E;
  __device__ static inline void load8(const E *p, float (&f)[8]) {
    const u32x4 a = load16(p), b = load16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(a[i]);
      f[4 + i] = __uint_as_float(b[i]);
    }
  }
  __device__ static inline float load1(const E *p) { return *p; }
};

__device__ inline double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ inline int wave_sum(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ inline float wave_max(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}

// Candidates of one piece, best first: (order32(value) << 32) | ~token.
__device__ inline uint64_t piece_key(float x, uint32_t token) {
  return (uint64_t(order32(x)) << 32) | uint32_t(~token);
}

// Block (piece, row): cand[row][piece][n_out] and stats[row][piece].
template <class T>
__global__ void __launch_bounds__(kBeamThreads) beam_piece_kernel(
    const typename Logit<T>::E *logits, const uint8_t *allowed, const uint8_t *finished,
    int64_t vocab, int pieces, int n_out, uint64_t *cand, PieceStats *stats) {
  const int64_t row = blockIdx.x / pieces;
  const int piece = int(blockIdx.x % pieces);
  if (finished && finished[row]) return;     // nothing of the row is read
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t base = int64_t(piece) * kBeamPiece;
  const int64_t left = vocab - base;         // values of the row from here on
  const typename Logit<T>::E *p = logits + row * vocab + base;
  const uint8_t *ok = allowed ? allowed + row * vocab + base : nullptr;

  __shared__ float s_top[4];
  __shared__ double s_sum[4];
  __shared__ float s_group[kBeamGroups];
  __shared__ float s_cut;
  __shared__ int s_count;
  __shared__ uint64_t s_list[kBeamList];

  float f[kBeamVecs][8];
#pragma unroll
  for (int v = 0; v < kBeamVecs; ++v) {
    const int at = (v * kBeamThreads + tid) * 8;
    if (at + 8 <= left) {
      Logit<T>::load8(p + at, f[v]);
      if (ok) {
        const AnyVec8 m = *reinterpret_cast<const AnyVec8 *>(ok + at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (((m.v[i >> 2] >> (8 * (i & 3))) & 0xff) == 0) f[v][i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[v][i] = at + i < left && (!ok || ok[at + i]) ? Logit<T>::load1(p + at + i) : -INFINITY;
    }
  }
  // NaN is passed over by fmaxf and shows in the sum.
  float mine = -INFINITY;
#pragma unroll
  for (int v = 0; v < kBeamVecs; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) mine = fmaxf(mine, f[v][i]);
  // groups of four neighbouring threads
  float group = fmaxf(mine, __shfl_xor(mine, 1));
  group = fmaxf(group, __shfl_xor(group, 2));
  if ((lane & 3) == 0) s_group[tid >> 2] = group;
  float top = wave_max(group);
  if (lane == 0) s_top[wave] = top;
  if (tid == 0) s_count = 0;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  const float m = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kBeamVecs; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sum += __builtin_amdgcn_exp2f((f[v][i] - m) * 1.4426950408889634f);
  const double wsum = wave_sum(double(sum));
  if (lane == 0) s_sum[wave] = wsum;
  // the n_out-th largest group maximum: the group whose rank is n_out - 1,
  // equal ones by place
  if (wave == 0) {
    const float g = s_group[lane];
    int rank = 0;
    for (int j = 0; j < kBeamGroups; ++j) {
      const float o = s_group[j];
      rank += (o > g || (o == g && j < lane)) ? 1 : 0;
    }
    if (rank == n_out - 1) s_cut = g;
  }
  __syncthreads();
  if (tid == 0) {
    PieceStats st;
    st.sum = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    st.top = top;
    st.pad = 0;
    stats[row * pieces + piece] = st;
  }
  // list the values at or above the cut (-inf is no candidate)
  const float cut = s_cut;
  if (mine >= cut) {
#pragma unroll
    for (int v = 0; v < kBeamVecs; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (f[v][i] >= cut && f[v][i] > -INFINITY) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kBeamList)
            s_list[at] = piece_key(f[v][i], uint32_t(base) + (v * kBeamThreads + tid) * 8 + i);
        }
      }
  }
  __syncthreads();
  int count = s_count;
  if (count > kBeamList) {
    // Bisection: the largest key that n_out keys reach.  The keys of the
    // listed values are all different and at least n_out of them exist.
    __shared__ int s_n[4];
    uint64_t lo = 0, hi = ~uint64_t(0);     // reached by >= n_out, by < n_out
    while (hi - lo > 1) {
      const uint64_t mid = lo + (hi - lo) / 2;
      int c = 0;
#pragma unroll
      for (int v = 0; v < kBeamVecs; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          c += f[v][i] > -INFINITY &&
               piece_key(f[v][i], uint32_t(base) + (v * kBeamThreads + tid) * 8 + i) >= mid;
      c = wave_sum(c);
      if (lane == 0) s_n[wave] = c;
      __syncthreads();
      c = s_n[0] + s_n[1] + s_n[2] + s_n[3];
      __syncthreads();
      if (c >= n_out) lo = mid;
      else hi = mid;
      if (c == n_out) break;
    }
    if (tid == 0) s_count = 0;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kBeamVecs; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t key = piece_key(f[v][i], uint32_t(base) + (v * kBeamThreads + tid) * 8 + i);
        if (f[v][i] > -INFINITY && key >= lo) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kBeamList) s_list[at] = key;
        }
      }
    __syncthreads();
    count = s_count;
  }
  uint64_t *out = cand + (row * pieces + piece) * n_out;
  for (int i = tid; i < count; i += kBeamThreads) {
    const uint64_t key = s_list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s_list[j] > key ? 1 : 0;
    if (rank < n_out) out[rank] = key;
  }
  for (int i = count + tid; i < n_out; i += kBeamThreads) out[i] = 0;
}

// A candidate of a sequence: larger total first, then the lower place
// beam * vocab + token.
struct BeamKey {
  uint64_t total;    // order64(total), 0: none
  uint64_t place;
};
__device__ inline bool before(uint64_t ta, uint64_t pa, uint64_t tb, uint64_t pb) {
  return ta > tb || (ta == tb && pa < pb);
}

// One block per sequence.
__global__ void __launch_bounds__(kBeamThreads) beam_merge_kernel(
    const uint64_t *cand, const PieceStats *stats, const float *scores, const uint8_t *finished,
    int beams, int64_t vocab, int pieces, int n_out, int64_t eos, float *out_scores,
    int64_t *out_parents, int64_t *out_tokens, uint8_t *out_finished) {
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __shared__ double s_lse[kMaxBeams];
  __shared__ int8_t s_state[kMaxBeams];     // 0: offers nothing, 1: open, 2: finished
  __shared__ BeamKey s_best[kBeamThreads];
  __shared__ BeamKey s_list[kBeamList];
  __shared__ BeamKey s_cut;
  __shared__ int s_count;

  // normalisers: one wave a beam, its lanes over the pieces
  for (int k = wave; k < beams; k += kBeamThreads / 64) {
    const int64_t row = seq * beams + k;
    const float score = scores[row];
    int state;
    double lse = 0.0;
    if (finished && finished[row]) {
      state = isfinite(score) ? 2 : 0;
    } else {
      float top = -INFINITY;
      for (int c = lane; c < pieces; c += 64) top = fmaxf(top, stats[row * pieces + c].top);
      top = wave_max(top);
      const double m = top == -INFINITY ? 0.0 : double(top);
      double sum = 0.0;
      for (int c = lane; c < pieces; c += 64) {
        const PieceStats st = stats[row * pieces + c];
        sum += st.top == -INFINITY && st.sum == 0.0 ? 0.0 : st.sum * exp(double(st.top) - m);
      }
      lse = m + log(wave_sum(sum));
      state = isfinite(score) && isfinite(lse) ? 1 : 0;   // NaN, +inf or nothing allowed: none
    }
    if (lane == 0) {
      s_lse[k] = lse;
      s_state[k] = int8_t(state);
    }
  }
  if (tid == 0) s_count = 0;
  __syncthreads();

  const int64_t per_beam = int64_t(pieces) * n_out, total_cand = beams * per_beam;
  auto candidate = [&](int64_t i) {
    const int k = int(i / per_beam);
    const int64_t j = i - k * per_beam, row = seq * beams + k;
    BeamKey c{0, ~uint64_t(0)};
    if (s_state[k] == 1) {
      const uint64_t key = cand[row * per_beam + j];
      if (key != 0) {
        const float x = unorder32(uint32_t(key >> 32));
        c.total = order64(double(scores[row]) + (double(x) - s_lse[k]));
        c.place = uint64_t(k) * uint64_t(vocab) + uint32_t(~uint32_t(key));
      }
    } else if (s_state[k] == 2 && j == 0) {
      c.total = order64(double(scores[row]));
      c.place = uint64_t(k) * uint64_t(vocab) + uint64_t(eos);
    }
    return c;
  };
  BeamKey best{0, ~uint64_t(0)};
  for (int64_t i = tid; i < total_cand; i += kBeamThreads) {
    const BeamKey c = candidate(i);
    if (before(c.total, c.place, best.total, best.place)) best = c;
  }
  s_best[tid] = best;
  if (tid == 0) s_cut = BeamKey{0, ~uint64_t(0)};
  __syncthreads();
  if (best.total != 0) {
    int rank = 0;
    for (int j = 0; j < kBeamThreads; ++j)
      rank += before(s_best[j].total, s_best[j].place, best.total, best.place) ? 1 : 0;
    if (rank == n_out - 1) s_cut = best;
  }
  __syncthreads();
  // at least n_out candidates are not behind the cut (all, where there is none)
  BeamKey cut = s_cut;
  auto listed = [&](const BeamKey &c) {
    return c.total != 0 && !before(cut.total, cut.place, c.total, c.place);
  };
  for (int64_t i = tid; i < total_cand; i += kBeamThreads) {
    const BeamKey c = candidate(i);
    if (listed(c)) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kBeamList) s_list[at] = c;
    }
  }
  __syncthreads();
  int count = s_count;
  const int64_t o = seq * n_out;
  auto emit = [&](int at, const BeamKey &c) {
    const bool real = c.total != 0;
    const int64_t token = real ? int64_t(c.place % uint64_t(vocab)) : -1;
    out_scores[o + at] = real ? float(unorder64(c.total)) : -INFINITY;
    out_parents[o + at] = real ? int64_t(c.place / uint64_t(vocab)) : -1;
    out_tokens[o + at] = token;
    if (out_finished) out_finished[o + at] = real && token == eos ? 1 : 0;
  };
  if (count <= kBeamList) {
    for (int i = tid; i < count; i += kBeamThreads) {
      const BeamKey c = s_list[i];
      int rank = 0;
      for (int j = 0; j < count; ++j)
        rank += before(s_list[j].total, s_list[j].place, c.total, c.place) ? 1 : 0;
      if (rank < n_out) emit(rank, c);
    }
    for (int i = count + tid; i < n_out; i += kBeamThreads) emit(i, BeamKey{0, ~uint64_t(0)});
    return;
  }
  // More than the list holds: take the best one n_out times, each after the
  // one before it.
  BeamKey last{~uint64_t(0), 0};
  for (int r = 0; r < n_out; ++r) {
    BeamKey b{0, ~uint64_t(0)};
    for (int64_t i = tid; i < total_cand; i += kBeamThreads) {
      const BeamKey c = candidate(i);
      if (before(last.total, last.place, c.total, c.place) &&
          before(c.total, c.place, b.total, b.place))
        b = c;
    }
    __syncthreads();
    s_best[tid] = b;
    __syncthreads();
    for (int half = kBeamThreads / 2; half > 0; half >>= 1) {
      if (tid < half && before(s_best[tid + half].total, s_best[tid + half].place,
                               s_best[tid].total, s_best[tid].place))
        s_best[tid] = s_best[tid + half];
      __syncthreads();
    }
    last = s_best[0];
    if (tid == 0) emit(r, last);
  }
}

// ------------------------------------------------------------- reordering --

constexpr int kMaxStates = 64;     // states per launch
struct StateList {
  const char *src[kMaxStates];
  char *dst[kMaxStates];
};

// Rows of `segs` segments, the first `bytes` of each `stride` bytes carried
// over: dst row (q, j) = src row (q, parents[q][j]), zeros where the parent is
// no beam.  A thread owns one 16-byte column of a sequence's rows and loads
// it for every destination before it stores any, so src may be dst; there a
// row that stays is neither read nor written.  Bound by memory: each source
// row that has a child is read once (its other children find it in cache).
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
  size_t off_stats = 0, off_cand = 0, total = 0;
};

static int32_t plan_beam(int64_t n_seq, int64_t beams, int64_t vocab, int64_t n_out, BeamPlan *p) {
  if (n_seq < 1 || beams < 1 || vocab < 1 || n_out < 1) return LCE_EMPTY_DIMENSION;
  if (n_seq > LCE_MAX_N_TOK || beams > kMaxBeams || vocab > LCE_MAX_VOCAB || n_out > kMaxBeamOut)
    return LCE_DIMENSION_TOO_LARGE;
  p->rows = n_seq * beams;
  p->pieces = ceil_div(vocab, kBeamPiece);
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
  auto run = [&](auto kernel, auto *x) {
    kernel<<<uint32_t(p.rows * p.pieces), kBeamThreads, 0, st>>>(x, ok, fin, vocab, int(p.pieces),
                                                                 int(n_out), cand, stats);
  };
  if (logits->dtype == LCE_F32)
    run(beam_piece_kernel<float>, static_cast<const float *>(logits->data));
  else if (logits->dtype == LCE_F16)
    run(beam_piece_kernel<Half8<true>>, static_cast<const uint16_t *>(logits->data));
  else
    run(beam_piece_kernel<Half8<false>>, static_cast<const uint16_t *>(logits->data));
  beam_merge_kernel<<<uint32_t(n_seq), kBeamThreads, 0, st>>>(
      cand, stats, static_cast<const float *>(scores->data), fin, int(beams), vocab,
      int(p.pieces), int(n_out), eos, static_cast<float *>(out_scores->data),
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
  if (n_seq > LCE_MAX_N_TOK || beams > kMaxBeams || n_out > kMaxBeams) return LCE_DIMENSION_TOO_LARGE;
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
  for (int32_t i = 0; i < n_states; ++i) {
    if (!holds(&src[i], n_seq * beams * row) || !holds(&dst[i], n_seq * n_out * row))
      return LCE_LENGTH_MISMATCH;
    const char *a = static_cast<const char *>(src[i].data);
    const char *b = static_cast<const char *>(dst[i].data);
    if (i == 0) same = a == b;
    if (same != (a == b) || (same && n_out != beams)) return LCE_LENGTH_MISMATCH;
    const int64_t an = n_seq * beams * row * int64_t(size), bn = n_seq * n_out * row * int64_t(size);
    if (!same && a < b + bn && b < a + an) return LCE_LENGTH_MISMATCH;   // they overlap
  }
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
