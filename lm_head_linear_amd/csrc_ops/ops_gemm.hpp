// ops_gemm.hpp -- 16-bit product C[m][c] = sum_k A[m][k] B[c][k] on the matrix
// cores for tiles smaller than the 256 x 256 core of lce_gemm2.hpp, and the
// epilogue that both share.
//
// Both operands are K-major with leading dimensions that are multiples of 8
// and 16-byte aligned bases.  Stages of 64 k go global -> LDS by DMA (no
// registers in between) into a ring of STAGES buffers, STAGES - 1 ahead; a
// k-step is one wait for its own stage, one barrier, the issue of the stage
// that takes the buffer just freed, and 4 MFMA substeps.  Chunks behind the
// last k and rows behind the last row are fetched from behind the buffer's
// end, which reads as zero.
//
// What bounds it: fitted over sweeps of the depth, a 64 x 64 tile's step takes
// 0.34 us alone on its compute unit and 0.41 beside a second.  A deeper ring (5
// and 9 stages), all fragments read ahead (3 to 5 %) and the step split over
// the waves changed little; which part of the step's chain of wait, barrier, LDS
// reads and products sets it has not been separated.
#pragma once

#include "../csrc/lce_gemm2.hpp"
#include "ops_common.h"

namespace lce {

enum Act { kNone = LCE_ACT_NONE, kRelu = LCE_ACT_RELU, kGelu = LCE_ACT_GELU, kSilu = LCE_ACT_SILU };

// The normal distribution function P(z) and e = exp(-z^2 / 2).  The lower tail
// of |z| is t Q(t) e with t = 1 / (1 + c |z|), which runs from 1 at z = 0 to 0:
// t Q(t) follows erfc(|z| / sqrt 2) exp(z^2 / 2) / 2, which falls as 1 / |z|.
// Q, of degree 7, is fitted to its relative error, 1e-7 for |z| up to 14.4 (fp32
// has no tail beyond), so a small result of gelu is as exact as a large one:
// within (21 + 1.2 z^2) 2^-24 relatively, where a sum 1 + erf loses the tail.
// One exponential and one reciprocal (8192 x 4096 outputs: 259 us a call; the
// library's erff took 32 more).
__device__ inline void normal_cdf(float z, float &cdf, float &e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.23405234515666962f, 1.0f));
  float q = fmaf(t, -0.0662810877f, 0.221980631f);
  q = fmaf(q, t, -0.163418442f);
  q = fmaf(q, t, 0.194321081f);
  q = fmaf(q, t, 0.0284388866f);
  q = fmaf(q, t, 0.0995572284f);
  q = fmaf(q, t, 0.0919526592f);
  q = fmaf(q, t, 0.0934489965f);
  e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  const float tail = q * t * e;
  cdf = z < 0.0f ? tail : 1.0f - tail;
}
__device__ inline float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
__device__ inline float act_value(float z, int act) {
  if (act == kRelu) return z > 0.0f || z != z ? z : 0.0f;
  if (act == kGelu) {
    float cdf, e;
    normal_cdf(z, cdf, e);
    return z * cdf;
  }
  if (act == kSilu) return z * sigmoid(z);
  return z;
}
__device__ inline float act_slope(float z, int act) {
  if (act == kRelu) return z > 0.0f ? 1.0f : 0.0f;
  if (act == kGelu) {
    float cdf, e;
    normal_cdf(z, cdf, e);
    return fmaf(z * 0.39894228040143268f, e, cdf);
  }
  if (act == kSilu) {
    const float s = sigmoid(z);
    return fmaf(z * s, 1.0f - s, s);
  }
  return 1.0f;
}

// ------------------------------------------------------------- epilogue --

// What becomes of C[m][c], element m of row c of the result.
struct OutParams {
  void *out;                 // [cols][ld]
  int64_t ld;
  int64_t rows, cols;        // valid m and c
  const void *bias;          // [rows], 16-bit or fp32, or null
  const uint16_t *residual;  // [cols][ld] or null
  uint16_t *preact;          // [cols][ld] or null
  int64_t split_stride;      // elements between the splits' results (fp32)
  int32_t out_f32, bias_f32, act, add;   // add: out += C
};

// The bias of elements m .. m + W - 1, of which `count` exist (0 behind).
template <bool F16, int W>
__device__ inline void load_bias(const OutParams &p, int64_t m, int count, float (&b)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) b[i] = 0.0f;
  if (!p.bias) return;
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < count)
      b[i] = p.bias_f32 ? static_cast<const float *>(p.bias)[m + i]
                        : widen<F16>(static_cast<const uint16_t *>(p.bias)[m + i]);
}

// W (4 or 8) consecutive 16-bit or fp32 values at any alignment; the first
// `count` of them exist.
template <bool F16, int W>
__device__ inline void read_half(const uint16_t *p, int count, float (&f)[W]) {
  if (count == W) {
    uint32_t v[W / 2];
    __builtin_memcpy(v, __builtin_assume_aligned(p, 2), W * 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      f[2 * i] = widen<F16>(uint16_t(v[i]));
      f[2 * i + 1] = widen<F16>(uint16_t(v[i] >> 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = i < count ? widen<F16>(p[i]) : 0.0f;
  }
}
template <bool F16, int W>
__device__ inline void write_half(uint16_t *p, int count, const float (&f)[W]) {
  if (count == W) {
    uint32_t v[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
      v[i] = uint32_t(narrow<F16>(f[2 * i])) | (uint32_t(narrow<F16>(f[2 * i + 1])) << 16);
    __builtin_memcpy(__builtin_assume_aligned(p, 2), v, W * 2);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < count) p[i] = narrow<F16>(f[i]);
  }
}

// Elements m .. m + W - 1 of row c of split `split`: z the sums, b the bias.
template <bool F16, int W>
__device__ __forceinline__ void finish(const OutParams &p, float (&z)[W], const float (&b)[W],
                                       int64_t m, int64_t c, int count, int split) {
  const int64_t at = c * p.ld + m;
#pragma unroll
  for (int i = 0; i < W; ++i) z[i] += b[i];
  if (p.preact) write_half<F16, W>(p.preact + at, count, z);
  if (p.act != kNone) {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] = act_value(z[i], p.act);
  }
  if (p.residual) {
    float r[W];
    read_half<F16, W>(p.residual + at, count, r);
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] += r[i];
  }
  if (p.out_f32) {
    float *o = static_cast<float *>(p.out) + split * p.split_stride + at;
    if (count == W) {
      if (p.add) {
        float r[W];
        __builtin_memcpy(r, __builtin_assume_aligned(o, 4), W * 4);
#pragma unroll
        for (int i = 0; i < W; ++i) z[i] += r[i];
      }
      __builtin_memcpy(__builtin_assume_aligned(o, 4), z, W * 4);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < count) o[i] = p.add ? o[i] + z[i] : z[i];
    }
  } else {
    uint16_t *o = static_cast<uint16_t *>(p.out) + at;
    if (p.add) {
      float r[W];
      read_half<F16, W>(o, count, r);
#pragma unroll
      for (int i = 0; i < W; ++i) z[i] += r[i];
    }
    write_half<F16, W>(o, count, z);
  }
}

// The same for eight elements that all exist and overwrite, the residual
// loaded before.
template <bool F16>
__device__ __forceinline__ void finish_whole(const OutParams &p, float (&z)[8], const float (&b)[8],
                                             const u32x4 &res, int64_t at, int split) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
  if (p.preact) store16(p.preact + at, narrow8<F16>(z));
  if (p.act == kGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kGelu);
  } else if (p.act == kSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kSilu);
  } else if (p.act == kRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kRelu);
  }
  if (p.residual) {
    float r[8];
    widen8<F16>(res, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
  if (p.out_f32) {
    float *o = static_cast<float *>(p.out) + split * p.split_stride + at;
    u32x4 x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __float_as_uint(z[i]);
      y[i] = __float_as_uint(z[4 + i]);
    }
    store16(o, x);
    store16(o + 4, y);
  } else {
    store16(static_cast<uint16_t *>(p.out) + at, narrow8<F16>(z));
  }
}

// Epilogue of both cores: a wave passes its accumulators through its own part
// of LDS, 32 rows of the result at a time, so that global accesses are 16
// bytes a lane along the rows.  The 16-byte chunks of an LDS row are XORed
// with the row's number, which spreads the column-wise writes over the banks.
template <class TR>
struct OutEpi {
  OutParams p;
  static constexpr bool kStaged = true;
  static constexpr int CH = TR::WTM / 4;                  // 16-byte chunks per row
  static constexpr int MASK = CH < 16 ? CH - 1 : 15;
  static constexpr int BYTES = 32 * TR::WTM * 4;          // LDS per wave

  __device__ __forceinline__ void staged(typename TR::AccBlock (&acc)[TR::FM][TR::FN], int64_t m0,
                                         int64_t n0, int wm, int wn, int lane, int split,
                                         char *lds, const char *) const {
    const int64_t mw = m0 + wm * TR::WTM, cw = n0 + wn * TR::WTN;
    if (mw >= p.rows || cw >= p.cols) return;             // wave-uniform
    char *region = lds + (wm * TR::WAVES_N + wn) * BYTES;
    constexpr int LPR = TR::WTM / 8;                      // lanes per row
    const int j = lane % LPR, r0 = lane / LPR;
    const int64_t m = mw + j * 8;
    const int count = m >= p.rows ? 0 : (p.rows - m >= 8 ? 8 : int(p.rows - m));
    float b[8];
    load_bias<TR::F16, 8>(p, m, count, b);
    constexpr int IT = 32 * LPR / 64;                     // rows of a lane in 32 rows
    const bool whole = mw + TR::WTM <= p.rows && !p.add;  // wave-uniform
#pragma unroll
    for (int fn = 0; fn < TR::FN; ++fn) {
      const int row = lane & 31;
      const int64_t c0 = cw + fn * 32 + r0;
      // the residual's loads go out before the accumulators are moved
      u32x4 res[IT];
      if (whole && p.residual) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int64_t col = c0 + i * (64 / LPR);
          res[i] = load16(p.residual + (col < p.cols ? col : cw) * p.ld + m);
        }
      }
#pragma unroll
      for (int fm = 0; fm < TR::FM; ++fm)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int ch = fm * 8 + 2 * q + (lane >> 5);
          f32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = acc[fm][fn][4 * q + i];
          *reinterpret_cast<f32x4 *>(region + row * (TR::WTM * 4) + ((ch ^ (row & MASK)) << 4)) = v;
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      auto sums = [&](int rr, float (&z)[8]) {
        const char *q = region + rr * (TR::WTM * 4);
        const f32x4 a = *reinterpret_cast<const f32x4 *>(q + (((2 * j) ^ (rr & MASK)) << 4));
        const f32x4 c = *reinterpret_cast<const f32x4 *>(q + (((2 * j + 1) ^ (rr & MASK)) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[i] = a[i];
          z[4 + i] = c[i];
        }
      };
      if (whole) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          float z[8];
          sums(r0 + i * (64 / LPR), z);
          const int64_t col = c0 + i * (64 / LPR);
          if (col < p.cols) finish_whole<TR::F16>(p, z, b, res[i], col * p.ld + m, split);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < IT; ++i) {
          float z[8];
          sums(r0 + i * (64 / LPR), z);
          const int64_t col = c0 + i * (64 / LPR);
          if (col < p.cols && count > 0) finish<TR::F16, 8>(p, z, b, m, col, count, split);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before it is overwritten
    }
  }
  typedef float f32x4 __attribute__((ext_vector_type(4)));
};

// ------------------------------------------------------------------ core --

template <int BM_, int BN_, int WM_, int WN_, int ST_, bool F16_>
struct Tile {
  static constexpr bool F16 = F16_;
  typedef f32x16 AccBlock;
  static constexpr int BM = BM_, BN = BN_, BK = 64, STAGES = ST_;
  static constexpr int WAVES_M = WM_, WAVES_N = WN_, NW = WM_ * WN_, NT = NW * 64;
  static constexpr int WTM = BM / WM_, WTN = BN / WN_, FM = WTM / 32, FN = WTN / 32;
  static constexpr int STAGE_BYTES = (BM + BN) * 128;
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr int EPI = NW * 32 * WTM * 4;
  static constexpr int LDS = RING > EPI ? RING : EPI;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole loads per wave");
};

struct TileParams {
  const void *A, *B;
  int64_t lda, ldb;          // elements
  int64_t M, N, K;           // K a multiple of 8
  int64_t k_per_split;       // multiple of 64
  uint32_t tiles_m, tiles_n; // of one split
  uint32_t blocks;           // tiles x splits
};

// ROWS rows of one operand.
template <class T, int ROWS>
struct TileOperand {
  static constexpr int INSTR = ROWS / 8 / T::NW;    // 1 KB loads per wave and stage
  __amdgpu_buffer_rsrc_t rs;
  uint32_t voff[INSTR];      // byte offset of this lane's chunk at k = 0
  int kc[INSTR];             // its k within a stage

  __device__ inline void init(const void *p, int64_t ld, int64_t row0, int64_t rows, int wave,
                              int lane) {
    const uint16_t *base = static_cast<const uint16_t *>(p) + row0 * ld;
    rs = make_rsrc(base, (rows - row0) * ld * 2);
#pragma unroll
    for (int i = 0; i < INSTR; ++i) {
      const int r = (wave * INSTR + i) * 8 + lane / 8;
      kc[i] = ((lane & 7) ^ kswz<128>(r)) * 8;
      voff[i] = uint32_t(r) * uint32_t(ld * 2) + uint32_t(kc[i] * 2);
    }
  }
  template <bool TAIL>
  __device__ inline void issue(int64_t k0, int64_t k_end, char *dst, int wave) const {
#pragma unroll
    for (int i = 0; i < INSTR; ++i) {
      uint32_t off = voff[i] + uint32_t(k0 * 2);
      if (TAIL && k0 + kc[i] >= k_end) off = 0x80000000u;     // behind the end: zero
      dma16<0>(rs, dst + (wave * INSTR + i) * 1024, off);
    }
  }
  static __device__ inline u32x4 frag(const char *src, int base, int kk, int lane) {
    const int r = base + (lane & 31), c = kk * 2 + (lane >> 5);
    return *reinterpret_cast<const u32x4 *>(src + r * 128 + ((c ^ kswz<128>(r)) << 4));
  }
};

// Tiles run in groups of kGroupM rows of tiles, column by column: the tiles
// that an XCD works on at a time (neighbours in this order) form a patch that
// shares operand rows in its L2, where a plain row-by-row order reads one
// operand once per tile.
constexpr uint32_t kGroupM = 4;
__device__ inline void tile_at(uint32_t L, uint32_t tiles_m, uint32_t tiles_n, uint32_t &m,
                               uint32_t &n) {
  const uint32_t per_group = kGroupM * tiles_n, g = L / per_group, r = L - g * per_group;
  const uint32_t first = g * kGroupM;
  const uint32_t rows = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
  n = r / rows;
  m = first + (r - n * rows);
}
// xcd_remap for grids below 2^32 (a 64-bit division costs a small kernel a
// good part of its time).
__device__ inline uint32_t xcd_order(uint32_t b, uint32_t nb) {
  const uint32_t xcd = b % 8, idx = b / 8, q = nb / 8, r = nb % 8;
  return xcd < r ? xcd * (q + 1) + idx : r * (q + 1) + (xcd - r) * q + idx;
}

// The 256 x 256 core in that order; workgroup `bid` of `blocks`.
template <class CFG, class TR, bool AK, bool BKM, class Epi>
__device__ __forceinline__ void big_block(const Gemm2Params &g, const Epi &epi, uint32_t bid,
                                          uint32_t blocks, char *smem) {
  const uint32_t LS = xcd_order(bid, blocks);
  const uint32_t tiles_m = uint32_t((g.M + CFG::BM - 1) / CFG::BM), tiles_n = uint32_t(g.tiles_n);
  const uint32_t tiles = tiles_m * tiles_n, split = LS / tiles;
  uint32_t m, n;
  tile_at(LS - split * tiles, tiles_m, tiles_n, m, n);
  gemm2_tile<CFG, TR, AK, BKM, Epi>(g, epi, int64_t(split * tiles + m * tiles_n + n), smem);
}
template <class CFG, class TR, bool AK, bool BKM, class Epi>
__global__ void __launch_bounds__(TR::NT) big_kernel(Gemm2Params g, Epi epi) {
  __shared__ __attribute__((aligned(1024))) char smem[gemm2_lds_bytes<CFG, Epi>()];
  big_block<CFG, TR, AK, BKM, Epi>(g, epi, blockIdx.x, gridDim.x, smem);
}

// One tile of one split; `bid` of `blocks` workgroups.
template <class T, class Epi>
__device__ __forceinline__ void tile_block(const TileParams &g, const Epi &epi, uint32_t bid,
                                           char *smem) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const uint32_t tiles = g.tiles_m * g.tiles_n, split = bid / tiles;
  uint32_t tm, tn;
  tile_at(bid - split * tiles, g.tiles_m, g.tiles_n, tm, tn);
  const int64_t m0 = int64_t(tm) * T::BM, n0 = int64_t(tn) * T::BN;
  const int64_t kb = split * g.k_per_split;
  const int64_t ke = kb + g.k_per_split < g.K ? kb + g.k_per_split : g.K;
  const int n_k = ke > kb ? int((ke - kb + 63) / 64) : 0;

  TileOperand<T, T::BM> oa;
  TileOperand<T, T::BN> ob;
  oa.init(g.A, g.lda, m0, g.M, wave, lane);
  ob.init(g.B, g.ldb, n0, g.N, wave, lane);
  constexpr int LPS = TileOperand<T, T::BM>::INSTR + TileOperand<T, T::BN>::INSTR;
  auto issue = [&](int s) {
    char *st = smem + (s % T::STAGES) * T::STAGE_BYTES;
    const int64_t k0 = kb + int64_t(s) * 64;
    if (k0 + 64 <= ke) {
      oa.template issue<false>(k0, ke, st, wave);
      ob.template issue<false>(k0, ke, st + T::BM * 128, wave);
    } else {
      oa.template issue<true>(k0, ke, st, wave);
      ob.template issue<true>(k0, ke, st + T::BM * 128, wave);
    }
  };

  f32x16 acc[T::FM][T::FN];
#pragma unroll
  for (int a = 0; a < T::FM; ++a)
#pragma unroll
    for (int b = 0; b < T::FN; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

#pragma unroll
  for (int s = 0; s < T::STAGES - 1; ++s)
    if (s < n_k) issue(s);
  for (int it = 0; it < n_k; ++it) {
    // stage `it` has landed everywhere, and every wave is done with stage it - 1
    wait_vm_barrier_stages<LPS, T::STAGES - 2>(n_k - 1 - it);
    if (it + T::STAGES - 1 < n_k) issue(it + T::STAGES - 1);
    const char *sa = smem + (it % T::STAGES) * T::STAGE_BYTES, *sb = sa + T::BM * 128;
    // The reads of the whole stage go out together: with one wave a SIMD each
    // substep would otherwise wait for its own.
    u32x4 fa[4][T::FM], fb[4][T::FN];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int a = 0; a < T::FM; ++a)
        fa[kk][a] = TileOperand<T, T::BM>::frag(sa, wm * T::WTM + a * 32, kk, lane);
#pragma unroll
      for (int b = 0; b < T::FN; ++b)
        fb[kk][b] = TileOperand<T, T::BN>::frag(sb, wn * T::WTN + b * 32, kk, lane);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int a = 0; a < T::FM; ++a)
#pragma unroll
        for (int b = 0; b < T::FN; ++b) acc[a][b] = mfma32<T>(fa[kk][a], fb[kk][b], acc[a][b]);
    __builtin_amdgcn_sched_group_barrier(0x100, 4 * (T::FM + T::FN), 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 4 * T::FM * T::FN, 0);
  }
  __syncthreads();     // the ring becomes the epilogue's staging space
  epi.staged(acc, m0, n0, wm, wn, lane, int(split), smem, nullptr);
}

template <class T, class Epi>
__global__ void __launch_bounds__(T::NT) tile_kernel(TileParams g, Epi epi) {
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
  tile_block<T>(g, epi, xcd_order(blockIdx.x, g.blocks), smem);
}

// The same tile of operands at any alignment: vector loads to registers, two
// or four stages ahead, and from there to LDS (the DMA needs aligned rows, so
// it would take a padded copy of both operands first).  Vector loads off a
// 16-byte boundary cost it: 777 x K -> 1531 takes 10.2 us at K = 1008 on the
// DMA tiles, here 13.9 at 1002 and 16.6 at 1003.  Whole words and a shift took
// longer (515 x 1003 -> 777: 15.1 us against 11.7).
template <class T, int ROWS>
struct AnyOperand {
  static constexpr int N = ROWS * 8 / T::NT;      // 16-byte chunks per thread
  const uint16_t *p[N];
  int at[N], kc[N];
  __device__ inline void init(const void *base, int64_t ld, int64_t row0, int64_t rows, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * T::NT, r = u >> 3, c = u & 7;
      const int64_t row = row0 + r < rows ? row0 + r : rows - 1;   // rows behind the last: unused
      p[i] = static_cast<const uint16_t *>(base) + row * ld + c * 8;
      kc[i] = c * 8;
      at[i] = r * 128 + ((c ^ kswz<128>(r)) << 4);
    }
  }
  __device__ inline void load(int64_t k0, int64_t k_end, u32x4 (&reg)[N]) const {
    if (k0 + 64 <= k_end) {
#pragma unroll
      for (int i = 0; i < N; ++i) reg[i] = load16(p[i] + k0);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t left = k_end - k0 - kc[i];
        u32x4 v = {0, 0, 0, 0};
        if (left >= 8) {
          v = load16(p[i] + k0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) v[e >> 1] |= uint32_t(p[i][k0 + e]) << (16 * (e & 1));
        }
        reg[i] = v;
      }
    }
  }
  __device__ inline void store(const u32x4 (&reg)[N], char *dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(dst + at[i]) = reg[i];
  }
};

template <class T, class Epi>
__global__ void __launch_bounds__(T::NT) any_tile_kernel(TileParams g, Epi epi) {
  // stages in flight, as far as 64 registers hold them
  constexpr int DEPTH = (T::BM + T::BN) * 8 / T::NT <= 4 ? 4 : 2;
  constexpr int RING = 2 * T::STAGE_BYTES;
  __shared__ __attribute__((aligned(1024))) char smem[RING > T::EPI ? RING : T::EPI];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const uint32_t bid = xcd_order(blockIdx.x, g.blocks);
  const uint32_t tiles = g.tiles_m * g.tiles_n, split = bid / tiles;
  uint32_t tm, tn;
  tile_at(bid - split * tiles, g.tiles_m, g.tiles_n, tm, tn);
  const int64_t m0 = int64_t(tm) * T::BM, n0 = int64_t(tn) * T::BN;
  const int64_t kb = split * g.k_per_split;
  const int64_t ke = kb + g.k_per_split < g.K ? kb + g.k_per_split : g.K;
  const int n_k = ke > kb ? int((ke - kb + 63) / 64) : 0;

  AnyOperand<T, T::BM> oa;
  AnyOperand<T, T::BN> ob;
  oa.init(g.A, g.lda, m0, g.M, tid);
  ob.init(g.B, g.ldb, n0, g.N, tid);
  u32x4 ra[DEPTH][AnyOperand<T, T::BM>::N], rb[DEPTH][AnyOperand<T, T::BN>::N];
  f32x16 acc[T::FM][T::FN];
#pragma unroll
  for (int a = 0; a < T::FM; ++a)
#pragma unroll
    for (int b = 0; b < T::FN; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
    if (s < n_k) {
      oa.load(kb + s * 64, ke, ra[s]);
      ob.load(kb + s * 64, ke, rb[s]);
    }
  for (int it0 = 0; it0 < n_k; it0 += DEPTH) {
#pragma unroll
    for (int h = 0; h < DEPTH; ++h) {
      const int it = it0 + h;
      if (it < n_k) {                                   // uniform
        char *sa = smem + (h & 1) * T::STAGE_BYTES, *sb = sa + T::BM * 128;
        // (stage it - 2, in this buffer, was read before the last barrier)
        oa.store(ra[h], sa);
        ob.store(rb[h], sb);
        __syncthreads();
        if (it + DEPTH < n_k) {
          oa.load(kb + int64_t(it + DEPTH) * 64, ke, ra[h]);
          ob.load(kb + int64_t(it + DEPTH) * 64, ke, rb[h]);
        }
        u32x4 fa[4][T::FM], fb[4][T::FN];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
          for (int a = 0; a < T::FM; ++a)
            fa[kk][a] = TileOperand<T, T::BM>::frag(sa, wm * T::WTM + a * 32, kk, lane);
#pragma unroll
          for (int b = 0; b < T::FN; ++b)
            fb[kk][b] = TileOperand<T, T::BN>::frag(sb, wn * T::WTN + b * 32, kk, lane);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int a = 0; a < T::FM; ++a)
#pragma unroll
            for (int b = 0; b < T::FN; ++b) acc[a][b] = mfma32<T>(fa[kk][a], fb[kk][b], acc[a][b]);
      }
    }
  }
  __syncthreads();
  epi.staged(acc, m0, n0, wm, wn, lane, int(split), smem, nullptr);
}

}  // namespace lce
