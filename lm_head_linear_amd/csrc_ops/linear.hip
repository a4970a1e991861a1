// linear.hip -- Y = act(X W^T + b) + R and its backward, 16-bit operands with
// fp32 sums on the matrix cores.
//
// Every product is computed as C[m][c] with m the contiguous index of the
// result's rows and c its row, so that a lane's four consecutive accumulators
// are four consecutive elements in memory:
//   forward   Y[t][o]   : m = o (W, K-major),  c = t (X, K-major),  depth d_in
//   d_x       dX[t][i]  : m = i (W^T copy),    c = t (G, K-major),  depth d_out
//   d_weight  dW[o][i]  : m = i (X, MN-major), c = o (G, MN-major), depth n
//                         (small tiles: X^T and G^T copies, K-major)
// with G = dY * act'(Z), rounded to the 16-bit type once (it feeds matrix
// instructions); the bias gradient sums the unrounded G, 64 tokens in fp32 and
// those sums in fp64.
//
// Up to 64 tokens run in few_tokens_kernel, which is bound by the read of W;
// more run on tiles in LDS: the 256 x 256 core of the losses where its tiles
// fill the chip, else smaller tiles, with the depth split over several tiles
// where there are few (plan_product).
//
// Measured (bf16, one box, us a call; a library product alone takes 212):
// 8192 x 4096 -> 4096 with bias, gelu, residual and pre-activation 259, 1.06
// PFLOP/s (255 to 266 from box to box): bound by the matrix cores (2 rounds of
// 64 steps of 1.59 us) and the epilogue's 201 MB, which all compute units move
// at the same time; its backward from 8-bit checkpoints 525 (511 to 531;
// traced: copies 81, products 509, medians of calls with gaps between them,
// which run slower than calls in a row).
#include <math.h>

#include <numeric>

#include "ops_gemm.hpp"

namespace lce {

// ------------------------------------------------------------- few tokens --

// Up to 64 tokens: the read of W bounds the call, so W goes straight from
// memory to the registers that feed the matrix instruction.  A wave owns 16
// rows of W and all tokens (16 T of them): per 32 k one 16-byte load a lane
// of W and T of X (the block's waves share X, which stays in L1), and T
// 16x16x32 products.  The loads of the next 128 k are in flight while the
// current ones are used.  Where d_out is small, KW waves of a block share 16
// rows, each a range of k, and their sums meet in LDS.  No alignment is asked
// for: vector loads take any address.
// Measured, W not in a cache: one token 1024 x 1024 4.4 us (a launch), 4096 x
// 4096 9.9 us (3.4 TB/s), 32768 x 4096 46 us (5.8 TB/s).  More tokens read more of X beside W (32768 x 4096,
// one W over and over: 93 us with 32 tokens, 146 with 64, against 53 and 55 in
// tiles), so large heads go to tiles: 151936 x 1024, 32 tokens, 60 us (5.2
// TB/s) against 111.
typedef float f32x4v __attribute__((ext_vector_type(4)));
template <bool F16>
__device__ inline f32x4v mfma16(u32x4 a, u32x4 b, f32x4v c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight values at p + k, zero from k_end on.
__device__ inline u32x4 load_k8(const uint16_t *p, int64_t k, int64_t k_end) {
  if (k + 8 <= k_end) return load16(p + k);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < k_end) v[i >> 1] |= uint32_t(p[k + i]) << (16 * (i & 1));
  return v;
}

template <bool F16, int T>
__global__ void __launch_bounds__(512) few_tokens_kernel(const uint16_t *x, const uint16_t *w,
                                                         int n, int64_t d_in, int64_t d_out,
                                                         int kw, int64_t k_part, OutParams out) {
  constexpr int U = 4;                   // loads of W in flight: 32 k each
  __shared__ f32x4v s_part[8 * T * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_block = int(blockDim.x >> 6) / kw;
  const int part = wave % kw;
  const int64_t group = int64_t(blockIdx.x) * per_block + wave / kw;
  const int64_t f0 = group * 16;
  const int r = lane & 15, kq = (lane >> 4) * 8;
  const int64_t feature = f0 + r < d_out ? f0 + r : d_out - 1;   // rows behind the last: unused
  const uint16_t *pw = w + feature * d_in + kq;
  const uint16_t *px[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int tok = t * 16 + r < n ? t * 16 + r : n - 1;
    px[t] = x + int64_t(tok) * d_in + kq;
  }
  f32x4v acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f32x4v{0, 0, 0, 0};

  const int64_t k0 = part * k_part, k1 = k0 + k_part < d_in ? k0 + k_part : d_in;
  const int64_t full = k1 > k0 ? (k1 - k0) / (32 * U) : 0;       // whole batches
  u32x4 cw[U], cx[U][T];
  auto load = [&](int64_t k, u32x4 (&a)[U], u32x4 (&b)[U][T]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u] = load16(pw + k + 32 * u);
#pragma unroll
      for (int t = 0; t < T; ++t) b[u][t] = load16(px[t] + k + 32 * u);
    }
  };
  auto use = [&](const u32x4 (&a)[U], const u32x4 (&b)[U][T]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[t] = mfma16<F16>(a[u], b[u][t], acc[t]);
  };
  if (full > 0) load(k0, cw, cx);
  for (int64_t i = 1; i < full; ++i) {
    u32x4 nw[U], nx[U][T];
    load(k0 + i * (32 * U), nw, nx);
    use(cw, cx);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      cw[u] = nw[u];
#pragma unroll
      for (int t = 0; t < T; ++t) cx[u][t] = nx[u][t];
    }
  }
  if (full > 0) use(cw, cx);
  for (int64_t k = k0 + full * (32 * U); k < k1; k += 32) {
    const u32x4 a = load_k8(pw, k, k1 - kq);
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = mfma16<F16>(a, load_k8(px[t], k, k1 - kq), acc[t]);
  }

  auto store = [&](int t, f32x4v v) {
    // lane: token t*16 + (lane & 15), features f0 + 4 (lane >> 4) .. + 3
    const int64_t m = f0 + (lane >> 4) * 4, c = t * 16 + r;
    const int count = m >= d_out ? 0 : (d_out - m >= 4 ? 4 : int(d_out - m));
    if (c >= n || count == 0) return;
    float z[4] = {v[0], v[1], v[2], v[3]}, b[4];
    load_bias<F16, 4>(out, m, count, b);
    finish<F16, 4>(out, z, b, m, c, count, 0);
  };
  if (kw == 1) {
#pragma unroll
    for (int t = 0; t < T; ++t) store(t, acc[t]);
    return;
  }
#pragma unroll
  for (int t = 0; t < T; ++t) s_part[(wave * T + t) * 64 + lane] = acc[t];
  __syncthreads();
  for (int t = part; t < T; t += kw) {
    const int first = wave - part;
    f32x4v v = s_part[(first * T + t) * 64 + lane];
    for (int q = 1; q < kw; ++q) v += s_part[((first + q) * T + t) * 64 + lane];
    store(t, v);
  }
}

// ---------------------------------------------------------- prepared copies --

// Operands as the tiled cores take them, from any alignment: one launch fills
// all copies a call needs.  A block turns a 64 x 64 tile of a [rows][cols]
// matrix into the padded row-major copy (columns behind the last are zero up
// to ld) and / or the padded transposed one, multiplying by the activation's
// slope and summing columns on the way where asked.
// Bound by memory and by the arithmetic of gelu's slope together: 8192 x 4096
// from 8-bit checkpoints with W's transposed copy, 337 MB, 81 us (4.2 TB/s; 73
// at best); one job after the other 92, and 64 x 256 tiles 96.
struct CopyJob {
  const void *src;          // [rows][cols], 16-bit, or e4m3 codes with scales
  const uint8_t *scales;
  const void *z;            // multiply by act'(z), null: do not
  const uint8_t *z_scales;
  int64_t rows, cols;
  uint16_t *dst;            // [rows][ld], null: none
  int64_t ld;
  uint16_t *dst_t;          // [cols][ld_t], null: none
  int64_t ld_t;
  float *sums;              // [tile rows][cols] sums over 64 rows, null: none
  uint32_t tiles_c, tiles;
  int32_t act;
};
constexpr int kMaxCopies = 3;
constexpr uint32_t kCopyRun = 64;
struct CopyJobs {
  CopyJob job[kMaxCopies];
  uint32_t stride;          // of the runs' order, prime to their number; 1: as they come
};

// Eight saved values from column c of a row on, `count` of them: as they lie
// in memory (loads of several may be in flight), then as fp32.
struct Raw8 {
  u32x4 v;
  int scale;
};
__device__ inline Raw8 load_saved(const void *v, const uint8_t *scales, int64_t row, int64_t cols,
                                  int64_t c, int count) {
  Raw8 r = {u32x4{0, 0, 0, 0}, 127};
  if (!scales) {
    const uint16_t *p = static_cast<const uint16_t *>(v) + row * cols + c;
    if (count == 8) {
      r.v = load16(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < count) r.v[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
    }
    return r;
  }
  const uint8_t *p = static_cast<const uint8_t *>(v) + row * cols + c;
  // (eight columns from a multiple of 8 on share a block of 32)
  r.scale = scales[row * ((cols + 31) / 32) + c / 32];
  if (count == 8) {
    const AnyVec8 q = *reinterpret_cast<const AnyVec8 *>(p);
    r.v[0] = q.v[0];
    r.v[1] = q.v[1];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) r.v[i >> 2] |= uint32_t(p[i]) << (8 * (i & 3));
  }
  return r;
}
template <bool F16>
__device__ inline void saved_values(const Raw8 &r, bool codes, float (&f)[8]) {
  if (!codes) {
    widen8<F16>(r.v, f);
    return;
  }
  codes_to_f32(r.v[0], r.v[1], r.scale - 127, f);
  // exact in the 16-bit type but where the largest codes pass its range
  if (r.scale >= 127 + (F16 ? 8 : 119) || r.scale < 127 + (F16 ? -15 : -117)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = widen<F16>(saturate16<F16>(f[i]));
  }
}

template <bool F16>
__global__ void __launch_bounds__(256) copies_kernel(CopyJobs jobs) {
  __shared__ uint32_t s_t[64 * 33];
  __shared__ float s_sum[4 * 64];
  // The jobs' blocks are mixed (some compute much, some move much), in runs of
  // kCopyRun neighbours of a job.
  const uint32_t runs = gridDim.x / kCopyRun;
  uint32_t b = blockIdx.x;
  if (jobs.stride > 1 && b < runs * kCopyRun) {
    const uint32_t run = b / kCopyRun;
    b = uint32_t(uint64_t(run) * jobs.stride % runs) * kCopyRun + b % kCopyRun;
  }
  int which = 0;
  while (which + 1 < kMaxCopies && b >= jobs.job[which].tiles) b -= jobs.job[which++].tiles;
  const CopyJob &j = jobs.job[which];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t tile_row = b / j.tiles_c;
  const int64_t tr = tile_row, r0 = tr * 64, c0 = int64_t(b - tile_row * j.tiles_c) * 64;
  const int cc = tid & 7, pair = tid >> 3;           // 8 columns, rows 2 pair and 2 pair + 1
  const int64_t c = c0 + cc * 8;
  const int count = c >= j.cols ? 0 : (j.cols - c >= 8 ? 8 : int(j.cols - c));
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  u32x4 v[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  Raw8 x[2] = {}, z[2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {           // all loads before the first use
    const int64_t row = r0 + 2 * pair + h;
    if (row < j.rows && count > 0) {
      x[h] = load_saved(j.src, j.scales, row, j.cols, c, count);
      if (j.z) z[h] = load_saved(j.z, j.z_scales, row, j.cols, c, count);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + 2 * pair + h;
    if (!j.z && !j.sums && !j.scales) {
      v[h] = x[h].v;                      // moved as it is
    } else if (row < j.rows && count > 0) {
      float f[8];
      saved_values<F16>(x[h], j.scales != nullptr, f);
      if (j.z) {
        float g[8];
        saved_values<F16>(z[h], j.z_scales != nullptr, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= act_slope(g[i], j.act);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= count) f[i] = 0.0f;
        sum[i] += f[i];
      }
      v[h] = narrow8<F16>(f);
    }
    if (j.dst && row < j.rows && c < j.ld)
      *reinterpret_cast<u32x4 *>(j.dst + row * j.ld + c) = v[h];
  }
  if (j.dst_t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = (v[0][i >> 1] >> (16 * (i & 1))) & 0xffffu;
      const uint32_t hi = (v[1][i >> 1] >> (16 * (i & 1))) & 0xffffu;
      s_t[(cc * 8 + i) * 33 + pair] = lo | (hi << 16);
    }
  }
  if (j.sums) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = 8; o < 64; o <<= 1) sum[i] += __shfl_xor(sum[i], o);
      if (lane < 8) s_sum[wave * 64 + cc * 8 + i] = sum[i];
    }
  }
  if (!j.dst_t && !j.sums) return;      // block-uniform
  __syncthreads();
  if (j.sums && tid < 64 && c0 + tid < j.cols)
    j.sums[tr * j.cols + c0 + tid] =
        ((s_sum[tid] + s_sum[64 + tid]) + s_sum[128 + tid]) + s_sum[192 + tid];
  if (j.dst_t) {
    const int col = tid >> 2, q = tid & 3;
    const int64_t t0 = r0 + q * 16;
    if (c0 + col < j.cols && t0 < j.ld_t) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = s_t[col * 33 + q * 8 + i];
      u32x4 *d = reinterpret_cast<u32x4 *>(j.dst_t + (c0 + col) * j.ld_t + t0);
      d[0] = u32x4{w[0], w[1], w[2], w[3]};
      d[1] = u32x4{w[4], w[5], w[6], w[7]};
    }
  }
}

// Adds the bias gradient's 64-row sums in fp64, as every sum over tokens (fp32
// drops what is below 2^-24 of the sum so far, and there may be 2^18 of them):
// 64 columns a block, a quarter of the rows a wave, each in order.
struct BiasGrad {
  const float *sums;       // [parts][d]
  int64_t parts, d;
  void *out;
  int32_t out_f32, add;
};
template <bool F16>
__device__ inline void bias_grad_block(const BiasGrad &a, uint32_t bid, double *s_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = int64_t(bid) * 64 + lane;
  const int64_t per = (a.parts + 3) / 4, begin = wave * per;
  const int64_t end = begin + per < a.parts ? begin + per : a.parts;
  if (wave < 4) {
    double s = 0.0;
    if (col < a.d) {
#pragma unroll 8
      for (int64_t i = begin; i < end; ++i) s += a.sums[i * a.d + col];
    }
    s_sum[wave * 64 + lane] = s;
  }
  __syncthreads();
  if (wave != 0 || col >= a.d) return;
  const float s = float(((s_sum[lane] + s_sum[64 + lane]) + s_sum[128 + lane]) + s_sum[192 + lane]);
  if (a.out_f32) {
    float *o = static_cast<float *>(a.out) + col;
    *o = a.add ? *o + s : s;
  } else {
    uint16_t *o = static_cast<uint16_t *>(a.out) + col;
    *o = narrow<F16>(a.add ? widen<F16>(*o) + s : s);
  }
}
template <bool F16>
__global__ void __launch_bounds__(256) bias_grad_kernel(BiasGrad a) {
  __shared__ double s_sum[256];
  bias_grad_block<F16>(a, blockIdx.x, s_sum);
}

// The small backward in one launch: two products on the same tiles and the
// bias gradient's sums, which need nothing of each other (515 x 1003 -> 777: the
// call took 26.3 us with a launch each, 19.4 with one and 32-bit tile numbers).
// Bound by the latency of the tiles' steps, about 0.3 us each.
template <class T>
__global__ void __launch_bounds__(T::NT) backward_kernel(TileParams g0, OutEpi<T> e0, TileParams g1,
                                                         OutEpi<T> e1, BiasGrad bias) {
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
  uint32_t b = blockIdx.x;
  if (b < g0.blocks) {
    tile_block<T>(g0, e0, xcd_order(b, g0.blocks), smem);
    return;
  }
  b -= g0.blocks;
  if (b < g1.blocks) {
    tile_block<T>(g1, e1, xcd_order(b, g1.blocks), smem);
    return;
  }
  bias_grad_block<T::F16>(bias, b - g1.blocks, reinterpret_cast<double *>(smem));
}

// The large backward in one launch: d_weight's tiles (operands as they lie),
// d_x's (K-major) and the bias gradient's sums.  One product's tail and its
// stores run beside the other's tiles (8192 x 4096 x 4096: 537 us for the call,
// 549 with three launches on the same box).
template <bool F16>
__global__ void __launch_bounds__(TraitsH16W8<F16>::NT) big_backward_kernel(
    Gemm2Params gw, OutEpi<TraitsH16W8<F16>> ew, uint32_t blocks_w, Gemm2Params gx,
    OutEpi<TraitsH16W8<F16>> ex, uint32_t blocks_x, BiasGrad bias) {
  typedef TraitsH16W8<F16> TR;
  typedef PipeCfg<64, 2> CFG;
  __shared__ __attribute__((aligned(1024))) char smem[gemm2_lds_bytes<CFG, OutEpi<TR>>()];
  const uint32_t b = blockIdx.x;
  if (b < blocks_w)
    big_block<CFG, TR, false, false, OutEpi<TR>>(gw, ew, b, blocks_w, smem);
  else if (b - blocks_w < blocks_x)
    big_block<CFG, TR, true, true, OutEpi<TR>>(gx, ex, b - blocks_w, blocks_x, smem);
  else
    bias_grad_block<F16>(bias, b - blocks_w - blocks_x, reinterpret_cast<double *>(smem));
}

// Adds the K-splits ([split][cols][ld] fp32) of one or two products in order
// and finishes.  Its cost is a launch and the partial results' read (fold_us).
struct FoldJob {
  const float *part;
  int64_t ld, stride;
  int32_t splits;
  uint32_t blocks;       // 0: nothing to fold
  OutParams out;
};
template <bool F16>
__device__ __forceinline__ void fold_block(const FoldJob &j, uint32_t bid) {
  const int64_t per_row = j.ld / 8, total = per_row * j.out.cols;
  for (int64_t u = int64_t(bid) * 256 + threadIdx.x; u < total; u += int64_t(j.blocks) * 256) {
    const int64_t c = u / per_row, m = (u - c * per_row) * 8;
    const int count = j.out.rows - m >= 8 ? 8 : int(j.out.rows - m);
    float z[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8];
    const float *p = j.part + c * j.ld + m;
#pragma unroll 4
    for (int s = 0; s < j.splits; ++s) {
      const u32x4 x = *reinterpret_cast<const u32x4 *>(p + s * j.stride);
      const u32x4 y = *reinterpret_cast<const u32x4 *>(p + s * j.stride + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[i] += __uint_as_float(x[i]);
        z[4 + i] += __uint_as_float(y[i]);
      }
    }
    load_bias<F16, 8>(j.out, m, count, b);
    finish<F16, 8>(j.out, z, b, m, c, count, 0);
  }
}
template <bool F16>
__global__ void __launch_bounds__(256) fold_kernel(FoldJob a, FoldJob b) {
  if (blockIdx.x < a.blocks) fold_block<F16>(a, blockIdx.x);
  else fold_block<F16>(b, blockIdx.x - a.blocks);
}

// ------------------------------------------------------------------- host --

constexpr int64_t kFewTokens = 64;

// How one product C[m][c], m < M, c < N, depth K runs.
enum Core {
  kGeneric,    // register-staged tiles of the losses: any alignment
  kFew,        // few_tokens_kernel
  k128x32, k64x64, k128x64, k128x128, k256x256
};
struct ProductPlan {
  Core core = kGeneric;
  int64_t splits = 1, k_per_split = 0;
  size_t part_bytes = 0;    // fp32 partial results of the splits
  double us = 0.0;          // modelled
};

static size_t partial_bytes(int64_t M, int64_t N, int64_t splits) {
  return splits > 1 ? size_t(splits * N * round_to(M, 8)) * 4 : 0;
}

struct Operand {
  const void *p;
  int64_t ld;
};

static int64_t tile_count(int64_t M, int64_t N, int64_t bm, int64_t bn) {
  return ceil_div(M, bm) * ceil_div(N, bn);
}

// Measured on the products alone (M 1024 to 151936, N 32 to 8192, K 512 to
// 4096, bf16): microseconds of a 64-deep step of one tile alone on a compute
// unit and with a second one beside it, and what a round of tiles costs
// besides its steps.  For example 4096 x 2048 x 1024: 36 us with 64 x 64
// tiles, 27 with 128 x 64, 23 with 128 x 128, 31 with 256 x 256; 1024 x 512 x
// 1024: 8.5, 10.6, 12.0, 27; 4096 x 4096 x 4096: 231, 167, 133, 109.
struct TileCost {
  Core core;
  int64_t bm, bn;
  double step_alone, step_shared, round;
  int64_t at_once;          // tiles the chip runs at a time
};
static const TileCost kTiles[] = {
    {k128x32, 128, 32, 0.28, 0.30, 1.5, 512},   {k64x64, 64, 64, 0.34, 0.41, 2.8, 512},
    {k128x64, 128, 64, 0.41, 0.62, 3.2, 512},   {k128x128, 128, 128, 0.64, 1.05, 2.5, 512},
    {k256x256, 256, 256, 1.59, 1.59, 8.0, 256},
};
constexpr double kBytesPerUs = 5.0e6;    // what a large copy moves

constexpr int64_t kMostSplits = 32;

// Microseconds that a product's K-splits add: a launch, and the partial
// results written and read.
static double fold_us(int64_t M, int64_t N, int64_t splits) {
  return splits > 1 ? 3.0 + double(splits) * double(M) * double(N) * 8.0 / kBytesPerUs : 0.0;
}

static ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool few) {
  ProductPlan best;
  double best_us = 1e30;
  int64_t best_tiles = 0;
  const int64_t steps = ceil_div(K, 64);
  const double memory_us = 2.0 * double(K) * double(M + N) / kBytesPerUs;
  for (const TileCost &t : kTiles) {
    if (t.core == k128x32 && N > 32) continue;
    const int64_t tiles = tile_count(M, N, t.bm, t.bn);
    for (int64_t sp = 1; sp <= kMostSplits && sp <= steps; sp *= 2) {
      const int64_t per = ceil_div(steps, sp);
      if ((sp - 1) * per >= steps) continue;
      const int64_t all = tiles * sp, last = all % t.at_once;
      double us = double(all / t.at_once) * (t.round + double(per) * t.step_shared);
      if (last)
        us += t.round + double(per) * (last <= kComputeUnits ? t.step_alone : t.step_shared);
      if (us < memory_us) us = memory_us;
      us += fold_us(M, N, sp);
      if (us < best_us) {
        best_us = us;
        best.core = t.core;
        best.splits = sp;
        best_tiles = all;
        best.k_per_split = per * 64;
      }
    }
  }
  best.part_bytes = partial_bytes(M, N, best.splits);
  best.us = best_us;
  // Up to 64 rows may stream A instead, with no ring to fill first: bound by the
  // read of A, at a rate that falls with the rows that share a wave.  Up to 16
  // rows both sides are lines measured with A not in a cache, where a step of
  // tiles that do not fill the chip takes 0.5 us: 32768 x 4096 takes 46, 54 and
  // 67 us with 1, 8 and 16 tokens (tiles 59 with each), 151936 x 1024 50, 63 and
  // 75 (tiles 52, 55, 57).  Fitted over 17 layers, and checked on nine others
  // with 1 to 14 tokens: 0.3 % over the better side on average, where 4.8 TB/s
  // for all and warm tile steps cost 2.3 %.  Beyond 16: 2.9 and 1.9 TB/s for up
  // to 32 and 64 rows, from one A read over and over.
  if (few && N <= 16) {
    const double cold_us = 1.5 + 0.5 * double(best.k_per_split / 64) + (best.splits > 1 ? 3.0 : 0.0);
    if (best_tiles <= kComputeUnits && best_us < cold_us) best_us = cold_us;
    const double us = 2.0 + 2.0e-6 * double(M) * double(K) * (0.165 + 0.007 * double(N - 1));
    if ((us > 4.8 ? us : 4.8) < best_us) {
      best = ProductPlan{};
      best.core = kFew;
    }
  } else if (few && N <= kFewTokens) {
    const double floor_us = N <= 32 ? 5.7 : 7.5, rate = N <= 32 ? 2.9e6 : 1.9e6;
    const double us = 2.0 + 2.0 * double(M) * double(K) / rate;
    if ((us > floor_us ? us : floor_us) < best_us + 2.5) {
      best = ProductPlan{};
      best.core = kFew;
    }
  }
  return best;
}

// The backward's two products (d_in x n over d_out, d_in x d_out over n) in
// one launch on one kind of tile, their splits folded by one more: taken when
// the model puts it ahead of separate launches (at about 2.5 us each).
static bool plan_joint(int64_t d_in, int64_t n, int64_t d_out, ProductPlan *px, ProductPlan *pw) {
  double best = px->us + pw->us + 2.5;
  bool found = false;
  const int64_t steps_x = ceil_div(d_out, 64), steps_w = ceil_div(n, 64);
  for (const TileCost &t : kTiles) {
    if (t.core == k128x32 || t.core == k256x256) continue;
    const int64_t tx = tile_count(d_in, n, t.bm, t.bn), tw = tile_count(d_in, d_out, t.bm, t.bn);
    for (int64_t sx = 1; sx <= kMostSplits && sx <= steps_x; sx *= 2)
      for (int64_t sw = 1; sw <= kMostSplits && sw <= steps_w; sw *= 2) {
        const int64_t per_x = ceil_div(steps_x, sx), per_w = ceil_div(steps_w, sw);
        if ((sx - 1) * per_x >= steps_x || (sw - 1) * per_w >= steps_w) continue;
        const bool alone = tx * sx + tw * sw <= kComputeUnits;
        const double step = alone ? t.step_alone : t.step_shared;
        const double cost_x = t.round + double(per_x) * step, cost_w = t.round + double(per_w) * step;
        double us = (double(tx * sx) * cost_x + double(tw * sw) * cost_w) / double(t.at_once);
        const double longest = cost_x > cost_w ? cost_x : cost_w;
        if (us < longest) us = longest;
        us += fold_us(d_in, n, sx) + fold_us(d_in, d_out, sw) - (sx > 1 && sw > 1 ? 3.0 : 0.0);
        if (us < best) {
          best = us;
          found = true;
          *px = ProductPlan{t.core, sx, per_x * 64, partial_bytes(d_in, n, sx), us};
          *pw = ProductPlan{t.core, sw, per_w * 64, partial_bytes(d_in, d_out, sw), us};
        }
      }
  }
  return found;
}

// The register-staged core of the losses: any alignment, 64-bit offsets.
template <class TR>
struct DirectEpi {
  OutParams p;
  __device__ __forceinline__ void operator()(typename TR::AccBlock (&acc)[TR::FM][TR::FN],
                                             int64_t m0, int64_t n0, int wm, int wn, int lane,
                                             int) const {
    // (rolled loops with the block picked by selects: 16 copies of the
    // epilogue would not be unrolled and the accumulators would go to memory)
#pragma unroll 1
    for (int f = 0; f < TR::FM * TR::FN; ++f) {
      const int fm = f / TR::FN, fn = f % TR::FN;
      const int64_t c = n0 + wn * TR::WTN + fn * TR::MF + TR::col_of(lane);
      f32x16 blk = acc[0][0];
#pragma unroll
      for (int a = 0; a < TR::FM; ++a)
#pragma unroll
        for (int b = 0; b < TR::FN; ++b)
          if (a == fm && b == fn) blk = acc[a][b];
      if (c >= p.cols) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t m = m0 + wm * TR::WTM + fm * TR::MF + TR::row_of(4 * q, lane);
        const int count = m >= p.rows ? 0 : (p.rows - m >= 4 ? 4 : int(p.rows - m));
        float z[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = blk[4 * q + i];
        load_bias<TR::F16, 4>(p, m, count, b);
        if (count > 0) finish<TR::F16, 4>(p, z, b, m, c, count, 0);
      }
    }
  }
};
template <bool F16, bool AK, bool BKM>
static void run_generic(Operand A, Operand B, int64_t M, int64_t N, int64_t K,
                        const OutParams &out, hipStream_t st) {
  typedef TraitsH16<F16> TR;
  GemmParams g = {};
  g.A = A.p; g.lda = A.ld; g.B = B.p; g.ldb = B.ld;
  g.M = M; g.N = N; g.K = K;
  g.k_per_split = round_to(K, TR::BK);
  g.tiles_n = ceil_div(N, TR::BN);
  const uint32_t tiles = uint32_t(tile_count(M, N, TR::BM, TR::BN));
  gemm_kernel<TR, AK, BKM, false><<<tiles, TR::NT, 0, st>>>(g, DirectEpi<TR>{out});
}

// f(tile type) for one of the K-major tiles.
template <bool F16, class F>
static void with_tile(Core core, F &&f) {
  if (core == k128x32) f(Tile<128, 32, 4, 1, 4, F16>());
  else if (core == k64x64) f(Tile<64, 64, 2, 2, 4, F16>());
  else if (core == k128x64) f(Tile<128, 64, 2, 2, 3, F16>());
  else f(Tile<128, 128, 2, 4, 2, F16>());
}
template <class T>
static TileParams tile_params(const ProductPlan &pl, Operand A, Operand B, int64_t M, int64_t N,
                              int64_t K) {
  TileParams g = {};
  g.A = A.p; g.lda = A.ld; g.B = B.p; g.ldb = B.ld;
  g.M = M; g.N = N; g.K = K;
  g.k_per_split = pl.k_per_split;
  g.tiles_m = uint32_t(ceil_div(M, T::BM));
  g.tiles_n = uint32_t(ceil_div(N, T::BN));
  g.blocks = uint32_t(g.tiles_m * g.tiles_n * pl.splits);
  return g;
}

static Gemm2Params big_params(const ProductPlan &pl, Operand A, Operand B, int64_t M, int64_t N,
                              int64_t K) {
  Gemm2Params g = {};
  g.A = A.p; g.lda = A.ld; g.B = B.p; g.ldb = B.ld;
  g.M = M; g.N = N; g.K = K;
  g.M_read = A.ld; g.N_read = B.ld;
  g.k_per_split = pl.k_per_split;
  g.tiles_n = ceil_div(N, 256);
  return g;
}

// Where the tiles of a planned product write, and how its splits are folded.
static OutParams product_out(const ProductPlan &pl, int64_t M, int64_t N, const OutParams &out,
                             char *part) {
  if (pl.splits == 1) return out;
  OutParams o = {};
  o.out = part;
  o.ld = round_to(M, 8);
  o.rows = out.rows;
  o.cols = out.cols;
  o.out_f32 = 1;
  o.split_stride = N * o.ld;
  return o;
}
static FoldJob fold_job(const ProductPlan &pl, int64_t M, int64_t N, const OutParams &out,
                        const char *part) {
  FoldJob j = {};
  if (pl.splits == 1) return j;
  j.part = reinterpret_cast<const float *>(part);
  j.ld = round_to(M, 8);
  j.stride = N * j.ld;
  j.splits = int32_t(pl.splits);
  const int64_t blocks = ceil_div(j.ld / 8 * out.cols, 256);
  j.blocks = uint32_t(blocks < 4096 ? blocks : 4096);
  j.out = out;
  return j;
}
template <bool F16>
static void run_folds(const FoldJob &a, const FoldJob &b, hipStream_t st) {
  if (a.blocks + b.blocks) fold_kernel<F16><<<a.blocks + b.blocks, 256, 0, st>>>(a, b);
}

// Runs a planned product of padded, aligned operands.  AK, BKM: the operand
// is K-major (the small tiles take K-major ones only).
// `any`: K-major operands at any alignment (not for the 256 x 256 core).
template <bool F16, bool AK, bool BKM>
static void run_product(const ProductPlan &pl, Operand A, Operand B, int64_t M, int64_t N,
                        int64_t K, const OutParams &out, char *part, hipStream_t st,
                        bool any = false) {
  const OutParams o = product_out(pl, M, N, out, part);
  if (pl.core == kGeneric) {
    run_generic<F16, AK, BKM>(A, B, M, N, K, out, st);
  } else if (pl.core == k256x256) {
    typedef TraitsH16W8<F16> TR;
    typedef PipeCfg<64, 2> CFG;
    const Gemm2Params g = big_params(pl, A, B, M, N, K);
    const int64_t wgs = tile_count(M, N, 256, 256) * pl.splits;
    big_kernel<CFG, TR, AK, BKM, OutEpi<TR>><<<uint32_t(wgs), TR::NT, 0, st>>>(g, OutEpi<TR>{o});
  } else if constexpr (AK && BKM) {
    with_tile<F16>(pl.core, [&](auto tile) {
      typedef decltype(tile) T;
      const TileParams g = tile_params<T>(pl, A, B, M, N, K);
      if (any) any_tile_kernel<T><<<g.blocks, T::NT, 0, st>>>(g, OutEpi<T>{o});
      else tile_kernel<T><<<g.blocks, T::NT, 0, st>>>(g, OutEpi<T>{o});
    });
  }
  run_folds<F16>(fold_job(pl, M, N, out, part), FoldJob{}, st);
}

// The tiled cores address 256 rows of an operand with 32-bit byte offsets.
static bool offsets_fit(int64_t ld) { return 256 * ld * 2 < (int64_t(1) << 31); }

struct LinearPlan {
  ProductPlan product;
  int64_t ld_in = 0;                      // padded d_in of the copies, 0: no copies
  bool any = false;                       // rows that are not aligned are read as they lie
  size_t off_x = 0, off_w = 0, off_part = 0, total = 0;
};

struct BackwardPlan {
  ProductPlan px, pw;                     // d_x and d_weight
  bool joint = false;                     // both in one launch, on the same tiles
  bool mn_x = false, mn_w = false;        // operands as they lie, not transposed copies
  int64_t ld_in = 0, ld_out = 0, ld_n = 0;
  int64_t sum_parts = 0;
  size_t off_g = 0, off_gt = 0, off_x = 0, off_xt = 0, off_w = 0, off_wt = 0;
  size_t off_part = 0, off_part_w = 0, off_sums = 0, total = 0;
};

struct Layout {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t here = at;
    at += size_t(round_to(int64_t(bytes), 256));
    return here;
  }
};

static int32_t plan_linear(int64_t n, int64_t d_in, int64_t d_out, int32_t dtype, LinearPlan *p) {
  if (const int32_t st = lce_dims_check(n, d_in, d_out); st != LCE_OK) return st;
  if (!half_type(dtype)) return LCE_DTYPE_MISMATCH;
  Layout l;
  p->product = plan_product(d_out, n, d_in, true);
  // Odd rows of up to 64 tokens stream, whatever the layer's size.  That is the
  // faster side for small layers (1003 -> 1531: 6.9, 8.5, 10.8, 16.1 us with 1,
  // 16, 32, 64 tokens, tiles that read the rows as they lie 13.2, 12.6, 12.9,
  // 12.1; 515 -> 777: 6.8 to 9.0 against 8.7 to 10.1) and not for large ones,
  // weights not in a cache: 1003 -> 151936 105, 168, 254, 441 against 76, 78,
  // 82, 108, 4097 -> 4097 18, 40, 64, 113 against 21, 23, 24, 27.  Padded copies
  // take longer than those tiles everywhere.
  if (n <= kFewTokens && d_in % 8 != 0) p->product = ProductPlan{kFew};
  if (p->product.core == kFew) return LCE_OK;
  if (p->product.core == k256x256 ? d_in % 64 != 0 : d_in % 8 != 0) {
    // Odd rows: read as they lie, where a step of a tile costs more (vector
    // loads off a 16-byte boundary), or from padded copies (a launch, and both
    // operands read and written).  515 x 1003 -> 777 fp16: 11.7 us against
    // 13.3; 777 x 1003 -> 1531: 16.7 either way; larger ones gain from copies.
    for (const TileCost &t : kTiles) {
      if (t.core != p->product.core || t.core == k256x256) continue;
      const int64_t all = tile_count(d_out, n, t.bm, t.bn) * p->product.splits;
      const double rounds = double(ceil_div(all, t.at_once)) * (all <= kComputeUnits ? 1.0 : 2.0);
      const double slower = 0.1 * double(t.bm + t.bn) / 64.0 * rounds *
                            double(p->product.k_per_split / 64);
      p->any = slower < 4.0 + 4.0 * double(d_in) * double(n + d_out) / kBytesPerUs;
    }
  }
  if (!p->any && (p->product.core == k256x256 ? d_in % 64 != 0 : d_in % 8 != 0)) {
    p->ld_in = round_to(d_in, 64);
    p->off_x = l.take(size_t(n * p->ld_in * 2));
    p->off_w = l.take(size_t(d_out * p->ld_in * 2));
  }
  p->off_part = l.take(p->product.part_bytes);
  p->total = l.at ? l.at + 256 : 0;
  return LCE_OK;
}

static int32_t plan_linear_backward(int64_t n, int64_t d_in, int64_t d_out, int32_t dtype,
                                    BackwardPlan *p) {
  if (const int32_t st = lce_dims_check(n, d_in, d_out); st != LCE_OK) return st;
  if (!half_type(dtype)) return LCE_DTYPE_MISMATCH;
  Layout l;
  p->px = plan_product(d_in, n, d_out, false);
  p->pw = plan_product(d_in, d_out, n, false);
  p->joint = plan_joint(d_in, n, d_out, &p->px, &p->pw);
  p->ld_in = round_to(d_in, 64);
  p->ld_out = round_to(d_out, 64);
  p->ld_n = round_to(n, 64);
  if (!offsets_fit(p->ld_out) || !offsets_fit(p->ld_n)) p->joint = false;
  if (!offsets_fit(p->ld_out)) p->px = p->pw = ProductPlan{};
  else if (!offsets_fit(p->ld_n) && p->pw.core != k256x256) {
    // (more than 4 million tokens: transposed copies would be too wide)
    p->pw = ProductPlan{k256x256, 16, round_to(ceil_div(n, 16), 64)};
    p->pw.part_bytes = partial_bytes(d_in, d_out, 16);
  }
  // Only the 256 x 256 core takes operands that are not K-major.  d_weight's
  // two are so as they lie and cost it less than copies would (8192 x 4096 x
  // 4096, traced: least 227 to 231 us, median 265 to 277, against d_x's 228 to
  // 233 and 245 to 252 K-major); d_x's W beside K-major G costs a fifth (least
  // 287, median 316), more than W's transposed copy unless few tokens share it.
  const double step_cost = 0.3 * double(ceil_div(tile_count(d_in, n, 256, 256), 256)) *
                           double(ceil_div(d_out, 64));
  p->mn_w = p->pw.core == k256x256 || p->pw.core == kGeneric;
  p->mn_x = p->px.core == kGeneric ||
            (p->px.core == k256x256 && step_cost < 4.0 * double(d_in) * double(d_out) / kBytesPerUs);
  p->sum_parts = ceil_div(n, 64);
  p->off_g = l.take(size_t(n * p->ld_out * 2));
  if (p->mn_x) p->off_w = l.take(size_t(d_out * p->ld_in * 2));
  else p->off_wt = l.take(size_t(d_in * p->ld_out * 2));
  if (p->mn_w) {
    p->off_x = l.take(size_t(n * p->ld_in * 2));
  } else {
    p->off_gt = l.take(size_t(d_out * p->ld_n * 2));
    p->off_xt = l.take(size_t(d_in * p->ld_n * 2));
  }
  p->off_part = l.take(p->px.part_bytes);
  p->off_part_w = l.take(p->pw.part_bytes);
  p->off_sums = l.take(size_t(p->sum_parts * d_out * 4));
  p->total = l.at + 256;
  return LCE_OK;
}

template <bool F16>
static void run_copies(CopyJobs &jobs, int count, hipStream_t st) {
  int64_t blocks = 0;
  for (int i = 0; i < kMaxCopies; ++i) {
    CopyJob &j = jobs.job[i];
    if (i >= count) {
      j.tiles = 0;
      j.tiles_c = 1;
      continue;
    }
    // tiles up to the padded columns of dst and the padded rows of dst_t: the
    // padding ends inside the last tile (multiples of 64)
    j.tiles_c = uint32_t(ceil_div(j.cols, 64));
    j.tiles = uint32_t(ceil_div(j.rows, 64)) * j.tiles_c;
    blocks += j.tiles;
  }
  jobs.stride = 1;
  const uint32_t runs = uint32_t(blocks) / kCopyRun;
  if (count > 1 && runs > 8) {
    jobs.stride = runs * 5 / 8;                  // far apart, any job next to any other
    while (std::gcd(jobs.stride, runs) != 1) ++jobs.stride;
  }
  if (blocks) copies_kernel<F16><<<uint32_t(blocks), 256, 0, st>>>(jobs);
}

static bool known_act(int32_t a) { return a >= LCE_ACT_NONE && a <= LCE_ACT_SILU; }

// A saved activation [n][d]: 16-bit, or codes with scales.
static int32_t check_saved(const lce_tensor *v, const lce_tensor *scales, int32_t dtype, int64_t n,
                           int64_t d, bool lengths) {
  const bool packed = given(scales);
  if (!lengths) {
    if (packed ? (v->dtype != LCE_U8 || scales->dtype != LCE_U8) : v->dtype != dtype)
      return LCE_DTYPE_MISMATCH;
  } else {
    if (!holds(v, n * d) || (packed && !holds(scales, n * ceil_div(d, LCE_PACK8_BLOCK))))
      return LCE_LENGTH_MISMATCH;
  }
  return LCE_OK;
}

template <bool F16>
static void linear_run(const LinearPlan &p, const lce_tensor *x, const lce_tensor *w,
                       const OutParams &out, int64_t n, int64_t d_in, int64_t d_out, char *ws,
                       hipStream_t st) {
  const bool aligned = aligned_to(x->data, 16) && aligned_to(w->data, 16);
  if (p.product.core == kFew || (n <= kFewTokens && !aligned)) {
    const int64_t groups = ceil_div(d_out, 16);
    // waves that share 16 rows, with 128 k each at least (1024 x 1024, one
    // token, W in a cache: 7.4, 6.0, 4.8, 4.9 us with 1, 2, 4, 8; 4096 x 4096:
    // 20, 12, 8.3, 8.2)
    const int most = groups <= 128 ? 8 : 4;
    int kw = 1;
    while (kw < most && d_in / (2 * kw) >= 128) kw *= 2;
    const int waves = kw > 4 ? kw : 4, per_block = waves / kw;
    const int64_t k_part = round_to(ceil_div(d_in, kw), 32);
    auto run = [&](auto kernel) {
      kernel<<<uint32_t(ceil_div(groups, per_block)), waves * 64, 0, st>>>(
          static_cast<const uint16_t *>(x->data), static_cast<const uint16_t *>(w->data), int(n),
          d_in, d_out, kw, k_part, out);
    };
    if (n <= 16) run(few_tokens_kernel<F16, 1>);
    else if (n <= 32) run(few_tokens_kernel<F16, 2>);
    else run(few_tokens_kernel<F16, 4>);
    return;
  }
  Operand X = {x->data, d_in}, W = {w->data, d_in};
  if (p.ld_in) {
    CopyJobs jobs = {};
    const Operand src[2] = {X, W};
    const int64_t rows[2] = {n, d_out};
    const size_t off[2] = {p.off_x, p.off_w};
    Operand *to[2] = {&X, &W};
    for (int i = 0; i < 2; ++i) {
      CopyJob &j = jobs.job[i];
      j.src = src[i].p; j.rows = rows[i]; j.cols = d_in;
      j.dst = reinterpret_cast<uint16_t *>(ws + off[i]); j.ld = p.ld_in;
      *to[i] = {j.dst, p.ld_in};
    }
    run_copies<F16>(jobs, 2, st);
  } else if (!aligned && p.product.core == k256x256) {
    run_generic<F16, true, true>(W, X, d_out, n, d_in, out, st);
    return;
  }
  const bool any = !p.ld_in && (!aligned || p.any);
  run_product<F16, true, true>(p.product, W, X, d_out, n, p.ld_in ? p.ld_in : d_in, out,
                               ws + p.off_part, st, any);
}

template <bool F16>
static void linear_backward_run(const BackwardPlan &p, const lce_tensor *dy, const lce_tensor *x,
                                const lce_tensor *x_scales, const lce_tensor *w,
                                const lce_tensor *z, const lce_tensor *z_scales, int64_t n,
                                int64_t d_in, int64_t d_out, int32_t act, lce_tensor *d_x,
                                lce_tensor *d_w, lce_tensor *d_b, int32_t add, char *ws,
                                hipStream_t st) {
  auto at = [&](size_t off) { return reinterpret_cast<uint16_t *>(ws + off); };
  auto scales_of = [](const lce_tensor *t) {
    return given(t) ? static_cast<const uint8_t *>(t->data) : nullptr;
  };
  const bool want_x = given(d_x), want_w = given(d_w), want_b = given(d_b);
  const bool slope = act != kNone;
  // which copies the products need; what is aligned and of the right kind
  // already is used where it lies
  CopyJobs jobs = {};
  int count = 0;
  Operand G = {dy->data, d_out}, GT = {nullptr, 0}, X = {nullptr, 0}, W = {nullptr, 0};
  const bool kk_x = want_x && !p.mn_x, kk_w = want_w && !p.mn_w;
  const bool mn_x = want_x && p.mn_x, mn_w = want_w && p.mn_w;
  const bool copy_g = slope || !aligned_to(dy->data, 16) ||
                      (want_x && p.px.core == k256x256 && d_out % 64 != 0) || d_out % 8 != 0;
  {
    CopyJob j = {};
    j.src = dy->data; j.rows = n; j.cols = d_out;
    if (slope) {
      j.z = z->data; j.z_scales = scales_of(z_scales);
      j.act = act;
    }
    if (copy_g && (want_x || mn_w)) {
      j.dst = at(p.off_g); j.ld = p.ld_out;
      G = {j.dst, j.ld};
    }
    if (kk_w) {
      j.dst_t = at(p.off_gt); j.ld_t = p.ld_n;
      GT = {j.dst_t, j.ld_t};
    }
    if (want_b) j.sums = reinterpret_cast<float *>(ws + p.off_sums);
    if (j.dst || j.dst_t || j.sums) jobs.job[count++] = j;
  }
  if (want_w) {
    CopyJob j = {};
    j.src = x->data; j.scales = scales_of(x_scales);
    j.rows = n; j.cols = d_in;
    if (kk_w) {
      j.dst_t = at(p.off_xt); j.ld_t = p.ld_n;
      X = {j.dst_t, j.ld_t};
    } else if (j.scales || !aligned_to(x->data, 16) || d_in % 8 != 0) {
      j.dst = at(p.off_x); j.ld = p.ld_in;
      X = {j.dst, j.ld};
    } else {
      X = {x->data, d_in};
    }
    if (j.dst || j.dst_t) jobs.job[count++] = j;
  }
  if (want_x) {
    CopyJob j = {};
    j.src = w->data; j.rows = d_out; j.cols = d_in;
    if (kk_x) {
      j.dst_t = at(p.off_wt); j.ld_t = p.ld_out;
      W = {j.dst_t, j.ld_t};
    } else if (!aligned_to(w->data, 16) || d_in % 8 != 0) {
      j.dst = at(p.off_w); j.ld = p.ld_in;
      W = {j.dst, j.ld};
    } else {
      W = {w->data, d_in};
    }
    if (j.dst || j.dst_t) jobs.job[count++] = j;
  }
  run_copies<F16>(jobs, count, st);

  const BiasGrad bias = {want_b ? reinterpret_cast<const float *>(ws + p.off_sums) : nullptr,
                         p.sum_parts, d_out, want_b ? d_b->data : nullptr,
                         want_b && d_b->dtype == LCE_F32, add};
  const uint32_t bias_blocks = want_b ? uint32_t(ceil_div(d_out, 64)) : 0;
  OutParams ox = {}, ow = {};
  if (want_x) {
    ox.out = d_x->data; ox.ld = d_in; ox.rows = d_in; ox.cols = n;
  }
  if (want_w) {
    ow.out = d_w->data; ow.ld = d_in; ow.rows = d_in; ow.cols = d_out;
    ow.out_f32 = d_w->dtype == LCE_F32;
    ow.add = add;
  }
  const int64_t k_x = p.px.core == k256x256 ? p.ld_out : round_to(d_out, 8);
  char *part_x = ws + p.off_part, *part_w = ws + p.off_part_w;
  if (p.joint && kk_x && kk_w) {
    with_tile<F16>(p.px.core, [&](auto tile) {
      typedef decltype(tile) T;
      const TileParams gx = tile_params<T>(p.px, W, G, d_in, n, k_x);
      const TileParams gw = tile_params<T>(p.pw, X, GT, d_in, d_out, p.ld_n);
      const OutEpi<T> ex = {product_out(p.px, d_in, n, ox, part_x)};
      const OutEpi<T> ew = {product_out(p.pw, d_in, d_out, ow, part_w)};
      // (the tiles that take longest first)
      const bool w_first = p.pw.k_per_split > p.px.k_per_split;
      backward_kernel<T><<<gx.blocks + gw.blocks + bias_blocks, T::NT, 0, st>>>(
          w_first ? gw : gx, w_first ? ew : ex, w_first ? gx : gw, w_first ? ex : ew, bias);
    });
    run_folds<F16>(fold_job(p.px, d_in, n, ox, part_x), fold_job(p.pw, d_in, d_out, ow, part_w), st);
    return;
  }
  if (kk_x && mn_w && p.px.core == k256x256 && p.pw.core == k256x256) {
    typedef TraitsH16W8<F16> TR;
    const uint32_t bx = uint32_t(tile_count(d_in, n, 256, 256) * p.px.splits);
    const uint32_t bw = uint32_t(tile_count(d_in, d_out, 256, 256) * p.pw.splits);
    big_backward_kernel<F16><<<bw + bx + bias_blocks, TR::NT, 0, st>>>(
        big_params(p.pw, X, G, d_in, d_out, n),
        OutEpi<TR>{product_out(p.pw, d_in, d_out, ow, part_w)}, bw,
        big_params(p.px, W, G, d_in, n, k_x), OutEpi<TR>{product_out(p.px, d_in, n, ox, part_x)},
        bx, bias);
    run_folds<F16>(fold_job(p.px, d_in, n, ox, part_x), fold_job(p.pw, d_in, d_out, ow, part_w), st);
    return;
  }
  if (want_b) bias_grad_kernel<F16><<<bias_blocks, 256, 0, st>>>(bias);
  if (mn_x) run_product<F16, false, true>(p.px, W, G, d_in, n, d_out, ox, part_x, st);
  if (kk_x) run_product<F16, true, true>(p.px, W, G, d_in, n, k_x, ox, part_x, st);
  if (mn_w) run_product<F16, false, false>(p.pw, X, G, d_in, d_out, n, ow, part_w, st);
  if (kk_w) run_product<F16, true, true>(p.pw, X, GT, d_in, d_out, p.ld_n, ow, part_w, st);
}

}  // namespace lce

using namespace lce;

extern "C" {

int64_t lce_linear_workspace_bytes(int64_t n_tok, int64_t d_in, int64_t d_out, int32_t dtype) {
  LinearPlan p;
  const int32_t st = plan_linear(n_tok, d_in, d_out, dtype, &p);
  return st == LCE_OK ? int64_t(p.total) : -int64_t(st);
}

int64_t lce_linear_backward_workspace_bytes(int64_t n_tok, int64_t d_in, int64_t d_out,
                                            int32_t dtype) {
  BackwardPlan p;
  const int32_t st = plan_linear_backward(n_tok, d_in, d_out, dtype, &p);
  return st == LCE_OK ? int64_t(p.total) : -int64_t(st);
}

int32_t lce_linear(const lce_tensor *x, const lce_tensor *weight, const lce_tensor *bias,
                   const lce_tensor *residual, int64_t n_tok, int64_t d_in, int64_t d_out,
                   int32_t activation, lce_tensor *preact, lce_tensor *out, lce_tensor *workspace,
                   void *stream) {
  if (const int32_t st = lce_dims_check(n_tok, d_in, d_out); st != LCE_OK) return st;
  if (!x || !weight || !out) return LCE_LENGTH_MISMATCH;
  const int32_t dt = x->dtype;
  if (!half_type(dt) || weight->dtype != dt || (out->dtype != dt && out->dtype != LCE_F32) ||
      (given(bias) && bias->dtype != dt && bias->dtype != LCE_F32) ||
      (given(residual) && residual->dtype != dt) || (given(preact) && preact->dtype != dt) ||
      (given(workspace) && workspace->dtype != LCE_U8))
    return LCE_DTYPE_MISMATCH;
  LinearPlan p;
  (void)plan_linear(n_tok, d_in, d_out, dt, &p);
  const int64_t cells = n_tok * d_out;
  if (!holds(x, n_tok * d_in) || !holds(weight, d_out * d_in) || !holds(out, cells) ||
      (given(bias) && bias->numel < d_out) || (given(residual) && residual->numel < cells) ||
      (given(preact) && preact->numel < cells) ||
      (p.total && !holds(workspace, int64_t(p.total))))
    return LCE_LENGTH_MISMATCH;
  if (!known_act(activation)) return LCE_UNKNOWN_OBJECTIVE;

  (void)hipGetLastError();
  OutParams o = {};
  o.out = out->data; o.ld = d_out; o.rows = d_out; o.cols = n_tok;
  o.bias = given(bias) ? bias->data : nullptr;
  o.residual = given(residual) ? static_cast<const uint16_t *>(residual->data) : nullptr;
  o.preact = given(preact) ? static_cast<uint16_t *>(preact->data) : nullptr;
  o.out_f32 = out->dtype == LCE_F32;
  o.bias_f32 = given(bias) && bias->dtype == LCE_F32;
  o.act = activation;
  const hipStream_t st = hipStream_t(stream);
  char *ws = p.total ? aligned_base(workspace) : nullptr;
  if (dt == LCE_F16) linear_run<true>(p, x, weight, o, n_tok, d_in, d_out, ws, st);
  else linear_run<false>(p, x, weight, o, n_tok, d_in, d_out, ws, st);
  return enqueued_status();
}

int32_t lce_linear_backward(const lce_tensor *d_out_grad, const lce_tensor *x,
                            const lce_tensor *x_scales, const lce_tensor *weight,
                            const lce_tensor *preact, const lce_tensor *preact_scales,
                            int64_t n_tok, int64_t d_in, int64_t d_out, int32_t activation,
                            lce_tensor *d_x, lce_tensor *d_weight, lce_tensor *d_bias,
                            int32_t accumulate, lce_tensor *workspace, void *stream) {
  if (const int32_t st = lce_dims_check(n_tok, d_in, d_out); st != LCE_OK) return st;
  if (!d_out_grad || !workspace) return LCE_LENGTH_MISMATCH;
  const int32_t dt = d_out_grad->dtype;
  const bool slope = activation != LCE_ACT_NONE;
  if ((given(d_x) && !given(weight)) || (given(d_weight) && !given(x)) ||
      (slope && !given(preact)) || (!given(d_x) && !given(d_weight) && !given(d_bias)))
    return LCE_LENGTH_MISMATCH;
  if (!half_type(dt) || (given(d_x) && (weight->dtype != dt || d_x->dtype != dt)) ||
      (given(d_weight) && d_weight->dtype != dt && d_weight->dtype != LCE_F32) ||
      (given(d_bias) && d_bias->dtype != dt && d_bias->dtype != LCE_F32) ||
      workspace->dtype != LCE_U8)
    return LCE_DTYPE_MISMATCH;
  for (const bool lengths : {false, true}) {
    if (given(d_weight))
      if (const int32_t st = check_saved(x, x_scales, dt, n_tok, d_in, lengths); st != LCE_OK) return st;
    if (slope)
      if (const int32_t st = check_saved(preact, preact_scales, dt, n_tok, d_out, lengths); st != LCE_OK)
        return st;
  }
  BackwardPlan p;
  (void)plan_linear_backward(n_tok, d_in, d_out, dt, &p);
  if (!holds(d_out_grad, n_tok * d_out) || (given(d_x) && (!holds(weight, d_out * d_in) || !holds(d_x, n_tok * d_in))) ||
      (given(d_weight) && !holds(d_weight, d_out * d_in)) ||
      (given(d_bias) && !holds(d_bias, d_out)) || !holds(workspace, int64_t(p.total)))
    return LCE_LENGTH_MISMATCH;
  if (!known_act(activation)) return LCE_UNKNOWN_OBJECTIVE;

  (void)hipGetLastError();
  char *ws = aligned_base(workspace);
  const hipStream_t st = hipStream_t(stream);
  if (dt == LCE_F16)
    linear_backward_run<true>(p, d_out_grad, x, x_scales, weight, preact, preact_scales, n_tok,
                              d_in, d_out, activation, d_x, d_weight, d_bias, accumulate != 0, ws,
                              st);
  else
    linear_backward_run<false>(p, d_out_grad, x, x_scales, weight, preact, preact_scales, n_tok,
                               d_in, d_out, activation, d_x, d_weight, d_bias, accumulate != 0,
                               ws, st);
  return enqueued_status();
}

}  // extern "C"
