// linear.hip -- Y = act(X W^T + b) + R and its backward, 16-bit operands with
// fp32 sums on the matrix cores.
//
// Every product is computed as C[m][c] with m the contiguous index of the
// result's rows and c its row, so that a lane's four consecutive accumulators
// are four consecutive elements in memory:
//   forward   Y[t][o]   : m = o (W, K-major),  c = t (X, K-major),  depth d_in
//   d_x       dX[t][i]  : m = i (W, MN-major), c = t (G, K-major),  depth d_out
//   d_weight  dW[o][i]  : m = i (X, MN-major), c = o (G, MN-major), depth n
// with G = dY * act'(Z), rounded to the 16-bit type once (it feeds matrix
// instructions); the bias gradient sums the unrounded G in fp32.
#include <math.h>

#include "ops_common.h"

namespace lce {

enum Act { kNone = LCE_ACT_NONE, kRelu = LCE_ACT_RELU, kGelu = LCE_ACT_GELU, kSilu = LCE_ACT_SILU };

__device__ inline float act_value(float z, int act) {
  switch (act) {
    case kRelu: return z > 0.0f || z != z ? z : 0.0f;
    case kGelu: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case kSilu: return z / (1.0f + __expf(-z));
    default: return z;
  }
}
__device__ inline float act_slope(float z, int act) {
  switch (act) {
    case kRelu: return z > 0.0f ? 1.0f : 0.0f;
    case kGelu:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
             z * 0.39894228040143268f * __expf(-0.5f * z * z);
    case kSilu: {
      const float s = 1.0f / (1.0f + __expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// What becomes of C[m][c], stored at row c, element m of the result.
struct OutParams {
  void *out;              // [cols][ld]
  int64_t ld;
  int64_t rows, cols;     // valid m and c
  const void *bias;       // [rows], 16-bit or fp32, or null
  const uint16_t *residual;  // [cols][ld] or null
  uint16_t *preact;       // [cols][ld] or null
  int32_t out_f32, bias_f32, act, add;   // add: out += C
};

template <class TR>
struct OutEpi {
  OutParams p;
  static constexpr bool F16 = TR::F16;

  __device__ __forceinline__ void one(float z, int64_t m, int64_t c) const {
    const int64_t at = c * p.ld + m;
    if (p.bias)
      z += p.bias_f32 ? static_cast<const float *>(p.bias)[m]
                      : widen<F16>(static_cast<const uint16_t *>(p.bias)[m]);
    if (p.preact) p.preact[at] = narrow<F16>(z);
    float y = act_value(z, p.act);
    if (p.residual) y += widen<F16>(p.residual[at]);
    if (p.out_f32) {
      float *o = static_cast<float *>(p.out) + at;
      *o = p.add ? *o + y : y;
    } else {
      uint16_t *o = static_cast<uint16_t *>(p.out) + at;
      *o = narrow<F16>(p.add ? widen<F16>(*o) + y : y);
    }
  }
  __device__ __forceinline__ void operator()(typename TR::AccBlock (&acc)[TR::FM][TR::FN],
                                             int64_t m0, int64_t n0, int wm, int wn, int lane,
                                             int) const {
#pragma unroll 1
    for (int fn = 0; fn < TR::FN; ++fn) {
      const int64_t c = n0 + wn * TR::WTN + fn * TR::MF + TR::col_of(lane);
      if (c >= p.cols) continue;
#pragma unroll 1
      for (int fm = 0; fm < TR::FM; ++fm) {
#pragma unroll
        for (int r = 0; r < TR::R; ++r) {
          const int64_t m = m0 + wm * TR::WTM + fm * TR::MF + TR::row_of(r, lane);
          float z = 0.0f;
#pragma unroll
          for (int a = 0; a < TR::FM; ++a)
#pragma unroll
            for (int b = 0; b < TR::FN; ++b)
              if (a == fm && b == fn) z = acc[a][b][r];
          if (m < p.rows) one(z, m, c);
        }
      }
    }
  }
};

// ---------------------------------------------------- the backward's inputs --

// Z as 16-bit values or as an 8-bit checkpoint.
struct Saved {
  const void *v;           // 16-bit values or codes, [n][d]; null: none
  const uint8_t *scales;   // [n][ceil(d/32)] for codes, else null
};
template <bool F16>
__device__ inline float saved_value(const Saved &s, int64_t row, int64_t col, int64_t d) {
  if (!s.scales) return widen<F16>(static_cast<const uint16_t *>(s.v)[row * d + col]);
  const uint32_t code = static_cast<const uint8_t *>(s.v)[row * d + col];
  const int e = int(s.scales[row * ((d + 31) / 32) + col / 32]) - 127;
  const float f = __builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8(int(code), 0), e);
  return widen<F16>(saturate16<F16>(f));
}

// Rows of `rows_per` tokens: G = dY act'(Z) stored when g is given, and the
// fp32 column sums of the unrounded G over these rows when sums is given
// ([gridDim.y][d]).  Thread = column.
template <bool F16>
__global__ void __launch_bounds__(256) slope_kernel(const uint16_t *dy, Saved z, int64_t n,
                                                    int64_t d, int act, int64_t rows_per,
                                                    uint16_t *g, float *sums) {
  const int64_t col = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (col >= d) return;
  const int64_t r0 = int64_t(blockIdx.y) * rows_per;
  const int64_t r1 = r0 + rows_per < n ? r0 + rows_per : n;
  float sum = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    float v = widen<F16>(dy[r * d + col]);
    if (z.v) v *= act_slope(saved_value<F16>(z, r, col, d), act);
    sum += v;
    if (g) g[r * d + col] = narrow<F16>(v);
  }
  if (sums) sums[int64_t(blockIdx.y) * d + col] = sum;
}

// Adds `parts` rows of sums in order.
template <bool F16>
__global__ void __launch_bounds__(256) bias_grad_kernel(const float *sums, int64_t parts, int64_t d,
                                                        void *out, int out_f32, int add) {
  const int64_t col = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (col >= d) return;
  float s = 0.0f;
  for (int64_t i = 0; i < parts; ++i) s += sums[i * d + col];
  if (out_f32) {
    float *o = static_cast<float *>(out) + col;
    *o = add ? *o + s : s;
  } else {
    uint16_t *o = static_cast<uint16_t *>(out) + col;
    *o = narrow<F16>(add ? widen<F16>(*o) + s : s);
  }
}

// ------------------------------------------------------------------- host --

template <class TR, bool AK, bool BKM>
static void run_product(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t M,
                        int64_t N, int64_t K, const OutParams &out, hipStream_t st) {
  const bool vec = aligned_to(A, 16) && aligned_to(B, 16) && lda % 8 == 0 && ldb % 8 == 0;
  GemmParams g = {};
  g.A = A; g.lda = lda; g.B = B; g.ldb = ldb;
  g.M = M; g.N = N; g.K = K;
  g.M_read = round_to(M, 8); g.N_read = round_to(N, 8);
  g.k_per_split = round_to(K, TR::BK);
  g.tiles_n = ceil_div(N, TR::BN);
  const int64_t tiles = ceil_div(M, TR::BM) * g.tiles_n;
  const OutEpi<TR> epi{out};
  if (vec) gemm_kernel<TR, AK, BKM, true><<<dim3(uint32_t(tiles)), TR::NT, 0, st>>>(g, epi);
  else gemm_kernel<TR, AK, BKM, false><<<dim3(uint32_t(tiles)), TR::NT, 0, st>>>(g, epi);
}

// Rows of dY that one block of slope_kernel sums.
static int64_t slope_rows(int64_t n) {
  const int64_t r = ceil_div(n, 256);
  return r < 16 ? 16 : r;
}

struct LinearPlan {
  size_t off_g = 0, off_x = 0, off_sums = 0, total = 0;
  int64_t sum_parts = 0;
};

static int32_t plan_linear(int64_t n, int64_t d_in, int64_t d_out, int32_t dtype) {
  if (const int32_t st = lce_dims_check(n, d_in, d_out); st != LCE_OK) return st;
  return half_type(dtype) ? LCE_OK : LCE_DTYPE_MISMATCH;
}
static int32_t plan_linear_backward(int64_t n, int64_t d_in, int64_t d_out, int32_t dtype,
                                    LinearPlan *p) {
  if (const int32_t st = plan_linear(n, d_in, d_out, dtype); st != LCE_OK) return st;
  p->sum_parts = ceil_div(n, slope_rows(n));
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += size_t(round_to(bytes, 256));
    return here;
  };
  p->off_g = take(n * d_out * 2);
  p->off_x = take(n * d_in * 2);
  p->off_sums = take(p->sum_parts * d_out * 4);
  p->total = at + 256;
  return LCE_OK;
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
static void linear_run(const lce_tensor *x, const lce_tensor *w, const OutParams &out, int64_t n,
                       int64_t d_in, int64_t d_out, hipStream_t st) {
  run_product<TraitsH16<F16>, true, true>(w->data, d_in, x->data, d_in, d_out, n, d_in, out, st);
}

template <bool F16>
static void linear_backward_run(const LinearPlan &p, const lce_tensor *dy, const lce_tensor *x,
                                const lce_tensor *x_scales, const lce_tensor *w, const Saved &z,
                                int64_t n, int64_t d_in, int64_t d_out, int32_t act,
                                lce_tensor *d_x, lce_tensor *d_w, lce_tensor *d_b, int32_t add,
                                char *ws, void *stream) {
  typedef TraitsH16<F16> TR;
  const hipStream_t st = hipStream_t(stream);
  const uint16_t *G = static_cast<const uint16_t *>(dy->data);
  const bool slope = act != kNone;
  if (slope || given(d_b)) {
    uint16_t *g = slope ? reinterpret_cast<uint16_t *>(ws + p.off_g) : nullptr;
    float *sums = given(d_b) ? reinterpret_cast<float *>(ws + p.off_sums) : nullptr;
    slope_kernel<F16><<<dim3(uint32_t(ceil_div(d_out, 256)), uint32_t(p.sum_parts)), 256, 0, st>>>(
        G, slope ? z : Saved{nullptr, nullptr}, n, d_out, act, slope_rows(n), g, sums);
    if (given(d_b))
      bias_grad_kernel<F16><<<uint32_t(ceil_div(d_out, 256)), 256, 0, st>>>(
          sums, p.sum_parts, d_out, d_b->data, d_b->dtype == LCE_F32, add);
    if (slope) G = g;
  }
  OutParams o = {};
  if (given(d_x)) {
    o.out = d_x->data; o.ld = d_in; o.rows = d_in; o.cols = n;
    run_product<TR, false, true>(w->data, d_in, G, d_out, d_in, n, d_out, o, st);
  }
  if (given(d_w)) {
    const void *X = x->data;
    if (given(x_scales)) {
      lce_tensor xt = {ws + p.off_x, n * d_in, F16 ? LCE_F16 : LCE_BF16};
      lce_unpack8(x, x_scales, n, d_in, &xt, stream);
      X = xt.data;
    }
    o = {};
    o.out = d_w->data; o.ld = d_in; o.rows = d_in; o.cols = d_out;
    o.out_f32 = d_w->dtype == LCE_F32;
    o.add = add;
    run_product<TR, false, false>(X, d_in, G, d_out, d_in, d_out, n, o, st);
  }
}

}  // namespace lce

using namespace lce;

extern "C" {

int64_t lce_linear_workspace_bytes(int64_t n_tok, int64_t d_in, int64_t d_out, int32_t dtype) {
  const int32_t st = plan_linear(n_tok, d_in, d_out, dtype);
  return st == LCE_OK ? 256 : -int64_t(st);
}

int64_t lce_linear_backward_workspace_bytes(int64_t n_tok, int64_t d_in, int64_t d_out,
                                            int32_t dtype) {
  LinearPlan p;
  const int32_t st = plan_linear_backward(n_tok, d_in, d_out, dtype, &p);
  return st == LCE_OK ? int64_t(p.total) : -int64_t(st);
}

int32_t lce_linear(const lce_tensor *x, const lce_tensor *weight, const lce_tensor *bias,
                   const lce_tensor *residual, int64_t n_tok, int64_t d_in, int64_t d_out,
                   int32_t activation, lce_tensor *preact, lce_tensor *out, lce_tensor *workspace,
                   void *stream) {
  if (const int32_t st = lce_dims_check(n_tok, d_in, d_out); st != LCE_OK) return st;
  if (!x || !weight || !out || !workspace) return LCE_LENGTH_MISMATCH;
  const int32_t dt = x->dtype;
  if (!half_type(dt) || weight->dtype != dt || (out->dtype != dt && out->dtype != LCE_F32) ||
      (given(bias) && bias->dtype != dt && bias->dtype != LCE_F32) ||
      (given(residual) && residual->dtype != dt) || (given(preact) && preact->dtype != dt) ||
      workspace->dtype != LCE_U8)
    return LCE_DTYPE_MISMATCH;
  const int64_t cells = n_tok * d_out;
  if (!holds(x, n_tok * d_in) || !holds(weight, d_out * d_in) || !holds(out, cells) ||
      (given(bias) && bias->numel < d_out) || (given(residual) && residual->numel < cells) ||
      (given(preact) && preact->numel < cells) ||
      !holds(workspace, lce_linear_workspace_bytes(n_tok, d_in, d_out, dt)))
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
  if (dt == LCE_F16) linear_run<true>(x, weight, o, n_tok, d_in, d_out, st);
  else linear_run<false>(x, weight, o, n_tok, d_in, d_out, st);
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
  LinearPlan p;
  (void)plan_linear_backward(n_tok, d_in, d_out, dt, &p);
  if (!holds(d_out_grad, n_tok * d_out) || (given(d_x) && (!holds(weight, d_out * d_in) || !holds(d_x, n_tok * d_in))) ||
      (given(d_weight) && !holds(d_weight, d_out * d_in)) ||
      (given(d_bias) && !holds(d_bias, d_out)) || !holds(workspace, int64_t(p.total)))
    return LCE_LENGTH_MISMATCH;
  if (!known_act(activation)) return LCE_UNKNOWN_OBJECTIVE;

  (void)hipGetLastError();
  const Saved z = {slope ? preact->data : nullptr,
                   slope && given(preact_scales)
                       ? static_cast<const uint8_t *>(preact_scales->data) : nullptr};
  char *ws = aligned_base(workspace);
  if (dt == LCE_F16)
    linear_backward_run<true>(p, d_out_grad, x, x_scales, weight, z, n_tok, d_in, d_out, activation,
                              d_x, d_weight, d_bias, accumulate != 0, ws, stream);
  else
    linear_backward_run<false>(p, d_out_grad, x, x_scales, weight, z, n_tok, d_in, d_out,
                               activation, d_x, d_weight, d_bias, accumulate != 0, ws, stream);
  return enqueued_status();
}

}  // extern "C"
