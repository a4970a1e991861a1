// checkpoint.hip -- 16-bit activations kept in 8 bits (e4m3 codes with a
// power-of-two scale per 32 values of a row) and read back.
//
// Per block of 32 values: A = max |x| over the finite ones, e the smallest
// integer with A <= 448 * 2^e, code = round_e4m3(x * 2^-e).  With A = m 2^E,
// m in [1, 2): e = E - 8 when m <= 1.75, else E - 7, read off A's bits.  The
// product by a power of two and the way back are exact, so the only rounding
// is the one to e4m3.
// Bound by memory: 2 + 1 + 1/32 bytes a value each way.  A lane holds 8 values
// (one 16-byte load); the four lanes of a quad share a block, so the maximum
// is two lane swaps within the quad and no value leaves its lane.  8192 x 4096
// bf16: 20 us packed, 17.5 read back (5.1 and 5.8 TB/s; a large copy: 5.0).
#include "ops_common.h"

namespace lce {

// Max over the four lanes of a quad.
__device__ inline uint32_t quad_max(uint32_t x) {
  uint32_t y = __builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xF, 0xF, true);   // lanes 1 0 3 2
  x = x > y ? x : y;
  y = __builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xF, 0xF, true);            // lanes 2 3 0 1
  return x > y ? x : y;
}

// The exponent of a block's scale from the bits of its largest magnitude.
template <bool F16> __device__ inline int scale_exponent(uint32_t amax_bits) {
  const int lowest = F16 ? -15 : -117;
  const int e = int(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > lowest ? e : lowest;
}

// Each wave takes 512 consecutive values (16 blocks) of one row, lane l the
// values 8 l .. 8 l + 7; FLAT (d a multiple of 32): rows follow one another
// without a gap, so the whole array is one row.
template <bool F16, bool FLAT>
__global__ void __launch_bounds__(256) pack8_kernel(const uint16_t *x, int64_t n, int64_t d,
                                                    uint8_t *codes, uint8_t *scales) {
  const int lane = threadIdx.x & 63;
  const int64_t cols = FLAT ? n * d : d, rows = FLAT ? 1 : n;
  const int64_t per_row = (cols + 511) / 512, units = rows * per_row;
  const int64_t blocks = (cols + 31) / 32;
  for (int64_t u = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units;
       u += int64_t(gridDim.x) * 4) {
    const int64_t row = FLAT ? 0 : u / per_row, c = (FLAT ? u : u % per_row) * 512 + lane * 8;
    const int64_t left = cols - c;      // values of this lane that exist
    const uint16_t *p = x + row * cols + c;
    float f[8];
    if (left >= 8) {
      widen8<F16>(load16(p), f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = i < left ? widen<F16>(p[i]) : 0.0f;
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __float_as_uint(f[i]) & 0x7fffffffu;
      if (m < 0x7f800000u) a = m > a ? m : a;
      else f[i] = __uint_as_float(0x7fc00000u);    // infinities have no code: NaN
    }
    const int e = scale_exponent<F16>(quad_max(a));
    const float unit = __uint_as_float(uint32_t(127 - e) << 23);   // 2^-e: e in [-117, 120]
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * unit, f[1] * unit, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * unit, f[3] * unit, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * unit, f[5] * unit, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * unit, f[7] * unit, hi, true);
    uint8_t *q = codes + row * cols + c;
    if (left >= 8) {
      *reinterpret_cast<AnyVec8 *>(q) = AnyVec8{{uint32_t(lo), uint32_t(hi)}};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = uint8_t(uint32_t(i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if ((lane & 3) == 0 && left > 0) scales[row * blocks + c / 32] = uint8_t(e + 127);
  }
}

template <bool F16, bool FLAT>
__global__ void __launch_bounds__(256) unpack8_kernel(const uint8_t *codes, const uint8_t *scales,
                                                      int64_t n, int64_t d, uint16_t *out) {
  const int lane = threadIdx.x & 63;
  const int64_t cols = FLAT ? n * d : d, rows = FLAT ? 1 : n;
  const int64_t per_row = (cols + 511) / 512, units = rows * per_row;
  const int64_t blocks = (cols + 31) / 32;
  for (int64_t u = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units;
       u += int64_t(gridDim.x) * 4) {
    const int64_t row = FLAT ? 0 : u / per_row, c = (FLAT ? u : u % per_row) * 512 + lane * 8;
    const int64_t left = cols - c;
    if (left <= 0) continue;
    const uint8_t *q = codes + row * cols + c;
    uint32_t w[2] = {0, 0};
    if (left >= 8) {
      const AnyVec8 v = *reinterpret_cast<const AnyVec8 *>(q);
      w[0] = v.v[0]; w[1] = v.v[1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 2] |= uint32_t(q[i]) << (8 * (i & 3));
    }
    float f[8];
    codes_to_f32(w[0], w[1], int(scales[row * blocks + c / 32]) - 127, f);
    uint16_t *p = out + row * cols + c;
    if (left >= 8) {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = uint32_t(saturate16<F16>(f[2 * i])) | (uint32_t(saturate16<F16>(f[2 * i + 1])) << 16);
      store16(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = saturate16<F16>(f[i]);
    }
  }
}

static int pack8_grid(int64_t n, int64_t d) {
  const int64_t units = d % 32 == 0 ? ceil_div(n * d, 512) : n * ceil_div(d, 512);
  const int64_t blocks = ceil_div(units, 4);
  return int(blocks < 65536 ? blocks : 65536);
}

static int32_t check_pack8(const lce_tensor *x, int64_t n, int64_t d, const lce_tensor *codes,
                           const lce_tensor *scales) {
  if (const int32_t st = lce_dims_check(n, 1, d); st != LCE_OK) return st;
  if (!x || !codes || !scales) return LCE_LENGTH_MISMATCH;
  if (!half_type(x->dtype) || codes->dtype != LCE_U8 || scales->dtype != LCE_U8)
    return LCE_DTYPE_MISMATCH;
  if (!holds(x, n * d) || !holds(codes, n * d) ||
      !holds(scales, n * ceil_div(d, LCE_PACK8_BLOCK)))
    return LCE_LENGTH_MISMATCH;
  return LCE_OK;
}

}  // namespace lce

using namespace lce;

extern "C" {

int32_t lce_pack8(const lce_tensor *x, int64_t n, int64_t d, lce_tensor *codes,
                  lce_tensor *scales, void *stream) {
  if (const int32_t st = check_pack8(x, n, d, codes, scales); st != LCE_OK) return st;
  (void)hipGetLastError();
  auto run = [&](auto kernel) {
    kernel<<<pack8_grid(n, d), 256, 0, hipStream_t(stream)>>>(
        static_cast<const uint16_t *>(x->data), n, d, static_cast<uint8_t *>(codes->data),
        static_cast<uint8_t *>(scales->data));
  };
  const bool flat = d % 32 == 0;
  if (x->dtype == LCE_F16) flat ? run(pack8_kernel<true, true>) : run(pack8_kernel<true, false>);
  else flat ? run(pack8_kernel<false, true>) : run(pack8_kernel<false, false>);
  return enqueued_status();
}

int32_t lce_unpack8(const lce_tensor *codes, const lce_tensor *scales, int64_t n, int64_t d,
                    lce_tensor *out, void *stream) {
  if (const int32_t st = check_pack8(out, n, d, codes, scales); st != LCE_OK) return st;
  (void)hipGetLastError();
  auto run = [&](auto kernel) {
    kernel<<<pack8_grid(n, d), 256, 0, hipStream_t(stream)>>>(
        static_cast<const uint8_t *>(codes->data), static_cast<const uint8_t *>(scales->data), n,
        d, static_cast<uint16_t *>(out->data));
  };
  const bool flat = d % 32 == 0;
  if (out->dtype == LCE_F16)
    flat ? run(unpack8_kernel<true, true>) : run(unpack8_kernel<true, false>);
  else
    flat ? run(unpack8_kernel<false, true>) : run(unpack8_kernel<false, false>);
  return enqueued_status();
}

}  // extern "C"
