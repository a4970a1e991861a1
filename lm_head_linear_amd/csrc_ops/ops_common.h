// ops_common.h -- host checks and device helpers shared by the operators that
// stand next to the loss kernels (linear layer, 8-bit checkpoints, beam step).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../csrc/lce_gemm.hpp"
#include "../csrc/lce_internal.h"

namespace lce {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_to(int64_t x, int64_t m) { return ceil_div(x, m) * m; }

inline bool given(const lce_tensor *t) { return t && t->data; }
inline bool half_type(int32_t dtype) { return dtype == LCE_BF16 || dtype == LCE_F16; }
inline bool holds(const lce_tensor *t, int64_t numel) { return given(t) && t->numel >= numel; }
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int32_t enqueued_status() {
  return hipGetLastError() == hipSuccess ? LCE_OK : LCE_DEVICE_ERROR;
}

// Workspaces are used from their first 256-byte boundary.
inline char *aligned_base(const lce_tensor *ws) {
  return reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(ws->data) + 255) & ~uintptr_t(255));
}

// ---- 16-byte accesses at any alignment ----------------------------------
// Global memory takes vector accesses at any byte address; the packed type
// tells the compiler that the address may be odd.
struct __attribute__((packed, aligned(1))) AnyVec16 { uint32_t v[4]; };
struct __attribute__((packed, aligned(1))) AnyVec8 { uint32_t v[2]; };

__device__ inline u32x4 load16(const void *p) {
  const AnyVec16 a = *static_cast<const AnyVec16 *>(p);
  return u32x4{a.v[0], a.v[1], a.v[2], a.v[3]};
}
__device__ inline void store16(void *p, u32x4 x) {
  *static_cast<AnyVec16 *>(p) = AnyVec16{{x[0], x[1], x[2], x[3]}};
}

// A 16-bit value to fp32 and back (round to nearest even).
template <bool F16> __device__ inline float widen(uint16_t h) {
  return F16 ? f16_to_f32(h) : bf16_to_f32(h);
}
template <bool F16> __device__ inline uint16_t narrow(float f) {
  return F16 ? f32_to_f16_rne(f) : f32_to_bf16_rne(f);
}
// Eight 16-bit values of a vector, as fp32.
template <bool F16> __device__ inline void widen8(u32x4 x, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = widen<F16>(uint16_t(x[i]));
    f[2 * i + 1] = widen<F16>(uint16_t(x[i] >> 16));
  }
}
template <bool F16> __device__ inline u32x4 narrow8(const float (&f)[8]) {
  u32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = uint32_t(narrow<F16>(f[2 * i])) | (uint32_t(narrow<F16>(f[2 * i + 1])) << 16);
  return x;
}

// Eight e4m3 codes times 2^e as fp32: exact (4 significant bits).
__device__ inline void codes_to_f32(uint32_t lo, uint32_t hi, int e, float (&f)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), false);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), true);
  f[0] = __builtin_ldexpf(a[0], e); f[1] = __builtin_ldexpf(a[1], e);
  f[2] = __builtin_ldexpf(b[0], e); f[3] = __builtin_ldexpf(b[1], e);
  f[4] = __builtin_ldexpf(c[0], e); f[5] = __builtin_ldexpf(c[1], e);
  f[6] = __builtin_ldexpf(d[0], e); f[7] = __builtin_ldexpf(d[1], e);
}
// A value read back from a checkpoint, held within the 16-bit type's finite
// range (NaN stays NaN).
template <bool F16> __device__ inline uint16_t saturate16(float f) {
  const float most = F16 ? 65504.0f : 3.3895313892515355e38f;
  return narrow<F16>(f > most ? most : f < -most ? -most : f);
}

}  // namespace lce
