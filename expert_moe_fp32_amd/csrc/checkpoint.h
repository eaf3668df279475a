// 8-bit checkpoints of activations: 128 neighbouring columns of a row share a
// power-of-two scale s = 2^e, the smallest with amax / s <= 448, and a value
// is kept as the E4M3 code nearest to v / s (ties to even).  Multiplying by a
// power of two rounds nothing, and a code has four significant bits, so
// code * s is exact in bf16: the backward pass multiplies exactly what the
// checkpoint says, in the matrix cores' own type.  (The weights' scales,
// amax / 448, would need a second rounding there.)  A power of two costs no
// precision either, only range: at most one of the 18 binades of a code.
#pragma once

#include "common.h"

namespace moe {

// smallest and largest exponent of a scale
constexpr int kCheckpointLow = -100, kCheckpointHigh = 120;

// Exponent of the scale for a group whose largest finite magnitude is `amax`
// (0 for a group of zeros): amax = m 2^x with m in [1, 2), and 448 = 1.75 2^8.
__device__ __forceinline__ int checkpoint_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 135 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return u == 0 ? 0 : max(e, kCheckpointLow);
}
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// the largest code magnitude: one step less where 2^8 times the largest scale
// would leave float32
__device__ __forceinline__ float checkpoint_limit(int e) {
  return e >= kCheckpointHigh ? 240.0f : 448.0f;
}

// Largest magnitude of finite values, 0 for the others: bits of infinities
// and NaN lie above every finite one.
__device__ __forceinline__ float finite_size(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? __uint_as_float(u) : 0.0f;
}

// Four codes of four values; `inv` = 1 / scale.  What is not finite becomes
// the code of NaN.
__device__ __forceinline__ uint32_t checkpoint_codes(float a, float b, float c,
                                                     float d, float inv,
                                                     float limit) {
  const float v[4] = {a, b, c, d};
  float q[4];
  uint32_t odd = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float w = v[i] * inv;
    q[i] = __builtin_fminf(__builtin_fmaxf(w, -limit), limit);
    if ((__float_as_uint(v[i]) & 0x7F800000u) == 0x7F800000u) odd |= 0x7Fu << (8 * i);
  }
  uint32_t r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], (int)r, true);
  return r | odd;
}

// max over the 16 lanes of a DPP row, in each of them
__device__ __forceinline__ float row16_max(float v) {
#define ROW_MAX(ctrl)                                                         \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xF, 0xF, true)));
  ROW_MAX(0x128) ROW_MAX(0x124) ROW_MAX(0x122) ROW_MAX(0x121)
#undef ROW_MAX
  return v;
}

// the four values of four codes, unscaled
__device__ __forceinline__ void code_values(uint32_t c, float* v) {
  typedef __attribute__((ext_vector_type(2))) float f32x2_t;
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  v[0] = lo.x; v[1] = lo.y; v[2] = hi.x; v[3] = hi.y;
}

// two values to bf16, rounded to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

}  // namespace moe
