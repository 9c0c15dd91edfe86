// Shared pieces of the low-precision operators: loads of 8 values, the e4m3
// quantizer and its scale.
#pragma once

#include "kernels.hpp"
#include "lanes.hpp"

namespace gptq {

constexpr int kFp8Block = 128;  // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;

struct Vals8 {
  float v[8];
};

// Values c0 .. c0 + 7 of a row (bf16 or fp32) as fp32, 0 past n.  `vec`: the
// row's address and c0 allow 16-byte loads (uniform over the grid).
template <int DT>
__device__ __forceinline__ Vals8 load_vals8(const void* row, int64_t c0, int64_t n, bool vec) {
  Vals8 o;
  if (vec && c0 + 8 <= n) {
    if (DT == GPTQ_BF16) {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + c0);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o.v[2 * k] = __uint_as_float(w[k] << 16);
        o.v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
      const float* p = reinterpret_cast<const float*>(row) + c0;
      const float4 a = *reinterpret_cast<const float4*>(p);
      const float4 b = *reinterpret_cast<const float4*>(p + 4);
      o.v[0] = a.x; o.v[1] = a.y; o.v[2] = a.z; o.v[3] = a.w;
      o.v[4] = b.x; o.v[5] = b.y; o.v[6] = b.z; o.v[7] = b.w;
    }
    return o;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) o.v[k] = c0 + k < n ? load_elem(row, DT, c0 + k) : 0.0f;
  return o;
}

// The largest finite magnitude of 8 values.
__device__ __forceinline__ float amax_finite8(const Vals8& x) {
  float a = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(x.v[k]));  // fmax passes over NaN
  if (a == __builtin_inff()) {  // rare: some value is infinite
    a = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (is_finite(x.v[k])) a = fmaxf(a, fabsf(x.v[k]));
  }
  return a;
}

// s = RN32(amax / 448), at least 2^-126 so that s and 1 / s are normal numbers;
// 1 where every value is 0.
__device__ __forceinline__ float e4m3_scale(float amax) {
  return amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, kE4m3Max), 0x1p-126f);
}

// The e4m3 code nearest to the real quotient x / s, ties to even, where its two
// candidates lo and hi = lo + 1 (magnitudes) are known: the sign of
// |x| - h s with h the border between them, which one fma gives exactly (small
// scales are lifted first, so that no partial result is below the subnormals).
__device__ __forceinline__ uint32_t e4m3_decide(float x, float s, uint32_t lo, uint32_t hi) {
  float a = fabsf(x);
  if (s < 0x1p-60f) {
    a *= 0x1p64f;
    s *= 0x1p64f;
  }
  const float vl = __builtin_amdgcn_cvt_f32_fp8((int)lo, 0), vh = __builtin_amdgcn_cvt_f32_fp8((int)hi, 0);
  const float h = 0.5f * (vl + vh);  // exact: 5 significant bits
  const float r = fmaf(-h, s, a);
  return r > 0.0f ? hi : r < 0.0f ? lo : ((lo & 1) ? hi : lo);
}

// 1 / s to within 2^-23 of itself, for a normal s and 1 / s
__device__ __forceinline__ float approx_recip(float s) { return __builtin_amdgcn_rcpf(s); }

// 8 codes of x / s, rs = approx_recip(s).  x * rs is within 2^-22 |x / s| of the
// quotient, so the hardware's rounding of that product lowered and raised by 2^-21 brackets the
// code; where the two differ (a border of the format is that close: about one
// value in 10^5) e4m3_decide takes the real quotient.  A non-finite value
// becomes the NaN code (the instruction's own result for it).
__device__ __forceinline__ uint2 e4m3_codes8(const Vals8& x, float s, float rs) {
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = x.v[4 * p + k] * rs;
    int a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * 0.99999952f, q[1] * 0.99999952f, a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * 0.99999952f, q[3] * 0.99999952f, a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * 1.00000048f, q[1] * 1.00000048f, b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * 1.00000048f, q[3] * 1.00000048f, b, true);
    lo[p] = (uint32_t)a;
    hi[p] = (uint32_t)b;
  }
  if (lo[0] != hi[0] || lo[1] != hi[1]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int sh = 8 * (k & 3);
      const uint32_t cl = (lo[k >> 2] >> sh) & 0x7F, ch = (hi[k >> 2] >> sh) & 0x7F;
      if (cl != ch && is_finite(x.v[k])) {
        const uint32_t c = e4m3_decide(x.v[k], s, cl, ch);
        lo[k >> 2] = (lo[k >> 2] & ~(0x7Fu << sh)) | (c << sh);
      }
    }
  }
  return make_uint2(lo[0], lo[1]);
}

}  // namespace gptq
