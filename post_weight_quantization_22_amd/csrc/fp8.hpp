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

// Values c0 .. c0 + 7 of a row (bf16 or fp32) as they lie in memory, 0 past n.
// `vec`: the row's address and c0 allow 16-byte loads (uniform over the grid).  Kept
// apart from their conversion: converted inside the branch below, each load would be
// waited for there, and several could not be in flight.
template <int DT>
struct Raw8 {
  uint32_t w[DT == GPTQ_BF16 ? 4 : 8];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* row, int64_t c0, int64_t n, bool vec) {
  Raw8<DT> o;
  const char* p = reinterpret_cast<const char*>(row) + c0 * (DT == GPTQ_BF16 ? 2 : 4);
  if (vec && c0 + 8 <= n) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
    if constexpr (DT != GPTQ_BF16) {
      const uint4 b = *reinterpret_cast<const uint4*>(p + 16);
      o.w[4] = b.x; o.w[5] = b.y; o.w[6] = b.z; o.w[7] = b.w;
    }
    return o;
  }
  if constexpr (DT == GPTQ_BF16) {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o.w[k] = c0 + 2 * k < n ? e[2 * k] : 0;
      if (c0 + 2 * k + 1 < n) o.w[k] |= (uint32_t)e[2 * k + 1] << 16;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) o.w[k] = c0 + k < n ? reinterpret_cast<const uint32_t*>(p)[k] : 0;
  }
  return o;
}

template <int DT>
__device__ __forceinline__ Vals8 vals_of(const Raw8<DT>& r) {
  Vals8 o;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if constexpr (DT == GPTQ_BF16)
      o.v[k] = __uint_as_float(k % 2 ? r.w[k / 2] & 0xFFFF0000u : r.w[k / 2] << 16);
    else
      o.v[k] = __uint_as_float(r.w[k]);
  }
  return o;
}

template <int DT>
__device__ __forceinline__ Vals8 load_vals8(const void* row, int64_t c0, int64_t n, bool vec) {
  return vals_of(load_raw8<DT>(row, c0, n, vec));
}

// Stores that do not stay in the caches (8- and 16-byte aligned).
__device__ __forceinline__ void stream_store(void* p, uint2 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(u32x2{v.x, v.y}, reinterpret_cast<u32x2*>(p));
}
__device__ __forceinline__ void stream_store(void* p, uint4 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
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

// 1 / s to within 2^-23 of itself, for a normal s and 1 / s
__device__ __forceinline__ float approx_recip(float s) { return __builtin_amdgcn_rcpf(s); }

// |x| / s so that the instruction's rounding of it (to nearest, ties to even)
// is the rounding of the real quotient: q = q0 + (x - q0 s) rs is a neighbour of the
// quotient, r = x - q s, which one fma gives exactly, says on which side; where it is
// not 0 the last bit is set on that side of q, whose neighbours on a border of the
// format end in 0.
__device__ __forceinline__ float sticky_quotient(float x, float s, float rs) {
  x = fabsf(x);
  const float q0 = x * rs, q = fmaf(fmaf(-q0, s, x), rs, q0), r = fmaf(-q, s, x);
  const uint32_t u = __float_as_uint(q) + (uint32_t)(__float_as_int(r) >> 31);
  return __uint_as_float(r != 0.0f ? u | 1u : u);
}

// 8 codes of x / s, rs = approx_recip(s).  A non-finite value becomes the NaN code
// (the instruction's own result for it).
// Of fp32 values about one in 10^5 lies near a border of the format: x * rs is within
// 2^-22 |x / s| of the quotient, the hardware's rounding of that product lowered and
// raised by 2^-21 brackets the code, and only where the two differ the sticky quotient
// is worked out.  Of bf16 values one in a few hundred lies on a border (a scale
// amax / 448 of 8 significant bits), one or more in nearly every wave: BF16 works it
// out at once.
template <bool BF16>
__device__ __forceinline__ uint2 e4m3_codes8(Vals8 x, float s, float rs) {
  uint32_t c[2];
  bool near = BF16;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = x.v[4 * p + k] * rs;
    int a = 0, b = 0;
    if (!BF16) {
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * 0.99999952f, q[1] * 0.99999952f, a, false);
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * 0.99999952f, q[3] * 0.99999952f, a, true);
      b = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * 1.00000048f, q[1] * 1.00000048f, b, false);
      b = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * 1.00000048f, q[3] * 1.00000048f, b, true);
      near |= a != b;
    }
    c[p] = (uint32_t)a;
  }
  if (near) {
    if (s < 0x1p-60f) {  // lifted, so that no remainder is below the subnormals
#pragma unroll
      for (int k = 0; k < 8; ++k) x.v[k] *= 0x1p64f;
      s *= 0x1p64f;
      rs *= 0x1p-64f;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[k] = sticky_quotient(x.v[4 * p + k], s, rs);
        if (BF16) q[k] = copysignf(q[k], x.v[4 * p + k]);
      }
      int a = 0;
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], a, false);
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
      c[p] = BF16 ? (uint32_t)a : (c[p] & 0x80808080u) | ((uint32_t)a & 0x7F7F7F7Fu);
    }
  }
  return make_uint2(c[0], c[1]);
}

// The 8 integer codes of quant_code(x, scale, zero, maxq), BITS each.  A quotient is at
// most 255 and its form by the reciprocal within 2^-22 of it, 6.1e-5: the integers
// agree unless a half-integer is that near, and then the division decides.
// kRound + an integer below 2^22 has that integer in its low bits, so one fma both
// rounds the quotient and adds the zero-point, and the codes' bit patterns can be
// shifted and added as they are, what kRound adds taken off at the end (modulo 2^32).
template <int BITS>
__device__ __forceinline__ uint2 int_codes8(const Vals8& x, float scale, float zero, float maxq) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  const float rs = approx_recip(scale), off = zero + kRound;
  float c[8], far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = fmaf(x.v[e], rs, off);
    far = fmaxf(far, fabsf(fmaf(x.v[e], rs, off - c[e])));
  }
  // (a NaN has code 0 either way)
  if (!(far < 0.4999f) || !(scale > 0x1p-120f && scale < 0x1p120f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = rintf(__fdiv_rn(x.v[e], scale)) + off;
  }
  constexpr int PER = 32 / BITS;  // codes in a word
  constexpr uint32_t ONES = BITS == 4 ? 0x11111111u : 0x01010101u;
  uint32_t w[8 / PER];
#pragma unroll
  for (int i = 0; i < 8 / PER; ++i) {
    w[i] = 0u - 0x4B400000u * ONES;  // kRound's bit pattern
#pragma unroll
    for (int e = 0; e < PER; ++e)  // (the middle of three passes over a NaN: code 0)
      w[i] += __float_as_uint(__builtin_amdgcn_fmed3f(c[PER * i + e], kRound, kRound + maxq))
              << (BITS * e);
  }
  return make_uint2(w[0], BITS == 4 ? 0u : w[8 / PER - 1]);
}

// Logits col .. col + 7 of n (col may lie up to 7 in front), 16-byte aligned where all
// of them are inside; 0 outside.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_chunk(const char* x, int64_t col, int64_t n) {
  Raw8<DT> o;
  if (col >= 0 && col + 8 <= n) return load_raw8<DT>(x, col, n, true);
  if constexpr (DT == GPTQ_BF16) {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = col + 2 * k;
      o.w[k] = i >= 0 && i < n ? e[i] : 0;
      if (i + 1 >= 0 && i + 1 < n) o.w[k] |= (uint32_t)e[i + 1] << 16;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o.w[k] = col + k >= 0 && col + k < n ? reinterpret_cast<const uint32_t*>(x)[col + k] : 0;
  }
  return o;
}

}  // namespace gptq
