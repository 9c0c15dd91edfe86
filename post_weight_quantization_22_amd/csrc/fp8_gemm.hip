// Product of two e4m3 matrices with block scales:
//   Y[t, r] = sum_b sx[b, t] sw[r / 128, b] sum_{k in block b} x[t, k] w[r, k]
// for X [tokens, n] with a scale per token and 128 columns and W [m, n] with a
// scale per 128 x 128 block, plus R[t, r] where a residual is given.  The inner
// sum runs on the matrix cores from a zero accumulator; the outer sum is fp32 in
// registers, one fma per element and block.
//
// Precision of the inner sum.  The e4m3 matrix instructions add their products in
// groups of 8 that are cut, toward zero, at 2^-13 of the group's largest product
// (measured: beside a product of 2^16 a product below 8 is lost): 1.5e-5 relative
// over normal data.  Turned into bf16 first (exact: e4m3 has 4 significant bits)
// the same operands are summed with fp32 accuracy (1e-8), at half the rate.  So
// fp32 results and all small batches take the bf16 instruction.
#include "fp8.hpp"

namespace gptq {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct GemmArgs {
  const uint8_t* X;
  int64_t ldx, tokens, n;
  const float* sx;  // [nb][lds]
  int64_t lds;
  const uint8_t* W;
  int64_t ldw, m;
  const float* sw;  // [ceil(m / 128)][ldsw]
  int64_t ldsw;
  void* Y;
  int64_t ldy;
  int ybf16;
  const void* R;  // residual of Y's type, or null
  int64_t ldr;
  int64_t nb, ntm, ntt;  // blocks of n, tiles of weight rows and of tokens
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 e4m3 codes as bf16
__device__ __forceinline__ bf16x8 to_bf16(int lo, int hi) {
  union {
    bf16x2 p[4];
    bf16x8 v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return u.v;
}

// The block's products of 16 weight rows and 16 tokens, summed with fp32
// accuracy.  Lane l holds 32 codes of weight row (token) l % 16, the same k on
// both sides; the result's lane l holds weight rows 4 (l / 16) + e, token l % 16.
__device__ __forceinline__ f32x4 block_exact(i32x8 w, i32x8 x) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(w[2 * i], w[2 * i + 1]),
                                                to_bf16(x[2 * i], x[2 * i + 1]), d, 0, 0, 0);
  return d;
}

__device__ __forceinline__ void store4(const GemmArgs& a, int64_t t, int64_t r, f32x4 v) {
  if (t >= a.tokens) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (r + e >= a.m) continue;
    if (a.ybf16) {
      const float res =
          a.R ? (float)reinterpret_cast<const __bf16*>(a.R)[t * a.ldr + r + e] : 0.0f;
      reinterpret_cast<__bf16*>(a.Y)[t * a.ldy + r + e] = (__bf16)(res + v[e]);
    } else {
      const float res = a.R ? reinterpret_cast<const float*>(a.R)[t * a.ldr + r + e] : 0.0f;
      reinterpret_cast<float*>(a.Y)[t * a.ldy + r + e] = res + v[e];
    }
  }
}

// 64 weight rows x 64 tokens a workgroup, 4 waves of 16 weight rows, operands
// straight from global memory.
__global__ __launch_bounds__(256) void fp8_gemm_direct_kernel(GemmArgs a) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int q = lane >> 4, l16 = lane & 15;
  const int64_t row0 = (int64_t)blockIdx.x * 64 + 16 * wv, tok0 = (int64_t)blockIdx.y * 64;
  const int64_t wr = row0 + l16 < a.m ? row0 + l16 : a.m - 1;
  const uint8_t* w = a.W + wr * a.ldw;
  const int64_t swrow = (row0 < a.m ? row0 : a.m - 1) / kFp8Block * a.ldsw;
  f32x4 acc[4];
  for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto ld = [&](const uint8_t* row, int64_t k0) {
    i32x8 v;
    for (int h = 0; h < 2; ++h) {
      const int64_t k = k0 + 32 * q + 16 * h;
      i32x4 u = {0, 0, 0, 0};
      if (k < a.n) u = *reinterpret_cast<const i32x4*>(row + k);
      for (int e = 0; e < 4; ++e) v[4 * h + e] = u[e];
    }
    return v;
  };
  for (int64_t b = 0; b < a.nb; ++b) {
    const i32x8 wf = ld(w, b * kFp8Block);
    const float sw = a.sw[swrow + b];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = tok0 + 16 * j + l16;
      const int64_t tc = t < a.tokens ? t : a.tokens - 1;
      const f32x4 d = block_exact(wf, ld(a.X + tc * a.ldx, b * kFp8Block));
      const float s = a.sx[b * a.lds + tc] * sw;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(d[e], s, acc[j][e]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) store4(a, tok0 + 16 * j + l16, row0 + 4 * q, acc[j]);
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t stream) {
  GemmArgs a;
  a.X = g.X; a.ldx = g.ldx; a.tokens = g.tokens; a.n = g.n;
  a.sx = g.sx; a.lds = g.lds;
  a.W = g.W; a.ldw = g.ldw; a.m = g.m;
  a.sw = g.sw; a.ldsw = g.ldsw;
  a.Y = g.Y; a.ldy = g.ldy; a.ybf16 = g.ydt == GPTQ_BF16;
  a.R = g.R; a.ldr = g.ldr;
  a.nb = ceil_div(g.n, (int64_t)kFp8Block);
  a.ntm = ceil_div(g.m, (int64_t)64);
  a.ntt = ceil_div(g.tokens, (int64_t)64);
  const int64_t per = 65535;
  for (int64_t t0 = 0; t0 < a.ntt; t0 += per) {
    GemmArgs p = a;
    p.X = a.X + t0 * 64 * a.ldx;
    p.sx = a.sx + t0 * 64;
    p.tokens = a.tokens - t0 * 64;
    p.Y = reinterpret_cast<char*>(a.Y) + t0 * 64 * a.ldy * (a.ybf16 ? 2 : 4);
    if (a.R) p.R = reinterpret_cast<const char*>(a.R) + t0 * 64 * a.ldr * (a.ybf16 ? 2 : 4);
    const dim3 grid((unsigned)a.ntm, (unsigned)hmin(a.ntt - t0, per));
    hipLaunchKernelGGL(fp8_gemm_direct_kernel, grid, dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

// ws: codes [tokens][ld16], scales [nb][tokens], then the product's own
static int64_t linear_ldc(int64_t n) { return (n + 127) / 128 * 128; }

size_t fp8_linear_ws_bytes(int64_t tokens, int64_t m, int64_t n) {
  return align_up((size_t)tokens * linear_ldc(n), 256) +
         align_up((size_t)ceil_div(n, (int64_t)kFp8Block) * tokens * 4, 256) +
         fp8_gemm_ws_bytes(tokens, m, n);
}

hipError_t launch_fp8_linear(const void* X, int xdt, int64_t ldx, const Fp8GemmArgs& g, void* ws,
                             hipStream_t stream) {
  Fp8GemmArgs p = g;
  uint8_t* codes = static_cast<uint8_t*>(ws);
  const int64_t ldc = linear_ldc(g.n);
  float* sx = reinterpret_cast<float*>(codes + align_up((size_t)g.tokens * ldc, 256));
  const size_t used = align_up((size_t)g.tokens * ldc, 256) +
                      align_up((size_t)ceil_div(g.n, (int64_t)kFp8Block) * g.tokens * 4, 256);
  const hipError_t e =
      launch_fp8_rows(X, ldx, nullptr, 0, xdt, g.tokens, g.n, codes, ldc, sx, g.tokens, stream);
  if (e != hipSuccess) return e;
  p.X = codes;
  p.ldx = ldc;
  p.sx = sx;
  p.lds = g.tokens;
  p.ws = static_cast<char*>(ws) + used;
  return launch_fp8_gemm(p, stream);
}

}  // namespace gptq
