// Quantizers to 8-bit floating point (OCP e4m3) with fp32 scales:
//   rows    one scale per token and 128 columns (activations)
//   blocks  one scale per 128 x 128 block (weights)
//   swiglu  silu(gate) * up, quantized as rows without leaving the chip
//
// "AWQ, MinMax, GPTQ calibration in Model Optimizer" (gtnt.cn news 115337),
// section 2: the max calibrator, scale = amax / qmax, which is the 8-bit
// floating-point formats' grid; here amax is taken per block of 128.
//   a = max |x| over the block's finite values
//   s = max(RN32(a / 448), 2^-126), 1 where a = 0
//   code = e4m3 nearest to the real quotient x / s, ties to even
// All three are bound by HBM: each value is read once and its code written once.
#include "fp8.hpp"

namespace gptq {

namespace {

constexpr int kLanes = kFp8Block / 8;  // lanes that share a row's block

// codes c0 .. c0 + 7 of a row of n
__device__ __forceinline__ void store_codes8(uint8_t* row, int64_t c0, int64_t n, bool vec,
                                             uint2 c) {
  if (vec && c0 + 8 <= n) {
    *reinterpret_cast<uint2*>(row + c0) = c;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (c0 + k < n) row[c0 + k] = (uint8_t)((k < 4 ? c.x : c.y) >> (8 * (k & 3)));
}

struct RowsArgs {
  const void* X;   // rows: X; swiglu: gate
  const void* X2;  // swiglu: up
  int64_t ldx, ldx2, tokens, n;
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  int64_t lds;
  int vec, vecc;
};

__device__ __forceinline__ float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// 16 lanes per token and block, a workgroup 16 tokens of one block: the scales
// of a block are stored for 16 tokens together.
template <int DT, bool SWIGLU>
__global__ __launch_bounds__(256) void fp8_rows_kernel(RowsArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t b = blockIdx.y;
  if (t >= a.tokens) return;
  const int64_t c0 = b * kFp8Block + 8 * (threadIdx.x & 15);
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  Vals8 x = load_vals8<DT>(reinterpret_cast<const char*>(a.X) + t * a.ldx * esz, c0, a.n, a.vec);
  if (SWIGLU) {
    const Vals8 u =
        load_vals8<DT>(reinterpret_cast<const char*>(a.X2) + t * a.ldx2 * esz, c0, a.n, a.vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = silu_times(x.v[k], u.v[k]);
  }
  const float s = e4m3_scale(lanes_max<kLanes>(amax_finite8(x)));
  const uint2 c = e4m3_codes8(x, s, approx_recip(s));
  store_codes8(a.codes + t * a.ldc, c0, a.n, a.vecc, c);
  if ((threadIdx.x & 15) == 0) a.scales[b * a.lds + t] = s;
}

// A workgroup per 128 x 128 block: 16 rows a step, the block's values held in
// registers between the maximum and the rounding.
template <int DT>
__global__ __launch_bounds__(256) void fp8_blocks_kernel(const void* __restrict__ W, int64_t m,
                                                         int64_t n, int64_t ldw, int vec,
                                                         uint8_t* __restrict__ codes, int64_t ldc,
                                                         int vecc, float* __restrict__ scales,
                                                         int64_t lds) {
  __shared__ float part[4];
  const int64_t r0 = (int64_t)blockIdx.y * kFp8Block + (threadIdx.x >> 4);
  const int64_t c0 = (int64_t)blockIdx.x * kFp8Block + 8 * (threadIdx.x & 15);
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  Vals8 x[8];
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < m) {
      x[i] = load_vals8<DT>(reinterpret_cast<const char*>(W) + r * ldw * esz, c0, n, vec);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i].v[k] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, amax_finite8(x[i]));
  am = lanes_max<kWave>(am);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = am;
  __syncthreads();
  am = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float s = e4m3_scale(am), rs = approx_recip(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < m) store_codes8(codes + r * ldc, c0, n, vecc, e4m3_codes8(x[i], s, rs));
  }
  if (threadIdx.x == 0) scales[blockIdx.y * lds + blockIdx.x] = s;
}

inline bool aligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

hipError_t launch_fp8_rows(const void* X, int64_t ldx, const void* X2, int64_t ldx2, int dt,
                           int64_t tokens, int64_t n, uint8_t* codes, int64_t ldc, float* scales,
                           int64_t lds, hipStream_t stream) {
  RowsArgs a;
  a.X = X; a.ldx = ldx; a.X2 = X2; a.ldx2 = ldx2;
  a.tokens = tokens; a.n = n;
  a.codes = codes; a.ldc = ldc;
  a.scales = scales; a.lds = lds;
  const int per16 = dt == GPTQ_BF16 ? 8 : 4;
  a.vec = aligned(X, 16) && ldx % per16 == 0 && (!X2 || (aligned(X2, 16) && ldx2 % per16 == 0));
  a.vecc = aligned(codes, 8) && ldc % 8 == 0;
  // tokens <= 2^24 and n <= 2^24: at most 2^20 x 2^17 workgroups, blocks in y up to 65535 a launch
  const int64_t nb = ceil_div(n, (int64_t)kFp8Block);
  const dim3 block(256);
  for (int64_t b0 = 0; b0 < nb; b0 += 65535) {
    RowsArgs p = a;
    const int64_t nbl = hmin(nb - b0, (int64_t)65535);
    const int64_t skip = b0 * kFp8Block;
    p.X = reinterpret_cast<const char*>(X) + skip * (dt == GPTQ_BF16 ? 2 : 4);
    if (X2) p.X2 = reinterpret_cast<const char*>(X2) + skip * (dt == GPTQ_BF16 ? 2 : 4);
    p.codes = codes + skip;
    p.scales = scales + b0 * lds;
    p.n = n - skip;
    const dim3 grid((unsigned)ceil_div(tokens, 16), (unsigned)nbl);
    if (X2) {
      if (dt == GPTQ_BF16) hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_BF16, true>), grid, block, 0, stream, p);
      else hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_F32, true>), grid, block, 0, stream, p);
    } else {
      if (dt == GPTQ_BF16) hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_BF16, false>), grid, block, 0, stream, p);
      else hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_F32, false>), grid, block, 0, stream, p);
    }
  }
  return hipGetLastError();
}

hipError_t launch_fp8_blocks(const void* W, int dt, int64_t m, int64_t n, int64_t ldw,
                             uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                             hipStream_t stream) {
  const int per16 = dt == GPTQ_BF16 ? 8 : 4;
  const int esz = dt == GPTQ_BF16 ? 2 : 4;
  const int vec = aligned(W, 16) && ldw % per16 == 0;
  const int vecc = aligned(codes, 8) && ldc % 8 == 0;
  const int64_t nb = ceil_div(n, (int64_t)kFp8Block), mb = ceil_div(m, (int64_t)kFp8Block);
  for (int64_t r0 = 0; r0 < mb; r0 += 65535) {  // rows of blocks in y, up to 65535 a launch
    const int64_t skip = r0 * kFp8Block;
    const void* Wp = reinterpret_cast<const char*>(W) + skip * ldw * esz;
    const dim3 grid((unsigned)nb, (unsigned)hmin(mb - r0, (int64_t)65535));
    if (dt == GPTQ_BF16)
      hipLaunchKernelGGL(fp8_blocks_kernel<GPTQ_BF16>, grid, dim3(256), 0, stream, Wp, m - skip, n,
                         ldw, vec, codes + skip * ldc, ldc, vecc, scales + r0 * lds, lds);
    else
      hipLaunchKernelGGL(fp8_blocks_kernel<GPTQ_F32>, grid, dim3(256), 0, stream, Wp, m - skip, n,
                         ldw, vec, codes + skip * ldc, ldc, vecc, scales + r0 * lds, lds);
  }
  return hipGetLastError();
}

}  // namespace gptq
