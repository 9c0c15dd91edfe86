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
// All three are bound by HBM: each value is read once and its code written once (rows
// of 2048 x 28672 bf16 35 us, 5.1 TB/s, fp32 52 us, 5.7; swiglu of that size 75 us, 3.9, in
// fp32 100 us, 5.3; blocks of 8192 x 28672 bf16 130 us, 5.4 TB/s, fp32
// 208 us, 5.6, of 4096 x 4096 bf16 12.8 us; a copy reaches 5.1 TB/s).
#include "fp8.hpp"

namespace gptq {

namespace {

constexpr int kLanes = kFp8Block / 8;  // lanes that share a row's block

// Codes c0 .. c0 + 7 of a row of n.  STREAM: past the caches, for codes that no kernel
// reads next (weights; 11008 x 4096 29 -> 25 us.  Activations' codes meet their product
// at once: 333 x 1000 x 4112 in all 19.0 us, 19.3 with it).
template <bool STREAM>
__device__ __forceinline__ void store_codes8(uint8_t* row, int64_t c0, int64_t n, bool vec,
                                             uint2 c) {
  if (vec && c0 + 8 <= n) {
    if (STREAM) stream_store(row + c0, c);
    else *reinterpret_cast<uint2*>(row + c0) = c;
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

// 16 lanes per token and block; a workgroup takes 16 tokens of B neighbouring
// blocks, its loads all in flight at once: rows are read in pieces of B * 256
// bytes, and a block's scales are stored for 16 tokens together.  Small inputs are
// bound by the launch and one round trip (333 x 4112: 3.4 us).
template <int DT, bool SWIGLU, int B>
__global__ __launch_bounds__(256) void fp8_rows_kernel(RowsArgs a) {
  const int64_t t = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4);
  const int64_t b0 = (int64_t)blockIdx.x * B;
  if (t >= a.tokens) return;
  const int64_t c0 = b0 * kFp8Block + 8 * (threadIdx.x & 15);
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  const char* row = reinterpret_cast<const char*>(a.X) + t * a.ldx * esz;
  const char* row2 = SWIGLU ? reinterpret_cast<const char*>(a.X2) + t * a.ldx2 * esz : nullptr;
  Raw8<DT> xr[B], ur[SWIGLU ? B : 1];
#pragma unroll
  for (int i = 0; i < B; ++i) {
    xr[i] = load_raw8<DT>(row, c0 + i * kFp8Block, a.n, a.vec);
    if (SWIGLU) ur[i] = load_raw8<DT>(row2, c0 + i * kFp8Block, a.n, a.vec);
  }
#pragma unroll
  for (int i = 0; i < B; ++i) {
    if ((b0 + i) * kFp8Block >= a.n) break;
    Vals8 x = vals_of(xr[i]);
    if (SWIGLU) {
      const Vals8 u = vals_of(ur[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) x.v[k] = silu_times(x.v[k], u.v[k]);
    }
    const float s = e4m3_scale(lanes_max<kLanes>(amax_finite8(x)));
    const uint2 c = e4m3_codes8<DT == GPTQ_BF16 && !SWIGLU>(x, s, approx_recip(s));
    store_codes8<false>(a.codes + t * a.ldc, c0 + i * kFp8Block, a.n, a.vecc, c);
    if ((threadIdx.x & 15) == 0) a.scales[(b0 + i) * a.lds + t] = s;
  }
}

// A workgroup per 128 x 128 block: 16 rows a step, the block's values held in
// registers between the maximum and the rounding.  (Two or four blocks a workgroup, and
// other orders of the blocks over the XCDs, measured slower.)
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
  Raw8<DT> x[8];
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // rows past the end: the last one again, the same maximum
    const int64_t r = min(r0 + 16 * i, m - 1);
    x[i] = load_raw8<DT>(reinterpret_cast<const char*>(W) + r * ldw * esz, c0, n, vec);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, amax_finite8(vals_of(x[i])));
  // (the packed values are kept and widened again below: kept wide they would take
  // twice the registers)
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (uint32_t& w : x[i].w) asm("" : "+v"(w));
  am = lanes_max<kWave>(am);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = am;
  __syncthreads();
  am = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float s = e4m3_scale(am), rs = approx_recip(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < m)
      store_codes8<true>(codes + r * ldc, c0, n, vecc,
                         e4m3_codes8<DT == GPTQ_BF16>(vals_of(x[i]), s, rs));
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
  // two blocks a workgroup where that still gives each CU eight of them (us, one / two
  // / four blocks: 512 x 8192 5.6 / 5.7, 1024 x 8192 8.6 / 8.4, 2048 x 28672 44 / 36 / 38)
  const int64_t nb = ceil_div(n, (int64_t)kFp8Block);
  const int per = ceil_div(nb, (int64_t)2) * ceil_div(tokens, (int64_t)16) >= 2048 ? 2 : 1;
  // 16-token rows of workgroups in y, up to 65535 a launch
  constexpr int64_t kRows = int64_t(65535) * 16;
  for (int64_t t0 = 0; t0 < tokens; t0 += kRows) {
    RowsArgs p = a;
    const int64_t esz = dt == GPTQ_BF16 ? 2 : 4;
    p.tokens = hmin(tokens - t0, kRows);
    p.X = reinterpret_cast<const char*>(X) + t0 * ldx * esz;
    if (X2) p.X2 = reinterpret_cast<const char*>(X2) + t0 * ldx2 * esz;
    p.codes = codes + t0 * ldc;
    p.scales = scales + t0;
    const dim3 grid((unsigned)ceil_div(nb, (int64_t)per), (unsigned)ceil_div(p.tokens, (int64_t)16));
    const dim3 block(256);
#define GPTQ_ROWS(DT, SW)                                                                   \
  if (per == 2) hipLaunchKernelGGL((fp8_rows_kernel<DT, SW, 2>), grid, block, 0, stream, p); \
  else hipLaunchKernelGGL((fp8_rows_kernel<DT, SW, 1>), grid, block, 0, stream, p);
    if (X2) {
      if (dt == GPTQ_BF16) { GPTQ_ROWS(GPTQ_BF16, true) }
      else { GPTQ_ROWS(GPTQ_F32, true) }
    } else {
      if (dt == GPTQ_BF16) { GPTQ_ROWS(GPTQ_BF16, false) }
      else { GPTQ_ROWS(GPTQ_F32, false) }
    }
#undef GPTQ_ROWS
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
