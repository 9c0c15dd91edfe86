// Product of two e4m3 matrices with block scales:
//   Y[t, r] = sum_b sx[b, t] sw[r / 128, b] sum_{k in block b} x[t, k] w[r, k]
// for X [tokens, n] with a scale per token and 128 columns and W [m, n] with a
// scale per 128 x 128 block, plus R[t, r] where a residual is given.  The inner
// sum runs on the matrix cores from a zero accumulator; the outer sum is fp32 in
// registers, one fma per element and block.
//
// Precision of the inner sum.  The e4m3 matrix instructions add their products in
// groups of 8 that are cut, toward zero, at 2^-13 of the group's largest product
// (measured: beside a product of 2^16 a product below 8 is lost).  That is a bias, not
// a rounding, and largest beside an outlier channel: over normal data 1.5e-5 of a
// result, and a gated MLP block's output, whose codes move where the cut moves a
// value over a border of their format, ends 0.003 from exact sums' instead of 0.0017.
// So every product here widens its codes to bf16 (exact: e4m3 has 4 significant bits)
// and takes the bf16 instruction, which sums them with fp32 accuracy (1e-8), at half
// the rate.
#include <type_traits>

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
  int vec4;  // rows of Y and R start on 4-element borders
  float* part;  // [ks][tokens][m], K splits only
  int64_t nb, ntm, ntt;  // blocks of n, tiles of weight rows and of tokens
  // gated products only: the up weights (W holds the gate's) and the codes of
  // silu(gate) * up
  const uint8_t* W2;
  int64_t ldw2;
  const float* sw2;
  int64_t ldsw2;
  uint8_t* codes;
  int64_t ldc;
  float* scales;  // [ceil(m / 128)][ldso]
  int64_t ldso;
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

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

// Y[t, r .. r + 3] = R + v, in one access where a.vec4 allows (rows of Y and R on
// 4-element borders)
__device__ __forceinline__ void store4(const GemmArgs& a, int64_t t, int64_t r, f32x4 v) {
  if (t >= a.tokens || r >= a.m) return;
  const int64_t o = t * a.ldy + r, ro = t * a.ldr + r;
  if (a.vec4 && r + 4 <= a.m) {
    if (a.ybf16) {
      if (a.R) {
        const bf16x4 res = *reinterpret_cast<const bf16x4*>(static_cast<const __bf16*>(a.R) + ro);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += (float)res[e];
      }
      bf16x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (__bf16)v[e];
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.Y) + o) = y;
    } else {
      if (a.R) v += *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.R) + ro);
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.Y) + o) = v;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (r + e >= a.m) continue;
    if (a.ybf16) {
      const float res = a.R ? (float)static_cast<const __bf16*>(a.R)[ro + e] : 0.0f;
      static_cast<__bf16*>(a.Y)[o + e] = (__bf16)(v[e] + res);
    } else {
      const float res = a.R ? static_cast<const float*>(a.R)[ro + e] : 0.0f;
      static_cast<float*>(a.Y)[o + e] = v[e] + res;
    }
  }
}

// a split's partial sums of 4 weight rows, `left` of them inside
__device__ __forceinline__ void store_part(float* p, int64_t left, int64_t m, f32x4 v) {
  if (left >= 4 && m % 4 == 0) {
    *reinterpret_cast<f32x4*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) p[e] = v[e];
}

// ---------------------------------------------------------------------------
// Tiles of TM weight rows x TT tokens, WM x WT waves of MI x NJ 16 x 16 results.
// A block (128 columns, one scale) of both operands arrives by LDS DMA in rows of
// 128 bytes whose 16-byte segments are XOR-swizzled by the row, two buffers: block
// c + 1 is on its way while block c is multiplied.  The results lie transposed
// (weight rows along a lane's registers), so that a lane has one token a column
// tile: one scale product per column tile and block, then one fma an element.
// Rows past the end are re-read from the last one and their results dropped; past
// n the last block's segments re-read the row's last ones and meet zeros in X.
//
// What bounds the 256 x 256 tile are the matrix cores and the widening beside them: a
// block is 4096 matrix cycles of a SIMD and 384 conversions, about 7 cycles each.  So
// that they, 192 KB of operand reads and 64 KB of DMA run beside each other
//  - a wave issues its DMA in pieces between the row tiles (all at once they hold it
//    behind the CU's address unit);
//  - a row tile's column tiles are summed two at a time: with all four sums open the
//    256 registers do not suffice;
//  - no branch comes between a matrix instruction and the reader of its result: past
//    the last block the last one is fetched again into buffers that nothing reads.
// Measured: 2048 x 8192 x 28672 in 256 x 256 tiles 755 us, 1.27 PFLOP/s (a library's
// bf16 product: 1.36 to 1.47); gated 512 x 11008 x 4096 111 us, 0.83 PFLOP/s (172
// tiles for 256 CUs); 512 x 4096 x 11008 in 128 x 128 tiles, two splits, 59 us, 0.78;
// 333 x 1000 x 4112 in 128 x 64 tiles, five splits, 13 us: a few blocks a
// workgroup, most of it the first blocks' latency.
constexpr int kRow = 128;  // bytes of a row of a block
constexpr uint32_t kXcds = 8;

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

struct Bf32 {
  bf16x8 k[4];
};

__device__ __forceinline__ Bf32 widen(i32x8 v) {
  Bf32 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.k[i] = to_bf16(v[2 * i], v[2 * i + 1]);
  return o;
}

// a scalar load (uniform p, memory that this kernel does not write)
__device__ __forceinline__ float const_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

// silu(g) u of the bf16 values nearest to the two products
__device__ __forceinline__ float gated(float g, float u) {
  g = (float)(__bf16)g;
  u = (float)(__bf16)u;
  return g / (1.0f + expf(-g)) * u;
}

// GATED: the tile's first half of rows are gate rows and its second half the up
// rows of the same 128 columns of h = silu(gate) * up, a whole scale block of h, so
// the tile quantizes its part of h itself: each pair of waves exchanges halves of
// their results through LDS, a lane then has 32 of a token's 128 values, and its
// three neighbours at the same token the others.
template <int N>
__device__ __forceinline__ void wait_vm() {  // at most N vector loads outstanding
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

template <int TM, int TT, int WM, int WT, int STAGES, bool GATED = false>
__global__ __launch_bounds__(WM * WT * 64) void fp8_gemm_tile_kernel(GemmArgs a) {
  static_assert(!GATED || (TM == 2 * kFp8Block && WM == 2), "a gate and an up block");
  constexpr int MI = TM / WM / 16, NJ = TT / WT / 16, NW = WM * WT;
  constexpr int W_BYTES = TM * kRow, X_BYTES = TT * kRow, STAGE = W_BYTES + X_BYTES;
  constexpr int PW = TM / 8 / NW, PX = TT / 8 / NW;  // a wave's DMA instructions, 8 rows each
  static_assert(PW % 2 == 0 || PW == 1, "the swizzle of a piece goes by its parity");
  static_assert(PX % 2 == 0 || PX == 1, "the swizzle of a piece goes by its parity");
  static_assert(TM / WM <= kFp8Block && kFp8Block % (TM / WM) == 0, "a wave's rows share a scale");
  static_assert(NJ % 2 == 0, "column tiles go in pairs");
  static_assert(TT % 64 == 0 && TT / 64 <= NW, "a wave fetches the scales of 64 tokens");
  constexpr int NS = TT / 64, LAG = STAGES - 1;  // waves that fetch scales; blocks in flight
  // with three buffers or more the next block is there while one is multiplied, and
  // its first operands are read behind this one's last matrix instructions
  constexpr bool AHEAD = STAGES >= 3;
  __shared__ __align__(16) uint8_t smem[STAGES * STAGE + STAGES * TT * 4];

  // tiles in runs per XCD; within a run, groups of 4 token tiles walked before the
  // next row tile, so that the workgroups of an XCD share both operands in its L2
  // (in 32 bits: a 64-bit division is a long sequence)
  const uint32_t ntm = (uint32_t)a.ntm, ntt = (uint32_t)a.ntt, ntiles = ntm * ntt;
  const uint32_t xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
  const uint32_t per = ntiles / kXcds, rem = ntiles % kXcds;
  if (idx >= per + (xcd < rem ? 1 : 0)) return;
  const uint32_t L = xcd * per + min(xcd, rem) + idx;
  const uint32_t grp = L / (4 * ntm), in = L - grp * 4 * ntm;
  const uint32_t gsz = min(4u, ntt - 4 * grp), rt = in / gsz;
  const int64_t tok0 = (int64_t)(4 * grp + (in - rt * gsz)) * TT;
  const int64_t row0 = (int64_t)rt * (GATED ? TM / 2 : TM);
  // the split's blocks
  const int nb = (int)a.nb, ks = gridDim.y, z = blockIdx.y;
  const int c0 = nb * z / ks, c1 = nb * (z + 1) / ks;  // at most 2^17 blocks, 16 splits

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WT, wt = wv % WT;
  const int q = lane >> 4, l16 = lane & 15;
  const int n = (int)a.n;
  const int rmax = (int)min((int64_t)(GATED ? TM / 2 : TM) - 1, a.m - 1 - row0);
  const int tmax = (int)min((int64_t)TT - 1, a.tokens - 1 - tok0);
  // (gated: the second half of the waves fetches up rows)
  const bool up = GATED && wv >= NW / 2;
  const int64_t ldw = up ? a.ldw2 : a.ldw;
  const uint8_t* wbase = up ? a.W2 + row0 * ldw : a.W + row0 * ldw;
  const int wp0 = (up ? wv - NW / 2 : wv) * PW;
  const uint8_t* xbase = a.X + tok0 * a.ldx;
  const uint32_t lds0 = lds_addr(smem);

  // lane l of a DMA lands on row l / 8, physical segment l % 8 of an 8-row piece,
  // so it loads the logical segment (l % 8) ^ swz(row)
  auto issue = [&](const uint8_t* base, int64_t ld, int last, int piece0, int j, int c,
                   uint32_t dst) {
    const int k0 = c * kRow, row = 8 * (piece0 + j) + (lane >> 3);
    const int sg = min(16 * ((lane & 7) ^ swz(row)), n - 16 - k0);
    lds_dma16(base + k0, __umul24(min(row, last), (uint32_t)ld) + sg, dst + 1024 * (piece0 + j));
  };
  auto issue_x = [&](int j, int c, int buf) {
    issue(xbase, a.ldx, tmax, wv * PX, j, c, lds0 + buf * STAGE + W_BYTES);
  };
  auto issue_w = [&](int j, int c, int buf) {
    issue(wbase, ldw, rmax, wp0, j, c, lds0 + buf * STAGE + 1024 * (wv * PW - wp0));
  };
  // scales of the tile's tokens, 64 by each of the first waves
  const uint32_t so = 4 * (uint32_t)min(64 * wv + lane, tmax);
  auto issue_s = [&](int c, int buf) {
    if (wv < NS)
      lds_dma4(a.sx + tok0 + c * a.lds, so, lds0 + STAGES * STAGE + buf * TT * 4 + 256 * wv);
  };
  const float* sxl = reinterpret_cast<const float*>(smem + STAGES * STAGE);
  const int64_t wrow = row0 + (GATED ? 0 : wm * (TM / WM));
  const int64_t srow = (wrow < a.m ? wrow : a.m - 1) / kFp8Block;
  const float* swp = GATED && wm == 1 ? a.sw2 + srow * a.ldsw2 : a.sw + srow * a.ldsw;

  const int seg0 = (q ^ swz(l16)) << 4, seg1 = ((4 + q) ^ swz(l16)) << 4;
  auto frag = [&](const uint8_t* st, int row) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(st + row * kRow + seg0);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(st + row * kRow + seg1);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };

  f32x4 acc[MI][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int p = 0; p < LAG; ++p) {
    const int c = min(c0 + p, c1 - 1);
    issue_s(c, p);
#pragma unroll
    for (int j = 0; j < PX; ++j) issue_x(j, c, p);
#pragma unroll
    for (int j = 0; j < PW; ++j) issue_w(j, c, p);
  }
  // this wave's DMA is there but for that of the LATER last blocks issued
  auto landed = [&](auto later) {
    constexpr int N = decltype(later)::value;
    if (N > 0 && wv < NS) wait_vm<N * (PX + PW + 1)>();
    else wait_vm<N * (PX + PW)>();
  };
  // the row's end: zeros in X past it
  auto zero_tail = [&](int c, uint8_t* xst) {
    for (int i = threadIdx.x; i < TT * 8; i += NW * 64) {
      const int row = i >> 3, sg = i & 7;
      if (c * kRow + 16 * sg >= n)
        *reinterpret_cast<i32x4*>(xst + row * kRow + ((sg ^ swz(row)) << 4)) = i32x4{0, 0, 0, 0};
    }
    __syncthreads();
  };
  float sw = const_load(swp + c0);
  int buf = 0;
  i32x8 x[NJ], w;
  if constexpr (AHEAD) {
    landed(std::integral_constant<int, LAG - 1>());
    __syncthreads();
    if ((c0 + 1) * kRow > n) zero_tail(c0, smem + W_BYTES);
    w = frag(smem, wm * (TM / WM) + l16);
#pragma unroll
    for (int j = 0; j < NJ; ++j) x[j] = frag(smem + W_BYTES, 16 * (wt * NJ + j) + l16);
  }
  for (int c = c0; c < c1; ++c) {
    // this wave's share of block c (AHEAD: of block c + 1) is there, then everyone's,
    // and block c - 1 has been read
    landed(std::integral_constant<int, AHEAD ? LAG - 2 : LAG - 1>());
    __syncthreads();
    const int after = buf == STAGES - 1 ? 0 : buf + 1;  // the next block's buffer
    const uint8_t* wst = smem + buf * STAGE;
    const uint8_t* xst = smem + buf * STAGE + W_BYTES;
    const uint8_t* wnx = smem + after * STAGE;
    const uint8_t* xnx = smem + after * STAGE + W_BYTES;
    const int ct = AHEAD ? c + 1 : c;
    if (ct < c1 && (ct + 1) * kRow > n)
      zero_tail(ct, smem + (AHEAD ? after : buf) * STAGE + W_BYTES);
    // the block to fetch, and the buffer that block c - 1 has left
    const int cn = min(c + LAG, c1 - 1), nbuf = buf == 0 ? STAGES - 1 : buf - 1;
    const int c2 = min(c + 1, c1 - 1);
    if constexpr (!AHEAD) {
      w = frag(wst, wm * (TM / WM) + l16);
#pragma unroll
      for (int j = 0; j < NJ; ++j) x[j] = frag(xst, 16 * (wt * NJ + j) + l16);
    }
    float s[NJ];
    issue_s(cn, nbuf);
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = sxl[buf * TT + 16 * (wt * NJ + j) + l16] * sw;
    sw = const_load(swp + c2);
    Bf32 xw[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      xw[j] = widen(x[j]);
      if (AHEAD) x[j] = frag(xnx, 16 * (wt * NJ + j) + l16);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const Bf32 ww = widen(w);
      if (i + 1 < MI) w = frag(wst, wm * (TM / WM) + 16 * (i + 1) + l16);
      else if (AHEAD) w = frag(wnx, wm * (TM / WM) + l16);
#pragma unroll
      for (int j = i * PX / MI; j < (i + 1) * PX / MI; ++j) issue_x(j, cn, nbuf);
#pragma unroll
      for (int j = i * PW / MI; j < (i + 1) * PW / MI; ++j) issue_w(j, cn, nbuf);
#pragma unroll
      for (int j0 = 0; j0 < NJ; j0 += 2) {
        f32x4 d[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.k[k], xw[j0 + j].k[k], d[j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j0 + j][e] = fmaf(d[j][e], s[j0 + j], acc[i][j0 + j][e]);
      }
    }
    buf = after;
  }
  wait_vm<0>();  // no DMA into this LDS outlives the workgroup
  if constexpr (GATED) {
    constexpr int NH = NJ / 2;  // column tiles that a wave of a pair quantizes
    __syncthreads();            // every operand has been read
    f32x4* mine = reinterpret_cast<f32x4*>(smem) + (wt * 2 + wm) * MI * NH * 64 + lane;
    const f32x4* theirs = reinterpret_cast<f32x4*>(smem) + (wt * 2 + 1 - wm) * MI * NH * 64 + lane;
    auto give = [&](auto first) {  // the other wave's column tiles
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NH; ++j) mine[(i * NH + j) * 64] = acc[i][first.value + j];
    };
    auto take = [&](auto first, bool gate) {
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        Vals8 h[MI / 2];
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const f32x4 own = acc[i][first.value + j], other = theirs[(i * NH + j) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = gate ? gated(own[e], other[e]) : gated(other[e], own[e]);
            h[i / 2].v[4 * (i % 2) + e] = row0 + 16 * i + 4 * q + e < a.m ? v : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < MI / 2; ++i) am = fmaxf(am, amax_finite8(h[i]));
        am = fmaxf(am, lane_xorf<16>(am));
        am = fmaxf(am, lane_xorf<32>(am));
        const float sc = e4m3_scale(am), rs = approx_recip(sc);
        const int64_t t = tok0 + 16 * (wt * NJ + first.value + j) + l16;
        if (t >= a.tokens) continue;
        if (q == 0) a.scales[row0 / kFp8Block * a.ldso + t] = sc;
#pragma unroll
        for (int i = 0; i < MI / 2; ++i) {
          const uint2 cc = e4m3_codes8<false>(h[i], sc, rs);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t four = k ? cc.y : cc.x;
            const int64_t col = row0 + 16 * (2 * i + k) + 4 * q;
            uint8_t* p = a.codes + t * a.ldc + col;
            if (a.vec4 && col + 4 <= a.m) {
              *reinterpret_cast<uint32_t*>(p) = four;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < a.m) p[e] = (uint8_t)(four >> (8 * e));
            }
          }
        }
      }
    };
    if (wm == 0) give(std::integral_constant<int, NH>());
    else give(std::integral_constant<int, 0>());
    __syncthreads();
    if (wm == 0) take(std::integral_constant<int, 0>(), true);
    else take(std::integral_constant<int, NH>(), false);
    return;
  }
  if (ks > 1) {
    float* part = a.part + z * a.tokens * a.m;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t t = tok0 + 16 * (wt * NJ + j) + l16, r = wrow + 16 * i + 4 * q;
        if (t < a.tokens) store_part(part + t * a.m + r, a.m - r, a.m, acc[i][j]);
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      store4(a, tok0 + 16 * (wt * NJ + j) + l16, wrow + 16 * i + 4 * q, acc[i][j]);
}

// ---------------------------------------------------------------------------
// Decode batches (at most 32 tokens): bound by the weights' HBM stream.  A
// workgroup of 8 waves owns 16 RT weight rows over the whole K range, so nothing
// is split across workgroups and no second kernel joins sums; the waves take
// every eighth block, their sums meet in LDS in wave order.  A lane loads the
// weights and codes of its matrix operand straight into registers (segments q
// and q + 4 of row l % 16 of the block: an instruction covers 64 bytes of 16
// rows), D blocks ahead.  SRC says where the activations come from: codes in
// memory, or bf16 / fp32 rows that the workgroup quantizes into LDS itself, each of its
// loads waiting for those in front of it, the first weights' among them (few tokens:
// every workgroup repeats that).
// Measured: 16 x 8192 x 28672 49 us (4.8 TB/s of weights), 1 x 28672 x 8192 48 us with
// the quantization (4.9), 1 x 4096 x 4096 6.2 us (2.7: launch and one round trip).
constexpr int SRC_CODES = -1;
constexpr int kGemvWaves = 8;

struct GemvArgs {
  GemmArgs g;
  const void* src;  // bf16 or fp32 rows, fused quantization only
  int64_t ldsrc;
  int vec;
};

template <int NT, int RT, int SRC>
__global__ __launch_bounds__(kGemvWaves * 64) void fp8_gemv_kernel(GemvArgs v) {
  const GemmArgs& a = v.g;
  constexpr int D = RT * (SRC == SRC_CODES ? NT : 1) == 1 ? 4 : 2;  // by the registers
  extern __shared__ __align__(16) uint8_t dyn[];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, l16 = lane & 15;
  const int nb = (int)a.nb, n = (int)a.n, T = (int)a.tokens;
  const int64_t row0 = (int64_t)blockIdx.x * 16 * RT;
  const uint8_t* wp[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    wp[i] = a.W + min(row0 + 16 * i + l16, a.m - 1) * a.ldw;
  const float* swp = a.sw + row0 / kFp8Block * a.ldsw;
  // past n the row's last segment is read again and meets zeros in X
  auto load = [&](const uint8_t* p, int c) -> i32x8 {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + min(kRow * c + 16 * q, n - 16));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(p + min(kRow * c + 16 * q + 64, n - 16));
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  struct Blk {
    i32x8 w[RT], x[SRC == SRC_CODES ? NT : 1];
    float sw, sx[SRC == SRC_CODES ? NT : 1];
  };
  const uint8_t* xp[NT];
  const float* sxp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = min(16 * j + l16, T - 1);
    xp[j] = a.X + t * a.ldx;
    sxp[j] = a.sx + t;
  }
  auto fetch = [&](int c) {
    Blk o;
    const int cc = min(c, nb - 1);  // past the end: re-read, never used
#pragma unroll
    for (int i = 0; i < RT; ++i) o.w[i] = load(wp[i], cc);
    o.sw = swp[cc];
    if (SRC == SRC_CODES) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o.x[j] = load(xp[j], cc);
        o.sx[j] = sxp[j][cc * a.lds];
      }
    }
    return o;
  };

  Blk cur[D];
#pragma unroll
  for (int d = 0; d < D; ++d) cur[d] = fetch(wv + kGemvWaves * d);

  // fused: codes [T][nb * 128 + 32], then scales [T][nb]
  const int xrow = nb * kRow + 32;
  float* xs = reinterpret_cast<float*>(dyn + T * xrow);
  if (SRC != SRC_CODES) {
    constexpr int DT = SRC == GPTQ_BF16 ? GPTQ_BF16 : GPTQ_F32;
    constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
    for (int t = 0; t < T; ++t) {
      const char* row = reinterpret_cast<const char*>(v.src) + t * v.ldsrc * esz;
      for (int b = threadIdx.x >> 4; b < nb; b += kGemvWaves * 4) {  // 16 lanes a block
        const Vals8 x = load_vals8<DT>(row, b * kRow + 8 * l16, n, v.vec);
        const float s = e4m3_scale(lanes_max<16>(amax_finite8(x)));
        *reinterpret_cast<uint2*>(dyn + t * xrow + b * kRow + 8 * l16) =
            e4m3_codes8<DT == GPTQ_BF16>(x, s, approx_recip(s));
        if (l16 == 0) xs[t * nb + b] = s;
      }
    }
    __syncthreads();
  }

  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = wv; c < nb; c += kGemvWaves * D) {
    Blk nxt[D];
    if (c + kGemvWaves * D < nb) {
#pragma unroll
      for (int d = 0; d < D; ++d) nxt[d] = fetch(c + kGemvWaves * (D + d));
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int cd = c + kGemvWaves * d;
      if (cd >= nb) break;
      // (before the block's first matrix instruction: with this branch between one
      // and the reader of its result, the compiler left out the wait states that
      // the reader needs on the path that takes the branch)
      if (SRC == SRC_CODES && kRow * (cd + 1) > n) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (kRow * cd + 16 * q + (e < 4 ? 0 : 64) >= n) cur[d].x[j][e] = 0;
      }
      Bf32 w[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) w[i] = widen(cur[d].w[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Bf32 x;
        float s;
        if (SRC == SRC_CODES) {
          x = widen(cur[d].x[j]);
          s = cur[d].sx[j] * cur[d].sw;
        } else {
          const int t = min(16 * j + l16, T - 1);
          const uint8_t* p = dyn + t * xrow + kRow * cd + 16 * q;
          const i32x4 lo = *reinterpret_cast<const i32x4*>(p);
          const i32x4 hi = *reinterpret_cast<const i32x4*>(p + 64);
          x = widen(i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
          s = xs[t * nb + cd] * cur[d].sw;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i].k[k], x.k[k], p, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s, acc[i][j][e]);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) cur[d] = nxt[d];
  }
  // the waves' sums in wave order (the activations' LDS is reused)
  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(dyn);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[((wv * RT + i) * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  if (wv < RT * NT) {
    f32x4 sum = part[wv * 64 + lane];
#pragma unroll
    for (int w = 1; w < kGemvWaves; ++w) {
      const f32x4 p = part[(w * RT * NT + wv) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += p[e];
    }
    const int i = wv / NT, j = wv % NT;
    store4(a, 16 * j + l16, row0 + 16 * i + 4 * q, sum);
  }
}

// Y = R + the splits' partial sums in their order, 4 outputs of a row a lane; the
// loads of up to 8 splits are in flight at once.  Bound by the launch and the
// partials' round trip (333 x 1000, five splits: 3.6 us).
__global__ __launch_bounds__(256) void fp8_gemm_reduce_kernel(GemmArgs a, int ks) {
  const int64_t per_row = (a.m + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * per_row) return;
  const int64_t t = i / per_row, r = 4 * (i - t * per_row);
  const float* p = a.part + t * a.m + r;
  const int64_t step = a.tokens * a.m;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (a.m % 4 == 0) {
    for (int z0 = 0; z0 < ks; z0 += 8) {
      f32x4 u[8];
#pragma unroll
      for (int z = 0; z < 8; ++z)
        if (z0 + z < ks) u[z] = *reinterpret_cast<const f32x4*>(p + (z0 + z) * step);
#pragma unroll
      for (int z = 0; z < 8; ++z)
        if (z0 + z < ks) v += u[z];
    }
  } else {
    for (int z = 0; z < ks; ++z)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e < a.m) v[e] += p[z * step + e];
  }
  store4(a, t, r, v);
}

// Batches that go through fp8_gemv_kernel: 16 tokens, and 32 over weights that a
// few microseconds read (32 x 4096 x 4096: 8.8 us, in narrow tiles 11.8, 32 x 8192 x 4096
// 11.0 and 15.9; but 32 x 4096 x 11008 19.6 and 18.6, 32 x 8192 x 28672 57 and 52, where
// the tiles' deeper DMA counts; 32 x 11008 x 4096 20 either way).
bool by_gemv(int64_t tokens, int64_t m, int64_t n) {
  return tokens <= 16 || (tokens <= 32 && m * n <= int64_t(1) << 25);
}

// 32 weight rows a workgroup (the activations are read, or quantized, half as often)
// where that still gives one to every CU and there are more than 2 tokens (us, 16 and
// 32 rows: 8 x 28672 x 8192 64 and 60, 16 x 8192 x 28672 73 and 54; but
// 1 x 28672 x 8192 57 and 59, quantizing itself 48 and 53)
template <int SRC>
hipError_t launch_gemv(const GemvArgs& v, size_t lds, hipStream_t stream) {
  constexpr bool codes = SRC == SRC_CODES;  // only these come with more than 16 tokens
  const int nt = codes && v.g.tokens > 16 ? 2 : 1, rt = v.g.m >= 8192 && v.g.tokens > 2 ? 2 : 1;
  lds = lds > (size_t)kGemvWaves * rt * nt * 1024 ? lds : (size_t)kGemvWaves * rt * nt * 1024;
  const dim3 grid((unsigned)ceil_div(v.g.m, (int64_t)16 * rt)), block(kGemvWaves * 64);
  if (nt == 1 && rt == 1)
    hipLaunchKernelGGL((fp8_gemv_kernel<1, 1, SRC>), grid, block, lds, stream, v);
  else if (nt == 1)
    hipLaunchKernelGGL((fp8_gemv_kernel<1, 2, SRC>), grid, block, lds, stream, v);
  else if (rt == 1)
    hipLaunchKernelGGL((fp8_gemv_kernel<codes ? 2 : 1, 1, SRC>), grid, block, lds, stream, v);
  else
    hipLaunchKernelGGL((fp8_gemv_kernel<codes ? 2 : 1, 2, SRC>), grid, block, lds, stream, v);
  return hipGetLastError();
}

// Few enough activations that every workgroup quantizes them itself, in at most 4
// rounds of 32 blocks of a token: no kernel before the product, whose launch costs about
// 2 us (us, in one and in two kernels: 1 x 4096 x 4096 5.6 and 7.7, 4 x 4096 x 4096 8.0
// and 8.2, 4 x 1024 x 4096 7.0 and 7.4, 1 x 8192 x 16384 29.7 and 32.2; but
// 8 x 4096 x 2048 8.6 and 7.6, 16 x 2048 x 1024 13.1 and 8.1).
bool quantizes_itself(int64_t tokens, int64_t n) {
  return tokens * ceil_div(n, (int64_t)kFp8Block * 4 * kGemvWaves) <= 4;
}

// How a product is cut: tile, and K splits where the tiles do not reach every CU.
// Measured (us):                              256x256  256x128  128x128 (split)
//   2048 x 8192 x 28672 (256 tiles of 256x256)    755      950      995
//   512 x 22016 x 4096  (172)                     119      139        -
//   1024 x 16640 x 4096 (260, 520 of 256x128)     213      198        -
//   4096 x 11008 x 4096 (688, 1376)               326      395        -
//   512 x 11008 x 4096  (86, 172)                 105       70       78
//   1024 x 4096 x 4096  (256 of 128x128)          104       67       42
//   512 x 4096 x 11008  (128, 2 splits)           259      167       61
// A CU takes one tile after another: a round of 256 x 256 tiles over the CUs takes as
// long as 1.6 rounds of 256 x 128 tiles, and the fewer of the two are taken.
enum Tile { T256x256, T256x128, T128x128, T128x64 };
struct Plan {
  Tile tile;
  int ks;
};

Plan plan_of(int64_t tokens, int64_t m, int64_t n) {
  const int64_t nb = ceil_div(n, (int64_t)kFp8Block);
  auto tiles = [&](int64_t tm, int64_t tt) { return ceil_div(m, tm) * ceil_div(tokens, tt); };
  auto rounds = [&](int64_t tm, int64_t tt) { return ceil_div(tiles(tm, tt), int64_t(256)); };
  if (tiles(128, 128) > 256)
    return {8 * rounds(256, 256) <= 5 * rounds(256, 128) ? T256x256 : T256x128, 1};
  // the narrow tile for narrow batches, and where there is little work for each CU
  // (128 x 128 and 128 x 64: 333 x 1000 x 4112 19.3 and 17.2 us, 128 x 4096 x 4096 21.3
  // and 18.5; but 128 x 8192 x 28672 80 and 101)
  const Tile tile = tokens <= 64 || tiles(128, 128) * nb < 8 * 256 ? T128x64 : T128x128;
  const int64_t t = tiles(128, tile == T128x64 ? 64 : 128);
  return {tile, (int)hmax(1, hmin(hmin(256 / t, nb / 4), 16))};
}

template <int TM, int TT, int WM, int WT, int STAGES, bool GATED = false>
void launch_tile(GemmArgs a, int ks, hipStream_t stream) {
  a.ntm = ceil_div(a.m, (int64_t)(GATED ? TM / 2 : TM));
  a.ntt = ceil_div(a.tokens, (int64_t)TT);
  const int64_t grid = ceil_div(a.ntm * a.ntt, kXcds) * kXcds;
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<TM, TT, WM, WT, STAGES, GATED>),
                     dim3((unsigned)grid, (unsigned)ks), dim3(WM * WT * 64), 0, stream, a);
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t tokens, int64_t m, int64_t n) {
  if (by_gemv(tokens, m, n)) return 0;
  const int ks = plan_of(tokens, m, n).ks;
  return ks == 1 ? 0 : (size_t)ks * tokens * m * 4;
}

static GemmArgs gemm_args(const Fp8GemmArgs& g) {
  GemmArgs a;
  a.X = g.X; a.ldx = g.ldx; a.tokens = g.tokens; a.n = g.n;
  a.sx = g.sx; a.lds = g.lds;
  a.W = g.W; a.ldw = g.ldw; a.m = g.m;
  a.sw = g.sw; a.ldsw = g.ldsw;
  a.Y = g.Y; a.ldy = g.ldy; a.ybf16 = g.ydt == GPTQ_BF16;
  a.R = g.R; a.ldr = g.ldr;
  a.part = static_cast<float*>(g.ws);
  const uintptr_t four = a.ybf16 ? 8 : 16;  // bytes of 4 elements
  a.vec4 = reinterpret_cast<uintptr_t>(g.Y) % four == 0 && g.ldy % 4 == 0 &&
           (!g.R || (reinterpret_cast<uintptr_t>(g.R) % four == 0 && g.ldr % 4 == 0));
  a.nb = ceil_div(g.n, (int64_t)kFp8Block);
  return a;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t stream) {
  const GemmArgs a = gemm_args(g);
  if (by_gemv(g.tokens, g.m, g.n)) return launch_gemv<SRC_CODES>(GemvArgs{a, nullptr, 0, 0}, 0, stream);
  const Plan p = plan_of(g.tokens, g.m, g.n);
  switch (p.tile) {
    case T256x256: launch_tile<256, 256, 2, 4, 2>(a, 1, stream); break;
    case T256x128: launch_tile<256, 128, 2, 4, 3>(a, 1, stream); break;
    case T128x128: launch_tile<128, 128, 2, 4, 4>(a, p.ks, stream); break;
    case T128x64: launch_tile<128, 64, 4, 2, 6>(a, p.ks, stream); break;
  }
  if (p.ks > 1) {
    const int64_t total = g.tokens * ceil_div(g.m, (int64_t)4);
    hipLaunchKernelGGL(fp8_gemm_reduce_kernel, dim3((unsigned)ceil_div(total, (int64_t)256)), dim3(256), 0,
                       stream, a, p.ks);
  }
  return hipGetLastError();
}

// The gated product in one kernel where more than one row of its 256 x 256 tiles is
// needed and they reach more than half of the CUs; else the two products into the
// workspace (bf16 [tokens][m] each) and the quantizer behind them.  In one and in three
// (us): 512 x 11008 x 4096 (172 tiles) 111 and 145, 300 x 11008 x 4096 111 and 141,
// 2048 x 11008 x 4096 332 and 427; but 512 x 8192 x 4096 (128 tiles) 111 and 91,
// 512 x 4096 x 4096 (64) 108 and 67, 256 x 11008 x 4096 110 and 86.
static bool gated_in_one(int64_t tokens, int64_t m) {
  return tokens > 256 && ceil_div(tokens, (int64_t)256) * ceil_div(m, (int64_t)128) > 128;
}

static int64_t gated_ld(int64_t m) { return (m + 7) / 8 * 8; }

size_t fp8_gated_ws_bytes(int64_t tokens, int64_t m, int64_t n) {
  if (gated_in_one(tokens, m)) return 0;
  return 2 * align_up((size_t)tokens * gated_ld(m) * 2, 256) + fp8_gemm_ws_bytes(tokens, m, n);
}

hipError_t launch_fp8_gated(const Fp8GemmArgs& g, const uint8_t* W2, int64_t ldw2,
                            const float* sw2, int64_t ldsw2, uint8_t* codes, int64_t ldc,
                            float* scales, int64_t ldso, hipStream_t stream) {
  if (gated_in_one(g.tokens, g.m)) {
    GemmArgs a = gemm_args(g);
    a.W2 = W2; a.ldw2 = ldw2;
    a.sw2 = sw2; a.ldsw2 = ldsw2;
    a.codes = codes; a.ldc = ldc;
    a.scales = scales; a.ldso = ldso;
    a.vec4 = reinterpret_cast<uintptr_t>(codes) % 4 == 0 && ldc % 4 == 0;
    launch_tile<256, 256, 2, 4, 2, true>(a, 1, stream);
    return hipGetLastError();
  }
  const int64_t ld = gated_ld(g.m);
  const size_t one = align_up((size_t)g.tokens * ld * 2, 256);
  char* ws = static_cast<char*>(g.ws);
  Fp8GemmArgs p = g;
  p.ydt = GPTQ_BF16;
  p.ldy = ld;
  p.R = nullptr;
  p.ws = ws + 2 * one;
  p.Y = ws;
  hipError_t e = launch_fp8_gemm(p, stream);
  if (e != hipSuccess) return e;
  p.W = W2; p.ldw = ldw2;
  p.sw = sw2; p.ldsw = ldsw2;
  p.Y = ws + one;
  e = launch_fp8_gemm(p, stream);
  if (e != hipSuccess) return e;
  return launch_fp8_rows(ws, ld, ws + one, ld, GPTQ_BF16, g.tokens, g.m, codes, ldc, scales, ldso,
                         stream);
}

// ws: codes [tokens][ld16], scales [nb][tokens], then the product's own
static int64_t linear_ldc(int64_t n) { return (n + 127) / 128 * 128; }

size_t fp8_linear_ws_bytes(int64_t tokens, int64_t m, int64_t n) {
  if (quantizes_itself(tokens, n)) return 0;
  return align_up((size_t)tokens * linear_ldc(n), 256) +
         align_up((size_t)ceil_div(n, (int64_t)kFp8Block) * tokens * 4, 256) +
         fp8_gemm_ws_bytes(tokens, m, n);
}

hipError_t launch_fp8_linear(const void* X, int xdt, int64_t ldx, const Fp8GemmArgs& g, void* ws,
                             hipStream_t stream) {
  Fp8GemmArgs p = g;
  if (quantizes_itself(g.tokens, g.n)) {
    GemvArgs v{gemm_args(g), X, ldx, 0};
    const int per16 = xdt == GPTQ_BF16 ? 8 : 4;
    v.vec = (reinterpret_cast<uintptr_t>(X) & 15) == 0 && ldx % per16 == 0;
    const size_t lds = (size_t)(g.tokens * (v.g.nb * (kRow + 4) + 32));
    return xdt == GPTQ_BF16 ? launch_gemv<GPTQ_BF16>(v, lds, stream)
                            : launch_gemv<GPTQ_F32>(v, lds, stream);
  }
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
