// New keys and values into a paged cache of 8-bit codes with one scale per block of
// tokens and head.
//
// "LLM quantization principles: GPTQ, AWQ, GGUF" (0539edu.com news 6111416), section 2.1
// (q = round(x / scale)) with the max calibrator's scale ("AWQ, MinMax, GPTQ calibration in
// Model Optimizer", gtnt.cn news 115337, section 2).  A block that begins with a new row has
// the scale of its new rows.  A block that rows are added to keeps its scale s0 where that
// covers them, and takes s0 2^k, the smallest that does, where not: the rows that it holds
// are then rounded anew.  Powers of two make that exact in e4m3 but for its subnormals, and
// bound what integers lose, a half step each time of a step twice as large, by one step in all.
//
// A unit of 16, 64 or 256 lanes, by how many values it has, takes one block of one head: its new rows are
// loaded once and held in registers, their largest value is a butterfly over the lanes.  What is read and
// written once bounds it: 2 x 8192 rows of 8 heads of 128 in blocks of 64 take 14.5 us, 3.4 TB/s (int8 14,
// fp32 rows 17, 4.9 TB/s; the copy of as many bytes 9.9); a token for each of 64 sequences 4.3 us in the
// kernel, a chain of four loads (starts, table, scale and rows; the scale's comparison needs both).
#include "kv_blocks.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256;
constexpr int kHold = 4;  // chunks of 8 values that a lane keeps; those behind are read twice

struct WriteSide {
  const char* rows;  // null: that cache is not touched
  int64_t tstride, hstride;  // elements
  int32_t vec;
  BlockCache c;
};

struct BlockWriteArgs {
  WriteSide s[2];
  Sequences q;
  int32_t heads, dim;
  Divisor by_chunks;  // dim / 8
};

// the smallest k >= 0 with need <= s0 2^k, both normal and positive
__device__ __forceinline__ int doublings(float need, float s0) {
  int en, e0;
  const float mn = frexpf(need, &en), m0 = frexpf(s0, &e0);
  return max(en - e0 + (mn > m0 ? 1 : 0), 0);
}

template <int FMT>
__device__ __forceinline__ uint2 rescaled8(uint2 c, float f) {
  uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if constexpr (FMT == GPTQ_KV_E4M3) {
      const float a = __builtin_amdgcn_cvt_f32_fp8((int)w[p], 0) * f;
      const float b = __builtin_amdgcn_cvt_f32_fp8((int)w[p], 1) * f;
      const float d = __builtin_amdgcn_cvt_f32_fp8((int)w[p], 2) * f;
      const float e = __builtin_amdgcn_cvt_f32_fp8((int)w[p], 3) * f;
      int o = 0;
      o = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, o, false);
      o = __builtin_amdgcn_cvt_pk_fp8_f32(d, e, o, true);
      w[p] = (uint32_t)o;
    } else {
      uint32_t o = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = (float)((w[p] >> (8 * k)) & 255u) - 128.0f;
        o |= (uint32_t)(rintf(v * f) + 128.0f) << (8 * k);
      }
      w[p] = o;
    }
  }
  return make_uint2(w[0], w[1]);
}

// W: the unit's threads.  256: the workgroup takes a head of a block; 64: its waves take four heads; 16: each
// wave takes four heads of a block of its own.
template <int DT, int FMT, int W>
__global__ __launch_bounds__(kThreads) void kv_block_write_kernel(BlockWriteArgs a) {
  const WriteSide& s = a.s[blockIdx.z];
  if (s.rows == nullptr) return;
  const Sequences& q = a.q;
  const int task = W == 16 ? blockIdx.x * 4 + (int)(threadIdx.x >> 6) : (int)blockIdx.x;
  int first;
  const Span sp = span_of(q, task, 1, q.by_block, 2, first);
  const int skip = max(sp.rows - sp.length, 0);  // rows in front of position 0
  const int p_new = max(sp.length - sp.rows, 0);
  if (sp.rows <= skip || task < first) return;
  const int64_t begin = (int64_t)(divided(p_new, q.by_block) + (task - first)) * q.block;
  if (begin >= sp.length) return;
  const int b0 = (int)begin;
  const int p0 = max(b0, p_new), p1 = (int)min((int64_t)b0 + q.block, (int64_t)sp.length);
  const int entry = divided(b0, q.by_page), slot0 = b0 - entry * q.page_size;
  const int page = entry < q.width ? q.table[sp.seq * q.ldt + entry] : -1;
  if (page < 0 || page >= q.pages) {
    if (q.info && threadIdx.x % 64 == 0) *q.info = 1;
    return;
  }
  const int h0 = W == 256 ? blockIdx.y : blockIdx.y * 4 + (W == 64 ? (int)threadIdx.x / 64 : 0);  // of the wave
  const int h = W == 16 ? h0 + (int)threadIdx.x % 64 / 16 : h0, lane = threadIdx.x % W;
  if (h0 >= a.heads) return;
  const bool on = W != 16 || h < a.heads;
  const int chunks = a.dim / 8, total = on ? (p1 - p0) * chunks : 0;
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  const char* rows = s.rows + ((int64_t)(sp.start + skip + p0 - p_new) * s.tstride + h * s.hstride) * esz;
  auto load = [&](int u) {
    const int r = divided(u, a.by_chunks);
    return load_raw8<DT>(rows + (int64_t)r * s.tstride * esz, 8 * (u - r * chunks), a.dim, s.vec);
  };
  float* const scale_at = s.c.scales + page * s.c.ppage + divided(slot0, q.by_block) * s.c.pblock + h * s.c.phead;
  const float s0 = on && p0 > b0 ? *scale_at : 0.0f;
  Raw8<DT> held[kHold] = {};
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (lane + k * W < total) held[k] = load(lane + k * W);
  float am = 0.0f;
#pragma unroll
  for (int k = 0; k < kHold; ++k) am = fmaxf(am, amax_finite8(vals_of(held[k])));
  for (int u = lane + kHold * W; u < total; u += W) am = fmaxf(am, amax_finite8(vals_of(load(u))));
  am = lanes_max<(W == 16 ? 16 : 64)>(am);
  if constexpr (W == 256) {  // (the unit is the workgroup: every thread is here)
    __shared__ float part[4];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = am;
    __syncthreads();
    am = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  const float need = FMT == GPTQ_KV_E4M3 ? fmaxf(__fdiv_rn(am, kE4m3Max), 0x1p-126f)
                                         : fmaxf(__fdiv_rn(am, 127.5f), 0x1p-126f);
  float scale = am > 0.0f ? need : 1.0f, f = 1.0f;
  // rows are added to a block (whose scale is a positive number, if it was ever written)
  if (s0 >= 0x1p-126f && is_finite(s0)) {
    const int k = am > 0.0f ? doublings(need, s0) : 0;
    scale = ldexpf(s0, k);
    f = ldexpf(1.0f, -k);
  }
  // codes of head rh that are there, times rf: N threads, several loads of each under way (a workgroup has enough
  // without, and no registers to spare: 2048 rows of 4 sequences 15.0 us, four loads 16.3)
  auto rescale = [&](int rh, float rf, int at, auto n) {
    constexpr int N = decltype(n)::value, AHEAD = N == 256 ? 1 : 4;
    const int before = (p0 - b0) * chunks;
    uint8_t* const codes = s.c.codes + page * s.c.cpage + (int64_t)slot0 * s.c.cslot + rh * s.c.chead;
    for (int u0 = at; u0 < before; u0 += AHEAD * N) {
      uint2* p[AHEAD];
      uint2 c[AHEAD];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int u = u0 + e * N, r = divided(u, a.by_chunks);
        p[e] = u < before ? reinterpret_cast<uint2*>(codes + (int64_t)r * s.c.cslot + 8 * (u - r * chunks)) : nullptr;
        if (p[e]) c[e] = *p[e];
      }
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
        if (p[e]) *p[e] = rescaled8<FMT>(c[e], rf);
    }
  };
  if constexpr (W == 16) {  // (the old rows may be many: the wave takes its heads in turn)
    if (__any(f != 1.0f))
      for (int i = 0; i < 4; ++i) {
        const float rf = __shfl(f, 16 * i);
        if (rf != 1.0f) rescale(h0 + i, rf, threadIdx.x % 64, std::integral_constant<int, 64>{});
      }
  } else if (f != 1.0f) {
    rescale(h, f, lane, std::integral_constant<int, W>{});
  }
  if (lane == 0 && on) *scale_at = scale;
  const float rs = approx_recip(scale);
  uint8_t* const out = s.c.codes + page * s.c.cpage + (int64_t)(slot0 + p0 - b0) * s.c.cslot + h * s.c.chead;
  auto store = [&](int u, const Raw8<DT>& x) {
    const int r = divided(u, a.by_chunks);
    uint2 code;
    if constexpr (FMT == GPTQ_KV_E4M3) code = e4m3_codes8<DT == GPTQ_BF16>(vals_of(x), scale, rs);
    else code = int_codes8<8>(vals_of(x), scale, 128.0f, 255.0f);
    *reinterpret_cast<uint2*>(out + (int64_t)r * s.c.cslot + 8 * (u - r * chunks)) = code;
  };
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (lane + k * W < total) store(lane + k * W, held[k]);
  for (int u = lane + kHold * W; u < total; u += W) store(u, load(u));
}

}  // namespace

hipError_t launch_kv_block_write(const KvRows& k, const KvRows& v, int dt, const KvSequences& seqs,
                                 const gptq_kv_blocks* kb, const gptq_kv_blocks* vb, int32_t* info,
                                 hipStream_t stream) {
  const gptq_kv_blocks* c = kb ? kb : vb;
  BlockWriteArgs a = {};
  const KvRows* rows[2] = {&k, &v};
  const gptq_kv_blocks* cs[2] = {kb, vb};
  const int per16 = dt == GPTQ_BF16 ? 8 : 4;
  for (int i = 0; i < 2; ++i) {
    if (!cs[i]) continue;
    a.s[i].rows = static_cast<const char*>(rows[i]->p);
    a.s[i].tstride = rows[i]->token_stride;
    a.s[i].hstride = rows[i]->head_stride;
    a.s[i].vec = (reinterpret_cast<uintptr_t>(rows[i]->p) & 15) == 0 &&
                 rows[i]->token_stride % per16 == 0 && rows[i]->head_stride % per16 == 0;
    a.s[i].c = block_cache_of(cs[i]);
  }
  a.q = sequences_of(seqs, c, info);
  a.heads = c->heads;
  a.dim = c->head_dim;
  a.by_chunks = divisor_of(c->head_dim / 8);
  // a sequence of n rows touches at most n / block + 2 blocks
  const int64_t tasks = seqs.tokens / c->block + 2 * seqs.seqs;
  // Lanes of a unit, by the values that most have: 16 hold 512 of them, a wave 2048 (8 heads of 128, 8192
  // tokens in blocks of one: a wave each 83 us, 16 lanes 25; a token for each of 1000 sequences: 18 and 10).
  // Few units whose blocks hold many old rows take a wave all the same, for the steps that rescale those
  // (64 sequences, blocks of 64, all rescaled: 16 lanes 21 us, a wave 10).
  const int64_t values = hmin(c->block, ceil_div(seqs.tokens, seqs.seqs)) * c->head_dim;
  const bool small = values <= kHold * 16 * 8 && ((int64_t)c->block * c->head_dim <= kHold * 64 * 8 || tasks * c->heads >= 8192);
  const int lanes = small ? 16 : values <= kHold * 64 * 8 ? 64 : 256;
  const int64_t groups = lanes == 16 ? ceil_div(tasks, 4) : tasks;
  if (!grid_fits(groups, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)groups, (unsigned)ceil_div(c->heads, lanes == 256 ? 1 : 4), 2);
#define GPTQ_KB(DT, F, W) \
  hipLaunchKernelGGL((kv_block_write_kernel<DT, F, W>), grid, dim3(kThreads), 0, stream, a)
#define GPTQ_KB_W(DT, F)                      \
  do {                                        \
    if (lanes == 256) GPTQ_KB(DT, F, 256);    \
    else if (lanes == 64) GPTQ_KB(DT, F, 64); \
    else GPTQ_KB(DT, F, 16);                  \
  } while (0)
  if (dt == GPTQ_BF16) {
    if (c->format == GPTQ_KV_E4M3) GPTQ_KB_W(GPTQ_BF16, GPTQ_KV_E4M3);
    else GPTQ_KB_W(GPTQ_BF16, GPTQ_KV_INT8);
  } else {
    if (c->format == GPTQ_KV_E4M3) GPTQ_KB_W(GPTQ_F32, GPTQ_KV_E4M3);
    else GPTQ_KB_W(GPTQ_F32, GPTQ_KV_INT8);
  }
#undef GPTQ_KB_W
#undef GPTQ_KB
  return hipGetLastError();
}

}  // namespace gptq
