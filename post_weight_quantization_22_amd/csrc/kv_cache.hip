// A key/value cache held in few bits: rows are quantized as they are written
// into their slots, and read back as bf16 or fp32.
//
// "LLM quantization principles: GPTQ, AWQ, GGUF" (0539edu.com news 6111416),
// section 2.1 (q = round(x / scale) + zero_point) and "Calibration algorithms
// guide" (bhfrc.com news 5741), section 2.2 (a min and max per group): a row of
// head_dim values of one token and head is cut into groups, each with its own
// fp32 scale (and 8-bit zero-point).  Integers take rtn_minmax's grid, bit for
// bit; e4m3 takes the 8-bit floating-point quantizers' grid, scale = amax / 448.
//
// Both directions are bound by HBM (2 + 1 or 2 + 1/2 bytes a value).  A lane
// owns 8 consecutive values of a row, a group spans LPG lanes of a wave and its
// range is a butterfly over them.  Keys and values of 8 heads of 128: 131072 tokens read
// from e4m3 in 156 us (5.2 TB/s), 8192 tokens written in 4 bits in 14 us (3.0 TB/s: the
// index arithmetic and the codes' rounding fill the issue slots), 5 tokens in 5 us (the
// launch and three dependent round trips: slots, rows, codes).
#include "bits.hpp"
#include "fp8.hpp"

namespace gptq {

namespace {

// Up to this many tokens a workgroup looks for a later token with the same slot by
// itself, T reads of 8 bytes from L2 and a compare for each of its tokens; beyond,
// two small kernels settle the slots' owners first (4.4 us; at 8192 tokens of 8
// heads of 128 the search would cost 11 to 20 us).
constexpr int64_t kScanTokens = GPTQ_KV_SMALL_TOKENS;
constexpr int kSeen = 16;  // slots that a lane compares at a time

constexpr int kThreads = 256;

struct Side {  // one of the two caches and its rows
  char* rows;
  int64_t tstride, hstride;  // elements
  uint8_t* codes;
  float* scales;
  uint8_t* zeros;
  int64_t cpage, cslot, chead;  // codes, bytes
  int64_t ppage, pslot, phead;  // scales and zeros, elements
  int32_t dim, ng;
  int32_t upt;       // units (lanes) per token: heads * ng << lg
  int32_t lg;        // log2 of the lanes per group
  float per_token, per_head;  // 1 / upt, 1 / (ng << lg)
  int32_t fmt, vec;
};

struct KvArgs {
  Side s[2];
  const int64_t* slots;
  int64_t tokens, nslots;
  int32_t page_size, page_shift;  // page_shift: log2 of page_size, -1 if it is no power of two
  int32_t flat;                   // a page's end is the next one's start, in all arrays
  int32_t* info;
  const int32_t* owner;  // writes: the token that each slot keeps, or null (search)
};

// x / d for 0 <= x < 2^21 + 2^10 (a token's lanes and a workgroup's) by the reciprocal:
// (x + 1/2) / d is 1 / (2 d) or more from an integer, nearly 2^-22 of the quotient, and
// the roundings of the reciprocal and the product move it by 2^-23 of itself at most
__device__ __forceinline__ int small_div(int x, float recip) {
  return (int)(((float)x + 0.5f) * recip);
}

struct Unit {
  int64_t t;
  int h, g, l, c0;
};

// Unit k * 256 + tid (V times 8 values) of a workgroup that starts at unit `rest` of
// token t0.
template <int V>
__device__ __forceinline__ Unit unit_of(const Side& s, int64_t t0, int rest, int k) {
  const int u = rest + k * kThreads + (int)threadIdx.x;
  const int dt = small_div(u, s.per_token), r = u - dt * s.upt;
  Unit o;
  o.t = t0 + dt;
  o.h = small_div(r, s.per_head);
  const int w = r - o.h * (s.ng << s.lg);
  o.g = w >> s.lg;
  o.l = w & ((1 << s.lg) - 1);
  o.c0 = 8 * V * w;
  return o;
}

struct Place {
  int64_t code, param;  // of the slot's first head
};

__device__ __forceinline__ Place place_of(const KvArgs& a, const Side& s, int64_t slot) {
  Place p;
  if (a.flat) {
    p.code = slot * s.cslot;
    p.param = slot * s.pslot;
    return p;
  }
  const int64_t page = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page_size;
  const int64_t off = slot - page * a.page_size;
  p.code = page * s.cpage + off * s.cslot;
  p.param = page * s.ppage + off * s.pslot;
  return p;
}

// Of two tokens of a call with the same slot the later one stays, as it would
// if they were written one after another: stale[i] says that the i-th token of
// this workgroup has a later namesake.
__device__ __forceinline__ void find_stale(const KvArgs& a, int64_t t0, int nt, int* sl,
                                           int* stale) {
  auto slot_at = [&](int64_t t) -> int {
    if (t >= a.tokens) return -1;
    const int64_t v = a.slots[t];
    return v < 0 || v >= a.nslots ? -1 : (int)v;
  };
  for (int i = threadIdx.x; i < nt; i += kThreads) {
    sl[i] = slot_at(t0 + i);
    stale[i] = 0;
  }
  __syncthreads();
  // among its own tokens, then all that come behind them
  for (int i = threadIdx.x; i < nt; i += kThreads)
    for (int j = i + 1; j < nt; ++j)
      if (sl[j] == sl[i]) stale[i] = 1;
  for (int64_t u0 = t0 + nt; u0 < a.tokens; u0 += kSeen * kThreads) {
    int seen[kSeen];
#pragma unroll
    for (int k = 0; k < kSeen; ++k) seen[k] = slot_at(u0 + threadIdx.x + k * kThreads);
    for (int i = 0; i < nt; ++i) {
      const int v = sl[i];
      bool hit = false;
#pragma unroll
      for (int k = 0; k < kSeen; ++k) hit |= seen[k] == v;
      if (hit) stale[i] = 1;  // (padding has no namesake that matters)
    }
  }
  __syncthreads();
}

// Group parameters of rtn_minmax's grid from the group's range, bit for bit
// minmax_params': the zero-point's quotient by the reciprocal of span (within
// 2^-21 of it, 255 at most: 1.3e-4), the IEEE division where a half-integer is near.
__device__ __forceinline__ void minmax_params_fast(float lo, float hi, float maxq, float& scale,
                                                   float& zero) {
  if (lo == hi) {
    lo = -1.0f;
    hi = 1.0f;
  }
  const float span = hi - lo, num = __fmul_rn(-lo, maxq);
  scale = __fdiv_rn(span, maxq);
  const float z = num * approx_recip(span);
  zero = rintf(z);
  // (false for a number only: a span whose reciprocal is no normal number divides)
  if (!(fabsf(z - zero) < 0.4998f) || !(span > 0x1p-120f && span < 0x1p120f))
    zero = rintf(__fdiv_rn(num, span));
}

// A lane takes 8 V consecutive values, LPG lanes a group.
template <int DT, int LPG, int V>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvArgs a) {
  const Side& s = a.s[blockIdx.y];
  if (s.codes == nullptr) return;
  const uint32_t base = blockIdx.x * kThreads;  // fewer than 2^31 units in all
  const int64_t t0 = base / (uint32_t)s.upt;
  if (t0 >= a.tokens) return;
  const int rest = (int)(base - (uint32_t)t0 * s.upt);
  // one lane a token at most, and a partial one in front
  __shared__ int sl[kThreads + 1], stale[kThreads + 1];
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  const Unit un = unit_of<V>(s, t0, rest, 0);
  bool live = un.t < a.tokens;
  const int64_t slot = live ? a.slots[un.t] : -1;
  Raw8<DT> xr[V] = {};
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (live && un.c0 + 8 * v < s.dim)
      xr[v] = load_raw8<DT>(s.rows + (un.t * s.tstride + un.h * s.hstride) * esz, un.c0 + 8 * v,
                            s.dim, s.vec);
  if (a.owner == nullptr)
    find_stale(a, t0, small_div(rest + kThreads - 1, s.per_token) + 1, sl, stale);
  if (slot >= a.nslots) {
    if (a.info) *a.info = 1;
    live = false;
  }
  if (slot < 0) live = false;
  if (live) live = a.owner ? a.owner[slot] == (int32_t)un.t : stale[un.t - t0] == 0;
  Vals8 x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = vals_of(xr[v]);
  float scale, zero = 0.0f;
  uint2 code[V];
  if (s.fmt == GPTQ_KV_E4M3) {
    float am = amax_finite8(x[0]);
    if (V == 2) am = fmaxf(am, amax_finite8(x[V - 1]));
    scale = e4m3_scale(lanes_max<LPG>(am));
    const float rs = approx_recip(scale);
#pragma unroll
    for (int v = 0; v < V; ++v) code[v] = e4m3_codes8<DT == GPTQ_BF16>(x[v], scale, rs);
  } else {
    const float maxq = s.fmt == GPTQ_KV_INT4 ? 15.0f : 255.0f;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo = fminf(lo, x[v].v[e]);
        hi = fmaxf(hi, x[v].v[e]);
      }
    lo = -lanes_max<LPG>(-lo);
    hi = lanes_max<LPG>(hi);
    if (s.zeros) minmax_params_fast(lo, hi, maxq, scale, zero);
    else sym_params(fmaxf(-lo, hi), maxq, scale, zero);
#pragma unroll
    for (int v = 0; v < V; ++v)
      code[v] = s.fmt == GPTQ_KV_INT4 ? int_codes8<4>(x[v], scale, zero, maxq)
                                      : int_codes8<8>(x[v], scale, zero, maxq);
  }
  if (!live || un.c0 >= s.dim) return;
  const Place p = place_of(a, s, slot);
  uint8_t* row = s.codes + p.code + un.h * s.chead;
  if (s.fmt == GPTQ_KV_INT4) {
    if (V == 2) stream_store(row + un.c0 / 2, make_uint2(code[0].x, code[V - 1].x));
    else *reinterpret_cast<uint32_t*>(row + un.c0 / 2) = code[0].x;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) stream_store(row + un.c0 + 8 * v, code[v]);
  }
  if (un.l == 0) {
    const int64_t i = p.param + un.h * s.phead + un.g;
    s.scales[i] = scale;
    if (s.zeros) s.zeros[i] = (uint8_t)zero;
  }
}

// owner[slot] = one of the call's tokens with that slot ...
__global__ __launch_bounds__(256) void kv_claim_kernel(const int64_t* slots, int64_t tokens,
                                                       int64_t nslots, int32_t* owner) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= tokens) return;
  const int64_t s = slots[t];
  if (s >= 0 && s < nslots) owner[s] = (int32_t)t;
}
// ... and then the last of them
__global__ __launch_bounds__(256) void kv_settle_kernel(const int64_t* slots, int64_t tokens,
                                                        int64_t nslots, int32_t* owner) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= tokens) return;
  const int64_t s = slots[t];
  if (s >= 0 && s < nslots && owner[s] < (int32_t)t) atomicMax(owner + s, (int32_t)t);
}

template <int DT>
__device__ __forceinline__ void store_vals8(char* row, int c0, bool vec, const float* v) {
  if (DT == GPTQ_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * k]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * k + 1]) << 16;
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + c0;
    if (vec) {
      stream_store(p, make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(row) + c0;
    if (vec) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[k]);
      stream_store(p, make_uint4(w[0], w[1], w[2], w[3]));
      stream_store(p + 4, make_uint4(w[4], w[5], w[6], w[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = v[k];
    }
  }
}

// K units a lane, their loads in flight together.
template <int DT, int K>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvArgs a) {
  const Side& s = a.s[blockIdx.y];
  if (s.codes == nullptr) return;
  const uint32_t base = blockIdx.x * (kThreads * K);
  const int64_t t0 = base / (uint32_t)s.upt;
  const int rest = (int)(base - (uint32_t)t0 * s.upt);
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  const float mid = s.fmt == GPTQ_KV_INT4 ? 8.0f : 128.0f;
  Unit un[K];
  bool live[K];
  int64_t slot[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    un[k] = unit_of<1>(s, t0, rest, k);
    live[k] = un[k].t < a.tokens && un[k].c0 < s.dim;
    slot[k] = live[k] ? a.slots[un[k].t] : -1;
  }
  uint2 code[K];
  float scale[K], zero[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    // padding reads as zeros: code and zero 0, scale 0
    code[k] = make_uint2(0, 0);
    scale[k] = zero[k] = 0.0f;
    if (slot[k] >= a.nslots && a.info) *a.info = 1;
    if (slot[k] < 0 || slot[k] >= a.nslots) continue;
    const Place p = place_of(a, s, slot[k]);
    const uint8_t* row = s.codes + p.code + un[k].h * s.chead;
    const int64_t i = p.param + un[k].h * s.phead + un[k].g;
    if (s.fmt == GPTQ_KV_INT4) code[k].x = *reinterpret_cast<const uint32_t*>(row + un[k].c0 / 2);
    else code[k] = *reinterpret_cast<const uint2*>(row + un[k].c0);
    scale[k] = s.scales[i];
    zero[k] = s.zeros ? (float)s.zeros[i] : mid;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!live[k]) continue;
    const uint2 c = code[k];
    float v[8];
    if (s.fmt == GPTQ_KV_E4M3) {
      v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 0);
      v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 1);
      v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 2);
      v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 3);
      v[4] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 0);
      v[5] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 1);
      v[6] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 2);
      v[7] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= scale[k];
    } else if (s.fmt == GPTQ_KV_INT4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ((float)((c.x >> (4 * e)) & 15u) - zero[k]) * scale[k];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = ((float)(((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 255u) - zero[k]) * scale[k];
    }
    store_vals8<DT>(s.rows + (un[k].t * s.tstride + un[k].h * s.hstride) * esz, un[k].c0, s.vec, v);
  }
}

// (a lane of `width` values)
Side side_of(const gptq_kv_cache* c, const KvRows& r, int dt, int width) {
  Side s = {};
  if (c == nullptr || r.p == nullptr) return s;
  s.rows = static_cast<char*>(r.p);
  s.tstride = r.token_stride;
  s.hstride = r.head_stride;
  s.codes = c->codes;
  s.scales = c->scales;
  s.zeros = c->format == GPTQ_KV_E4M3 ? nullptr : c->zeros;
  s.cpage = c->page_stride; s.cslot = c->slot_stride; s.chead = c->head_stride;
  s.ppage = c->param_page_stride; s.pslot = c->param_slot_stride; s.phead = c->param_head_stride;
  s.dim = c->head_dim;
  // a group as long as the head or longer is the whole head
  const int g = c->group_size > 0 && c->group_size < c->head_dim ? c->group_size : c->head_dim;
  s.lg = log2_at_least((g + width - 1) / width);
  s.ng = (int)ceil_div(c->head_dim, g);
  s.upt = c->heads * (s.ng << s.lg);
  s.per_token = 1.0f / (float)s.upt;
  s.per_head = 1.0f / (float)(s.ng << s.lg);
  s.fmt = c->format;
  const int per16 = dt == GPTQ_BF16 ? 8 : 4;
  s.vec = (reinterpret_cast<uintptr_t>(r.p) & 15) == 0 && r.token_stride % per16 == 0 &&
          r.head_stride % per16 == 0;
  return s;
}

// 16 values a lane when many rows are written, where whole heads and the codes'
// alignment allow it: the group's parameters and the indexes are worked out half as
// often (8192 tokens of 8 heads of 128, 4 bits: 19 -> 17 us; 8 tokens: 5.2 -> 5.9,
// twice the work in a row)
bool takes_16(const gptq_kv_cache* c) {
  return !c || (c->head_dim % 16 == 0 &&
                (c->format != GPTQ_KV_INT4 ||
                 ((reinterpret_cast<uintptr_t>(c->codes) | c->page_stride | c->slot_stride |
                   c->head_stride) % 8) == 0));
}

bool flat(const gptq_kv_cache* c) {
  return !c || (c->page_stride == c->page_size * c->slot_stride &&
                c->param_page_stride == c->page_size * c->param_slot_stride);
}

KvArgs args_of(const gptq_kv_cache* kc, const gptq_kv_cache* vc, const int64_t* slots,
               int64_t tokens, const KvRows& k, const KvRows& v, int dt, int width,
               int32_t* info) {
  KvArgs a = {};
  a.s[0] = side_of(kc, k, dt, width);
  a.s[1] = side_of(vc, v, dt, width);
  const gptq_kv_cache* c = kc ? kc : vc;
  a.slots = slots;
  a.tokens = tokens;
  a.nslots = c->pages * c->page_size;
  a.page_size = c->page_size;
  a.page_shift = log2_exact(c->page_size);
  a.flat = flat(kc) && flat(vc);
  a.info = info;
  return a;
}

// four units a lane where that still gives every CU four workgroups (8 heads of 128, us,
// one and four units: 4096 tokens 7.7 and 8.5, 8192 tokens 12.0 and 11.3, 131072 tokens
// 204 and 168)
int units_a_lane(int64_t units) { return units >= int64_t(1) << 20 ? 4 : 1; }

}  // namespace

size_t kv_write_ws_bytes(int64_t tokens, int64_t slots) {
  return tokens > kScanTokens ? (size_t)slots * 4 : 0;
}

hipError_t launch_kv_write(const KvRows& k, const KvRows& v, int dt, int64_t tokens,
                           const int64_t* slots, const gptq_kv_cache* kc, const gptq_kv_cache* vc,
                           int32_t* info, void* ws, hipStream_t stream) {
  const int wide = tokens > kScanTokens && takes_16(kc) && takes_16(vc) ? 2 : 1;
  KvArgs a = args_of(kc, vc, slots, tokens, k, v, dt, 8 * wide, info);
  if (tokens > kScanTokens) {
    int32_t* owner = static_cast<int32_t*>(ws);
    const dim3 grid((unsigned)ceil_div(tokens, 256));
    hipLaunchKernelGGL(kv_claim_kernel, grid, dim3(256), 0, stream, slots, tokens, a.nslots, owner);
    hipLaunchKernelGGL(kv_settle_kernel, grid, dim3(256), 0, stream, slots, tokens, a.nslots, owner);
    a.owner = owner;
  }
  // one launch for both caches where their groups span the same lanes
  const int la = a.s[0].codes ? 1 << a.s[0].lg : 0, lb = a.s[1].codes ? 1 << a.s[1].lg : 0;
  const bool together = la == lb || la == 0 || lb == 0;
  for (int pass = 0; pass < (together ? 1 : 2); ++pass) {
    KvArgs p = a;
    int lpg = la ? la : lb;
    if (!together) {
      p.s[1 - pass] = Side{};
      lpg = pass == 0 ? la : lb;
    }
    const int64_t units = tokens * hmax(p.s[0].upt, p.s[1].upt);
    const dim3 grid((unsigned)ceil_div(units, (int64_t)kThreads), 2), block(kThreads);
#define GPTQ_KV_LAUNCH(L, V)                                                             \
  if (dt == GPTQ_BF16)                                                                   \
    hipLaunchKernelGGL((kv_write_kernel<GPTQ_BF16, L, V>), grid, block, 0, stream, p);   \
  else                                                                                   \
    hipLaunchKernelGGL((kv_write_kernel<GPTQ_F32, L, V>), grid, block, 0, stream, p);
#define GPTQ_KV(L)                             \
  case L:                                      \
    if (wide == 2) { GPTQ_KV_LAUNCH(L, 2) }    \
    else { GPTQ_KV_LAUNCH(L, 1) }              \
    break;
    switch (lpg) {
      GPTQ_KV(1)
      GPTQ_KV(2)
      GPTQ_KV(4)
      GPTQ_KV(8)
      GPTQ_KV(16)
      GPTQ_KV(32)
      GPTQ_KV(64)
      default: return hipErrorInvalidValue;
    }
#undef GPTQ_KV
#undef GPTQ_KV_LAUNCH
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const gptq_kv_cache* kc, const gptq_kv_cache* vc, const int64_t* slots,
                          int64_t tokens, const KvRows& k, const KvRows& v, int dt, int32_t* info,
                          hipStream_t stream) {
  const KvArgs a = args_of(kc, vc, slots, tokens, k, v, dt, 8, info);
  const int64_t units = tokens * hmax(a.s[0].upt, a.s[1].upt);
  const int per = units_a_lane(units);
  const dim3 grid((unsigned)ceil_div(units, (int64_t)kThreads * per), 2), block(kThreads);
  if (per == 4) {
    if (dt == GPTQ_BF16) hipLaunchKernelGGL((kv_read_kernel<GPTQ_BF16, 4>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((kv_read_kernel<GPTQ_F32, 4>), grid, block, 0, stream, a);
  } else {
    if (dt == GPTQ_BF16) hipLaunchKernelGGL((kv_read_kernel<GPTQ_BF16, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((kv_read_kernel<GPTQ_F32, 1>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace gptq
