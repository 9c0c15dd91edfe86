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
// range is a butterfly over them.
#include "fp8.hpp"

namespace gptq {

namespace {

// up to this many tokens a workgroup looks for a later token with the same slot
// by itself; beyond, two small kernels settle the slots' owners first
constexpr int64_t kScanTokens = GPTQ_KV_SMALL_TOKENS;

// the most tokens that the 256 lanes of a workgroup touch (one lane a token, and
// a partial one)
constexpr int kMaxTokensPerGroup = 257;

struct Side {  // one of the two caches and its rows
  char* rows;
  int64_t tstride, hstride;  // elements
  uint8_t* codes;
  float* scales;
  uint8_t* zeros;
  int64_t cpage, cslot, chead;  // codes, bytes
  int64_t ppage, pslot, phead;  // scales and zeros, elements
  int32_t heads, dim, glanes;   // glanes: 8-value chunks per group
  int32_t upt;                  // units (lanes) per token: heads * ng * glanes
  int32_t ng;
  int32_t fmt, vec;
};

struct KvArgs {
  Side s[2];
  const int64_t* slots;
  int64_t tokens, nslots;
  int32_t page_size;
  int32_t* info;
  const int32_t* owner;  // writes: the token that each slot keeps, or null (scan)
};

__device__ __forceinline__ void unit_of(const KvArgs& a, const Side& s, int64_t& t, int& h, int& g,
                                        int& l, bool& live) {
  const int64_t base = (int64_t)blockIdx.x * 256;
  const int64_t t0 = base / s.upt;
  const uint32_t u = (uint32_t)(base - t0 * s.upt) + threadIdx.x;
  const uint32_t dt = u / (uint32_t)s.upt, r = u - dt * (uint32_t)s.upt;
  t = t0 + dt;
  live = t < a.tokens;
  const uint32_t per_head = (uint32_t)(s.ng * s.glanes);
  h = (int)(r / per_head);
  const uint32_t w = r - (uint32_t)h * per_head;
  g = (int)(w / (uint32_t)s.glanes);
  l = (int)(w - (uint32_t)g * s.glanes);
}

// Of two tokens of a call with the same slot the later one stays, as it would
// if they were written one after another: stale[i] says that the i-th token of
// this workgroup has a later namesake.
__device__ __forceinline__ void find_stale(const KvArgs& a, int64_t t0, int nt, int64_t* sl,
                                           int* stale) {
  for (int i = threadIdx.x; i < nt; i += 256) {
    sl[i] = t0 + i < a.tokens ? a.slots[t0 + i] : -1;
    stale[i] = 0;
  }
  __syncthreads();
  for (int64_t u = t0 + 1 + threadIdx.x; u < a.tokens; u += 256) {
    const int64_t v = a.slots[u];
    for (int i = 0; i < nt; ++i)
      if (sl[i] == v && u > t0 + i) stale[i] = 1;
  }
  __syncthreads();
}

template <int LPG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = 1; off < LPG; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, LPG));
  return v;
}

template <int DT, int LPG>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a) {
  const Side& s = a.s[blockIdx.y];
  if (s.codes == nullptr) return;
  const int64_t first = (int64_t)blockIdx.x * 256 / s.upt;
  if (first >= a.tokens) return;
  __shared__ int64_t sl[kMaxTokensPerGroup];
  __shared__ int stale[kMaxTokensPerGroup];
  int64_t t;
  int h, g, l;
  bool live;
  unit_of(a, s, t, h, g, l, live);
  if (a.owner == nullptr) {
    const int nt = (int)(((int64_t)blockIdx.x * 256 + 255) / s.upt - first) + 1;
    find_stale(a, first, nt, sl, stale);
  }
  const int64_t slot = live ? a.slots[t] : -1;
  if (slot >= a.nslots) {
    if (a.info) *a.info = 1;
    live = false;
  }
  if (slot < 0) live = false;
  if (live) {
    if (a.owner) live = a.owner[slot] == (int32_t)t;
    else live = stale[t - first] == 0;
  }
  const int c0 = (g * s.glanes + l) * 8;
  const bool here = live && c0 < s.dim;
  Vals8 x;
#pragma unroll
  for (int k = 0; k < 8; ++k) x.v[k] = 0.0f;
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  if (here)
    x = load_vals8<DT>(s.rows + (t * s.tstride + h * s.hstride) * esz, c0, s.dim, s.vec);
  float scale, zero = 0.0f;
  uint2 code;
  if (s.fmt == GPTQ_KV_E4M3) {
    scale = e4m3_scale(group_max<LPG>(amax_finite8(x)));
    code = e4m3_codes8(x, scale, 1.0f / scale);
  } else {
    const float maxq = s.fmt == GPTQ_KV_INT4 ? 15.0f : 255.0f;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo = fminf(lo, x.v[k]);
      hi = fmaxf(hi, x.v[k]);
    }
    lo = -group_max<LPG>(-lo);
    hi = group_max<LPG>(hi);
    if (s.zeros) minmax_params(lo, hi, maxq, scale, zero);
    else sym_params(fmaxf(-lo, hi), maxq, scale, zero);
    const float rs = 1.0f / scale;
    uint32_t q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = (uint32_t)quant_code_fast(x.v[k], scale, rs, zero, maxq);
    if (s.fmt == GPTQ_KV_INT4) {
      code.x = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) code.x |= q[k] << (4 * k);
    } else {
      code.x = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
      code.y = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
    }
  }
  if (!here) return;
  const int64_t page = slot / a.page_size, off = slot - page * a.page_size;
  uint8_t* row = s.codes + page * s.cpage + off * s.cslot + h * s.chead;
  if (s.fmt == GPTQ_KV_INT4) *reinterpret_cast<uint32_t*>(row + c0 / 2) = code.x;
  else *reinterpret_cast<uint2*>(row + c0) = code;
  if (l == 0) {
    const int64_t p = page * s.ppage + off * s.pslot + h * s.phead + g;
    s.scales[p] = scale;
    if (s.zeros) s.zeros[p] = (uint8_t)zero;
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
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(row) + c0;
    if (vec) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = v[k];
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a) {
  const Side& s = a.s[blockIdx.y];
  if (s.codes == nullptr) return;
  int64_t t;
  int h, g, l;
  bool live;
  unit_of(a, s, t, h, g, l, live);
  const int c0 = (g * s.glanes + l) * 8;
  if (!live || c0 >= s.dim) return;
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  char* out = s.rows + (t * s.tstride + h * s.hstride) * esz;
  float v[8];
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.nslots) {  // padding reads as zeros
    if (slot >= 0 && a.info) *a.info = 1;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    store_vals8<DT>(out, c0, s.vec, v);
    return;
  }
  const int64_t page = slot / a.page_size, off = slot - page * a.page_size;
  const uint8_t* row = s.codes + page * s.cpage + off * s.cslot + h * s.chead;
  const int64_t p = page * s.ppage + off * s.pslot + h * s.phead + g;
  const float scale = s.scales[p];
  if (s.fmt == GPTQ_KV_E4M3) {
    const uint2 c = *reinterpret_cast<const uint2*>(row + c0);
    v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 0);
    v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 1);
    v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 2);
    v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 3);
    v[4] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 0);
    v[5] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 1);
    v[6] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 2);
    v[7] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 3);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= scale;
  } else if (s.fmt == GPTQ_KV_INT4) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(row + c0 / 2);
    const float z = s.zeros ? (float)s.zeros[p] : 8.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = ((float)((c >> (4 * k)) & 15u) - z) * scale;
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(row + c0);
    const float z = s.zeros ? (float)s.zeros[p] : 128.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = ((float)(((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 255u) - z) * scale;
  }
  store_vals8<DT>(out, c0, s.vec, v);
}

inline int pow2_at_least(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

Side side_of(const gptq_kv_cache* c, const KvRows& r, int dt) {
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
  s.heads = c->heads;
  s.dim = c->head_dim;
  // a group as long as the head or longer is the whole head
  const int g = c->group_size > 0 && c->group_size < c->head_dim ? c->group_size : c->head_dim;
  s.glanes = pow2_at_least((g + 7) / 8);
  s.ng = (int)ceil_div(c->head_dim, g);
  s.upt = s.heads * s.ng * s.glanes;
  s.fmt = c->format;
  const int per16 = dt == GPTQ_BF16 ? 8 : 4;
  s.vec = (reinterpret_cast<uintptr_t>(r.p) & 15) == 0 && r.token_stride % per16 == 0 &&
          r.head_stride % per16 == 0;
  return s;
}

KvArgs args_of(const gptq_kv_cache* kc, const gptq_kv_cache* vc, const int64_t* slots,
               int64_t tokens, const KvRows& k, const KvRows& v, int dt, int32_t* info) {
  KvArgs a = {};
  a.s[0] = side_of(kc, k, dt);
  a.s[1] = side_of(vc, v, dt);
  const gptq_kv_cache* c = kc ? kc : vc;
  a.slots = slots;
  a.tokens = tokens;
  a.nslots = c->pages * c->page_size;
  a.page_size = c->page_size;
  a.info = info;
  return a;
}

}  // namespace

size_t kv_write_ws_bytes(int64_t tokens, int64_t slots) {
  return tokens > kScanTokens ? (size_t)slots * 4 : 0;
}

hipError_t launch_kv_write(const KvRows& k, const KvRows& v, int dt, int64_t tokens,
                           const int64_t* slots, const gptq_kv_cache* kc, const gptq_kv_cache* vc,
                           int32_t* info, void* ws, hipStream_t stream) {
  KvArgs a = args_of(kc, vc, slots, tokens, k, v, dt, info);
  if (tokens > kScanTokens) {
    int32_t* owner = static_cast<int32_t*>(ws);
    const dim3 grid((unsigned)ceil_div(tokens, 256));
    hipLaunchKernelGGL(kv_claim_kernel, grid, dim3(256), 0, stream, slots, tokens, a.nslots, owner);
    hipLaunchKernelGGL(kv_settle_kernel, grid, dim3(256), 0, stream, slots, tokens, a.nslots, owner);
    a.owner = owner;
  }
  // one launch for both caches where their groups span the same lanes
  for (int pass = 0; pass < 2; ++pass) {
    KvArgs p = a;
    const int la = a.s[0].codes ? a.s[0].glanes : 0, lb = a.s[1].codes ? a.s[1].glanes : 0;
    int lpg;
    if (la == lb || la == 0 || lb == 0) {
      if (pass == 1) break;
      lpg = la ? la : lb;
    } else {
      p.s[1 - pass] = Side{};
      lpg = pass == 0 ? la : lb;
    }
    const int64_t upt = hmax(p.s[0].upt, p.s[1].upt);
    const dim3 grid((unsigned)ceil_div(tokens * upt, 256), 2);
#define GPTQ_KV(L)                                                                               \
  case L:                                                                                        \
    if (dt == GPTQ_BF16)                                                                         \
      hipLaunchKernelGGL((kv_write_kernel<GPTQ_BF16, L>), grid, dim3(256), 0, stream, p);        \
    else                                                                                         \
      hipLaunchKernelGGL((kv_write_kernel<GPTQ_F32, L>), grid, dim3(256), 0, stream, p);         \
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
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const gptq_kv_cache* kc, const gptq_kv_cache* vc, const int64_t* slots,
                          int64_t tokens, const KvRows& k, const KvRows& v, int dt, int32_t* info,
                          hipStream_t stream) {
  const KvArgs a = args_of(kc, vc, slots, tokens, k, v, dt, info);
  const int64_t upt = hmax(a.s[0].upt, a.s[1].upt);
  const dim3 grid((unsigned)ceil_div(tokens * upt, 256), 2);
  if (dt == GPTQ_BF16) hipLaunchKernelGGL(kv_read_kernel<GPTQ_BF16>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(kv_read_kernel<GPTQ_F32>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace gptq
