// Attention to a paged cache of 8-bit codes with one scale per block of tokens and head.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = ks[block of j] codes_j, v_j likewise,
// the quantized keys and values ("LLM quantization principles", 0539edu.com news 6111416,
// section 2.1) never written out in 16 bits.
//
// Codes are exact in bf16 (e4m3: 4 significant bits, integers: 8), so both products run on the
// bf16 matrix instruction on bare codes.  A key's scale multiplies its scores behind the first
// product; a value's scale multiplies its probability in front of the second.
//
// A wave takes MT x 16 rows (query heads that share a key head, times new tokens) over tiles of 32
// keys.  Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane holds
// one query row throughout: 8 of its scores a tile, its running maximum and sum, a quarter of its
// output.  The order of the summed index is free in both products, and is chosen so that nothing
// has to change lanes: over head_dim a lane group takes consecutive bytes of a key, which it loads
// 16 at a time; over keys it takes the very keys whose scores it holds.  Columns of V are dealt
// so that a lane loads consecutive bytes of a row; bytes of two keys are brought together by
// v_perm before the conversion.  K and V go from memory to registers, no LDS in between.
//
// The four waves of a workgroup take tiles in turn, their results are joined through LDS;
// where rows are few, the keys are also split over workgroups and joined by a second kernel.
//
// With few rows the codes' stream bounds it: 16 sequences of 12000 tokens, 64 query heads on 8 of 128, e4m3,
// a row each: 76 us and 5 for the join, 4.7 TB/s (1 x 131072: 59 and 6, 4.1, integers too).  A small step, 5
// sequences of 300 tokens on 32 heads, 9 us: a chain of four round trips (starts, table, keys and
// values, the sum), the launch, the join of the waves.  fp32 rows (three terms each, three times the
// products) of 13 sequences of up to 2777 in pages of 100, windows of 1000: 14.5 us and 4.
#include "kv_blocks.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 32;  // keys
constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

union Frag {  // 8 operands of one lane
  bf16x8 v;
  bf16x2 p[4];
  uint32_t w[4];
};

struct AttnArgs {
  const char* q;
  char* out;
  int64_t qt, qh, ot, oh;  // strides, elements
  float* lse;
  Sequences s;
  BlockCache k, v;
  int32_t heads, group, dim;  // group: query heads of a key head
  int32_t causal, window, qvec, ovec;
  float scale;  // times log2(e)
  int32_t splits;
  Divisor by_rows, by_group, by_splits;  // rows of a tile, query heads of a key head
  float* parts;     // [task][head][split][rows][DP]
  float2* stats;    // [task][head][split][rows]: maximum, sum
};

// Two codes of a word as bf16: bytes 2 hi and 2 hi + 1.
template <int FMT, bool HI>
__device__ __forceinline__ bf16x2 pair_of(uint32_t w) {
  if constexpr (FMT == GPTQ_KV_E4M3) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
  } else {  // bytes are signed here (the caller has flipped their top bits)
    bf16x2 r;
    r[0] = (__bf16)(float)(int8_t)(w >> (HI ? 16 : 0));
    r[1] = (__bf16)(float)(int8_t)(w >> (HI ? 24 : 8));
    return r;
  }
}

template <int FMT>
__device__ __forceinline__ uint32_t signed_codes(uint32_t w) {
  return FMT == GPTQ_KV_INT8 ? w ^ 0x80808080u : w;
}

// bit 7 of each byte of w that is e4m3's NaN (the other bits: anything)
__device__ __forceinline__ uint32_t nan_marks(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }

// bytes of w that are e4m3's NaN, as 0xFF
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((nan_marks(w) & 0x80808080u) >> 7) * 255u;
}

__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// TERMS bf16 numbers whose sum is x (1: rounded; 3: 24 bits and more)
template <int TERMS>
__device__ __forceinline__ void split_terms(float x, __bf16 (&t)[TERMS]) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    t[k] = (__bf16)x;
    x = x - (float)t[k];
    if (!is_finite(x)) x = 0.0f;  // an infinity or a NaN is in its first term
  }
}

// All ones where bit k of `bits` is set, else 0 (masks of lanes in scalar registers, one for each
// of so many values, would crowd out what is kept there).
__device__ __forceinline__ uint32_t spread_bit(uint32_t bits, int k) { return (uint32_t)((int32_t)(bits << (31 - k)) >> 31); }
__device__ __forceinline__ float kept(float x, uint32_t mask) { return __uint_as_float(__float_as_uint(x) & mask); }
__device__ __forceinline__ float kept_or_neg_inf(float x, uint32_t mask) {
  return __uint_as_float((__float_as_uint(x) & mask) | (0xFF800000u & ~mask));
}

// The largest of 8 (written out: the compiler would first turn each that went through a mask into a
// quiet number, 8 instructions more).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  __asm__("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float max_of(const f32x4 (&s)[2]) {
  return max3(max3(max3(s[0][0], s[0][1], s[0][2]), s[0][3], s[1][0]), s[1][1], max3(s[1][2], s[1][3], s[1][3]));
}

// Which of the keys base + 16 u + i (u < 2, i < 4; bit 4 u + i) lie in lo .. hi.
__device__ __forceinline__ uint32_t keys_between(int base, int lo, int hi) {
  uint32_t bits = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int to = min(max(hi - base - 16 * u + 1, 0), 4), from = min(max(lo - base - 16 * u, 0), 4);
    bits |= (((1u << to) - 1) & ~((1u << from) - 1)) << (4 * u);
  }
  return bits;
}

// The weights of one row, keys 16 u + 4 g + i, as the second product's operands: e^(s - base) times
// the values' scales; their sum is added to l.  MASKED: a weight whose key is not seen is 0, whatever
// its scale is (apart from the other form, which costs half as many instructions).
template <bool MASKED, int TERMS>
__device__ __forceinline__ void weights_of(const f32x4 (&s)[2], const float (&vs)[2][4], uint32_t seen, float base,
                                           float& l, Frag (&p)[TERMS]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // pairs
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int u = k / 2, i = 2 * (k % 2) + e;
      const float w = __builtin_amdgcn_exp2f(s[u][i] - base);
      l += w;
      x[e] = w * vs[u][i];
      if (MASKED) x[e] = kept(x[e], spread_bit(seen, 4 * u + i));
    }
    if constexpr (TERMS == 1) {
      p[0].p[k][0] = (__bf16)x[0];
      p[0].p[k][1] = (__bf16)x[1];
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        __bf16 t[TERMS];
        split_terms<TERMS>(x[e], t);
#pragma unroll
        for (int n = 0; n < TERMS; ++n) p[n].p[k][e] = t[n];
      }
    }
  }
}

struct TileRows {  // what a workgroup works on
  Span sp;
  int row0, rows;  // of the sequence's rows * group
  int lo, hi;      // its keys, lo a multiple of 16
  bool bad;        // keys that the table has no entry for
};

__device__ __forceinline__ TileRows tile_rows(const AttnArgs& a, int task, int per) {
  TileRows t;
  int first;
  t.sp = span_of(a.s, task, a.group, a.by_rows, 1, first);
  t.row0 = (task - first) * per;
  t.rows = task < first ? 0 : max(min(per, t.sp.rows * a.group - t.row0), 0);
  // positions of the first and last row; keys that any of them sees
  const int base = t.sp.length - t.sp.rows;
  t.hi = t.sp.length;
  t.lo = 0;
  if (t.rows > 0 && a.causal) {
    const int p0 = base + divided(t.row0, a.by_group), p1 = base + divided(t.row0 + t.rows - 1, a.by_group);
    t.hi = max(min(t.hi, p1 + 1), 0);
    if (a.window > 0) t.lo = max(max(p0, 0) - a.window + 1, 0) & ~15;  // (a row in front of position 0 sees nothing)
  }
  t.bad = t.hi > a.s.room;
  t.hi = min(t.hi, a.s.room);
  return t;
}

// a split's keys: whole rounds of the workgroup's waves (counted in 32 bits: a 64-bit comparison has
// no scalar form, and what hangs on it would be held in every lane)
__device__ __forceinline__ void split_keys(const AttnArgs& a, const TileRows& t, int i, int& k0, int& k1) {
  const uint32_t n = (uint32_t)max(t.hi - t.lo, 0);
  const uint32_t per = ((uint32_t)divided((int)n, a.by_splits) + kTile * kWaves) & ~(uint32_t)(kTile * kWaves - 1);
  const uint32_t b = (uint32_t)i * per;  // (at most n + 64 rounds)
  k0 = t.lo + (int)min(n, b);
  k1 = t.lo + (int)min(n, b + per);
}

// N values of row rr (of rows * group) of the sequence from column c on, and its statistics.
template <int N, bool F32>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const Span& sp, int head, int rr, int c,
                                           const float* o, float m, float l) {
  const int r = divided(rr, a.by_group);
  const int64_t row = sp.start + r;
  const int qh = head * a.group + (rr - r * a.group);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // (no key: zeros)
  if (c < a.dim) {
    char* p = a.out + (row * a.ot + qh * a.oh + c) * (F32 ? 4 : 2);
    if constexpr (F32) {
      float* f = reinterpret_cast<float*>(p);
      if (a.ovec) {
#pragma unroll
        for (int k = 0; k < N; k += 4)
          *reinterpret_cast<float4*>(f + k) = make_float4(o[k] * inv, o[k + 1] * inv, o[k + 2] * inv, o[k + 3] * inv);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = o[k] * inv;
      }
    } else {
      uint16_t* f = reinterpret_cast<uint16_t*>(p);
      uint32_t w[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) w[k] = bf16_bits(o[2 * k] * inv) | bf16_bits(o[2 * k + 1] * inv) << 16;
      if (a.ovec) {
        if constexpr (N == 4) *reinterpret_cast<uint2*>(f) = make_uint2(w[0], w[1]);
        else {
#pragma unroll
          for (int k = 0; k < N / 8; ++k)
            *reinterpret_cast<uint4*>(f + 8 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
      }
    }
  }
  if (a.lse && c == 0)
    a.lse[row * (int64_t)(a.heads * a.group) + qh] = l == 0.0f ? kNegInf : m * kLn2 + logf(l);
}

// The same for a split: its part in the workspace.
template <int N, int DP>
__device__ __forceinline__ void store_part(const AttnArgs& a, int64_t at, int c, const float* v, float m, float l) {
  float* d = a.parts + at * DP + c;
#pragma unroll
  for (int n = 0; n < N; n += 4) *reinterpret_cast<float4*>(d + n) = make_float4(v[n], v[n + 1], v[n + 2], v[n + 3]);
  if (c == 0) a.stats[at] = make_float2(m, l);
}

// One of the two caches, at the workgroup's head.
struct Side {
  const uint8_t* codes;
  const float* scales;
  int64_t cpage, ppage;
  int32_t cslot, pblock;
};

__device__ __forceinline__ Side side_of(const BlockCache& c, int head) {
  return Side{c.codes + head * c.chead, c.scales + head * c.phead, c.cpage, c.ppage, (int32_t)c.cslot, (int32_t)c.pblock};
}

// A zero that the compiler takes for a lane's own: loads that all lanes make of one address go the
// vector loads' way, and are waited for where they are used, in order with the others (a scalar
// load is waited for as soon as its value is put anywhere).
__device__ __forceinline__ int lane_zero() {
  int z = 0;
  __asm__ volatile("" : "+v"(z));
  return z;
}

// Where the 32 keys of a tile lie.  EVEN: the 16 keys of a half tile share a page and a block, and
// all of this is the same in every lane; else lane i (and i + 32) knows key i.  A key behind the
// end, or whose page is none, has page 0 and is marked as such: its loads go somewhere and count
// for nothing, so that no load depends on a branch.
template <bool EVEN>
struct Place {
  static constexpr int N = EVEN ? 2 : 1;
  int page[N], slot[N];
  bool there[N];
};

// The table's entries for the tile at k0 (loads under way until place_of).
template <bool EVEN>
struct Entries {
  int v[EVEN ? 2 : 1];
};

template <bool EVEN>
__device__ __forceinline__ Entries<EVEN> entries_of(const AttnArgs& a, const int32_t* table, int k0, int ke, int zero) {
  Entries<EVEN> e;
#pragma unroll
  for (int u = 0; u < Place<EVEN>::N; ++u) {
    const int kk = min(EVEN ? k0 + 16 * u : k0 + ((int)threadIdx.x & 31), ke - 1);
    e.v[u] = table[min(divided(kk, a.s.by_page), a.s.width - 1) + zero];
  }
  return e;
}

template <bool EVEN>
__device__ __forceinline__ Place<EVEN> place_of(const AttnArgs& a, const Entries<EVEN>& e, int k0, int ke, bool& bad) {
  Place<EVEN> p;
#pragma unroll
  for (int u = 0; u < Place<EVEN>::N; ++u) {
    const int key = EVEN ? k0 + 16 * u : k0 + ((int)threadIdx.x & 31), kk = min(key, ke - 1);
    const int entry = divided(kk, a.s.by_page);
    const int page = EVEN ? __builtin_amdgcn_readfirstlane(e.v[u]) : e.v[u];
    const bool ok = entry < a.s.width && (uint32_t)page < (uint32_t)a.s.pages;
    bad = bad || (key < ke && !ok);
    p.there[u] = key < ke && ok;
    p.page[u] = ok ? page : 0;
    p.slot[u] = kk - entry * a.s.page_size;
    if (EVEN) p.slot[u] &= ~15;  // (kk may have been moved to the last key)
  }
  return p;
}

// The scales of a lane's 8 keys, 16 u + 4 g + i: EVEN: of the half tiles; else of key i in lane i.
template <bool EVEN>
struct Scales {
  float v[EVEN ? 2 : 1];
};
template <bool EVEN>
__device__ __forceinline__ Scales<EVEN> scales_of(const AttnArgs& a, const Side& c, const Place<EVEN>& p, int zero) {
  Scales<EVEN> s;
#pragma unroll
  for (int u = 0; u < Place<EVEN>::N; ++u)
    s.v[u] = c.scales[p.page[u] * c.ppage + (int64_t)divided(p.slot[u], a.s.by_block) * c.pblock + zero];
  return s;
}
template <bool EVEN>
__device__ __forceinline__ void spread(const Scales<EVEN>& s, float (&v)[2][4]) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (EVEN) v[u][i] = s.v[u];
      else v[u][i] = __shfl(s.v[0], 16 * u + 4 * (((int)threadIdx.x & 63) >> 4) + i);
    }
}

// The codes of key row 16 u + r in cache c.
template <bool EVEN>
__device__ __forceinline__ const uint8_t* row_of(const Side& c, const Place<EVEN>& p, int u, int r) {
  if constexpr (EVEN) {
    return c.codes + (p.page[u] * c.cpage + (int64_t)p.slot[u] * c.cslot) + (uint32_t)(r * c.cslot);
  } else {
    const int page = __shfl(p.page[0], 16 * u + r), slot = __shfl(p.slot[0], 16 * u + r);
    return c.codes + (page * c.cpage + (int64_t)slot * c.cslot);
  }
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (W == 1) w[0] = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  }
}

// 8 codes as an operand of the first product
template <int FMT>
__device__ __forceinline__ Frag frag_of(uint32_t w0, uint32_t w1) {
  Frag f;
  w0 = signed_codes<FMT>(w0);
  w1 = signed_codes<FMT>(w1);
  f.p[0] = pair_of<FMT, false>(w0);
  f.p[1] = pair_of<FMT, true>(w0);
  f.p[2] = pair_of<FMT, false>(w1);
  f.p[3] = pair_of<FMT, true>(w1);
  return f;
}

// Byte b of each of 8 words (the lane's keys): an operand of the second product
template <int FMT, int B>
__device__ __forceinline__ Frag column_of(const uint32_t (&two)[2][4]) {
  Frag f;
#pragma unroll
  for (int k = 0; k < 4; ++k) f.p[k] = pair_of<FMT, (B & 1) != 0>(two[B / 2][k]);
  return f;
}
template <int FMT, typename F>
__device__ __forceinline__ void columns_of(const uint32_t (&w)[8], F&& use) {
  uint32_t two[2][4];  // bytes 0, 1 and 2, 3 of keys 2 k and 2 k + 1
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = signed_codes<FMT>(w[2 * k]), y = signed_codes<FMT>(w[2 * k + 1]);
    two[0][k] = __builtin_amdgcn_perm(y, x, 0x05010400u);
    two[1][k] = __builtin_amdgcn_perm(y, x, 0x07030602u);
  }
  use(0, column_of<FMT, 0>(two));
  use(1, column_of<FMT, 1>(two));
  use(2, column_of<FMT, 2>(two));
  use(3, column_of<FMT, 3>(two));
}

// Queries of 16 rows: lane (row c16, group g) holds columns 64 (s / 2) + 16 g + 8 (s % 2) .. + 7 of
// step s, as the keys' rows are loaded.
template <int STEPS, int TERMS>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const TileRows& t, int head, int r16, int g,
                                             Frag (&q)[STEPS][TERMS], int& pos) {  // (r16: the row in the tile)
  constexpr bool F32 = TERMS == 3;
  constexpr int DT = F32 ? GPTQ_F32 : GPTQ_BF16;
  // (rows behind the tile's last are its first one's: nothing of them is stored)
  const int rr = t.row0 + (r16 < t.rows ? r16 : 0), r = divided(rr, a.by_group);
  pos = t.sp.length - t.sp.rows + r;
  const char* p = a.q + ((int64_t)(t.sp.start + r) * a.qt + (int64_t)(head * a.group + (rr - r * a.group)) * a.qh) * (F32 ? 4 : 2);
  Raw8<DT> raw[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = 64 * (s / 2) + 16 * g + 8 * (s % 2);
    const bool in = c < a.dim;  // (head_dim is a multiple of 16)
    const char* x = p + (in ? c : 0) * (F32 ? 4 : 2);
    if (a.qvec) {
#pragma unroll
      for (int k = 0; k < (F32 ? 2 : 1); ++k) load_words<4>(reinterpret_cast<const uint8_t*>(x) + 16 * k, raw[s].w + 4 * k);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (F32) raw[s].w[k] = reinterpret_cast<const uint32_t*>(x)[k];
        else if (k % 2 == 0) raw[s].w[k / 2] = reinterpret_cast<const uint16_t*>(x)[k] | (uint32_t)reinterpret_cast<const uint16_t*>(x)[k + 1] << 16;
      }
    }
    if (!in) raw[s] = {};
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        __bf16 tm[TERMS];
        split_terms<TERMS>(__uint_as_float(raw[s].w[e]), tm);
#pragma unroll
        for (int k = 0; k < TERMS; ++k) q[s][k].v[e] = tm[k];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) q[s][0].w[e] = raw[s].w[e];
    }
  }
}

// DP: head_dim rounded up to 64, 128 or 256.  fp32 rows: queries and probabilities as three
// bf16 terms each.
template <int DP, int FMT, bool F32, int MT, bool EVEN>
__global__ __launch_bounds__(kThreads, F32 || DP == 256 ? 1 : MT == 1 ? 3 : 2) void kv_attention_kernel(AttnArgs a) {
  constexpr int TERMS = F32 ? 3 : 1;
  constexpr int STEPS = DP / 32;   // of the first product
  constexpr int NT = DP / 16;      // tiles of 16 columns of the output; bytes of a V row in a lane
  constexpr int KW = DP / 16;      // words of a K row in a lane (4 lanes a row)
  constexpr int VW = DP / 64;      // words of a V row in a lane (16 lanes a row)
  constexpr int LD = DP + 4;
  __shared__ __align__(16) float so[kWaves][16][LD];
  __shared__ float sm[kWaves][16], sl[kWaves][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int head = blockIdx.y;
  const TileRows t = tile_rows(a, (int)blockIdx.x, 16 * MT);
  if (t.rows <= 0) return;
  int kb, ke;
  split_keys(a, t, (int)blockIdx.z, kb, ke);
  const int32_t* table = a.s.table + t.sp.seq * a.s.ldt;
  const int kfirst = kb + kTile * wave;
  const Side kc = side_of(a.k, head), vc = side_of(a.v, head);
  bool bad = t.bad;

  const int zero = lane_zero();
  uint32_t kraw[2][KW], vraw[VW][8];
  Scales<EVEN> ksc, vsc;
  // (columns behind head_dim: the row's first ones, whose queries and outputs are not there)
  int ck[KW / 4];
#pragma unroll
  for (int p = 0; p < KW / 4; ++p) ck[p] = 64 * p + 16 * g < a.dim ? 64 * p + 16 * g : 0;
  const int cv = NT * c16 < a.dim ? NT * c16 : 0;
  auto load_keys = [&](const Place<EVEN>& p) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* row = row_of<EVEN>(kc, p, u, c16);
#pragma unroll
      for (int w = 0; w < KW / 4; ++w) load_words<4>(row + ck[w], kraw[u] + 4 * w);
    }
    ksc = scales_of<EVEN>(a, kc, p, zero);
  };
  auto load_values = [&](const Place<EVEN>& p) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[VW];
        load_words<VW>(row_of<EVEN>(vc, p, u, 4 * g + i) + cv, w);
#pragma unroll
        for (int x = 0; x < VW; ++x) vraw[x][4 * u + i] = w[x];
      }
    vsc = scales_of<EVEN>(a, vc, p, zero);
  };

  Place<EVEN> now = {};
  Entries<EVEN> ahead = {};
  if (kfirst < ke) {
    const Entries<EVEN> e = entries_of<EVEN>(a, table, kfirst, ke, zero);
    ahead = entries_of<EVEN>(a, table, kfirst + kTile * kWaves, ke, zero);
    now = place_of<EVEN>(a, e, kfirst, ke, bad);
    load_keys(now);
    load_values(now);
  }
  Frag q[MT][STEPS][TERMS];
  int pos[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) load_queries<STEPS, TERMS>(a, t, head, 16 * mt + c16, g, q[mt], pos[mt]);
  // (bounds of the tile's rows, for its masks)
  const int pos_first = t.sp.length - t.sp.rows + divided(t.row0, a.by_group);
  const int pos_last = t.sp.length - t.sp.rows + divided(t.row0 + t.rows - 1, a.by_group);

  f32x4 o[NT][MT];
  float m[MT], l[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = kNegInf;
    l[mt] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // A tile's registers are refilled as soon as they have been used: the next keys travel during the
  // softmax and the second product, the next values during the first product behind it, the
  // places two tiles ahead.
  for (int k0 = kfirst; k0 < ke; k0 += kTile * kWaves) {
    const int k1 = k0 + kTile * kWaves;
    float ks[2][4], vs[2][4];
    spread<EVEN>(ksc, ks);
    // S^T = K Q^T: two tiles of 16 keys
    f32x4 s[MT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const Frag f = frag_of<FMT>(kraw[u][2 * st], kraw[u][2 * st + 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) s[mt][u] = mfma(f, q[mt][st][k], s[mt][u]);
      }
    }
    // scores of the lane's row, keys 16 u + 4 g + i (scaled before any branch: a branch between a
    // matrix instruction and its result's reader has cost wait states)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][u][i] *= ks[u][i] * a.scale;
    const Place<EVEN> at = now;
    if (k1 < ke) {
      now = place_of<EVEN>(a, ahead, k1, ke, bad);
      ahead = entries_of<EVEN>(a, table, k1 + kTile * kWaves, ke, zero);
      load_keys(now);
    }
    spread<EVEN>(vsc, vs);
    // which of them count: a tile inside every row's range has no mask
    bool whole = true;
#pragma unroll
    for (int u = 0; u < Place<EVEN>::N; ++u) whole = whole && at.there[u];
    if constexpr (!EVEN) whole = __all(whole);
    const bool partial = !whole || k0 + kTile > ke ||
                         (a.causal && (k0 + kTile > pos_first + 1 ||
                                       (a.window > 0 && k0 <= pos_last - a.window)));
    uint32_t seen[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) seen[mt] = 0xFF;
    if (partial) {
      uint32_t there = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool known;  // (every lane takes part in the exchange)
          if constexpr (EVEN) known = at.there[u];
          else known = __shfl((int)at.there[0], 16 * u + 4 * g + i) != 0;
          there |= (known && k0 + 16 * u + 4 * g + i < ke ? 1u : 0u) << (4 * u + i);
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        seen[mt] = there;
        if (a.causal) seen[mt] &= keys_between(k0 + 4 * g, a.window > 0 ? pos[mt] - a.window + 1 : 0, pos[mt]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][u][i] = kept_or_neg_inf(s[mt][u][i], spread_bit(seen[mt], 4 * u + i));
      }
    }
    // running maximum, probabilities, P^T as the second product's operand
    Frag p[MT][TERMS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float mx = fmaxf(fmaxf(fmaxf(s[mt][0][0], s[mt][0][1]), fmaxf(s[mt][0][2], s[mt][0][3])),
                       fmaxf(fmaxf(s[mt][1][0], s[mt][1][1]), fmaxf(s[mt][1][2], s[mt][1][3])));
      mx = fmaxf(mx, lane_xorf<16>(mx));
      mx = fmaxf(mx, lane_xorf<32>(mx));
      const float mn = fmaxf(m[mt], mx);
      const float base = mn == kNegInf ? 0.0f : mn;
      const float alpha = __builtin_amdgcn_exp2f(m[mt] - base);
      m[mt] = mn;
      l[mt] *= alpha;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][mt] *= alpha;
      if (partial) weights_of<true, TERMS>(s[mt], vs, seen[mt], base, l[mt], p[mt]);
      else weights_of<false, TERMS>(s[mt], vs, 0, base, l[mt], p[mt]);
    }
    // masked places may hold e4m3's NaN: it must reach the rows that see it, and no other
    if (FMT == GPTQ_KV_E4M3 && partial) {
      uint32_t any = 0;
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= nan_marks(vraw[w][i]);
      if (__any((any & 0x80808080u) != 0)) {
        Frag ind[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 8; ++i) ind[mt].v[i] = (__bf16)(seen[mt] >> i & 1 ? 1.0f : 0.0f);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t ones[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t nb = nan_bytes(vraw[w][i]);
            vraw[w][i] &= ~nb;
            ones[i] = nb & 0x38383838u;  // e4m3's 1
          }
          columns_of<FMT>(ones, [&](int b, const Frag& f) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const f32x4 c = mfma(f, ind[mt], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[4 * w + b][mt][i] += c[i] > 0.0f ? __builtin_nanf("") : 0.0f;
            }
          });
        }
      }
    }
    // O^T += V^T P^T: column NT r + n of V is row r of tile n
#pragma unroll
    for (int w = 0; w < VW; ++w)
      columns_of<FMT>(vraw[w], [&](int b, const Frag& f) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) o[4 * w + b][mt] = mfma(f, p[mt][k], o[4 * w + b][mt]);
      });
    if (k1 < ke) load_values(now);
  }
  // the loop's branch stands between the last product and its readers: wait the product's length
  __asm__ volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  if (bad && a.s.info) *a.s.info = 1;

  // join the waves, 16 rows at a time
  const int64_t part = ((int64_t)blockIdx.x * a.heads + head) * a.splits + blockIdx.z;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt > 0) __syncthreads();
    if (16 * mt >= t.rows) break;
    float sum = l[mt];
    sum += lane_xorf<16>(sum);
    sum += lane_xorf<32>(sum);
    if (g == 0) {
      sm[wave][c16] = m[mt];
      sl[wave][c16] = sum;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NT; n += 4)
        *reinterpret_cast<float4*>(&so[wave][c16][NT * (4 * g + i) + n]) =
            make_float4(o[n][mt][i], o[n + 1][mt][i], o[n + 2][mt][i], o[n + 3][mt][i]);
    __syncthreads();
    const int row = tid >> 4, c = (tid & 15) * NT;
    float mx = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, sm[w][row]);
    const float base = mx == kNegInf ? 0.0f : mx;
    float v[NT] = {}, tl = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][row] - base);
      tl += sl[w][row] * f;
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] += so[w][row][c + n] * f;
    }
    if (16 * mt + row >= t.rows) continue;
    if (a.splits == 1) {
      finish_row<NT, F32>(a, t.sp, head, t.row0 + 16 * mt + row, c, v, mx, tl);
    } else {
      store_part<NT, DP>(a, part * (16 * MT) + 16 * mt + row, c, v, mx, tl);
    }
  }
}

// Many rows: a workgroup takes 64 MT rows, each wave 16 MT of them, over tiles of 8192 / DP keys.
// What a tile's codes become on the way to the matrix instructions is the same for all rows, so
// the waves share that work: each converts a quarter of a tile to operands (two 16-byte pieces of
// 16 keys, one 4-byte column of 32 values), which lie in LDS as the lanes take them, 16 bytes each
// in order, without conflicts.  Two tiles alternate; while one is multiplied, the codes of the
// next are on their way, and the places of the one behind it are looked up, a key a thread.
// An operand read from LDS feeds MT matrix instructions: 4 waves read 1 KB each in 16 MT cycles.
//
// The running maximum is a reference that the true one passes by kSlack at most (scores are powers of two): scores
// are compared with it lane by lane, and only where one of a wave passes it (the first tiles) are
// maxima exchanged and sums rescaled.  The weights are then up to 2^kSlack, which fp32 sums and
// bf16 weights hold as well as 1.
//
// 2 sequences of 2048 rows over 4096 tokens, 32 query heads on 8 of 128, e4m3: 279 us, 0.74 PFLOP/s (int8
// 293; 4 x 2048 rows over themselves 212 us, 0.65; fp32 0.25; head_dim 64 0.48, 256 0.40).  No unit is full:
// matrix cores 28% of the time, vector units 46%, LDS 31%; two waves a SIMD hide each other's chains only in
// part, and a third has no registers (it spills: 656 us).  8 waves that share a tile: 269 us here, but 230
// for 4 x 2048, whose beginnings and ends nothing else fills.  Codes are unpacked once for four waves
// in LDS (each wave by itself, without LDS: 730 us).
constexpr float kSlack = 8.0f;

template <int DP>
struct TileShared {
  static constexpr int KEYS = 8192 / DP;
  uint4 k[2][KEYS / 16][DP / 32][64];  // operands of both products
  uint4 v[2][KEYS / 32][DP / 16][64];
  float ks[2][KEYS], vs[2][KEYS];
  int64_t kat[2][KEYS], vat[2][KEYS];  // where a key's codes begin
  uint8_t there[2][KEYS];              // 0: no such key
  uint8_t nan[2][KEYS][DP / 4];        // bit n: value 4 c + n of a key is e4m3's NaN (and 0 in v), where
  uint32_t odd[3];                     // (tiles in turn) bit w: wave w's part of the values has any; bit 4: a key is not there
};

template <int DP, int FMT, bool F32, int MT>
__global__ __launch_bounds__(kThreads, DP == 256 && F32 ? 1 : 2) void kv_attention_tile_kernel(AttnArgs a) {
  constexpr int TERMS = F32 ? 3 : 1;
  constexpr int STEPS = DP / 32, NT = DP / 16, P = DP / 64;
  constexpr int KEYS = TileShared<DP>::KEYS;
  extern __shared__ __align__(16) char shared_bytes[];
  TileShared<DP>& sh = *reinterpret_cast<TileShared<DP>*>(shared_bytes);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  // heads run fastest, so that the tiles of a head meet in one L2; the last tiles, which have the
  // most keys where masked, come first
  const int task = (int)(gridDim.x / a.heads) - 1 - (int)(blockIdx.x / a.heads), head = (int)(blockIdx.x % a.heads);
  const TileRows t = tile_rows(a, task, 64 * MT);
  if (t.rows <= 0) return;
  int kb, ke;
  split_keys(a, t, (int)blockIdx.z, kb, ke);
  const int32_t* table = a.s.table + t.sp.seq * a.s.ldt;
  const Side kc = side_of(a.k, head), vc = side_of(a.v, head);

  Frag q[MT][STEPS][TERMS];
  int pos[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    load_queries<STEPS, TERMS>(a, t, head, 16 * (MT * wave + mt) + c16, g, q[mt], pos[mt]);
  const int w0 = min(16 * MT * wave, t.rows - 1), w1 = min(16 * MT * (wave + 1), t.rows) - 1;
  const bool idle = 16 * MT * wave >= t.rows;
  const int pos_first = t.sp.length - t.sp.rows + divided(t.row0 + w0, a.by_group);
  const int pos_last = t.sp.length - t.sp.rows + divided(t.row0 + max(w0, w1), a.by_group);

  // this wave's part of the conversion
  const int ku[2] = {(2 * wave) / P, (2 * wave + 1) / P}, kp[2] = {(2 * wave) % P, (2 * wave + 1) % P};
  const int vh = wave / P, vw = wave % P;
  // (columns behind head_dim: the row's first ones, whose queries and outputs are not there)
  int ck[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) ck[i] = 64 * kp[i] + 16 * g < a.dim ? 64 * kp[i] + 16 * g : 0;
  const int cv = 64 * vw + 4 * c16 < a.dim ? 64 * vw + 4 * c16 : 0;
  uint32_t kraw[2][4], vraw[8];
  auto load_codes = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_words<4>(kc.codes + sh.kat[b][16 * ku[i] + c16] + ck[i], kraw[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      load_words<1>(vc.codes + sh.vat[b][32 * vh + 16 * (i / 4) + 4 * g + i % 4] + cv, vraw + i);
  };
  auto convert = [&](int b, int mark) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const Frag f = frag_of<FMT>(kraw[i][2 * st], kraw[i][2 * st + 1]);
        sh.k[b][ku[i]][2 * kp[i] + st][lane] = make_uint4(f.w[0], f.w[1], f.w[2], f.w[3]);
      }
    if (FMT == GPTQ_KV_E4M3) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= nan_marks(vraw[i]);
      if (__any((any & 0x80808080u) != 0)) {  // no operand holds a NaN, which would reach every row
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = nan_bytes(vraw[i]);
          vraw[i] &= ~x;
          sh.nan[b][32 * vh + 16 * (i / 4) + 4 * g + i % 4][16 * vw + c16] =
              (uint8_t)((x & 1u) | (x >> 7 & 2u) | (x >> 14 & 4u) | (x >> 21 & 8u));
        }
        if (lane == 0) atomicOr(&sh.odd[mark], 1u << wave);
      }
    }
    columns_of<FMT>(vraw, [&](int n, const Frag& f) {
      sh.v[b][vh][4 * vw + n][lane] = make_uint4(f.w[0], f.w[1], f.w[2], f.w[3]);
    });
  };
  // places: thread i looks up key i of a tile for the keys' cache, thread KEYS + i for the values',
  // the table's entries a round ahead
  const bool looks = tid < 2 * KEYS, of_keys = tid < KEYS;
  const int ti = of_keys ? tid : tid - KEYS;
  const int64_t tpage = of_keys ? kc.cpage : vc.cpage, tppage = of_keys ? kc.ppage : vc.ppage;
  const int32_t tslot = of_keys ? kc.cslot : vc.cslot, tblock = of_keys ? kc.pblock : vc.pblock;
  const float* const tscales = of_keys ? kc.scales : vc.scales;
  bool bad = t.bad, known = false;
  float sc = 0.0f;
  auto entry_of = [&](int k0) {
    return looks ? table[min(divided(min(k0 + ti, ke - 1), a.s.by_page), a.s.width - 1)] : 0;
  };
  auto look_up = [&](int k0, int e, int b) {  // (its scale goes to LDS with the tile's operands)
    if (!looks) return;
    const int kk = min(k0 + ti, ke - 1), entry = divided(kk, a.s.by_page);
    const bool ok = entry < a.s.width && (uint32_t)e < (uint32_t)a.s.pages;
    bad = bad || (k0 + ti < ke && !ok);
    known = k0 + ti < ke && ok;
    const int page = ok ? e : 0, slot = kk - entry * a.s.page_size, blk = divided(slot, a.s.by_block);
    (of_keys ? sh.kat : sh.vat)[b][ti] = page * tpage + (int64_t)slot * tslot;
    sc = tscales[page * tppage + (int64_t)blk * tblock];
  };
  auto put_scales = [&](int b, int mark) {
    if (!looks) return;
    (of_keys ? sh.ks : sh.vs)[b][ti] = of_keys ? sc * a.scale : sc;
    if (of_keys) sh.there[b][ti] = known;
    if (!known) atomicOr(&sh.odd[mark], 16u);
  };

  f32x4 o[NT][MT];
  float m[MT], l[MT];
  bool set[MT];  // whether a row has seen a key, and m is its reference
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = l[mt] = 0.0f;
    set[mt] = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  if (kb < ke) {  // the first tile, the second one's places, the third one's entries
    if (tid < 3) sh.odd[tid] = 0;
    look_up(kb, entry_of(kb), 0);
    __syncthreads();
    load_codes(0);
    put_scales(0, 0);
    look_up(kb + KEYS, entry_of(kb + KEYS), 1);
    convert(0, 0);
  }
  int e = kb < ke ? entry_of(kb + 2 * KEYS) : 0;
  // One barrier a tile: what is written behind it belongs to the next tile's buffers, which were read
  // last in front of it, or to marks that are read two barriers later.
  for (int k0 = kb, b = 0, mark = 0; k0 < ke; k0 += KEYS, b ^= 1) {
    __syncthreads();  // tile b's operands, the next one's places
    const uint32_t odd = __builtin_amdgcn_readfirstlane(sh.odd[mark]);
    load_codes(b ^ 1);  // (behind the last tile: somewhere)
    uint4 kw[2][STEPS];
    auto read_keys = [&](int h, int i) { kw[i / STEPS][i % STEPS] = sh.k[b][2 * h + i / STEPS][i % STEPS][lane]; };
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i) read_keys(0, i);
#pragma unroll 1
    for (int h = 0; h < KEYS / 32; ++h) {
      const int kh = k0 + 32 * h, ahead = min(h + 1, KEYS / 32 - 1);
      // keys that none of the wave's rows sees
      if (idle || kh >= ke || (a.causal && (kh > pos_last || (a.window > 0 && kh + 31 <= max(pos_first, 0) - a.window)))) {
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) read_keys(ahead, i);
        continue;
      }
      f32x4 s[MT][2];
      {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            Frag f;
            f.w[0] = kw[u][st].x; f.w[1] = kw[u][st].y; f.w[2] = kw[u][st].z; f.w[3] = kw[u][st].w;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int k = 0; k < TERMS; ++k) s[mt][u] = mfma(f, q[mt][st][k], s[mt][u]);
          }
        }
      }
      uint4 vw_[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) vw_[n] = sh.v[b][h][n][lane];
      float vs[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 x = *reinterpret_cast<const float4*>(&sh.ks[b][32 * h + 16 * u + 4 * g]);
        const float4 y = *reinterpret_cast<const float4*>(&sh.vs[b][32 * h + 16 * u + 4 * g]);
        vs[u][0] = y.x; vs[u][1] = y.y; vs[u][2] = y.z; vs[u][3] = y.w;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {  // scores relative to the row's reference
          s[mt][u][0] = fmaf(s[mt][u][0], x.x, -m[mt]); s[mt][u][1] = fmaf(s[mt][u][1], x.y, -m[mt]);
          s[mt][u][2] = fmaf(s[mt][u][2], x.z, -m[mt]); s[mt][u][3] = fmaf(s[mt][u][3], x.w, -m[mt]);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      const bool partial = (odd & 16u) || kh + 32 > ke ||
                           (a.causal && (kh + 32 > pos_first + 1 || (a.window > 0 && kh <= pos_last - a.window)));
      uint32_t seen[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) seen[mt] = 0xFF;
      if (partial) {
        uint32_t there = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(&sh.there[b][32 * h + 16 * u + 4 * g]);  // 4 bytes, 0 or 1
          there |= ((x | x >> 7 | x >> 14 | x >> 21) & 15u) << (4 * u);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          seen[mt] = there;
          if (a.causal) seen[mt] &= keys_between(kh + 4 * g, a.window > 0 ? pos[mt] - a.window + 1 : 0, pos[mt]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][u][i] = kept_or_neg_inf(s[mt][u][i], spread_bit(seen[mt], 4 * u + i));
        }
      }
      float mx[MT];
      bool grows = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mx[mt] = max_of(s[mt]);
        grows = grows || mx[mt] > (set[mt] ? kSlack : kNegInf);
      }
      if (__any(grows)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float x = fmaxf(mx[mt], lane_xorf<16>(mx[mt]));
          x = fmaxf(x, lane_xorf<32>(x));
          if (set[mt]) x = fmaxf(x, 0.0f);
          const bool moves = x > kNegInf;
          const float by = moves ? x : 0.0f, alpha = set[mt] ? __builtin_amdgcn_exp2f(-by) : 1.0f;
          set[mt] = set[mt] || moves;
          m[mt] += by;
          l[mt] *= alpha;
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][mt] *= alpha;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][u][i] -= by;
        }
      }
      Frag p[MT][TERMS];
      if (partial) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          weights_of<true, TERMS>(s[mt], vs, seen[mt], 0.0f, l[mt], p[mt]);
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) weights_of<false, TERMS>(s[mt], vs, 0, 0.0f, l[mt], p[mt]);
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        f.w[0] = vw_[n].x; f.w[1] = vw_[n].y; f.w[2] = vw_[n].z; f.w[3] = vw_[n].w;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) o[n][mt] = mfma(f, p[mt][k], o[n][mt]);
        if (KEYS > 32) {  // (the next half's keys travel beside these products)
#pragma unroll
          for (int i = n * 2 * STEPS / NT; i < (n + 1) * 2 * STEPS / NT; ++i) read_keys(ahead, i);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      if (FMT == GPTQ_KV_E4M3 && (odd >> (P * h) & ((1u << P) - 1)) != 0) {
        // a NaN among the values reaches the rows that see its key
        __asm__ volatile("s_nop 15" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll 1
        for (int key = 0; key < 32; ++key) {
          uint32_t sees[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            sees[mt] = spread_bit(__shfl((int)seen[mt], 16 * (key % 16 / 4) + c16), 4 * (key / 16) + key % 4) & 0x7FC00000u;
#pragma unroll
          for (int w = 0; w < P; ++w) {
            if ((odd >> (P * h + w) & 1u) == 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = sh.nan[b][32 * h + key][16 * w + 4 * g + i];
#pragma unroll
              for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  o[4 * w + n][mt][i] = __uint_as_float(__float_as_uint(o[4 * w + n][mt][i]) | (sees[mt] & spread_bit(x, n)));
            }
          }
        }
      }
    }
    mark = mark == 2 ? 0 : mark + 1;
    if (tid == 0) sh.odd[mark == 2 ? 0 : mark + 1] = 0;
    put_scales(b ^ 1, mark);
    convert(b ^ 1, mark);
    look_up(k0 + 2 * KEYS, e, b);
    e = entry_of(k0 + 3 * KEYS);
  }
  // (the loop's branch stands between the last product and its readers: wait the product's length)
  __asm__ volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  if (bad && a.s.info) *a.s.info = 1;

  const int64_t part = ((int64_t)task * a.heads + head) * a.splits + blockIdx.z;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = 16 * (MT * wave + mt) + c16;
    float sum = l[mt];
    sum += lane_xorf<16>(sum);
    sum += lane_xorf<32>(sum);
    if (row >= t.rows) continue;
#pragma unroll
    for (int w = 0; w < P; ++w) {
      float v[16];  // columns 64 w + 16 g + 4 i + n
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) v[4 * i + n] = o[4 * w + n][mt][i];
      if (a.splits == 1) finish_row<16, F32>(a, t.sp, head, t.row0 + row, 64 * w + 16 * g, v, m[mt], sum);
      else store_part<16, DP>(a, part * (64 * MT) + row, 64 * w + 16 * g, v, set[mt] ? m[mt] : kNegInf, sum);
    }
  }
}

// A wave joins the splits of a row of a tile: a group of 16 lanes takes every fourth one, in order, their
// sums are joined in a fixed order.
template <int DP, bool F32>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(AttnArgs a, int per) {
  constexpr int NT = DP / 16;
  constexpr int B = 4;  // parts of a lane whose loads are under way together
  const int lane = threadIdx.x & 63, head = blockIdx.y, row = blockIdx.z * kWaves + (threadIdx.x >> 6);
  const TileRows t = tile_rows(a, (int)blockIdx.x, per);
  if (row >= t.rows) return;
  const int64_t part = ((int64_t)blockIdx.x * a.heads + head) * a.splits;
  const int c = (lane & 15) * NT, sub = lane >> 4;
  float m = kNegInf, l = 0.0f, v[NT] = {};
  for (int s0 = sub; s0 < a.splits; s0 += 4 * B) {
    float2 st[B];
    float4 d[B][NT / 4];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int64_t at = (part + min(s0 + 4 * k, a.splits - 1)) * per + row;
      st[k] = a.stats[at];
#pragma unroll
      for (int n = 0; n < NT / 4; ++n) d[k][n] = reinterpret_cast<const float4*>(a.parts + at * DP + c)[n];
    }
    float mx = m;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (s0 + 4 * k >= a.splits) st[k] = make_float2(kNegInf, 0.0f);
      mx = fmaxf(mx, st[k].x);
    }
    const float base = mx == kNegInf ? 0.0f : mx;
    const float f0 = __builtin_amdgcn_exp2f(m - base);
    m = mx;
    l *= f0;
#pragma unroll
    for (int n = 0; n < NT; ++n) v[n] *= f0;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const bool in = s0 + 4 * k < a.splits;  // (what stands in for a part behind the last one may hold anything)
      const float f = __builtin_amdgcn_exp2f(st[k].x - base);
      l += st[k].y * f;
#pragma unroll
      for (int n = 0; n < NT / 4; ++n) {
        v[4 * n] += in ? d[k][n].x * f : 0.0f;
        v[4 * n + 1] += in ? d[k][n].y * f : 0.0f;
        v[4 * n + 2] += in ? d[k][n].z * f : 0.0f;
        v[4 * n + 3] += in ? d[k][n].w * f : 0.0f;
      }
    }
  }
  float mx = fmaxf(m, lane_xorf<16>(m));
  mx = fmaxf(mx, lane_xorf<32>(mx));
  const float f = __builtin_amdgcn_exp2f(m - (mx == kNegInf ? 0.0f : mx));
  l *= f;
  l += lane_xorf<16>(l);
  l += lane_xorf<32>(l);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    v[n] *= f;
    v[n] += lane_xorf<16>(v[n]);
    v[n] += lane_xorf<32>(v[n]);
  }
  if (sub == 0) finish_row<NT, F32>(a, t.sp, head, t.row0 + row, c, v, mx, l);
}

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

struct Plan {
  bool tiles;   // the tile kernel
  int mt;       // 16 rows each, of a wave
  int per;      // rows of a workgroup
  int64_t tasks;
  int splits;
};

// 16 rows each of a wave in the tile kernel: as many as 256 registers hold beside the operands that
// are read ahead (2 x 2048 rows over 4096 tokens: 2 277 us, 3, which spills, 373).
constexpr int tile_mt(int dp, bool f32) { return dp == 64 ? (f32 ? 2 : 3) : f32 ? 1 : dp == 128 ? 2 : 1; }

Plan plan_of(const gptq_kv_blocks* c, int q_heads, int dt, int64_t tokens, int64_t seqs, int64_t width) {
  Plan p;
  const bool f32 = dt == GPTQ_F32;
  const int dp = padded_dim(c->head_dim);
  const int64_t group = q_heads / c->heads;
  const int64_t each = ceil_div(tokens * group, seqs);  // rows of a sequence on average
  // 8 sequences of 8000, 32 query heads on 8 of 128, 20 rows a key head: 32 rows a wave 47 us, twice 16
  // 92, the tile kernel 74; 36 rows: 32 rows a wave 86, the tile kernel 63 (its waves with 16 rows); fp32,
  // 20 rows: 16 rows a wave 74, the tile kernel 102
  p.tiles = each > (f32 || dp <= 128 ? 32 : 16);
  p.mt = p.tiles ? (each <= 64 ? 1 : tile_mt(dp, f32)) : each > 16 && !f32 ? 2 : 1;
  p.per = p.tiles ? 64 * p.mt : 16 * p.mt;
  p.tasks = tokens * group / p.per + seqs;
  // Splits: as many as give 512 workgroups, two a CU, whose waves' loads fill the memory's queue
  // (16 sequences of 12000, 8 heads of 128: 128 workgroups 115 us, 512 80, 768 88, 1024 91, 2048 87),
  // 512 keys each at least (5 sequences of 300: one 8.7 us; the 13 that a table for 32768 tokens gives them and
  // their join 12.9).  Kernel, tiles and splits go by the call's averages and its table, which the host knows:
  // sequences of very different kinds are right in one call, but faster in calls of their own.
  const int64_t tiles = hmin(p.tasks, seqs * ceil_div(each, p.per)) * c->heads;
  const int64_t keys = hmin(width * c->page_size, int64_t(1) << 30);
  p.splits = (int)hmax(1, hmin(hmin(ceil_div(512, tiles), 64), keys / 512));
  return p;
}

template <int DP, int FMT, bool F32, int MT>
hipError_t launch_tiles(const AttnArgs& a, const dim3& grid, hipStream_t stream) {
  auto* kernel = kv_attention_tile_kernel<DP, FMT, F32, MT>;
  constexpr int bytes = (int)sizeof(TileShared<DP>);
  // (more than 64 KB of LDS has to be asked for; the same each time)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), bytes, stream, a);
  return hipGetLastError();
}

template <int FMT, bool F32>
hipError_t launch_tiles_of(int dp, int mt, const AttnArgs& a, const dim3& grid, hipStream_t stream) {
  if (mt == 1) {
    if (dp == 64) return launch_tiles<64, FMT, F32, 1>(a, grid, stream);
    if (dp == 128) return launch_tiles<128, FMT, F32, 1>(a, grid, stream);
    return launch_tiles<256, FMT, F32, 1>(a, grid, stream);
  }
  if (dp == 64) return launch_tiles<64, FMT, F32, tile_mt(64, F32)>(a, grid, stream);
  if (dp == 128) return launch_tiles<128, FMT, F32, tile_mt(128, F32)>(a, grid, stream);
  return launch_tiles<256, FMT, F32, tile_mt(256, F32)>(a, grid, stream);
}

}  // namespace

size_t kv_attention_ws_bytes(const gptq_kv_blocks* c, int q_heads, int dt, int64_t tokens,
                             int64_t seqs, int64_t width) {
  const Plan p = plan_of(c, q_heads, dt, tokens, seqs, width);
  if (p.splits == 1) return 0;
  return (size_t)p.tasks * c->heads * p.splits * p.per * (padded_dim(c->head_dim) + 2) * 4;
}

hipError_t launch_kv_attention(const KvAttention& t, const KvSequences& seqs,
                               const gptq_kv_blocks* kb, const gptq_kv_blocks* vb, int32_t* info,
                               void* ws, hipStream_t stream) {
  const Plan p = plan_of(kb, t.q_heads, t.dt, seqs.tokens, seqs.seqs, seqs.width);
  if (!grid_fits(p.tiles ? p.tasks * kb->heads : p.tasks, kThreads)) return hipErrorInvalidConfiguration;
  const bool f32 = t.dt == GPTQ_F32;
  const int dp = padded_dim(kb->head_dim), per16 = f32 ? 4 : 8;
  AttnArgs a = {};
  a.q = static_cast<const char*>(t.q.p);
  a.out = static_cast<char*>(t.out.p);
  a.qt = t.q.token_stride; a.qh = t.q.head_stride;
  a.ot = t.out.token_stride; a.oh = t.out.head_stride;
  a.lse = t.lse;
  a.s = sequences_of(seqs, kb, info);
  a.k = block_cache_of(kb);
  a.v = block_cache_of(vb);
  a.heads = kb->heads;
  a.group = t.q_heads / kb->heads;
  a.dim = kb->head_dim;
  a.causal = t.causal;
  a.window = t.window;
  a.qvec = (reinterpret_cast<uintptr_t>(t.q.p) & 15) == 0 && a.qt % per16 == 0 && a.qh % per16 == 0;
  a.ovec = (reinterpret_cast<uintptr_t>(t.out.p) & 15) == 0 && a.ot % per16 == 0 && a.oh % per16 == 0;
  a.scale = t.scale * kLog2e;
  a.splits = p.splits;
  a.by_rows = divisor_of(p.per);
  a.by_group = divisor_of(a.group);
  a.by_splits = divisor_of(p.splits);
  a.stats = static_cast<float2*>(ws);
  a.parts = reinterpret_cast<float*>(a.stats + p.tasks * kb->heads * p.splits * p.per);
  const bool even = kb->page_size % 16 == 0 && kb->block % 16 == 0;
  const dim3 block(kThreads);
  if (p.tiles) {
    const dim3 tgrid((unsigned)(p.tasks * kb->heads), 1, (unsigned)p.splits);
    const hipError_t e =
        kb->format == GPTQ_KV_E4M3
            ? (f32 ? launch_tiles_of<GPTQ_KV_E4M3, true>(dp, p.mt, a, tgrid, stream) : launch_tiles_of<GPTQ_KV_E4M3, false>(dp, p.mt, a, tgrid, stream))
            : (f32 ? launch_tiles_of<GPTQ_KV_INT8, true>(dp, p.mt, a, tgrid, stream) : launch_tiles_of<GPTQ_KV_INT8, false>(dp, p.mt, a, tgrid, stream));
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)p.tasks, (unsigned)kb->heads, (unsigned)p.splits);
#define GPTQ_ATTN_E(DP, F, W, MT)                                                                  \
  do {                                                                                             \
    if (even) hipLaunchKernelGGL((kv_attention_kernel<DP, F, W, MT, true>), grid, block, 0, stream, a); \
    else hipLaunchKernelGGL((kv_attention_kernel<DP, F, W, MT, false>), grid, block, 0, stream, a);  \
  } while (0)
#define GPTQ_ATTN_F(DP, W, MT)                                            \
  do {                                                                    \
    if (kb->format == GPTQ_KV_E4M3) GPTQ_ATTN_E(DP, GPTQ_KV_E4M3, W, MT); \
    else GPTQ_ATTN_E(DP, GPTQ_KV_INT8, W, MT);                            \
  } while (0)
#define GPTQ_ATTN(DP)                         \
  do {                                        \
    if (f32) GPTQ_ATTN_F(DP, true, 1);        \
    else if (p.mt == 1) GPTQ_ATTN_F(DP, false, 1); \
    else GPTQ_ATTN_F(DP, false, 2);           \
  } while (0)
  if (p.tiles) {}
  else if (dp == 64) GPTQ_ATTN(64);
  else if (dp == 128) GPTQ_ATTN(128);
  else if (f32) GPTQ_ATTN_F(256, true, 1);
  else GPTQ_ATTN_F(256, false, 1);
#undef GPTQ_ATTN
#undef GPTQ_ATTN_F
#undef GPTQ_ATTN_E
  if (p.splits > 1) {
    const dim3 jgrid((unsigned)p.tasks, (unsigned)kb->heads, (unsigned)(p.per / kWaves));
#define GPTQ_JOIN(DP)                                                                                     \
  do {                                                                                                    \
    if (f32) hipLaunchKernelGGL((kv_attention_join_kernel<DP, true>), jgrid, block, 0, stream, a, p.per); \
    else hipLaunchKernelGGL((kv_attention_join_kernel<DP, false>), jgrid, block, 0, stream, a, p.per);    \
  } while (0)
    if (dp == 64) GPTQ_JOIN(64);
    else if (dp == 128) GPTQ_JOIN(128);
    else GPTQ_JOIN(256);
#undef GPTQ_JOIN
  }
  return hipGetLastError();
}

}  // namespace gptq
