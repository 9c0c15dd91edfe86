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
  Divisor by_rows;  // rows of a tile
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

// bytes of w that are e4m3's NaN, as 0xFF
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return (t >> 7) * 255u;
}

__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// TERMS bf16 numbers whose sum is x (1: rounded; 3: 24 bits and more)
template <int TERMS>
__device__ __forceinline__ void split_terms(float x, float (&t)[TERMS]) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    t[k] = (float)(__bf16)x;
    x = x - t[k];
    if (!is_finite(x)) x = 0.0f;  // an infinity or a NaN is in its first term
  }
}

struct TileRows {  // what a workgroup works on
  Span sp;
  int row0, rows;  // of the sequence's rows * group
  int lo, hi;      // its keys, lo a multiple of 16
};

__device__ __forceinline__ TileRows tile_rows(const AttnArgs& a, int task, int per) {
  TileRows t;
  int first;
  t.sp = span_of(a.s, task, a.group, a.by_rows, 1, first);
  t.row0 = (task - first) * per;
  t.rows = max(min(per, t.sp.rows * a.group - t.row0), 0);
  // positions of the first and last row; keys that any of them sees
  const int base = t.sp.length - t.sp.rows;
  t.hi = t.sp.length;
  t.lo = 0;
  if (t.rows > 0 && a.causal) {
    const int p0 = base + t.row0 / a.group, p1 = base + (t.row0 + t.rows - 1) / a.group;
    t.hi = max(min(t.hi, p1 + 1), 0);
    if (a.window > 0) t.lo = max(p0 - a.window + 1, 0) & ~15;
  }
  return t;
}

// a split's keys: whole rounds of the workgroup's waves
__device__ __forceinline__ void split_keys(const TileRows& t, int splits, int i, int& k0, int& k1) {
  const int n = max(t.hi - t.lo, 0);
  const int per = ((n + splits - 1) / splits + kTile * kWaves - 1) / (kTile * kWaves) * (kTile * kWaves);
  const int64_t b = (int64_t)i * per;
  k0 = t.lo + (int)min((int64_t)n, b);
  k1 = t.lo + (int)min((int64_t)n, b + per);
}

// Row rr (of rows * group) of the sequence: DP / 16 values from column c on, and its statistics.
template <int DP, bool F32>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const Span& sp, int head, int rr, int c,
                                           const float* o, float m, float l) {
  constexpr int N = DP / 16;
  const int r = rr / a.group;
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

// DP: head_dim rounded up to 64, 128 or 256.  EVEN: the 16 keys of a half tile share a page and
// a block.  fp32 rows: queries and probabilities as three bf16 terms each.
template <int DP, int FMT, bool F32, int MT, bool EVEN>
__global__ __launch_bounds__(kThreads) void kv_attention_kernel(AttnArgs a) {
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
  split_keys(t, a.splits, (int)blockIdx.z, kb, ke);

  // queries: lane (row c16, group g) holds columns (DP / 4) g .. + DP / 4 - 1
  Frag q[MT][STEPS][TERMS];
  int pos[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int rr = t.row0 + 16 * mt + c16;
    const bool live = 16 * mt + c16 < t.rows;
    const int r = live ? rr / a.group : 0;
    pos[mt] = t.sp.length - t.sp.rows + r;
    const char* p = a.q + ((int64_t)(t.sp.start + r) * a.qt +
                           (int64_t)(head * a.group + (live ? rr - r * a.group : 0)) * a.qh) * (F32 ? 4 : 2);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c0 = (DP / 4) * g + 8 * s;
      const Raw8<F32 ? GPTQ_F32 : GPTQ_BF16> raw =
          load_raw8<F32 ? GPTQ_F32 : GPTQ_BF16>(p, c0, live ? a.dim : 0, a.qvec);
      if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float tm[TERMS];
          split_terms<TERMS>(__uint_as_float(raw.w[e]), tm);
#pragma unroll
          for (int k = 0; k < TERMS; ++k) q[mt][s][k].v[e] = (__bf16)tm[k];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[mt][s][0].w[e] = raw.w[e];
      }
    }
  }
  // (bounds of the tile's rows, for its masks)
  const int pos_first = t.sp.length - t.sp.rows + t.row0 / a.group;
  const int pos_last = t.sp.length - t.sp.rows + (t.row0 + t.rows - 1) / a.group;

  f32x4 o[NT][MT];
  float m[MT], l[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = kNegInf;
    l[mt] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t* table = a.s.table + t.sp.seq * a.s.ldt;
  const int ck = KW * 4 * g;           // first column of the lane's part of a K row
  const int cv = NT * c16;             // of a V row
  for (int k0 = kb + kTile * wave; k0 < ke; k0 += kTile * kWaves) {
    // where the keys lie: pages and slots
    bool bad = false;
    uint32_t kraw[2][KW], vraw[8][VW];
    float ks[2][4], vs[2][4];
    bool usable[2] = {true, true};
    uint32_t good = 0xFF;  // the lane's 8 keys: a bit each
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (EVEN) {
        const int kk = k0 + 16 * u;
        const int entry = divided(kk, a.s.by_page);
        int page = -1;
        if (kk < ke) {
          page = entry < a.s.width ? table[entry] : -1;
          if (page < 0 || page >= a.s.pages) { bad = true; page = -1; }
        }
        page = __builtin_amdgcn_readfirstlane(page);
        usable[u] = page >= 0;
        const int slot = kk - entry * a.s.page_size;
        const int64_t ko = page * a.k.cpage + slot * a.k.cslot + head * a.k.chead;
        const int64_t vo = page * a.v.cpage + slot * a.v.cslot + head * a.v.chead;
        const int blk = divided(slot, a.s.by_block);
        float sk = 0.0f, sv = 0.0f;
        if (usable[u]) {
          sk = a.k.scales[page * a.k.ppage + blk * a.k.pblock + head * a.k.phead];
          sv = a.v.scales[page * a.v.ppage + blk * a.v.pblock + head * a.v.phead];
        } else {
          good &= u ? 0x0F : 0xF0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) { ks[u][i] = sk; vs[u][i] = sv; }
#pragma unroll
        for (int w = 0; w < KW; w += 4) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (usable[u] && kk + c16 < ke && ck + 4 * w < a.dim)
            x = *reinterpret_cast<const uint4*>(a.k.codes + ko + c16 * a.k.cslot + ck + 4 * w);
          kraw[u][w] = x.x; kraw[u][w + 1] = x.y; kraw[u][w + 2] = x.z; kraw[u][w + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = usable[u] && kk + 4 * g + i < ke && cv < a.dim;
          const uint8_t* p = a.v.codes + vo + (4 * g + i) * a.v.cslot + cv;
          if constexpr (VW == 1) vraw[4 * u + i][0] = in ? *reinterpret_cast<const uint32_t*>(p) : 0;
          else if constexpr (VW == 2) {
            uint2 x = make_uint2(0, 0);
            if (in) x = *reinterpret_cast<const uint2*>(p);
            vraw[4 * u + i][0] = x.x; vraw[4 * u + i][1] = x.y;
          } else {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4*>(p);
            vraw[4 * u + i][0] = x.x; vraw[4 * u + i][1] = x.y; vraw[4 * u + i][2] = x.z; vraw[4 * u + i][3] = x.w;
          }
        }
      }
    }
    if constexpr (!EVEN) {
      // lane i (and i + 32) looks up key k0 + i
      const int kk = k0 + (lane & 31);
      int page = -1, slot = 0;
      float sk = 0.0f, sv = 0.0f;
      if (kk < ke) {
        const int entry = divided(kk, a.s.by_page);
        page = entry < a.s.width ? table[entry] : -1;
        slot = kk - entry * a.s.page_size;
        if (page < 0 || page >= a.s.pages) { bad = true; page = -1; }
        else {
          const int blk = divided(slot, a.s.by_block);
          sk = a.k.scales[page * a.k.ppage + blk * a.k.pblock + head * a.k.phead];
          sv = a.v.scales[page * a.v.ppage + blk * a.v.pblock + head * a.v.phead];
        }
      }
      usable[0] = usable[1] = __all(page >= 0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int pg = __shfl(page, 16 * u + c16), sl_ = __shfl(slot, 16 * u + c16);
        const uint8_t* p = a.k.codes + pg * a.k.cpage + sl_ * a.k.cslot + head * a.k.chead + ck;
#pragma unroll
        for (int w = 0; w < KW; w += 4) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (pg >= 0 && ck + 4 * w < a.dim) x = *reinterpret_cast<const uint4*>(p + 4 * w);
          kraw[u][w] = x.x; kraw[u][w + 1] = x.y; kraw[u][w + 2] = x.z; kraw[u][w + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int from = 16 * u + 4 * g + i;
          const int pv = __shfl(page, from), sv_ = __shfl(slot, from);
          ks[u][i] = __shfl(sk, from);
          vs[u][i] = __shfl(sv, from);
          if (pv < 0) good &= ~(1u << (4 * u + i));
          const bool in = pv >= 0 && cv < a.dim;
          const uint8_t* pp = a.v.codes + pv * a.v.cpage + sv_ * a.v.cslot + head * a.v.chead + cv;
#pragma unroll
          for (int w = 0; w < VW; ++w)
            vraw[4 * u + i][w] = in ? reinterpret_cast<const uint32_t*>(pp)[w] : 0;
        }
      }
    }
    if (bad && a.s.info) *a.s.info = 1;

    // S^T = K Q^T: two tiles of 16 keys
    f32x4 s[2][MT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[u][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const uint32_t w0 = signed_codes<FMT>(kraw[u][2 * st]), w1 = signed_codes<FMT>(kraw[u][2 * st + 1]);
        Frag f;
        f.p[0] = pair_of<FMT, false>(w0);
        f.p[1] = pair_of<FMT, true>(w0);
        f.p[2] = pair_of<FMT, false>(w1);
        f.p[3] = pair_of<FMT, true>(w1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) s[u][mt] = mfma(f, q[mt][st][k], s[u][mt]);
      }
    }
    // scores of the lane's row, keys 16 u + 4 g + i (scaled before any branch: a branch between a
    // matrix instruction and its result's reader has cost wait states)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][mt][i] *= ks[u][i] * a.scale;
    // which of them count: a tile inside every row's range has no mask
    const bool partial = !usable[0] || !usable[1] || k0 + kTile > ke ||
                         (a.causal && (k0 + kTile > pos_first + 1 ||
                                       (a.window > 0 && k0 <= pos_last - a.window)));
    uint32_t seen[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) seen[mt] = 0xFF;
    if (partial) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        seen[mt] = good;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = k0 + 16 * u + 4 * g + i;
            if (key >= ke || (a.causal && (key > pos[mt] || (a.window > 0 && key <= pos[mt] - a.window))))
              seen[mt] &= ~(1u << (4 * u + i));
            if (!(seen[mt] >> (4 * u + i) & 1)) s[u][mt][i] = kNegInf;
          }
      }
    }
    // running maximum, probabilities, P^T as the second product's operand
    Frag p[MT][TERMS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float mx = fmaxf(fmaxf(fmaxf(s[0][mt][0], s[0][mt][1]), fmaxf(s[0][mt][2], s[0][mt][3])),
                       fmaxf(fmaxf(s[1][mt][0], s[1][mt][1]), fmaxf(s[1][mt][2], s[1][mt][3])));
      mx = fmaxf(mx, lane_xorf<16>(mx));
      mx = fmaxf(mx, lane_xorf<32>(mx));
      const float mn = fmaxf(m[mt], mx);
      const float base = mn == kNegInf ? 0.0f : mn;
      const float alpha = __builtin_amdgcn_exp2f(m[mt] - base);
      m[mt] = mn;
      l[mt] *= alpha;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][mt] *= alpha;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(s[u][mt][i] - base);
          l[mt] += e;
          float x = e * vs[u][i];
          if (partial && !(seen[mt] >> (4 * u + i) & 1)) x = 0.0f;  // (a scale may be anything there)
          float tm[TERMS];
          split_terms<TERMS>(x, tm);
#pragma unroll
          for (int k = 0; k < TERMS; ++k) p[mt][k].v[4 * u + i] = (__bf16)tm[k];
        }
    }
    // masked places may hold e4m3's NaN: it must reach the rows that see it, and no other
    bool nans = false;
    if (FMT == GPTQ_KV_E4M3 && partial) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int w = 0; w < VW; ++w) any |= nan_bytes(vraw[i][w]);
      nans = __any(any != 0);
      if (nans) {
        Frag ind[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 8; ++i) ind[mt].v[i] = (__bf16)(seen[mt] >> i & 1 ? 1.0f : 0.0f);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t nb[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            nb[i] = nan_bytes(vraw[i][w]);
            vraw[i][w] &= ~nb[i];
            nb[i] &= 0x38383838u;  // e4m3's 1
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            Frag f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t two = __builtin_amdgcn_perm(nb[2 * k + 1], nb[2 * k], b < 2 ? 0x05010400u : 0x07030602u);
              f.p[k] = b & 1 ? pair_of<FMT, true>(two) : pair_of<FMT, false>(two);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const f32x4 c = mfma(f, ind[mt], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[4 * w + b][mt][i] += c[i] > 0.0f ? __builtin_nanf("") : 0.0f;
            }
          }
        }
      }
    }
    // O^T += V^T P^T: column NT r + n of V is row r of tile n
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = signed_codes<FMT>(vraw[2 * k][w]), y = signed_codes<FMT>(vraw[2 * k + 1][w]);
        lo[k] = __builtin_amdgcn_perm(y, x, 0x05010400u);
        hi[k] = __builtin_amdgcn_perm(y, x, 0x07030602u);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        Frag f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t two = b < 2 ? lo[k] : hi[k];
          f.p[k] = b & 1 ? pair_of<FMT, true>(two) : pair_of<FMT, false>(two);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) o[4 * w + b][mt] = mfma(f, p[mt][k], o[4 * w + b][mt]);
      }
    }
  }
  // the loop's branch stands between the last product and its readers: wait the product's length
  __asm__ volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);

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
      finish_row<DP, F32>(a, t.sp, head, t.row0 + 16 * mt + row, c, v, mx, tl);
    } else {
      const int64_t at = part * (16 * MT) + 16 * mt + row;
      float* d = a.parts + at * DP + c;
#pragma unroll
      for (int n = 0; n < NT; n += 4) *reinterpret_cast<float4*>(d + n) = make_float4(v[n], v[n + 1], v[n + 2], v[n + 3]);
      if (c == 0) a.stats[at] = make_float2(mx, tl);
    }
  }
}

// A workgroup per tile and head joins its splits, in their order.
template <int DP, bool F32>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(AttnArgs a, int per) {
  constexpr int NT = DP / 16;
  const int tid = threadIdx.x, head = blockIdx.y;
  const TileRows t = tile_rows(a, (int)blockIdx.x, per);
  const int64_t part = ((int64_t)blockIdx.x * a.heads + head) * a.splits;
  for (int row = tid >> 4; row < t.rows; row += 16) {
    const int c = (tid & 15) * NT;
    float mx = kNegInf;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, a.stats[(part + s) * per + row].x);
    const float base = mx == kNegInf ? 0.0f : mx;
    float v[NT] = {}, tl = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
      const int64_t at = (part + s) * per + row;
      const float2 st = a.stats[at];
      const float f = __builtin_amdgcn_exp2f(st.x - base);
      tl += st.y * f;
      const float* d = a.parts + at * DP + c;
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] += d[n] * f;
    }
    finish_row<DP, F32>(a, t.sp, head, t.row0 + row, c, v, mx, tl);
  }
}

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

struct Plan {
  int mt;       // tiles of 16 rows
  int64_t tasks;
  int splits;
};

Plan plan_of(const gptq_kv_blocks* c, int q_heads, int dt, int64_t tokens, int64_t seqs, int64_t width) {
  Plan p;
  const int64_t group = q_heads / c->heads;
  const int64_t each = ceil_div(tokens * group, seqs);  // rows of a sequence on average
  p.mt = each > 16 && dt == GPTQ_BF16 && c->head_dim <= 128 ? 4 : 1;
  p.tasks = tokens * group / (16 * p.mt) + seqs;
  // splits: as many as give 1024 workgroups, 256 keys each at least
  const int64_t tiles = hmin(p.tasks, seqs * ceil_div(each, int64_t(16) * p.mt)) * c->heads;
  const int64_t keys = hmin(width * c->page_size, int64_t(1) << 30);
  p.splits = (int)hmax(1, hmin(hmin(ceil_div(1024, tiles), 64), keys / 256));
  return p;
}

}  // namespace

size_t kv_attention_ws_bytes(const gptq_kv_blocks* c, int q_heads, int dt, int64_t tokens,
                             int64_t seqs, int64_t width) {
  const Plan p = plan_of(c, q_heads, dt, tokens, seqs, width);
  if (p.splits == 1) return 0;
  return (size_t)p.tasks * c->heads * p.splits * 16 * p.mt * (padded_dim(c->head_dim) + 2) * 4;
}

hipError_t launch_kv_attention(const KvAttention& t, const KvSequences& seqs,
                               const gptq_kv_blocks* kb, const gptq_kv_blocks* vb, int32_t* info,
                               void* ws, hipStream_t stream) {
  const Plan p = plan_of(kb, t.q_heads, t.dt, seqs.tokens, seqs.seqs, seqs.width);
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
  a.by_rows = divisor_of(16 * p.mt);
  a.stats = static_cast<float2*>(ws);
  a.parts = reinterpret_cast<float*>(a.stats + p.tasks * kb->heads * p.splits * 16 * p.mt);
  const bool even = kb->page_size % 16 == 0 && kb->block % 16 == 0;
  const dim3 grid((unsigned)p.tasks, (unsigned)kb->heads, (unsigned)p.splits), block(kThreads);
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
    else GPTQ_ATTN_F(DP, false, 4);           \
  } while (0)
  if (dp == 64) GPTQ_ATTN(64);
  else if (dp == 128) GPTQ_ATTN(128);
  else if (f32) GPTQ_ATTN_F(256, true, 1);
  else GPTQ_ATTN_F(256, false, 1);
#undef GPTQ_ATTN
#undef GPTQ_ATTN_F
#undef GPTQ_ATTN_E
  if (p.splits > 1) {
    const dim3 jgrid((unsigned)p.tasks, (unsigned)kb->heads);
#define GPTQ_JOIN(DP)                                                                                     \
  do {                                                                                                    \
    if (f32) hipLaunchKernelGGL((kv_attention_join_kernel<DP, true>), jgrid, block, 0, stream, a, 16 * p.mt); \
    else hipLaunchKernelGGL((kv_attention_join_kernel<DP, false>), jgrid, block, 0, stream, a, 16 * p.mt);    \
  } while (0)
    if (dp == 64) GPTQ_JOIN(64);
    else if (dp == 128) GPTQ_JOIN(128);
    else GPTQ_JOIN(256);
#undef GPTQ_JOIN
  }
  return hipGetLastError();
}

}  // namespace gptq
