// Drafted tokens against the model that judges them, from given random numbers.
//
// A sequence's rows t0 .. t0 + d hold the target's logits behind each of its d drafted tokens;
// ids[t] is the token that row t judges.  With p and q the target's and the drafter's
// probabilities, token x of row t is accepted while u[t] q(x) < p(x); behind the first refusal
// the next token has the weights max(p - q, 0), behind the last accepted one p, and is the
// smallest v with C(v) > u' C(vocab - 1), C the running sum of the weights: the tokens are
// then distributed as if the target had drawn each of them.
//
// The acceptance needs both models' logits once, one sum over each row, in fp32: with d = (m - x) / temperature a
// probability is off by 4 (d + ln vocab) 2^-24 and some roundings more at most, four of them in each exponent and the
// mean of d over the sum at most ln vocab.  A token moves across u q = p with that chance.  The draw compares a sum
// over up to the whole vocabulary with a border; fp32's error would be as wide as many a token's
// share, so the one row per sequence that is drawn from is summed in fp64.
//
// Three kernels: statistics of every row (the logits' stream: 64 sequences of 8 rows, 32000 fp32 logits of
// both models in 20 us, 6 TB/s), acceptance with the sums of the row that is drawn from (12 us) and the draw
// (16): chains of four and six round trips to memory, with some 50 fp64 operations a logit between them.
// 4 sequences of 5 rows, 128000 bf16 logits: 6, 9 and 13 us.
#include "kv_blocks.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxSegs = 64;  // a lane each
constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;

struct Stat {  // of a row or a part of it: the largest logit, the sum of e^((x - m) / temperature), its place
  float m, sum;
  int32_t at;
};

struct VerifyCall {
  VerifyArgs v;
  Stat* stats;     // [2][tokens][segs]
  double* sums;    // [3][seqs][dsegs]: e^((x - m) / temperature) of the target, of the drafter, the weights
  int4* draws;     // [seqs]: the row that is drawn from (-1: none), whether the drafter's law is taken off,
                   // the bits of both maxima
  int32_t segs, dsegs;
  int64_t seg, dseg;  // logits of a segment
};

__device__ __forceinline__ float temperature(const VerifyCall& a, int seq) {
  return a.v.temps ? a.v.temps[seq] : 1.0f;
}

// log2(e) / t, at most fp32's largest number (which t < 2^-127 would pass): logits 2^-100 apart are then far apart
// still, and a difference of 0 stays 0
__device__ __forceinline__ float exponent_scale(float t) {
  const float c = kLog2e / t;
  return c == __builtin_inff() ? 0x1.fffffep127f : c;
}

// TD, DD: the types of the target's and the drafter's logits
template <int TD, int DD>
__device__ __forceinline__ float logit(const VerifyCall& a, bool draft, int64_t row, int64_t i) {
  return draft ? load_elem(a.v.draft, DD, row * a.v.ldd + i) : load_elem(a.v.target, TD, row * a.v.ldt + i);
}

// lane sums, the same in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += lane_xorf<1>(v);
  v += lane_xorf<2>(v);
  v += lane_xorf<7>(v);
  v += lane_xorf<15>(v);
  v += lane_xorf<16>(v);
  v += lane_xorf<32>(v);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
  v = min(v, (int)lane_xor<1>(v));
  v = min(v, (int)lane_xor<2>(v));
  v = min(v, (int)lane_xor<7>(v));
  v = min(v, (int)lane_xor<15>(v));
  v = min(v, (int)lane_xor<16>(v));
  v = min(v, (int)lane_xor<32>(v));
  return v;
}

// the wave's parts as one; c: log2(e) / temperature, 0 where only the largest logit counts
__device__ __forceinline__ Stat wave_join(Stat s, float c) {
  Stat o;
  o.m = lanes_max<64>(s.m);
  // (a part that holds nothing finite has sum 0, or NaN where it holds a NaN or +inf; maxima may be farther
  // apart than any number, and infinity times 0 is none)
  o.sum = wave_sum(s.m == kNegInf || c == 0.0f ? s.sum : s.sum * __builtin_amdgcn_exp2f((s.m - o.m) * c));
  o.at = wave_min(s.m == o.m ? s.at : INT32_MAX);
  return o;
}

// s + a for a long sum: c is what the additions so far have added too much
__device__ __forceinline__ void add_to(float& s, float& c, float a) {
  const float y = a - c, n = s + y;
  c = (n - s) - y;
  s = n;
}

// A lane's logits c .. c + 7 into its statistics.  GREEDY: only the largest and its place count, the sum
// is 1 where something is finite, NaN where something is NaN or +inf.
template <bool GREEDY>
__device__ __forceinline__ void take8(const Vals8& v, int64_t c, float scale, Stat& s, float& carry) {
  float cm = v.v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) cm = fmaxf(cm, v.v[k]);
  if (cm > s.m) {
    if constexpr (GREEDY) {
      int first = 0;
#pragma unroll
      for (int k = 7; k >= 0; --k)
        if (v.v[k] == cm) first = k;
      s.at = (int32_t)c + first;
      if (!(s.sum != s.sum)) s.sum = 1.0f;
    } else if (s.m != kNegInf) {
      const float w = __builtin_amdgcn_exp2f((s.m - cm) * scale);
      s.sum *= w;
      carry *= w;
    }
    s.m = cm;
  }
  if constexpr (GREEDY) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!(v.v[k] < __builtin_inff())) s.sum = __builtin_nanf("");
  } else {
    const float base = s.m == kNegInf ? 0.0f : s.m;
    float e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = __builtin_amdgcn_exp2f((v.v[k] - base) * scale);
    add_to(s.sum, carry, ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
  }
}

template <int DT, bool GREEDY>
__device__ __forceinline__ Stat part_stat(const char* x, int64_t n, float scale) {
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  constexpr int AHEAD = 4;  // chunks under way
  // chunks of 8 lie on 16-byte borders, the first one beginning `off` places in front of the row
  const int off = (int)(reinterpret_cast<uintptr_t>(x) / esz % (16 / esz));
  Stat s{kNegInf, 0.0f, 0};
  float carry = 0.0f;
  for (int64_t p = 8 * (int)threadIdx.x - off; p < n; p += AHEAD * 8 * kThreads) {
    Raw8<DT> raw[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) raw[k] = load_chunk<DT>(x, p + k * 8 * kThreads, n);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t c = p + k * 8 * kThreads;
      Vals8 v = vals_of(raw[k]);
      if (c < 0 || c + 8 > n) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < 0 || c + e >= n) v.v[e] = kNegInf;
      }
      take8<GREEDY>(v, c, scale, s, carry);
    }
  }
  return s;
}

// A workgroup per row, segment and model.
__global__ __launch_bounds__(kThreads) void verify_stats_kernel(VerifyCall a) {
  __shared__ Stat part[kWaves];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const bool draft = blockIdx.z == 1;
  Sequences q = {};
  q.starts = a.v.starts;
  q.lengths = a.v.starts;  // (not used)
  q.seqs = (int32_t)a.v.seqs;
  q.tokens = (int32_t)a.v.tokens;
  int first;
  const Span sp = span_of(q, (int)row, 1, Divisor{1, 0}, 0, first);
  if (row < sp.start || row >= sp.start + sp.rows) return;
  if (draft && row == sp.start + sp.rows - 1) return;  // its logits judge nothing
  const float t = temperature(a, sp.seq);
  if (draft && t == 0.0f) return;
  const float c = exponent_scale(t);
  const int64_t c0 = blockIdx.y * a.seg, n = min(a.seg, a.v.vocab - c0);
  const int dt = draft ? a.v.ddt : a.v.tdt;
  const char* x = static_cast<const char*>(draft ? a.v.draft : a.v.target) +
                  (row * (draft ? a.v.ldd : a.v.ldt) + c0) * (dt == GPTQ_BF16 ? 2 : 4);
  Stat s;
  if (t == 0.0f) s = dt == GPTQ_BF16 ? part_stat<GPTQ_BF16, true>(x, n, 0.0f) : part_stat<GPTQ_F32, true>(x, n, 0.0f);
  else s = dt == GPTQ_BF16 ? part_stat<GPTQ_BF16, false>(x, n, c) : part_stat<GPTQ_F32, false>(x, n, c);
  s.at += (int32_t)c0;
  const float jc = t == 0.0f ? 0.0f : c;
  s = wave_join(s, jc);
  if ((tid & 63) == 0) part[tid >> 6] = s;
  __syncthreads();
  if (tid < 64) {
    s = wave_join(tid < kWaves ? part[tid] : Stat{kNegInf, 0.0f, INT32_MAX}, jc);
    if (tid == 0) a.stats[((draft ? a.v.tokens : 0) + row) * a.segs + blockIdx.y] = s;
  }
}

// e^d for d <= 0 (a little more does no harm) to about 2^-42 of itself: 2^n times Taylor's series of
// e^x, x = f ln 2, |f| <= 1/2, whose next term is below 2^-42, its even and odd terms apart.  (The
// library's is correct to the last of 53 places; the sums are compared with multiples of 2^-24, and
// what they are off moves a token with a chance of 10^-7.)
__device__ __forceinline__ double exp64(double d) {
  const double y = fmax(d * 1.4426950408889634074, -1100.0);  // (2^-1100 is 0; a NaN is seen to below)
  const double n = rint(y), x = (y - n) * 0.69314718055994530942, z = x * x;
  double e = fma(z, 1.0 / 3628800.0, 1.0 / 40320.0), o = fma(z, 1.0 / 362880.0, 1.0 / 5040.0);
  e = fma(e, z, 1.0 / 720.0);
  o = fma(o, z, 1.0 / 120.0);
  e = fma(e, z, 1.0 / 24.0);
  o = fma(o, z, 1.0 / 6.0);
  e = fma(e, z, 0.5);
  o = fma(o, z, 1.0);
  e = fma(e, z, 1.0);
  const double r = ldexp(fma(o, x, e), (int)n);
  return d == d ? r : d;
}

__device__ __forceinline__ double lane_xor_d(double v, int m) { return __shfl_xor(v, m); }

__device__ __forceinline__ double block_sum(double v, double* part) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += lane_xor_d(v, m);
  __syncthreads();
  if ((tid & 63) == 0) part[tid >> 6] = v;
  __syncthreads();
  return ((part[0] + part[1]) + part[2]) + part[3];
}

// A workgroup per sequence and segment: how many drafted tokens are accepted (the first one writes what
// follows from it), then the segment's sums of the row that the next token is drawn from.
template <int TD, int DD>
__global__ __launch_bounds__(kThreads) void verify_accept_kernel(VerifyCall a) {
  constexpr int EACH = 2, ROUND = EACH * kWaves;  // rows of a wave, of the workgroup, at a time
  __shared__ int refused;
  __shared__ Stat seen[ROUND];
  __shared__ float seen_mq[ROUND];
  __shared__ bool seen_in[ROUND];  // the id is in the vocabulary
  __shared__ double part[kWaves];
  const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool writes = blockIdx.y == 0;
  const int T = (int)a.v.tokens;
  const int s0 = min(max(a.v.starts[seq], 0), T), n = min(max(a.v.starts[seq + 1], 0), T) - s0;
  const float t = temperature(a, seq);
  if (n <= 0) {
    if (writes && tid == 0) {
      a.v.accepted[seq] = 0;
      a.draws[seq].x = -1;
    }
    return;
  }
  const bool sure = t == 0.0f, law_q = a.v.draft != nullptr && !sure;
  const float c = sure ? 0.0f : exponent_scale(t);
  if (tid == 0) refused = n - 1;  // (the last row judges nothing)
  __syncthreads();
  int taken = 0, at = 0;
  for (int k = 0;; k += ROUND) {
    int64_t row[EACH], id[EACH];
    Stat st[EACH], sd[EACH];
    float u[EACH], xt[EACH], xd[EACH];
    bool in[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {  // (behind the last row: that row once more)
      row[e] = s0 + min(k + e * kWaves + wave, n - 1);
      id[e] = a.v.ids[row[e]];
      u[e] = a.v.u[row[e]];
      st[e] = a.stats[row[e] * a.segs + min(lane, a.segs - 1)];
      sd[e] = st[e];
      if (law_q && row[e] < s0 + n - 1) sd[e] = a.stats[(a.v.tokens + row[e]) * a.segs + min(lane, a.segs - 1)];
      in[e] = id[e] >= 0 && id[e] < a.v.vocab;
    }
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      xt[e] = logit<TD, DD>(a, false, row[e], in[e] ? id[e] : 0);
      xd[e] = law_q ? logit<TD, DD>(a, true, row[e], in[e] ? id[e] : 0) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int j = k + e * kWaves + wave;
      const Stat none{kNegInf, 0.0f, INT32_MAX};
      const Stat p = wave_join(lane < a.segs ? st[e] : none, c), q = wave_join(lane < a.segs ? sd[e] : none, c);
      bool good = in[e] && j < n - 1;
      if (sure) {
        good = good && p.sum > 0.0f && p.at == id[e];
      } else {
        const float qx = law_q ? __builtin_amdgcn_exp2f((xd[e] - q.m) * c) / q.sum : 1.0f;
        good = good && u[e] * qx < __builtin_amdgcn_exp2f((xt[e] - p.m) * c) / p.sum;
      }
      if (lane == 0 && j < n) {
        if (!good) atomicMin(&refused, j);
        seen[e * kWaves + wave] = p;
        seen_mq[e * kWaves + wave] = q.m;
        seen_in[e * kWaves + wave] = in[e];
        if (writes && j < n - 1) {
          a.v.out[row[e]] = id[e];
          if (a.v.logprobs) a.v.logprobs[row[e]] = sure ? 0.0f : (xt[e] - p.m) / t - logf(p.sum);
        }
      }
    }
    __syncthreads();
    taken = refused;
    at = taken - k;
    if (at < ROUND) break;
    __syncthreads();  // (everyone has read it)
  }
  const int64_t row = s0 + taken;
  if (writes)
    for (int j = taken + tid; j < n; j += kThreads) {
      a.v.out[s0 + j] = -1;
      if (a.v.logprobs) a.v.logprobs[s0 + j] = 0.0f;
    }
  const bool judged = taken < n - 1 && (a.v.draft || seen_in[at]);
  const Stat top = seen[at];
  const float mq = seen_mq[at];
  const bool law = top.sum > 0.0f && top.sum < __builtin_inff();  // numbers, one of them finite
  __syncthreads();  // (-1 is written before what may follow it)
  if (writes && tid == 0) {
    a.v.accepted[seq] = taken;
    a.draws[seq] = make_int4(law && !sure ? (int)row : -1, judged, __float_as_int(top.m), __float_as_int(mq));
    if (law && sure) a.v.out[row] = top.at;
  }
  if (sure || !law) return;
  constexpr int AHEAD = 8;  // logits of a thread and model under way
  const bool both = judged && a.v.draft;
  const double it = 1.0 / (double)t, m = top.m, md = mq;
  const int64_t c0 = blockIdx.y * a.dseg, c1 = min(c0 + a.dseg, a.v.vocab);
  double s = 0.0, sq = 0.0;
  for (int64_t i = c0 + tid; i < c1; i += AHEAD * kThreads) {
    float x[AHEAD], y[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      const int64_t k = min(i + e * kThreads, c1 - 1);
      x[e] = logit<TD, DD>(a, false, row, k);
      y[e] = both ? logit<TD, DD>(a, true, row, k) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      const double v = exp64(((double)x[e] - m) * it);
      if (i + e * kThreads < c1) s += v;
    }
    if (both) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const double v = exp64(((double)y[e] - md) * it);
        if (i + e * kThreads < c1) sq += v;
      }
    }
  }
  s = block_sum(s, part);
  if (both) sq = block_sum(sq, part);
  if (tid == 0) {
    a.sums[(int64_t)seq * a.dsegs + blockIdx.y] = s;
    a.sums[(a.v.seqs + seq) * a.dsegs + blockIdx.y] = sq;
    a.sums[(2 * a.v.seqs + seq) * a.dsegs + blockIdx.y] = -1.0;  // (not known yet)
  }
}

struct Law {  // of the row that is drawn from
  double it, m, mq, zp, zq;  // zp, zq: 1 / the sums
  int64_t row, id;
  bool judged, draft;
};

// the weight of token i from its two logits
__device__ __forceinline__ double weight_of(const Law& w, int64_t i, float xt, float xd) {
  const double p = exp64(((double)xt - w.m) * w.it) * w.zp;
  if (!w.judged) return p;
  double q;
  if (w.draft) q = exp64(((double)xd - w.mq) * w.it) * w.zq;
  else q = i == w.id ? 1.0 : 0.0;
  return fmax(p - q, 0.0);
}

// logits of tokens i, i + kThreads, .. (behind c1: the last one's)
template <int N>
struct Pairs {
  float xt[N], xd[N];
};
template <int TD, int DD, int N>
__device__ __forceinline__ Pairs<N> pairs_at(const VerifyCall& a, int64_t row, bool both, int64_t i, int64_t c1) {
  Pairs<N> p;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int64_t k = min(i + e * kThreads, c1 - 1);
    p.xt[e] = logit<TD, DD>(a, false, row, k);
    p.xd[e] = both ? logit<TD, DD>(a, true, row, k) : 0.0f;
  }
  return p;
}

// their weights, 0 from c1 on
template <int N>
__device__ __forceinline__ void weights_of(const Law& w, const Pairs<N>& p, int64_t i, int64_t c1, double (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const double x = weight_of(w, i + e * kThreads, p.xt[e], p.xd[e]);
    v[e] = i + e * kThreads < c1 ? x : 0.0;
  }
}

// the sum of the lanes' numbers
__device__ __forceinline__ double total_of(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += lane_xor_d(v, m);
  return v;
}

// the wave's running sums
__device__ __forceinline__ double wave_scan(double v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(v, s);
    if (lane >= s) v += y;
  }
  return v;
}

// A workgroup per sequence and segment sums the segment's weights; one that finds all of the sequence's
// sums there finds the segment that holds the border, and in it the token.  That is the last one to be
// done; others that are done at the same time may find them too, and write the same.
template <int TD, int DD>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyCall a) {
  constexpr int AHEAD = 8, CHUNK = AHEAD * kThreads;
  __shared__ double part[kWaves];
  __shared__ double held[CHUNK + CHUNK / AHEAD];  // a thread's run of 8 apart from the next one's, by a place
  __shared__ int chosen;
  const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // two round trips in front of the sums: what hangs on the sequence alone, what hangs on the row
  const int4 d = a.draws[seq];
  const float t = temperature(a, seq), next = a.v.u_next[seq];
  const double sum_p = lane < a.dsegs ? a.sums[(int64_t)seq * a.dsegs + lane] : 0.0;
  const double sum_q = lane < a.dsegs ? a.sums[(a.v.seqs + seq) * a.dsegs + lane] : 0.0;
  if (d.x < 0) return;
  Law w;
  w.row = d.x;
  w.judged = d.y != 0;
  w.draft = a.v.draft != nullptr;
  const bool both = w.judged && w.draft;
  const int64_t s0 = blockIdx.y * a.dseg, s1 = min(s0 + a.dseg, a.v.vocab);
  Pairs<AHEAD> pairs = pairs_at<TD, DD, AHEAD>(a, w.row, both, s0 + tid, s1);
  w.id = a.v.ids[d.x];
  w.it = 1.0 / (double)t;
  w.m = __int_as_float(d.z);
  w.mq = __int_as_float(d.w);
  w.zp = 1.0 / total_of(sum_p);
  w.zq = both ? 1.0 / total_of(sum_q) : 1.0;
  double* const sums = a.sums + (2 * a.v.seqs + seq) * a.dsegs;
  {
    double s = 0.0;
    for (int64_t b = s0; b < s1; b += CHUNK) {
      if (b > s0) pairs = pairs_at<TD, DD, AHEAD>(a, w.row, both, b + tid, s1);
      double v[AHEAD];
      weights_of(w, pairs, b + tid, s1, v);
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) s += v[e];
    }
    s = block_sum(s, part);
    if (tid == 0) {
      // The sum goes past the caches by itself and has arrived before the others' are read: a store and loads at
      // the device's scope with a wait between them, which is how sequentially consistent ones are made on this
      // chip, less the fence in front of them, which nothing here needs and which would write back everything
      // that this part of the chip holds (64 sequences: 37 us, not 14).  So of two workgroups one at least sees
      // the other's sum, and the one whose sum arrives last sees them all.
      __hip_atomic_store(sums + blockIdx.y, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    __syncthreads();
  }
  double mine = lane < a.dsegs ? __hip_atomic_load(sums + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  if (__syncthreads_or(mine < 0.0)) return;
  double total = mine;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) total += lane_xor_d(total, m);
  if (!(total > 0.0)) {  // p = q, or no number among the drafter's: the target's own law
    w.judged = false;
    mine = sum_p * w.zp;
    total = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) total += lane_xor_d(total, m);
  }
  const double border = fmin(fmax((double)next, 0.0), 0x1.fffffep-1) * total;
  // running sums over the segments: the first one that passes the border (rounding may leave it behind
  // all of them: the last one with any weight)
  const double upto = wave_scan(mine);
  const uint64_t pass = __ballot(lane < a.dsegs && mine > 0.0 && upto > border), any = __ballot(mine > 0.0);
  if (any == 0) return;
  const int g = pass ? __ffsll((unsigned long long)pass) - 1 : 63 - __clzll((long long)any);
  double lead = __shfl(upto - mine, g);
  const int64_t c0 = g * a.dseg, c1 = min(c0 + a.dseg, a.v.vocab);
  // then over it, 8 consecutive tokens a thread
  int token = -1;
  for (int64_t b = c0; b < c1; b += CHUNK) {
    double v[AHEAD];
    weights_of(w, pairs_at<TD, DD, AHEAD>(a, w.row, w.judged && w.draft, b + tid, c1), b + tid, c1, v);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) held[(tid + e * kThreads) / AHEAD + tid + e * kThreads] = v[e];
    if (tid == 0) chosen = INT32_MAX;
    __syncthreads();
    double own = 0.0;
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      v[e] = held[tid + AHEAD * tid + e];
      own += v[e];
    }
    const double run = wave_scan(own);
    if (lane == 63) part[wave] = run;
    __syncthreads();
    double before = lead;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      if (k < wave) before += part[k];
      lead += part[k];
    }
    double c = before + (run - own);
    int latest = -1, first = -1;
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      c += v[e];
      if (v[e] > 0.0) {
        latest = AHEAD * tid + e;
        if (first < 0 && c > border) first = latest;
      }
    }
    if (first >= 0) atomicMin(&chosen, first);
    __syncthreads();
    if (chosen != INT32_MAX) {
      token = (int)b + chosen;
      break;
    }
    // nothing passes it here: keep the last token with any weight
    __syncthreads();
    if (tid == 0) chosen = -1;
    __syncthreads();
    if (latest >= 0) atomicMax(&chosen, latest);
    __syncthreads();
    if (chosen >= 0) token = (int)b + chosen;
  }
  if (token < 0 || tid != 0) return;
  a.v.out[w.row] = token;
  if (a.v.logprobs)
    a.v.logprobs[w.row] = (float)(((double)logit<TD, DD>(a, false, w.row, token) - w.m) * w.it + log(w.zp));
}

// Segments of a row of the statistics (rows and models in all), of a sequence's draw: as many as give
// 1024 workgroups, of whole rounds of 8 logits a thread.
struct Segments {
  int32_t count;
  int64_t size;
};
Segments segments(int64_t rows, int64_t vocab) {
  constexpr int64_t kRound = 8 * kThreads;
  const int64_t want = hmin(ceil_div(1024, hmax(rows, 1)), kMaxSegs);
  const int64_t size = ceil_div(ceil_div(vocab, want), kRound) * kRound;
  return Segments{(int32_t)ceil_div(vocab, size), size};
}

struct Layout {
  size_t draws, sums, bytes;
};

Layout layout_of(int64_t tokens, int64_t seqs, int64_t segs, int64_t dsegs) {
  Layout l;
  l.draws = align_up(2 * tokens * segs * sizeof(Stat), 16);
  l.sums = l.draws + seqs * sizeof(int4);
  l.bytes = l.sums + 3 * seqs * dsegs * sizeof(double);
  return l;
}

}  // namespace

size_t verify_ws_bytes(int64_t tokens, int64_t vocab, int64_t seqs) {
  return layout_of(tokens, seqs, segments(2 * tokens, vocab).count, segments(seqs, vocab).count).bytes;
}

hipError_t launch_verify(const VerifyArgs& v, hipStream_t stream) {
  if (!grid_fits(hmax(v.tokens, v.seqs), kThreads)) return hipErrorInvalidConfiguration;
  VerifyCall a;
  a.v = v;
  const Segments ss = segments(2 * v.tokens, v.vocab), ds = segments(v.seqs, v.vocab);
  a.segs = ss.count; a.seg = ss.size;
  a.dsegs = ds.count; a.dseg = ds.size;
  const Layout l = layout_of(v.tokens, v.seqs, a.segs, a.dsegs);
  char* ws = static_cast<char*>(v.ws);
  a.stats = reinterpret_cast<Stat*>(ws);
  a.draws = reinterpret_cast<int4*>(ws + l.draws);
  a.sums = reinterpret_cast<double*>(ws + l.sums);
  const dim3 block(kThreads);
  const unsigned models = v.draft ? 2 : 1;
  if (v.tokens > 0)
    hipLaunchKernelGGL(verify_stats_kernel, dim3((unsigned)v.tokens, (unsigned)a.segs, models), block, 0,
                       stream, a);
  const dim3 dgrid((unsigned)v.seqs, (unsigned)a.dsegs);
  // (a call without rows writes accepted = 0 and draws nothing: its u_next may be null)
#define GPTQ_DRAW(TD, DD)                                                                  \
  do {                                                                                     \
    hipLaunchKernelGGL((verify_accept_kernel<TD, DD>), dgrid, block, 0, stream, a);        \
    if (v.tokens > 0)                                                                      \
      hipLaunchKernelGGL((verify_draw_kernel<TD, DD>), dgrid, block, 0, stream, a);        \
  } while (0)
  if (v.tdt == GPTQ_BF16 && (!v.draft || v.ddt == GPTQ_BF16)) GPTQ_DRAW(GPTQ_BF16, GPTQ_BF16);
  else if (v.tdt == GPTQ_BF16) GPTQ_DRAW(GPTQ_BF16, GPTQ_F32);
  else if (!v.draft || v.ddt == GPTQ_F32) GPTQ_DRAW(GPTQ_F32, GPTQ_F32);
  else GPTQ_DRAW(GPTQ_F32, GPTQ_BF16);
#undef GPTQ_DRAW
  return hipGetLastError();
}

}  // namespace gptq
