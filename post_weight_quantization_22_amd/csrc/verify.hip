// Drafted tokens against the model that judges them, from given random numbers.
//
// A sequence's rows t0 .. t0 + d hold the target's logits behind each of its d drafted tokens;
// ids[t] is the token that row t judges.  With p and q the target's and the drafter's
// probabilities, token x of row t is accepted while u[t] q(x) < p(x); behind the first refusal
// the next token has the weights max(p - q, 0), behind the last accepted one p, and is the
// smallest v with C(v) > u' C(vocab - 1), C the running sum of the weights: the tokens are
// then distributed as if the target had drawn each of them.
//
// The acceptance needs both models' logits once, one sum over each row (fp32, relative error
// a few 2^-24, which moves a token across u q = p with that chance).  The draw compares a sum
// over up to the whole vocabulary with a border; fp32's error would be as wide as many a token's
// share, so the one row per sequence that is drawn from is summed in fp64.
#include "kv_blocks.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256;
constexpr int kStep = 8 * kThreads;  // logits of one step of a workgroup
constexpr float kNegInf = -__builtin_inff();

struct Stat {  // of a row or a part of it: maximum, sum of e^(x - maximum), where the maximum is
  float m, sum;
  int32_t at;
};

struct Draw {  // the row that a sequence's next token is drawn from
  int32_t row;    // -1: nothing is drawn
  int32_t judged; // whether the drafter's probabilities are taken off
  float m, mq;    // maxima of the target's and the drafter's logits
};

struct Kernel {
  VerifyArgs v;
  Stat* stats;    // [2][tokens][segs]
  Draw* draws;    // [seqs]
  double* sums;   // [3][seqs][segs]: e^(x - m) of the target, of the drafter, the weights
  int32_t segs;
  int64_t seg;    // logits of a segment
};

__device__ __forceinline__ float inverse_temp(const Kernel& a, int seq) {
  if (!a.v.temps) return 1.0f;
  const float t = a.v.temps[seq];
  return t == 0.0f ? 1.0f : 1.0f / t;
}
__device__ __forceinline__ bool greedy(const Kernel& a, int seq) {
  return a.v.temps && a.v.temps[seq] == 0.0f;
}

__device__ __forceinline__ Span row_span(const Kernel& a, int row) {
  Sequences q = {};
  q.starts = a.v.starts;
  q.lengths = a.v.starts;  // (not used)
  q.seqs = (int32_t)a.v.seqs;
  q.tokens = (int32_t)a.v.tokens;
  int first;
  return span_of(q, row, 1, Divisor{1, 0}, 0, first);
}

__device__ __forceinline__ float logit(const Kernel& a, bool draft, int64_t row, int64_t i) {
  return draft ? load_elem(a.v.draft, a.v.ddt, row * a.v.ldd + i) : load_elem(a.v.target, a.v.tdt, row * a.v.ldt + i);
}

__device__ __forceinline__ Stat joined(const Stat& a, const Stat& b) {
  Stat o;
  const bool first = a.m > b.m || (a.m == b.m && a.at < b.at) || b.at < 0;
  o.at = first ? a.at : b.at;
  o.m = fmaxf(a.m, b.m);
  const float base = o.m == kNegInf ? 0.0f : o.m;
  o.sum = a.sum * expf(a.m - base) + b.sum * expf(b.m - base);
  return o;
}

__global__ __launch_bounds__(kThreads) void verify_stats_kernel(Kernel a) {
  __shared__ Stat part[kThreads];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const bool draft = blockIdx.z == 1;
  const Span sp = row_span(a, (int)row);
  if (row < sp.start || row >= sp.start + sp.rows) return;
  if (draft && row == sp.start + sp.rows - 1) return;  // its logits judge nothing
  const float it = inverse_temp(a, sp.seq);
  const int64_t c0 = blockIdx.y * a.seg, c1 = min(c0 + a.seg, a.v.vocab);
  Stat s{kNegInf, 0.0f, -1};
  for (int64_t i = c0 + tid; i < c1; i += kThreads) {
    const float x = logit(a, draft, row, i) * it;
    s = joined(s, Stat{x, x == kNegInf ? 0.0f : 1.0f, (int32_t)i});
  }
  part[tid] = s;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d >>= 1) {
    if (tid < d) part[tid] = joined(part[tid], part[tid + d]);
    __syncthreads();
  }
  if (tid == 0) a.stats[((draft ? a.v.tokens : 0) + row) * a.segs + blockIdx.y] = part[0];
}

__device__ __forceinline__ Stat row_stat(const Kernel& a, bool draft, int64_t row) {
  const Stat* p = a.stats + ((draft ? a.v.tokens : 0) + row) * a.segs;
  Stat s = p[0];
  for (int i = 1; i < a.segs; ++i) s = joined(s, p[i]);
  return s;
}

// A wave per sequence: how many drafted tokens are accepted, and where the next one comes from.
__global__ __launch_bounds__(64) void verify_accept_kernel(Kernel a) {
  const int seq = blockIdx.x, lane = threadIdx.x;
  const int T = (int)a.v.tokens;
  const int s0 = min(max(a.v.starts[seq], 0), T), s1 = min(max(a.v.starts[seq + 1], 0), T);
  const int n = s1 - s0;
  if (n <= 0) {
    if (lane == 0) {
      a.v.accepted[seq] = 0;
      a.draws[seq].row = -1;
    }
    return;
  }
  const float it = inverse_temp(a, seq);
  const bool sure = greedy(a, seq);
  int k = 0;
  for (; k < n - 1; k += 64) {
    const int j = k + lane;
    bool good = false;
    if (j < n - 1) {
      const int64_t row = s0 + j, id = a.v.ids[row];
      if (id >= 0 && id < a.v.vocab) {
        const Stat t = row_stat(a, false, row);
        if (sure) {
          good = t.at == id && t.sum > 0.0f;
        } else {
          const float p = expf(logit(a, false, row, id) * it - t.m) / t.sum;
          float q = 1.0f;
          if (a.v.draft) {
            const Stat d = row_stat(a, true, row);
            q = expf(logit(a, true, row, id) * it - d.m) / d.sum;
          }
          good = a.v.u[row] * q < p;
        }
      }
    }
    const uint64_t no = __ballot(!good);
    if (no) {
      k += __ffsll((unsigned long long)no) - 1;
      break;
    }
  }
  const int taken = min(k, n - 1);
  for (int j = lane; j < n; j += 64) {
    const int64_t row = s0 + j;
    float lp = 0.0f;
    if (j < taken && !sure) {
      const Stat t = row_stat(a, false, row);
      lp = logit(a, false, row, a.v.ids[row]) * it - t.m - logf(t.sum);
    }
    a.v.out[row] = j < taken ? a.v.ids[row] : -1;
    if (a.v.logprobs) a.v.logprobs[row] = lp;
  }
  if (lane != 0) return;
  a.v.accepted[seq] = taken;
  const int row = s0 + taken;
  const Stat t = row_stat(a, false, row);
  const bool law = t.sum > 0.0f && t.sum < __builtin_inff();  // a row of numbers, one of them finite
  Draw d{-1, 0, t.m, 0.0f};
  if (sure) {
    a.v.out[row] = law ? t.at : -1;
  } else if (law) {
    d.row = row;
    const int64_t id = a.v.ids[row];
    d.judged = taken < n - 1 && (a.v.draft || (id >= 0 && id < a.v.vocab));
    if (d.judged && a.v.draft) d.mq = row_stat(a, true, row).m;
  }
  a.draws[seq] = d;
}

__device__ __forceinline__ double block_sum(double v, double* part) {
  const int tid = threadIdx.x;
  __syncthreads();
  part[tid] = v;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d >>= 1) {
    if (tid < d) part[tid] += part[tid + d];
    __syncthreads();
  }
  return part[0];
}

__device__ __forceinline__ double total_of(const double* p, int n) {
  double s = 0.0;
  for (int i = 0; i < n; ++i) s += p[i];
  return s;
}

// e^(x - m) of a segment, summed in fp64
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(Kernel a) {
  __shared__ double part[kThreads];
  const int seq = blockIdx.x, tid = threadIdx.x;
  const Draw d = a.draws[seq];
  if (d.row < 0) return;
  const bool draft = blockIdx.z == 1;
  if (draft && !d.judged) return;
  const double it = a.v.temps ? 1.0 / (double)a.v.temps[seq] : 1.0;
  const int64_t c0 = blockIdx.y * a.seg, c1 = min(c0 + a.seg, a.v.vocab);
  const double m = draft ? d.mq : d.m;
  double s = 0.0;
  for (int64_t i = c0 + tid; i < c1; i += kThreads) s += exp((double)logit(a, draft, d.row, i) * it - m);
  s = block_sum(s, part);
  if (tid == 0) a.sums[(int64_t)(draft ? a.v.seqs + seq : seq) * a.segs + blockIdx.y] = s;
}

struct Law {
  double it, m, mq, zp, zq;
  int64_t row, id;
  bool judged, draft;
};

__device__ __forceinline__ double weight_of(const Kernel& a, const Law& w, int64_t i) {
  const double p = exp((double)logit(a, false, w.row, i) * w.it - w.m) / w.zp;
  if (!w.judged) return p;
  double q;
  if (w.draft) q = exp((double)logit(a, true, w.row, i) * w.it - w.mq) / w.zq;
  else q = i == w.id ? 1.0 : 0.0;
  return fmax(p - q, 0.0);
}

__device__ __forceinline__ Law law_of(const Kernel& a, int seq, const Draw& d) {
  Law w;
  w.it = a.v.temps ? 1.0 / (double)a.v.temps[seq] : 1.0;
  w.m = d.m; w.mq = d.mq;
  w.row = d.row;
  w.judged = d.judged;
  w.draft = a.v.draft != nullptr;
  w.id = a.v.ids[d.row];
  w.zp = total_of(a.sums + (int64_t)seq * a.segs, a.segs);
  w.zq = w.judged && w.draft ? total_of(a.sums + (a.v.seqs + seq) * a.segs, a.segs) : 1.0;
  return w;
}

__global__ __launch_bounds__(kThreads) void verify_weights_kernel(Kernel a) {
  __shared__ double part[kThreads];
  const int seq = blockIdx.x, tid = threadIdx.x;
  const Draw d = a.draws[seq];
  if (d.row < 0) return;
  const Law w = law_of(a, seq, d);
  const int64_t c0 = blockIdx.y * a.seg, c1 = min(c0 + a.seg, a.v.vocab);
  double s = 0.0;
  for (int64_t i = c0 + tid; i < c1; i += kThreads) s += weight_of(a, w, i);
  s = block_sum(s, part);
  if (tid == 0) a.sums[(2 * a.v.seqs + seq) * a.segs + blockIdx.y] = s;
}

// A workgroup per sequence: the segment that holds the border, then the token in it.
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(Kernel a) {
  __shared__ double part[kThreads];
  __shared__ int pick;
  const int seq = blockIdx.x, tid = threadIdx.x;
  const Draw d = a.draws[seq];
  if (d.row < 0) return;
  Law w = law_of(a, seq, d);
  const double* sums = a.sums + (2 * a.v.seqs + seq) * a.segs;
  double total = total_of(sums, a.segs);
  if (!(total > 0.0)) {  // p = q, or no number among the drafter's: the target's own law
    w.judged = false;
    sums = a.sums + (int64_t)seq * a.segs;
    total = w.zp;
  }
  const double unit = sums == a.sums + (int64_t)seq * a.segs ? w.zp : 1.0;  // (these are not divided yet)
  const double border = fmax((double)a.v.u_next[seq], 0.0) * (total / unit);
  // the last segment with any weight, if rounding leaves the border behind all of them
  int s = -1, last = 0;
  double before = 0.0, upto = 0.0;
  for (int i = 0; i < a.segs; ++i) {
    const double x = sums[i] / unit;
    if (x > 0.0) last = i;
    if (s < 0 && upto + x > border) {
      s = i;
      before = upto;
    }
    upto += x;
  }
  if (s < 0) {
    s = last;
    before = upto;
  }
  const int64_t c0 = s * a.seg, c1 = min(c0 + a.seg, a.v.vocab);
  if (tid == 0) pick = -1;
  int latest = -1;  // the last token with any weight
  double run = before;
  bool found = false;
  for (int64_t i0 = c0; i0 < c1 && !found; i0 += kThreads) {
    const int64_t i = i0 + tid;
    const double x = i < c1 ? weight_of(a, w, i) : 0.0;
    if (x > 0.0) latest = (int)i;
    __syncthreads();
    part[tid] = x;
    __syncthreads();
    for (int st = 1; st < kThreads; st <<= 1) {  // running sums
      const double y = tid >= st ? part[tid - st] : 0.0;
      __syncthreads();
      part[tid] += y;
      __syncthreads();
    }
    const double mine = run + part[tid], prev = tid ? run + part[tid - 1] : run;
    if (i < c1 && mine > border && !(prev > border)) pick = (int)i;
    run += part[kThreads - 1];
    found = run > border;
    __syncthreads();
  }
  int best = pick;
  if (best < 0) {
    __shared__ int lasts[kThreads];
    lasts[tid] = latest;
    __syncthreads();
    for (int i = 0; i < kThreads; ++i) best = max(best, lasts[i]);
  }
  if (tid == 0 && best >= 0) {
    a.v.out[d.row] = best;
    if (a.v.logprobs)
      a.v.logprobs[d.row] = (float)((double)logit(a, false, d.row, best) * w.it - w.m - log(w.zp));
  }
}

int segments(int64_t rows, int64_t vocab) {
  return (int)hmax(1, hmin(hmin(ceil_div(1024, rows), 64), vocab / kStep));
}

struct Layout {
  size_t stats, draws, sums, bytes;
};

Layout layout_of(int64_t tokens, int64_t seqs, int64_t segs) {
  Layout l;
  l.stats = 0;
  l.draws = align_up(2 * tokens * segs * sizeof(Stat), 16);
  l.sums = align_up(l.draws + seqs * sizeof(Draw), 16);
  l.bytes = l.sums + 3 * seqs * segs * sizeof(double);
  return l;
}

}  // namespace

size_t verify_ws_bytes(int64_t tokens, int64_t vocab, int64_t seqs) {
  return layout_of(tokens, seqs, segments(seqs, vocab)).bytes;
}

hipError_t launch_verify(const VerifyArgs& v, hipStream_t stream) {
  Kernel a;
  a.v = v;
  a.segs = segments(v.seqs, v.vocab);
  a.seg = ceil_div(v.vocab, a.segs);
  const Layout l = layout_of(v.tokens, v.seqs, a.segs);
  char* ws = static_cast<char*>(v.ws);
  a.stats = reinterpret_cast<Stat*>(ws + l.stats);
  a.draws = reinterpret_cast<Draw*>(ws + l.draws);
  a.sums = reinterpret_cast<double*>(ws + l.sums);
  const dim3 block(kThreads);
  const unsigned models = v.draft ? 2 : 1;
  if (v.tokens > 0)
    hipLaunchKernelGGL(verify_stats_kernel, dim3((unsigned)v.tokens, (unsigned)a.segs, models), block, 0,
                       stream, a);
  hipLaunchKernelGGL(verify_accept_kernel, dim3((unsigned)v.seqs), dim3(64), 0, stream, a);
  hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)v.seqs, (unsigned)a.segs, models), block, 0,
                     stream, a);
  hipLaunchKernelGGL(verify_weights_kernel, dim3((unsigned)v.seqs, (unsigned)a.segs), block, 0, stream, a);
  hipLaunchKernelGGL(verify_draw_kernel, dim3((unsigned)v.seqs), block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace gptq
