// Log probabilities of given tokens, the entropy and the top alternatives of
// each row of logits, in one pass over the logits.
//
// "Quantized deployment, 1.5 TB to 250 GB" (lmnt.cn news 123823), section 3.1:
// a quantized model is judged by its perplexity, exp of the mean negative log
// probability of the text's tokens.  For a row x of V logits with largest
// element m (one instance of it left out of the sums below):
//   r = sum e^(x - m),  t = sum e^(x - m) (x - m)
//   log p(id) = x[id] - m - log1p(r)
//   entropy   = log1p(r) - t / (1 + r)
// Leaving the largest element out keeps the digits of a row whose best token is
// almost certain (log p of that token is -log1p(r), not log of a sum near 1).
// (m, r, t) of two parts join: with m1 >= m2, d = m2 - m1, w = e^d
//   r = r1 + w (1 + r2),  t = t1 + w (t2 + d (1 + r2)).
// A lane of a long row adds hundreds of terms to one sum: each chunk's 8 are added in a
// tree, and the chunks with what each addition rounds off carried along, so the sums'
// error does not grow with V (one term after another, 1024 equal ones, it is 2^-16).
//
// Bound by HBM: each logit is read once (2048 x 32000 fp32 in 51 us, 5.1 TB/s, with 5
// alternatives 57; bf16 halves the bytes, not the sums' instructions: 34 and 40 us).  Few
// rows by latency: 4 x 128000 7.9 us and 5.4 us to join the segments.
// A workgroup of 256 takes a row (or a segment of it, where there are few rows; a
// second kernel joins the segments).
// A lane keeps (m, r, t) of its own logits and the place of its m.  The top
// alternatives are found among few candidates: with K the k-th best of the 256
// lanes' best (value, place) pairs, at least k logits are no worse than K, and
// only the k lanes whose best is no worse than K can hold one; the logits of
// those lanes are read once more (from L2) and listed.  Pairs are ordered by value,
// then by the lower index, so all are distinct and the result does not depend
// on the order in which the list was filled.
#include "fp8.hpp"
#include "lanes.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256;
constexpr int kTopMax = 32;
constexpr int kList = 1024;  // candidates held in LDS
constexpr float kNegInf = -__builtin_inff();
// differences are held to this before they are multiplied: e^kFar is 0, and 0
// times a difference of masked logits (-inf, or the type's lowest value) stays 0
constexpr float kFar = -1000.0f;

struct Part {
  float m, r, t;
};

// e^d as 2^(d log2 e), the product rounded to 32 bits: off by |d| 2^-24 of itself and an
// ulp, at most 2^-25 of the largest term (|d| e^d <= 1 / e).  2048 x 50257 bf16 over and
// over 51 us, with expf 78.
__device__ __forceinline__ float exp_of(float d) { return __expf(d); }

// s + a for a long sum: c is what the additions so far have added too much
__device__ __forceinline__ void add_to(float& s, float& c, float a) {
  const float y = a - c, n = s + y;
  c = (n - s) - y;
  s = n;
}

__device__ __forceinline__ Part join(Part a, Part b) {
  if (b.m > a.m) {
    const Part c = a;
    a = b;
    b = c;
  }
  if (b.m == kNegInf) {  // nothing on that side but, possibly, a NaN
    a.r += b.r;
    return a;
  }
  const float d = fmaxf(b.m - a.m, kFar), w = expf(d);
  a.r += w * (1.0f + b.r);
  a.t += w * (b.t + d * (1.0f + b.r));
  return a;
}

// 64-bit order of (value, index): larger is better; ties and both zeros go to
// the lower index; NaN ranks with -inf.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t idx) {
  if (v != v) v = kNegInf;
  uint32_t u = __float_as_uint(v + 0.0f);
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return (uint64_t)u << 32 | (uint32_t)~idx;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

__device__ __forceinline__ uint64_t umax(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Of the pair (lane, lane ^ M) the lane without bit LOW keeps the larger key.
template <int M, int LOW>
__device__ __forceinline__ uint64_t exchange(uint64_t v) {
  const uint64_t o = lane_xor64<M>(v);
  return ((threadIdx.x & LOW) == 0) == (v > o) ? v : o;
}
// a bitonic run of 2 LOW lanes into descending order
template <int LOW>
__device__ __forceinline__ uint64_t merge_down(uint64_t v) {
  v = exchange<LOW, LOW>(v);
  if constexpr (LOW > 1) v = merge_down<LOW / 2>(v);
  return v;
}
// the wave's 64 keys in descending order: runs of 2, 4, .. 64, each from its two
// halves by a mirror exchange and a merge of each half
template <int SIZE = 2>
__device__ __forceinline__ uint64_t sort64(uint64_t v) {
  v = exchange<SIZE - 1, SIZE / 2>(v);
  if constexpr (SIZE > 2) v = merge_down<SIZE / 4>(v);
  if constexpr (SIZE < 64) v = sort64<2 * SIZE>(v);
  return v;
}

// the wave's parts as one, the same bits in every lane: the largest m, then each
// lane's sums taken to it, one of the lanes that hold it leaving it out
__device__ __forceinline__ Part wave_join(Part p) {
  float m = p.m;
  m = fmaxf(m, lane_xorf<1>(m));
  m = fmaxf(m, lane_xorf<2>(m));
  m = fmaxf(m, lane_xorf<7>(m));
  m = fmaxf(m, lane_xorf<15>(m));
  m = fmaxf(m, lane_xorf<16>(m));
  m = fmaxf(m, lane_xorf<32>(m));
  const uint64_t holders = __ballot(p.m == m);
  const bool owner = (int)(threadIdx.x & 63) == __ffsll((unsigned long long)holders) - 1;
  if (!owner && p.m != kNegInf) {
    const float d = fmaxf(p.m - m, kFar), w = expf(d);
    p.t = w * (p.t + d * (1.0f + p.r));
    p.r = w * (1.0f + p.r);
  }
  p.m = m;
  // (a lane and its mirror hold the same sum by then)
  p.r += lane_xorf<1>(p.r);   p.t += lane_xorf<1>(p.t);
  p.r += lane_xorf<2>(p.r);   p.t += lane_xorf<2>(p.t);
  p.r += lane_xorf<7>(p.r);   p.t += lane_xorf<7>(p.t);
  p.r += lane_xorf<15>(p.r);  p.t += lane_xorf<15>(p.t);
  p.r += lane_xorf<16>(p.r);  p.t += lane_xorf<16>(p.t);
  p.r += lane_xorf<32>(p.r);  p.t += lane_xorf<32>(p.t);
  return p;
}

struct Shared {
  uint64_t list[kList];
  uint64_t best[4 * kTopMax];
  uint64_t kth;
  Part part[4];
  int count;
};

// The best `top` of the workgroup's keys, one per lane (0: none), in descending
// order in best[0 .. top): every wave sorts its own, then the first wave merges.
__device__ __forceinline__ void best_of_lanes(Shared& sh, uint64_t mine) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint64_t v = sort64(mine);
  __syncthreads();
  if (lane < kTopMax) sh.best[wv * kTopMax + lane] = v;
  __syncthreads();
  if (wv == 0) {
    // of two descending lists of 32, the larger of a[i] and b[31 - i] are the best 32
    const int i = lane & 31, pair = lane >> 5;
    uint64_t k = umax(sh.best[pair * 64 + i], sh.best[pair * 64 + 63 - i]);
    k = merge_down<16>(k);
    k = merge_down<16>(umax(k, lane_xor64<63>(k)));
    if (lane < kTopMax) sh.best[lane] = k;
  }
  __syncthreads();
}

// The best `top` of list[0 .. n), n <= kList, in descending order in best[].
__device__ __forceinline__ void best_of_list(Shared& sh, int n, int top) {
  const int tid = threadIdx.x;
  if (n > 64) {
    // bring it down to few: only keys no worse than the top-th of the lanes' best
    uint64_t mine = 0, own[kList / kThreads];
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int i = j * kThreads + tid;
      own[j] = i < n ? sh.list[i] : 0;
      mine = umax(mine, own[j]);
    }
    best_of_lanes(sh, mine);
    const uint64_t kth = sh.best[top - 1];
    if (tid == 0) sh.count = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j)
      if (own[j] != 0 && own[j] >= kth) sh.list[atomicAdd(&sh.count, 1)] = own[j];
    __syncthreads();
    n = sh.count;
  }
  // at most top * kList / kThreads = 128 are left: two keys a lane of one wave
  if (tid < 64) {
    uint64_t a = tid < n ? sh.list[tid] : 0, b = 64 + tid < n ? sh.list[64 + tid] : 0;
    a = sort64(a);
    if (n > 64) {
      b = sort64(b);
      // both descending: the larger of a[i] and b[63 - i] are the best 64
      a = merge_down<32>(umax(a, lane_xor64<63>(b)));
    }
    if (tid < kTopMax) sh.best[tid] = a;
  }
  __syncthreads();
}

struct LpArgs {
  const void* X;
  int64_t tokens, vocab, ldx;
  const int64_t* ids;
  float* logprob;
  float* entropy;
  int top;
  int32_t* top_ids;
  float* top_logprobs;
  int64_t seg;  // logits of a segment, a multiple of 2048 (or the whole row)
  int nseg;
  Part* parts;      // [tokens][nseg], segments only
  uint64_t* keys;   // [tokens][nseg][top], segments only
};

__device__ __forceinline__ void write_row(const LpArgs& a, int64_t row, const Part& p,
                                          const uint64_t* best, int dt) {
  // a row with +inf has no distribution; a NaN is in r already
  const bool empty = p.m == kNegInf && p.r == 0.0f;
  const float bad = p.m == __builtin_inff() ? __builtin_nanf("") : 0.0f;
  const float l1 = log1pf(p.r) + bad;
  const int tid = threadIdx.x;
  if (tid == 0) {
    if (a.entropy) a.entropy[row] = empty ? 0.0f : l1 - p.t / (1.0f + p.r);
    if (a.ids) {
      const int64_t id = a.ids[row];
      float lp = 0.0f;
      if (id >= a.vocab) {
        lp = __builtin_nanf("");
      } else if (id >= 0) {
        const float x = load_elem(a.X, dt, row * a.ldx + id);
        lp = empty ? kNegInf : (x - p.m) - l1;
      }
      a.logprob[row] = lp;
    }
  }
  if (tid < a.top) {
    const uint64_t k = best[tid];
    a.top_ids[row * a.top + tid] = (int32_t)key_index(k);
    a.top_logprobs[row * a.top + tid] = empty ? kNegInf : (key_value(k) - p.m) - l1;
  }
}

// A workgroup per row and segment.  Its chunks of 8 logits lie on 16-byte borders, the
// first one beginning `off` places in front of the row (2048 x 50257 bf16, rows that start
// on any border: 51 us; loads of single logits took 2.3 times as long).
template <int DT>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LpArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int64_t c0 = (int64_t)blockIdx.y * a.seg;
  const int64_t n = min(a.seg, a.vocab - c0);
  constexpr int esz = DT == GPTQ_BF16 ? 2 : 4;
  const char* x = reinterpret_cast<const char*>(a.X) + (row * a.ldx + c0) * esz;

  const int off = (int)(reinterpret_cast<uintptr_t>(x) / esz % (16 / esz));
  const int64_t end = n + off;  // chunks are counted from 8 c - off on

  float m = kNegInf, mr = 0.0f, r = 0.0f, t = 0.0f;  // mr: m, or 0 before the first finite logit
  float rc = 0.0f, tc = 0.0f;                        // add_to's
  uint32_t at = max(8 * tid - off, 0);
  Raw8<DT> next;
  if (8 * tid < end) next = load_chunk<DT>(x, 8 * tid - off, n);
  for (int64_t p = 8 * tid; p < end; p += 8 * kThreads) {
    const int64_t c = p - off;
    Vals8 v = vals_of(next);
    if (p + 8 * kThreads < end) next = load_chunk<DT>(x, c + 8 * kThreads, n);
    if (c < 0 || c + 8 > n) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < 0 || c + k >= n) v.v[k] = kNegInf;
    }
    float cm = v.v[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) cm = fmaxf(cm, v.v[k]);
    if (cm > m) {  // rescale to the new largest, which the sums below leave out
      if (m != kNegInf) {
        const float d = fmaxf(m - cm, kFar), w = expf(d);
        t = w * (t + d * (1.0f + r));
        r = w * (1.0f + r);
        rc *= w;
        tc *= w;
      }
      int first = 0;
#pragma unroll
      for (int k = 7; k >= 0; --k)
        if (v.v[k] == cm) first = k;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k == first) v.v[k] = kNegInf;
      at = (uint32_t)c + first;
      m = mr = cm;
    }
    float e[8], f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = v.v[k] - mr;
      e[k] = exp_of(d);
      f[k] = e[k] * fmaxf(d, kFar);
    }
    add_to(r, rc, ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
    add_to(t, tc, ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7])));
  }

  Part p = wave_join(Part{m, r, t});
  if ((tid & 63) == 0) sh.part[tid >> 6] = p;

  if (a.top > 0) {
    const uint64_t mine = 8 * tid < end ? key_of(m, at) : 0;
    best_of_lanes(sh, mine);
    const uint64_t kth = sh.best[a.top - 1];
    if (tid == 0) sh.count = 0;
    __syncthreads();
    // the chunks of the lanes that hold candidates, dealt to all lanes: a key's
    // index says which lane it came from
    const int chunks = (int)((end + 8 * kThreads - 1) / (8 * kThreads));
    for (int u = tid; u < chunks * a.top; u += kThreads) {
      const uint64_t of = sh.best[u % a.top];
      const uint32_t lane = ((key_index(of) + off) >> 3) & (kThreads - 1);
      const int64_t c = 8 * (lane + (int64_t)(u / a.top) * kThreads) - off;
      if (of == 0 || c >= n) continue;
      const Vals8 v = vals_of(load_chunk<DT>(x, c, n));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t key = key_of(v.v[k], (uint32_t)c + k);
        if (c + k >= 0 && c + k < n && key >= kth) {
          const int i = atomicAdd(&sh.count, 1);
          if (i < kList) sh.list[i] = key;
        }
      }
    }
    __syncthreads();
    const int count = sh.count;
    __syncthreads();
    if (count <= kList) {
      best_of_list(sh, count, a.top);
    } else {
      // more candidates than the list holds (a few lanes hold most of the row's
      // large logits): one alternative after another, over the whole row
      uint64_t last = ~0ull;
      for (int i = 0; i < a.top; ++i) {
        uint64_t b = 0;
        for (int64_t c = 8 * tid - off; c < n; c += 8 * kThreads) {
          const Vals8 v = vals_of(load_chunk<DT>(x, c, n));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t key = key_of(v.v[k], (uint32_t)c + k);
            if (c + k >= 0 && c + k < n && key < last) b = umax(b, key);
          }
        }
        b = sort64(b);
        if ((tid & 63) == 0) sh.list[tid >> 6] = b;
        __syncthreads();
        last = umax(umax(sh.list[0], sh.list[1]), umax(sh.list[2], sh.list[3]));
        if (tid == 0) sh.best[i] = last;
        __syncthreads();
      }
    }
  } else {
    __syncthreads();
  }
  p = join(join(sh.part[0], sh.part[1]), join(sh.part[2], sh.part[3]));
  if (a.nseg == 1) {
    write_row(a, row, p, sh.best, DT);
    return;
  }
  const int64_t s = row * a.nseg + blockIdx.y;
  if (tid == 0) a.parts[s] = p;
  if (tid < a.top) {  // segments shorter than top leave none (0)
    const uint64_t k = sh.best[tid];
    a.keys[s * a.top + tid] = k == 0 ? 0 : key_of(key_value(k), key_index(k) + (uint32_t)c0);
  }
}

// A workgroup per row joins its segments.
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(LpArgs a, int dt) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  Part p = tid < a.nseg ? a.parts[row * a.nseg + tid] : Part{kNegInf, 0.0f, 0.0f};
  p = wave_join(p);
  if (tid == 0) sh.part[0] = p;  // at most 64 segments
  if (a.top > 0) {
    // nseg lists in descending order: a lane takes the j-th of 256 / nseg of them in turn
    const int total = a.nseg * a.top;
    uint64_t mine = 0;
    for (int i = tid; i < total; i += kThreads) mine = umax(mine, a.keys[row * total + i]);
    best_of_lanes(sh, mine);
    const uint64_t kth = sh.best[a.top - 1];
    if (tid == 0) sh.count = 0;
    __syncthreads();
    for (int i = tid; i < total; i += kThreads) {
      const uint64_t k = a.keys[row * total + i];
      if (k != 0 && k >= kth) sh.list[atomicAdd(&sh.count, 1)] = k;  // <= top * 2048 / 256
    }
    __syncthreads();
    const int n = sh.count;
    __syncthreads();
    best_of_list(sh, n, a.top);
  }
  __syncthreads();
  write_row(a, row, sh.part[0], sh.best, dt);
}

// Segments of a row: none from 256 rows on and for short rows, else as many as give 512
// workgroups; at least 2048 logits each, at most 64 of them (us, whole rows and
// segments: 1 x 16384 9.5 and 10.8, 1 x 24576 11.4 and 10.8, 4 x 128000 35 and 12.4,
// 200 x 128000 37 and 29; twice as many segments: the same).
int segments(int64_t tokens, int64_t vocab) {
  if (tokens >= 256 || vocab < 24576) return 1;
  const int64_t want = ceil_div(512, tokens);
  return (int)hmax(1, hmin(hmin(want, 64), vocab / 2048));
}

}  // namespace

size_t logprobs_ws_bytes(int64_t tokens, int64_t vocab, int top) {
  const int ns = segments(tokens, vocab);
  if (ns == 1) return 0;
  return align_up((size_t)tokens * ns * sizeof(Part), 16) + (size_t)tokens * ns * top * 8;
}

hipError_t launch_logprobs(const void* X, int dt, int64_t tokens, int64_t vocab, int64_t ldx,
                           const int64_t* ids, float* logprob, float* entropy, int top,
                           int32_t* top_ids, float* top_logprobs, void* ws, hipStream_t stream) {
  const int ns = segments(tokens, vocab);
  LpArgs a;
  a.vocab = vocab; a.ldx = ldx; a.top = top;
  a.seg = ns == 1 ? vocab : (ceil_div(vocab, ns) + 2047) / 2048 * 2048;
  a.nseg = (int)ceil_div(vocab, a.seg);
  a.parts = static_cast<Part*>(ws);
  a.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) +
                                       align_up((size_t)tokens * ns * sizeof(Part), 16));
  // rows of one launch: 256 threads each, fewer than 2^32 in all (more than 256
  // rows are never cut into segments, so the workspace is not offset)
  constexpr int64_t kRows = int64_t(1) << 20;
  for (int64_t t0 = 0; t0 < tokens; t0 += kRows) {
    a.X = static_cast<const char*>(X) + t0 * ldx * (dt == GPTQ_BF16 ? 2 : 4);
    a.tokens = hmin(tokens - t0, kRows);
    a.ids = ids ? ids + t0 : nullptr;
    a.logprob = logprob ? logprob + t0 : nullptr;
    a.entropy = entropy ? entropy + t0 : nullptr;
    a.top_ids = top ? top_ids + t0 * top : nullptr;
    a.top_logprobs = top ? top_logprobs + t0 * top : nullptr;
    const dim3 grid((unsigned)a.tokens, (unsigned)a.nseg);
    if (dt == GPTQ_BF16)
      hipLaunchKernelGGL(logprobs_kernel<GPTQ_BF16>, grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL(logprobs_kernel<GPTQ_F32>, grid, dim3(kThreads), 0, stream, a);
    if (a.nseg > 1)
      hipLaunchKernelGGL(logprobs_join_kernel, dim3((unsigned)a.tokens), dim3(kThreads), 0, stream,
                         a, dt);
  }
  return hipGetLastError();
}

}  // namespace gptq
