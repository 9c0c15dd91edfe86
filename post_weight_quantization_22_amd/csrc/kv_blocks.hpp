// Shared pieces of the operators on a paged cache with a scale per block of tokens
// and head: where a sequence's rows and keys lie.
#pragma once

#include "fp8.hpp"

namespace gptq {

// n / d for 0 <= n < 2^31: mul = floor(2^(32 + shift) / d) + 1, shift = floor(log2 d), is
// off by at most d < 2^(shift + 1) of 2^(32 + shift), too little to reach the next
// quotient; mul == 0 where d is a power of two.
struct Divisor {
  uint32_t mul;
  int32_t shift;
};

inline Divisor divisor_of(int64_t d) {
  int s = 0;
  while ((int64_t(2) << s) <= d) ++s;
  if ((d & (d - 1)) == 0) return Divisor{0, s};
  return Divisor{(uint32_t)((uint64_t(1) << (32 + s)) / (uint64_t)d + 1), s};
}

__device__ __forceinline__ int divided(int n, const Divisor& d) {
  return d.mul ? (int)(__umulhi((uint32_t)n, d.mul) >> d.shift) : n >> d.shift;
}

struct BlockCache {  // one of the two caches
  uint8_t* codes;
  float* scales;
  int64_t cpage, cslot, chead;   // codes, bytes
  int64_t ppage, pblock, phead;  // scales, elements
};

// The sequences of a call: new rows starts[i] .. starts[i + 1] - 1 stand at the last
// positions of lengths[i], whose pages table[i] lists.
struct Sequences {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  int64_t ldt;
  int32_t width, seqs, tokens;
  int32_t pages, page_size, block;
  Divisor by_page, by_block;
  int32_t* info;
};

struct Span {  // a sequence's new rows (none where the starts do not ascend)
  int seq, start, rows, length;
};

// The sequence that task t belongs to, and its first task: sequence i has the tasks from
// starts[i] * num / den + i * extra on (each wave finds it by itself, 64 sequences a step;
// starts that do not ascend lead to some sequence of the call all the same).
// tokens * num < 2^31.
__device__ __forceinline__ Span span_of(const Sequences& q, int t, int num, const Divisor& den,
                                        int extra, int& first) {
  const int lane = threadIdx.x & 63;
  auto start_at = [&](int i) { return min(max(q.starts[i], 0), q.tokens); };
  auto task_at = [&](int i) { return divided(start_at(i) * num, den) + i * extra; };
  int lo = 0, n = q.seqs;  // the last i in lo .. lo + n - 1 with task_at(i) <= t
  while (n > 1) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    const bool below = lane * step < n && task_at(i) <= t;
    const int k = max(__popcll(__ballot(below)) - 1, 0);
    n = min(step, n - k * step);
    lo += k * step;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  Span s;
  s.seq = lo;
  s.start = start_at(lo);
  s.rows = max(start_at(lo + 1) - s.start, 0);
  s.length = max(q.lengths[lo], 0);
  first = task_at(lo);
  return s;
}

inline BlockCache block_cache_of(const gptq_kv_blocks* c) {
  return BlockCache{c->codes,       c->scales,            c->page_stride,        c->slot_stride,
                    c->head_stride, c->param_page_stride, c->param_block_stride, c->param_head_stride};
}

inline Sequences sequences_of(const KvSequences& q, const gptq_kv_blocks* c, int32_t* info) {
  Sequences s;
  s.table = q.table; s.lengths = q.lengths; s.starts = q.starts;
  s.ldt = q.ldt; s.width = (int32_t)q.width; s.seqs = (int32_t)q.seqs; s.tokens = (int32_t)q.tokens;
  s.pages = (int32_t)c->pages; s.page_size = c->page_size; s.block = c->block;
  s.by_page = divisor_of(c->page_size);
  s.by_block = divisor_of(c->block);
  s.info = info;
  return s;
}

}  // namespace gptq
