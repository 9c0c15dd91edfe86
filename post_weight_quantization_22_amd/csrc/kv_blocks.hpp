// Shared pieces of the operators on a paged cache with a scale per block of tokens
// and head: where a sequence's rows and keys lie.
#pragma once

#include "fp8.hpp"

namespace gptq {

// n / d for 0 <= n < 2^31 as n * mul >> shift: with 2^k >= d, mul = ceil(2^(31 + k) / d) is off by
// less than d <= 2^k of 2^(31 + k), and n times that is less than 2^(31 + k), too little to reach
// the next quotient.
struct Divisor {
  uint32_t mul;
  int32_t shift;
};

inline Divisor divisor_of(int64_t d) {
  int k = 0;
  while ((int64_t(1) << k) < d) ++k;
  return Divisor{(uint32_t)(((uint64_t(1) << (31 + k)) + (uint64_t)d - 1) / (uint64_t)d), 31 + k};
}

__device__ __forceinline__ int divided(int n, const Divisor& d) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
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
  int32_t room;  // positions that the table has entries for
  Divisor by_page, by_block;
  int32_t* info;
};

struct Span {  // a sequence's new rows (none where the starts do not ascend)
  int seq, start, rows, length;
};

// The sequence that task t belongs to, and its first task: sequence i has the tasks from
// starts[i] * num / den + i * extra on (each wave finds it by itself, 64 sequences a step;
// starts that do not ascend lead to some sequence of the call all the same).  Tasks of rows in front of
// starts[0] have a first task behind them: nothing is to be done for those.
// tokens * num < 2^31.
__device__ __forceinline__ Span span_of(const Sequences& q, int t, int num, const Divisor& den,
                                        int extra, int& first) {
  const int lane = threadIdx.x & 63;
  auto start_at = [&](int i) { return min(max(q.starts[i], 0), q.tokens); };
  auto task_at = [&](int start, int i) { return divided(start * num, den) + i * extra; };
  int lo = 0, n = q.seqs;  // the last i in lo .. lo + n - 1 with task_at(i) <= t
  while (n > 64) {
    const int step = (n + 63) / 64, i = lo + min(lane * step, n - 1);
    const bool below = (lane * step < n) & (task_at(start_at(i), i) <= t);
    const int k = max((int)__popcll(__ballot(below)) - 1, 0);
    n = min(step, n - k * step);
    lo += k * step;
  }
  // the last step reads all that the answer may need: one round trip for up to 64 sequences
  const int i = lo + min(lane, n - 1);
  const int s0 = start_at(i), s1 = start_at(i + 1), len = q.lengths[i];
  // (& and no branch: what is computed on both sides of one counts as different in every lane)
  const int k = max((int)__popcll(__ballot((lane < n) & (task_at(s0, i) <= t))) - 1, 0);  // (it counts without a sign)
  Span s;
  s.seq = __builtin_amdgcn_readfirstlane(lo + k);
  s.start = __builtin_amdgcn_readlane(s0, k);
  s.rows = max(__builtin_amdgcn_readlane(s1, k) - s.start, 0);
  s.length = max(__builtin_amdgcn_readlane(len, k), 0);
  first = task_at(s.start, s.seq);
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
  s.room = (int32_t)hmin(q.width * c->page_size, INT32_MAX - 65536);  // (tiles are counted past the end)
  s.by_page = divisor_of(c->page_size);
  s.by_block = divisor_of(c->block);
  s.info = info;
  return s;
}

}  // namespace gptq
