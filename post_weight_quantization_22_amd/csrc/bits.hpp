// Integer helpers of the host side (no HIP in here).
#pragma once

#include <stdint.h>

namespace gptq {

// the smallest p with 2^p >= v
constexpr int log2_at_least(int64_t v) {
  int p = 0;
  while ((int64_t(1) << p) < v) ++p;
  return p;
}

// log2 of v > 0, -1 where v is no power of two
constexpr int log2_exact(int64_t v) { return (v & (v - 1)) == 0 ? log2_at_least(v) : -1; }

}  // namespace gptq
