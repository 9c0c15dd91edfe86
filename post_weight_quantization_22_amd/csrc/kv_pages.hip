// The pages of a cache: sequences that share them, grow, end, and are moved together.
//
// refs[page] counts the sequences that hold a page (0: free).  Everything is settled on the
// device in whole numbers, so a captured step may fork, grow and free; the result does not
// depend on the order of atomics, which only add, or take a maximum.
//
// Forking copies no page.  A page is copied when a sequence is about to write into it while
// others hold it: kv_pages_resize gives that sequence a page of its own and names the pair,
// which kv_pages_copy then copies in every layer's arrays.  Pages are taken lowest first.
//
// Launches bound all of this but the copies (a call's host time, some 2 us between kernels, a few round
// trips in each): a table of some thousand entries is settled by one workgroup in one launch (fork 3.5
// us, growth with what it takes back 7, compaction 4 to 6), which a larger one would keep waiting for
// one workgroup's loads (6 rows forked, grown and copied: two launches for a fork and for a resize 26 us,
// one 22; 250 pages compacted and copied 17.5 and 15.8).  Copies go at the memory's rate (2000 pages' halves of
// 64 KB in 8 arrays: 4.8 TB/s).
#include "kernels.hpp"

namespace gptq {

namespace {

constexpr int kWide = 1024;   // threads of the kernels that settle pages
constexpr int kPer = 4;       // pages that a thread looks at in one step
constexpr int kStep = kWide * kPer;
constexpr int kRows = 4096;   // rows whose last pages are compared at a time
constexpr int kHeld = 8192;   // fresh pages that LDS holds
constexpr int kSmall = 8192;  // pages and table entries that one workgroup settles by itself

__device__ __forceinline__ int pages_of(int len, int page_size) {
  return (int)(((int64_t)max(len, 0) + page_size - 1) / page_size);
}

// The sum of v over the threads in front of this one; total: over all of them.
__device__ __forceinline__ int scan_wide(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWide / 64; ++w) {
    const int s = part[w];
    before += w < wave ? s : 0;
    total += s;
  }
  return before + x - v;
}

struct ForkArgs {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* refs;
  const int32_t* parents;
  int32_t* new_table;
  int32_t* new_lengths;
  int32_t* new_refs;
  int32_t* info;
  int64_t ldt, ldn;
  int32_t rows, new_rows, width, pages, page_size;
};

// A workgroup per new row; those behind them copy refs.
__global__ __launch_bounds__(256) void pages_rows_kernel(ForkArgs a) {
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= a.new_rows) {
    const int i = ((int)blockIdx.x - a.new_rows) * 256 + tid;
    if (i < a.pages) a.new_refs[i] = a.refs[i];
    return;
  }
  const int row = blockIdx.x;
  int p = a.parents[row];
  if (p >= a.rows) {
    if (a.info && tid == 0) atomicOr(a.info, 1);
    p = -1;
  }
  const int len = p < 0 ? 0 : max(a.lengths[p], 0);
  const int n = pages_of(len, a.page_size);
  if (n > a.width && a.info && tid == 0) atomicOr(a.info, 1);
  if (tid == 0) a.new_lengths[row] = len;
  const int32_t* from = a.table + max(p, 0) * a.ldt;
  int32_t* to = a.new_table + row * a.ldn;
  for (int j0 = tid; j0 < a.width; j0 += 4 * 256) {
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = j0 + k * 256 < min(n, a.width) ? from[j0 + k * 256] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j0 + k * 256 < a.width) to[j0 + k * 256] = page[k];
  }
}

// A workgroup per old row: its pages have as many more holders as it has children, less itself.
__global__ __launch_bounds__(256) void pages_refs_kernel(ForkArgs a) {
  __shared__ int part[4];
  const int tid = threadIdx.x, row = blockIdx.x;
  int c = 0;
  for (int i = tid; i < a.new_rows; i += 256) c += a.parents[i] == row;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) c += __shfl_xor(c, d);
  if ((tid & 63) == 0) part[tid >> 6] = c;
  __syncthreads();
  c = part[0] + part[1] + part[2] + part[3] - 1;
  if (c == 0) return;
  const int n = min(pages_of(a.lengths[row], a.page_size), a.width);
  const int32_t* const entries = a.table + row * a.ldt;
  for (int j0 = tid; j0 < n; j0 += 4 * 256) {
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = entries[min(j0 + k * 256, n - 1)];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j0 + k * 256 >= n) break;
      if (page[k] >= 0 && page[k] < a.pages) atomicAdd(a.new_refs + page[k], c);
      else if (a.info) atomicOr(a.info, 1);
    }
  }
}

// Both for few rows and pages, in one workgroup: a launch less, and what pages gain is added up in LDS.
__global__ __launch_bounds__(kWide) void pages_fork_kernel(ForkArgs a) {
  __shared__ int children[kWide];
  __shared__ int gain[kSmall];
  const int tid = threadIdx.x;
  children[tid] = -1;  // (less the row itself)
  for (int i = tid; i < a.pages; i += kWide) gain[i] = 0;
  __syncthreads();
  auto parent = [&](int row) {
    const int p = a.parents[row];
    return p < a.rows ? p : -1;
  };
  auto outside = [&] {
    if (a.info) atomicOr(a.info, 1);
  };
  for (int i = tid; i < a.new_rows; i += kWide) {
    const int p = parent(i);
    if (p >= 0) atomicAdd(children + p, 1);
    const int len = p < 0 ? 0 : max(a.lengths[p], 0);
    a.new_lengths[i] = len;
    if (a.parents[i] >= a.rows || pages_of(len, a.page_size) > a.width) outside();
  }
  // four entries of a thread under way
  for (int u0 = tid; u0 < a.new_rows * a.width; u0 += 4 * kWide) {
    int p[4], len[4], page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = min(u0 + k * kWide, a.new_rows * a.width - 1);
      p[k] = parent(u / a.width);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = min(u0 + k * kWide, a.new_rows * a.width - 1);
      len[k] = p[k] < 0 ? 0 : a.lengths[p[k]];
      page[k] = p[k] < 0 ? -1 : a.table[p[k] * a.ldt + u % a.width];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k * kWide;
      if (u >= a.new_rows * a.width) break;
      const int row = u / a.width, j = u - row * a.width;
      a.new_table[row * a.ldn + j] = j < pages_of(len[k], a.page_size) ? page[k] : -1;
    }
  }
  __syncthreads();
  for (int u = tid; u < a.rows * a.width; u += kWide) {
    const int row = u / a.width, j = u - row * a.width, c = children[row];
    const int n = pages_of(a.lengths[row], a.page_size), page = a.table[row * a.ldt + j];
    if (c == 0 || j >= n) continue;
    if (page >= 0 && page < a.pages) atomicAdd(gain + page, c);
    else outside();
  }
  __syncthreads();
  for (int i = tid; i < a.pages; i += kWide) a.new_refs[i] = a.refs[i] + gain[i];
}

struct ResizeArgs {
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  const int32_t* new_lengths;
  int32_t* src;
  int32_t* dst;
  int32_t* info;
  int32_t* taken;    // [pages]: the free pages in use from now on, in order (kHeld of them at most: in LDS)
  int32_t* base;     // [rows]: where a row's fresh pages begin among those (more than kWide rows)
  int64_t ldt;
  int32_t rows, width, pages, page_size;
};

// the length that a row is to have, its own where it stays or where the table has no room
__device__ __forceinline__ int wanted(const ResizeArgs& a, int row, int len, bool& bad) {
  const int n = a.new_lengths[row];
  bad = n > 0 && pages_of(n, a.page_size) > a.width;
  return n < 0 || bad ? len : n;
}

// A workgroup per row: pages past a shorter end go back, four entries of a thread under way.
__global__ __launch_bounds__(256) void pages_drop_kernel(ResizeArgs a) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const int len = a.lengths[row];
  bool bad;
  const int want = wanted(a, row, len, bad);
  if (bad && a.info && tid == 0) atomicOr(a.info, 1);
  if (tid == 0) {
    a.src[row] = -1;
    a.dst[row] = -1;
  }
  if (want >= len) return;
  const int o = min(pages_of(len, a.page_size), a.width), n = pages_of(want, a.page_size);
  int32_t* const entries = a.table + row * a.ldt;
  for (int j0 = n + tid; j0 < o; j0 += 4 * 256) {
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = entries[min(j0 + k * 256, o - 1)];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j0 + k * 256 >= o) break;
      entries[j0 + k * 256] = -1;
      if (page[k] >= 0 && page[k] < a.pages) atomicSub(a.refs + page[k], 1);
      else if (a.info) atomicOr(a.info, 1);
    }
  }
  __syncthreads();  // (everyone has read the length)
  if (tid == 0) a.lengths[row] = want;
}

// A load that sees what the same kernel's atomics have done (past the first-level cache).
__device__ __forceinline__ int settled(const int* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One workgroup: who gets which free pages.  A step of a batch waits for it, so it is one chain of few
// round trips: rows and the first free pages are read at once, shared pages are found among the rows'
// last ones in LDS, nothing is fenced (what waves exchange in memory goes through one first-level cache).
// DROP: few rows and entries, whose shorter ends it takes back first, a launch less.
template <bool DROP>
__global__ __launch_bounds__(kWide) void pages_grow_kernel(ResizeArgs a) {
  __shared__ int part[kWide / 64];
  __shared__ __align__(16) int lasts[kRows];  // (DROP: where the rows' entries to take back begin and end first)
  __shared__ int held_taken[kHeld];
  const int tid = threadIdx.x, lane = tid & 63;
  struct Row {
    int len, want, last, held;  // last: the page that it grows inside of, -1: none
  };
  auto row_at = [&](int row) {
    Row r{0, 0, -1, 0};
    if (row >= a.rows) return r;
    r.len = max(a.lengths[row], 0);
    bool bad;
    r.want = wanted(a, row, r.len, bad);
    const int j = r.len / a.page_size;
    if (r.want > r.len && j * (int64_t)a.page_size < r.len) {
      const int page = j < a.width ? a.table[row * a.ldt + j] : -1;
      if (page >= 0 && page < a.pages) r.last = page;
      else if (a.info) atomicOr(a.info, 1);
    }
    return r;
  };
  bool dropped = false;
  auto refs_at = [&](int p) { return DROP && dropped ? settled(a.refs + p) : a.refs[p]; };
  auto free_at = [&](int p0, int (&free)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int p = p0 + tid * kPer + k;
      free[k] = p < a.pages && refs_at(p) == 0;
    }
  };
  int free[kPer];
  free_at(0, free);
  if constexpr (DROP) {  // (a thread's row: kWide of them at most)
    const int len = tid < a.rows ? a.lengths[tid] : 0;
    bool bad = false;
    const int want = tid < a.rows ? wanted(a, tid, len, bad) : 0;
    if (tid < a.rows) a.src[tid] = a.dst[tid] = -1;
    if (bad && a.info) atomicOr(a.info, 1);
    if (want < len) a.lengths[tid] = want;
    const int from = pages_of(want, a.page_size), to = want < len ? min(pages_of(len, a.page_size), a.width) : 0;
    lasts[tid] = from;
    lasts[kWide + tid] = to;
    dropped = __syncthreads_or(from < to);
    if (dropped) {
      for (int u0 = tid; u0 < a.rows * a.width; u0 += 4 * kWide) {  // entries, four of a thread under way
        int32_t* e[4];
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = u0 + k * kWide, row = u / a.width, j = u - row * a.width;
          e[k] = u < a.rows * a.width && j >= lasts[row] && j < lasts[kWide + row] ? a.table + row * a.ldt + j : nullptr;
          if (e[k]) page[k] = *e[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!e[k]) continue;
          *e[k] = -1;
          if (page[k] >= 0 && page[k] < a.pages) atomicSub(a.refs + page[k], 1);
          else if (a.info) atomicOr(a.info, 1);
        }
      }
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (they have arrived in front of the barrier)
      __syncthreads();
      free_at(0, free);
    }
  }
  // A shared page stays with the last of its holders if all of them write into it.
  Row r;
  bool copy = false;
  int total = 0, base = 0;
  for (int r0 = 0; r0 < a.rows; r0 += kWide) {
    r = row_at(r0 + tid);
    r.held = r.last < 0 ? 0 : refs_at(r.last);
    const bool shared = r.held > 1;
    int writers = 0, top = -1;
    if (__syncthreads_or(shared)) {
      for (int t0 = 0; t0 < a.rows; t0 += kRows) {
        const int n = min(kRows, a.rows - t0);
        __syncthreads();
        for (int i = tid; i < (n + 3) / 4 * 4; i += kWide)
          lasts[i] = i >= n ? -1 : t0 + i == r0 + tid ? r.last : row_at(t0 + i).last;
        __syncthreads();
        if (shared)
          for (int i = 0; i < n; i += 4) {
            const int4 x = *reinterpret_cast<const int4*>(lasts + i);
            writers += (x.x == r.last) + (x.y == r.last) + (x.z == r.last) + (x.w == r.last);
            if (x.x == r.last) top = t0 + i;
            if (x.y == r.last) top = t0 + i + 1;
            if (x.z == r.last) top = t0 + i + 2;
            if (x.w == r.last) top = t0 + i + 3;
          }
      }
    }
    copy = shared && !(writers == r.held && top == r0 + tid);
    const int need = max(pages_of(r.want, a.page_size) - pages_of(r.len, a.page_size), 0) + (copy ? 1 : 0);
    int sum;
    base = total + scan_wide(need, part, sum);
    if (a.rows > kWide && r0 + tid < a.rows) a.base[r0 + tid] = base << 1 | (copy ? 1 : 0);
    total += sum;
  }
  // the lowest free pages, as many as that
  int* const taken = total <= kHeld || a.pages <= kHeld ? held_taken : a.taken;
  int found = 0;
  for (int p0 = 0; p0 < a.pages && found < total; p0 += kStep) {
    if (p0 > 0) free_at(p0, free);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) n += free[k];
    int sum;
    int at = found + scan_wide(n, part, sum);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (free[k]) {
        if (at < total) taken[at] = p0 + tid * kPer + k;
        ++at;
      }
    found += sum;
  }
  __syncthreads();
  if (found < total) {  // nobody grows
    if (tid == 0 && a.info) atomicOr(a.info, 2);
    return;
  }
  for (int r0 = 0; r0 < a.rows; r0 += kWide) {
    const int row = r0 + tid;
    if (a.rows > kWide) {
      r = row_at(row);
      const int b = row < a.rows ? a.base[row] : 0;
      base = b >> 1;
      copy = b & 1;
    }
    const bool grows = row < a.rows && r.want > r.len;
    const int o = pages_of(r.len, a.page_size), n = grows ? pages_of(r.want, a.page_size) : o;
    int32_t* const e = a.table + (int64_t)row * a.ldt;
    if (grows) {
      a.lengths[row] = r.want;
      if (copy) {
        const int page = taken[base];
        a.src[row] = r.last;
        a.dst[row] = page;
        e[o - 1] = page;
        atomicSub(a.refs + r.last, 1);
        a.refs[page] = 1;
      }
    }
    // a few pages a row by its thread, many by its wave
    constexpr int kFew = 4;
    const int first = base + (copy ? 1 : 0), more = n - o;
    if (more > 0 && more <= kFew)
      for (int k = 0; k < more; ++k) {
        const int page = taken[first + k];
        e[o + k] = page;
        a.refs[page] = 1;
      }
    for (uint64_t many = __ballot(more > kFew); many; many &= many - 1) {
      const int of = __ffsll((unsigned long long)many) - 1;
      const int f = __shfl(first, of), m = __shfl(more, of), at = __shfl(o, of);
      int32_t* const w = a.table + (int64_t)(r0 + (tid & ~63) + of) * a.ldt + at;
      for (int k = lane; k < m; k += 64) {
        const int page = taken[f + k];
        w[k] = page;
        a.refs[page] = 1;
      }
    }
  }
}

struct CompactArgs {
  const int32_t* table;
  const int32_t* refs;
  int32_t* new_table;
  int32_t* new_refs;
  int32_t* src;
  int32_t* dst;
  int32_t* count;
  int32_t* place;  // [pages]: where a page goes
  int64_t ldt, ldn, capacity;
  int32_t rows, width, pages;
};

// One workgroup: the k-th page in use behind their count goes into the k-th hole in front of it.  With r the
// pages in use in front of page p, a hole is the (p - r)-th, a page behind the count the (r - r0)-th one to
// move, r0 the pages in use in front of the count: one running sum gives both lists.
// SMALL: few pages and entries, whose new names it writes too, from the places that it keeps in LDS.
template <bool SMALL>
__global__ __launch_bounds__(kWide) void pages_place_kernel(CompactArgs a) {
  __shared__ int part[kWide / 64];
  __shared__ int in_front;
  __shared__ int places[SMALL ? kSmall : 1];
  int* const place = SMALL ? places : a.place;
  const int tid = threadIdx.x;
  auto refs_at = [&](int p0, int (&refs)[kPer]) {
    int live = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int p = p0 + tid * kPer + k;
      refs[k] = p < a.pages ? a.refs[p] : 0;
      live += refs[k] > 0;
    }
    return live;
  };
  int refs[kPer], live = 0, total;
  for (int p0 = 0; p0 < a.pages; p0 += kStep) live += refs_at(p0, refs);
  scan_wide(live, part, total);
  if (tid == 0) in_front = 0;
  int found = 0;
  for (int p0 = 0; p0 < a.pages; p0 += kStep) {
    live = a.pages > kStep ? refs_at(p0, refs) : live;
    int sum;
    const int before = found + scan_wide(live, part, sum);
    int r = before;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (p0 + tid * kPer + k == total) in_front = r;
      r += refs[k] > 0;
    }
    __syncthreads();
    const int r0 = in_front;
    r = before;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int p = p0 + tid * kPer + k;
      if (p >= a.pages) break;
      const bool used = refs[k] > 0;
      if (p < total && used) a.new_refs[p] = refs[k];
      if (p >= total) a.new_refs[p] = 0;
      if (!(p >= total && used)) place[p] = p;
      if (p < total && !used) a.dst[p - r] = p;
      if (p >= total && used) a.src[r - r0] = p;
      r += used;
    }
    found += sum;
  }
  __syncthreads();
  // (as many holes in front as pages behind: the count less those in use in front)
  const int moves = total < a.pages ? total - in_front : 0;
  for (int64_t i = tid; i < a.capacity; i += kWide) {
    if (i >= moves) {
      a.src[i] = a.dst[i] = -1;
      continue;
    }
    const int s = a.src[i], d = a.dst[i];
    place[s] = d;
    a.new_refs[d] = a.refs[s];
  }
  if (tid == 0) *a.count = total;
  if constexpr (SMALL) {
    __syncthreads();
    for (int u = tid; u < a.rows * a.width; u += kWide) {
      const int row = u / a.width, j = u - row * a.width, p = a.table[row * a.ldt + j];
      a.new_table[row * a.ldn + j] = p >= 0 && p < a.pages ? places[p] : p;
    }
  }
}

__global__ __launch_bounds__(256) void pages_rename_kernel(CompactArgs a) {
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x)
    for (int j = threadIdx.x; j < a.width; j += 256) {
      const int p = a.table[row * a.ldt + j];
      a.new_table[row * a.ldn + j] = p >= 0 && p < a.pages ? a.place[p] : p;
    }
}

constexpr int kArrays = 32;  // arrays of one launch (its arguments stay below 4 KB)

struct CopyArgs {
  gptq_page_array v[kArrays];
  const int32_t* src;
  const int32_t* dst;
  int32_t* info;
  int64_t pairs;
};

// A workgroup copies pairs of one array in turn, V bytes a lane; rows of several runs of strides
// are counted through.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename V>
__device__ __forceinline__ void copy_page(const gptq_page_array& v, int64_t s, int64_t d) {
  const char* from = static_cast<const char*>(v.data) + s * v.page_stride;
  char* to = static_cast<char*>(v.data) + d * v.page_stride;
  const int64_t n = v.row_bytes / (int)sizeof(V);
  constexpr int AHEAD = 4;
  if (v.outer * v.inner == 1) {
    const V* f = reinterpret_cast<const V*>(from);
    V* t = reinterpret_cast<V*>(to);
    int64_t b = threadIdx.x;
    for (; b + (AHEAD - 1) * 256 < n; b += AHEAD * 256) {
      const V x0 = f[b], x1 = f[b + 256], x2 = f[b + 512], x3 = f[b + 768];
      t[b] = x0; t[b + 256] = x1; t[b + 512] = x2; t[b + 768] = x3;
    }
    for (; b < n; b += 256) t[b] = f[b];
    return;
  }
  for (int64_t u = threadIdx.x; u < v.outer * v.inner * n; u += 256) {
    const int64_t row = u / n, o = row / v.inner, i = row - o * v.inner;
    const int64_t at = o * v.outer_stride + i * v.inner_stride + (u - row * n) * (int)sizeof(V);
    *reinterpret_cast<V*>(to + at) = *reinterpret_cast<const V*>(from + at);
  }
}

__global__ __launch_bounds__(256) void pages_copy_kernel(CopyArgs a) {
  const gptq_page_array& v = a.v[blockIdx.y];
  const int64_t all = reinterpret_cast<uintptr_t>(v.data) | v.page_stride | v.outer_stride |
                      v.inner_stride | v.row_bytes;
  for (int64_t k = blockIdx.x; k < a.pairs; k += gridDim.x) {
    const int s = a.src[k], d = a.dst[k];
    if (s < 0 || d < 0 || s == d) continue;
    if (s >= v.pages || d >= v.pages) {
      if (a.info && threadIdx.x == 0) *a.info = 1;
      continue;
    }
    if (all % 16 == 0) copy_page<u32x4>(v, s, d);
    else if (all % 4 == 0) copy_page<uint32_t>(v, s, d);
    else copy_page<uint8_t>(v, s, d);
  }
}

}  // namespace

hipError_t launch_kv_pages_fork(const int32_t* table, int64_t ldt, const int32_t* lengths,
                                int64_t rows, const int32_t* refs, int64_t pages,
                                const int32_t* parents, int64_t new_rows, int page_size,
                                int32_t* new_table, int64_t ldn, int64_t width,
                                int32_t* new_lengths, int32_t* new_refs, int32_t* info,
                                hipStream_t stream) {
  ForkArgs a{table,     lengths,   refs, parents,       new_table,         new_lengths,
             new_refs,  info,      ldt,  ldn,           (int32_t)rows,     (int32_t)new_rows,
             (int32_t)width, (int32_t)pages, page_size};
  const dim3 block(256);
  if (rows <= kWide && pages <= kSmall && hmax(rows, new_rows) * width <= kSmall) {
    hipLaunchKernelGGL(pages_fork_kernel, dim3(1), dim3(kWide), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t groups = new_rows + ceil_div(pages, 256);
  if (!grid_fits(hmax(groups, rows), 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(pages_rows_kernel, dim3((unsigned)groups), block, 0, stream, a);
  if (rows > 0) hipLaunchKernelGGL(pages_refs_kernel, dim3((unsigned)rows), block, 0, stream, a);
  return hipGetLastError();
}

size_t kv_pages_resize_ws_bytes(int64_t rows, int64_t pages) {
  return (size_t)((pages > kHeld ? pages : 0) + (rows > kWide ? rows : 0)) * 4;
}

hipError_t launch_kv_pages_resize(int32_t* table, int64_t ldt, int64_t width, int32_t* lengths,
                                  int64_t rows, int32_t* refs, int64_t pages,
                                  const int32_t* new_lengths, int page_size, int32_t* src,
                                  int32_t* dst, int32_t* info, void* ws, hipStream_t stream) {
  int32_t* w = static_cast<int32_t*>(ws);
  ResizeArgs a{table, lengths, refs, new_lengths, src, dst, info, w, w + (pages > kHeld ? pages : 0),
               ldt, (int32_t)rows, (int32_t)width, (int32_t)pages, page_size};
  if (!grid_fits(rows, 256)) return hipErrorInvalidConfiguration;
  if (rows <= kWide && rows * width <= kSmall) {
    hipLaunchKernelGGL(pages_grow_kernel<true>, dim3(1), dim3(kWide), 0, stream, a);
  } else {
    hipLaunchKernelGGL(pages_drop_kernel, dim3((unsigned)rows), dim3(256), 0, stream, a);
    hipLaunchKernelGGL(pages_grow_kernel<false>, dim3(1), dim3(kWide), 0, stream, a);
  }
  return hipGetLastError();
}

size_t kv_pages_compact_ws_bytes(int64_t pages) { return (size_t)pages * 4; }

hipError_t launch_kv_pages_compact(const int32_t* table, int64_t ldt, int64_t rows, int64_t width,
                                   const int32_t* refs, int64_t pages, int32_t* new_table,
                                   int64_t ldn, int32_t* new_refs, int32_t* src, int32_t* dst,
                                   int64_t capacity, int32_t* count, void* ws, hipStream_t stream) {
  CompactArgs a{table, refs, new_table, new_refs, src, dst, count, static_cast<int32_t*>(ws), ldt, ldn,
                capacity, (int32_t)rows, (int32_t)width, (int32_t)pages};
  if (pages <= kSmall && rows * width <= kSmall) {
    hipLaunchKernelGGL(pages_place_kernel<true>, dim3(1), dim3(kWide), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(pages_place_kernel<false>, dim3(1), dim3(kWide), 0, stream, a);
  if (rows > 0)
    hipLaunchKernelGGL(pages_rename_kernel, dim3((unsigned)hmin(rows, 4096)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_pages_copy(const gptq_page_array* arrays, int64_t n, const int32_t* src,
                                const int32_t* dst, int64_t pairs, int32_t* info,
                                hipStream_t stream) {
  for (int64_t i = 0; i < n; i += kArrays) {
    CopyArgs a = {};
    const int64_t m = hmin(n - i, kArrays);
    for (int64_t k = 0; k < m; ++k) a.v[k] = arrays[i + k];
    a.src = src;
    a.dst = dst;
    a.info = info;
    a.pairs = pairs;
    const dim3 grid((unsigned)hmin(pairs, 1024), (unsigned)m);
    hipLaunchKernelGGL(pages_copy_kernel, grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace gptq
