// The pages of a cache: sequences that share them, grow, end, and are moved together.
//
// refs[page] counts the sequences that hold a page (0: free).  Everything is settled on the
// device in whole numbers, so a captured step may fork, grow and free; the result does not
// depend on the order of atomics, which only add, or take a maximum.
//
// Forking copies no page.  A page is copied when a sequence is about to write into it while
// others hold it: kv_pages_resize gives that sequence a page of its own and names the pair,
// which kv_pages_copy then copies in every layer's arrays.  Pages are taken lowest first.
#include "kernels.hpp"

namespace gptq {

namespace {

constexpr int kWide = 1024;   // threads of the kernels that settle pages
constexpr int kPer = 4;       // pages that a thread looks at in one step

// values that other waves of the workgroup have changed by atomics
__device__ __forceinline__ int32_t fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

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
  for (int j = tid; j < a.width; j += 256) to[j] = j < n ? from[j] : -1;
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
  for (int j = tid; j < n; j += 256) {
    const int page = a.table[row * a.ldt + j];
    if (page >= 0 && page < a.pages) atomicAdd(a.new_refs + page, c);
    else if (a.info) atomicOr(a.info, 1);
  }
}

struct ResizeArgs {
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  const int32_t* new_lengths;
  int32_t* src;
  int32_t* dst;
  int32_t* info;
  int32_t* writers;  // [pages]: rows that write into a page
  int32_t* top;      // [pages]: the last of them
  int32_t* taken;    // [pages]: the free pages in use from now on, in order
  int32_t* base;     // [rows]: where a row's fresh pages begin in `taken`
  int64_t ldt;
  int32_t rows, width, pages, page_size;
};

// the length that a row is to have, its own where it stays or where the table has no room
__device__ __forceinline__ int wanted(const ResizeArgs& a, int row, int len, bool& bad) {
  const int n = a.new_lengths[row];
  bad = n > 0 && pages_of(n, a.page_size) > a.width;
  return n < 0 || bad ? len : n;
}

// A wave per row: pages past a shorter end go back.
__global__ __launch_bounds__(256) void pages_drop_kernel(ResizeArgs a) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  const int len = a.lengths[row];
  bool bad;
  const int want = wanted(a, row, len, bad);
  if (bad && a.info && lane == 0) atomicOr(a.info, 1);
  if (lane == 0) {
    a.src[row] = -1;
    a.dst[row] = -1;
  }
  if (want >= len) return;
  const int o = min(pages_of(len, a.page_size), a.width), n = pages_of(want, a.page_size);
  for (int j = n + lane; j < o; j += 64) {
    int32_t* e = a.table + row * a.ldt + j;
    const int page = *e;
    *e = -1;
    if (page >= 0 && page < a.pages) atomicSub(a.refs + page, 1);
    else if (a.info) atomicOr(a.info, 1);
  }
  if (lane == 0) a.lengths[row] = want;
}

// One workgroup: who gets which free pages.
__global__ __launch_bounds__(kWide) void pages_grow_kernel(ResizeArgs a) {
  __shared__ int part[kWide / 64];
  __shared__ int short_of;
  const int tid = threadIdx.x;
  // the last page of a row that grows inside it, -1 for the others
  auto last_page = [&](int row, int& len, int& want) {
    bool bad;
    len = max(a.lengths[row], 0);
    want = wanted(a, row, len, bad);
    const int rest = len % a.page_size;
    if (want <= len || rest == 0) return -1;
    const int j = len / a.page_size;
    const int page = j < a.width ? a.table[row * a.ldt + j] : -1;
    if (page >= 0 && page < a.pages) return page;
    if (a.info) atomicOr(a.info, 1);
    return -1;
  };
  int len, want;
  for (int row = tid; row < a.rows; row += kWide) {
    const int p = last_page(row, len, want);
    if (p >= 0) {
      atomicExch(a.writers + p, 0);
      atomicExch(a.top + p, -1);
    }
  }
  __threadfence();
  __syncthreads();
  for (int row = tid; row < a.rows; row += kWide) {
    const int p = last_page(row, len, want);
    if (p >= 0) {
      atomicAdd(a.writers + p, 1);
      atomicMax(a.top + p, row);
    }
  }
  __threadfence();
  __syncthreads();
  // a shared page stays with the last of its holders if all of them write into it
  int total = 0;
  for (int r0 = 0; r0 < a.rows; r0 += kWide) {
    const int row = r0 + tid;
    int need = 0;
    bool copy = false;
    if (row < a.rows) {
      const int p = last_page(row, len, want);
      if (p >= 0) {
        const int held = fresh(a.refs + p);
        copy = held > 1 && !(fresh(a.writers + p) == held && fresh(a.top + p) == row);
      }
      need = max(pages_of(want, a.page_size) - pages_of(len, a.page_size), 0) + (copy ? 1 : 0);
    }
    int sum;
    const int before = scan_wide(need, part, sum);
    if (row < a.rows) a.base[row] = (total + before) << 1 | (copy ? 1 : 0);
    total += sum;
  }
  // the lowest free pages, as many as that
  int found = 0;
  for (int p0 = 0; p0 < a.pages && found < total; p0 += kWide * kPer) {
    int free[kPer], n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int p = p0 + tid * kPer + k;
      free[k] = p < a.pages && fresh(a.refs + p) == 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) n += free[k];
    int sum;
    int at = found + scan_wide(n, part, sum);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (free[k]) {
        if (at < total) a.taken[at] = p0 + tid * kPer + k;
        ++at;
      }
    found += sum;
  }
  if (tid == 0) short_of = found < total;
  __threadfence();
  __syncthreads();
  if (short_of) {  // nobody grows
    if (tid == 0 && a.info) atomicOr(a.info, 2);
    return;
  }
  // a wave per row hands them out
  for (int row = tid >> 6; row < a.rows; row += kWide / 64) {
    bool bad;
    const int lane = tid & 63, l0 = max(a.lengths[row], 0);
    const int w = wanted(a, row, l0, bad);
    if (w <= l0) continue;
    const int o = pages_of(l0, a.page_size), n = pages_of(w, a.page_size);
    const int b = fresh(a.base + row), copy = b & 1, at = b >> 1;
    int32_t* e = a.table + row * a.ldt;
    if (lane == 0) {
      a.lengths[row] = w;
      if (copy) {
        const int old = e[o - 1], page = fresh(a.taken + at);
        a.src[row] = old;
        a.dst[row] = page;
        e[o - 1] = page;
        atomicSub(a.refs + old, 1);
        atomicExch(a.refs + page, 1);
      }
    }
    for (int j = o + lane; j < n; j += 64) {
      const int page = fresh(a.taken + at + copy + j - o);
      e[j] = page;
      atomicExch(a.refs + page, 1);
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

// One workgroup: the k-th page in use behind their count goes into the k-th hole in front of it.
__global__ __launch_bounds__(kWide) void pages_place_kernel(CompactArgs a) {
  __shared__ int part[kWide / 64];
  const int tid = threadIdx.x;
  int live = 0;
  for (int p = tid; p < a.pages; p += kWide) live += a.refs[p] > 0;
  int total;
  scan_wide(live, part, total);
  for (int pass = 0; pass < 2; ++pass) {  // holes, then the pages that fill them
    int32_t* const list = pass == 0 ? a.dst : a.src;
    int found = 0;
    const int from = pass == 0 ? 0 : total, to = pass == 0 ? total : a.pages;
    for (int p0 = from; p0 < to; p0 += kWide) {
      const int p = p0 + tid;
      const bool hit = p < to && (a.refs[p] > 0) == (pass == 1);
      int sum;
      const int at = found + scan_wide(hit, part, sum);
      if (hit && at < a.capacity) list[at] = p;
      found += sum;
    }
    for (int64_t i = found + tid; i < a.capacity; i += kWide) list[i] = -1;
  }
  for (int p = tid; p < a.pages; p += kWide) {
    a.place[p] = p;
    const int n = a.refs[p];
    a.new_refs[p] = p < total ? n : 0;
  }
  __threadfence();
  __syncthreads();
  for (int64_t i = tid; i < a.capacity; i += kWide) {
    const int s = fresh(a.src + i), d = fresh(a.dst + i);
    if (s < 0 || d < 0) break;
    a.place[s] = d;
    a.new_refs[d] = a.refs[s];
  }
  if (tid == 0) *a.count = total;
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

// A workgroup copies pairs of one array in turn, V bytes a lane.
template <typename V>
__device__ __forceinline__ void copy_page(const gptq_page_array& v, int64_t s, int64_t d) {
  const char* from = static_cast<const char*>(v.data) + s * v.page_stride;
  char* to = static_cast<char*>(v.data) + d * v.page_stride;
  const int64_t n = v.row_bytes / (int)sizeof(V);
  for (int64_t o = 0; o < v.outer; ++o)
    for (int64_t i = 0; i < v.inner; ++i) {
      const V* f = reinterpret_cast<const V*>(from + o * v.outer_stride + i * v.inner_stride);
      V* t = reinterpret_cast<V*>(to + o * v.outer_stride + i * v.inner_stride);
      for (int64_t b = threadIdx.x; b < n; b += 256) t[b] = f[b];
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
    if (all % 16 == 0) copy_page<uint4>(v, s, d);
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
  hipLaunchKernelGGL(pages_rows_kernel, dim3((unsigned)(new_rows + ceil_div(pages, 256))), block, 0,
                     stream, a);
  if (rows > 0) hipLaunchKernelGGL(pages_refs_kernel, dim3((unsigned)rows), block, 0, stream, a);
  return hipGetLastError();
}

size_t kv_pages_resize_ws_bytes(int64_t rows, int64_t pages) { return (size_t)(3 * pages + rows) * 4; }

hipError_t launch_kv_pages_resize(int32_t* table, int64_t ldt, int64_t width, int32_t* lengths,
                                  int64_t rows, int32_t* refs, int64_t pages,
                                  const int32_t* new_lengths, int page_size, int32_t* src,
                                  int32_t* dst, int32_t* info, void* ws, hipStream_t stream) {
  int32_t* w = static_cast<int32_t*>(ws);
  ResizeArgs a{table, lengths, refs, new_lengths, src, dst, info, w, w + pages, w + 2 * pages,
               w + 3 * pages, ldt, (int32_t)rows, (int32_t)width, (int32_t)pages, page_size};
  hipLaunchKernelGGL(pages_drop_kernel, dim3((unsigned)ceil_div(rows, 4)), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(pages_grow_kernel, dim3(1), dim3(kWide), 0, stream, a);
  return hipGetLastError();
}

size_t kv_pages_compact_ws_bytes(int64_t pages) { return (size_t)pages * 4; }

hipError_t launch_kv_pages_compact(const int32_t* table, int64_t ldt, int64_t rows, int64_t width,
                                   const int32_t* refs, int64_t pages, int32_t* new_table,
                                   int64_t ldn, int32_t* new_refs, int32_t* src, int32_t* dst,
                                   int64_t capacity, int32_t* count, void* ws, hipStream_t stream) {
  CompactArgs a{table, refs, new_table, new_refs, src, dst, count, static_cast<int32_t*>(ws), ldt, ldn,
                capacity, (int32_t)rows, (int32_t)width, (int32_t)pages};
  hipLaunchKernelGGL(pages_place_kernel, dim3(1), dim3(kWide), 0, stream, a);
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
