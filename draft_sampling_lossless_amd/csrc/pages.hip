// The cache's rows and pages: accepted paths moved together, pages copied, and the pages'
// bookkeeping.  Tables, lengths and counts live on the device, so that rounds in a captured
// graph take and give back pages without the host.
//
// A page's count is the number of table entries that name it; a page of count 0 is free.
// Nothing else is kept: the lowest free pages are found by reading the counts.
#include "attention.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

// a store of what this launch does not read again
typedef uint32_t uint32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_streaming(uint4* p, const uint4& v) {
  __builtin_nontemporal_store(uint32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<uint32x4*>(p));
}

// ------------------------------------------------------------------ rows and pages
// Bytes copied, nothing else: memory's rate is the bound, 4.9 TB/s for a copy of 2 GiB.  A thread
// has kFlight pieces of 16 bytes on their way, and stores them past the caches' order of
// replacement: 192 pages of 32 KB in five layers, keys and values, 29 us so (4.3 TB/s) and 33 with plain
// stores; 19 and 28 for the same pages again and again, which the last-level cache holds in part.
constexpr int kCopyThreads = 256, kFlight = 4;

// Path entry i of request b moves from place ctx + path[i] to ctx + i, for one layer of keys or
// values a workgroup.  Paths ascend, so path[i] >= i and no row is written that a later one
// still reads: batches of rows in their order, each read whole before it is written.  256 trees of
// 64 nodes with paths of up to 17, five layers of 8 x 128, 90 MB: 27 us, 3.3 TB/s, and 35 with plain
// stores; in the same caches again and again, of which the last-level cache holds a part, 17 and 28
// (there a thread for every piece of a row and no barriers, which leaves short rows to few threads,
// gained nothing).  3 us without a row to move.
__global__ __launch_bounds__(kCopyThreads) void kv_compact_rows(CompactArgs a) {
  __shared__ int from[kMaxPath], to[kMaxPath], valid, lead;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int node = tid < a.max_path ? a.path[(size_t)b * a.max_path + tid] : -1;
  const int n = max(a.cu_q[b + 1] - a.cu_q[b], 0), kv = clampi(a.kv_len[b], 0, a.width << a.page_shift), ctx = kv - n;
  const int len = clampi(a.accepted[b], 0, a.max_path);
  if (tid < kMaxPath) to[tid] = node;
  if (tid == 0) valid = lead = len;
  __syncthreads();
  const int before = tid > 0 && tid < len ? to[tid - 1] : -1;
  __syncthreads();
  if (tid < len) {
    auto slot_of = [&](int key) {
      if (key < 0 || key >= kv) return -1;
      const int page = a.page_table[(size_t)b * a.width + (key >> a.page_shift)];
      return page >= 0 && page < a.num_pages ? (page << a.page_shift) + (key & ((1 << a.page_shift) - 1)) : -1;
    };
    if (node <= before || node >= n) atomicMin(&valid, tid);    // the path ends before it
    else if (node != tid) atomicMin(&lead, tid);                // what stands in its place already
    from[tid] = node >= 0 && node < n ? slot_of(ctx + node) : -1;
    to[tid] = slot_of(ctx + tid);
  }
  __syncthreads();
  const int rows = valid;
  if (a.new_len && blockIdx.y == 0 && tid == 0) a.new_len[b] = max(ctx + rows, 0);
  const int first = min(lead, rows);
  uint4* cache = reinterpret_cast<uint4*>(blockIdx.y & 1 ? a.v_cache : a.k_cache) + (size_t)(blockIdx.y >> 1) * a.layer_pieces;
  const uint32_t pieces = a.row_pieces, total = (uint32_t)(rows - first) * pieces;
  for (uint32_t base = 0; base < total; base += kCopyThreads * kFlight) {
    uint4 v[kFlight];
    int64_t dst[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const uint32_t x = base + u * kCopyThreads + tid, r = x / pieces, p = x - r * pieces;
      dst[u] = -1;
      if (x < total && from[first + r] >= 0 && to[first + r] >= 0) {
        v[u] = cache[(int64_t)from[first + r] * pieces + p];
        dst[u] = (int64_t)to[first + r] * pieces + p;
      }
    }
    // every load of the batch has returned, everyone's: its rows may be written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (dst[u] >= 0) store_streaming(cache + dst[u], v[u]);
  }
}

__global__ __launch_bounds__(kCopyThreads) void kv_copy_page(CopyArgs a) {
  const int2 c = reinterpret_cast<const int2*>(a.copies)[blockIdx.x];
  if (c.x < 0 || c.x >= a.num_pages || c.y < 0 || c.y >= a.num_pages || c.x == c.y) return;
  uint4* cache = reinterpret_cast<uint4*>(blockIdx.y & 1 ? a.v_cache : a.k_cache) + (size_t)(blockIdx.y >> 1) * a.layer_pieces;
  const uint4* src = cache + (int64_t)c.x * a.page_pieces;
  uint4* dst = cache + (int64_t)c.y * a.page_pieces;
  for (int64_t base = (int64_t)blockIdx.z * kCopyThreads * kFlight; base < a.page_pieces; base += (int64_t)gridDim.z * kCopyThreads * kFlight) {
    uint4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t x = base + u * kCopyThreads + threadIdx.x;
      if (x < a.page_pieces) v[u] = src[x];
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t x = base + u * kCopyThreads + threadIdx.x;
      if (x < a.page_pieces) store_streaming(dst + x, v[u]);
    }
  }
}

// ------------------------------------------------------------------ rows of the table
// One workgroup a row: the new ones copied and counted, the old ones counted off.  The counts
// are added by atomics, whose order does not matter to a sum.
__global__ __launch_bounds__(256) void pages_select_rows(SelectArgs a) {
  const bool fresh = (int)blockIdx.x < a.rows;
  const int row = fresh ? blockIdx.x : blockIdx.x - a.rows;
  const int s = fresh ? a.src[row] : row;
  const bool there = s >= 0 && s < a.B;
  const int len = there ? clampi(a.kv_len[s], 0, a.width << a.page_shift) : 0;
  const int hold = (len + (1 << a.page_shift) - 1) >> a.page_shift;
  const int32_t* from = a.page_table + (size_t)(there ? s : 0) * a.width;
  if (fresh && threadIdx.x == 0) a.new_len[row] = len;
  for (int c = threadIdx.x; c < (fresh ? a.width : hold); c += 256) {
    const int page = c < hold ? from[c] : -1;
    if (fresh) a.new_table[(size_t)row * a.width + c] = page;
    if (page >= 0 && page < a.num_pages) atomicAdd(a.refs + page, fresh ? 1 : -1);
  }
}

// ------------------------------------------------------------------ lengths
// One workgroup for the whole call, its four steps told apart by barriers: pages given back,
// needs counted, free pages found and dealt, lengths set.  A thread has up to kEach requests in
// a row; the r-th need of all requests gets the r-th free page.  A call is a chain of dependent
// loads and barriers: 64 requests that grow by two pages 7 us, that shrink 7; 256 in groups of four
// on a page 12, 4096 of them 32, and 144 where all share one page, whose count is one after the
// other's.
constexpr int kThreads = 1024, kEach = 4;
constexpr int kSpan = 4, kPass = kSpan * 4 * kThreads;   // counts looked through at once
static_assert(kThreads * kEach >= 4096, "DSPARK_MAX_SEQS requests");

// exclusive sum over the workgroup; `part` is LDS of its waves
__device__ __forceinline__ int block_sum_before(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  const int of_wave = lane < kThreads / 64 ? part[lane] : 0;
  int run = of_wave;
#pragma unroll
  for (int o = 1; o < kThreads / 64; o <<= 1) {
    const int x = __shfl_up(run, o);
    if (lane >= o) run += x;
  }
  total = __shfl(run, kThreads / 64 - 1);
  return inc - v + __shfl(run - of_wave, wave);
}

__global__ __launch_bounds__(kThreads) void pages_resize_all(ResizeArgs a) {
  // offs: first item of each request; col0: the column of a request's first item; list: free
  // pages in their order
  __shared__ int offs[kThreads * kEach + 1], col0[kThreads * kEach];
  __shared__ int list[4 * kThreads];
  __shared__ int part[kThreads / 64], torn;
  const int tid = threadIdx.x, each = (a.B + kThreads - 1) / kThreads, b0 = tid * each;
  const int size = 1 << a.page_shift, most = a.width << a.page_shift;
  int was[kEach], now[kEach], hold[kEach], want[kEach], before, total;
  // the request that item x belongs to
  auto owner = [&](int x) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offs[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  auto publish = [&](const int (&items)[kEach]) {  // fills offs and total
    int sum = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum += items[e];
    before = block_sum_before(sum, part, total);
    int at = before;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (e < each && b0 + e < a.B) {
        offs[b0 + e] = at;
        at += items[e];
      }
    __syncthreads();
  };

  auto counts_at = [&](int first) {
    int4 v = make_int4(1, 1, 1, 1);
    if (first + 4 <= a.num_pages) {
      v = *reinterpret_cast<const int4*>(a.refs + first);
    } else {
      if (first < a.num_pages) v.x = a.refs[first];
      if (first + 1 < a.num_pages) v.y = a.refs[first + 1];
      if (first + 2 < a.num_pages) v.z = a.refs[first + 2];
    }
    return v;
  };

  // The counts to look through first are asked for at once, and hold if no page is given back.
  int4 next[kSpan];
  auto first_counts = [&]() {
#pragma unroll
    for (int k = 0; k < kSpan; ++k) next[k] = counts_at(k * 4 * kThreads + 4 * tid);
  };
  first_counts();

  // Everyone's atomics, and loads of what they change, are done.  (They are carried out by the
  // second-level cache, which this workgroup alone writes to: a fence for the whole device, some
  // 3 us, is more than is needed.)
  auto everyone = [&]() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };

  // pages given back
  int items[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = b0 + e;
    was[e] = now[e] = 0;
    if (e < each && b < a.B) {
      was[e] = clampi(a.kv_len[b], 0, most);
      now[e] = clampi(a.new_len[b], 0, most);
    }
    hold[e] = (was[e] + size - 1) >> a.page_shift;
    want[e] = (now[e] + size - 1) >> a.page_shift;
    items[e] = max(hold[e] - want[e], 0);
    if (e < each && b < a.B) col0[b] = want[e];
  }
  // (the last page of a request that grows: not one that is given back)
  int end[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    end[e] = now[e] > was[e] && (was[e] & (size - 1)) ? a.page_table[(size_t)(b0 + e) * a.width + hold[e] - 1] : -1;
  publish(items);
  if (total > 0) {
    for (int x = tid; x < total; x += kThreads) {
      const int b = owner(x);
      int32_t* entry = a.page_table + (size_t)b * a.width + col0[b] + x - offs[b];
      const int page = *entry;
      *entry = -1;
      if (page >= 0 && page < a.num_pages) atomicSub(a.refs + page, 1);
    }
    everyone();
    // (the atomics went to the second-level cache, and the first may hold what was asked for before)
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    first_counts();
  }

  // A growing request whose last page is not full writes into it.  If others share the page the
  // request takes a copy; if all who share it do, the last of them keeps it.  All are counted off
  // at once: where none is left, the count serves to find the last, which counts itself again.
  int shared[kEach];
  bool copied[kEach] = {};
  bool any = false;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    shared[e] = end[e] >= 0 && end[e] < a.num_pages && a.refs[end[e]] > 1 ? end[e] : -1;
    copied[e] = shared[e] >= 0;
    any |= copied[e];
  }
  if (__syncthreads_or(any)) {
    everyone();                                   // (the first counts too: some of them pass through 0 here)
    auto count_of = [&](int page) { return __hip_atomic_load(a.refs + page, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (copied[e]) atomicSub(a.refs + shared[e], 1);
    everyone();
    bool left[kEach];                             // nobody has it any more
#pragma unroll
    for (int e = 0; e < kEach; ++e) left[e] = copied[e] && count_of(shared[e]) == 0;
    everyone();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (left[e]) atomicMax(a.refs + shared[e], b0 + e + 1);
    everyone();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (left[e] && count_of(shared[e]) == b0 + e + 1) copied[e] = false;
    everyone();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (left[e] && !copied[e]) __hip_atomic_store(a.refs + shared[e], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    everyone();
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    items[e] = now[e] > was[e] ? want[e] - hold[e] + copied[e] : 0;
    if (e < each && b0 + e < a.B) col0[b0 + e] = hold[e] - copied[e];
  }
  if (tid == 0) torn = -1;
  publish(items);

  // The lowest free pages, dealt in order: kSpan times 4 kThreads counts a pass, the next pass's on
  // their way.  Spans without a free page, which most are where a pool is nearly full, take no more
  // than the pass's barrier: with the free pages at the end of 131072 a call takes 16 us, 35 with a pass
  // for every 4096.
  int found = 0;
  const int needed = total;
  for (int base = 0; base < a.num_pages && found < needed; base += kPass) {
    int4 v[kSpan];
    bool some = false;
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      v[k] = next[k];
      some |= v[k].x == 0 || v[k].y == 0 || v[k].z == 0 || v[k].w == 0;
      next[k] = counts_at(base + kPass + k * 4 * kThreads + 4 * tid);
    }
    if (!__syncthreads_or(some)) continue;
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      if (found >= needed) break;
      const int first = base + k * 4 * kThreads + 4 * tid;
      int here;
      const int mine = (v[k].x == 0) + (v[k].y == 0) + (v[k].z == 0) + (v[k].w == 0);
      int at = block_sum_before(mine, part, here);
      if (v[k].x == 0) list[at++] = first;
      if (v[k].y == 0) list[at++] = first + 1;
      if (v[k].z == 0) list[at++] = first + 2;
      if (v[k].w == 0) list[at++] = first + 3;
      __syncthreads();
      const int use = min(here, needed - found);
      for (int x = tid; x < use; x += kThreads) {
        const int b = owner(found + x);
        a.page_table[(size_t)b * a.width + col0[b] + found + x - offs[b]] = list[x];
        a.refs[list[x]] = 1;
      }
      found += use;
      __syncthreads();
    }
  }

  // A request is served if its pages were found; one that got some of them gives them back.
  int at = before;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = b0 + e;
    if (e < each && b < a.B) {
      const bool waits = now[e] > was[e] && (items[e] > 0 || shared[e] >= 0);
      const bool ok = !waits || at + items[e] <= found;
      int32_t* last = a.page_table + (size_t)b * a.width + hold[e] - 1;
      int2 copy = make_int2(-1, -1);
      if (copied[e] && ok) copy = make_int2(shared[e], *last);
      if (copied[e] && !ok) atomicAdd(a.refs + shared[e], 1);   // (it still has the page)
      if (!ok && at < found) torn = b;            // (one at most: the needs lie in a row)
      a.kv_len[b] = ok ? now[e] : was[e];
      if (a.copies) reinterpret_cast<int2*>(a.copies)[b] = copy;
      if (a.served) a.served[b] = ok;
    }
    at += items[e];
  }
  __syncthreads();
  if (torn >= 0) {
    const int b = torn, got = found - offs[b];
    for (int x = tid; x < got; x += kThreads) {
      int32_t* entry = a.page_table + (size_t)b * a.width + col0[b] + x;
      a.refs[*entry] = 0;
      *entry = -1;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (b0 + e == b && e < each && copied[e]) a.page_table[(size_t)b * a.width + hold[e] - 1] = shared[e];
  }
}

}  // namespace

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(kv_compact_rows, dim3(a.B, 2 * a.layers), dim3(kCopyThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const CopyArgs& a, hipStream_t stream) {
  const int64_t parts = (a.page_pieces + kCopyThreads * kFlight - 1) / (kCopyThreads * kFlight);
  hipLaunchKernelGGL(kv_copy_page, dim3(a.n, 2 * a.layers, parts < 64 ? (int)parts : 64), dim3(kCopyThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_select(const SelectArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(pages_select_rows, dim3(a.rows + a.B), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_resize(const ResizeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(pages_resize_all, dim3(1), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dspark
