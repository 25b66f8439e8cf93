// Pages of a paged cache: who owns them, and moving them.
//
// The bookkeeping is three integer arrays on the device: the page table
// [R, max_pages] (row r names the pages of sequence r, in order; -1 behind
// them), n_pages [R] and the reference counts ref [pages] (how many rows name
// a page; 0 = free).  Every operation hands out the lowest free pages first,
// in the order of its rows or pairs, and moves the lowest page first, so its
// result does not depend on timing.
//
// Planning (resize_kernel, fork_kernel, compact_kernel, check_kernel) is one
// CTA: it scans 4 counts a thread and step, 4096 pages at once, which for the
// pools that fit a GPU is a few microseconds, less than a second launch and a
// grid-wide prefix sum would cost (1800 pages: resize 5.6 us, compact 4.3; 48
// forks 10 us, the latency of its phases).  Moving (move_kernel) is a grid-wide
// copy bound by HBM: it reads the planned list of (source, destination) items on
// the device (481 pages of 64 entries, 126 MB, 19 us).
#pragma once

#include "hca_ptx.cuh"

namespace hca {
namespace pages {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

struct Table {
  int* table;          // row r at table + r * ld
  long long ld;
  int rows, max_pages;
  int* n_pages;        // [rows]
  int* ref;            // [num_pages]
  int num_pages;
  int page_shift;
};

__device__ __forceinline__ int pages_of(const Table& t, int entries) {
  return static_cast<int>((static_cast<long long>(entries) + (1 << t.page_shift) - 1) >>
                          t.page_shift);
}

// Exclusive prefix of `x` over the CTA, and the sum (all threads call).
__device__ __forceinline__ int block_scan(int x, int* red, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();   // `red` of an earlier scan has been read
  if (lane == 31) red[w] = y;
  __syncthreads();
  if (w == 0) {
    int z = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += v;
    }
    red[lane] = z;
  }
  __syncthreads();
  *total = red[kPlanWarps - 1];
  return y - x + (w > 0 ? red[w - 1] : 0);
}

// Calls found(k, page) for the k-th page (k < want) in [lo, hi) whose count
// satisfies pred, in ascending order; returns how many there are, up to want.
template <typename Pred, typename Found>
__device__ __forceinline__ int scan_pages(const int* ref, int lo, int hi, int want, int* red,
                                          Pred&& pred, Found&& found) {
  int seen = 0;
  for (int base = lo; base < hi && seen < want; base += 4 * kPlanThreads) {
    const int p0 = base + 4 * threadIdx.x;
    int m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      // counts may just have been changed by this CTA's atomics: read past L1
      if (p0 + q < hi && pred(__ldcg(ref + p0 + q))) m |= 1 << q;
    int total;
    int k = seen + block_scan(__popc(m), red, &total);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if ((m >> q) & 1) {
        if (k < want) found(k, p0 + q);
        ++k;
      }
    seen += total;
  }
  return min(seen, want);
}

// Drops one reference of `page`; a page that has none, or lies outside of the
// pool, is reported.
__device__ __forceinline__ void drop_ref(const Table& t, int page) {
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(t.num_pages)) {
    record_error(DEVERR_BAD_INPUT, 220);
  } else if (atomicSub(t.ref + page, 1) <= 0) {
    atomicAdd(t.ref + page, 1);
    record_error(DEVERR_BAD_INPUT, 221);
  }
}

// ---------------------------------------------------------------------------
// resize: row r is to hold ceil(entries[r] / P) pages (entries[r] < 0: as
// many as it has).  First every row that shrinks gives its last pages back,
// then rows that grow take the lowest free pages, row by row, while there are
// any; n_pages tells what each row got.
// With `src` (lists of pages to copy, for move_kernel) a row whose last page is
// now partly used, and named by other rows too, gets a fresh page in its place
// before any row grows, so that what is appended to it stays its own; of rows
// that share that page with nobody else the last one keeps it.  Without a free
// page it keeps the shared one, which is reported.
// Workspace: free list [num_pages], growth prefix [rows + 1]; then src, dst
// [rows] and their length.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int clamped_pages(const Table& t, int r) {
  const int n = t.n_pages[r];
  if (n < 0 || n > t.max_pages) record_error(DEVERR_BAD_INPUT, 222);
  return min(max(n, 0), t.max_pages);
}

__global__ void __launch_bounds__(kPlanThreads)
    resize_kernel(const Table t, const int* __restrict__ entries, int* __restrict__ free_list,
                  int* __restrict__ prefix, int* __restrict__ src, int* __restrict__ dst,
                  int* __restrict__ count) {
  __shared__ int red[kPlanWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  // growth of every row, and its prefix
  int grown = 0;
  for (int base = 0; base < t.rows; base += kPlanThreads) {
    const int r = base + threadIdx.x;
    int grow = 0;
    if (r < t.rows) {
      const int have = clamped_pages(t, r), e = entries[r];
      int want = e < 0 ? have : pages_of(t, e);
      if (want > t.max_pages) {
        record_error(DEVERR_BAD_INPUT, 223);
        want = t.max_pages;
      }
      grow = want - have;   // negative: shrinks by that many
    }
    int total;
    const int before = block_scan(max(grow, 0), red, &total);
    if (r < t.rows) prefix[r] = grow >= 0 ? grown + before : grow;
    grown += total;
  }
  if (threadIdx.x == 0) prefix[t.rows] = grown;
  __syncthreads();
  // shrink: a warp a row
  for (int r = w; r < t.rows; r += kPlanWarps) {
    const int d = prefix[r];
    if (d >= 0) continue;
    const int have = min(max(t.n_pages[r], 0), t.max_pages);
    int* row = t.table + r * t.ld;
    for (int c = have + d + lane; c < have; c += 32) {
      drop_ref(t, row[c]);
      row[c] = -1;
    }
    __syncwarp();
    if (lane == 0) t.n_pages[r] = have + d;
  }
  __syncthreads();
  // rows that need their partly used page for themselves
  int own = 0;
  auto partial = [&](int r) -> int {   // that page, or -1
    const int e = entries[r], c = e >> t.page_shift;
    if (e <= 0 || (e & ((1 << t.page_shift) - 1)) == 0 || c >= min(t.n_pages[r], t.max_pages))
      return -1;
    const int page = t.table[r * t.ld + c];
    return static_cast<unsigned>(page) < static_cast<unsigned>(t.num_pages) &&
                   __ldcg(t.ref + page) > 1
               ? page
               : -1;
  };
  if (src != nullptr) {
    for (int r = threadIdx.x; r < t.rows; r += kPlanThreads) dst[r] = partial(r);
    __syncthreads();
    for (int base = 0; base < t.rows; base += kPlanThreads) {
      const int r = base + threadIdx.x;
      const int page = r < t.rows ? dst[r] : -1;
      int left = 0;                    // references of it when it is this row's turn
      if (page >= 0) {
        left = __ldcg(t.ref + page);
        for (int q = 0; q < r; ++q) left -= dst[q] == page ? 1 : 0;
      }
      int total;
      const int k = own + block_scan(left > 1 ? 1 : 0, red, &total);
      if (left > 1) src[k] = r;        // the row, for now
      own += total;
    }
  }
  if (grown + own == 0) {
    if (src != nullptr && threadIdx.x == 0) *count = 0;
    return;
  }
  const int found = scan_pages(
      t.ref, 0, t.num_pages, grown + own, red, [](int c) { return c <= 0; },
      [&](int k, int page) { free_list[k] = page; });
  __syncthreads();
  if (src != nullptr) {
    for (int k = threadIdx.x; k < own; k += kPlanThreads) {
      const int r = src[k];
      int* at = t.table + r * t.ld + (entries[r] >> t.page_shift);
      if (k < found) {
        src[k] = *at;
        dst[k] = free_list[k];
        drop_ref(t, *at);
        t.ref[free_list[k]] = 1;
        *at = free_list[k];
      } else {
        src[k] = dst[k] = -1;
        record_error(DEVERR_BAD_INPUT, 228);
      }
    }
    if (threadIdx.x == 0) *count = own;
  }
  const int got = max(found - own, 0);
  free_list += own;
  for (int r = w; r < t.rows; r += kPlanWarps) {
    const int first = prefix[r];
    if (first < 0) continue;
    int next = t.rows;      // the next row's first page: of the next row that does not shrink
    for (int q = r + 1; q <= t.rows; ++q)
      if (prefix[q] >= 0) {
        next = prefix[q];
        break;
      }
    const int take = min(next, got) - first;
    if (take <= 0) continue;
    const int have = min(max(t.n_pages[r], 0), t.max_pages);
    int* row = t.table + r * t.ld;
    for (int c = lane; c < take; c += 32) {
      const int page = free_list[first + c];
      row[have + c] = page;
      t.ref[page] = 1;
    }
    __syncwarp();
    if (lane == 0) t.n_pages[r] = have + take;
  }
}

// ---------------------------------------------------------------------------
// fork: pair i makes the empty row child[i] a branch of parent[i] at
// entries[i] entries: the full pages are shared (ref + 1), the partly filled
// one is given a fresh page, whose copy is left to move_kernel.  A pair is
// refused (ok = 0, reported) when a row number is out of range, the child has
// pages, is a parent in this call or appeared before, or the parent has fewer
// pages than the entries need; ok = 0 without a report when no page is free.
// Lists: item i copies page src[i] to dst[i] (-1: nothing) and ring row
// rsrc[i] to rdst[i].
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads)
    fork_kernel(const Table t, const int* __restrict__ parent, const int* __restrict__ child,
                const int* __restrict__ entries, int n, int* __restrict__ ok,
                int* __restrict__ src, int* __restrict__ dst, int* __restrict__ rsrc,
                int* __restrict__ rdst) {
  __shared__ int red[kPlanWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  // validity; dst[i] = rank of the pair's fresh page, or -1
  int fresh = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    bool good = false, part = false;
    if (i < n) {
      const int a = parent[i], b = child[i], e = entries[i];
      good = static_cast<unsigned>(a) < static_cast<unsigned>(t.rows) &&
             static_cast<unsigned>(b) < static_cast<unsigned>(t.rows) && e >= 0;
      if (good) {
        const int have = t.n_pages[a];
        good = t.n_pages[b] == 0 && have <= t.max_pages && pages_of(t, e) <= have;
        part = (e & ((1 << t.page_shift) - 1)) != 0;
      }
      for (int q = 0; q < n && good; ++q)
        if (parent[q] == b || (q < i && child[q] == b)) good = false;
      if (!good) record_error(DEVERR_BAD_INPUT, 224);
    }
    int total;
    const int rank = block_scan(good && part ? 1 : 0, red, &total);
    if (i < n) {
      ok[i] = good ? 1 : 0;
      dst[i] = good && part ? fresh + rank : -1;
      src[i] = -1;
    }
    fresh += total;
  }
  __syncthreads();
  // the fresh pages: rsrc serves as their list first
  const int got = fresh == 0 ? 0
                             : scan_pages(
                                   t.ref, 0, t.num_pages, fresh, red, [](int c) { return c <= 0; },
                                   [&](int k, int page) { rsrc[k] = page; });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int k = dst[i];
    if (k >= got) ok[i] = 0;
    rdst[i] = k >= 0 && k < got ? rsrc[k] : -1;
  }
  __syncthreads();
  // a warp a pair: the child's row
  for (int i = w; i < n; i += kPlanWarps) {
    if (!ok[i]) {
      if (lane == 0) dst[i] = -1;
      continue;
    }
    const int a = parent[i], b = child[i], e = entries[i];
    const int full = e >> t.page_shift;
    const int page = rdst[i];
    const int* from = t.table + a * t.ld;
    int* row = t.table + b * t.ld;
    for (int c = lane; c < t.max_pages; c += 32) {
      int v = -1;
      if (c < full) {
        v = from[c];
        if (static_cast<unsigned>(v) < static_cast<unsigned>(t.num_pages)) {
          atomicAdd(t.ref + v, 1);
        } else {
          record_error(DEVERR_BAD_INPUT, 225);
          v = -1;
        }
      } else if (c == full && page >= 0) {
        v = page;
        t.ref[page] = 1;
      }
      row[c] = v;
    }
    if (lane == 0) {
      t.n_pages[b] = full + (page >= 0 ? 1 : 0);
      dst[i] = page;
      if (page >= 0) {
        const int old = from[full];
        src[i] = static_cast<unsigned>(old) < static_cast<unsigned>(t.num_pages) ? old : -1;
        if (src[i] < 0) record_error(DEVERR_BAD_INPUT, 225);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    rsrc[i] = ok[i] ? parent[i] : -1;
    rdst[i] = ok[i] ? child[i] : -1;
  }
}

// ---------------------------------------------------------------------------
// compact: with `live` pages in use, those numbered live and above move, in
// order, into the free ones below.  Lists (src, dst), their length, and the
// new number of every page that moves; the table is rewritten and the pages
// are copied by move_kernel.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads)
    compact_kernel(int* __restrict__ ref, int num_pages, int* __restrict__ src,
                   int* __restrict__ dst, int* __restrict__ count, int* __restrict__ remap,
                   int* __restrict__ live_out) {
  __shared__ int red[kPlanWarps];
  __shared__ int live_s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();
  int m = 0;
  for (int p = threadIdx.x; p < num_pages; p += kPlanThreads) m += ref[p] > 0 ? 1 : 0;
  atomicAdd(&live_s, m);
  __syncthreads();
  const int live = live_s;
  scan_pages(
      ref, 0, live, num_pages, red, [](int c) { return c <= 0; },
      [&](int k, int page) { dst[k] = page; });
  const int moves = scan_pages(
      ref, live, num_pages, num_pages, red, [](int c) { return c > 0; },
      [&](int k, int page) { src[k] = page; });
  for (int p = live + threadIdx.x; p < num_pages; p += kPlanThreads) remap[p] = p;
  __syncthreads();
  for (int k = threadIdx.x; k < moves; k += kPlanThreads) {
    const int a = src[k], b = dst[k];
    remap[a] = b;
    ref[b] = ref[a];
    ref[a] = 0;
  }
  if (threadIdx.x == 0) {
    *count = moves;
    *live_out = live;
  }
}

// ---------------------------------------------------------------------------
// copy: a list from the caller.  Items out of range are refused, and so are
// all pairs of a destination that is named twice or is also a source (what
// they would leave there depends on timing); an item onto itself is nothing.
// mark [items], zero-filled: times an item is a destination, bit 30 = source.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads)
    check_kernel(const int* __restrict__ from, const int* __restrict__ to, int n, int items,
                 int* __restrict__ mark, int* __restrict__ src, int* __restrict__ dst) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto in = [&](int x) { return static_cast<unsigned>(x) < static_cast<unsigned>(items); };
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int a = from[i], b = to[i];
    if (!in(a) || !in(b)) {
      record_error(DEVERR_BAD_INPUT, 226);
    } else if (a != b) {
      atomicAdd(mark + b, 1);
      atomicOr(mark + a, 1 << 30);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int a = from[i], b = to[i];
    bool good = in(a) && in(b) && a != b;
    if (good && __ldcg(mark + b) != 1) {
      record_error(DEVERR_BAD_INPUT, 227);
      good = false;
    }
    src[i] = good ? a : -1;
    dst[i] = good ? b : -1;
  }
}

// ---------------------------------------------------------------------------
// move: items (pages, or ring rows) of several arrays, by the lists above.
// Units of up to 16 KB, one CTA step each: 256 threads x 4 x 16 bytes in
// flight.
// ---------------------------------------------------------------------------
constexpr int kMaxArrays = 8;
constexpr int kMoveThreads = 256;
constexpr int kUnit = 16384;

struct MoveArray {
  uint8_t* base;
  long long bytes;     // of an item, a multiple of 16
  unsigned per;        // units of an item; all units of a call are fewer than 2^31
  const int* src;      // list
  const int* dst;
};

struct Move {
  MoveArray a[kMaxArrays];
  int arrays;
  int n;               // list length, or its upper bound
  long long units;     // of all arrays (host)
  const int* count;    // list length on the device, or null
  // compact: table entries to renumber (null: none)
  int* table;
  long long table_ld;
  int rows, max_pages;
  const int* remap;
  const int* live;
  int num_pages;
};

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Move m) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan's lists
  const int n = m.count != nullptr ? min(*m.count, m.n) : m.n;
  if (m.table != nullptr) {
    const int live = *m.live;
    const long long total = static_cast<long long>(m.rows) * m.max_pages;
    for (long long x = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x; x < total;
         x += static_cast<long long>(gridDim.x) * kMoveThreads) {
      const long long r = x / m.max_pages;
      int* e = m.table + r * m.table_ld + (x - r * m.max_pages);
      const int page = *e;
      if (page >= live && page < m.num_pages) *e = m.remap[page];
    }
  }
  // 32-bit unit numbers: with 64-bit divisions the kernel was bound by them (48 forks: 59 % of
  // the issue slots)
  unsigned skip = 0;     // units of the arrays before this one, modulo the grid
  for (int q = 0; q < m.arrays; ++q) {
    const MoveArray& a = m.a[q];
    const unsigned units = a.per * static_cast<unsigned>(n);
    // this CTA's units of the array: u = blockIdx.x (mod gridDim.x), counted over all arrays
    const unsigned first = blockIdx.x >= skip ? blockIdx.x - skip : blockIdx.x + gridDim.x - skip;
    for (unsigned u = first; u < units; u += gridDim.x) {
      const unsigned item = u / a.per;
      const int s = a.src[item], d = a.dst[item];
      if (s < 0 || d < 0) continue;
      const long long off = static_cast<long long>(u - item * a.per) * kUnit;
      const int len = static_cast<int>(min(static_cast<long long>(kUnit), a.bytes - off));
      const uint4* from = reinterpret_cast<const uint4*>(a.base + s * a.bytes + off);
      uint4* to = reinterpret_cast<uint4*>(a.base + d * a.bytes + off);
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int o = threadIdx.x + k * kMoveThreads;
        if (16 * o < len) x[k] = __ldcs(from + o);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int o = threadIdx.x + k * kMoveThreads;
        if (16 * o < len) __stcs(to + o, x[k]);
      }
    }
    skip = (skip + units % gridDim.x) % gridDim.x;
  }
}

}  // namespace pages
}  // namespace hca
