// Appending ragged chunks of new tokens to a paged cache.
//
// The cache of sequence i is its ring (the newest 128 raw tokens, slot =
// position mod 128) and the pages that its page table row names: entry j lies
// in page table[i][j / P], slot j mod P.  A chunk brings the tokens
// [q_start[i], q_start[i + 1]) of the packed inputs as the newest ones of
// sequence i, at positions L0 .. L1 - 1 with L1 = ctx_len[i].
//
// entries_kernel: every block of 128 positions that the chunk completes,
//   w = softmax(s), ck = sum w k, cv = sum w v ('BaiduがERNIE 5.5 Flash Baseを
//   公開' §2.1), its tokens taken from the ring (positions before L0) and from
//   the chunk.  Same thread layout and order of sums as the whole-sequence
//   compressor, so the entries are bit-identical to it.  Without kRaw it is the
//   whole append: the ring takes the newest tokens as well.  With kRaw it lays
//   the 127 tokens before the chunk, the chunk and 17 zero rows one after
//   another in the workspace, where the attention of the chunk reads the raw
//   windows of all its tokens as contiguous rows;
// finish_kernel, launched behind that, updates the ring (which may only change
//   once the rows before the chunk have been read) and writes the item list and
//   the copies of last pages for the attention.
//
// Both move bytes only: 2 KB a token in (and out again with kRaw).  Measured: 32768
// tokens of one sequence 13.8 us (4.9 TB/s), 32 pieces of up to 256 tokens 7.9 us, 2000
// sequences of a token or two 73 us, of which latency is all but the first.
#pragma once

#include "compress.cuh"
#include "hca_ptx.cuh"

namespace hca {
namespace paged {

constexpr int kD = 512;
constexpr int kBlk = 128;
constexpr int kBack = 127;      // tokens before the chunk that its first window needs
constexpr int kPad = 144;       // workspace rows of a sequence beyond its n tokens
constexpr int kThreads = 128;
// blocks that n + kPad rows (kRaw), or n, can touch beyond n / 128
template <bool kRaw>
constexpr int kUnitsExtra = kRaw ? 4 : 2;

struct Cache {
  uint16_t* wk;        // [S, 128, 512]
  uint16_t* wv;
  uint16_t* ws;        // [S, 128]
  uint16_t* ck;        // [pages, P, 512]
  uint16_t* cv;
  const int* table;    // row i at table + i * table_ld
  long long table_ld;
  int max_pages;       // columns of the table
  int num_pages;
  int page_shift;
};

struct Chunk {
  const uint16_t* k;   // [N, 512]
  const uint16_t* v;
  const uint16_t* s;   // [N]
  const int* q_start;  // [S + 1], null: one token a sequence
  const int* ctx_len;  // [S]
  int S, N;
};

struct Span {
  int qs, n, L0, L1;   // first packed token, tokens, positions [L0, L1)
};

// Bounds of sequence i.  Offsets outside of 0 .. N, or falling, and lengths
// below the number of tokens or above 2^30 are clamped and (by the one caller
// that asks) reported.
__device__ __forceinline__ Span span_of(const Chunk& c, int i, bool report) {
  Span r;
  const int a = c.q_start != nullptr ? c.q_start[i] : i;
  const int b = c.q_start != nullptr ? c.q_start[i + 1] : i + 1;
  const int L = c.ctx_len[i];
  r.qs = min(max(a, 0), c.N);
  r.n = max(min(max(b, 0), c.N) - r.qs, 0);
  r.L1 = min(max(L, r.n), 1 << 30);
  r.L0 = r.L1 - r.n;
  if (report && (r.qs != a || r.qs + r.n != b || (r.L1 != L && r.n > 0)))
    record_error(DEVERR_BAD_INPUT, 210);
  return r;
}

// first workspace row of sequence i: position L0 - 127
__device__ __forceinline__ int raw_base(const Span& sp, int i) { return sp.qs + kPad * i; }

// Row of entry j of sequence i in the page pools, or -1 (reported) where the
// table has no page for it.
__device__ __forceinline__ long long entry_row(const Cache& c, int i, int j, unsigned where) {
  const int col = j >> c.page_shift;
  int pg = -1;
  if (col < c.max_pages) pg = c.table[i * c.table_ld + col];
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(c.num_pages)) {
    if (threadIdx.x == 0) record_error(DEVERR_BAD_INPUT, where);
    return -1;
  }
  return (static_cast<long long>(pg) << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

// Sequence of work unit u when sequence i owns the units from
// floor(q_start[i] / 128) + extra i on (at least as many as it can need): the last that
// does not start behind u, found by counting in two rounds, every 1/128th of the offsets
// and then the 1/128th that it names (one round up to 128 sequences), without a prefix
// sum.  Counting all offsets took 90 us for 2000 sequences of a token or two.
__device__ __forceinline__ int unit_seq(const Chunk& c, int u, int extra, int* red) {
  auto count = [&](bool in) -> int {
    const unsigned some = __ballot_sync(0xffffffffu, in);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = __popc(some);
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
  };
  auto starts = [&](int i) -> bool {   // at or before u
    const int qs = c.q_start != nullptr ? min(max(c.q_start[i], 0), c.N) : i;
    return qs / kBlk + extra * i <= u;
  };
  const int step = (c.S + kThreads - 1) / kThreads, tid = threadIdx.x;
  int at = max(count(tid * step < c.S && starts(tid * step)) - 1, 0) * step;
  const int end = min(at + step, c.S);
  for (int base = at + 1; base < end; base += kThreads)
    at += count(base + tid < end && starts(base + tid));
  return at;
}

// Newest position of ring slot `slot` with L1 tokens.
__device__ __forceinline__ int newest(int L1, int slot) {
  return L1 - 1 - ((L1 - 1 - slot) & (kBlk - 1));
}

// grid.x = floor(N / 128) + kUnitsExtra S units, grid.y = 8 (K/V x 4 channel quarters);
// without kRaw the 8 CTAs of a unit are a cluster
template <bool kRaw>
__global__ void __launch_bounds__(kThreads)
    entries_kernel(const Chunk c, const Cache cache, uint16_t* __restrict__ raw_k,
                   uint16_t* __restrict__ raw_v) {
  __shared__ float w[kBlk];
  __shared__ float red[2][4];
  __shared__ int cnt[4];
  __shared__ float part[8][kBlk + 4];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5;
  const int u = blockIdx.x;
  const int which = blockIdx.y >> 2, quarter = blockIdx.y & 3;
  const int i = unit_seq(c, u, kUnitsExtra<kRaw>, cnt);
  const Span sp = span_of(c, i, false);
  if (!kRaw && u == 0 && blockIdx.y == 0)
    for (int j = tid; j < c.S; j += kThreads) span_of(c, j, true);
  const int ubase = sp.qs / kBlk + kUnitsExtra<kRaw> * i;
  if (u < ubase || sp.n == 0) return;
  // block b, positions p0 .. p0 + 127; the first block is that of position L0 - 127 (kRaw) or L0
  const int b = (kRaw ? ((sp.L0 - kBack + kBlk) >> 7) - 1 : sp.L0 >> 7) + (u - ubase);
  const int p0 = b * kBlk;
  if (p0 > sp.L1 + 16) return;
  const bool completes = b >= 0 && p0 + kBlk <= sp.L1 && p0 + kBlk > sp.L0;
  // Only the block of the first new token takes tokens from the ring: its CTAs bring the
  // ring up to date, each the channels that it reads itself, so that only the scores, which
  // all of them read and one writes, make them wait for one another.
  const bool renews = !kRaw && u == ubase;
  if (!kRaw && !completes && !renews) return;

  if (completes) {   // within-block softmax of the scores (fp32)
    const int p = p0 + tid;
    const uint16_t sb = p < sp.L0 ? cache.ws[static_cast<size_t>(i) * kBlk + tid]
                                  : c.s[static_cast<size_t>(sp.qs) + (p - sp.L0)];
    const float sv = __uint_as_float(static_cast<uint32_t>(sb) << 16);
    float m = warp_max(sv);
    if ((tid & 31) == 0) red[0][warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float e = expf(sv - m);
    float z = warp_sum(e);
    if ((tid & 31) == 0) red[1][warp] = z;
    __syncthreads();
    z = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    w[tid] = e / z;
    __syncthreads();
    if (renews) cluster_arrive();   // the scores have been read
  }

  // thread (r, c): tokens r, r + 8, .. and channels 8 c .. 8 c + 7 of the quarter
  uint16_t* ring = (which ? cache.wv : cache.wk) + static_cast<size_t>(i) * kBlk * kD;
  const uint16_t* fresh = (which ? c.v : c.k) + static_cast<size_t>(sp.qs) * kD;
  uint16_t* raw = which ? raw_v : raw_k;
  const int col = quarter * 128 + (tid & 15) * 8;
  const int r = tid >> 4;
  uint4 x[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int p = p0 + q * 8 + r;
    x[q] = make_uint4(0u, 0u, 0u, 0u);
    if (!kRaw && !completes) continue;
    if (p >= sp.L0) {
      if (p < sp.L1)
        x[q] = __ldg(reinterpret_cast<const uint4*>(fresh + static_cast<size_t>(p - sp.L0) * kD + col));
    } else if (p >= max(0, sp.L0 - kBack)) {
      x[q] = *reinterpret_cast<const uint4*>(ring + static_cast<size_t>(p & (kBlk - 1)) * kD + col);
    }
  }
  if constexpr (kRaw) {
    const long long row0 = static_cast<long long>(raw_base(sp, i)) + kBack - sp.L0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int p = p0 + q * 8 + r;
      if (p >= sp.L0 - kBack && p <= sp.L1 + 16)
        *reinterpret_cast<uint4*>(raw + (row0 + p) * kD + col) = x[q];
    }
  }
  if (renews) {   // a thread writes the ring where it read it
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int p = newest(sp.L1, q * 8 + r);
      if (p >= sp.L0)
        *reinterpret_cast<uint4*>(ring + static_cast<size_t>(q * 8 + r) * kD + col) =
            __ldg(reinterpret_cast<const uint4*>(fresh + static_cast<size_t>(p - sp.L0) * kD + col));
    }
  }
  if (completes) {
    float acc[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) acc[a] = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const float wi = w[q * 8 + r];
      const uint32_t uu[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        acc[2 * a] = fmaf(wi, bf16lo_to_f32(uu[a]), acc[2 * a]);
        acc[2 * a + 1] = fmaf(wi, bf16hi_to_f32(uu[a]), acc[2 * a + 1]);
      }
    }
#pragma unroll
    for (int a = 0; a < 8; ++a) part[r][(tid & 15) * 8 + a] = acc[a];
    __syncthreads();
    float tot = 0.f;
#pragma unroll
    for (int rr = 0; rr < 8; ++rr) tot += part[rr][tid];
    const long long row = entry_row(cache, i, b, 211);
    if (row >= 0) {
      __nv_bfloat16 hb = __float2bfloat16_rn(tot);
      (which ? cache.cv : cache.ck)[row * kD + quarter * 128 + tid] =
          *reinterpret_cast<uint16_t*>(&hb);
    }
    if (renews) cluster_wait();
  }
  if (renews && blockIdx.y == 0) {
    const int p = newest(sp.L1, tid);
    if (p >= sp.L0)
      cache.ws[static_cast<size_t>(i) * kBlk + tid] = c.s[static_cast<size_t>(sp.qs) + (p - sp.L0)];
  }
}

constexpr int kFinishY = 8;     // CTAs of a sequence, 16 ring slots each
constexpr int kFinishThreads = 256;

// What the attention reads beside the cache (null pointers: not wanted).
struct Queries {
  // four positions at a time; one at a time needs nothing
  int4* items;     // [cap] {table row, first packed token, its position, positions}
  int cap;
  int* tail16;     // [S] first entry of the last group of 16 when it is not full, or INT_MAX
  uint16_t* tail;  // [S, 16, 512] V rows of that group, zeros behind the last entry
  int* count;      // items in all
};

// Sum over the CTA (kFinishThreads threads).
__device__ __forceinline__ long long finish_sum(long long x, long long* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  long long t = 0;
  for (int w = 0; w < 8; ++w) t += red[w];
  return t;
}


// grid (S, kFinishY)
__global__ void __launch_bounds__(kFinishThreads)
    finish_kernel(const Chunk c, const Cache cache, const Queries qr) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = blockIdx.x, tid = threadIdx.x;
  const Span sp = span_of(c, i, blockIdx.y == 0 && tid == 0);
  // launched while entries_kernel may still read the rings
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (qr.items != nullptr) {
    __shared__ long long red[8];
    if (blockIdx.y == 0) {
      // Place of this sequence's items: behind those of all sequences with a longer context
      // (of equal ones, with a smaller number), so that the longest items are taken first.
      long long before = 0, all = 0;
      for (int j = tid; j < c.S; j += kFinishThreads) {
        const Span o = span_of(c, j, false);
        const int m = (o.n + 3) >> 2;
        all += m;
        if (o.L1 > sp.L1 || (o.L1 == sp.L1 && j < i)) before += m;
      }
      before = finish_sum(before, red);
      const int m = (sp.n + 3) >> 2;
      for (int r = tid; r < m; r += kFinishThreads) {
        const long long at = before + (m - 1 - r);
        if (at < qr.cap)   // always, unless offsets fall
          qr.items[at] = make_int4(i, sp.qs + 4 * r, sp.L0 + 4 * r, min(4, sp.n - 4 * r));
      }
      if (i == 0) {
        all = finish_sum(all, red);
        if (tid == 0) *qr.count = static_cast<int>(min(all, static_cast<long long>(qr.cap)));
      }
    }
    // the last group of 16 entries, rows 2 y and 2 y + 1
    const int cap = cache.max_pages << cache.page_shift;
    const int E = min(sp.L1 >> 7, cap);
    if (blockIdx.y == 0 && tid == 0 && sp.n > 0 && (sp.L1 >> 7) - 1 > cap)
      record_error(DEVERR_BAD_INPUT, 214);   // more entries visible than the table has room for
    if (blockIdx.y == 0 && tid == 0) qr.tail16[i] = (E & 15) != 0 ? E & ~15 : 0x7fffffff;
    if ((E & 15) != 0 && sp.n > 0 && tid < 128) {
      const int r = 2 * blockIdx.y + (tid >> 6), e = (E & ~15) + r, col = (tid & 63) * 8;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (e < E) {
        const int pg = cache.table[i * cache.table_ld + (e >> cache.page_shift)];
        if (static_cast<unsigned>(pg) < static_cast<unsigned>(cache.num_pages))
          x = *reinterpret_cast<const uint4*>(
              cache.cv +
              ((static_cast<size_t>(pg) << cache.page_shift) + (e & ((1 << cache.page_shift) - 1))) *
                  kD + col);
      }
      *reinterpret_cast<uint4*>(qr.tail + (static_cast<size_t>(i) * 16 + r) * kD + col) = x;
    }
  }
  constexpr int kSlots = kBlk / kFinishY;
  // 16 slots x (K, V) x 64 chunks of 16 bytes
#pragma unroll
  for (int q = 0; q < kSlots * 2 * 64 / kFinishThreads; ++q) {
    const int idx = q * kFinishThreads + tid;
    const int slot = blockIdx.y * kSlots + (idx >> 7), which = (idx >> 6) & 1, col = (idx & 63) * 8;
    const int p = newest(sp.L1, slot);
    if (sp.n > 0 && p >= sp.L0) {
      const size_t tok = static_cast<size_t>(sp.qs) + (p - sp.L0);
      const size_t dst = (static_cast<size_t>(i) * kBlk + slot) * kD + col;
      *reinterpret_cast<uint4*>((which ? cache.wv : cache.wk) + dst) =
          __ldg(reinterpret_cast<const uint4*>((which ? c.v : c.k) + tok * kD + col));
      if (col == 0 && which == 0) cache.ws[static_cast<size_t>(i) * kBlk + slot] = c.s[tok];
    }
  }
}

// One token a sequence, which completes a block: the ring is that block, its newest row
// in slot 127.  K or V and channel quarter y of sequence i by 128 threads that `sync`
// joins; the newest row and score come from the inputs, so that nobody waits for the
// ring's update.
struct RingScratch {
  float w[kBlk];
  float red[2][4];
  float part[8][kBlk + 4];
};
template <typename Sync>
__device__ __forceinline__ void entry_of_ring(const Chunk& c, const Cache& cache, int i, int L,
                                              int y, int tid, RingScratch& sm, Sync sync) {
  const int warp = tid >> 5, which = y >> 2, quarter = y & 3;
  const uint16_t* ring = (which ? cache.wv : cache.wk) + static_cast<size_t>(i) * kBlk * kD;
  const uint16_t* fresh = (which ? c.v : c.k) + static_cast<size_t>(i) * kD;
  const int col = quarter * 128 + (tid & 15) * 8;
  const int r = tid >> 4;
  const uint16_t sb = tid == kBlk - 1 ? c.s[i] : cache.ws[static_cast<size_t>(i) * kBlk + tid];
  uint4 x[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int t = q * 8 + r;
    x[q] = t == kBlk - 1 ? __ldg(reinterpret_cast<const uint4*>(fresh + col))
                         : *reinterpret_cast<const uint4*>(ring + static_cast<size_t>(t) * kD + col);
  }
  const float sv = __uint_as_float(static_cast<uint32_t>(sb) << 16);
  float m = warp_max(sv);
  if ((tid & 31) == 0) sm.red[0][warp] = m;
  sync();
  m = fmaxf(fmaxf(sm.red[0][0], sm.red[0][1]), fmaxf(sm.red[0][2], sm.red[0][3]));
  const float e = expf(sv - m);
  float z = warp_sum(e);
  if ((tid & 31) == 0) sm.red[1][warp] = z;
  sync();
  z = sm.red[1][0] + sm.red[1][1] + sm.red[1][2] + sm.red[1][3];
  sm.w[tid] = e / z;
  sync();
  float acc[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) acc[a] = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float wi = sm.w[q * 8 + r];
    const uint32_t uu[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      acc[2 * a] = fmaf(wi, bf16lo_to_f32(uu[a]), acc[2 * a]);
      acc[2 * a + 1] = fmaf(wi, bf16hi_to_f32(uu[a]), acc[2 * a + 1]);
    }
  }
#pragma unroll
  for (int a = 0; a < 8; ++a) sm.part[r][(tid & 15) * 8 + a] = acc[a];
  sync();
  float tot = 0.f;
#pragma unroll
  for (int rr = 0; rr < 8; ++rr) tot += sm.part[rr][tid];
  const int j = L / kBlk - 1, page = j >> cache.page_shift;
  int pg = -1;
  if (page < cache.max_pages) pg = cache.table[i * cache.table_ld + page];
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(cache.num_pages)) {
    if (tid == 0) record_error(DEVERR_BAD_INPUT, 213);
    return;
  }
  __nv_bfloat16 hb = __float2bfloat16_rn(tot);
  (which ? cache.cv : cache.ck)[((static_cast<size_t>(pg) << cache.page_shift) +
                                 (j & ((1 << cache.page_shift) - 1))) * kD + quarter * 128 + tid] =
      *reinterpret_cast<uint16_t*>(&hb);
}

// The append of one token a sequence (ring write and, where a block completes,
// its entry) in one launch: grid (S, 8), CTA (i, y) = (K or V, channel quarter)
// of sequence i, 128 threads.  Latency-bound.  (hca_paged_decode_step does the
// same inside the attention kernel for up to kInlineSeqs sequences.)
__global__ void __launch_bounds__(kThreads) step_kernel(const Chunk c, const Cache cache) {
  __shared__ RingScratch sm;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = blockIdx.x, tid = threadIdx.x;
  const int which = blockIdx.y >> 2, quarter = blockIdx.y & 3;
  const int L = c.ctx_len[i];
  if (L < 1) {
    if (tid == 0 && blockIdx.y == 0) record_error(DEVERR_BAD_INPUT, 212);
    return;
  }
  const size_t row = static_cast<size_t>(i) * kBlk + ((L - 1) & (kBlk - 1));
  if (tid < 16) {
    const int col = quarter * 128 + tid * 8;
    *reinterpret_cast<uint4*>((which ? cache.wv : cache.wk) + row * kD + col) =
        __ldg(reinterpret_cast<const uint4*>((which ? c.v : c.k) + static_cast<size_t>(i) * kD + col));
  }
  if (tid == 32 && blockIdx.y == 0) cache.ws[row] = c.s[i];
  if ((L & (kBlk - 1)) == 0)
    entry_of_ring(c, cache, i, L, blockIdx.y, tid, sm, [] { __syncthreads(); });
}

}  // namespace paged
}  // namespace hca
