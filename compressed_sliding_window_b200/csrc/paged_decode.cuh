// HCA decode over a paged cache: one query token at a time, split over the keys.
//
// For query i with context length L, page table row r and raw window rows
// w .. w + 127 (the ring of sequence i, or rows that a chunk laid out), one
// softmax over the entries j < nc(L-1) of row r's pages and the raw window, then
// out = sigmoid(g) * (P . V), as in decode.cuh; from there also the mapping
// onto the tensor cores (keys on the 128 lanes, heads on N):
//   S^T[key, head] = K_tile[key, :] . Q[head, :]        (M=128, N=64, K=512)
//   O^T[dv, head] += V_tile[:, dv]^T . P^T[:, head]      (4 x M=128 dv, N=64, K=128)
// TMEM: O^T (4 x 64 columns) and two 64-column S^T buffers.
//
// Pages.  A 16 KB stage is one 64-wide slab of 128 keys, brought by one box
// per page (1 to 8), each issued by a lane of the producer warp that keeps its
// page number in a register, read one tile ahead.  Boxes past the last visible
// entry use a page number outside of the pool, which fills their rows with
// zeros.  Rows of the last page behind the last visible entry may hold
// anything: their probabilities are set to 0, P.V stops at the next multiple of
// 16 keys, and the MMA warp clears the (at most 15) V rows up to there, because
// 0 x NaN would reach the sums otherwise.
//
// Softmax.  Eight warps: two per TMEM lane quadrant, one for each 32 heads, a
// thread owning one key.  The running maximum m of a head only has to be near
// the true one, so a tile whose scores all stay below m + 8 (in log2 units)
// keeps m: that takes one fused multiply-add and one maximum per score inside
// the thread and one vote, instead of a reduction over the 128 keys of every
// head.  Only a tile that exceeds the bound (the first of a segment always)
// reduces (redux.sync over the lanes, shared memory over the quadrants) and
// rescales.  Row sums stay in the thread, per head, until the segment ends.
// (The cross-lane form of decode.cuh, 124 shuffles a tile in four warps, takes
// 4.8 us a tile of 128 keys from L2.)
//
// Work split.  A query whose keys are all one CTA's is written straight out; one
// whose keys several CTAs share leaves partial results (O / l in fp32, m, l),
// which they merge.  When giving each CTA whole queries costs only a few tiles
// more than an even cut, that is done, and nothing is merged.  Else, with fewer
// queries than CTAs, each CTA has a part of one query; else the key tiles of all
// queries laid end to end are cut evenly.  With CTAs to spare, 2 or 4 of them take
// the same keys and each a half or a quarter of the value columns: 64 sequences at
// 131000 tokens 45.6 -> 39.8 us, one at 131073 20.5 -> 16.9 us, at 300 17.4 -> 11.6
// us, eight at 40000 25.0 -> 17.1 us.
#pragma once

#include "decode.cuh"
#include "hca_ptx.cuh"
#include "paged.cuh"

namespace hca {
namespace pdecode {

constexpr int kHeads = 64;
constexpr int kDim = 512;
constexpr int kKeyTile = 128;
constexpr int kWin = 128;
constexpr int kStages = 4;
constexpr int kSlab = 16384;        // [128 keys x 64 bf16] swizzled
constexpr int kStage = 2 * kSlab;
constexpr int kQSlab = 8192;        // [64 heads x 64 bf16] swizzled
constexpr int kProducers = 2;        // warps 0, 1; then the MMA warp, then the softmax warps
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kProducers + 1 + kSoftWarps);
constexpr int kWarps = kThreads / 32;
constexpr int kInlineSeqs = 512;    // up to this many queries each CTA plans for itself
// Tiles that the longest CTA may have beyond an even share for whole queries to be cheaper
// than parts of one query (80 sequences at 40000 tokens 26.7 us against 27.9) or than an even
// cut (200 sequences at 60000 tokens 67.9 us against 81.0, at 100000 94.1 against 100.2).
constexpr int kWholeTiles = 3;
constexpr int kWholeTilesCut = 5;
constexpr float kTau = 8.0f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

constexpr int kSmemQ = 0;                                   // 8 x 8 KB
constexpr int kSmemRing = 65536;                            // 4 x 32 KB
constexpr int kSmemPT = kSmemRing + kStages * kStage;       // P^T [128 keys x 64 heads] bf16
constexpr int kSmemM = kSmemPT + 16384;                     // [8 warps][32 m | 32 factors]
constexpr int kSmemMax = kSmemM + 8 * 64 * 4;               // [2 halves][4 quadrants][32]
constexpr int kSmemSum = kSmemMax + 2 * 4 * 32 * 4;
constexpr int kSmemFlag = kSmemSum + 2 * 4 * 32 * 4;        // [2 parities][2 halves][4]
constexpr int kSmemBar = kSmemFlag + 64;
constexpr int kSmemTiles = kSmemBar + 320;                  // [kInlineSeqs + 1] int64 prefix
constexpr int kSmemLen = kSmemTiles + 8 * (kInlineSeqs + 1) + 8;
constexpr int kSmemRow = kSmemLen + 4 * kInlineSeqs;        // [kInlineSeqs] table row
constexpr int kSmemBytes = kSmemRow + 4 * kInlineSeqs;
constexpr int kSmemAlloc = kSmemBytes + 1024;
static_assert(kSmemAlloc <= 232448 - 1024, "shared memory budget");
static_assert(kStages * kStage == kKeyTile * kDim * 2, "a tile's K or V is one round of the ring");

enum {
  B_QFULL = 0, B_QEMPTY = 1, B_FULL = 2, B_EMPTY = B_FULL + kStages, B_SFULL = B_EMPTY + kStages,
  B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_PFREE = B_PFULL + 1, B_OFULL = B_PFREE + 1,
  B_OFREE = B_OFULL + 1, B_DRAIN = B_OFREE + 1, B_MERGE = B_DRAIN + 1, B_RENEWED = B_MERGE + 1,
  B_COUNT = B_RENEWED + 1
};
constexpr int kTmemSlot = 8 * B_COUNT;
constexpr int kAbortSlot = kTmemSlot + 4;
static_assert(kAbortSlot + 4 <= 320, "barrier region overflow");

constexpr uint32_t kTmemO = 0, kTmemS0 = 256, kTmemS1 = 320, kTmemCols = 512;

// Workspace (bytes): partial O / l in fp32, [slots][64 chunks][16 heads][32
// value columns], chunk 16 (column / 128) + 4 (head / 16) + column / 32 % 4;
// then [slots][2][64] fp32 (m, l) in log2 units (CTAs that share keys write the
// same); slots = grid + S.
__host__ __device__ inline size_t ws_o_bytes(int slots) {
  return static_cast<size_t>(slots) * kHeads * kDim * 4;
}
__host__ __device__ inline size_t ws_bytes(int slots) {
  return ws_o_bytes(slots) + static_cast<size_t>(slots) * 2 * kHeads * 4;
}

struct Params {
  const int* ctx_len;  // [S]
  int S;
  int max_nc;
  float scale_log2;
  float* ws_o;
  float* ws_ml;
  long long* seq_tile; // [S + 2] tile prefix and longest query (plan_kernel, S > kInlineSeqs)
  unsigned* arrived;   // [grid] arrivals at the merge of the query whose first CTA is c: zero
                       // between calls
  unsigned long long* gsync;   // grid barrier of the head mix
  const uint16_t* g;   // [S, 64, 512]
  uint16_t* out;
  const uint16_t* vha_down;
  const uint16_t* vha_up;
  int vha_rank;
  const int* table;    // row r at table + r * table_ld
  long long table_ld;
  int num_pages;
  int page_shift;
  // Queries that are the tokens of a chunk (chunk.q_start set; S: at most as many): query i
  // is token first + i, first = q_start[0] (what lies before is no sequence's); as one of
  // sequence j it has the window rows first + i + kPad j .. of the laid out raw tokens.
  // Else query i is sequence i, its window the ring at row 128 i; with chunk.k set the call
  // first appends token i of the chunk to `cache` (step).
  paged::Chunk chunk;
  paged::Cache cache;
  // The kernel in front writes nothing that is read here but the window rows: only
  // the loads of those wait for it.  (An entry that it completes is not visible yet:
  // a block is seen 128 positions after its last token, and a chunk in this form has
  // fewer.)
  int only_window;
};

struct Maps {
  CUtensorMap q;    // (64, S*64, 8, 1),  box (64, 64, 8, 1): the whole q of one query
  CUtensorMap g;    // (64, S*64, 8, 1),  box (64, 64, 2, 1): 128 columns of one query's gate
  CUtensorMap ck;   // (64, page, 8, pages), box (64, page, 1, 1)
  CUtensorMap cv;
  CUtensorMap wk;   // (64, rows, 8, 1),  box (64, 128, 2, 1)
  CUtensorMap wv;
};

struct SeqInfo {
  int L, nc, nct;   // context length, visible entries, compressed tiles
};
__device__ __forceinline__ SeqInfo seq_info(int L, int max_nc) {
  SeqInfo r;
  r.L = max(1, L);
  r.nc = min(max(decode::nc_of_len(r.L), 0), max_nc);
  r.nct = (r.nc + kKeyTile - 1) / kKeyTile;
  return r;
}
// tiles of a query of length L; a length out of range is reported by one caller
__device__ __forceinline__ int tiles_of(int L, int max_nc, bool report) {
  if (report && (L < 1 || decode::nc_of_len(L) > max_nc)) record_error(DEVERR_BAD_INPUT, 103);
  return seq_info(L, max_nc).nct + 1;
}

// Sequence of query i of a chunk: the last whose first token is not behind it.
__device__ __forceinline__ int seq_of(const paged::Chunk& c, int i) {
  int lo = 0, hi = c.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.q_start[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tile prefix of S queries by one CTA of NT threads, each a run of queries:
// out[i], out[S] = total, and the longest query in *longest.  first: token that is query 0 of a
// chunk.  lens, rows (may be null): context length and table row of each query.
template <int NT>
__device__ __forceinline__ void plan_tiles(const Params& p, int first, long long* out, int* lens,
                                           int* rows, int* longest, bool report) {
  __shared__ long long wsum[NT / 32];
  __shared__ int wmax[NT / 32];
  const int S = p.S;
  const int per = (S + NT - 1) / NT;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, S), i1 = min(i0 + per, S);
  long long run = 0;
  int most = 0;
  for (int i = i0; i < i1; ++i) {
    int L, row = i;
    if (p.chunk.q_start != nullptr) {
      row = seq_of(p.chunk, first + i);
      const paged::Span sp = paged::span_of(p.chunk, row, false);
      L = sp.L0 + min(max(first + i - sp.qs, 0), max(sp.n - 1, 0)) + 1;
    } else {
      L = p.ctx_len[i];
    }
    const int n = tiles_of(L, p.max_nc, report);
    if (lens != nullptr) {
      lens[i] = L;
      rows[i] = row;
    }
    out[i] = n;
    run += n;
    most = max(most, n);
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long x = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    wsum[w] = x;
    wmax[w] = most;
  }
  __syncthreads();
  long long before = x - run;
  for (int v = 0; v < w; ++v) before += wsum[v];
  for (int i = i0; i < i1; ++i) {
    const long long n = out[i];
    out[i] = before;
    before += n;
  }
  if (threadIdx.x == NT - 1) {
    out[S] = before;
    int m = 0;
    for (int v = 0; v < NT / 32; ++v) m = max(m, wmax[v]);
    *longest = m;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(1024) plan_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int longest;
  plan_tiles<1024>(p, 0, p.seq_tile, nullptr, nullptr, &longest, true);
  if (threadIdx.x == 0) p.seq_tile[p.S + 1] = longest;
}

// largest s in [0, S) with first[s] <= x
__device__ __forceinline__ int find_seq(const long long* first, int S, long long x) {
  return decode::find_seq(first, S, x);
}

// Page number of box `b` of the 128-entry tile `j`: num_pages (zero fill) for a
// box past the last visible entry or a page number outside the pool (reported).
__device__ __forceinline__ int box_page(const Params& p, const int* row, int nc, int j, int b) {
  const int e = j * kKeyTile + (b << p.page_shift);
  if (e >= nc) return p.num_pages;
  const int pg = row[e >> p.page_shift];
  if (static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages)) return pg;
  record_error(DEVERR_BAD_INPUT, 102);
  return p.num_pages;
}

// Clears rows [valid, next multiple of 16) of a stage (one warp).
__device__ __forceinline__ void clear_rows(uint8_t* stage, int valid, int lane) {
  const int end = (valid + 15) & ~15;
  for (int i = valid * 8 + lane; i < end * 8; i += 32) {
    *reinterpret_cast<uint4*>(stage + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(stage + kSlab + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums 32 per-lane values over the lanes of a warp: lane l gets value l's sum.
__device__ __forceinline__ float lanes_sum32(float (&a)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16, n = 32; o >= 1; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = up ? a[i] : a[i + n / 2];
      const float keep = up ? a[i + n / 2] : a[i];
      a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return a[0];
}

// CTAs of a query of `t` tiles when each takes at most T (or, by rounding, a tile
// more: what counts is that all CTAs find the same)
__device__ __forceinline__ int parts_of(int t, float inv) {
  return max(1, static_cast<int>(ceilf(static_cast<float>(t) * inv - 1e-3f)));
}

// With fewer queries than CTAs each CTA works for one query: query s is shared
// by parts_of(t_s, T) CTAs, T the smallest for which all fit on the grid (found
// by bisection, every warp for itself).  Sets the CTA's query, its part of n,
// or n = 0 for a CTA that is left over.
__device__ __forceinline__ void own_query(const long long* tiles, int S, int longest, int G, int cta,
                                          int& s, int& part, int& n) {
  const int lane = threadIdx.x & 31;
  auto all_parts = [&](int T) -> int {
    const float inv = __frcp_rn(static_cast<float>(T));
    int x = 0;
    for (int i = lane; i < S; i += 32) x += parts_of(static_cast<int>(tiles[i + 1] - tiles[i]), inv);
    return __reduce_add_sync(0xffffffffu, x);
  };
  // sum of ceil(t / T) < N / T + S: T = ceil(N / (G - S)) always fits
  const int N = static_cast<int>(tiles[S]);
  int lo = max(1, (N + G - 1) / G), hi = max(lo, min(longest, (N + G - S - 1) / (G - S)));
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (all_parts(mid) <= G) hi = mid; else lo = mid + 1;
  }
  const float inv = __frcp_rn(static_cast<float>(lo));
  int before = 0;
  n = 0;
  for (int base = 0; base < S && n == 0; base += 32) {
    const int i = base + lane;
    const int m = i < S ? parts_of(static_cast<int>(tiles[i + 1] - tiles[i]), inv) : 0;
    int x = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int first = before + x - m;
    const unsigned hit = __ballot_sync(0xffffffffu, m > 0 && cta >= first && cta < first + m);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      s = base + l;
      n = __shfl_sync(0xffffffffu, m, l);
      part = cta - __shfl_sync(0xffffffffu, first, l);
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
}

// ---------------------------------------------------------------------------
// Merge of a query whose tiles n CTAs share, by all of them: CTA i of the n
// takes the i-th of n equal runs of the chunks (16 heads x 32 value columns) of
// their column groups in all n partials, once all have been written (a counter per query; a CTA waits
// only for those that share its first or last query, and only after its own
// tiles).  A split's share is contiguous, so one bulk copy brings it into shared
// memory (a CTA's own stays there from the start where its tiles are one part
// of one query); meanwhile the warps find the weights w = l_f 2^(m_f - M) / L of
// all splits and heads.  Then a warp adds up a chunk, lane l holding heads
// 4 q + l / 8 and columns 4 (l % 8) .. + 3.  With fewer chunks than warps, several
// warps share a chunk's splits and add up through shared memory.
// ---------------------------------------------------------------------------
// Splits up to which the weights fit the P^T buffer; with more the Q buffer
// takes them, and the data have the ring alone.
constexpr int kFewSplits = 64;
__device__ __forceinline__ int merge_room(int n) { return n <= kFewSplits ? 96 : 64; }   // chunks
__device__ __forceinline__ uint32_t merge_data(int n) { return n <= kFewSplits ? kSmemQ : kSmemRing; }
// first chunk of CTA i of the n that merge column groups cg .. cg + nv - 1
__device__ __forceinline__ int merge_first(int i, int n, int cg, int nv) {
  return 16 * cg + 16 * nv * i / n;
}

__device__ __forceinline__ void merge_query(const Params& p, int s, size_t slot, unsigned* arrived,
                                            int i, int n, int cg, int nv, bool kept, uint8_t* smem, uint32_t sbase, uint32_t bar_m,
                                            uint32_t& phase, volatile int* abort_flag, int warp,
                                            int lane) {
  const int k0 = merge_first(i, n, cg, nv), nk = merge_first(i + 1, n, cg, nv) - k0;
  const int batch = nk > 0 ? min(n, merge_room(n) / nk) : n;   // splits at a time
  const uint32_t data = merge_data(n);
  const float* po = p.ws_o + slot * kHeads * kDim + 512 * k0;
  __shared__ int late;
  auto load = [&](int f0, int f1) {   // one thread
    uint32_t bytes = 0;
    for (int f = f0; f < f1; ++f) bytes += (kept && f == i) ? 0u : 2048u * nk;
    mbar_expect_tx(bar_m, bytes);
    for (int f = f0; f < f1; ++f)
      if (!(kept && f == i))
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1], %2, [%3];" ::"r"(sbase + data + 2048u * nk * (f - f0)),
            "l"(po + static_cast<size_t>(f) * kHeads * kDim), "r"(2048u * nk), "r"(bar_m)
            : "memory");
  };
  if (threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    late = 0;
    for (uint32_t k = 1;; ++k) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
      if (v >= static_cast<unsigned>(n)) break;
      if ((k & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(DEVERR_TIMEOUT, 72);
        late = 1;
        break;
      }
    }
    if (nk > 0 && !late) {
      fence_proxy_async_all();   // read by bulk copies; and this memory's earlier generic uses
      load(0, batch);
    }
  }
  __syncthreads();
  if (nk > 0 && !late) {
    // heads 2 lane, 2 lane + 1: M and L over the splits, every warp for itself, then the
    // weights of splits warp, warp + kWarps, ..
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml + slot * 128);
    float* w = reinterpret_cast<float*>(smem + (n <= kFewSplits ? kSmemPT : kSmemQ));   // [n][64]
    float2 M = make_float2(-INFINITY, -INFINITY), L = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int f0 = 0; f0 < n; f0 += 8) {
      float2 m[8], l[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool in = f0 + u < n;
        m[u] = in ? __ldcg(ml + 64 * (f0 + u) + lane) : make_float2(-INFINITY, -INFINITY);
        l[u] = in ? __ldcg(ml + 64 * (f0 + u) + 32 + lane) : make_float2(0.f, 0.f);
      }
      float2 T = M;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        T.x = fmaxf(T.x, m[u].x);
        T.y = fmaxf(T.y, m[u].y);
      }
      L.x *= ex2_approx(M.x - T.x);   // the first time 0 x 2^-inf
      L.y *= ex2_approx(M.y - T.y);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        L.x = fmaf(l[u].x, ex2_approx(m[u].x - T.x), L.x);
        L.y = fmaf(l[u].y, ex2_approx(m[u].y - T.y), L.y);
      }
      M = T;
    }
    const float2 inv = make_float2(1.f / L.x, 1.f / L.y);
    for (int f = warp; f < n; f += kWarps) {
      const float2 m = __ldcg(ml + 64 * f + lane), l = __ldcg(ml + 64 * f + 32 + lane);
      *reinterpret_cast<float2*>(w + 64 * f + 2 * lane) =
          make_float2(l.x * ex2_approx(m.x - M.x) * inv.x, l.y * ex2_approx(m.y - M.y) * inv.y);
    }
    __syncthreads();
    const int share = nk < kWarps ? kWarps / nk : 1;            // warps per chunk
    const int part = warp % share, slot0 = warp / share, chunks = kWarps / share;
    // More than one batch only where nk <= 2 (and so one round of chunks).
    for (int r0 = 0; r0 < nk; r0 += chunks) {
      const int r = r0 + slot0, k = k0 + r;
      const bool mine = slot0 < chunks && r < nk;
      const int h0 = 16 * ((k >> 2) & 3) + (lane >> 3);         // heads h0 + 4 q
      const size_t at = (static_cast<size_t>(s) * kHeads + h0) * kDim + 128 * (k >> 4) +
                        32 * (k & 3) + 4 * (lane & 7);
      float acc[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) acc[t] = 0.f;
      uint2 gv[4];
      if (mine) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          gv[q] = __ldg(reinterpret_cast<const uint2*>(p.g + at + 4 * q * kDim));
      }
      for (int f0 = 0; f0 < n; f0 += batch) {
        const int f1 = min(n, f0 + batch);
        if (f0 > 0) {
          __syncthreads();   // the last batch has been read
          if (threadIdx.x == 0) {
            fence_proxy_async_all();
            load(f0, f1);
          }
        }
        if (r0 == 0) {
          // late copies may still land: nobody may leave before abort_drain
          if (!mbar_wait_warp(bar_m, phase, abort_flag, kWaitLimitNs, 73) && lane == 0)
            abort_drain(abort_flag);
          phase ^= 1;
        }
        if (mine) {
          const float4* src = reinterpret_cast<const float4*>(smem + data) + 128 * r + lane;
#pragma unroll 2
          for (int f = f0 + part; f < f1; f += share) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 x = src[128 * nk * (f - f0) + 32 * q];
              const float wf = w[64 * f + h0 + 4 * q];
              acc[4 * q] = fmaf(wf, x.x, acc[4 * q]);
              acc[4 * q + 1] = fmaf(wf, x.y, acc[4 * q + 1]);
              acc[4 * q + 2] = fmaf(wf, x.z, acc[4 * q + 2]);
              acc[4 * q + 3] = fmaf(wf, x.w, acc[4 * q + 3]);
            }
          }
        }
      }
      if (share > 1) {   // uniform in the CTA; the data have been read by all
        float* add = reinterpret_cast<float*>(smem + data);       // [warps][512]
        __syncthreads();
        if (mine && part > 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(add + warp * 512 + 128 * q + 4 * lane) =
                make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        }
        __syncthreads();
        if (mine && part == 0) {
          for (int v = 1; v < share; ++v) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 x =
                  *reinterpret_cast<const float4*>(add + (warp + v) * 512 + 128 * q + 4 * lane);
              acc[4 * q] += x.x;
              acc[4 * q + 1] += x.y;
              acc[4 * q + 2] += x.z;
              acc[4 * q + 3] += x.w;
            }
          }
        }
      }
      if (mine && part == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(p.out + at + 4 * q * kDim) =
              make_uint2(pack_bf16x2(gate32(acc[4 * q], bf16lo_to_f32(gv[q].x)),
                                     gate32(acc[4 * q + 1], bf16hi_to_f32(gv[q].x))),
                         pack_bf16x2(gate32(acc[4 * q + 2], bf16lo_to_f32(gv[q].y)),
                                     gate32(acc[4 * q + 3], bf16hi_to_f32(gv[q].y))));
      }
    }
  }
  // Everybody's second arrival, after the wait above; the last one leaves the
  // counter at zero for the next call.
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned old;
    asm volatile("atom.add.relaxed.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(old)
                 : "l"(arrived)
                 : "memory");
    if (old == 2u * n - 1) *arrived = 0u;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ Maps maps, const Params p0) {
  Params p = p0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kSmemQ, sRing = sbase + kSmemRing, sPT = sbase + kSmemPT;
  auto bar = [&](int i) -> uint32_t { return sbase + kSmemBar + 8u * static_cast<uint32_t>(i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmemBar + kAbortSlot);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemBar + kTmemSlot);
  long long* sT = reinterpret_cast<long long*>(smem + kSmemTiles);
  int* sL = reinterpret_cast<int*>(smem + kSmemLen);
  __shared__ int longest, first;   // longest query in tiles; first token of a chunk

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == kThreads - 32) {   // a warp with nothing to plan for, as a rule
    mbar_init(bar(B_QFULL), 1);
    mbar_init(bar(B_QEMPTY), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_SFREE + s), kSoftWarps);
    }
    mbar_init(bar(B_PFULL), kSoftWarps);
    mbar_init(bar(B_PFREE), 1);
    mbar_init(bar(B_OFULL), 1);
    mbar_init(bar(B_OFREE), kSoftWarps);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_MERGE), 1);
    mbar_init(bar(B_RENEWED), kSoftWarps);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.ck);
    tma_prefetch_desc(&maps.cv);
    tma_prefetch_desc(&maps.wk);
    tma_prefetch_desc(&maps.wv);
    tma_prefetch_desc(&maps.g);
  }
  if (warp == kProducers) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  // The plan, here for up to kInlineSeqs queries.  The kernel may have been
  // launched while the one in front of it still runs.
  const bool inl = p.S <= kInlineSeqs;
  int* sRow = reinterpret_cast<int*>(smem + kSmemRow);
  if (!p.only_window) asm volatile("griddepcontrol.wait;" ::: "memory");
  int skip = 0;   // first token of a chunk
  if (inl) {
    if (p.chunk.q_start != nullptr) {
      skip = min(max(p.chunk.q_start[0], 0), p.S);
      p.S = max(min(p.chunk.q_start[p.chunk.S], p.S) - skip, 0);
    }
    if (threadIdx.x == 0) first = skip;   // read behind the plan's barriers
    plan_tiles<kThreads>(p, skip, sT, sL, sRow, &longest, blockIdx.x == 0);
  } else {
    if (threadIdx.x == 0) {
      first = 0;
      longest = static_cast<int>(p.seq_tile[p.S + 1]);
    }
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long* tiles = inl ? sT : p.seq_tile;
  const int* lens = inl ? sL : p.ctx_len;
  // How the tiles are split: whole queries per CTA where that costs little, else
  // one query per CTA where there are fewer queries than CTAs, else an even cut
  // of all tiles laid end to end.
  const long long N = tiles[p.S];
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const long long even = decode::div_nn(N + grid - 1, grid);
  // Column split (lcs > 0): 2 or 4 CTAs, 1 << lcs, share the keys of a query or of a part
  // of one and take a half or a quarter of its value columns each: the keys come from L2
  // again, but a CTA loads less, and its epilogue and what it merges are as much shorter.
  // Whole queries are split where that leaves no CTA with two; parts where every CTA still
  // has one tile only.
  int lcs = 4 * p.S <= grid ? 2 : 2 * p.S <= grid ? 1 : 0;
  // Whole with 1 to 37 queries takes about 6 + 2.8 us a tile of the longest, with 64 of them
  // 8 + 3.6; in parts 16.3 us with a tile a CTA and four column groups, else 13 + 5.8 us a
  // tile of the even share.  Longest and share in tiles: 3 and 1 14.9 us whole against 16.3,
  // 4 and 1 17.3 against 16.3; 9 and 2 33.2 against 28.7; 9 and 4 39.8 against 45.6.
  const bool whole = lcs > 0 ? 4 * static_cast<long long>(longest) <= 7 * even + 8
                             : static_cast<long long>(longest) * ((p.S + grid - 1) / grid) <=
                                   even + (p.S < grid ? kWholeTiles : kWholeTilesCut);
  const bool own = !whole && p.S < grid;
  if (!whole) {
    lcs = 0;
    if (own)
      while (lcs < 2 && (N << (lcs + 1)) <= grid && p.S < grid >> (lcs + 1)) ++lcs;
  }
  const int nv = kStages >> lcs;                  // 128-column groups of this CTA
  const int cg = (cta & ((1 << lcs) - 1)) * nv;   // the first of them
  const int vcta = cta >> lcs;                    // CTA of the split by keys
  const int G = static_cast<int>(min(static_cast<long long>(grid), max(N, 1LL)));   // even cut
  long long A0 = 0, A1 = 0;
  int mine = 0, part = 0, parts = 0;   // own: this CTA's query
  if (whole && lcs > 0) {
    if (vcta < p.S) {
      A0 = tiles[vcta];
      A1 = tiles[vcta + 1];
    }
  } else if (whole) {
    A0 = tiles[decode::div_nn(static_cast<long long>(p.S) * cta, grid)];
    A1 = tiles[decode::div_nn(static_cast<long long>(p.S) * (cta + 1), grid)];
  } else if (own) {
    own_query(tiles, p.S, longest, grid >> lcs, vcta, mine, part, parts);
    if (parts > 0) {
      const int t = static_cast<int>(tiles[mine + 1] - tiles[mine]);
      A0 = tiles[mine] + t * part / parts;
      A1 = tiles[mine] + t * (part + 1) / parts;
    }
  } else if (cta < G) {
    A0 = decode::div_nn(N * cta, G);
    A1 = decode::div_nn(N * (cta + 1), G);
  }
  // own: this CTA's share of its own partial stays in shared memory, where nothing
  // follows its only segment, if all splits' shares fit there at once
  const int k0 = own && parts > 1 ? merge_first(part, parts, cg, nv) : 0;
  const int nk = own && parts > 1 ? merge_first(part + 1, parts, cg, nv) - k0 : 0;
  const bool kept = nk > 0 && parts * nk <= merge_room(parts);
  auto owner = [&](long long x) -> int {   // even cut: CTA of tile x
    return static_cast<int>(decode::div_nn((x + 1) * G + N - 1, N)) - 1;
  };
  // Segments: maximal runs of this CTA's tiles inside one query.
  const int s_first = A0 < A1 ? find_seq(tiles, p.S, A0) : 0;
  // A step's append, by the warps that have nothing to do until the first scores are there.
  // The new rows go into the rings of the queries whose windows this CTA reads (CTAs that
  // read the same one write the same); only the window's loads wait for that.  The entries
  // of the blocks that the tokens complete, which no query of this call sees, are dealt out
  // over all CTAs, a unit of K or V and channel quarter to four warps.  Against the append as
  // a launch of its own: 148 sequences at 300 tokens 22.0 -> 20.3 us, 64 at 131072 (each
  // completes a block) 48.6 -> 47.6 us, 200 at 30000 53.7 -> 51.2 us; only many blocks at once
  // lose, 200 at 30080 (each completes one) 60.3 -> 66.7 us.  The host picks the form and does
  // not know the lengths; even sequences in lockstep complete their blocks in one step of 128.
  const bool step = p.chunk.k != nullptr && p.chunk.q_start == nullptr;
  const bool renews = step && A0 < A1 && tiles[s_first + 1] <= A1;
  if (step && warp > kProducers) {
    const int t = threadIdx.x - 32 * (kProducers + 1);   // 0 .. 255
    if (renews) {
      for (int s = s_first; s < p.S && tiles[s + 1] <= A1; ++s) {
        if (sL[s] < 1) continue;
        const size_t row = static_cast<size_t>(s) * kWin + ((sL[s] - 1) & (kWin - 1));
        if (t < 128) {
          const size_t to = row * kDim + 8 * (t & 63), from = static_cast<size_t>(s) * kDim + 8 * (t & 63);
          *reinterpret_cast<uint4*>((t < 64 ? p.cache.wk : p.cache.wv) + to) =
              __ldg(reinterpret_cast<const uint4*>((t < 64 ? p.chunk.k : p.chunk.v) + from));
        } else if (t == 128) {
          p.cache.ws[row] = p.chunk.s[s];
        }
      }
      __threadfence();           // read next by the window's copies, which go to L2
      fence_proxy_async_all();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_RENEWED));
    }
    const int half = t >> 7;
    paged::RingScratch& sm = *reinterpret_cast<paged::RingScratch*>(smem + kSmemPT + 8192 * half);
    for (long long u = 2 * cta + half; u < 8LL * p.S; u += 2 * grid) {
      const int s = static_cast<int>(u >> 3), L = sL[s];
      if (L >= 1 && (L & (kWin - 1)) == 0) {
        paged::entry_of_ring(p.chunk, p.cache, s, L, static_cast<int>(u & 7), t & 127, sm,
                             [&] { named_bar_sync(1 + half, 128); });
        named_bar_sync(1 + half, 128);   // the scratch may be written again
      }
    }
    // A half's scratch lies in the P^T buffer, whose rows both halves write: nobody stores
    // P before the other half's last entry is out.
    named_bar_sync(3, 32 * kSoftWarps);
  }
  if (A0 < A1) {  // uniform across the CTA

  if (warp < kProducers) {
    // ------------------------------------------------------------ producers
    // Two warps take turns at the stages; lane b (+ boxes for the second slab)
    // loads box b of a stage.
    const int me = warp;
    const int boxes = kKeyTile >> p.page_shift;
    const int bx = lane & (boxes - 1), slab = lane / boxes;
    const uint32_t boff = slab * kSlab + bx * (kSlab / boxes);
    // Uses of the ring so far: use u takes stage u & 3, which warp u & 1 loads.  A K tile
    // is four uses, a V tile one for each of this CTA's column groups.
    uint32_t u = 0, quse = 0;
    bool ok = true;
    bool waited = !p.only_window && !renews;
    // The eight slabs of a K tile, or those of this CTA's columns of a V tile: entries of
    // the page `pg` of this lane's box, or (pg < 0) the window rows from y on
    auto load = [&](const CUtensorMap* map, int pg, int y, bool values) {
      if (pg < 0 && !waited) {
        if (step) {
          // bounded, as all waits: a producer that gave up elsewhere is not waited for
          ok = ok && mbar_wait_warp(bar(B_RENEWED), 0, abort_flag, kWaitLimitNs, 42);
          fence_proxy_async_all();
        } else {
          asm volatile("griddepcontrol.wait;" ::: "memory");
        }
        waited = true;
      }
      const int n = values ? nv : kStages, z = values ? 2 * cg : 0;
#pragma unroll
      for (int t = 0; t < kStages / kProducers; ++t) {
        const int i = kProducers * t + ((u ^ me) & 1);
        if (i >= n) break;
        const int st = (u + i) & (kStages - 1);
        if (lane == 0) {
          ok = ok && mbar_wait(bar(B_EMPTY + st), (((u + i) / kStages) & 1) ^ 1, abort_flag,
                               kWaitLimitNs, 40);
          if (ok) mbar_expect_tx(bar(B_FULL + st), kStage);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        __syncwarp();
        if (ok && pg >= 0 && slab < 2)
          decode::tma_load_4d_dec(sRing + st * kStage + boff, map, bar(B_FULL + st), 0, 0,
                                  z + 2 * i + slab, pg);
        else if (ok && pg < 0 && lane == 0)
          decode::tma_load_4d_dec(sRing + st * kStage, map, bar(B_FULL + st), 0, y, z + 2 * i, 0);
      }
      u += n;
    };
    long long x = A0;
    for (int s = s_first; x < A1 && ok; ++s) {
      const SeqInfo si = seq_info(lens[s], p.max_nc);
      const long long seg_end = min(A1, tiles[s + 1]);
      const int j0 = static_cast<int>(x - tiles[s]);
      const int j1 = static_cast<int>(seg_end - tiles[s]);
      if (me == 0) {
        if (lane == 0) {
          ok = mbar_wait(bar(B_QEMPTY), (quse & 1) ^ 1, abort_flag, kWaitLimitNs, 41);
          if (ok) {
            mbar_expect_tx(bar(B_QFULL), 8 * kQSlab);
            decode::tma_load_4d_dec(sQ, &maps.q, bar(B_QFULL), 0, (skip + s) * kHeads, 0, 0);
          }
          if (j0 == 0 && seg_end == tiles[s + 1])   // a whole query: its gate, into L2
            for (int c = cg; c < cg + nv; ++c)
              prefill3::tma_prefetch_4d(&maps.g, 0, (skip + s) * kHeads, 2 * c, 0);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      ++quse;
      const int trow = inl ? sRow[s] : s;
      const int* prow = p.table + trow * p.table_ld;
      const int win = p.chunk.q_start != nullptr ? skip + s + paged::kPad * trow : s * kWin;
      auto page_of = [&](int j) -> int {
        return j < si.nct ? box_page(p, prow, si.nc, j, bx) : -1;
      };
      int pg = page_of(j0), pg1 = j0 + 1 < j1 ? page_of(j0 + 1) : -1;
      load(pg >= 0 ? &maps.ck : &maps.wk, pg, win, false);
      for (int j = j0; j < j1 && ok; ++j) {
        const int pg2 = j + 2 < j1 ? page_of(j + 2) : -1;   // needed one tile later
        if (j + 1 < j1) load(pg1 >= 0 ? &maps.ck : &maps.wk, pg1, win, false);
        load(pg >= 0 ? &maps.cv : &maps.wv, pg, win, true);
        pg = pg1;
        pg1 = pg2;
      }
      x = seg_end;
    }
    // The last copies are out: bring the gate of the columns that this CTA will merge
    // into L2.
    if (own && nk > 0 && me == 0 && lane == 0)
      for (int c = k0 >> 4; c <= (k0 + nk - 1) >> 4; ++c)
        prefill3::tma_prefetch_4d(&maps.g, 0, (skip + mine) * kHeads, 2 * c, 0);
  } else if (warp == kProducers) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp waits and walks the tiles; one elected lane issues.  Under
    // a branch on elect.sync in warp-uniform code the descriptors stay in
    // uniform registers: 49 cycles an MMA of 128 x 64 x 16 (what its operands
    // take from shared memory) against 115 under a branch on the lane number.
    // `ok` is uniform; after a failed wait the loops run on without waiting.
    bool ok = true;
    uint32_t u = 0, quse = 0, sidx = 0, pvidx = 0, nseg = 0;   // as the producers'
    const uint32_t idesc_s = idesc_bf16_f32(128, 64, false, false);
    const uint32_t idesc_o = idesc_bf16_f32(128, 64, true, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait = [&](int b, uint32_t par, unsigned where) {
      if (ok && !__all_sync(0xffffffffu, mbar_try_wait(bar(b), par)))
        ok = mbar_wait_warp(bar(b), par, abort_flag, kWaitLimitNs, where);
    };
    auto issue_s = [&]() {
      const uint32_t buf = sidx & 1;
      wait(B_SFREE + buf, ((sidx >> 1) & 1) ^ 1, 50);
      const uint32_t dS = tm + (buf ? kTmemS1 : kTmemS0);
      const uint32_t u0 = __shfl_sync(0xffffffffu, u, 0);   // in a uniform register
#pragma unroll 1
      for (int i = 0; i < kStages; ++i) {
        const uint32_t use = u0 + i;
        const int st = use & (kStages - 1);
        wait(B_FULL + st, (use / kStages) & 1, 51);
        tc_fence_after();
        const uint64_t ad = sdesc_sw128(sRing + st * kStage, 16, 1024);
        const uint64_t bd = sdesc_sw128(sQ + i * 2 * kQSlab, 16, 1024);
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)   // 16 channels each: 32 bytes on, or the next slab
            umma_bf16(dS, ad + 2 * (k & 3) + (k >> 2) * (kSlab >> 4),
                      bd + 2 * (k & 3) + (k >> 2) * (kQSlab >> 4), idesc_s, (i | k) != 0);
          umma_commit(bar(B_EMPTY + st));
          if (i == kStages - 1) umma_commit(bar(B_SFULL + buf));
        }
        __syncwarp();
      }
      u += kStages;
      ++sidx;
    };
    auto issue_pv = [&](bool first, int valid) {
      wait(B_PFULL, pvidx & 1, 52);
      if (first) wait(B_OFREE, (nseg & 1) ^ 1, 53);
      const int ksteps = (valid + 15) >> 4;
      const uint32_t u0 = __shfl_sync(0xffffffffu, u, 0);
#pragma unroll 1
      for (int c = 0; c < nv; ++c) {   // 128 value columns each
        const uint32_t use = u0 + c;
        const int st = use & (kStages - 1);
        wait(B_FULL + st, (use / kStages) & 1, 54);
        if (ok && (valid & 15) != 0) {
          clear_rows(smem + kSmemRing + st * kStage, valid, lane);
          fence_proxy_async_smem();               // read next by the tensor core
        }
        __syncwarp();
        tc_fence_after();
        const uint64_t ad = sdesc_sw128(sRing + st * kStage, kSlab, 1024);
        const uint64_t bd = sdesc_sw128(sPT, kSlab, 1024);
        if (ok && elect_one()) {
          if (ksteps == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_bf16(tm + kTmemO + 64 * c, ad + 128 * k, bd + 128 * k, idesc_o,
                        (!first || k > 0) ? 1u : 0u);
          } else {
#pragma unroll 1
            for (int k = 0; k < ksteps; ++k)
              umma_bf16(tm + kTmemO + 64 * c, ad + 128 * k, bd + 128 * k, idesc_o,
                        (!first || k > 0) ? 1u : 0u);
          }
          umma_commit(bar(B_EMPTY + st));
          if (c == nv - 1) umma_commit(bar(B_PFREE));
        }
        __syncwarp();
      }
      u += nv;
      ++pvidx;
    };
    auto commit = [&](int b) {
      if (ok && elect_one()) umma_commit(bar(b));
      __syncwarp();
    };
    long long x = A0;
    for (int s = s_first; x < A1; ++s) {
      const SeqInfo si = seq_info(lens[s], p.max_nc);
      const long long seg_end = min(A1, tiles[s + 1]);
      const int j0 = static_cast<int>(x - tiles[s]);
      const int j1 = static_cast<int>(seg_end - tiles[s]);
      wait(B_QFULL, quse & 1, 56);
      ++quse;
      issue_s();
      if (j1 - j0 == 1) commit(B_QEMPTY);
      for (int j = j0; j < j1; ++j) {
        if (j + 1 < j1) {
          issue_s();
          if (j + 2 == j1) commit(B_QEMPTY);
        }
        issue_pv(j == j0, j < si.nct ? min(kKeyTile, si.nc - j * kKeyTile)
                          : p.chunk.q_start != nullptr ? kWin : min(si.L, kWin));
      }
      commit(B_OFULL);
      ++nseg;
      x = seg_end;
    }
    if (elect_one()) umma_commit(bar(B_DRAIN));
    __syncwarp();
    mbar_wait_warp(bar(B_DRAIN), 0, abort_flag, kWaitLimitNs, 57);
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    const int sw = warp - kProducers - 1;    // 0..7
    const int half = sw >> 2;                // heads [32 half, 32 half + 32)
    const int wq = warp & 3;                 // TMEM lane quadrant
    const int key = wq * 32 + lane;          // key row of S^T / value column of O^T
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 32 * half;
    float* mrow = reinterpret_cast<float*>(smem + kSmemM) + 64 * sw;   // m | factors, by head
    float* smax = reinterpret_cast<float*>(smem + kSmemMax) + 128 * half;
    float* ssum = reinterpret_cast<float*>(smem + kSmemSum) + 128 * half;
    volatile int* flag = reinterpret_cast<volatile int*>(smem + kSmemFlag) + 4 * half;
    uint32_t sidx = 0, pvidx = 0, nseg = 0;
    // A failed wait leaves `ok` false and the loops running (without waiting),
    // so that the four warps of a half keep meeting at their barrier.
    bool ok = true;
    const float sc = p.scale_log2;
    long long x = A0;
    for (int s = s_first; x < A1; ++s) {
      const SeqInfo si = seq_info(lens[s], p.max_nc);
      const long long seg_end = min(A1, tiles[s + 1]);
      const int j0 = static_cast<int>(x - tiles[s]);
      const int j1 = static_cast<int>(seg_end - tiles[s]);
      float m = -INFINITY;                   // of head 32 half + lane
      float lsum[32];                        // of this key lane, by head
#pragma unroll
      for (int h = 0; h < 32; ++h) lsum[h] = 0.f;
      for (int j = j0; j < j1; ++j) {
        const uint32_t buf = sidx & 1;
        if (ok)
          ok = mbar_wait_warp(bar(B_SFULL + buf), (sidx >> 1) & 1, abort_flag, kWaitLimitNs, 60);
        tc_fence_after();
        uint32_t r[32];
        tmem_ld32(tl + (buf ? kTmemS1 : kTmemS0), r);
        tmem_wait_ld_dep32(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SFREE + buf));
        ++sidx;
        bool valid;
        if (j < si.nct) valid = j * kKeyTile + key < si.nc;
        else if (p.chunk.q_start != nullptr) valid = key >= kWin - si.L;   // positions >= 0
        else valid = (si.L >= kWin) || (key < si.L);

        // d = scale s - m by head; does any pass the bound?
        float d[32];
        bool over = j == j0;
        if (j > j0) {
          float top = -INFINITY;
#pragma unroll
          for (int h4 = 0; h4 < 8; ++h4) {
            const float4 mm = *reinterpret_cast<const float4*>(mrow + 4 * h4);
            const float mv[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int h = 4 * h4 + q;
              d[h] = fmaf(__uint_as_float(r[h]), sc, -mv[q]);
              top = fmaxf(top, d[h]);
            }
          }
          over = valid && top > kTau;
        }
        over = __any_sync(0xffffffffu, over);
        volatile int* fl = flag + 8 * (sidx & 1);
        if (lane == 0) fl[wq] = over ? 1 : 0;
        named_bar_sync(1 + half, 128);
        bool resc = false;
        if ((fl[0] | fl[1] | fl[2] | fl[3]) != 0) {
          // maximum over the keys of the tile, by head: lane h keeps head h's
          float mine = -INFINITY;
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            const float v = redux_max(valid ? __uint_as_float(r[h]) : -INFINITY);
            if (lane == h) mine = v;
          }
          smax[32 * wq + lane] = mine;
          named_bar_sync(1 + half, 128);
          const float tm = sc * fmaxf(fmaxf(smax[lane], smax[32 + lane]),
                                      fmaxf(smax[64 + lane], smax[96 + lane]));
          float alpha = 1.f;
          if (tm > m + kTau) {
            alpha = m == -INFINITY ? 0.f : ex2_approx(m - tm);
            m = tm;
          }
          resc = __any_sync(0xffffffffu, alpha != 1.f) && j > j0;
          mrow[lane] = m == -INFINITY ? 0.f : m;
          mrow[32 + lane] = alpha;
          __syncwarp();
#pragma unroll
          for (int h4 = 0; h4 < 8; ++h4) {
            const float4 mm = *reinterpret_cast<const float4*>(mrow + 4 * h4);
            const float mv[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              d[4 * h4 + q] = fmaf(__uint_as_float(r[4 * h4 + q]), sc, -mv[q]);
          }
          if (resc) {
#pragma unroll
            for (int h = 0; h < 32; ++h) lsum[h] *= mrow[32 + h];
          }
        }
        // P is rounded to bf16 (half a step, 2^-8 of each probability): the MMA takes it with
        // V, in V's type.  The row sums add the 32-bit values.  Outputs are 2.3e-3 from the
        // 64-bit result in place of 1.7e-3, which the rounding of the output alone gives.
        uint32_t pk[16];
#pragma unroll
        for (int h = 0; h < 32; h += 2) {
          // a masked score may be NaN: selected away, not multiplied
          const float e0 = valid ? ex2_approx(d[h]) : 0.f;
          const float e1 = valid ? ex2_approx(d[h + 1]) : 0.f;
          lsum[h] += e0;
          lsum[h + 1] += e1;
          pk[h / 2] = pack_bf16x2(e0, e1);
        }
        // P^T and O^T are free once the previous tile's P.V is done
        if (ok)
          ok = mbar_wait_warp(bar(B_PFREE), (pvidx & 1) ^ 1, abort_flag, kWaitLimitNs, 61);
        tc_fence_after();
        if (resc) {   // rarely: this quadrant's value columns of these heads
#pragma unroll 1
          for (int c = 0; c < nv; ++c) {
            uint32_t o[32];
            tmem_ld32(tl + kTmemO + 64 * c, o);
            tmem_wait_ld_dep32(o);
#pragma unroll
            for (int h = 0; h < 32; ++h)
              o[h] = __float_as_uint(__uint_as_float(o[h]) * mrow[32 + h]);
            tmem_st32(tl + kTmemO + 64 * c, o);
          }
          tmem_wait_st();
        }
        uint8_t* pt = smem + kSmemPT;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(pt + sw128_offset(key, 4 * half + c)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL));
        ++pvidx;
      }
      // ---------------------------------------------------------- end of the segment
      const bool direct = j0 == 0 && seg_end == tiles[s + 1];   // the whole query is here
      const float lw = lanes_sum32(lsum);
      ssum[32 * wq + lane] = lw;
      named_bar_sync(1 + half, 128);
      const float l = ssum[lane] + ssum[32 + lane] + ssum[64 + lane] + ssum[96 + lane];
      mrow[32 + lane] = l > 0.f ? 1.f / l : 0.f;
      __syncwarp();
      named_bar_sync(1 + half, 128);   // ssum is written again by the next segment
      // The output (gate O / l of a whole query) or the partial O / l, in a short loop: this
      // code runs once a segment, and much of what it costs is its way into the instruction
      // cache.  A chunk of 16 heads x 32 value columns goes through this warp's 2 KB of the
      // P^T buffer: from TMEM a thread has one column of many heads, in global memory it
      // takes 4 columns of one head, 64 bytes in a row for 8 lanes (single columns took
      // 4.9 us a query, and 2.8 us a partial).  The gate comes straight from L2, one step
      // ahead; through the ring it kept the next query's tiles out of two stages (512
      // sequences at 300 tokens 71.6 -> 66.3 us, one 11.6 -> 10.8 us).
      // (opaque: else the addresses are computed ahead of the tiles and more is spilled, 67.1
      // us in place of 66.2)
      int ln = lane, sq = s;
      asm volatile("" : "+r"(ln), "+r"(sq));
      const size_t slot = static_cast<size_t>(vcta) + sq;
      sq += first;
      const int h0 = 32 * half + (ln >> 3);        // heads h0 + 16 hb + 4 q
      const size_t at = (static_cast<size_t>(sq) * kHeads + h0) * kDim + 128 * cg + 32 * wq +
                        4 * (ln & 7);
      if (!direct && wq == 0) {
        p.ws_ml[slot * 128 + 32 * half + ln] = m;
        p.ws_ml[slot * 128 + 64 + 32 * half + ln] = l;
      }
      float* stage = reinterpret_cast<float*>(smem + kSmemPT) + 512 * sw;
      float inv[8];                      // 1 / l of heads (lane >> 3) + 4 t of this half
#pragma unroll
      for (int t = 0; t < 8; ++t) inv[t] = mrow[32 + (ln >> 3) + 4 * t];
      // chunk hb of the 32 heads, from dst
      auto chunk = [&](const uint32_t(&o)[32], int hb, float* dst, float4(&v)[4]) {
#pragma unroll
        for (int h = 0; h < 16; ++h) dst[32 * h + ln] = __uint_as_float(o[16 * hb + h]);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 w = reinterpret_cast<const float4*>(dst)[32 * q + ln];
          const float f = inv[4 * hb + q];
          v[q] = make_float4(w.x * f, w.y * f, w.z * f, w.w * f);
        }
        __syncwarp();
      };
      if (direct) {
        uint2 gv[8];
        auto load_gate = [&](int c, int t) {
          gv[t] = __ldg(reinterpret_cast<const uint2*>(p.g + at + 128 * c + 4 * t * kDim));
        };
#pragma unroll
        for (int t = 0; t < 8; ++t) load_gate(0, t);
        if (ok) ok = mbar_wait_warp(bar(B_OFULL), nseg & 1, abort_flag, kWaitLimitNs, 62);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < nv; ++c) {   // value columns 128 (cg + c) + key
          uint32_t o[32];
          tmem_ld32(tl + kTmemO + 64 * c, o);
          tmem_wait_ld_dep32(o);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            float4 v[4];
            chunk(o, hb, stage, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint2 gq = gv[4 * hb + q];
              *reinterpret_cast<uint2*>(p.out + at + 128 * c + (16 * hb + 4 * q) * kDim) =
                  make_uint2(pack_bf16x2(gate32(v[q].x, bf16lo_to_f32(gq.x)),
                                         gate32(v[q].y, bf16hi_to_f32(gq.x))),
                             pack_bf16x2(gate32(v[q].z, bf16lo_to_f32(gq.y)),
                                         gate32(v[q].w, bf16hi_to_f32(gq.y))));
              if (c + 1 < nv) load_gate(c + 1, 4 * hb + q);
            }
          }
        }
      } else {
        if (ok) ok = mbar_wait_warp(bar(B_OFULL), nseg & 1, abort_flag, kWaitLimitNs, 62);
        tc_fence_after();
        float* wo = p.ws_o + slot * kHeads * kDim;
        float* keep = reinterpret_cast<float*>(smem + merge_data(parts)) + 512 * nk * part;
#pragma unroll 1
        for (int c = 0; c < nv; ++c) {
          uint32_t o[32];
          tmem_ld32(tl + kTmemO + 64 * c, o);
          tmem_wait_ld_dep32(o);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const int k = 16 * (cg + c) + 4 * (2 * half + hb) + wq;
            const bool here = kept && k >= k0 && k < k0 + nk;
            float* dst = here ? keep + 512 * (k - k0) : stage;
            float4 v[4];
            chunk(o, hb, dst, v);
            float4* to = reinterpret_cast<float4*>(here ? dst : wo + 512 * k) + ln;
#pragma unroll
            for (int q = 0; q < 4; ++q) to[32 * q] = v[q];
          }
        }
      }
      // Everybody has left the P^T buffer, and a partial is written: one arrival for the
      // CTAs that share the query.
      named_bar_sync(3, 32 * kSoftWarps);
      if (!direct && sw == 0 && lane == 0)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(
                         p.arrived + (own ? cta - (part << lcs) : owner(tiles[s])))
                     : "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_OFREE));
      ++nseg;
      x = seg_end;
    }
  }

  }  // A0 < A1
  if (threadIdx.x == 0) {
    abort_drain(abort_flag);
    // whoever follows this kernel may count on the one before it being done, too
    if (p.only_window) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  __syncthreads();
  if (warp == kProducers) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }

  // ---------------------------------------------------------------- merge, head mix
  // The launch is cooperative: CTAs wait for one another.  Grid barrier of the
  // head mix: a counter that is never reset, each barrier adding exactly
  // gridDim.x, as in decode.cuh.
  __shared__ unsigned long long bar_target;
  __shared__ int bar_done;
  auto grid_arrive = [&]() {
    __syncthreads();
    if (threadIdx.x == 0) {
      const unsigned long long G = gridDim.x;
      unsigned long long old;
      asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;"
                   : "=l"(old)
                   : "l"(p.gsync)
                   : "memory");
      bar_target = (old / G + 1) * G;
      bar_done = (old + 1 == bar_target) ? 1 : 0;
    }
  };
  auto grid_wait = [&]() {
    if (threadIdx.x == 0 && !bar_done) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1;; ++i) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p.gsync) : "memory");
        if (v >= bar_target) break;
        if ((i & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
          record_error(DEVERR_TIMEOUT, 72);
          break;
        }
      }
      bar_done = 1;
    }
    __syncthreads();
  };
  uint32_t merges = 0;   // phase of B_MERGE
  if (own ? parts > 1 : !whole && A0 < A1) {
    // of an even cut the first and the last query may be shared with others
    const int sa = own ? mine : find_seq(tiles, p.S, A0);
    const int sb = own ? mine : find_seq(tiles, p.S, A1 - 1);
#pragma unroll 1
    for (int s = sa; s <= sb; s += max(sb - sa, 1)) {
      const int c0 = own ? cta - (part << lcs) : owner(tiles[s]);   // first CTA of the query
      const int n = own ? parts : owner(tiles[s + 1] - 1) - c0 + 1;
      if (n > 1)
        merge_query(p, first + s, static_cast<size_t>(own ? vcta - part : c0) + s, p.arrived + c0,
                    own ? part : cta - c0, n, cg, nv, kept, smem, sbase, bar(B_MERGE), merges,
                    abort_flag, warp, lane);
    }
  }
  if (p.vha_rank > 0) {
    grid_arrive();  // this CTA's rows of out are written
    grid_wait();
    float* fd = reinterpret_cast<float*>(smem + kSmemQ);   // [64][r8]
    float* fu = fd + kHeads * kHeads;
    uint16_t* mix = reinterpret_cast<uint16_t*>(fu + kHeads * kHeads);   // 1 KB per warp
    decode::vha_load_factors<kThreads>(p, fd, fu);
    __syncthreads();
    p.out += static_cast<size_t>(first) * kHeads * kDim;
    decode::vha_mix_columns<kThreads>(p, fd, fu, mix + warp * kHeads * 8, warp, lane);
  }
}

}  // namespace pdecode
}  // namespace hca
