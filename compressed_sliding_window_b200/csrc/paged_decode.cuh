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
// Work split.  The key tiles of all queries laid end to end are cut into one
// contiguous range per CTA; a query that is whole inside one CTA is written
// straight out, the others leave partial results (O / l in fp32, m, l), which
// the CTAs that share the query merge.  When giving each CTA whole queries costs
// at most kWholeTiles tiles more than an even cut, that is done, and nothing is
// merged (which takes about as long).
#pragma once

#include "decode.cuh"
#include "hca_ptx.cuh"

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
constexpr int kWholeTiles = 3;
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
constexpr int kSmemBytes = kSmemLen + 4 * kInlineSeqs;
constexpr int kSmemAlloc = kSmemBytes + 1024;
static_assert(kSmemAlloc <= 232448 - 1024, "shared memory budget");
static_assert(kStages * kStage == kKeyTile * kDim * 2, "a tile's K or V is one round of the ring");

enum {
  B_QFULL = 0, B_QEMPTY = 1, B_FULL = 2, B_EMPTY = B_FULL + kStages, B_SFULL = B_EMPTY + kStages,
  B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_PFREE = B_PFULL + 1, B_OFULL = B_PFREE + 1,
  B_OFREE = B_OFULL + 1, B_DRAIN = B_OFREE + 1, B_COUNT = B_DRAIN + 1
};
constexpr int kTmemSlot = 8 * B_COUNT;
constexpr int kAbortSlot = kTmemSlot + 4;
static_assert(kAbortSlot + 4 <= 320, "barrier region overflow");

constexpr uint32_t kTmemO = 0, kTmemS0 = 256, kTmemS1 = 320, kTmemCols = 512;

// Workspace (bytes): [slots][64][512] fp32 partial O / l, then [slots][2][64]
// fp32 (m, l) in log2 units; slots = grid + S.
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
  unsigned* arrived;   // [S] arrivals at each query's merge: zero between calls
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
  const int* row_of;   // [S] table row of each query, null: query s has row s
  const int* win_row;  // [S] first window row (positions L-128 .. L-1), null: a ring at 128 s
  const int* count;    // number of queries on the device (at most S), null: S
  int plan_early;      // ctx_len is older than the kernel in front: plan before waiting for it
};

struct Maps {
  CUtensorMap q;    // (64, S*64, 8, 1),  box (64, 64, 8, 1): the whole q of one query
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

// Tile prefix of S queries by one CTA of NT threads, each a run of queries:
// out[i], out[S] = total, and the longest query in *longest.
template <int NT>
__device__ __forceinline__ void plan_tiles(const int* ctx_len, int S, int max_nc, long long* out,
                                           int* lens, int* longest, bool report) {
  __shared__ long long wsum[NT / 32];
  __shared__ int wmax[NT / 32];
  const int per = (S + NT - 1) / NT;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, S), i1 = min(i0 + per, S);
  long long run = 0;
  int most = 0;
  for (int i = i0; i < i1; ++i) {
    const int L = ctx_len[i];
    const int n = tiles_of(L, max_nc, report);
    if (lens != nullptr) lens[i] = L;
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

__global__ void __launch_bounds__(1024)
    plan_kernel(const int* ctx_len, int S, int max_nc, long long* seq_tile, const int* count) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (count != nullptr) S = min(max(*count, 0), S);
  __shared__ int longest;
  plan_tiles<1024>(ctx_len, S, max_nc, seq_tile, nullptr, &longest, true);
  if (threadIdx.x == 0) seq_tile[S + 1] = longest;
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

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}" : "=r"(r));
  return r != 0;
}

// names the destination registers of a finished tcgen05.ld (see tmem_wait_ld_dep32)
__device__ __forceinline__ void reg_dep16(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
               "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
               "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
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

// 1 / (1 + 2^(-x log2 e))
__device__ __forceinline__ float sigmoid32(float x) {
  return __fdividef(1.f, 1.f + ex2_approx(-1.4426950408889634f * x));
}

// How a launch is split, the same in every CTA.
struct Split {
  long long N;   // tiles
  int G;         // CTAs with tiles
  bool whole;    // whole queries per CTA
};

// ---------------------------------------------------------------------------
// Merge of a query whose tiles n CTAs share, by all of them: CTA i of the n
// takes the rows (heads) [64 i / n, 64 (i + 1) / n) of all n partials, once
// all have been written (a counter per query; a CTA waits only for those that
// share its first or last query, and only after its own tiles).  First every
// warp finds the weights w_f = l_f 2^(m_f - M) / L of its rows' splits, lane =
// split; then lane l adds up value columns 128 q + 4 l .. + 3 (a partial row is
// four 16-byte loads a lane, four splits in flight).  With fewer rows than
// warps, several warps share a row's splits and add up through shared memory.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void merge_query(const Params& p, int s, int c0, int n, uint8_t* smem,
                                            int warp, int lane) {
  const int i = static_cast<int>(blockIdx.x) - c0;
  const int h0 = kHeads * i / n, nr = kHeads * (i + 1) / n - h0;
  __shared__ int late;
  if (threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    late = 0;
    for (uint32_t k = 1;; ++k) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.arrived + s) : "memory");
      if (v >= static_cast<unsigned>(n)) break;
      if ((k & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(DEVERR_TIMEOUT, 72);
        late = 1;
        break;
      }
    }
  }
  __syncthreads();
  if (nr > 0 && !late) {
    const int share = nr < kWarps ? kWarps / nr : 1;           // warps per row
    const int part = warp % share, slot0 = warp / share, rows = kWarps / share;
    float* add = reinterpret_cast<float*>(smem + kSmemRing);    // [warps][512]
    float* wt = reinterpret_cast<float*>(smem + kSmemQ);        // [warps][grid]
    float* w = wt + warp * gridDim.x;
    for (int r0 = 0; r0 < nr; r0 += rows) {
      const int r = r0 + slot0;
      const bool mine = slot0 < rows && r < nr;
      const int h = h0 + r;
      const size_t row = static_cast<size_t>(s) * kHeads + h;
      float acc[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) acc[t] = 0.f;
      uint2 gv[4];
      if (mine) {
        const float* ml = p.ws_ml + static_cast<size_t>(c0 + s) * 128 + h;
        const uint2* gp = reinterpret_cast<const uint2*>(p.g + row * kDim + 4 * lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) gv[q] = __ldg(gp + 32 * q);
        float M = -INFINITY, L = 0.f;
        for (int f = lane; f < n; f += 32) {
          const float m = __ldcg(ml + 128 * f);
          w[f] = m;
          M = fmaxf(M, m);
        }
        M = redux_max(M);
        const float mu = M == -INFINITY ? 0.f : M;
        for (int f = lane; f < n; f += 32) {
          const float x = __ldcg(ml + 128 * f + 64) * ex2_approx(w[f] - mu);
          w[f] = x;
          L += x;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        __syncwarp();
        const float inv = 1.f / L;
        const float4* po = reinterpret_cast<const float4*>(
                               p.ws_o + (static_cast<size_t>(c0 + s) * kHeads + h) * kDim) + lane;
#pragma unroll 1
        for (int f0 = part; f0 < n; f0 += 4 * share) {
          float4 x[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int f = min(f0 + u * share, n - 1);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              x[u][q] = __ldcg(po + static_cast<size_t>(f) * (kHeads * kDim / 4) + 32 * q);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int f = f0 + u * share;
            const float wf = f < n ? w[f] * inv : 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[4 * q] = fmaf(wf, x[u][q].x, acc[4 * q]);
              acc[4 * q + 1] = fmaf(wf, x[u][q].y, acc[4 * q + 1]);
              acc[4 * q + 2] = fmaf(wf, x[u][q].z, acc[4 * q + 2]);
              acc[4 * q + 3] = fmaf(wf, x[u][q].w, acc[4 * q + 3]);
            }
          }
        }
      }
      if (share > 1) {   // uniform in the CTA
        __syncthreads();
        if (mine && part > 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(add + warp * kDim + 128 * q + 4 * lane) =
                make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        }
        __syncthreads();
        if (mine && part == 0) {
          for (int v = 1; v < share; ++v) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 x =
                  *reinterpret_cast<const float4*>(add + (warp + v) * kDim + 128 * q + 4 * lane);
              acc[4 * q] += x.x;
              acc[4 * q + 1] += x.y;
              acc[4 * q + 2] += x.z;
              acc[4 * q + 3] += x.w;
            }
          }
        }
      }
      if (mine && part == 0) {
        uint2* op = reinterpret_cast<uint2*>(p.out + row * kDim + 4 * lane);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          op[32 * q] = make_uint2(pack_bf16x2(acc[4 * q] * sigmoid32(bf16lo_to_f32(gv[q].x)),
                                              acc[4 * q + 1] * sigmoid32(bf16hi_to_f32(gv[q].x))),
                                  pack_bf16x2(acc[4 * q + 2] * sigmoid32(bf16lo_to_f32(gv[q].y)),
                                              acc[4 * q + 3] * sigmoid32(bf16hi_to_f32(gv[q].y))));
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
                 : "l"(p.arrived + s)
                 : "memory");
    if (old == 2u * n - 1) p.arrived[s] = 0u;
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
  __shared__ int longest;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
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
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.ck);
    tma_prefetch_desc(&maps.cv);
    tma_prefetch_desc(&maps.wk);
    tma_prefetch_desc(&maps.wv);
  }
  if (warp == kProducers) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  // The plan, here for up to kInlineSeqs queries.  The kernel may have been
  // launched while the one in front of it still runs: it waits before it reads
  // anything that one writes.
  const bool inl = p0.S <= kInlineSeqs;
  if (inl && p.plan_early)
    plan_tiles<kThreads>(p.ctx_len, p.S, p.max_nc, sT, sL, &longest, blockIdx.x == 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.count != nullptr) p.S = min(max(*p.count, 0), p0.S);
  if (inl && !p.plan_early)
    plan_tiles<kThreads>(p.ctx_len, p.S, p.max_nc, sT, sL, &longest, blockIdx.x == 0);
  if (!inl) {
    if (threadIdx.x == 0) longest = static_cast<int>(p.seq_tile[p.S + 1]);
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long* tiles = inl ? sT : p.seq_tile;
  const int* lens = inl ? sL : p.ctx_len;
  Split sp;
  sp.N = tiles[p.S];
  sp.G = static_cast<int>(min(static_cast<long long>(gridDim.x), max(sp.N, 1LL)));
  const int per = (p.S + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  sp.whole = static_cast<long long>(longest) * per <=
             decode::div_nn(sp.N + gridDim.x - 1, gridDim.x) + kWholeTiles;
  long long A0 = 0, A1 = 0;
  if (sp.whole) {
    A0 = tiles[decode::div_nn(static_cast<long long>(p.S) * blockIdx.x, gridDim.x)];
    A1 = tiles[decode::div_nn(static_cast<long long>(p.S) * (blockIdx.x + 1), gridDim.x)];
  } else if (static_cast<int>(blockIdx.x) < sp.G) {
    A0 = decode::div_nn(sp.N * blockIdx.x, sp.G);
    A1 = decode::div_nn(sp.N * (blockIdx.x + 1), sp.G);
  }
  if (A0 < A1) {  // uniform across the CTA

  // Segments: maximal runs of this CTA's tiles inside one query.
  const int s_first = find_seq(tiles, p.S, A0);

  if (warp < kProducers) {
    // ------------------------------------------------------------ producers
    // Two warps take turns at the stages; lane b (+ boxes for the second slab)
    // loads box b of a stage.
    const int me = warp;
    const int boxes = kKeyTile >> p.page_shift;
    const int bx = lane & (boxes - 1), slab = lane / boxes;
    const uint32_t boff = slab * kSlab + bx * (kSlab / boxes);
    uint32_t u = 0, quse = 0;   // u: rounds of the ring
    bool ok = true;
    // The eight slabs of a tile: entries of the page `pg` of this lane's box, or
    // (pg < 0) the window rows from y on
    auto load = [&](const CUtensorMap* map, int pg, int y) {
#pragma unroll
      for (int i = 0; i < kStages / kProducers; ++i) {
        const int st = kProducers * i + me;
        if (lane == 0) {
          ok = ok && mbar_wait(bar(B_EMPTY + st), (u & 1) ^ 1, abort_flag, kWaitLimitNs, 40);
          if (ok) mbar_expect_tx(bar(B_FULL + st), kStage);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        __syncwarp();
        if (ok && pg >= 0 && slab < 2)
          decode::tma_load_4d_dec(sRing + st * kStage + boff, map, bar(B_FULL + st), 0, 0,
                                  2 * st + slab, pg);
        else if (ok && pg < 0 && lane == 0)
          decode::tma_load_4d_dec(sRing + st * kStage, map, bar(B_FULL + st), 0, y, 2 * st, 0);
      }
      ++u;
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
            decode::tma_load_4d_dec(sQ, &maps.q, bar(B_QFULL), 0, s * kHeads, 0, 0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      ++quse;
      const int* prow = p.table + (p.row_of != nullptr ? p.row_of[s] : s) * p.table_ld;
      const int win = p.win_row != nullptr ? p.win_row[s] : s * kWin;
      auto page_of = [&](int j) -> int {
        return j < si.nct ? box_page(p, prow, si.nc, j, bx) : -1;
      };
      int pg = page_of(j0), pg1 = j0 + 1 < j1 ? page_of(j0 + 1) : -1;
      load(pg >= 0 ? &maps.ck : &maps.wk, pg, win);
      for (int j = j0; j < j1 && ok; ++j) {
        const int pg2 = j + 2 < j1 ? page_of(j + 2) : -1;   // needed one tile later
        if (j + 1 < j1) load(pg1 >= 0 ? &maps.ck : &maps.wk, pg1, win);
        load(pg >= 0 ? &maps.cv : &maps.wv, pg, win);
        pg = pg1;
        pg1 = pg2;
      }
      x = seg_end;
    }
  } else if (warp == kProducers) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp waits and walks the tiles; one elected lane issues.  Under
    // a branch on elect.sync in warp-uniform code the descriptors stay in
    // uniform registers: 49 cycles an MMA of 128 x 64 x 16 (what its operands
    // take from shared memory) against 115 under a branch on the lane number.
    // `ok` is uniform; after a failed wait the loops run on without waiting.
    bool ok = true;
    uint32_t ring = 0, quse = 0, sidx = 0, pvidx = 0, nseg = 0;   // ring: rounds
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
#pragma unroll 1
      for (int st = 0; st < kStages; ++st) {
        wait(B_FULL + st, ring & 1, 51);
        tc_fence_after();
        const uint64_t ad = sdesc_sw128(sRing + st * kStage, 16, 1024);
        const uint64_t bd = sdesc_sw128(sQ + st * 2 * kQSlab, 16, 1024);
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)   // 16 channels each: 32 bytes on, or the next slab
            umma_bf16(dS, ad + 2 * (k & 3) + (k >> 2) * (kSlab >> 4),
                      bd + 2 * (k & 3) + (k >> 2) * (kQSlab >> 4), idesc_s, (st | k) != 0);
          umma_commit(bar(B_EMPTY + st));
          if (st == kStages - 1) umma_commit(bar(B_SFULL + buf));
        }
        __syncwarp();
      }
      ++ring;
      ++sidx;
    };
    auto issue_pv = [&](bool first, int valid) {
      wait(B_PFULL, pvidx & 1, 52);
      if (first) wait(B_OFREE, (nseg & 1) ^ 1, 53);
      const int ksteps = (valid + 15) >> 4;
#pragma unroll 1
      for (int c = 0; c < kStages; ++c) {   // 128 value columns each
        wait(B_FULL + c, ring & 1, 54);
        if (ok && (valid & 15) != 0) {
          clear_rows(smem + kSmemRing + c * kStage, valid, lane);
          fence_proxy_async_smem();               // read next by the tensor core
        }
        __syncwarp();
        tc_fence_after();
        const uint64_t ad = sdesc_sw128(sRing + c * kStage, kSlab, 1024);
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
          umma_commit(bar(B_EMPTY + c));
          if (c == kStages - 1) umma_commit(bar(B_PFREE));
        }
        __syncwarp();
      }
      ++ring;
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
                          : p.win_row != nullptr ? kWin : min(si.L, kWin));
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
        else if (p.win_row != nullptr) valid = key >= kWin - si.L;   // positions >= 0
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
          for (int c = 0; c < 4; ++c) {
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
      const size_t hrow = static_cast<size_t>(s) * kHeads + 32 * half;
      const float lw = lanes_sum32(lsum);
      ssum[32 * wq + lane] = lw;
      named_bar_sync(1 + half, 128);
      const float l = ssum[lane] + ssum[32 + lane] + ssum[64 + lane] + ssum[96 + lane];
      mrow[32 + lane] = l > 0.f ? 1.f / l : 0.f;
      __syncwarp();
      named_bar_sync(1 + half, 128);   // ssum is written again by the next segment
      // 16 heads of 128 value columns at a time, in a short loop: this code runs
      // once a segment, and what it costs is above all its way into the
      // instruction cache.
      if (direct) {
        // gate: 16-byte chunk lane % 4 of rows (heads) lane / 4 and + 8, value columns 128 c + 32 wq
        const size_t goff = (hrow + (lane >> 2)) * kDim + 32 * wq + 8 * (lane & 3);
        // this warp's 1 KB of the P^T buffer: [16 heads][32 value columns] bf16
        uint8_t* stage = smem + kSmemPT + 1024 * sw;
        uint4 ga = __ldg(reinterpret_cast<const uint4*>(p.g + goff));
        uint4 gb = __ldg(reinterpret_cast<const uint4*>(p.g + goff + 8 * kDim));
        if (ok) ok = mbar_wait_warp(bar(B_OFULL), nseg & 1, abort_flag, kWaitLimitNs, 62);
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {      // heads 16 (i & 1), value columns 128 (i >> 1)
          uint32_t o[16];
          tmem_ld16(tl + kTmemO + 64 * (i >> 1) + 16 * (i & 1), o);
          *reinterpret_cast<uint4*>(stage + 16 * lane) = ga;
          *reinterpret_cast<uint4*>(stage + 512 + 16 * lane) = gb;
          const size_t at = goff + 16 * (i & 1) * kDim + 128 * (i >> 1);
          if (i < 7) {
            const size_t nx = goff + 16 * ((i + 1) & 1) * kDim + 128 * ((i + 1) >> 1);
            ga = __ldg(reinterpret_cast<const uint4*>(p.g + nx));
            gb = __ldg(reinterpret_cast<const uint4*>(p.g + nx + 8 * kDim));
          }
          tmem_wait_ld();
          reg_dep16(o);
          __syncwarp();
          const float* inv = mrow + 32 + 16 * (i & 1);
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            uint16_t* e = reinterpret_cast<uint16_t*>(stage + 64 * h) + lane;
            const float gate = sigmoid32(__uint_as_float(static_cast<uint32_t>(*e) << 16));
            const __nv_bfloat16 v = __float2bfloat16_rn(__uint_as_float(o[h]) * inv[h] * gate);
            *e = *reinterpret_cast<const uint16_t*>(&v);
          }
          __syncwarp();
          *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(stage + 16 * lane);
          *reinterpret_cast<uint4*>(p.out + at + 8 * kDim) =
              *reinterpret_cast<const uint4*>(stage + 512 + 16 * lane);
          __syncwarp();
        }
        named_bar_sync(3, 32 * kSoftWarps);   // the next query's P^T overwrites the stages
      } else {
        const size_t slot = static_cast<size_t>(blockIdx.x) + s;
        float* wo = p.ws_o + (slot * kHeads + 32 * half) * kDim + key;
        if (wq == 0) {
          p.ws_ml[slot * 128 + 32 * half + lane] = m;
          p.ws_ml[slot * 128 + 64 + 32 * half + lane] = l;
        }
        if (ok) ok = mbar_wait_warp(bar(B_OFULL), nseg & 1, abort_flag, kWaitLimitNs, 62);
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          uint32_t o[16];
          tmem_ld16(tl + kTmemO + 64 * (i >> 1) + 16 * (i & 1), o);
          tmem_wait_ld();
          reg_dep16(o);
          const float* inv = mrow + 32 + 16 * (i & 1);
          float* dst = wo + 16 * (i & 1) * kDim + 128 * (i >> 1);
#pragma unroll
          for (int h = 0; h < 16; ++h) dst[h * kDim] = __uint_as_float(o[h]) * inv[h];
        }
        // the partial is written: one arrival for the CTAs that share the query
        named_bar_sync(3, 32 * kSoftWarps);
        if (sw == 0 && lane == 0)
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.arrived + s) : "memory");
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_OFREE));
      ++nseg;
      x = seg_end;
    }
  }

  }  // A0 < A1
  if (threadIdx.x == 0) abort_drain(abort_flag);
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
  if (!sp.whole && A0 < A1) {
    auto owner = [&](long long x) -> int {   // CTA of tile x
      return static_cast<int>(decode::div_nn((x + 1) * sp.G + sp.N - 1, sp.N)) - 1;
    };
    // the first and the last query of this CTA may be shared with others
    const int sa = find_seq(tiles, p.S, A0), sb = find_seq(tiles, p.S, A1 - 1);
    for (int s = sa; s <= sb; s += max(sb - sa, 1)) {
      const int c0 = owner(tiles[s]), n = owner(tiles[s + 1] - 1) - c0 + 1;
      if (n > 1) merge_query(p, s, c0, n, smem, warp, lane);
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
    decode::vha_mix_columns<kThreads>(p, fd, fu, mix + warp * kHeads * 8, warp, lane);
  }
}

}  // namespace pdecode
}  // namespace hca
