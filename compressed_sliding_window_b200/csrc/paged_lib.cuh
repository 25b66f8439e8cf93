// Host side of the paged cache: argument checks, maps and launches of the
// calls that include/hca.h declares under "Paged cache".  Part of the one
// translation unit of hca_lib.cu, whose helpers it uses.
#pragma once

namespace {

// log2 of a page size the kernels take (16, 32, 64 or 128 entries), or -1
int page_shift_of(int page_size) {
  for (int s = 4; s <= 7; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Checks what every call on a paged cache shares and fills `c`.
hca_status_t paged_cache(hca::paged::Cache& c, const hca_paged_cache_t* p, int S, bool ring_scores) {
  if (p == nullptr) return HCA_ERR_INVALID_ARG;
  if (p->num_pages < 0 || p->max_pages < 0 || p->table_stride < p->max_pages)
    return HCA_ERR_INVALID_ARG;
  const int shift = page_shift_of(p->page_size);
  if (shift < 0) return HCA_ERR_UNSUPPORTED;
  if (p->wk == nullptr || p->wv == nullptr || !aligned16(p->wk) || !aligned16(p->wv) ||
      (ring_scores && p->ws == nullptr))
    return HCA_ERR_INVALID_ARG;
  if (p->num_pages > 0 && (p->ck == nullptr || p->cv == nullptr || !aligned16(p->ck) ||
                           !aligned16(p->cv)))
    return HCA_ERR_INVALID_ARG;
  if (p->max_pages > 0 && (p->page_table == nullptr || !aligned4(p->page_table)))
    return HCA_ERR_INVALID_ARG;
  // entry numbers and ring rows are 32-bit
  if (static_cast<long long>(p->max_pages) * p->page_size > 0x7fffffffLL / HCA_BLOCK ||
      S > 0x7fffffff / HCA_BLOCK)
    return HCA_ERR_UNSUPPORTED;
  c.wk = p->wk;
  c.wv = p->wv;
  c.ws = p->ws;
  c.ck = p->ck;
  c.cv = p->cv;
  c.table = p->page_table;
  c.table_ld = p->table_stride;
  c.max_pages = p->max_pages;
  c.num_pages = p->num_pages;
  c.page_shift = shift;
  return HCA_OK;
}

hca_status_t chunk_args(hca::paged::Chunk& c, const hca_bf16* k_new, const hca_bf16* v_new,
                        const hca_bf16* s_new, const int32_t* q_start, const int32_t* ctx_len,
                        int S, int N) {
  if (S < 1 || N < 0 || k_new == nullptr || v_new == nullptr || s_new == nullptr ||
      ctx_len == nullptr || !aligned16(k_new) || !aligned16(v_new) || !aligned4(ctx_len) ||
      !aligned4(q_start))
    return HCA_ERR_INVALID_ARG;
  c = {k_new, v_new, s_new, q_start, ctx_len, S, N};
  return HCA_OK;
}

// A launch that may begin while the kernel before it on the stream still runs
// (it waits for its results inside).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream,
                          const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// grid.x of entries_kernel: the units of all sequences
template <bool kRaw>
long long entry_units(int S, int N) {
  return N / hca::paged::kBlk + static_cast<long long>(hca::paged::kUnitsExtra<kRaw>) * S;
}

// The zero-filled head of a workspace, the same for every call: grid barrier,
// counters of the merges.
constexpr int kMaxGrid = 960;
constexpr size_t kHeadBytes = 256 + 4 * kMaxGrid;
static_assert(kHeadBytes % 256 == 0, "what follows is aligned");

// One query at a time, split over the keys: the rest of `prm`, maps, launches.
hca_status_t paged_attend(const hca::paged::Cache& c, const hca_bf16* q, const hca_bf16* g,
                          hca_bf16* out, const hca_bf16* wk, const hca_bf16* wv,
                          uint64_t win_rows, hca::pdecode::Params& prm, uint8_t* ws,
                          cudaStream_t stream) {
  namespace D = hca::pdecode;
  const int sms = device_sms();
  if (sms <= 0) return HCA_ERR_CUDA;
  const int slots = sms + prm.S;
  prm.max_nc = c.num_pages > 0 ? c.max_pages << c.page_shift : 0;
  prm.gsync = reinterpret_cast<unsigned long long*>(ws);
  if (sms > kMaxGrid) return HCA_ERR_UNSUPPORTED;
  prm.arrived = reinterpret_cast<unsigned*>(ws + 256);
  ws += kHeadBytes;
  prm.ws_o = reinterpret_cast<float*>(ws);
  prm.ws_ml = reinterpret_cast<float*>(ws + D::ws_o_bytes(slots));
  prm.seq_tile = reinterpret_cast<long long*>(ws + align256(D::ws_bytes(slots)));
  prm.g = g;
  prm.out = out;
  prm.table = c.table;
  prm.table_ld = c.table_ld;
  prm.num_pages = c.num_pages;
  prm.page_shift = c.page_shift;
  D::Maps maps;
  const uint32_t box = 1u << c.page_shift;
  bool ok = make_map4(&maps.q, q, static_cast<uint64_t>(prm.S) * HCA_NUM_HEADS, 1, 64, 8) &&
            make_map4(&maps.g, g, static_cast<uint64_t>(prm.S) * HCA_NUM_HEADS, 1, 64, 2) &&
            make_map4(&maps.wk, wk, win_rows, 1, 128, 2) &&
            make_map4(&maps.wv, wv, win_rows, 1, 128, 2);
  if (ok && c.num_pages > 0) {
    ok = make_map4(&maps.ck, c.ck, box, c.num_pages, box, 1) &&
         make_map4(&maps.cv, c.cv, box, c.num_pages, box, 1);
  } else if (ok) {   // no entry can be visible: never used
    maps.ck = maps.wk;
    maps.cv = maps.wv;
  }
  if (!ok) return HCA_ERR_CUDA;
  if (once_per_device<2>([] {
        return cudaFuncSetAttribute(D::paged_decode_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, D::kSmemAlloc);
      }) != cudaSuccess)
    return HCA_ERR_CUDA;
  if (prm.S > D::kInlineSeqs) {
    D::plan_kernel<<<1, 1024, 0, stream>>>(prm);
    if (cudaGetLastError() != cudaSuccess) return HCA_ERR_CUDA;
  }
  // cooperative: CTAs that share a query wait for one another
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(D::kThreads);
  cfg.dynamicSmemBytes = D::kSmemAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, D::paged_decode_kernel, maps, prm) != cudaSuccess)
    return HCA_ERR_CUDA;
  return launch_status();
}

// What an attention call shares beside its cache.
hca_status_t attend_args(const hca_bf16* q, const hca_bf16* g, const hca_bf16* out, int H,
                         float scale, const hca_bf16* vha_down, const hca_bf16* vha_up,
                         int vha_rank, const void* ws) {
  if (H != HCA_NUM_HEADS) return HCA_ERR_UNSUPPORTED;
  if (!scale_ok(scale) || q == nullptr || g == nullptr || out == nullptr || ws == nullptr)
    return HCA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(g) || !aligned16(out)) return HCA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return HCA_ERR_INVALID_ARG;
  if (vha_rank < 0 || vha_rank > HCA_NUM_HEADS ||
      (vha_rank > 0 && (vha_down == nullptr || vha_up == nullptr)))
    return HCA_ERR_INVALID_ARG;
  return HCA_OK;
}

// Does `out` [rows, 64, 512] share memory with q or g?  (CTAs that split a query read both
// while others already write.)
bool out_overlaps(const hca_bf16* out, const hca_bf16* q, const hca_bf16* g, long long rows) {
  const uintptr_t bytes = static_cast<uintptr_t>(rows) * HCA_NUM_HEADS * HCA_HEAD_DIM * 2;
  const uintptr_t o = reinterpret_cast<uintptr_t>(out);
  for (const hca_bf16* in : {q, g}) {
    const uintptr_t i = reinterpret_cast<uintptr_t>(in);
    if (o < i + bytes && i < o + bytes) return true;
  }
  return false;
}

// Which form the attention of a chunk takes.  The split form reads a sequence's entries
// once per token and works on 64 rows at a time, on every SM whatever N is; the items form
// reads them once per four tokens with 256-row tiles, an item a cluster at a time (33 of
// them).  GPU time of one sequence, split and items: 44 tokens at 20000 24.6 and 27.8 us, at
// 1M 100 and 122; 64 tokens at 20000 24.8 and 28.2, at 131072 42.2 and 37.5, at 1M 140 and
// 123: up to 56 split.  Of many sequences with a token or two the items fill more than one
// round of the clusters: 32 x 2 at 40000 27.4 and 31.2, at 131072 49.0 and 45.6; 64 x 1 at
// 20000 27.5 and 41.9, at 131072 58.5 and 72.3; but 24 x 4 at 40000 33.0 and 30.3.  With two
// rounds the limit is half of the 148 SMs: up to there the split form has two CTAs for each
// query, which share its value columns.  (Where long contexts would rather have the items, as
// 32 x 2 at 131072 by 7 %, the host cannot tell: the lengths are on the device.)
constexpr int kSplitTokens = 56;
constexpr int kSplitTwoRounds = 148 / 2;
constexpr int kSplitMost = 127;      // with more than two rounds
static_assert(kSplitMost <= 128, "a block that the chunk completes must not become visible in it");
// room for the items of N tokens: the sum of ceil(n / 4) over S sequences
int item_room(int S, int N) { return static_cast<int>((static_cast<long long>(N) + 3LL * S) / 4); }
bool split_form(int S, int N, int clusters) {
  if (N <= kSplitTokens) return true;
  const int items = item_room(S, N);
  return (N <= kSplitTwoRounds && items > clusters) || (N <= kSplitMost && items > 2 * clusters);
}
constexpr int kMaxChunkSeqs = 4096;

struct PagedPrefillLayout {
  bool split;   // one query at a time, split over the keys; else four positions at a time
  int items;    // room in the item list
  size_t list, tail16, tail, scratch, count, raw_k, raw_v, total;
};

PagedPrefillLayout paged_prefill_layout(int S, int N, int clusters, bool split) {
  PagedPrefillLayout L = {};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.split = split;
  L.items = item_room(S, N);
  // the split form's workspace is at its start, and its head is nobody else's
  take(L.split ? hca_paged_decode_workspace_size(N) : kHeadBytes);
  if (!L.split) {
    L.count = take(4);
    L.list = take(static_cast<size_t>(L.items) * 16);
    L.tail16 = take(static_cast<size_t>(S) * 4);
    L.tail = take(static_cast<size_t>(S) * 16 * HCA_HEAD_DIM * 2);
    L.scratch = take(static_cast<size_t>(clusters) * hca::prefill3::kScratchPerCluster);
  }
  const size_t raw = (static_cast<size_t>(N) + static_cast<size_t>(hca::paged::kPad) * S) *
                     HCA_HEAD_DIM * 2;
  L.raw_k = take(raw);
  L.raw_v = take(raw);
  L.total = off;
  return L;
}

// Four positions at a time: the prefill kernel over the item list in `w`.
hca_status_t paged_items(const hca::paged::Cache& c, const PagedPrefillLayout& L, uint8_t* w,
                         const hca_bf16* q, const hca_bf16* g, hca_bf16* out, int S, int N,
                         float scale, const hca_bf16* vha_down, const hca_bf16* vha_up,
                         int vha_rank, int clusters, cudaStream_t stream) {
  namespace P = hca::prefill3;
  P::PagedMaps maps;
  const uint64_t rows = static_cast<uint64_t>(N) * HCA_NUM_HEADS;
  const uint64_t raw = static_cast<uint64_t>(N) + static_cast<uint64_t>(hca::paged::kPad) * S;
  const uint64_t prows = static_cast<uint64_t>(clusters) * P::kScratchPerCluster / 256;
  const uint32_t page = 1u << c.page_shift;
  bool ok = make_map4(&maps.q4, q, rows, 1, 128, 4) && make_map4(&maps.g4, g, rows, 1, 128, 2) &&
            make_map4(&maps.out4, out, rows, 1, 128, 2) &&
            make_map4(&maps.out1, out, rows, 1, 64, 1) &&
            make_map(&maps.kwin, w + L.raw_k, HCA_HEAD_DIM, raw, 1, P::kWinHalf) &&
            make_map4(&maps.v4, w + L.raw_v, raw, 1, 128, 2) &&
            make_map4(&maps.v4t, w + L.raw_v, raw, 1, 16, 1) &&
            make_map4(&maps.tail, w + L.tail, static_cast<uint64_t>(S) * 16, 1, 16, 1) &&
            make_map_bytes(&maps.p128, w + L.scratch, prows, 128) &&
            make_map_bytes(&maps.p16, w + L.scratch, prows, 16);
  if (ok && c.num_pages > 0) {
    ok = make_map(&maps.ck, c.ck, HCA_HEAD_DIM, page, c.num_pages, page < 64 ? page : 64) &&
         make_map4(&maps.cv4, c.cv, page, c.num_pages, page, 1) &&
         make_map4(&maps.cv16, c.cv, page, c.num_pages, 16, 1);
  } else if (ok) {   // no entry can be visible: never used
    maps.ck = maps.kwin;
    maps.cv4 = maps.cv16 = maps.v4t;
  }
  if (!ok) return HCA_ERR_CUDA;
  P::Params prm = {};
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.pscratch = w + L.scratch;
  prm.vha_down = vha_down;
  prm.vha_up = vha_up;
  prm.vha_rank = vha_rank;
  prm.item_list = reinterpret_cast<const int4*>(w + L.list);
  prm.item_count = reinterpret_cast<const int*>(w + L.count);
  prm.tail16 = reinterpret_cast<const int*>(w + L.tail16);
  prm.table = c.table;
  prm.table_ld = c.table_ld;
  prm.num_pages = c.num_pages;
  prm.page_shift = c.page_shift;
  prm.max_nc = c.num_pages > 0 ? c.max_pages << c.page_shift : 0;
  prm.raw_pad = hca::paged::kPad;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * clusters);
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmemAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t err = vha_rank > 0
                              ? cudaLaunchKernelEx(&cfg, P::prefill3_kernel<true, true>, maps, prm)
                              : cudaLaunchKernelEx(&cfg, P::prefill3_kernel<false, true>, maps, prm);
  return err == cudaSuccess ? launch_status() : HCA_ERR_CUDA;
}

// clusters of the prefill kernel for at most `items` items
int paged_clusters(int items) {
  const int most = prefill_max_clusters<true>();
  return items < most ? items : most;
}

}  // namespace

extern "C" {

hca_status_t hca_paged_append(const hca_bf16* k_new, const hca_bf16* v_new, const hca_bf16* s_new,
                              const int32_t* q_start, const int32_t* ctx_len, int S, int N,
                              const hca_paged_cache_t* cache, hca_stream_t stream) {
  namespace G = hca::paged;
  G::Cache c;
  G::Chunk ch;
  hca_status_t st = chunk_args(ch, k_new, v_new, s_new, q_start, ctx_len, S, N);
  if (st != HCA_OK) return st;
  if (q_start == nullptr && N != S) return HCA_ERR_INVALID_ARG;
  st = paged_cache(c, cache, S, true);
  if (st != HCA_OK) return st;
  if (N == 0) return HCA_OK;
  if (q_start == nullptr) {
    G::step_kernel<<<dim3(S, 8), G::kThreads, 0, stream>>>(ch, c);
    return launch_status();
  }
  const long long units = entry_units<false>(S, N);
  if (units > 0x7fffffffLL) return HCA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units), 8);
  cfg.blockDim = dim3(G::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1;
  attr.val.clusterDim.y = 8;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  uint16_t* none = nullptr;
  if (cudaLaunchKernelEx(&cfg, G::entries_kernel<false>, ch, c, none, none) != cudaSuccess)
    return HCA_ERR_CUDA;
  return launch_status();
}

size_t hca_paged_prefill_workspace_size(int S, int N) {
  if (S < 1 || N < 1) return 0;
  const int clusters = paged_clusters(0x7fffffff);
  if (clusters <= 0) return 0;
  // no smaller for fewer tokens: one workspace serves every call of at most S and N
  const size_t a = paged_prefill_layout(S, N < kSplitMost ? N : kSplitMost, clusters, true).total;
  const size_t b = N > kSplitTokens ? paged_prefill_layout(S, N, clusters, false).total : 0;
  return a > b ? a : b;
}

hca_status_t hca_paged_prefill(const hca_bf16* q, const hca_bf16* g, const hca_bf16* k_new,
                               const hca_bf16* v_new, const hca_bf16* s_new,
                               const int32_t* q_start, const int32_t* ctx_len, int S, int N, int H,
                               float scale, const hca_bf16* vha_down, const hca_bf16* vha_up,
                               int vha_rank, const hca_paged_cache_t* cache, hca_bf16* out,
                               void* ws, size_t ws_bytes, hca_stream_t stream) {
  namespace G = hca::paged;
  G::Cache c;
  G::Chunk ch;
  hca_status_t st = attend_args(q, g, out, H, scale, vha_down, vha_up, vha_rank, ws);
  if (st != HCA_OK) return st;
  st = chunk_args(ch, k_new, v_new, s_new, q_start, ctx_len, S, N);
  if (st != HCA_OK) return st;
  if (q_start == nullptr) return HCA_ERR_INVALID_ARG;
  st = paged_cache(c, cache, S, true);
  if (st != HCA_OK) return st;
  if (N == 0) return HCA_OK;
  if (S > kMaxChunkSeqs || static_cast<long long>(N) + static_cast<long long>(G::kPad) * S >
                               0x7fffffffLL / HCA_NUM_HEADS)
    return HCA_ERR_UNSUPPORTED;
  const long long units = entry_units<true>(S, N);
  const int most = prefill_max_clusters<true>();
  if (most <= 0) return HCA_ERR_CUDA;
  const PagedPrefillLayout L = paged_prefill_layout(S, N, most, split_form(S, N, most));
  if (ws_bytes < L.total || out_overlaps(out, q, g, N)) return HCA_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint16_t* raw_k = reinterpret_cast<uint16_t*>(w + L.raw_k);
  uint16_t* raw_v = reinterpret_cast<uint16_t*>(w + L.raw_v);
  G::Queries qr = {};
  if (!L.split) {
    qr.count = reinterpret_cast<int*>(w + L.count);
    qr.items = reinterpret_cast<int4*>(w + L.list);
    qr.cap = L.items;
    qr.tail16 = reinterpret_cast<int*>(w + L.tail16);
    qr.tail = reinterpret_cast<uint16_t*>(w + L.tail);
  }
  G::entries_kernel<true>
      <<<dim3(static_cast<unsigned>(units), 8), G::kThreads, 0, stream>>>(ch, c, raw_k, raw_v);
  if (launch_behind(G::finish_kernel, dim3(S, G::kFinishY), G::kFinishThreads, stream, ch, c, qr) !=
      cudaSuccess)
    return HCA_ERR_CUDA;
  if (!L.split)
    return paged_items(c, L, w, q, g, out, S, N, scale, vha_down, vha_up, vha_rank,
                       paged_clusters(L.items), stream);
  hca::pdecode::Params prm = {};
  prm.chunk = ch;
  prm.only_window = 1;
  prm.S = N;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.vha_down = vha_down;
  prm.vha_up = vha_up;
  prm.vha_rank = vha_rank;
  return paged_attend(c, q, g, out, raw_k, raw_v,
                      static_cast<uint64_t>(N) + static_cast<uint64_t>(G::kPad) * S, prm,
                      w, stream);
}

size_t hca_paged_decode_workspace_size(int S) {
  if (S < 1) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  // head, split partials, tile prefix
  return kHeadBytes + align256(hca::pdecode::ws_bytes(sms + S)) + static_cast<size_t>(S + 2) * 8;
}

}  // extern "C"

namespace {
// hca_paged_decode; `step`: with the append of these tokens
hca_status_t paged_decode(const hca_bf16* q, const hca_bf16* g, const int32_t* ctx_len, int S,
                          int H, float scale, const hca_bf16* vha_down, const hca_bf16* vha_up,
                          int vha_rank, const hca_paged_cache_t* cache, hca_bf16* out, void* ws,
                          size_t ws_bytes, const hca::paged::Chunk* step, cudaStream_t stream) {
  namespace G = hca::paged;
  G::Cache c;
  hca_status_t st = attend_args(q, g, out, H, scale, vha_down, vha_up, vha_rank, ws);
  if (st != HCA_OK) return st;
  if (S < 1 || ctx_len == nullptr || !aligned4(ctx_len)) return HCA_ERR_INVALID_ARG;
  if (S > 65535) return HCA_ERR_UNSUPPORTED;
  st = paged_cache(c, cache, S, step != nullptr);
  if (st != HCA_OK) return st;
  if (ws_bytes < hca_paged_decode_workspace_size(S) || out_overlaps(out, q, g, S))
    return HCA_ERR_INVALID_ARG;
  hca::pdecode::Params prm = {};
  prm.ctx_len = ctx_len;
  prm.S = S;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.vha_down = vha_down;
  prm.vha_up = vha_up;
  prm.vha_rank = vha_rank;
  if (step != nullptr && S <= hca::pdecode::kInlineSeqs) {
    // one launch instead of two: both sides at the append in paged_decode_kernel
    prm.chunk = *step;
    prm.cache = c;
  } else if (step != nullptr) {   // the CTAs do not have the lengths at hand
    G::step_kernel<<<dim3(S, 8), G::kThreads, 0, stream>>>(*step, c);
    if (cudaGetLastError() != cudaSuccess) return HCA_ERR_CUDA;
  }
  return paged_attend(c, q, g, out, c.wk, c.wv, static_cast<uint64_t>(S) * HCA_WINDOW, prm,
                      static_cast<uint8_t*>(ws), stream);
}
}  // namespace

extern "C" {

hca_status_t hca_paged_decode(const hca_bf16* q, const hca_bf16* g, const int32_t* ctx_len, int S,
                              int H, float scale, const hca_bf16* vha_down,
                              const hca_bf16* vha_up, int vha_rank,
                              const hca_paged_cache_t* cache, hca_bf16* out, void* ws,
                              size_t ws_bytes, hca_stream_t stream) {
  return paged_decode(q, g, ctx_len, S, H, scale, vha_down, vha_up, vha_rank, cache, out, ws,
                      ws_bytes, nullptr, stream);
}

hca_status_t hca_paged_decode_step(const hca_bf16* q, const hca_bf16* g, const hca_bf16* k_new,
                                   const hca_bf16* v_new, const hca_bf16* s_new,
                                   const int32_t* ctx_len, int S, int H, float scale,
                                   const hca_bf16* vha_down, const hca_bf16* vha_up, int vha_rank,
                                   const hca_paged_cache_t* cache, hca_bf16* out, void* ws,
                                   size_t ws_bytes, hca_stream_t stream) {
  hca::paged::Chunk step;
  const hca_status_t st = chunk_args(step, k_new, v_new, s_new, nullptr, ctx_len, S, S);
  if (st != HCA_OK) return H == HCA_NUM_HEADS ? st : HCA_ERR_UNSUPPORTED;
  return paged_decode(q, g, ctx_len, S, H, scale, vha_down, vha_up, vha_rank, cache, out, ws,
                      ws_bytes, &step, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Page management
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxForks = 8192;

hca_status_t page_rows(hca::pages::Table& t, const hca_page_table_t* p) {
  if (p == nullptr || p->rows < 1 || p->max_pages < 1 || p->num_pages < 1 ||
      p->table_stride < p->max_pages)
    return HCA_ERR_INVALID_ARG;
  const int shift = page_shift_of(p->page_size);
  if (shift < 0) return HCA_ERR_UNSUPPORTED;
  if (p->page_table == nullptr || p->n_pages == nullptr || p->ref == nullptr ||
      !aligned4(p->page_table) || !aligned4(p->n_pages) || !aligned4(p->ref))
    return HCA_ERR_INVALID_ARG;
  t = {p->page_table, p->table_stride, p->rows, p->max_pages, p->n_pages, p->ref, p->num_pages,
       shift};
  return HCA_OK;
}

// Adds `n` arrays with the given lists to `m` (whose list length is set).
hca_status_t move_arrays(hca::pages::Move& m, const hca_page_array_t* arrays, int n, const int* src,
                         const int* dst) {
  if (n < 0 || (n > 0 && arrays == nullptr)) return HCA_ERR_INVALID_ARG;
  if (m.arrays + n > hca::pages::kMaxArrays) return HCA_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    if (arrays[i].data == nullptr || !aligned16(arrays[i].data) || arrays[i].item_bytes < 16 ||
        arrays[i].item_bytes % 16 != 0)
      return HCA_ERR_INVALID_ARG;
    const long long per = (arrays[i].item_bytes - 1) / hca::pages::kUnit + 1;
    if (per > 0x7fffffffLL || m.units + per * m.n > 0x7fffffffLL) return HCA_ERR_UNSUPPORTED;
    m.units += per * m.n;
    m.a[m.arrays++] = {static_cast<uint8_t*>(arrays[i].data), arrays[i].item_bytes,
                       static_cast<unsigned>(per), src, dst};
  }
  return HCA_OK;
}

hca_status_t launch_move(const hca::pages::Move& m, cudaStream_t stream) {
  namespace P = hca::pages;
  if (m.n < 1 || (m.arrays == 0 && m.table == nullptr)) return launch_status();
  const int sms = device_sms();
  if (sms <= 0) return HCA_ERR_CUDA;
  long long units = m.units;
  const long long table = (static_cast<long long>(m.rows) * m.max_pages + 1023) / 1024;
  units = units > table ? units : table;
  const long long most = 8LL * sms;
  if (launch_behind(P::move_kernel, dim3(static_cast<unsigned>(units < most ? units : most)),
                    P::kMoveThreads, stream, m) != cudaSuccess)
    return HCA_ERR_CUDA;
  return launch_status();
}

hca_status_t pages_resize(const hca_page_table_t* table, const int32_t* entries,
                          const hca_page_array_t* pools, int n_pools, bool copy, void* ws,
                          size_t ws_bytes, cudaStream_t stream) {
  namespace P = hca::pages;
  P::Table t;
  hca_status_t st = page_rows(t, table);
  if (st != HCA_OK) return st;
  if (entries == nullptr || ws == nullptr || !aligned4(entries) || !aligned16(ws) ||
      ws_bytes < hca_pages_workspace_size(t.rows, t.num_pages, 0) || (copy && n_pools < 1))
    return HCA_ERR_INVALID_ARG;
  int* free_list = static_cast<int*>(ws);
  int* prefix = free_list + t.num_pages;
  P::Move m = {};
  int *src = nullptr, *dst = nullptr, *count = nullptr;
  if (copy) {
    src = prefix + t.rows + 1;
    dst = src + t.rows;
    count = dst + t.rows;
    m.n = t.rows;
    m.count = count;
    st = move_arrays(m, pools, n_pools, src, dst);
    if (st != HCA_OK) return st;
  }
  P::resize_kernel<<<1, P::kPlanThreads, 0, stream>>>(t, entries, free_list, prefix, src, dst,
                                                      count);
  st = launch_status();
  return st == HCA_OK && copy ? launch_move(m, stream) : st;
}

}  // namespace

extern "C" {

size_t hca_pages_workspace_size(int rows, int num_pages, int n) {
  if (rows < 1 || num_pages < 1 || n < 0) return 0;
  // the largest of: resize (free list, prefix, two lists, count), fork (four lists), compact
  // (two half lists, remap, count), copy (marks, two lists)
  const size_t pages = num_pages, list = n;
  const size_t resize = pages + 3 * static_cast<size_t>(rows) + 2, fork = 4 * list, compact = 2 * (pages / 2 + 1) + pages + 1,
               copy = pages + 2 * list;
  size_t most = resize;
  for (const size_t x : {fork, compact, copy}) most = x > most ? x : most;
  return align256(most * 4);
}

hca_status_t hca_pages_resize(const hca_page_table_t* table, const int32_t* entries, void* ws,
                              size_t ws_bytes, hca_stream_t stream) {
  return pages_resize(table, entries, nullptr, 0, false, ws, ws_bytes, stream);
}

hca_status_t hca_pages_resize_copy(const hca_page_table_t* table, const int32_t* entries,
                                   const hca_page_array_t* pools, int n_pools, void* ws,
                                   size_t ws_bytes, hca_stream_t stream) {
  return pages_resize(table, entries, pools, n_pools, true, ws, ws_bytes, stream);
}

hca_status_t hca_pages_fork(const hca_page_table_t* table, const int32_t* parents,
                            const int32_t* children, const int32_t* entries, int n,
                            const hca_page_array_t* pools, int n_pools,
                            const hca_page_array_t* rings, int n_rings, int32_t* ok, void* ws,
                            size_t ws_bytes, hca_stream_t stream) {
  namespace P = hca::pages;
  P::Table t;
  hca_status_t st = page_rows(t, table);
  if (st != HCA_OK) return st;
  if (n < 0 || parents == nullptr || children == nullptr || entries == nullptr || ok == nullptr ||
      ws == nullptr || !aligned4(parents) || !aligned4(children) || !aligned4(entries) ||
      !aligned4(ok) || !aligned16(ws) ||
      ws_bytes < hca_pages_workspace_size(t.rows, t.num_pages, n))
    return HCA_ERR_INVALID_ARG;
  if (n > kMaxForks) return HCA_ERR_UNSUPPORTED;
  int* src = static_cast<int*>(ws);
  int *dst = src + n, *rsrc = src + 2 * n, *rdst = src + 3 * n;
  P::Move m = {};
  m.n = n;
  st = move_arrays(m, pools, n_pools, src, dst);
  if (st == HCA_OK) st = move_arrays(m, rings, n_rings, rsrc, rdst);
  if (st != HCA_OK) return st;
  if (n == 0) return HCA_OK;
  P::fork_kernel<<<1, P::kPlanThreads, 0, stream>>>(t, parents, children, entries, n, ok, src, dst,
                                                    rsrc, rdst);
  st = launch_status();
  return st == HCA_OK ? launch_move(m, stream) : st;
}

hca_status_t hca_pages_compact(const hca_page_table_t* table, const hca_page_array_t* pools,
                               int n_pools, int32_t* live, void* ws, size_t ws_bytes,
                               hca_stream_t stream) {
  namespace P = hca::pages;
  P::Table t;
  hca_status_t st = page_rows(t, table);
  if (st != HCA_OK) return st;
  if (live == nullptr || ws == nullptr || !aligned4(live) || !aligned16(ws) ||
      ws_bytes < hca_pages_workspace_size(t.rows, t.num_pages, 0))
    return HCA_ERR_INVALID_ARG;
  const int half = t.num_pages / 2 + 1;
  int* src = static_cast<int*>(ws);
  int *dst = src + half, *remap = src + 2 * half, *count = remap + t.num_pages;
  P::Move m = {};
  m.n = t.num_pages / 2;
  m.count = count;
  m.table = t.table;
  m.table_ld = t.ld;
  m.rows = t.rows;
  m.max_pages = t.max_pages;
  m.remap = remap;
  m.live = live;
  m.num_pages = t.num_pages;
  st = move_arrays(m, pools, n_pools, src, dst);
  if (st != HCA_OK) return st;
  P::compact_kernel<<<1, P::kPlanThreads, 0, stream>>>(t.ref, t.num_pages, src, dst, count, remap,
                                                       live);
  st = launch_status();
  return st == HCA_OK ? launch_move(m, stream) : st;
}

hca_status_t hca_pages_copy(const hca_page_array_t* arrays, int n_arrays, int items,
                            const int32_t* src, const int32_t* dst, int n, void* ws,
                            size_t ws_bytes, hca_stream_t stream) {
  namespace P = hca::pages;
  if (items < 1 || n < 0 || n >= 1 << 30 || src == nullptr || dst == nullptr || ws == nullptr ||
      !aligned4(src) || !aligned4(dst) || !aligned16(ws) ||
      ws_bytes < hca_pages_workspace_size(1, items, n))
    return HCA_ERR_INVALID_ARG;
  int* mark = static_cast<int*>(ws);
  int *from = mark + items, *to = from + n;
  P::Move m = {};
  m.n = n;
  const hca_status_t st = move_arrays(m, arrays, n_arrays, from, to);
  if (st != HCA_OK) return st;
  if (n == 0) return HCA_OK;
  if (cudaMemsetAsync(mark, 0, static_cast<size_t>(items) * 4, stream) != cudaSuccess)
    return HCA_ERR_CUDA;
  P::check_kernel<<<1, P::kPlanThreads, 0, stream>>>(src, dst, n, items, mark, from, to);
  return launch_move(m, stream);
}

}  // extern "C"
