/*
 * hca.h — C ABI of libhca.so, a B200 (sm_100a) implementation of the forward
 * hot path of Heavily Compressed Attention (HCA).
 *
 * The method.  'BaiduがERNIE 5.5 Flash Baseを公開' §2.1 (Latent-Gated Sparse
 * Attention) and its Chinese twin 'ERNIE 5.5 Flash Base 正式发布' §2.1 describe
 * HCA layers that turn every 128 tokens into one cache entry and run one dense
 * softmax over all of those entries plus a short window of recent raw tokens,
 * with 64 query heads of width 512; every layer multiplies its attention
 * output by a learned gate.  The xenospectrum analysis of the same release
 * (section 活性140億パラメータと長文処理を支える仕組み) gives the window: the
 * newest 128 tokens, kept uncompressed.  Where the pages are silent this
 * library fixes: one shared KV head; entry j = softmax(s over block j)-weighted
 * sum of the block's K rows (and, with the same weights, of its V rows), with s
 * a per-token score; query t sees entry j only when block j lies wholly before
 * its window, i.e. j < nc(t) = max(0, floor((t - 127) / 128)), and the raw keys
 * max(0, t - 127) .. t; out = sigmoid(g) * o elementwise.
 *
 * Conventions shared by every call:
 *  - bf16 values are passed as raw 16-bit patterns (hca_bf16).  Every tensor is
 *    dense, row-major, on the current CUDA device, and 16-byte aligned.
 *  - The caller owns every buffer and the stream; the library allocates no
 *    memory and keeps no per-call state.  Calls are asynchronous on `stream`
 *    (NULL = legacy default stream).
 *  - Arguments are validated on the host before anything is launched; a
 *    rejected call returns HCA_ERR_INVALID_ARG or HCA_ERR_UNSUPPORTED and
 *    launches nothing.  HCA_ERR_CUDA reports a launch failure.
 *  - Kernels never trap.  Every wait inside them is bounded; a wait that runs
 *    out, or a device-resident argument found out of range (decode context
 *    lengths), is recorded in a device-side error word that
 *    hca_get_device_error() reads back.
 *  - No C++ exception crosses this interface.
 */
#ifndef HCA_H
#define HCA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HCA_OK = 0,
  HCA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size or scale       */
  HCA_ERR_UNSUPPORTED = 2, /* a shape outside what the kernels implement       */
  HCA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed                */
  HCA_ERR_TIMEOUT = 4,     /* a device-side bounded wait ran out               */
  HCA_ERR_DEVICE_INPUT = 5 /* a device-resident argument was out of range      */
} hca_status_t;

typedef uint16_t hca_bf16;              /* raw bfloat16 bits                   */
typedef struct CUstream_st* hca_stream_t; /* same type as cudaStream_t         */

#define HCA_HEAD_DIM 512 /* width of q, k, v and o rows                        */
#define HCA_NUM_HEADS 64 /* query heads sharing the single KV head             */
#define HCA_BLOCK 128    /* tokens per compressed entry                        */
#define HCA_WINDOW 128   /* raw tokens each query attends (itself included)    */

/*
 * hca_compress — block compressor.
 *   'BaiduがERNIE 5.5 Flash Baseを公開' §2.1: 128 tokens -> one cache entry.
 *   For every complete block j < nb = floor(T / 128) of every batch b:
 *     w = softmax(s[b, 128j : 128j + 128])            (fp32)
 *     ck[b, j, :] = sum_i w_i * k[b, 128j + i, :]      (fp32 accumulate, bf16 RNE)
 *     cv[b, j, :] = sum_i w_i * v[b, 128j + i, :]
 *   Tokens of a trailing partial block are not compressed.
 * Layout:  k, v  [B, T, 512] bf16;  s [B, T] bf16;  ck, cv [B, nb, 512] bf16.
 * Errors:  B < 1 or T < 1 -> HCA_ERR_INVALID_ARG.  nb == 0 launches nothing.
 */
hca_status_t hca_compress(const hca_bf16* k, const hca_bf16* v, const hca_bf16* s, int B, int T,
                          hca_bf16* ck, hca_bf16* cv, hca_stream_t stream);

/*
 * hca_prefill_workspace_size — bytes of device scratch hca_prefill_fwd needs
 * on the current device (probability tiles in flight between the CTAs of
 * each cluster; under 10 MB on a B200).  The answer depends on how many
 * clusters fit on the device, which is queried once per device.  Returns 0
 * for B < 1 or T < 1 or when the query fails.
 */
size_t hca_prefill_workspace_size(int B, int T);

/*
 * hca_prefill_fwd — HCA attention for every position of B sequences.
 *   For query t of batch b and head h (page sources as above):
 *     keys   = [ck[b, 0 : nc(t)] ; k[b, max(0, t-127) : t+1]]
 *     values = [cv[b, 0 : nc(t)] ; v[b, max(0, t-127) : t+1]]
 *     p      = softmax(scale * keys . q[b, t, h])      (one softmax over both sets)
 *     out[b, t, h, :] = sigmoid(g[b, t, h, :]) * (p . values)
 *   lse (optional) receives ln(sum exp(scale * keys . q)) per (b, t, h).
 * Layout:  q, g, out [B, T, H, 512] bf16 (H = 64);  k, v [B, T, 512] bf16;
 *          ck, cv [B, floor(T/128), 512] bf16 as written by hca_compress;
 *          lse [B, T, H] fp32 or NULL;  ws: caller-owned device scratch of at
 *          least hca_prefill_workspace_size(B, T) bytes, 256-byte aligned (its
 *          contents need no initialisation and are meaningless afterwards;
 *          two calls in flight at once need two workspaces).
 * Errors:  H != 64 -> HCA_ERR_UNSUPPORTED; B < 1, T < 1, a null pointer (other
 *          than lse), a pointer not 16-byte aligned, a workspace too small or
 *          misaligned, or a non-finite or non-positive scale ->
 *          HCA_ERR_INVALID_ARG.
 */
hca_status_t hca_prefill_fwd(const hca_bf16* q, const hca_bf16* k, const hca_bf16* v,
                             const hca_bf16* ck, const hca_bf16* cv, const hca_bf16* g, int B,
                             int T, int H, float scale, hca_bf16* out, float* lse, void* ws,
                             size_t ws_bytes, hca_stream_t stream);

/*
 * hca_prefill_fwd_vha — hca_prefill_fwd followed, inside the same kernel, by
 *   virtual head attention ('BaiduがERNIE 5.5 Flash Baseを公開' §2.1 and
 *   'ERNIE 5.5 Flash Base 正式发布' §2.1, VHA: after attention, a light
 *   low-rank mix across heads with an identity skip, fused into the attention
 *   kernel at inference).  With x[b, t] the [H, 512] gated output above:
 *     out[b, t, h, :] = x[h, :] + sum_r up[h, r] * sum_k down[k, r] * x[k, :]
 *   (the pages give no rank and do not say where the gate sits; this reads
 *   the mix as acting on the gated output of each position).
 * Layout:  as hca_prefill_fwd;  vha_down, vha_up [64, vha_rank] bf16
 *          row-major, device memory, 1 <= vha_rank <= 64.  The mix runs in
 *          fp32 on bf16 operands: x rounded to bf16 and the 64 x 64 product
 *          up down^T formed in fp32 and rounded to bf16 once per launch.
 * Errors:  those of hca_prefill_fwd; HCA_ERR_INVALID_ARG for a rank outside
 *          [1, 64] or a NULL factor.
 */
hca_status_t hca_prefill_fwd_vha(const hca_bf16* q, const hca_bf16* k, const hca_bf16* v,
                                 const hca_bf16* ck, const hca_bf16* cv, const hca_bf16* g,
                                 int B, int T, int H, float scale, const hca_bf16* vha_down,
                                 const hca_bf16* vha_up, int vha_rank, hca_bf16* out, float* lse,
                                 void* ws, size_t ws_bytes, hca_stream_t stream);

/*
 * hca_prefill_bwd_workspace_size — bytes of device scratch hca_prefill_bwd
 * needs: dO, the probabilities and their gradients over every visited
 * (row, key) pair in bf16, and the fp32 entry gradients (about 2 KB per
 * (position, head) row per 512 compressed entries, plus 1.6 KB per row).
 * Returns 0 for B < 1 or T < 1.
 */
size_t hca_prefill_bwd_workspace_size(int B, int T);

/*
 * hca_prefill_bwd — gradients of L = sum(dout * out) for out =
 *   hca_prefill_fwd(q, k, v, hca_compress(k, v, s), g) (the model trains at
 *   128K context, 'BaiduがERNIE 5.5 Flash Baseを公開' §3).  With o the
 *   ungated output and P the softmax of each query:
 *     dg = dout * out * (1 - sigmoid(g)),  dO = dout * sigmoid(g)
 *     dS = P (dO . value - sum_d dout * out),  dq = scale sum dS key,
 *     dkey = scale sum dS q,  dvalue = sum P dO  (raw keys and entries),
 *   and the entry gradients through each block's compressor into dk, dv and
 *   ds (ds_i = w_i (a_i - sum w a), a_i = dcK . k_i + dcV . v_i).
 * Layout:  q, g, out, dout, dq, dg [B, T, 64, 512] bf16;  k, v [B, T, 512]
 *          bf16;  s [B, T] bf16;  ck, cv the forward's [B, T/128, 512];
 *          lse [B, T, 64] fp32 as written by hca_prefill_fwd;  dk, dv
 *          [B, T, 512] fp32;  ds [B, T] fp32 (0 for tokens of a partial
 *          block).  All device memory, 16-byte aligned; ws 256-byte aligned,
 *          at least hca_prefill_bwd_workspace_size(B, T) bytes, contents
 *          meaningless before and after.  Five launches on `stream`.
 * Errors:  HCA_ERR_UNSUPPORTED for H != 64 or T * 64 >= 2^31;
 *          HCA_ERR_INVALID_ARG for a NULL or misaligned pointer, B, T < 1, a
 *          non-finite or non-positive scale, or a short workspace;
 *          HCA_ERR_CUDA for a launch failure.
 */
hca_status_t hca_prefill_bwd(const hca_bf16* q, const hca_bf16* k, const hca_bf16* v,
                             const hca_bf16* s, const hca_bf16* ck, const hca_bf16* cv,
                             const hca_bf16* g, const hca_bf16* out, const float* lse,
                             const hca_bf16* dout, int B, int T, int H, float scale, hca_bf16* dq,
                             float* dk, float* dv, float* ds, hca_bf16* dg, void* ws,
                             size_t ws_bytes, hca_stream_t stream);

/*
 * hca_decode_workspace_size — bytes of scratch hca_decode needs for S
 * sequences on the current device (partial results of the split-KV pass and
 * a grid-barrier counter).  A workspace must be zero-filled once before its
 * first hca_decode call (e.g. cudaMemsetAsync); every call leaves it valid for
 * the next one, whatever S, on the same device.
 */
size_t hca_decode_workspace_size(int S);

/*
 * hca_decode — one new token per sequence (split-KV over all SMs, then a
 * log-sum-exp combine, in one cooperative launch of one CTA per SM; above
 * 1024 sequences a one-CTA plan kernel runs first).
 *   For sequence i with context length L = ctx_len[i] (which counts the new
 *   token, so the query sits at t = L - 1):
 *     keys   = [ck[i, 0 : nc(L-1)] ; the min(L, 128) newest raw keys]
 *     out[i, h, :] = sigmoid(g[i, h, :]) * softmax(scale * keys . q[i, h]) . values
 *   The raw window is a ring: the token at position p lives in slot p mod 128
 *   of wk/wv; when L < 128 only slots 0 .. L-1 are read.  Slot order does not
 *   change the result (no positional term).
 * Layout:  q, g, out [S, H, 512] bf16 (H = 64);  ck, cv [S, max_nc, 512] bf16;
 *          wk, wv [S, 128, 512] bf16;  ctx_len [S] int32 on the device;
 *          ws: caller-owned device scratch of at least
 *          hca_decode_workspace_size(S) bytes, 256-byte aligned, zero-filled
 *          before its first use; one call at a time per workspace.
 * Errors:  host-checked as for prefill (and ws_bytes too small ->
 *          HCA_ERR_INVALID_ARG).  A device-side ctx_len < 1 or one needing more
 *          than max_nc entries is clamped and reported later by
 *          hca_get_device_error() as HCA_ERR_DEVICE_INPUT.
 */
hca_status_t hca_decode(const hca_bf16* q, const hca_bf16* ck, const hca_bf16* cv, int max_nc,
                        const hca_bf16* wk, const hca_bf16* wv, const int32_t* ctx_len,
                        const hca_bf16* g, int S, int H, float scale, void* ws, size_t ws_bytes,
                        hca_bf16* out, hca_stream_t stream);

/*
 * hca_decode_vha — hca_decode followed, inside the same kernel, by virtual
 *   head attention on each sequence's gated output (same passage and reading
 *   as hca_prefill_fwd_vha):
 *     out[s, h, :] = x[h, :] + sum_r up[h, r] * sum_k down[k, r] * x[k, :]
 *   with x[s] the [64, 512] output hca_decode would write.  The mix runs in
 *   fp32 on x rounded to bf16 (a second grid barrier of the launch separates
 *   the two phases).
 * Layout:  as hca_decode;  vha_down, vha_up [64, vha_rank] bf16 row-major,
 *          device memory, 1 <= vha_rank <= 64.
 * Errors:  those of hca_decode; HCA_ERR_INVALID_ARG for a rank outside
 *          [1, 64] or a NULL factor.
 */
hca_status_t hca_decode_vha(const hca_bf16* q, const hca_bf16* ck, const hca_bf16* cv,
                            int max_nc, const hca_bf16* wk, const hca_bf16* wv,
                            const int32_t* ctx_len, const hca_bf16* g, int S, int H, float scale,
                            const hca_bf16* vha_down, const hca_bf16* vha_up, int vha_rank,
                            void* ws, size_t ws_bytes, hca_bf16* out, hca_stream_t stream);

/*
 * hca_decode_noalloc — hca_decode for callers that cannot allocate device
 * memory.  The paper has no counterpart: this is a deployment variant.
 *   Some callers have no way to provide scratch: a plugin loaded into a host
 *   program that owns all device memory and exposes no allocator, or a
 *   latency-critical serving loop where a cudaMalloc (which can synchronise
 *   the whole device) is not allowed.  This entry point takes the same
 *   inputs and output as hca_decode but no workspace; its scratch lives in
 *   one fixed device array inside the library (224 split slots of 66,048
 *   bytes plus a small index and the grid-barrier counter: about 14.8 MB),
 *   which every GPU that loads the library keeps until the process exits.
 *   Limits: S <= HCA_NOALLOC_MAX_SEQS (64); larger S returns
 *   HCA_ERR_UNSUPPORTED without launching.  The split uses at most
 *   HCA_NOALLOC_MAX_CTAS (160) CTAs.
 *   Set-up: every call looks up the array's device address in the current
 *   device's context (cudaGetSymbolAddress, with that device current; the
 *   array's name in host code is only a handle).  The first call on a device
 *   also loads the library's module there, so make that first call outside
 *   any stream capture.  Nothing is allocated, ever.
 *   Sharing: every call uses the same array.  Its grid-barrier counter starts
 *   at zero when the library loads and every call leaves it valid (each call
 *   writes every other scratch value it later reads), but two calls that
 *   overlap on the GPU (other streams, other threads) race on it: serialise
 *   them.
 */
#define HCA_NOALLOC_MAX_SEQS 64
#define HCA_NOALLOC_MAX_CTAS 160
hca_status_t hca_decode_noalloc(const hca_bf16* q, const hca_bf16* ck, const hca_bf16* cv,
                                int max_nc, const hca_bf16* wk, const hca_bf16* wv,
                                const int32_t* ctx_len, const hca_bf16* g, int S, int H,
                                float scale, hca_bf16* out, hca_stream_t stream);

/*
 * hca_cache_append — incremental update of a decode cache by one new token per
 * sequence (the step on either side of hca_decode in serving).
 *   'BaiduがERNIE 5.5 Flash Baseを公開' §2.1: every 128 tokens become one
 *   cache entry; the xenospectrum analysis (section 活性140億パラメータと
 *   長文処理を支える仕組み): the newest 128 tokens stay raw.
 *   For sequence i with L = ctx_len[i] (which counts the new token, at
 *   position p = L - 1):
 *     wk[i, p mod 128] = k_new[i];  wv[i, p mod 128] = v_new[i];
 *     ws[i, p mod 128] = s_new[i]                       (the ring of raw tokens)
 *   and when L is a multiple of 128, block j = L/128 - 1 (now exactly the ring)
 *   is compressed into entry j:
 *     w = softmax(ws[i, 0:128]) (fp32);  ck[i, j] = sum_r w_r wk[i, r];
 *     cv[i, j] = sum_r w_r wv[i, r]           (fp32 accumulate, bf16 RNE)
 *   -- the value hca_compress gives for that block of the raw sequence.
 * Layout:  k_new, v_new [S, 512] bf16;  s_new [S] bf16;  ctx_len [S] int32 on
 *          the device;  wk, wv [S, 128, 512] bf16 and ws [S, 128] bf16 rings,
 *          updated in place;  ck, cv [S, max_nc, 512] bf16, entry j written in
 *          place (may be NULL when max_nc = 0).
 * Errors:  host-checked: S < 1, max_nc < 0, a null or (for the 512-wide
 *          tensors) misaligned pointer -> HCA_ERR_INVALID_ARG.  A device-side
 *          ctx_len < 1, or a completed block j >= max_nc, writes nothing for
 *          that sequence (ctx_len < 1) or skips the entry, and is reported by
 *          hca_get_device_error() as HCA_ERR_DEVICE_INPUT.
 */
hca_status_t hca_cache_append(const hca_bf16* k_new, const hca_bf16* v_new,
                              const hca_bf16* s_new, const int32_t* ctx_len, int S, hca_bf16* wk,
                              hca_bf16* wv, hca_bf16* ws, hca_bf16* ck, hca_bf16* cv, int max_nc,
                              hca_stream_t stream);

/*
 * hca_decode_step — one serving step: hca_cache_append of the new tokens,
 * then hca_decode of their queries against the updated cache, in stream
 * order on `stream` (two launches).  Arguments as in those two calls;
 * everything is validated before either kernel is launched.
 */
hca_status_t hca_decode_step(const hca_bf16* q, const hca_bf16* g, const hca_bf16* k_new,
                             const hca_bf16* v_new, const hca_bf16* s_new,
                             const int32_t* ctx_len, int S, int H, float scale, hca_bf16* wk,
                             hca_bf16* wv, hca_bf16* ws, hca_bf16* ck, hca_bf16* cv, int max_nc,
                             void* workspace, size_t ws_bytes, hca_bf16* out,
                             hca_stream_t stream);

/*
 * hca_quantize_e4m3 — FP8 storage of 512-wide bf16 rows (e.g. cache entries
 * and window rows for hca_decode_e4m3).
 *   The pages train with FP8 mixed precision and ship FP8 weights
 *   ('BaiduがERNIE 5.5 Flash Baseを公開' §3 and §5); the library stores a
 *   decode cache the same way.  Per row r:
 *     scale[r] = amax(|x[r, :]|) / 448            (fp32; 1 for an all-zero row)
 *     codes[r, c] = e4m3(x[r, c] / scale[r])      (fp32 division, round to
 *                                                   nearest even, saturating at
 *                                                   +-448)
 *   so the stored value is e4m3_value(codes) * scale.
 * Layout:  x [rows, 512] bf16 (16-byte aligned);  codes [rows, 512] bytes
 *          (16-byte aligned);  scale [rows] fp32.  Rows must be finite.
 * Errors:  rows < 0 or a null / misaligned pointer -> HCA_ERR_INVALID_ARG.
 */
hca_status_t hca_quantize_e4m3(const hca_bf16* x, long long rows, uint8_t* codes, float* scale,
                               hca_stream_t stream);

/*
 * hca_decode_e4m3 — hca_decode over an FP8 cache: the compressed entries and
 * the raw window rows stored by hca_quantize_e4m3 (half the bytes a decode
 * step streams).  The result is the HCA decode of the stored values
 * (code * row scale), as defined for hca_decode; q and g stay bf16, and q must
 * satisfy |q| < 65504 (the kernel runs its MMAs in f16: every e4m3 value and
 * every such bf16 value is exact in f16).
 * Layout:  q, g, out [S, 64, 512] bf16;  ck, cv [S, max_nc, 512] codes with
 *          ck_scale, cv_scale [S, max_nc] fp32;  wk, wv [S, 128, 512] codes (ring,
 *          slot = position mod 128) with wk_scale, wv_scale [S, 128] fp32;
 *          ctx_len [S] int32 on the device;  ws as for hca_decode (the same
 *          workspace serves both calls).
 * Errors:  as hca_decode; every scale pointer is required (ck / cv scales only
 *          when max_nc > 0).
 */
hca_status_t hca_decode_e4m3(const hca_bf16* q, const uint8_t* ck, const float* ck_scale,
                             const uint8_t* cv, const float* cv_scale, int max_nc,
                             const uint8_t* wk, const float* wk_scale, const uint8_t* wv,
                             const float* wv_scale, const int32_t* ctx_len, const hca_bf16* g,
                             int S, int H, float scale, void* ws, size_t ws_bytes, hca_bf16* out,
                             hca_stream_t stream);

/* ---------------------------------------------------------------------------
 * Paged cache
 *
 * The compressed entries of many sequences share one pool of pages, each of
 * `page_size` entries (16, 32, 64 or 128; an entry stands for 128 tokens).
 * Entry j of sequence i is row j % page_size of page
 * page_table[i][j / page_size].  The raw window of sequence i is row i of the
 * rings, as for hca_decode.  Rows of the pool behind a sequence's last entry,
 * ring slots without a token, other sequences' pages and table columns that no
 * entry needs may hold anything, NaN included.  A page number outside of the
 * pool where one is needed reads as zero rows (a write there is left out) and
 * is reported by hca_get_device_error() as HCA_ERR_DEVICE_INPUT.
 * ------------------------------------------------------------------------- */
typedef struct {
  hca_bf16* wk; /* [S, 128, 512] raw window rings (slot = position mod 128)    */
  hca_bf16* wv;
  hca_bf16* ws; /* [S, 128] their scores (not read by hca_paged_decode)        */
  hca_bf16* ck; /* [num_pages, page_size, 512] entry pools                     */
  hca_bf16* cv;
  const int32_t* page_table; /* row i at page_table + i * table_stride         */
  long long table_stride;    /* >= max_pages                                   */
  int max_pages;             /* columns                                        */
  int num_pages;
  int page_size;
} hca_paged_cache_t;

/*
 * hca_paged_append — append a chunk of new tokens per sequence to a paged cache
 *   (hca_cache_append for any number of tokens; same sources).
 *   Sequence i brings the tokens q_start[i] .. q_start[i + 1] - 1 (possibly
 *   none) of the packed inputs; ctx_len[i] counts them, so they sit at
 *   positions ctx_len[i] - n .. ctx_len[i] - 1.  Every block of 128 positions
 *   that they complete becomes an entry in its page, bit-identical to
 *   hca_compress of the whole sequence; the ring takes the newest tokens.
 *   q_start NULL: one token per sequence (N = S).
 * Layout:  k_new, v_new [N, 512] bf16;  s_new [N] bf16;  q_start [S + 1] and
 *          ctx_len [S] int32 on the device.  A page that is written must not
 *          be shared with another sequence (hca_pages_fork and, for a sequence
 *          that is cut, hca_pages_resize_copy see to that).
 * Errors:  HCA_ERR_INVALID_ARG for S < 1, N < 0, a NULL or misaligned pointer,
 *          q_start NULL with N != S; HCA_ERR_UNSUPPORTED for another page size
 *          or a table of more than 2^31 / 128 entries a row.  On the device:
 *          offsets that fall or leave 0 .. N, and lengths below the tokens
 *          brought or above 2^30, are clamped and reported.
 */
hca_status_t hca_paged_append(const hca_bf16* k_new, const hca_bf16* v_new, const hca_bf16* s_new,
                              const int32_t* q_start, const int32_t* ctx_len, int S, int N,
                              const hca_paged_cache_t* cache, hca_stream_t stream);

/*
 * hca_paged_prefill_workspace_size — bytes of scratch hca_paged_prefill needs
 * for up to S sequences with up to N new tokens in all.  Returns 0 for S < 1
 * or N < 1 or when the device cannot be asked.
 */
size_t hca_paged_prefill_workspace_size(int S, int N);

/*
 * hca_paged_prefill — hca_paged_append, and the attention of every new token
 *   over its sequence (chunked prefill, drafts of several tokens, mixed
 *   batches).  For the token at position t:
 *     keys = [entries 0 .. nc(t) - 1 ; raw keys max(0, t - 127) .. t]
 *     out  = sigmoid(g) * softmax(scale * keys . q) . values
 *   with nc(t) as above, then (vha_rank > 0) the head mix of hca_decode_vha.
 * Layout:  q, g, out [N, H, 512] bf16 (H = 64), packed as k_new; out shares no
 *          memory with q or g; rows before q_start[0] and from q_start[S] on
 *          are not written.  vha_down, vha_up [64, vha_rank] bf16
 *          (vha_rank = 0: none, may be NULL).  ws: at least
 *          hca_paged_prefill_workspace_size(S, N) bytes, 256-byte aligned,
 *          zero-filled before its first use (every call leaves it valid for
 *          the next, whatever its S and N); calls that overlap need one each.
 *          Tokens must be finite: one that is not may also reach outputs of
 *          its sequence, in this call or a later one, that give it no weight
 *          (zero times infinity is NaN); other sequences are not touched.
 * Errors:  those of hca_paged_append (q_start is required), of hca_decode_vha,
 *          and HCA_ERR_UNSUPPORTED for S > 4096 or (N + 144 S) * 64 >= 2^31.
 */
hca_status_t hca_paged_prefill(const hca_bf16* q, const hca_bf16* g, const hca_bf16* k_new,
                               const hca_bf16* v_new, const hca_bf16* s_new,
                               const int32_t* q_start, const int32_t* ctx_len, int S, int N, int H,
                               float scale, const hca_bf16* vha_down, const hca_bf16* vha_up,
                               int vha_rank, const hca_paged_cache_t* cache, hca_bf16* out,
                               void* ws, size_t ws_bytes, hca_stream_t stream);

/*
 * hca_paged_decode_workspace_size — bytes of scratch hca_paged_decode needs for
 * S sequences, zero-filled before its first use as for hca_decode.
 */
size_t hca_paged_decode_workspace_size(int S);

/*
 * hca_paged_decode — hca_decode (vha_rank > 0: hca_decode_vha) over a paged
 *   cache: one query per sequence, the cache already holding its token.
 *   Reads the cache only.  q, g, out [S, 64, 512], out apart from both; ws: at
 *   least hca_paged_decode_workspace_size(S) bytes, one call at a time.
 * Errors:  as hca_decode_vha and hca_paged_append; HCA_ERR_UNSUPPORTED for
 *          S > 65535.
 */
hca_status_t hca_paged_decode(const hca_bf16* q, const hca_bf16* g, const int32_t* ctx_len, int S,
                              int H, float scale, const hca_bf16* vha_down,
                              const hca_bf16* vha_up, int vha_rank,
                              const hca_paged_cache_t* cache, hca_bf16* out, void* ws,
                              size_t ws_bytes, hca_stream_t stream);

/*
 * hca_paged_decode_step — one serving step: hca_paged_append of one token per
 *   sequence, then hca_paged_decode; one launch for up to 512 sequences.
 */
hca_status_t hca_paged_decode_step(const hca_bf16* q, const hca_bf16* g, const hca_bf16* k_new,
                                   const hca_bf16* v_new, const hca_bf16* s_new,
                                   const int32_t* ctx_len, int S, int H, float scale,
                                   const hca_bf16* vha_down, const hca_bf16* vha_up, int vha_rank,
                                   const hca_paged_cache_t* cache, hca_bf16* out, void* ws,
                                   size_t ws_bytes, hca_stream_t stream);

/* ---------------------------------------------------------------------------
 * Pages
 *
 * Who owns the pages of a pool: page_table [rows, max_pages] int32 (row r:
 * the pages of a sequence in order, -1 behind them), n_pages [rows] and
 * ref [num_pages] (rows that name a page; 0 = free), all on the device.
 * Free pages are handed out lowest number first, in the order of the rows or
 * pairs, so results do not depend on timing.  ws: at least
 * hca_pages_workspace_size(rows, num_pages, n) bytes (n: list length, 0 where
 * there is none), 16-byte aligned, no initialisation; calls that overlap
 * need one each.  A call that may move 2^31 units of 16 KB (an item takes
 * whole units) or more is HCA_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t* page_table;
  long long table_stride; /* >= max_pages                                      */
  int rows, max_pages;
  int32_t* n_pages;
  int32_t* ref;
  int num_pages;
  int page_size; /* entries: 16, 32, 64 or 128                                 */
} hca_page_table_t;

/* An array of items (pages, or rows of a ring): item x at data + x * item_bytes. */
typedef struct {
  void* data;           /* 16-byte aligned                                     */
  long long item_bytes; /* a multiple of 16                                    */
} hca_page_array_t;

size_t hca_pages_workspace_size(int rows, int num_pages, int n);

/*
 * hca_pages_resize — give every row the pages of entries[r] entries
 *   (ceil(entries[r] / page_size); 0 frees the row, a negative number leaves
 *   it as it is).  Rows that shrink give up their last pages first (ref - 1);
 *   rows that grow then take free pages, row by row, while there are any:
 *   n_pages[r] afterwards tells what row r has.
 * Layout:  entries [rows] int32 on the device.
 * Errors:  HCA_ERR_INVALID_ARG / HCA_ERR_UNSUPPORTED on the host as above; on
 *          the device a row that would exceed max_pages is cut there, and
 *          inconsistent counts or page numbers are skipped, and reported.
 */
hca_status_t hca_pages_resize(const hca_page_table_t* table, const int32_t* entries, void* ws,
                              size_t ws_bytes, hca_stream_t stream);

/*
 * hca_pages_resize_copy — hca_pages_resize that leaves every row free to be
 *   appended to.  A row cut to a number of entries that ends inside a page
 *   which other rows name too (a branch cut below the place where it left its
 *   parent, or a parent below a branch) would go on writing into their page.
 *   Here it gets a fresh page, with the contents copied in each of the `pools`
 *   (as for hca_pages_fork), before any row grows; of rows that share such a
 *   page with nobody else, the last keeps it.
 * Errors:  those of hca_pages_resize, HCA_ERR_INVALID_ARG for n_pools < 1; on
 *          the device a row for which no page is free keeps the shared page,
 *          which is reported.
 */
hca_status_t hca_pages_resize_copy(const hca_page_table_t* table, const int32_t* entries,
                                   const hca_page_array_t* pools, int n_pools, void* ws,
                                   size_t ws_bytes, hca_stream_t stream);

/*
 * hca_pages_fork — branch sequences: the empty row children[i] becomes a copy
 *   of parents[i] cut at entries[i] entries.  Pages that are full are shared
 *   (ref + 1); the partly filled one is copied to a fresh page in each of the
 *   `pools` (arrays of num_pages items), and row parents[i] of each of the
 *   `rings` (arrays of `rows` items) to row children[i].
 *   ok[i] = 1 when the branch was made, 0 when no page was free for it.
 * Layout:  parents, children, entries, ok [n] int32 on the device; pools and
 *          rings are host arrays of at most 8 arrays together.
 * Errors:  host checks as above; n > 8192 or more arrays -> HCA_ERR_UNSUPPORTED.
 *          On the device a pair with a row out of range, a child that has
 *          pages, is a parent of this call or was named before, or a parent
 *          with fewer pages than the entries need, is left out (ok[i] = 0) and
 *          reported.
 */
hca_status_t hca_pages_fork(const hca_page_table_t* table, const int32_t* parents,
                            const int32_t* children, const int32_t* entries, int n,
                            const hca_page_array_t* pools, int n_pools,
                            const hca_page_array_t* rings, int n_rings, int32_t* ok, void* ws,
                            size_t ws_bytes, hca_stream_t stream);

/*
 * hca_pages_compact — close up a pool: with `live` pages in use, those
 *   numbered live and above move, in order, into the free ones below; the
 *   table and ref follow.  live (int32 on the device) receives the count:
 *   every page from there on is free.
 * Errors:  as above (at most 8 pools).
 */
hca_status_t hca_pages_compact(const hca_page_table_t* table, const hca_page_array_t* pools,
                               int n_pools, int32_t* live, void* ws, size_t ws_bytes,
                               hca_stream_t stream);

/*
 * hca_pages_copy — copy item src[i] to item dst[i] of every array, i < n
 *   (src, dst int32 on the device; items: number of items of the arrays).
 *   A source may be named often.  Left out and reported: items out of range,
 *   and every pair whose destination is named twice or is also a source.
 *   ws for hca_pages_workspace_size(1, items, n).
 */
hca_status_t hca_pages_copy(const hca_page_array_t* arrays, int n_arrays, int items,
                            const int32_t* src, const int32_t* dst, int n, void* ws,
                            size_t ws_bytes, hca_stream_t stream);

/*
 * hca_get_device_error — synchronises `stream`, then reads and clears the
 * device-side error word of the current device.  Returns HCA_OK,
 * HCA_ERR_TIMEOUT, HCA_ERR_DEVICE_INPUT or HCA_ERR_CUDA.  `where`, if not
 * NULL, receives an internal code naming the wait that gave up.
 * The error word is one per device for the whole process: every stream and
 * every host thread that launches this library's kernels on that device
 * records into it, and this call reads and clears it for all of them.  A
 * caller that drives one device from several threads or streams therefore
 * sees (and clears) errors of the others' launches too; serialise the checks
 * or attribute errors per device, not per stream.
 */
hca_status_t hca_get_device_error(hca_stream_t stream, unsigned int* where);

/*
 * hca_selftest_bounded_wait — launches one CTA that waits on an mbarrier
 * nobody arrives on, with a limit of `limit_us` microseconds (1 .. 10^7).
 * The kernel gives up, records HCA_ERR_TIMEOUT and exits normally; the
 * context stays usable.  Exists to test the failure path without faulting.
 */
hca_status_t hca_selftest_bounded_wait(int limit_us, hca_stream_t stream);

/* hca_status_string — static, human-readable name of a status code. */
const char* hca_status_string(hca_status_t status);

/* hca_version — library version as major*10000 + minor*100 + patch. */
int hca_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HCA_H */
