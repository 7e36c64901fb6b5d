/*
 * libkvq -- quantized KV cache with fused decode attention, for GB300 (sm_103a).
 *
 * C ABI.  Plain pointers and sizes only; no CUDA or framework types in the
 * signatures (a stream is passed as `void *`, meaning a cudaStream_t; NULL is
 * the legacy default stream).  Every device buffer is allocated and owned by
 * the caller; the library never allocates device or host memory.  Calls are
 * asynchronous on the given stream unless stated otherwise.
 *
 * Method (page title, section):
 *   [KIVI]   "大模型量化技术原理：KIVI、IntactKV、KVQuant" (juejin.cn), KIVI /
 *            背景 and 工作原理: keys quantized per channel in groups of G
 *            tokens, values per token; the newest tokens stay fp16 in a
 *            residual that is quantized and appended every R tokens.
 *   [HF]     pgsm.cn KV-cache quantization how-to, §2.1 (asymmetric form
 *            X_Q = round(X/S) - Z) and §3.1 (fp16 residual buffer, quantized
 *            as a batch when full).
 *   [INNERQ] "【论文】InnerQ：硬件感知免调优KV缓存量化用于大语言模型"
 *            (euno.news), 方法论 1-5: groups along the inner (head) dimension,
 *            per-group symmetric/asymmetric choice, fp16 sink and recent
 *            windows, dequantization fused into the GEMV.
 *   [KVQ5]   the juejin page, KVQuant / 技术原理 五: first token kept fp16.
 *   [IKV]    the juejin page, IntactKV / KV Cache量化: fp16 tokens joined
 *            with the dequantized cache at attention time.
 *
 * Quantization formula (asymmetric, fp32, IEEE round-to-nearest-even):
 *   scale = (max - min) / (2^b - 1), zero = min,
 *   code  = clamp(rint((x - min) / scale), 0, 2^b - 1); x_hat = code*scale + zero.
 *   A constant group stores scale 0 and code 0.
 * Symmetric (InnerQ groups whose midpoint |max + min| <= (max - min)/(2^b - 1)):
 *   scale = max(|min|, |max|) / (2^(b-1) - 1), q = clamp(rint(x / scale)),
 *   code = q + 2^(b-1), zero = -2^(b-1) * scale (same dequantization formula).
 *
 * Packed layout.  cap = max_ctx rounded up to a multiple of 128 is the
 * per-head token capacity.  Every per-token quantity of the quantized region
 * lives in 32-token blocks, so one contiguous read fetches everything a
 * 32-token tile needs except the KIVI key statistics for G >= 64.  M below is
 * f32, or fp16 under KVQ_META_F16 (m = its size in bytes, 4 or 2):
 *   blocks  u8 [B][H][cap/32][block_bytes]; block j of a head holds tokens
 *           32j .. 32j+31 (token t at row i = t mod 32) as
 *             K codes  [32][d*bits/8]    channel c of a row at bits
 *             V codes  [32][d*bits/8]    (c mod (8/bits))*bits of byte c/(8/bits)
 *             V scale  M [32][d/v_group]   (per token, channel group)
 *             V zero   M [32][d/v_group]
 *             InnerQ only:
 *             K scale  M [32][d/k_group]   (per token, channel group)
 *             K zero   M [32][d/k_group]
 *             KIVI with G <= 32 only:
 *             K stats  M [32/G][2][d]  per key group of the block: scale
 *                      row, then zero (= min) row, one value per channel
 *             KIVI with o = cfg.outliers > 0 only:
 *             K outliers u32 [32][o]  per token: (channel << 16) | fp16 bits
 *             V outliers u32 [32][o]  of its o outliers, channels ascending
 *           block_bytes = 64*d*bits/8 + 64*m*(d/v_group + (InnerQ ? d/k_group : 0))
 *                         + (KIVI, G <= 32 ? (32/G)*2*m*d : 0) + 256*o,
 *           a multiple of 128.
 *           KVQ_INNERQ_KNORM: the blocks buffer ends with the key factors
 *             f32 [B][H][d] (n_c above), after the last head's blocks.
 *   KIVI with G >= 64:
 *           k_meta  M [B][H][cap/G][2][d]  the same two rows per key group
 *           (the buffer carries 64 bytes of slack after the last head)
 *   KIVI:   k_res, v_res   fp16 [B][H][R][d]  residual, oldest first; with
 *                           KVQ_VALUE_QUEUE, v_res is a ring: the fp16 value
 *                           of token t sits in slot t mod R
 *   InnerQ: k_mode, v_mode  u32 [B][H][cap*(d/group)/32]  bit i = group
 *                           i % (d/group) of token i / (d/group); 1 = symmetric
 *           k_res, v_res   fp16 [B][H][W][d]   recent window, a ring (see ring_head)
 *           k_sink, v_sink fp16 [B][H][S][d]   first S tokens
 *   KVQ_RAGGED: seq_prompt int32 [B]  each sequence's prompt length
 *   Quantized tokens occupy slots [0, n_quant) in arrival order.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes.  Validation happens before any launch; on a negative return
 * no cache state (host counters or device buffers) has changed. */
#define KVQ_OK 0
#define KVQ_EINVAL (-1)       /* null pointer, negative size, inconsistent config */
#define KVQ_EUNSUPPORTED (-2) /* valid but not built: head_dim, bits, group sizes */
#define KVQ_ECAPACITY (-3)    /* the call would exceed max_ctx, the pages or the workspace */
#define KVQ_EALIGN (-4)       /* a device buffer is not 16-byte aligned */
#define KVQ_ECUDA (-5)        /* a CUDA launch or copy failed */
#define KVQ_ETIMEOUT (-6)     /* a bounded device-side wait gave up (status word) */
#define KVQ_EPAGE (-7)        /* a token's page is not in the block table (status word) */

#define KVQ_KIVI 0
#define KVQ_INNERQ 1
#define KVQ_INNERQ_KNORM 2 /* InnerQ with the one-shot per-channel key normalization */

/* Cache-format options (kvq_config.flags). */
#define KVQ_META_F16 1u    /* scales and zero points stored in fp16 */
#define KVQ_VALUE_QUEUE 2u /* KIVI: values leave the fp16 residual one at a time */
#define KVQ_RAGGED 4u      /* every sequence of the batch has its own length */

/*
 * Cache configuration.
 *   batch, n_q_heads, n_kv_heads: n_q_heads % n_kv_heads == 0; query head hq
 *     reads KV head hq / (n_q_heads / n_kv_heads) (GQA; MHA when equal).
 *   head_dim d: 64 or 128.   bits: 2 or 4.
 *   scheme KVQ_KIVI: k_group = G tokens per key group (16, 32, 64 or 128),
 *     v_group = channels per value group (multiple of 16 dividing d),
 *     residual = R (multiple of G, <= 1024), n_sink must be 0.
 *   scheme KVQ_INNERQ: k_group and v_group = channels per group (multiples of
 *     16 dividing d), residual = W recent fp16 tokens (0..1024), n_sink = S
 *     fp16 sink tokens (0..1024).
 *   scheme KVQ_INNERQ_KNORM: KVQ_INNERQ plus the one-shot per-channel key
 *     normalization ("InnerQ" paper summary, key contributions and
 *     methodology 4: keys scaled once per channel at prefill, the factor
 *     folded into the query).  kvq_quantize_prefill sets the factor n_c of
 *     channel c of every head to the largest |K[t][c]| over the T prompt
 *     tokens (1 if that is 0 or T = 0); every key that is quantized (now or
 *     when it later leaves the window) is first multiplied, in fp32, by
 *     r_c = 1 / n_c (fp32 division); decode multiplies q by n_c for the
 *     quantized tokens.  Sinks and window stay the raw fp16 keys.
 *   max_ctx: most tokens one sequence will hold (prompt + appended), at most
 *     2^30 (KVQ_EUNSUPPORTED above).
 *   flags: any of
 *     KVQ_META_F16 (pgsm.cn how-to §3.1 stores the residual design without
 *       fixing the statistics' precision): the fp32 scale and zero of the
 *       formula are each rounded once to fp16 (IEEE nearest-even) and the
 *       codes are taken with the stored values, code = clamp(rint((x -
 *       zero16) / scale16)) (symmetric: q = clamp(rint(x / scale16)), zero =
 *       -2^(b-1) * scale16), so dequantization uses exactly what is stored; a
 *       scale that rounds to 0 is a constant group.  Needs |x| small enough
 *       that every stored value is finite (|x| <= 8192 covers every case).
 *     KVQ_VALUE_QUEUE (KIVI only; [KIVI] 工作原理, value paragraph: the
 *       newest values wait in a queue, and once it reaches R the oldest is
 *       quantized): after n tokens the last min(n, R - 1) values are fp16 and
 *       the first max(0, n - R + 1) are quantized per token; keys still flush
 *       every R tokens.
 *     KVQ_RAGGED: sequences have their own prompt lengths
 *       (kvq_quantize_prefill_ragged); every append adds one token to every
 *       sequence.
 *   outliers (KIVI only; "大模型量化技术原理", KVQuant / 技术原理 四: per
 *     vector, the outliers are kept apart in fp16 and the rest quantized over
 *     the narrower range): o in 0..8.  Each token's o largest-magnitude key
 *     elements and o largest value elements (equal magnitudes: the lower
 *     channel) are kept as (channel, fp16) lists; the statistics of every key
 *     group (each channel over its G tokens) and value group come from the
 *     other elements only (none left: scale 0, zero 0), outlier positions
 *     store code 0, and decode uses the fp16 value there.
 */
typedef struct kvq_config {
  int32_t batch;
  int32_t n_q_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t bits;
  int32_t scheme;
  int32_t k_group;
  int32_t v_group;
  int32_t residual;
  int32_t n_sink;
  int64_t max_ctx;
  uint32_t flags;
  int32_t outliers;
} kvq_config;

/* Byte sizes of the cache buffers for a configuration (0 = unused). */
typedef struct kvq_sizes {
  size_t blocks;  /* 32-token blocks of codes and per-token statistics */
  size_t k_meta;  /* KIVI key statistics for G >= 64 (0 otherwise) */
  size_t k_mode, v_mode;
  size_t k_res, v_res;
  size_t k_sink, v_sink;
  size_t status;     /* one int32 status word */
  size_t seq_prompt; /* KVQ_RAGGED: int32 per sequence (0 otherwise) */
} kvq_sizes;

/*
 * Cache view.  The caller allocates every buffer (sizes from kvq_cache_sizes,
 * 16-byte aligned), zero-fills `dev_status` once, and keeps this struct; the
 * library updates the host counters below.  Copying the struct together with
 * the buffers checkpoints the cache.
 *   n_quant   tokens in the quantized region (slots [0, n_quant))
 *   n_resid   KIVI: fp16 residual tokens (< R); InnerQ: window tokens (<= W)
 *   n_sink    InnerQ: sink tokens held (<= S)
 *   ring_head InnerQ: window slot of the oldest token once the window is full
 *   n_appended  tokens appended to every sequence since the prefill
 * Without KVQ_RAGGED lengths are uniform across the batch and the counters
 * describe every sequence.  With KVQ_RAGGED they describe the longest
 * sequence (capacity checks and launch sizes use them); sequence b holds
 * seq_prompt[b] + n_appended tokens, and its own counters follow from that
 * length exactly as a uniform cache's would (the device reads seq_prompt).
 * Every call except the prefills (which reset them) first checks that the
 * counters describe a reachable state (n_sink <= S, n_resid <= R or W, KIVI
 * n_resid < R and n_quant a multiple of R, ring_head < W, n_quant <=
 * capacity, all tokens <= max_ctx, n_appended <= all tokens) and returns
 * KVQ_EINVAL otherwise.
 */
typedef struct kvq_cache {
  void *blocks;
  void *k_meta;
  uint32_t *k_mode, *v_mode;
  uint16_t *k_res, *v_res, *k_sink, *v_sink;
  int64_t n_quant, n_resid, n_sink, ring_head;
  int32_t *dev_status;
  int32_t *seq_prompt; /* KVQ_RAGGED: device int32 [B], written by the prefill */
  int64_t n_appended;
} kvq_cache;

/* Fills *out with the byte size of each cache buffer.  Returns KVQ_OK,
 * KVQ_EINVAL or KVQ_EUNSUPPORTED.  Host only, no CUDA call. */
int kvq_cache_sizes(const kvq_config *cfg, kvq_sizes *out);

/* Bytes of scratch (device) that kvq_decode_attention needs for any cache
 * state of this configuration.  The scratch must be zero-filled before its
 * first use; every decode call that succeeds leaves it zero again.  It must
 * not be shared by decode calls that can run at the same time. */
int kvq_workspace_bytes(const kvq_config *cfg, size_t *bytes);

/*
 * Prefill: quantize a prompt of T tokens into an empty cache.
 * K, V: device fp16 [B][H][T][d], contiguous.  Resets the cache counters.
 * KIVI ([KIVI] 工作原理): tokens [0, T - T mod R) are quantized (keys per
 *   channel in groups of G tokens, values per token in groups of v_group
 *   channels); the last T mod R tokens go to the fp16 residual.
 * InnerQ ([INNERQ] 方法论 1-4): the first min(S, T) tokens go to the sink,
 *   the last min(W, T - S) to the window, the rest are quantized per token in
 *   groups of k_group / v_group channels with a per-group mode.
 *   KVQ_INNERQ_KNORM: the per-channel key factors are computed first over all
 *   T tokens and the quantized keys are normalized by them (see the scheme).
 * Errors: KVQ_EINVAL (null, T < 0), KVQ_ECAPACITY (T > max_ctx), KVQ_EALIGN,
 *   KVQ_EUNSUPPORTED, KVQ_ECUDA.
 */
int kvq_quantize_prefill(const kvq_config *cfg, kvq_cache *cache, const uint16_t *K,
                         const uint16_t *V, int64_t T, void *stream);

/*
 * Prefill of sequences with their own prompt lengths (KVQ_RAGGED; pgsm.cn
 * how-to §3.1 keeps a residual per sequence).  K, V: device fp16
 * [B][H][T_max][d], sequence b's prompt in rows [0, lens[b]) (later rows are
 * not read).  lens: HOST int32 [B], 0 <= lens[b] <= T_max <= max_ctx, copied
 * to cache->seq_prompt on `stream` (a pageable host copy: the call returns
 * once lens is no longer needed).  Each sequence is quantized exactly as
 * kvq_quantize_prefill quantizes a prompt of its length; the host counters
 * then describe the longest one.  kvq_quantize_prefill on a KVQ_RAGGED cache
 * gives every sequence the length T.
 * Errors: as kvq_quantize_prefill; KVQ_EINVAL without KVQ_RAGGED.
 */
int kvq_quantize_prefill_ragged(const kvq_config *cfg, kvq_cache *cache, const uint16_t *K,
                                const uint16_t *V, int64_t T_max, const int32_t *lens,
                                void *stream);

/*
 * Append one decode token per (batch, kv head).  k, v: device fp16 [B][H][d].
 * KIVI ([KIVI] 工作原理; [HF] §3.1): the token enters residual slot n_resid;
 *   when the residual reaches R tokens the same launch quantizes all R of them
 *   to slots [n_quant, n_quant + R) and empties the residual.
 * InnerQ: the sink fills first, then the window; once the window holds W
 *   tokens its oldest token is quantized to slot n_quant (normalized by the
 *   prompt's key factors under KVQ_INNERQ_KNORM) and the new token takes its
 *   ring slot.
 * Errors: KVQ_EINVAL, KVQ_ECAPACITY (total tokens would exceed max_ctx),
 *   KVQ_EALIGN, KVQ_ECUDA.
 */
int kvq_append(const kvq_config *cfg, kvq_cache *cache, const uint16_t *k,
               const uint16_t *v, void *stream);

/*
 * Fused decode attention over the packed cache ([KIVI] 背景: each decode
 * step reads the whole cache; [INNERQ] 方法论 3: dequantization folded into
 * the q.K^T and P.V GEMVs; [IKV]: fp16 sink / residual tokens joined with
 * the quantized ones by an online-softmax merge).
 *   q:   device fp16 [B][n_q_heads][d]
 *   out: device fp32 [B][n_q_heads][d] = softmax(softmax_scale * q.K^T) V over
 *        every token held (sink, quantized, residual / window).  An empty
 *        cache yields zeros.
 *   ws:  device scratch of ws_bytes >= kvq_workspace_bytes (see there).
 * A decode step is kvq_append followed by kvq_decode_attention.
 * Errors: KVQ_EINVAL, KVQ_ECAPACITY (ws too small), KVQ_EALIGN, KVQ_ECUDA.
 */
int kvq_decode_attention(const kvq_config *cfg, const kvq_cache *cache, const uint16_t *q,
                         float *out, float softmax_scale, void *ws, size_t ws_bytes,
                         void *stream);

/*
 * Decode attention over keys cached BEFORE the rotary position embedding
 * ("大模型量化技术原理：KIVI、IntactKV、KVQuant", KVQuant / 技术原理 二: keys
 * are quantized pre-RoPE, and the embedding is applied after dequantization
 * inside the q.K^T kernel).  The cache holds the keys exactly as they were
 * given to kvq_quantize_prefill / kvq_append (un-rotated); q is un-rotated
 * too.  RoPE (RoFormer's rotation; the pages do not spell it out): channels
 * 2i and 2i+1 of a vector at position p are turned counter-clockwise by the
 * angle p * theta_i, theta_i = rope_base^(-2i/d).  Positions: the tokens held
 * are numbered 0, 1, ... in arrival order (sinks, quantized tokens,
 * residual / window oldest first), and q belongs to the newest token.
 *   out = softmax(softmax_scale * RoPE(q) . RoPE(K)^T) V, fp32, as
 *   kvq_decode_attention (values are not rotated; an empty cache gives zeros).
 *   ws: the decode scratch (kvq_workspace_bytes; zero-filled, left zero).
 * Errors: as kvq_decode_attention; KVQ_EINVAL for rope_base <= 0 or not
 *   finite; KVQ_EUNSUPPORTED for n_q_heads / n_kv_heads = 8, max_ctx > 2^24
 *   (positions are exact in fp32), or any kvq_config.flags / outliers option.
 */
int kvq_decode_attention_rope(const kvq_config *cfg, const kvq_cache *cache, const uint16_t *q,
                              float *out, float softmax_scale, double rope_base, void *ws,
                              size_t ws_bytes, void *stream);

/*
 * One decode step on device buffers: kvq_append(k, v) then
 * kvq_decode_attention(q) with the same arguments, results and errors.  When
 * the append only stores the new token (KIVI without a flush) and the decode
 * runs on the tensor-core path (head_dim 128, MHA), both happen in ONE kernel
 * launch: the decode reads the new token's rows from k, v directly and stores
 * them into the residual; otherwise it is the two launches.
 */
int kvq_append_decode(const kvq_config *cfg, kvq_cache *cache, const uint16_t *k,
                      const uint16_t *v, const uint16_t *q, float *out, float softmax_scale,
                      void *ws, size_t ws_bytes, void *stream);

/*
 * One decode step from HOST buffers, with one copy in and one copy out.
 *   h_in:  host fp16, the step's inputs back to back: k [B][H][d], then
 *          v [B][H][d], then q [B][n_q_heads][d] (2*B*H*d + B*n_q_heads*d
 *          halves).
 *   d_in:  device staging buffer of the same layout and size (16-byte aligned).
 *   h_out: host fp32 [B][n_q_heads][d]; d_out: its device staging buffer.
 * Enqueued on `stream`, no synchronization: one host-to-device copy of h_in,
 * kvq_append_decode on the staged rows, one device-to-host copy of the output.
 * Host buffers should be pinned for the copies to be asynchronous.  Errors:
 * as kvq_append_decode; KVQ_ECUDA when a copy fails to enqueue.
 */
int kvq_decode_step_host(const kvq_config *cfg, kvq_cache *cache, const uint16_t *h_in,
                         float *h_out, uint16_t *d_in, float *d_out, float softmax_scale,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * Decode attention that allocates nothing, not even its scratch.  The pages
 * have no counterpart: this is a deployment convenience of the library.
 *
 * For callers that cannot hand the library a device buffer for scratch: code
 * that runs where no device allocator may be called (a plugin or callback
 * handed only its input and output tensors, a real-time or certified path
 * that forbids run-time device allocation, a process whose device memory is
 * entirely owned by another pool).  Same arguments, result and errors as
 * kvq_decode_attention minus ws / ws_bytes.
 *
 * The scratch is one file-scope device array of KVQ_NOALLOC_SCRATCH_BYTES
 * (16 MiB) that every GPU which loads the library holds until the process
 * exits.  Configurations whose kvq_workspace_bytes exceeds it are rejected
 * with KVQ_ECAPACITY; every other check of kvq_decode_attention runs too, and
 * a rejected call enqueues nothing and leaves the array alone.  The first call
 * on a device (with that device current) looks up the array's device address
 * with cudaGetSymbolAddress and keeps it; make that first call before any
 * stream capture.  Only the device's primary context (the CUDA runtime's) is
 * supported: the kept address is not valid in another context, nor after
 * cudaDeviceReset.  Each call clears the part of the scratch its
 * configuration uses (an asynchronous memset of kvq_workspace_bytes on
 * `stream`), then launches the decode, so a call that stopped early (a
 * timeout) leaves nothing behind for the next one.  All calls share the one
 * array: calls whose work can overlap on the GPU (different streams,
 * different caches) race and give wrong results; serialize them.
 */
#define KVQ_NOALLOC_SCRATCH_BYTES (16u << 20)
int kvq_decode_attention_noalloc(const kvq_config *cfg, const kvq_cache *cache,
                                 const uint16_t *q, float *out, float softmax_scale,
                                 void *stream);

/* Synchronizes `stream`, reads and clears the cache's device status word.
 * Returns KVQ_OK, or the error a kernel recorded (KVQ_ETIMEOUT), or KVQ_ECUDA. */
int kvq_get_device_status(kvq_cache *cache, void *stream);

/* Debug switch for the failure path of the decode kernel's bounded waits.
 * Every wait of the shared-memory pipeline gives up after a fixed poll cap
 * (2^24 polls, about a second or more), records KVQ_ETIMEOUT in the status
 * word, waits (bounded) for the block's own copies in flight and returns.
 * With iterations > 0, each block of later tensor-core decode launches first
 * waits, with that cap, on a barrier that nothing completes, so the timeout
 * path runs for certain; 0 switches it off.  After a timeout the output and
 * the workspace are undefined: zero-fill the workspace again.
 * Process-wide; not for production use. */
void kvq_debug_stall_waits(int64_t iterations);

/* Name of the decode kernel, with its template arguments, that
 * kvq_decode_attention launches for this configuration when n_quant tokens
 * are quantized (e.g. "tc_decode_kernel<bits=2,scheme=kivi,ngv=4,ngk=1,km=1>"),
 * written NUL-terminated into buf[len].  Host only, no CUDA call.  Returns
 * KVQ_OK, KVQ_EINVAL (null, n_quant < 0, buf too small) or a config error. */
int kvq_decode_kernel_name(const kvq_config *cfg, int64_t n_quant, char *buf, size_t len);

/* The same for kvq_decode_attention_rope (e.g.
 * "tc_decode_kernel<bits=2,scheme=kivi,ngv=4,km=1,rope=1>": the tensor-core
 * form, taken for head_dim 128, one query head per KV head, KIVI with key
 * groups of 32 or more and no cache options; other shapes name
 * "rope_decode_kernel<...>").  Host only, no CUDA call; same returns. */
int kvq_rope_kernel_name(const kvq_config *cfg, int64_t n_quant, char *buf, size_t len);

/* ---- Paged cache ---------------------------------------------------------
 *
 * A cache whose tokens live in fixed-size pages, for serving: sequences grow,
 * end and share prefixes without moving data.  A sequence is a row of a block
 * table (its pages in order), so several sequences may name the same page to
 * read it.  Every token is quantized as it is written, per token and head in
 * groups of 32 channels, keys and values alike: there is no fp16 residual and
 * no per-sequence state beyond the lengths, which the caller keeps on the
 * device.  The calls read lengths and tables on the device only, so a captured
 * CUDA graph follows them from replay to replay.
 *
 * Stored form (b bits, per group of 32 channels of one token and head; x the
 * 16-bit input, infinities and |x| > 32768 saturated to +-32768, NaN taken as
 * 0, so the cache holds finite values only):
 *   scale = fp16((max - min) / (2^b - 1)), zero = fp16(min),
 *   code  = clamp(rint((x - zero) / scale), 0, 2^b - 1), 0 where scale is 0,
 *   x_hat = code * scale + zero          (fp32; each rounding to nearest even)
 *
 * Layout.  pages u8 [n_pages][n_kv_heads][page_size/16][atom]; an atom holds
 * 16 consecutive tokens of one head, rb = d*b/8 bytes of codes per row:
 *   K codes [16][rb], V codes [16][rb],
 *   K statistics fp16 [16][2][d/32], V statistics fp16 [16][2][d/32]
 *     (per token the scales of its groups, then their zeros)
 *   atom = 32 * (rb + 4*d/32) bytes.
 * Within a row the codes are permuted so that a tensor-core fragment is a
 * plain load.  Slot s of a row is its bits [s*b, (s+1)*b) (little endian):
 *   K: channel 32*G + 8*j + 2*k + e (j, k in 0..3, e in 0..1) sits in 32-bit
 *      word floor(p*b/16) of quarter j of the row, p = 4*G + k, at bit
 *      (p*b mod 16) + 16*e;
 *   V: channel 32*(2*h + e) + 4*g + i (g in 0..7, i in 0..3) sits in eighth g
 *      of the row, p = 4*h + i, in its unit floor(p*b/w) of 2*w bits at bit
 *      (p*b mod w) + w*e, w = 16 (8 when d = 64, b = 2).
 */
#define KVQ_F16 0
#define KVQ_BF16 1
#define KVQ_F32 2 /* logits only */

/*
 *   n_q_heads, n_kv_heads: n_q_heads = r * n_kv_heads, 1 <= r <= 128; query
 *     head hq reads KV head hq / r.
 *   head_dim d: 64 or 128.  bits: 2, 4 or 8.  page_size: tokens per page, 16,
 *     32, 64, 128 or 256.  dtype: type of keys, values, queries and outputs.
 *   n_pages: pages in the pool.
 */
typedef struct kvq_paged_config {
  int32_t n_q_heads, n_kv_heads, head_dim, bits, page_size, dtype;
  int64_t n_pages;
} kvq_paged_config;

/* Caller's buffers: the pages (kvq_paged_cache_bytes, 16-byte aligned; pages
 * need no initial value) and one int32 status word, zero-filled once. */
typedef struct kvq_paged_cache {
  void *pages;
  int32_t *dev_status;
} kvq_paged_cache;

/*
 * One call's sequences.  Device arrays:
 *   block_table int32 [n_seqs][table_width]  page of tokens [i*page_size,
 *     (i+1)*page_size) of sequence b at [b][i]; entries behind a sequence's
 *     last page are not read
 *   seq_lens    int32 [n_seqs]   tokens sequence b holds, the call's included
 *   cu_tokens   int32 [n_seqs+1] the call's rows [cu[b], cu[b+1]) belong to
 *     sequence b and are its LAST n_b = cu[b+1] - cu[b] tokens: row cu[b] + i
 *     is position seq_lens[b] - n_b + i.  cu[0] = 0, not decreasing.
 * Host values: n_seqs (1..2048), table_width, n_tokens = rows of the packed
 * arrays (rows from cu[n_seqs] on are padding: never read, never written),
 * max_tokens >= every n_b.
 * What the device arrays say is checked there: a row at a negative position
 * is skipped (write), reads as zeros (read), attends to nothing (attention);
 * a token whose page entry lies outside [0, n_pages) or behind table_width is
 * skipped, reads as zeros or is not attended to, and KVQ_EPAGE goes to the
 * status word; a sequence with more than max_tokens rows, with rows behind
 * n_tokens, or whose cu_tokens decrease, is not attended for and gives
 * KVQ_EINVAL there.
 */
typedef struct kvq_paged_batch {
  const int32_t *block_table, *seq_lens, *cu_tokens;
  int64_t table_width, n_tokens;
  int32_t n_seqs, max_tokens;
} kvq_paged_batch;

/* Bytes of the page pool, and of one page (out parameters may be null).
 * Returns KVQ_OK, KVQ_EINVAL or KVQ_EUNSUPPORTED.  Host only. */
int kvq_paged_cache_bytes(const kvq_paged_config *cfg, size_t *pool, size_t *page);

/* Bytes of scratch kvq_paged_attention needs (any batch).  Zero-fill it once;
 * every call leaves what must be zero at zero again, unless a wait ran out
 * (KVQ_ETIMEOUT in the status word): zero-fill it then.  Calls that can run at
 * the same time need scratch of their own. */
int kvq_paged_workspace_bytes(const kvq_paged_config *cfg, size_t *bytes);

/*
 * Quantize the call's tokens into their pages.  k, v: device, row t of head h
 * at k + t*k_stride + h*head_dim (dtype elements; strides in elements, at
 * least n_kv_heads*head_dim, multiples of 8), so a slice of a fused q-k-v
 * projection can be given as it is.  Each written token must have a slot of
 * its own: where two rows of a call name one slot (a page shared by two
 * sequences that both write to it) that slot holds a mixture of the two.
 * Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EALIGN, KVQ_ECUDA.
 */
int kvq_paged_write(const kvq_paged_config *cfg, kvq_paged_cache *cache,
                    const kvq_paged_batch *batch, const void *k, int64_t k_stride, const void *v,
                    int64_t v_stride, void *stream);

/*
 * Read the call's tokens back: x_hat rounded once to dtype, k_out and v_out
 * [n_tokens][n_kv_heads][head_dim] contiguous, apart from each other.
 * cu_tokens = running sums of seq_lens reads whole sequences.  Errors as
 * kvq_paged_write.
 */
int kvq_paged_read(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                   const kvq_paged_batch *batch, void *k_out, void *v_out, void *stream);

/*
 * Causal attention of the call's rows over the pages: row i of sequence b, at
 * position p = seq_lens[b] - n_b + i, sees the sequence's tokens 0..p (its own
 * included: write first).  One row per sequence is a decode step; chunks of
 * any length, and batches that mix both, are one call.
 *   q: device, row t of query head h at q + t*q_stride + h*head_dim
 *   out [n_tokens][n_q_heads][head_dim], contiguous, dtype, apart from q:
 *     softmax(softmax_scale * q.K^T) V; zeros for a row that sees nothing.
 *   softmax_scale: any finite number.  A score (times log2 e) of 2^23 or more in
 *     magnitude, or a bf16 query beyond 2^90, may make its row NaN: fp32 no longer
 *     tells such scores apart.  A query with a NaN or an infinity makes its own
 *     row and head NaN and no other.
 *   ws: device scratch, ws_bytes >= kvq_paged_workspace_bytes.
 * Arithmetic: scores, weights' sums and outputs are held in fp32; the operands
 * of the two products are rounded to fp16.  A sequence's rows are its tokens in
 * the call times r, the query heads of a KV head.  Few rows are at most 8, or at
 * most 16 where r > 8 or max_tokens * r <= 16 (so the rounding of a sequence with
 * 9 to 16 rows depends on max_tokens).  With few rows the rounded operands are the
 * query (relative to the largest of its row) and each weight times its value's
 * scale, with more the query, the weights and the keys and values x_hat.
 * fp16's range costs what is small beside something large: of few rows a weight
 * times scale below 2^-25 of the largest such product is off by up to 2^-36 of
 * it; of more rows a weight below 2^-18 of the row's largest by up to 2^-29 of
 * it, and an x_hat below 2^-14 by up to 2^-25.
 * Measured over 1900 calls of mixed shapes (normal keys with a few channels 8
 * times larger, fp16; norm of a call's error over the norm of its output): few
 * rows up to 5.0e-4, in the median 2.8e-4; more rows up to 1.6e-3, in the median
 * 4.7e-4, single rows of those up to 7.4e-3.  The output's own rounding is 2.1e-4
 * of that; to bf16 it alone is 1.7e-3.
 * Errors: as kvq_paged_write; KVQ_EINVAL also where q and out overlap;
 *   KVQ_ECAPACITY (ws too small).
 */
int kvq_paged_attention(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                        const kvq_paged_batch *batch, const void *q, int64_t q_stride, void *out,
                        float softmax_scale, void *ws, size_t ws_bytes, void *stream);

/*
 * Cross attention of the call's rows over the pages: every row of sequence b sees
 * all seq_lens[b] tokens (an encoder's states, written once), whatever the number
 * of its rows, which may be larger: the rows are no tokens of the sequence.  Rows
 * that read the same states (beams, samples) go in as rows of one sequence and
 * share its reads.  Arguments, arithmetic (fp16 operands, with their errors), results
 * and errors are otherwise those of kvq_paged_attention; a sequence without tokens
 * gives its rows zeros, one longer than its table ends with that (KVQ_EPAGE).
 */
int kvq_paged_cross_attention(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                              const kvq_paged_batch *batch, const void *q, int64_t q_stride,
                              void *out, float softmax_scale, void *ws, size_t ws_bytes,
                              void *stream);

/*
 * Copy pages inside the pool.  copies: device int32 [n_copies][2], 8-byte aligned:
 * pairs (from, to), ended by n_copies or by the first pair whose `from` is
 * negative.  Pairs run in no order: a page may be copied to several others, but no
 * `to` is named twice or is another pair's `from`.  A pair that names a page
 * outside [0, n_pages) is skipped and gives KVQ_EPAGE in the status word.  Whole
 * pages are copied, slots without tokens too.
 * Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EALIGN, KVQ_ECUDA.
 */
int kvq_paged_copy(const kvq_paged_config *cfg, kvq_paged_cache *cache, const int32_t *copies,
                   int64_t n_copies, void *stream);

/* Synchronizes `stream`, reads and clears the status word; KVQ_OK, or what a
 * kernel recorded there, or KVQ_ECUDA.  Of several errors it holds the first
 * (KVQ_EPAGE, KVQ_EINVAL), but KVQ_ETIMEOUT before either. */
int kvq_paged_status(kvq_paged_cache *cache, void *stream);

/* The same for any status word. */
int kvq_read_status(int32_t *dev_status, void *stream);

/* ---- Page tables ----------------------------------------------------------
 *
 * Who holds which page, kept on the device: pages for a step's new tokens, copies
 * of shared pages before they are written, tokens taken back, sequences forked,
 * reordered and ended, the pool made compact.  One set of tables serves the page
 * pools of all layers: the tables change once a step, and the copies they ask for
 * (kvq_paged_copy) run in every pool.  Nothing is read back by the host, so a step
 * with all of these calls can be captured in a CUDA graph.
 *
 *   block_table, seq_lens: as in kvq_paged_batch, for n_seqs slots (1..2048).  A
 *     sequence of n tokens holds ceil(n / page_size) entries; those behind them are
 *     -1.  A slot without tokens is free.
 *   page_refs int32 [n_pages]: how many entries of all tables name each page; 0 is
 *     a free page.
 *   state: kvq_pages_state_bytes of device memory, 16-byte aligned: the free pages'
 *     map and scratch of the calls.
 *   dev_status: an int32 status word, zero-filled once.
 *   n_pages: 1..2^26.  page_size: 16, 32, 64, 128 or 256.
 * The buffers are the caller's.  kvq_pages_recount has to run before any other
 * call, and again after the caller has written to tables or lengths itself.  Calls
 * on one table never run at the same time.
 *
 * What the device arrays say is checked there, and goes to the status word: an
 * entry that is no page (KVQ_EPAGE, skipped), a negative length (KVQ_EINVAL) or one
 * beyond the table (KVQ_EPAGE; such a sequence stays as it is, and none becomes it),
 * holder counts that do not agree with the tables (KVQ_EINVAL).
 * Every call returns KVQ_OK, KVQ_EINVAL (null, sizes), KVQ_EUNSUPPORTED, KVQ_EALIGN
 * or KVQ_ECUDA, and what is said there.
 */
typedef struct kvq_page_table {
  int32_t *block_table, *seq_lens, *page_refs;
  void *state;
  int32_t *dev_status;
  int64_t n_pages, table_width;
  int32_t n_seqs, page_size;
} kvq_page_table;

/* Bytes of `state`; only the sizes of *table are looked at.  Host only. */
int kvq_pages_state_bytes(const kvq_page_table *table, size_t *bytes);

/* Count the holders of every page from block_table and seq_lens (all zero: an
 * empty pool), and set entries behind a sequence's last to -1. */
int kvq_pages_recount(const kvq_page_table *table, void *stream);

/*
 * Pages for new tokens: sequence b is about to get n_b = cu_tokens[b+1] -
 * cu_tokens[b] more (0: left alone), seq_lens[b] grows by them, and its table gets
 * the pages they need, the lowest-numbered free ones first, by sequence and entry.
 * A partly filled last page that others hold too is copied before it is written:
 * the sequence gets a page of its own (the first of its new ones).  Of sequences
 * that get tokens in this call and are all the holders of such a page, the first
 * keeps it.
 *   cu_tokens int32 [n_seqs+1], as in kvq_paged_batch.
 *   copies int32 [n_seqs][2], 8-byte aligned: the copies to make before the tokens
 *     are written, for kvq_paged_copy; (-1, -1) behind the last.
 *   cu_call int32 [n_seqs+1], apart from cu_tokens: cu_tokens again, or zeros where
 *     the call failed; given as cu_tokens to every call of the step that follows
 *     (kvq_paged_write, kvq_paged_attention, kvq_paged_cross_attention,
 *     kvq_verify_drafts), it makes a failed step write, attend to and judge nothing,
 *     so that no token is dropped that was not reserved.
 * All or nothing: where pages (KVQ_ECAPACITY) or table entries (KVQ_ECAPACITY) do
 * not suffice or the arrays are wrong (KVQ_EINVAL, KVQ_EPAGE), the status word says
 * so, nothing changes and there are no copies.
 */
int kvq_pages_reserve(const kvq_page_table *table, const int32_t *cu_tokens, int32_t *copies,
                      int32_t *cu_call, void *stream);

/* Take back the newest tokens[b] (device int32 [n_seqs]) tokens of every sequence
 * (none where <= 0, all where as many or more: the sequence ends), and let go of
 * the pages that hold nothing else of it. */
int kvq_pages_drop(const kvq_page_table *table, const int32_t *tokens, void *stream);

/* Sequence b becomes what sequence parents[b] (device int32 [n_seqs]) was before
 * the call: b itself stays, -1 empties b, others fork or reorder; the pages are
 * shared, and pages nobody holds any more are free.  A parent outside [-1, n_seqs)
 * leaves b as it is and gives KVQ_EINVAL in the status word. */
int kvq_pages_select(const kvq_page_table *table, const int32_t *parents, void *stream);

/* Bring the n live pages to [0, n): the k-th live page from n on moves to the k-th
 * free page before n, and tables and counts follow.  copies int32 [n_copies][2],
 * 8-byte aligned, n_copies >= n_pages / 2 (KVQ_ECAPACITY): the moves, for
 * kvq_paged_copy in every pool; (-1, -1) behind the last. */
int kvq_pages_compact(const kvq_page_table *table, int32_t *copies, int64_t n_copies,
                      void *stream);

/* ---- Drafted tokens --------------------------------------------------------
 *
 * Speculative decoding's decision.  A step runs the model on rows
 * [cu_tokens[b], cu_tokens[b+1]) of sequence b: its newest token, then its drafts.
 * Row t's logits are those of the token after tokens[t], so row t judges
 * tokens[t+1], and the last row has the token after the last draft.
 */
typedef struct kvq_draft_batch {
  const int32_t *cu_tokens; /* device [n_seqs+1], as in kvq_paged_batch */
  const int32_t *tokens;    /* device [n_tokens] */
  int32_t *dev_status;      /* device status word, zero-filled once */
  int64_t n_tokens;         /* rows of the packed arrays, 0..65535; rows from
                               cu_tokens[n_seqs] on are padding */
  int32_t n_seqs, vocab, dtype; /* 1..2048; 1..2^24; KVQ_F16, KVQ_BF16 or KVQ_F32 */
} kvq_draft_batch;

/* Bytes of scratch kvq_verify_drafts needs for these sizes (the pointers are not
 * looked at); it does not shrink as sizes grow.  Zero-fill it once; every call
 * leaves what must be zero at zero again.  Calls that can run at the same time need
 * scratch of their own.  Host only. */
int kvq_verify_workspace_bytes(const kvq_draft_batch *batch, size_t *bytes);

/*
 * Accept or refuse drafts and draw the next token (Leviathan et al. 2023, "Fast
 * inference from transformers via speculative decoding", algorithm 1).
 *   logits: device, row t at logits + t*stride (dtype elements, stride >= vocab, any
 *     alignment of the dtype): x.  draft_logits: y, the draft model's for the same
 *     rows (a sequence's last row is not read), or NULL: each draft was certain
 *     (found by lookup).
 *   temperature: device [n_seqs], T > 0; a sequence where it is not (0, NaN) is
 *     greedy.  NULL: all are.
 *   uniform: device [n_tokens], in [0, 1): row t's number judges tokens[t+1].
 *   noise: device, row b at noise + b*noise_stride: e_i of the exponential
 *     distribution (-log of a uniform number), one for every token of the vocabulary.
 *   (uniform and noise may be NULL where temperature is; greedy sequences read
 *   neither, nor y.)
 * With p = softmax(x / T), q = softmax(y / T) (1 at the draft for NULL), draft c of
 * row t stays while every earlier one does and uniform[t] * q_c < p_c.  The next
 * token is at the first refused row the i of the largest max(p_i - q_i, 0) / e_i
 * (p_i / e_i if all are 0), at the last row, if all stay, of the largest p_i / e_i;
 * of equal ones the lowest.  Its distribution is p's, whatever the drafts.  Greedy:
 * a draft stays while it is the lowest index of x's maximum, and that is the next
 * token.
 *   out_tokens [n_tokens], apart from tokens: for each sequence from its first row on,
 *     the drafts that stayed, then the next token, then -1.
 *   logprobs fp32 [n_tokens]: ln p of each of those tokens (greedy: at T = 1), 0
 *     for -1.
 *   accepted, dropped [n_seqs]: drafts that stayed, and the others: what
 *     kvq_pages_drop takes back, since the cache holds the rows' tokens.
 * Masked: a logit of -infinity or NaN has probability 0; +infinity counts as the
 * type's largest number.  A row of masked logits has no next token: -1.
 * e_i below 2^-126 counts as that, NaN takes i out.  T is held to 2^-100..2^100.
 * A draft outside [0, vocab) is refused and gives KVQ_EINVAL in the status word; so
 * do cu_tokens that decrease, begin below 0 or end behind n_tokens: then no sequence is
 * judged, and outputs are left alone but for 0 accepted, 0 dropped.  A sequence without
 * rows gets those too.
 * Arithmetic: fp32, sums in fp32 in a fixed order, exponents in two parts of fp32.
 * A token t_i = (max x - x_i) / (T ln 2) powers of two below its row's likeliest has
 * its probability within (t_i + 64 + vocab / 2^13) 2^-23 of the exact one (relative),
 * in p and in q, so numbers that close to a border may fall on its other side.  In the
 * sums and in the race a token with t_i beyond 126 counts as 0; as a draft it is
 * judged like any other.
 * Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EALIGN, KVQ_ECAPACITY (ws too small),
 *   KVQ_ECUDA.
 */
int kvq_verify_drafts(const kvq_draft_batch *batch, const void *logits, int64_t stride,
                      const void *draft_logits, int64_t draft_stride, const float *temperature,
                      const float *uniform, const float *noise, int64_t noise_stride,
                      int32_t *out_tokens, int32_t *accepted, int32_t *dropped, float *logprobs,
                      void *ws, size_t ws_bytes, void *stream);

/* The same, and every row of out_tokens and logprobs is written: rows that no
 * sequence owns (padding; all of them where no sequence is judged, or after a failed
 * kvq_pages_reserve) get -1 and 0. */
int kvq_verify_drafts_padded(const kvq_draft_batch *batch, const void *logits, int64_t stride,
                             const void *draft_logits, int64_t draft_stride,
                             const float *temperature, const float *uniform, const float *noise,
                             int64_t noise_stride, int32_t *out_tokens, int32_t *accepted,
                             int32_t *dropped, float *logprobs, void *ws, size_t ws_bytes,
                             void *stream);

/* Number of kernel launches the last successful call of this thread enqueued. */
int kvq_last_launch_count(void);

/* Static description of a return code. */
const char *kvq_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
