/*
 * mla.h -- C ABI of libmla: Multi-head Latent Attention (MLA) over a paged latent KV
 * cache on GB300 (sm_103a).
 *
 * Sources.  The operations follow the TokenSpeed pages:
 *  [TALK]  "构建面向 Agentic 推理的下一代 LLM 推理引擎" (AICon 2026 Shenzhen talk
 *          transcript), section "Kernel：让 MLA 真正跑满 GPU": MLA keeps one latent
 *          state shared by all heads; decode's first matmul is query x latent key with a
 *          query length of one, so query tokens are folded into the head axis; the KV
 *          loop is split into a partial stage and a reduction stage whose split count
 *          and workspace size are computed automatically at run time and cached; the
 *          prefill path is a ragged no-padding batch whose Q and KV lengths differ
 *          because a long prefix (>90% hit rate) is cached and only a few hundred tokens
 *          are appended.  Even with 8-bit KV, loading KV is the bottleneck.
 *  [BLOG]  "英偉達力薦，小團隊兩個月開源一款「光速級」智能體推理引擎" (Synced repost of the
 *          TokenSpeed launch blog), sections "TokenSpeed 技術簡介" and "TokenSpeed 性能
 *          預覽": the decode kernel folds the query-sequence axis into the head axis to
 *          fill the M tile of the first batched matmul; decode is benchmarked with
 *          speculative decoding at batch 4/8/16 over long prefixes; prefill is "prefill
 *          with a long prefix KV cache".
 *  [READ]  "TokenSpeed 深度解析" (gitread.org), section "核心技术揭秘": KV is managed in
 *          fixed-size blocks reached through a table (paged KV).
 *
 * Shapes used throughout: B requests, T = q_len draft tokens per request (1..8192; beyond
 * a few drafts this is the prefill of T new tokens over a paged prefix, absorbed form), H heads,
 * D = 576 latent columns (512 latent + 64 rope), Dv = 512 (the value is the first 512
 * latent columns).  Prefill: 16-bit q/k with Dqk = 192 and v with Dv' = 128.
 *
 * Conventions shared by every call:
 *  - Every pointer argument that is not documented as host memory is DEVICE memory owned
 *    by the caller.  The library never allocates or frees device memory and, but for
 *    mla_get_status, never synchronises the stream.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *  - Tensors are dense and row-major (last index fastest), with the layouts given below.
 *  - Every call returns an mla_status_t code; no C++ exception crosses this ABI.
 *    Host-side argument checks run before anything is enqueued; on a non-zero return
 *    nothing was launched unless the code is MLA_ERR_CUDA.
 *  - The first call of an entry point on each device and host thread sets its kernels up: make
 *    it before a stream capture.
 *  - Device-side failures (a bounded wait that ran out, a length beyond the plan) are
 *    recorded in a per-device status word that mla_get_status() reads and clears.
 */
#ifndef MLA_GB300_MLA_H_
#define MLA_GB300_MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mla_status_t {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,         /* null pointer, negative size, inconsistent shapes   */
  MLA_ERR_UNSUPPORTED = 2,         /* shape the kernels do not implement (see each call) */
  MLA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < plan->workspace_bytes            */
  MLA_ERR_CUDA = 4,                /* a CUDA runtime/driver call or launch failed        */
  MLA_ERR_TIMEOUT = 5,             /* a device-side bounded wait expired (status word)   */
  MLA_ERR_DEVICE_ARG = 6           /* device-side argument check failed (status word)    */
} mla_status_t;

typedef enum mla_kv_dtype_t {
  MLA_KV_BF16 = 0, /* latent pool stored as bfloat16                                     */
  MLA_KV_E4M3 = 1, /* latent pool stored as OCP FP8 e4m3fn codes times one kv_scale      */
  MLA_KV_INT8 = 2, /* latent pool stored as two's-complement int8 codes times one kv_scale.
                    * (The TokenSpeed talk, section "Kernel：让 MLA 真正跑满 GPU", names INT8
                    * among the KV quantisations that keep decode bandwidth-bound; a
                    * per-tensor scale is the plainest form it leaves open.)               */
  MLA_KV_INT8_PAGE = 3 /* int8 codes, each page with its own scale: a latent element is its
                        * code times the scale of the page that holds its row (the other
                        * INT8 form the talk leaves open); decoded by mla_decode_int8_paged  */,
  MLA_KV_FP4 = 4 /* 336 bytes a latent row, all values in units of one kv_scale:
                    *   0..255   columns 0..511, eight to a 32-bit little-endian word: column 8w + i has its
                    *            e2m1 magnitude code (0, 1/2, 1, 3/2, 2, 3, 4, 6) in bits 4i..4i+2 and its
                    *            sign in bit 8i + 7 (i < 4) or 8 (i - 4) + 3; the value is the magnitude times
                    *            2^(e-5) with the exponent e of its 16 columns
                    *   256..271 the exponents e, 0..11, of columns 16g..16g+15: a nibble each, low first
                    *            (12..15 do not occur; they read as some finite value)
                    *   272..335 the 64 rotated columns as e4m3 codes                               */
} mla_kv_dtype_t;

/* Decode plan: a plain value struct filled by mla_decode_plan(); callers treat the
 * fields as read-only.  It fixes the launch shape of mla_decode for one batch layout. */
typedef struct mla_decode_plan_t {
  int32_t batch;             /* B                                                        */
  int32_t q_len;             /* T, draft tokens per request                              */
  int32_t num_heads;         /* H                                                        */
  int32_t page_size;         /* tokens per page                                          */
  int32_t max_pages_per_seq; /* row stride of page_table                                 */
  int32_t kv_dtype;          /* mla_kv_dtype_t                                           */
  int64_t num_pages;         /* pages in the pool (first dimension of kv_pages)          */
  int32_t num_sms;           /* SMs the split count was sized for                        */
  int32_t rows;              /* T*H folded query rows per request                        */
  int32_t head_groups;       /* CTAs along the folded row axis (64 rows each; over a 4-bit
                                pool 32, or 16 for at most 16 rows)                      */
  int32_t chunk_tokens;      /* keys per split (multiple of 64)                          */
  int32_t max_splits;        /* splits of the longest request                            */
  int32_t max_seq_len;       /* longest planned request; device seq_lens must not exceed */
  int32_t split_major;       /* launch order of the partial kernel's CTAs: 1 = split by
                                split (plans of more than one wave), 0 = request by request,
                                2 = whole splits, then remainders (4-bit pools)          */
  int32_t num_splits;        /* split_major 2: splits of the planned requests in all;
                                else 0                                                  */
  size_t workspace_bytes;    /* bytes mla_decode needs in `workspace` (0 = none)         */
} mla_decode_plan_t;

/* Plan one decode launch: pick the keys-per-split chunk (whole 64-key tiles) and size the
 * workspace for the split partials.  The partial kernel runs one CTA per (request, split,
 * 64-row group); the plan estimates the call's duration by dispatching those CTAs in
 * launch order onto the SM that frees first (each costing its tiles plus a fixed
 * start-up and epilogue cost that depends on the pool format, plus the combine when a
 * request is split), over these chunks: the longest request in 1-4 splits (1-32 with more
 * than one row group when the others leave the SMs idle over a tenth of the call), the
 * smallest
 * chunk that keeps the call in one wave of CTAs when the unsplit call fits one, and, with
 * one row group, the chunks that share all tiles evenly over one or two waves (and up to
 * 8 tiles more than the one-wave one).  The chunk
 * with the shortest estimate wins (fewer splits on a tie), so a split is never taken when
 * it lengthens the call by that estimate.  A plan of one row group and more than one wave
 * launches its CTAs split by split (every request's first split, then every request's
 * second, ...: split_major = 1), so that short remainders go last; every other plan
 * launches them request by request.
 * Plans are memoised on all arguments
 * (the split count and workspace are "computed automatically at run time and cached",
 * [TALK] Kernel section).
 *   seq_lens_host : HOST int32[batch], tokens cached per request INCLUDING the q_len
 *                   draft tokens (the drafts are the last q_len positions).
 *   num_sms       : SMs to plan for; 0 = query the current device.
 * Errors: MLA_ERR_INVALID_ARG (null pointers, batch < 1, a length < q_len or beyond
 * max_pages_per_seq*page_size), MLA_ERR_UNSUPPORTED (q_len > 8192, page_size not one
 * of 8,16,32,64,128,256, or more than 131072 folded rows), MLA_ERR_CUDA (device query). */
int mla_decode_plan(int batch, const int32_t* seq_lens_host, int q_len, int num_heads,
                    int page_size, int max_pages_per_seq, int64_t num_pages, int kv_dtype,
                    int num_sms, mla_decode_plan_t* plan_out);

/* Absorbed MLA decode with speculative draft tokens over the paged latent cache.
 *   q          : [B, T, H, 576] bf16.  Folded row m = t*H + h of request b.
 *   kv_pages   : [num_pages, page_size, 576] bf16, e4m3 or int8 bytes, or [.., 336] bytes of
 *                MLA_KV_FP4 (plan->kv_dtype); the allocation must hold all num_pages pages in the plan's format (the
 *                library cannot check it: a pool of another format is read out of bounds).
 *   page_table : [B, max_pages_per_seq] int32; latent row j of request b is
 *                kv_pages[page_table[b, j / page_size], j % page_size, :].
 *   seq_lens   : [B] int32 device copy of the planned lengths (each <= max_seq_len).
 *   scale      : softmax scale applied to q . k.
 *   kv_scale   : per-tensor dequantisation scale of an 8-bit or 4-bit pool (ignored for bf16).
 *                (Over a 4-bit pool a query element is exact down to 2^-9 of its row's largest and taken to 2^-17 of that
 *                below.  A key's weight is carried to 2^-9 of itself or, where that is more, to the lesser of 2^-20 of its
 *                row's largest and 2^-9 of its row's largest among the 128 keys of its tile (tiles begin at multiples of
 *                128); beside a key far above all others of its tile and in the three tiles behind it, up to nine where such
 *                keys come again and again, to 2^-20 of that key's.)
 *   out        : [B, T, H, 512] bf16, out[b,t,h] = sum_j softmax_j(scale q.k_j) v_j with
 *                draft t seeing keys 0 .. L_b - T + t and v_j = k_j[:512].
 *   lse        : [B, T, H] fp32, natural-log log-sum-exp of the scaled scores.
 *   workspace  : device scratch of workspace_bytes >= plan->workspace_bytes, 256-byte
 *                aligned; may be NULL when plan->workspace_bytes == 0.  Its contents are
 *                overwritten; calls that share one workspace must be stream-ordered.
 * Enqueues the split-KV partial kernel and, when any request has more than one split,
 * the LSE-merge combine kernel on `stream`.  No allocation, no host synchronisation.
 * Both are programmatic dependent launches: the partial kernel may set itself up while the
 * stream's previous kernel finishes, but reads no input before that kernel has completed;
 * the combine waits in the same way for the partial kernel.  A kernel enqueued after this
 * call as a programmatic dependent must itself wait (griddepcontrol.wait or
 * cudaGridDependencySynchronize) before it reads out or lse.
 * Errors: MLA_ERR_INVALID_ARG (null pointers, q_len/num_heads differ from the plan,
 * misaligned pointers: q, kv_pages 16-byte, out 16-byte), MLA_ERR_WORKSPACE_TOO_SMALL,
 * MLA_ERR_CUDA (tensor-map encoding or launch failure).  Device-side, recorded in the
 * status word as MLA_ERR_DEVICE_ARG (read by mla_get_status): a length below q_len or
 * beyond the plan (that request is skipped, its out/lse rows left unwritten), and a page
 * id outside [0, num_pages) (the rows it names are read as zeros, never from outside the
 * pool). */
int mla_decode(const mla_decode_plan_t* plan, const void* q, const void* kv_pages,
               const int32_t* page_table, const int32_t* seq_lens, int q_len, int num_heads,
               float scale, float kv_scale, void* out, float* lse, void* workspace,
               size_t workspace_bytes, void* stream);

/* mla_decode over an int8 pool with one scale per page (plan->kv_dtype ==
 * MLA_KV_INT8_PAGE; mla_decode and mla_decode_partial reject such plans).  Arguments,
 * layouts and errors as mla_decode, with:
 *   kv_pages    : [num_pages, page_size, 576] int8 codes.
 *   page_scales : [num_pages] fp32 on the device, 4-byte aligned: the scale of each page's
 *                 codes (element = code * page_scales[page]).
 *   kv_scale    : a reference scale > 0 (the largest page scale is the natural choice).
 *                 Each page scale must lie in [0, 255 * kv_scale]; a page scale outside it
 *                 (or not finite) on a page a request reads is reported as
 *                 MLA_ERR_DEVICE_ARG and that request's split is skipped.
 * The codes are multiplied exactly as int8 values; each key's page scale relative to
 * kv_scale multiplies its score (in fp32) and the softmax weight its value row receives,
 * and kv_scale itself is folded into the softmax scale and the output.  The combine
 * stage is the one of mla_decode: mla_decode_combine accepts these plans. */
int mla_decode_int8_paged(const mla_decode_plan_t* plan, const void* q, const void* kv_pages,
                          const float* page_scales, const int32_t* page_table, const int32_t* seq_lens,
                          int q_len, int num_heads, float scale, float kv_scale, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Decode of a TREE of drafted tokens: as mla_decode, but the drafts do not follow one another;
 * draft t of request b sees the whole prefix (keys 0 .. L_b - T - 1) and, of the T drafts at the
 * request's last positions, those whose bit is set in its mask word.
 *   plan        : from mla_decode_tree_plan: mla_decode_plan with q_len = T <= 64 and a workspace for
 *                 a tree's split partials (fp32 over a bf16 pool; mla_decode_plan's own plans run
 *                 too, given a workspace of that size).
 *   page_scales : as mla_decode_int8_paged for an MLA_KV_INT8_PAGE plan, else NULL.
 *   tree_mask   : [B, T] uint64, 8-byte aligned: bit u of word (b, t) = draft t sees draft u (usually
 *                 its ancestors and itself; any word is accepted, bits from T on are ignored).
 *   out, lse    : as mla_decode; a draft that sees no key at all (an empty mask over an empty
 *                 prefix) gets out 0 and lse -infinity.
 * An infinity or NaN in a draft's latent row reaches only the drafts that see it: NaN everywhere, or,
 * where the score is -infinity and so the weight 0, in the columns that hold it.  (A draft all of whose
 * scores are -infinity counts as one that sees no key.)  Launches,
 * workspace rules and every other argument and error as mla_decode; also MLA_ERR_UNSUPPORTED for
 * more than 64 drafts. */
int mla_decode_tree_plan(int batch, const int32_t* seq_lens_host, int q_len, int num_heads,
                         int page_size, int max_pages_per_seq, int64_t num_pages, int kv_dtype,
                         int num_sms, mla_decode_plan_t* plan_out);
int mla_decode_tree(const mla_decode_plan_t* plan, const void* q, const void* kv_pages, const float* page_scales,
                    const int32_t* page_table, const int32_t* seq_lens, const uint64_t* tree_mask,
                    int q_len, int num_heads, float scale, float kv_scale, void* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream);

/* The two stages of mla_decode, for callers that schedule them apart (e.g. to put other
 * work between them, or to time the split-KV partial kernel on its own).  The TokenSpeed
 * talk ("构建面向 Agentic 推理的下一代 LLM 推理引擎", section "Kernel：让 MLA 真正跑满 GPU")
 * describes the kernel as a split-KV partial stage followed by a reduction stage; these
 * calls expose that split.  mla_decode(...) is exactly mla_decode_partial(...) followed by
 * mla_decode_combine(...) on the same stream with the same plan, workspace, out and lse.
 *
 * mla_decode_partial: arguments, layouts and errors as mla_decode.  Enqueues the split-KV
 * partial kernel only.  Requests whose plan gives them one split get their final out/lse
 * rows; the others leave per-split bf16 partial outputs and fp32 log-sum-exps in the
 * workspace, which stay valid until the workspace is next written.
 *
 * mla_decode_combine: merges those partials into out/lse (log-sum-exp weighted mean over
 * the splits of each request).  plan, seq_lens, q_len, num_heads, out, lse and workspace
 * must be the ones given to the mla_decode_partial call it completes, stream-ordered
 * after it.  Enqueues nothing when no request has more than one split.  Errors:
 * MLA_ERR_INVALID_ARG (null plan/seq_lens/out/lse, q_len/num_heads differ from the plan,
 * out not 16-byte or lse not 4-byte aligned, workspace missing or not 256-byte aligned),
 * MLA_ERR_WORKSPACE_TOO_SMALL, MLA_ERR_CUDA (launch failure). */
int mla_decode_partial(const mla_decode_plan_t* plan, const void* q, const void* kv_pages,
                       const int32_t* page_table, const int32_t* seq_lens, int q_len, int num_heads,
                       float scale, float kv_scale, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);
int mla_decode_combine(const mla_decode_plan_t* plan, const int32_t* seq_lens, int q_len,
                       int num_heads, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/* mla_decode for callers that cannot allocate device memory.  (The pages have no
 * counterpart: this is a library convenience.)  Some callers cannot call cudaMalloc, e.g.
 * a serving engine whose memory manager gives every free byte of the device to its
 * KV-cache pool at start-up and refuses later allocations, or a plugin loaded into a host
 * program that offers it no allocator.  This entry point takes the same arguments as
 * mla_decode minus the workspace, and uses as scratch a fixed 32 MiB buffer that lives in
 * the library's own device data: every GPU that loads libmla holds those 32 MiB until the
 * process exits.  It allocates and frees nothing.
 *  - Limit: plan->workspace_bytes must be <= 32 MiB (33554432); larger plans are rejected
 *    with MLA_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.
 *  - The first call on each device looks up the buffer's device address (with that device
 *    current); make that first call before any stream capture.
 *  - All calls on a device share the one buffer, which keeps the previous call's
 *    contents.  Nothing in it has to start at zero: each call writes every partial it
 *    later reads.  Calls whose kernels overlap on the GPU (other streams, other threads)
 *    race on the buffer and corrupt each other's results: order them on one stream.
 * Errors: as mla_decode, plus MLA_ERR_WORKSPACE_TOO_SMALL for plans beyond the limit. */
int mla_decode_noalloc(const mla_decode_plan_t* plan, const void* q, const void* kv_pages,
                       const int32_t* page_table, const int32_t* seq_lens, int q_len, int num_heads,
                       float scale, float kv_scale, void* out, float* lse, void* stream);

/* Ragged (no padding) causal MLA prefill on top of a cached prefix.
 *   q             : [total_q, H, 192] bf16; request b's n_b new tokens are rows
 *                   cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1.
 *   k             : [total_kv, H, 192] bf16; request b's p_b + n_b keys (prefix first) are
 *                   rows cu_seqlens_kv[b] .. cu_seqlens_kv[b+1]-1.
 *   v             : [total_kv, H, 128] bf16, same rows as k.
 *   cu_seqlens_q, cu_seqlens_kv : [batch+1] int32 prefix sums (device).
 *   prefix_lens   : [batch] int32 p_b (device); kv length must equal p_b + n_b.
 *   max_seqlen_q  : host bound on n_b (sizes the grid).
 *   total_q, total_kv : host row counts of q and k/v (bounds of the tensor maps).
 *   out           : [total_q, H, 128] bf16; new token i of request b attends to keys
 *                   0 .. p_b + i of its own request.
 *   lse           : [total_q, H] fp32 natural-log log-sum-exp.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (num_heads < 1 or > 256),
 * MLA_ERR_CUDA.  Device-side, recorded in the status word as MLA_ERR_DEVICE_ARG (read by
 * mla_get_status) before any load or store of the request: its kv length differs from
 * p_b + n_b, n_b > max_seqlen_q, or its rows reach beyond total_q / total_kv.  That
 * request is skipped and its out/lse rows are left unwritten.
 * Scratch: a q block with 8 or more tiles of 128 keys runs as two CTAs over the halves of
 * its keys, which merge through this library's own device scratch (32 MiB per GPU, 1024
 * slots; q blocks past them are not split).  Prefill calls whose kernels overlap on the
 * GPU (other streams, other threads) race on it: order them on one stream.  The first
 * call on each device and host thread looks the scratch up; make it before any stream
 * capture. */
int mla_prefill_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                       const int32_t* cu_seqlens_kv, const int32_t* prefix_lens, int batch,
                       int num_heads, int max_seqlen_q, int total_q, int total_kv, float scale,
                       void* out, float* lse, void* stream);

/* The same prefill with K/V read from a paged cache of per-head k/v rows instead of
 * contiguous per-request rows.  The TokenSpeed pages describe the prefill as "prefill with a
 * long prefix KV cache" ([BLOG] "TokenSpeed 性能預覽"; [TALK] "Kernel：让 MLA 真正跑满 GPU",
 * last paragraph) and keep KV in fixed-size blocks behind a table ([READ] "核心技术揭秘");
 * this call reads both the cached prefix and the new tokens' k/v from such blocks.
 *   q             : [total_q, H, 192] bf16; request b's n_b new tokens are rows
 *                   cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1.
 *   k_pages       : [num_pages, page_size, H, 192] bf16.
 *   v_pages       : [num_pages, page_size, H, 128] bf16.
 *   page_table    : [batch, max_pages_per_seq] int32; key j of request b (prefix first,
 *                   then its new tokens) is row j % page_size of page
 *                   page_table[b, j / page_size] of k_pages / v_pages.
 *   kv_lens       : [batch] int32 (device), p_b + n_b: the request's cached prefix plus
 *                   its new tokens, whose k/v are the last n_b positions.
 *   page_size     : 16, 32, 64, 128 or 256 tokens.
 *   num_pages     : pages in each pool (num_pages * page_size < 2^31).
 *   out, lse      : as mla_prefill_varlen: new token i of request b attends to keys
 *                   0 .. p_b + i.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (num_heads outside 1..256, another page
 * size, too many pool rows), MLA_ERR_CUDA.  Device-side, recorded in the status word as
 * MLA_ERR_DEVICE_ARG: n_b > max_seqlen_q, kv_lens[b] < n_b or beyond the table row, q rows
 * beyond total_q (the request is skipped, before any access), and a page id outside
 * [0, num_pages) (its rows are read as zeros, never from outside the pools).
 * Scratch: as mla_prefill_varlen (the same library-owned scratch: order every prefill
 * call, contiguous or paged, on one stream). */
int mla_prefill_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                      const int32_t* cu_seqlens_q, const int32_t* kv_lens, int batch, int num_heads,
                      int page_size, int max_pages_per_seq, int64_t num_pages, int max_seqlen_q,
                      int total_q, float scale, void* out, float* lse, void* stream);

/* One pass that prepares a step's queries and latent keys and writes the keys into the paged
 * latent cache that mla_decode reads: norm, position rotation and (quantised) paged write.
 * For token n at position x = positions[n] (all arithmetic in fp32, one rounding at the store):
 *   key  : c = kv_in[n, :512]; c' = c / sqrt(mean(c^2) + eps) * kv_weight (kv_weight NULL: c' = c);
 *          the latent row [c', rot(kv_in[n, 512:576], x)] goes to pool row slots[n], as bf16, or as
 *          the codes of the values over kv_scale (nearest, ties to even; saturated to +-448 or
 *          +-127; a NaN encodes as the e4m3 NaN, as int8 0).  A 4-bit row: y = value times 1/kv_scale (rounded
 *          to fp32); 16 columns whose largest |y| is t take the smallest exponent e of 0..11 with t <= 7 2^(e-5), and
 *          the nearest code of y 2^(5-e) (ties to the even code; saturated to +-6; a NaN encodes as 0); the rotated columns
 *          are e4m3 codes.  Here the mean is that of the exact squares, rounded once to fp32, and no product is fused
 *          with a sum, so that the codes are those of the formula to the bit.  (With kv_weight one NaN or infinity among the 512
 *          columns leaves nothing of the others: 512 zeros in a 4-bit or int8 row, which nothing reports.)
 *   query: v = q_in[n, h, :q_dim]; v' = v / sqrt(mean(v^2) + eps) * q_weight over the whole width
 *          (q_weight NULL: v' = v); q_out[n, h] = [v'[:q_dim-64], rot(v'[q_dim-64:], x)].
 *   rot  : pair i of 32 is columns (2i, 2i+1) (interleaved != 0) or (i, i+32); (a, b) becomes
 *          (a cos - b sin, b cos + a sin) with cos = cos_sin[x, i], sin = cos_sin[x, 32 + i].
 *   q_in, q_out : bf16, element [n, h, c] at n * token_stride + h * head_stride + c; strides are
 *                 in elements, multiples of 8 (q_in's may be 0; q_out's rows may not overlap).
 *                 q_out may be q_in with the same strides; else the two spans of memory are apart.
 *                 q_in NULL: keys only (every q argument is ignored).
 *   q_dim       : 64..576, a multiple of 8: 64 rotates a [.., 64] view alone (for example columns
 *                 512.. of absorbed queries), 192 is the prefill's width.
 *   q_weight    : [q_dim] bf16 or NULL.   kv_weight : [512] bf16 or NULL.
 *   kv_in       : bf16 [num_tokens, 576], rows kv_in_token_stride apart (a multiple of 8).
 *                 NULL: queries only (slots, kv_pages, num_slots are ignored).
 *   cos_sin     : [max_positions, 64] fp32, 16-byte aligned.
 *   positions   : [num_tokens] int32.
 *   slots       : [num_tokens] int64: page id * page_size + offset of the key's pool row; negative =
 *                 a padded token whose key is not stored (its queries still are).  Slots that are
 *                 not negative must differ: a row that two tokens name holds bytes of either.
 *   kv_pages    : the pool, num_slots = num_pages * page_size rows of kv_dtype.
 *   kv_scale    : scale of an e4m3, int8 or 4-bit pool (ignored for bf16).
 * Pointers are 16-byte aligned (positions 4, slots 8).  kv_in, q_in and q_out lie outside the pool, and
 * q_out holds no element of kv_in, the weights, cos_sin, positions or slots.
 * Rows that no token names are left as they were.  num_tokens 0 does nothing.  Launched as a programmatic dependent like mla_decode.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (num_heads > 1024, another q_dim, num_tokens >
 * 2^20, an MLA_KV_INT8_PAGE pool, whose page scales cannot follow new rows), MLA_ERR_CUDA.
 * Device-side, recorded as MLA_ERR_DEVICE_ARG: a position outside [0, max_positions) (the token's
 * rows are left unwritten; a padded token's position counts too unless kv_in alone is given) and a
 * slot >= num_slots (its key is left unwritten). */
int mla_kv_append(const void* q_in, int64_t q_in_token_stride, int64_t q_in_head_stride, void* q_out,
                  int64_t q_out_token_stride, int64_t q_out_head_stride, int num_heads, int q_dim,
                  const void* q_weight, const void* kv_in, int64_t kv_in_token_stride, const void* kv_weight,
                  float eps, const float* cos_sin, int max_positions, const int32_t* positions,
                  const int64_t* slots, int num_tokens, int interleaved, void* kv_pages, int64_t num_slots,
                  int kv_dtype, float kv_scale, void* stream);

/* Latent rows of requests, read out of the pages of any pool format into contiguous bf16 rows (a prefill that
 * projects a cached prefix up again needs them so): for r = cu_rows[b] .. cu_rows[b+1] - 1,
 *   out[r, :] = bf16(value of row r - cu_rows[b] of request b),
 * a value being its code times kv_scale (MLA_KV_INT8_PAGE: its page's scale) in fp32, rounded once; bf16 rows are
 * copied.
 *   kv_pages, page_table : as mla_decode, [batch, max_pages_per_seq].
 *   page_scales : [num_pages] for an MLA_KV_INT8_PAGE pool, else NULL.
 *   kv_scale    : > 0 (ignored for bf16 and for a scale per page).
 *   cu_rows     : [batch + 1] int32 prefix sums on the device.
 *   total_rows  : host bound on cu_rows[batch], the rows of out.  0 does nothing.
 *   out         : bf16, rows out_row_stride elements apart (at least 576, a multiple of 8), 16-byte aligned; it lies
 *                 outside the pool, the table, cu_rows and the scales.  Rows of no request are left as they were.
 * Launched as a programmatic dependent like mla_decode.  Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (page_size),
 * MLA_ERR_CUDA.  Device-side, recorded as MLA_ERR_DEVICE_ARG: cu_rows below 0 or beyond total_rows (those rows are not
 * written), a request longer than its page-table row (the rows beyond are not written), a page id outside
 * [0, num_pages) (its rows are zeros). */
int mla_kv_gather(const void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float kv_scale, const float* page_scales,
                  const int32_t* page_table, int max_pages_per_seq, const int32_t* cu_rows, int batch, int total_rows,
                  void* out, int64_t out_row_stride, void* stream);

/* The attention weight that each cached key received in a decode step, accumulated over steps:
 *   mass[b, j] = decay * mass[b, j] + sum over rows (t, h) that see key j of
 *                exp(scale q[b,t,h] . k_j - lse[b,t,h]),   j < L_b
 * Call it after the step's mla_decode / mla_decode_tree, with that call's arguments and lse; each
 * row then adds a total weight of 1.  Sums are fp32, in a fixed order.
 *   plan        : from mla_decode_plan or mla_decode_tree_plan.
 *   q, kv_pages, page_table, seq_lens, scale, kv_scale : as mla_decode.
 *   page_scales : as mla_decode_int8_paged for an MLA_KV_INT8_PAGE plan, else NULL.
 *   tree_mask   : as mla_decode_tree, or NULL: draft t sees keys 0 .. L_b - T + t.
 *   lse         : [B, T, H] fp32; a row whose lse is not finite adds nothing.
 *   decay       : >= 0; 0 overwrites mass without reading it.
 *   mass        : fp32, row b at mass + b * mass_stride (elements; >= plan->max_seq_len); entries from
 *                 L_b on are left as they were.
 *   workspace   : device scratch of the size mla_key_mass_workspace gives for the plan, 256-byte
 *                 aligned (NULL when that is 0, as it is for at most 128 rows q_len * num_heads);
 *                 overwritten; calls that share one are stream-ordered.
 * Launched as a programmatic dependent like mla_decode.  Errors: MLA_ERR_INVALID_ARG,
 * MLA_ERR_UNSUPPORTED (tree_mask with more than 64 drafts; a 4-bit pool; batch times the longest request beyond
 * 2^38 keys), MLA_ERR_WORKSPACE_TOO_SMALL, MLA_ERR_CUDA.  Device-side, recorded as
 * MLA_ERR_DEVICE_ARG: a length below q_len or beyond the plan (that request's row is left as it
 * was), a page id outside [0, num_pages) (its rows count as zeros) and, on a page that a request
 * reads, a page scale outside [0, 255 * kv_scale] or not finite (its keys get no weight: their mass
 * only decays). */
int mla_key_mass_workspace(const mla_decode_plan_t* plan, size_t* bytes_out);
int mla_key_mass(const mla_decode_plan_t* plan, const void* q, const void* kv_pages, const float* page_scales,
                 const int32_t* page_table, const int32_t* seq_lens, const uint64_t* tree_mask,
                 const float* lse, int q_len, int num_heads, float scale, float kv_scale, float decay,
                 float* mass, int64_t mass_stride, void* workspace, size_t workspace_bytes, void* stream);

/* Eviction by accumulated attention weight: choose the keys that each request keeps and copy their
 * latent rows, in order, into new pages of the same pool.  Request b with L = seq_lens[b] cached
 * keys keeps K = min(keep_lens[b], L): the first s = min(sink, K), the last r = min(recent, K - s),
 * and the K - s - r keys between them with the largest mass[b, j] (equal masses: the lower index;
 * -0 equals 0; NaN is below every number).  With kept = those keys in ascending order:
 *   row i of the destination pages = row kept[i] of the source pages, i < K
 *   kept[b, i] = kept[i], mass_out[b, i] = mass[b, kept[i]], new_lens[b] = K
 * Entries of kept and mass_out from K on, and pool rows that are no destination, are left as they
 * were.  Rows are copied because a source page may be a prefix that other requests share; the
 * caller releases the old pages.  Keys keep the rotation of their old positions.  (mla_key_mass does not take a 4-bit
 * pool: masses of its keys are the caller's own.)
 *   kv_pages       : [num_pages, page_size] rows of kv_dtype (bf16, e4m3, int8 or 4-bit).
 *   page_table     : [batch, max_pages_per_seq] int32 source pages.
 *   seq_lens, keep_lens : [batch] int32 (device).
 *   mass           : fp32, row b at mass + b * mass_stride (elements; >= max_seq_len).
 *   dst_page_table : [batch, max_dst_pages] int32 destination pages, which must be distinct and no
 *                    source page of any request of the call.
 *   max_seq_len, max_keep : host bounds on the lengths and on K (0: mass, or kept and mass_out, may be NULL).
 *   kept, mass_out : row b at b * kept_stride / b * mass_out_stride (elements; >= max_keep).
 *                    mass_out may not overlap mass, new_lens neither seq_lens nor keep_lens.
 * Two kernels on `stream` (selection, copy), programmatic dependents like mla_decode.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (page_size not 8..256, batch > 65535,
 * max_seq_len > 2^24, an MLA_KV_INT8_PAGE pool, whose codes mean something else under another
 * page's scale), MLA_ERR_CUDA.  Device-side, recorded as MLA_ERR_DEVICE_ARG: a length below 0,
 * beyond max_seq_len or beyond its page-table row, keep_lens[b] < 0, K beyond max_keep or the
 * destination row (the request is skipped, nothing of it written), and a page id outside
 * [0, num_pages) (its rows are not copied). */
int mla_kv_evict(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, const int32_t* page_table,
                 int max_pages_per_seq, const int32_t* seq_lens, const int32_t* keep_lens, const float* mass,
                 int64_t mass_stride, const int32_t* dst_page_table, int max_dst_pages, int batch, int sink,
                 int recent, int max_seq_len, int max_keep, int32_t* kept, int64_t kept_stride,
                 int32_t* new_lens, float* mass_out, int64_t mass_out_stride, void* stream);

/* The pages of a cache, kept on the device.  A cache has num_slots requests, slot s with the pages
 * page_table[s, 0 .. ceil(seq_lens[s] / page_size) - 1] (entries from there on mean nothing), and a count refs[page]
 * of the entries that refer to each page; 0 is a free page.  Pages may be shared: full ones only, since appended rows
 * go into the last.  (A slot that mla_page_free shrinks into a page that others share is forked before rows are appended to
 * it: the fork's partial last page is its own.)  The caller takes new pages from the free ones (mla_page_free lists
 * them) and sets their counts to 1.
 *   kv_pages   : the pool, [num_pages, page_size] rows of kv_dtype (any).
 *   page_scales: [num_pages] for an MLA_KV_INT8_PAGE pool (they go with the pages), else NULL.
 *   page_table : [num_slots, max_pages_per_seq] int32.    seq_lens : [num_slots] int32.    refs : [num_pages] int32.
 * All on the device; what a call writes shares no memory with anything else that it takes.  Kernels are programmatic
 * dependents like mla_decode's.  Counts are not negative.  Errors of all: MLA_ERR_INVALID_ARG (more than 2^30 pages
 * too), MLA_ERR_UNSUPPORTED (page_size not 8..256, more than 65535 listed slots), MLA_ERR_CUDA.
 *
 * mla_page_fork: for each i < count, slot children[i] becomes a copy of slot parents[i]: it shares the full pages
 * (their counts go up by 1); a partial last page is copied to page new_pages[i], whose count becomes 1 (not looked at
 * where the parent's last page is full); the length is the parent's.  What the child held before is not given back.
 * children differ from one another and from every parent of the call, new pages differ and are free.
 * Device-side, recorded as MLA_ERR_DEVICE_ARG, that child left as it was: a slot outside the table, a child that a
 * child before it or a parent names, a length below 0 or beyond the row, and, where one is needed, a new page outside the
 * pool, not free, or named before in new_pages, or a last page outside the pool.  A full page outside the pool is
 * copied as it is, and recorded.
 *
 * mla_page_free: for each i < count, slot slots[i] shrinks to keep_lens[i] <= its length (0: it ends): the counts
 * of the pages behind go down by 1, and seq_lens[slots[i]] = keep_lens[i].  The pages whose count came to 0 by this call
 * stand in freed[0 .. *num_freed - 1] in ascending order; entries behind are left as they were.  page_table is
 * not changed.
 *   freed : [num_pages] int32.    num_freed : int32.
 * Device-side, recorded as MLA_ERR_DEVICE_ARG: a slot outside the table or listed before, a length beyond the row or
 * below keep_lens[i], keep_lens[i] < 0 (that slot is left as it was); an entry outside the pool, or one more for a page
 * than its count (the entry is passed over).
 *
 * mla_page_compact: pages with a count move so that they are 0 .. *num_live - 1: the k-th free page below *num_live
 * takes the k-th counted page from *num_live on.  Rows, counts, page scales and the tables of all slots follow; free pages
 * keep their rows.  Entries from a slot's length on are not rewritten, although a page there that has a count may move: pages are
 * taken ahead of the length after this call, not before.
 *   num_live  : int32.
 *   workspace : of the size mla_page_compact_workspace gives, 256-byte aligned; overwritten; calls that share one are
 *               stream-ordered.  MLA_ERR_WORKSPACE_TOO_SMALL.
 * Device-side, recorded as MLA_ERR_DEVICE_ARG: a table entry outside the pool, or from *num_live on whose page
 * has no count (left as it was), a length beyond the row (its whole row is rewritten). */
int mla_page_fork(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float* page_scales, int32_t* page_table,
                  int max_pages_per_seq, int32_t* seq_lens, int num_slots, int32_t* refs, const int32_t* parents,
                  const int32_t* children, const int32_t* new_pages, int count, void* stream);
int mla_page_free(const int32_t* page_table, int max_pages_per_seq, int32_t* seq_lens, int num_slots, int page_size, int32_t* refs,
                  int64_t num_pages, const int32_t* slots, const int32_t* keep_lens, int count, int32_t* freed, int32_t* num_freed,
                  void* stream);
int mla_page_compact_workspace(int64_t num_pages, size_t* bytes_out);
int mla_page_compact(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float* page_scales, int32_t* page_table,
                     int max_pages_per_seq, const int32_t* seq_lens, int num_slots, int32_t* refs, int32_t* num_live,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Read and clear the current device's status word after synchronising `stream`.
 * Returns MLA_OK, MLA_ERR_TIMEOUT or MLA_ERR_DEVICE_ARG (first recorded), or
 * MLA_ERR_CUDA if the read itself fails.  This call synchronises: keep it off the hot
 * path. */
int mla_get_status(void* stream);

/* Measurement hook: when start/stop are non-NULL cudaEvent_t handles, subsequent
 * mla_decode calls made from the calling host thread record `start` immediately before
 * and `stop` immediately after the split-KV partial kernel (on the call's stream), and
 * mla_prefill_varlen records them around its kernel.  NULL, NULL turns recording off.
 * The library does not own the events.  Returns MLA_OK. */
int mla_set_profile_events(void* start_event, void* stop_event);

/* Elapsed milliseconds between two events recorded through the hook above (including
 * event nodes replayed from a captured CUDA graph).  Returns MLA_ERR_CUDA if either event
 * has not completed. */
int mla_profile_elapsed_ms(void* start_event, void* stop_event, float* ms_out);

/* Watchdog self-test: enqueue a one-warp kernel that waits, through the same bounded
 * mbarrier wait every MLA kernel uses, on a barrier nothing ever arrives on.  The wait
 * gives up after its limit (1 s) and records MLA_ERR_TIMEOUT in the status word, which
 * the next mla_get_status() returns; the CUDA context stays usable.  Returns MLA_OK once
 * enqueued.  (No counterpart on the pages: it exercises the failure-detection path of
 * this library without faulting or hanging the GPU.) */
int mla_selftest_wait_timeout(void* stream);

/* Static, human-readable name of a status code. */
const char* mla_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_GB300_MLA_H_ */
