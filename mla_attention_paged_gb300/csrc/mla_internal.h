// mla_internal.h -- launch parameter blocks and launcher declarations shared by the host
// API (mla_api.cu) and the kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

constexpr int kLatentDim = 576;  // 512 latent + 64 rope columns
constexpr int kValueDim = 512;   // value = first 512 latent columns
constexpr int kTileKeys = 64;    // keys per decode tile
constexpr int kGroupRows = 64;   // folded query rows per decode CTA
constexpr int kTreeNarrowRows = 48;  // most rows of a tree over a bf16 pool that one CTA takes

// Formats of the split partials (see DecodeParams).
constexpr int kPartBf16 = 0;
constexpr int kPartF32 = 1;
constexpr int kPartF16 = 2;

constexpr int kMaxTreeDrafts = 64;  // drafts of a tree: one bit each of a 64-bit word

// Pool formats of the decode kernel (the values of mla_kv_dtype_t).
constexpr int kKvBf16 = 0;
constexpr int kKvE4m3 = 1;
constexpr int kKvInt8 = 2;
constexpr int kKvInt8Page = 3;  // int8 codes times a scale per page
constexpr int kKvFp4 = 4;       // e2m1 codes times a power of two per 16 columns, e4m3 rotated columns

constexpr int kFp4RowBytes = 336;  // a latent row: 256 bytes of codes, 16 of exponents, 64 rotated
constexpr int kFp4TileKeys = 128;  // keys per decode tile

// Device status word bits (OR-ed by kernels, read and cleared by mla_get_status).
constexpr unsigned kStatusTimeout = 1u;
constexpr unsigned kStatusDeviceArg = 2u;

struct DecodeParams {
  int B, T, H, R;               // R = T*H folded rows per request
  int page_size, max_pages;     // page geometry and page_table row stride
  int chunk, max_splits, max_seq;
  int num_splits;               // split_major 2: of the planned lengths, all requests (0: not known)
  int split_major;              // grid: 1 (groups, B, splits), 0 (groups, splits, B), 2 a list of (split, group), kKvFp4 only
  int kv_dtype;                 // kKvBf16, kKvE4m3, kKvInt8, kKvInt8Page or kKvFp4
  int64_t num_pages;            // pages in the pool: a page id outside [0, num_pages) is reported
  float scale_log2;             // softmax scale * log2(e) (* kv_scale for an 8-bit pool)
  float v_scale;                // 1, or kv_scale for an 8-bit pool (applied in the epilogue)
  const int32_t* page_table;
  const int32_t* seq_lens;
  const __nv_bfloat16* q;       // [B, T, H, 576] (kKvFp4; the others read it through a tensor map)
  const uint8_t* kv_pool;       // pool base (the int8 path reads raw rows from here)
  const float* page_scales;     // kKvInt8Page: [num_pages] scale of each page's codes
  float inv_ref_scale;          // kKvInt8Page: 1 / kv_scale (page scales are applied relative to it)
  __nv_bfloat16* out;           // [B, T, H, 512]
  float* lse;                   // [B, T, H]
  __nv_bfloat16* ws_o;          // [B, max_splits, R, 512] partial outputs (normalised, bf16; kKvFp4: f16 in units of the codes)
  float* ws_lse;                // [B, max_splits, R] partial log-sum-exp (natural log)
  float* part_scale;            // kKvFp4: v_scale for the combine, left by the partial kernel in the workspace's
                                // first bytes (a combine on its own is not given kv_scale); else null
  unsigned* status;             // device status word
  // tree decode (tree_mask non-null): [B, T] bit u of word (b, t) = draft t sees draft u; the
  // split partials are f16 in units of the codes in ws_o (8-bit pools), or fp32 in ws_of
  const uint64_t* tree_mask;
  float* ws_of;                 // [B, max_splits, R, 512] partial outputs of a tree decode over a bf16 pool
};

struct PrefillParams {
  int B, H, max_q_blocks;
  int max_seqlen_q;             // host bound on new tokens per request (sizes the grid)
  float scale_log2;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  const int32_t* prefix_lens;
  __nv_bfloat16* out;           // [total_q, H, 128]
  float* lse;                   // [total_q, H]
  int total_q, total_kv;        // rows of q/out/lse and of k/v
  unsigned* status;
  // paged K/V (page_table non-null): row j of request b is row j % page_size of page
  // page_table[b * max_pages + j / page_size]; kv_lens[b] = prefix + new tokens
  const int32_t* page_table;
  const int32_t* kv_lens;
  int page_size, max_pages;
  int64_t num_pages;
};

// One pass that norms and rotates queries and latent keys and writes the keys into the pages.
struct AppendParams {
  const __nv_bfloat16* q_in;    // null: keys only
  __nv_bfloat16* q_out;
  int64_t q_in_token, q_in_head, q_out_token, q_out_head;  // strides in elements
  int heads, q_dim;
  const __nv_bfloat16* q_weight;   // [q_dim] or null (no norm)
  const __nv_bfloat16* kv_in;      // null: queries only
  int64_t kv_in_token;
  const __nv_bfloat16* kv_weight;  // [512] or null (no norm)
  float eps;
  const float* cos_sin;         // [max_positions][64]: 32 cosines, 32 sines
  int max_positions;
  const int32_t* positions;
  const int64_t* slots;
  int tokens;
  int interleaved;
  uint8_t* kv_pages;
  int64_t num_slots;
  int kv_dtype;
  float kv_scale;
  unsigned* status;
};

// Pages of a cache: counts of the table entries that refer to each.
struct ForkParams {
  uint8_t* kv_pages;
  int num_pages, page_size, row_bytes;
  float* page_scales;           // kKvInt8Page: [num_pages]
  int32_t* page_table;          // [slots][max_pages]
  int max_pages;
  int32_t* seq_lens;            // [slots]
  int slots;
  int32_t* refs;                // [num_pages]
  const int32_t* parents;       // [n] slots
  const int32_t* children;
  const int32_t* new_pages;
  int n;
  unsigned* status;
};

struct FreeParams {
  const int32_t* page_table;
  int max_pages;
  int32_t* seq_lens;
  int slots, page_size;
  int32_t* refs;
  int num_pages;
  const int32_t* list;          // [n] slots
  const int32_t* keep_lens;
  int n;
  int32_t* freed;
  int32_t* num_freed;
  unsigned* status;
};

struct CompactParams {
  uint8_t* kv_pages;
  int num_pages, page_size, row_bytes;
  float* page_scales;
  int32_t* page_table;
  int max_pages;
  const int32_t* seq_lens;
  int slots;
  int32_t* refs;
  int32_t* num_live;
  // workspace: live pages and moves; where each page from the live ones on goes (-1: nowhere); holes ascending; pages that
  // move, from the last and from the first
  int32_t* head;
  int32_t* remap;
  int32_t* holes;
  int32_t* movers;
  int32_t* movers_up;
  unsigned* status;
};

// Rows of requests out of the pages, as contiguous bf16 rows.
struct GatherParams {
  const uint8_t* kv_pages;
  int64_t num_pages;
  int page_size, kv_dtype;
  float kv_scale;
  const float* page_scales;     // kKvInt8Page: [num_pages]
  const int32_t* page_table;
  int max_pages, B, total;
  const int32_t* cu_rows;       // [B + 1]
  __nv_bfloat16* out;
  int64_t out_stride;           // elements
  unsigned* status;
};

// Eviction: selection of the kept keys, then the copy of their rows into new pages.
struct EvictParams {
  uint8_t* kv_pages;
  int64_t num_pages;
  int page_size, row_bytes;
  const int32_t* page_table;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* keep_lens;
  const float* mass;
  int64_t mass_stride;
  const int32_t* dst_page_table;
  int max_dst_pages;
  int B, sink, recent, max_seq, max_keep;
  int32_t* kept;
  int64_t kept_stride;
  int32_t* new_lens;
  float* mass_out;
  int64_t mass_out_stride;
  int cached;                   // images a CTA keeps in shared memory (launch_kv_evict)
  unsigned* status;
};

// Attention weight of each key of a decode step, accumulated.
struct KeyMassParams {
  int B, T, H, R;               // R = T*H folded rows per request
  int page_size, max_pages, max_seq;
  int kv_dtype;
  int64_t num_pages;
  float scale_log2;             // softmax scale * log2(e) (* kv_scale for an 8-bit pool)
  float decay;
  const __nv_bfloat16* q;       // [B, T, H, 576]
  const uint8_t* kv_pool;
  const float* page_scales;     // kKvInt8Page: [num_pages]
  float inv_ref_scale;          // kKvInt8Page: 1 / kv_scale
  const int32_t* page_table;
  const int32_t* seq_lens;
  const uint64_t* tree_mask;    // [B, T], or null: drafts in order
  const float* lse;             // [B, T, H]
  float* mass;                  // row b at b * mass_stride
  int64_t mass_stride;
  float* part;                  // row groups' sums [groups, B, max_seq] (more than one group)
  int group_rows, groups, sets, stages, raw_stages;  // launch shape (launch_key_mass)
  unsigned* status;
};

// Host helpers of mla_api.cu that every entry point uses.
unsigned* status_ptr();  // device address of the current device's status word
// Tiled tensor map (128-byte swizzle unless given).  dims/strides innermost first; strides
// in bytes for dims 1..rank-1.
bool make_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const uint64_t* dims,
              const uint64_t* strides, const uint32_t* box,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
inline bool kv_dtype_ok(int t) { return t >= kKvBf16 && t <= kKvFp4; }
inline int kv_row_bytes(int t) { return t == kKvBf16 ? 2 * kLatentDim : t == kKvFp4 ? kFp4RowBytes : kLatentDim; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool page_size_ok(int P) { return P == 8 || P == 16 || P == 32 || P == 64 || P == 128 || P == 256; }

cudaError_t launch_page_fork(const ForkParams& p, cudaStream_t stream);
cudaError_t launch_page_free(const FreeParams& p, cudaStream_t stream);
cudaError_t launch_page_compact(const CompactParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_gather(const GatherParams& p, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
// tm_q: bf16 pools only.
cudaError_t launch_key_mass(const KeyMassParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv, int num_sms,
                            cudaStream_t stream);
int key_mass_group_rows(int R);  // query rows a CTA holds: the height of tm_q's box
size_t key_mass_part_bytes(int B, int R, int max_seq);  // scratch of KeyMassParams::part
cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t stream);

// Decode: split-KV partial kernel (tensor maps over q and the latent pool).
cudaError_t launch_decode_partial(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv,
                                  int head_groups, cudaStream_t stream);
// Decode over an e4m3 pool: the split-KV partial kernel that runs BMM1 on the raw codes.
cudaError_t launch_decode_partial_e4m3(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv,
                                       int head_groups, cudaStream_t stream);
// Decode over a bf16 pool for requests of at most 32 folded rows (trees: 48): Q held in
// tensor memory, a three-tile ring (mla_decode_narrow_sm103a.cu).
cudaError_t launch_decode_partial_narrow(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv,
                                         cudaStream_t stream);
// Decode over a 4-bit pool (trees too).
cudaError_t launch_decode_partial_fp4(const DecodeParams& p, const CUtensorMap& tm_kv, cudaStream_t stream);
int fp4_group_rows(int R);  // folded rows per CTA
// Tree decode over a bf16 pool for requests of more than kTreeNarrowRows folded rows (pairs of CTAs).
cudaError_t launch_decode_tree_pair(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t stream);
int tree_pair_groups(int R);  // pairs along the folded row axis
// Decode: LSE-merge of the split partials for requests with more than one split.
cudaError_t launch_decode_combine(const DecodeParams& p, cudaStream_t stream);
// Watchdog self-test kernel (a wait nothing satisfies; must time out and report).
cudaError_t launch_selftest_timeout(unsigned* status, cudaStream_t stream);
// Prefill: ragged causal prefill with prefix offset (contiguous or paged K/V, by p.page_table).
cudaError_t launch_prefill(const PrefillParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                           const CUtensorMap& tm_v, cudaStream_t stream);

}  // namespace mla
