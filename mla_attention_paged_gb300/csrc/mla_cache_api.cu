// mla_cache_api.cu -- host side of the entry points that keep the paged latent cache
// (include/mla.h): mla_kv_append writes it, mla_key_mass weighs its keys and mla_kv_evict
// shrinks it.
// Argument checks run before anything is enqueued; nothing is allocated and no stream is
// synchronised.
#include <cstring>

#include "../../include/mla.h"
#include "mla_internal.h"

using namespace mla;

namespace {

// Whether heads x tokens rows of `dim` elements at these strides are rows of their own.
bool rows_apart(int64_t token, int64_t head, int tokens, int heads, int dim) {
  if (token < 0 || head < 0) return false;
  if (tokens == 1 && heads == 1) return true;
  if (tokens == 1) return head >= dim;
  if (heads == 1) return token >= dim;
  return (head >= dim && token >= (heads - 1) * head + dim) || (token >= dim && head >= (tokens - 1) * token + dim);
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// Whether two sets of `rows` rows (addresses, strides and lengths in bytes) share memory.  Rows of one
// stride may lie side by side, as column ranges of one buffer; of two strides, the spans decide.
bool rows_overlap(const void* a, int64_t a_stride, int64_t a_len, const void* b, int64_t b_stride, int64_t b_len, int64_t rows) {
  if (a_len == 0 || b_len == 0) return false;
  if (!overlap(a, (rows - 1) * a_stride + a_len, b, (rows - 1) * b_stride + b_len)) return false;
  if (a_stride != b_stride || rows == 1) return true;
  // row i + k of b lies at `off` + k strides from row i of a, k in (-rows, rows)
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t k0 = -off / a_stride;  // the rows of b that come near a's
  for (int64_t k = k0 - 1; k <= k0 + 1; ++k)
    if (k > -rows && k < rows && off + k * b_stride < a_len && off + k * b_stride + b_len > 0) return true;
  return false;
}

}  // namespace

extern "C" {

int mla_kv_append(const void* q_in, int64_t q_in_token_stride, int64_t q_in_head_stride, void* q_out,
                  int64_t q_out_token_stride, int64_t q_out_head_stride, int num_heads, int q_dim,
                  const void* q_weight, const void* kv_in, int64_t kv_in_token_stride, const void* kv_weight, float eps,
                  const float* cos_sin, int max_positions, const int32_t* positions, const int64_t* slots,
                  int num_tokens, int interleaved, void* kv_pages, int64_t num_slots, int kv_dtype, float kv_scale,
                  void* stream) {
  const bool has_q = q_in != nullptr, has_kv = kv_in != nullptr;
  if (num_tokens < 0 || max_positions < 1 || !(eps >= 0.f)) return MLA_ERR_INVALID_ARG;
  if (!kv_dtype_ok(kv_dtype)) return MLA_ERR_INVALID_ARG;
  if (has_q) {
    if (num_heads < 1 || q_in_token_stride < 0 || q_in_head_stride < 0) return MLA_ERR_INVALID_ARG;
    if (num_heads > 1024 || q_dim < 64 || q_dim > 576 || q_dim % 8 != 0) return MLA_ERR_UNSUPPORTED;
  }
  if (num_tokens > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  // the scale of a page that already holds rows cannot follow a new row's range
  if (has_kv && kv_dtype == MLA_KV_INT8_PAGE) return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLA_OK;
  if (!has_q && !has_kv) return MLA_ERR_INVALID_ARG;
  if (!cos_sin || !positions || !aligned(cos_sin, 16) || !aligned(positions, 4)) return MLA_ERR_INVALID_ARG;
  const size_t pool_bytes = num_slots < 1 ? 0 : static_cast<size_t>(num_slots) * kv_row_bytes(kv_dtype);
  if (has_q) {
    if (!q_out || !aligned(q_in, 16) || !aligned(q_out, 16) || (q_weight && !aligned(q_weight, 16)))
      return MLA_ERR_INVALID_ARG;
    if ((q_in_token_stride | q_in_head_stride | q_out_token_stride | q_out_head_stride) % 8 != 0)
      return MLA_ERR_INVALID_ARG;
    if (!rows_apart(q_out_token_stride, q_out_head_stride, num_tokens, num_heads, q_dim)) return MLA_ERR_INVALID_ARG;
    // in place, or apart: a warp writes its row while others still read theirs
    const bool in_place = q_in == q_out && (num_tokens == 1 || q_in_token_stride == q_out_token_stride) &&
                          (num_heads == 1 || q_in_head_stride == q_out_head_stride);
    const auto span = [&](int64_t token, int64_t head) {
      return static_cast<size_t>((num_tokens - 1) * token + (num_heads - 1) * head + q_dim) * 2;
    };
    const size_t in_span = span(q_in_token_stride, q_in_head_stride), out_span = span(q_out_token_stride, q_out_head_stride);
    if (!in_place && overlap(q_in, in_span, q_out, out_span)) return MLA_ERR_INVALID_ARG;
    // the same pass writes the pool's rows
    if (has_kv && (overlap(q_in, in_span, kv_pages, pool_bytes) || overlap(q_out, out_span, kv_pages, pool_bytes)))
      return MLA_ERR_INVALID_ARG;
  }
  if (has_kv) {
    if (!kv_pages || !slots || num_slots < 1 || !aligned(kv_in, 16) || !aligned(kv_pages, 16) || !aligned(slots, 8) ||
        (kv_weight && !aligned(kv_weight, 16)) || kv_in_token_stride < 0 || kv_in_token_stride % 8 != 0)
      return MLA_ERR_INVALID_ARG;
    if (kv_dtype != MLA_KV_BF16 && !(kv_scale > 0.f)) return MLA_ERR_INVALID_ARG;
    // a row may be written while another of the pool's is still to be read
    if (overlap(kv_in, static_cast<size_t>((num_tokens - 1) * kv_in_token_stride + kLatentDim) * 2, kv_pages, pool_bytes))
      return MLA_ERR_INVALID_ARG;
  }
  AppendParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  if (has_q) {
    p.q_in = static_cast<const __nv_bfloat16*>(q_in);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.q_in_token = q_in_token_stride;
    p.q_in_head = q_in_head_stride;
    p.q_out_token = q_out_token_stride;
    p.q_out_head = q_out_head_stride;
    p.heads = num_heads;
    p.q_dim = q_dim;
    p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  }
  if (has_kv) {
    p.kv_in = static_cast<const __nv_bfloat16*>(kv_in);
    p.kv_in_token = kv_in_token_stride;
    p.kv_weight = static_cast<const __nv_bfloat16*>(kv_weight);
    p.slots = slots;
    p.kv_pages = static_cast<uint8_t*>(kv_pages);
    p.num_slots = num_slots;
  }
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.max_positions = max_positions;
  p.positions = positions;
  p.tokens = num_tokens;
  p.interleaved = interleaved;
  p.kv_dtype = kv_dtype;
  p.kv_scale = kv_scale;
  return launch_kv_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_kv_gather(const void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float kv_scale, const float* page_scales,
                  const int32_t* page_table, int max_pages_per_seq, const int32_t* cu_rows, int batch, int total_rows,
                  void* out, int64_t out_row_stride, void* stream) {
  if (batch < 1 || total_rows < 0 || num_pages < 1 || max_pages_per_seq < 1 || !kv_dtype_ok(kv_dtype)) return MLA_ERR_INVALID_ARG;
  if ((kv_dtype == MLA_KV_INT8_PAGE) != (page_scales != nullptr)) return MLA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED;
  if (total_rows == 0) return MLA_OK;
  if (!kv_pages || !page_table || !cu_rows || !out) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(page_scales, 4) || !aligned(page_table, 4) || !aligned(cu_rows, 4) || !aligned(out, 16))
    return MLA_ERR_INVALID_ARG;
  if (out_row_stride < kLatentDim || out_row_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_INT8_PAGE && !(kv_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  // rows are written while others of the pool, and lengths, are still to be read
  const size_t span = (static_cast<size_t>(total_rows - 1) * out_row_stride + kLatentDim) * 2;
  if (overlap(kv_pages, static_cast<size_t>(num_pages) * page_size * kv_row_bytes(kv_dtype), out, span) ||
      overlap(page_table, static_cast<size_t>(batch) * max_pages_per_seq * 4, out, span) ||
      overlap(cu_rows, (static_cast<size_t>(batch) + 1) * 4, out, span) ||
      (page_scales && overlap(page_scales, static_cast<size_t>(num_pages) * 4, out, span)))
    return MLA_ERR_INVALID_ARG;
  GatherParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.kv_pages = static_cast<const uint8_t*>(kv_pages);
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.kv_dtype = kv_dtype;
  p.kv_scale = kv_scale;
  p.page_scales = page_scales;
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.B = batch;
  p.total = total_rows;
  p.cu_rows = cu_rows;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride = out_row_stride;
  return launch_kv_gather(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_key_mass_workspace(const mla_decode_plan_t* plan, size_t* bytes_out) {
  if (!plan || !bytes_out) return MLA_ERR_INVALID_ARG;
  *bytes_out = key_mass_part_bytes(plan->batch, plan->rows, plan->max_seq_len);
  return MLA_OK;
}

int mla_key_mass(const mla_decode_plan_t* plan, const void* q, const void* kv_pages, const float* page_scales,
                 const int32_t* page_table, const int32_t* seq_lens, const uint64_t* tree_mask, const float* lse,
                 int q_len, int num_heads, float scale, float kv_scale, float decay, float* mass, int64_t mass_stride,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan || !q || !kv_pages || !page_table || !seq_lens || !lse || !mass) return MLA_ERR_INVALID_ARG;
  if ((plan->kv_dtype == MLA_KV_INT8_PAGE) != (page_scales != nullptr)) return MLA_ERR_INVALID_ARG;
  if (q_len != plan->q_len || num_heads != plan->num_heads || plan->rows != q_len * num_heads) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(page_scales, 4) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(tree_mask, 8) || !aligned(lse, 4) || !aligned(mass, 4))
    return MLA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(kv_scale > 0.f) || !(decay >= 0.f) || mass_stride < plan->max_seq_len) return MLA_ERR_INVALID_ARG;
  if (tree_mask && q_len > kMaxTreeDrafts) return MLA_ERR_UNSUPPORTED;
  if (plan->kv_dtype == MLA_KV_FP4) return MLA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(plan->batch) * (plan->max_seq_len / 128 + 1) >= (int64_t(1) << 31)) return MLA_ERR_UNSUPPORTED;
  size_t need = 0;
  mla_key_mass_workspace(plan, &need);
  if (need > 0) {
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  KeyMassParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.B = plan->batch;
  p.T = q_len;
  p.H = num_heads;
  p.R = plan->rows;
  p.page_size = plan->page_size;
  p.max_pages = plan->max_pages_per_seq;
  p.max_seq = plan->max_seq_len;
  p.kv_dtype = plan->kv_dtype;
  p.num_pages = plan->num_pages;
  p.scale_log2 = scale * 1.4426950408889634f * (plan->kv_dtype != MLA_KV_BF16 ? kv_scale : 1.f);
  p.decay = decay;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv_pool = static_cast<const uint8_t*>(kv_pages);
  p.page_scales = page_scales;
  p.inv_ref_scale = 1.f / kv_scale;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.tree_mask = tree_mask;
  p.lse = lse;
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.part = static_cast<float*>(workspace);
  // Queries as nine 128-byte-swizzled blocks of 64 columns; the pool as boxes of 64 columns by
  // a page's share of a 128-key tile.
  CUtensorMap tm_q, tm_kv;
  memset(&tm_q, 0, sizeof tm_q);
  memset(&tm_kv, 0, sizeof tm_kv);
  const uint64_t pool_rows = static_cast<uint64_t>(plan->num_pages) * plan->page_size;
  const uint32_t box_kv[2] = {64, static_cast<uint32_t>(plan->page_size < 128 ? plan->page_size : 128)};
  if (plan->kv_dtype == MLA_KV_BF16) {
    const uint64_t dims[3] = {64, static_cast<uint64_t>(plan->batch) * plan->rows, kLatentDim / 64};
    const uint64_t strides[2] = {kLatentDim * 2, 128};
    const uint32_t box[3] = {64, static_cast<uint32_t>(key_mass_group_rows(plan->rows)), kLatentDim / 64};
    const uint64_t kv_dims[2] = {kLatentDim, pool_rows};
    const uint64_t kv_strides[1] = {kLatentDim * 2};
    if (!make_map(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box) ||
        !make_map(&tm_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kv_pages, kv_dims, kv_strides, box_kv))
      return MLA_ERR_CUDA;
  } else {
    const uint64_t kv_dims[2] = {kLatentDim, pool_rows};
    const uint64_t kv_strides[1] = {kLatentDim};
    if (!make_map(&tm_kv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, kv_pages, kv_dims, kv_strides, box_kv,
                  plan->kv_dtype == MLA_KV_E4M3 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE))
      return MLA_ERR_CUDA;
  }
  return launch_key_mass(p, tm_q, tm_kv, plan->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK
                                                                                                           : MLA_ERR_CUDA;
}

int mla_kv_evict(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, const int32_t* page_table,
                 int max_pages_per_seq, const int32_t* seq_lens, const int32_t* keep_lens, const float* mass,
                 int64_t mass_stride, const int32_t* dst_page_table, int max_dst_pages, int batch, int sink, int recent,
                 int max_seq_len, int max_keep, int32_t* kept, int64_t kept_stride, int32_t* new_lens, float* mass_out,
                 int64_t mass_out_stride, void* stream) {
  if (batch < 1 || num_pages < 1 || max_pages_per_seq < 1 || max_dst_pages < 1 || sink < 0 || recent < 0 ||
      max_seq_len < 0 || max_keep < 0)
    return MLA_ERR_INVALID_ARG;
  if (!kv_dtype_ok(kv_dtype)) return MLA_ERR_INVALID_ARG;
  // a row's codes mean something else under another page's scale
  if (kv_dtype == MLA_KV_INT8_PAGE) return MLA_ERR_UNSUPPORTED;
  if (!page_size_ok(page_size) || batch > 65535 || max_seq_len > (1 << 24)) return MLA_ERR_UNSUPPORTED;
  if (!kv_pages || !page_table || !seq_lens || !keep_lens || !dst_page_table || !new_lens || (!mass && max_seq_len > 0) ||
      ((!kept || !mass_out) && max_keep > 0))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(keep_lens, 4) ||
      !aligned(mass, 4) || !aligned(dst_page_table, 4) || !aligned(kept, 4) || !aligned(new_lens, 4) ||
      !aligned(mass_out, 4))
    return MLA_ERR_INVALID_ARG;
  if (mass_stride < max_seq_len || kept_stride < max_keep || mass_out_stride < max_keep) return MLA_ERR_INVALID_ARG;
  // the copy reads mass while it writes mass_out, and lengths while it writes new ones
  const size_t B = static_cast<size_t>(batch);
  if (rows_overlap(mass, mass_stride * 4, int64_t(max_seq_len) * 4, mass_out, mass_out_stride * 4, int64_t(max_keep) * 4, batch) ||
      overlap(seq_lens, B * 4, new_lens, B * 4) || overlap(keep_lens, B * 4, new_lens, B * 4))
    return MLA_ERR_INVALID_ARG;
  EvictParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.kv_pages = static_cast<uint8_t*>(kv_pages);
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.row_bytes = kv_row_bytes(kv_dtype);
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.dst_page_table = dst_page_table;
  p.max_dst_pages = max_dst_pages;
  p.B = batch;
  p.sink = sink;
  p.recent = recent;
  p.max_seq = max_seq_len;
  p.max_keep = max_keep;
  p.kept = kept;
  p.kept_stride = kept_stride;
  p.new_lens = new_lens;
  p.mass_out = mass_out;
  p.mass_out_stride = mass_out_stride;
  return launch_kv_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
