// mla_pages_api.cu -- host side of the entry points that keep the pages of a cache (include/mla.h): fork, free and
// compact.  Argument checks run before anything is enqueued; nothing is allocated and no stream is synchronised.
#include <cstring>

#include "../../include/mla.h"
#include "mla_internal.h"

using namespace mla;

namespace {

struct Span {
  const void* at;
  size_t bytes;
};

// Whether one of `written` shares memory with another of them or with one of `read` (empty spans do not).
template <size_t W, size_t R>
bool clash(const Span (&written)[W], const Span (&read)[R]) {
  const auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.at && b.at && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
  };
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return true;
    for (size_t j = 0; j < R; ++j)
      if (meet(written[i], read[j])) return true;
  }
  return false;
}

// Pages are int32, with room above for the scan's strides.
bool pages_ok(int64_t num_pages) { return num_pages >= 1 && num_pages <= (int64_t(1) << 30); }

}  // namespace

extern "C" {

int mla_page_fork(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float* page_scales, int32_t* page_table,
                  int max_pages_per_seq, int32_t* seq_lens, int num_slots, int32_t* refs, const int32_t* parents,
                  const int32_t* children, const int32_t* new_pages, int count, void* stream) {
  if (count < 0 || num_slots < 1 || max_pages_per_seq < 1 || !pages_ok(num_pages) || !kv_dtype_ok(kv_dtype)) return MLA_ERR_INVALID_ARG;
  if ((kv_dtype == MLA_KV_INT8_PAGE) != (page_scales != nullptr)) return MLA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || count > 65535) return MLA_ERR_UNSUPPORTED;
  if (count == 0) return MLA_OK;
  if (!kv_pages || !page_table || !seq_lens || !refs || !parents || !children || !new_pages) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(page_scales, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(refs, 4) ||
      !aligned(parents, 4) || !aligned(children, 4) || !aligned(new_pages, 4))
    return MLA_ERR_INVALID_ARG;
  const size_t N = static_cast<size_t>(num_pages), n = static_cast<size_t>(count) * 4;
  const Span written[] = {{kv_pages, N * page_size * kv_row_bytes(kv_dtype)}, {page_scales, N * 4},
                          {page_table, static_cast<size_t>(num_slots) * max_pages_per_seq * 4},
                          {seq_lens, static_cast<size_t>(num_slots) * 4}, {refs, N * 4}};
  const Span read[] = {{parents, n}, {children, n}, {new_pages, n}};
  if (clash(written, read)) return MLA_ERR_INVALID_ARG;
  ForkParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.kv_pages = static_cast<uint8_t*>(kv_pages);
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = page_size;
  p.row_bytes = kv_row_bytes(kv_dtype);
  p.page_scales = page_scales;
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.slots = num_slots;
  p.refs = refs;
  p.parents = parents;
  p.children = children;
  p.new_pages = new_pages;
  p.n = count;
  return launch_page_fork(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_page_free(const int32_t* page_table, int max_pages_per_seq, int32_t* seq_lens, int num_slots, int page_size, int32_t* refs,
                  int64_t num_pages, const int32_t* slots, const int32_t* keep_lens, int count, int32_t* freed, int32_t* num_freed,
                  void* stream) {
  if (count < 0 || num_slots < 1 || max_pages_per_seq < 1 || !pages_ok(num_pages)) return MLA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || count > 65535) return MLA_ERR_UNSUPPORTED;
  if (!refs || !freed || !num_freed || (count > 0 && (!page_table || !seq_lens || !slots || !keep_lens))) return MLA_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(refs, 4) || !aligned(slots, 4) || !aligned(keep_lens, 4) ||
      !aligned(freed, 4) || !aligned(num_freed, 4))
    return MLA_ERR_INVALID_ARG;
  const size_t N = static_cast<size_t>(num_pages), n = static_cast<size_t>(count) * 4;
  const Span written[] = {{seq_lens, count ? static_cast<size_t>(num_slots) * 4 : 0}, {refs, N * 4}, {freed, N * 4}, {num_freed, 4}};
  const Span read[] = {{page_table, count ? static_cast<size_t>(num_slots) * max_pages_per_seq * 4 : 0}, {slots, n}, {keep_lens, n}};
  if (clash(written, read)) return MLA_ERR_INVALID_ARG;
  FreeParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.slots = num_slots;
  p.page_size = page_size;
  p.refs = refs;
  p.num_pages = static_cast<int>(num_pages);
  p.list = slots;
  p.keep_lens = keep_lens;
  p.n = count;
  p.freed = freed;
  p.num_freed = num_freed;
  return launch_page_free(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_page_compact_workspace(int64_t num_pages, size_t* bytes_out) {
  if (!bytes_out || !pages_ok(num_pages)) return MLA_ERR_INVALID_ARG;
  // head | where each page goes | holes, pages that move (from the last, from the first): at most half of the pages each
  const size_t N = static_cast<size_t>(num_pages), half = N / 2 + 1;
  *bytes_out = 256 + 4 * (N + 3 * half);
  return MLA_OK;
}

int mla_page_compact(void* kv_pages, int64_t num_pages, int page_size, int kv_dtype, float* page_scales, int32_t* page_table,
                     int max_pages_per_seq, const int32_t* seq_lens, int num_slots, int32_t* refs, int32_t* num_live,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (num_slots < 1 || max_pages_per_seq < 1 || !pages_ok(num_pages) || !kv_dtype_ok(kv_dtype)) return MLA_ERR_INVALID_ARG;
  if ((kv_dtype == MLA_KV_INT8_PAGE) != (page_scales != nullptr)) return MLA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED;
  if (!kv_pages || !page_table || !seq_lens || !refs || !num_live || !workspace) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(page_scales, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(refs, 4) ||
      !aligned(num_live, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  size_t need = 0;
  mla_page_compact_workspace(num_pages, &need);
  if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const size_t N = static_cast<size_t>(num_pages), half = N / 2 + 1;
  const Span written[] = {{kv_pages, N * page_size * kv_row_bytes(kv_dtype)}, {page_scales, N * 4},
                          {page_table, static_cast<size_t>(num_slots) * max_pages_per_seq * 4}, {refs, N * 4}, {num_live, 4},
                          {workspace, need}};
  const Span read[] = {{seq_lens, static_cast<size_t>(num_slots) * 4}};
  if (clash(written, read)) return MLA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MLA_ERR_CUDA;
  CompactParams p;
  memset(&p, 0, sizeof p);
  p.status = status_ptr();
  if (!p.status) return MLA_ERR_CUDA;
  p.kv_pages = static_cast<uint8_t*>(kv_pages);
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = page_size;
  p.row_bytes = kv_row_bytes(kv_dtype);
  p.page_scales = page_scales;
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.slots = num_slots;
  p.refs = refs;
  p.num_live = num_live;
  p.head = static_cast<int32_t*>(workspace);
  p.remap = p.head + 64;
  p.holes = p.remap + N;
  p.movers = p.holes + half;
  p.movers_up = p.movers + half;
  return launch_page_compact(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
