// mla_evict_sm103a.cu -- eviction from the paged latent cache by accumulated attention
// weight, sm_103a: choose the keys that every request keeps and copy their rows, in order,
// into new pages.
//
// What it computes, per request b with L cached keys and K = min(keep_lens[b], L):
//   kept = the first min(sink, K) keys, the last min(recent, K - those) keys, and of the keys
//   between them the K - those heaviest by mass[b, j] (equal masses: the lower index; NaN is
//   the lightest; -0 equals 0), in ascending order;
//   row i of the request's destination pages = row kept[i] of its source pages;
//   mass_out[b, i] = mass[b, kept[i]];  new_lens[b] = K.
// Rows are copied, not moved in place: a source page may be a prefix that other requests
// share.
//
// Selection: a radix select over the order-preserving 32-bit image of the masses (four
// passes of 8 bits, counted in shared memory) gives the K-th heaviest value; one more pass
// emits the kept indices in order with a block scan.  Copy: bound by memory, one warp per
// row.
#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kCopyWarps = 8;

// Order-preserving image of a mass: larger mass, larger image; NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The request's kept count, or -1 for lengths that reach past the bounds the call was given.
__device__ __forceinline__ int keep_count(const EvictParams& p, int b, int& L) {
  L = p.seq_lens[b];
  const int keep = p.keep_lens[b];
  if (L < 0 || keep < 0 || L > p.max_seq || L > static_cast<int64_t>(p.max_pages) * p.page_size) return -1;
  const int K = min(keep, L);
  if (K > p.max_keep || K > static_cast<int64_t>(p.max_dst_pages) * p.page_size) return -1;
  return K;
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_need;
  __shared__ unsigned long long warp_tot[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x;
  const int tid = threadIdx.x;
  int L;
  const int K = keep_count(p, b, L);
  if (K < 0) {
    if (tid == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const int lo = min(p.sink, K);
  const int tail = min(p.recent, K - lo);
  const int hi = L - tail;
  const int m = K - lo - tail;  // to choose from [lo, hi)
  const float* mass = p.mass + static_cast<int64_t>(b) * p.mass_stride;
  int32_t* kept = p.kept + static_cast<int64_t>(b) * p.kept_stride;
  if (tid == 0) p.new_lens[b] = K;
  for (int i = tid; i < lo; i += kSelectThreads) kept[i] = i;
  for (int i = tid; i < tail; i += kSelectThreads) kept[K - tail + i] = hi + i;
  if (m == 0) return;
  // threshold: the m-th largest image; `need` of the images equal to it are kept
  uint32_t prefix = 0;
  int need = m;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = lo + tid; i < hi; i += kSelectThreads) {
      const uint32_t k = mass_key(mass[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, left = need;
      while (left > hist[d]) left -= hist[d--];
      s_digit = d;
      s_need = left;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_need;
    __syncthreads();
  }
  // emission in order: a scan of (heavier, equal) counts
  int gt_base = 0, eq_base = 0;
  for (int c = lo; c < hi; c += kSelectThreads) {
    const int i = c + tid;
    const uint32_t k = i < hi ? mass_key(mass[i]) : 0u;
    const bool gt = i < hi && k > prefix, eq = i < hi && k == prefix;
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const int lane = tid & 31, warp = tid >> 5;
    if (lane == 0) warp_tot[warp] = (static_cast<unsigned long long>(__popc(bg)) << 32) | __popc(be);
    __syncthreads();
    unsigned long long before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w == warp) before = all;
      all += warp_tot[w];
    }
    const unsigned below = (1u << lane) - 1u;
    const int gt_rank = gt_base + static_cast<int>(before >> 32) + __popc(bg & below);
    const int eq_rank = eq_base + static_cast<int>(before & 0xffffffffull) + __popc(be & below);
    if (gt || (eq && eq_rank < need)) kept[lo + gt_rank + min(eq_rank, need)] = i;
    gt_base += static_cast<int>(all >> 32);
    eq_base += static_cast<int>(all & 0xffffffffull);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(32 * kCopyWarps) kv_copy_kernel(const EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  int L;
  const int K = keep_count(p, b, L);
  if (i >= K) return;
  const int j = p.kept[static_cast<int64_t>(b) * p.kept_stride + i];
  const int P = p.page_size;
  const int64_t src_page = p.page_table[static_cast<int64_t>(b) * p.max_pages + j / P];
  const int64_t dst_page = p.dst_page_table[static_cast<int64_t>(b) * p.max_dst_pages + i / P];
  if (lane == 0)
    p.mass_out[static_cast<int64_t>(b) * p.mass_out_stride + i] = p.mass[static_cast<int64_t>(b) * p.mass_stride + j];
  if (src_page < 0 || src_page >= p.num_pages || dst_page < 0 || dst_page >= p.num_pages) {
    if (lane == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(p.kv_pages + (src_page * P + j % P) * p.row_bytes);
  uint4* dst = reinterpret_cast<uint4*>(p.kv_pages + (dst_page * P + i % P) * p.row_bytes);
  for (int c = lane; c < p.row_bytes / 16; c += 32) dst[c] = src[c];
}

template <typename K>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, const EvictParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t stream) {
  cudaError_t e = launch_dependent(kv_select_kernel, dim3(p.B), kSelectThreads, p, stream);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  return launch_dependent(kv_copy_kernel, dim3((p.max_keep + kCopyWarps - 1) / kCopyWarps, p.B), 32 * kCopyWarps, p, stream);
}

}  // namespace mla
