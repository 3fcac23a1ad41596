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
// Selection: a radix select over the order-preserving 32-bit image of the masses (three
// passes of 11, 11 and 10 bits, counted in shared memory), then one pass that emits the kept
// indices in order.  Bound by latency (a few hundred KB per request): a request of many keys
// is spread over a cluster of CTAs, each keeping the images of its share in shared memory;
// they read each other's counts there, one cluster barrier a pass.
// Copy: bound by memory.  A warp copies a few consecutive rows with all their loads in
// flight before the first store.
#include <cooperative_groups.h>

#include <algorithm>

#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kCluster = 8;            // CTAs per request
constexpr int kMaxCached = 48 * 1024;  // images a CTA keeps in shared memory; longer shares are read again
constexpr int kOneCtaKeys = 8192;      // up to this length a request has one CTA
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

// Keys of a CTA's share: whole rounds of 32 lanes for each of the 32 warps.
__host__ __device__ inline int share_of(int span, int ctas) {
  const int per_warp = (span + ctas * kSelectThreads - 1) / (ctas * kSelectThreads) * 32;
  return per_warp * kSelectWarps;
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t images[];  // p.cached of them
  __shared__ int hist[3][kBins];
  __shared__ int warp_sum[kSelectWarps];
  __shared__ int s_digit, s_need;
  __shared__ int2 warp_count[kSelectWarps];
  __shared__ int2 cta_count;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int L;
  const int K = keep_count(p, b, L);
  if (K < 0) {  // (every return before a cluster barrier is the whole cluster's)
    if (tid == 0 && rank == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const int lo = min(p.sink, K);
  const int tail = min(p.recent, K - lo);
  const int hi = L - tail;
  const int m = K - lo - tail;  // to choose from [lo, hi)
  int32_t* kept = p.kept + static_cast<int64_t>(b) * p.kept_stride;
  if (tid == 0 && rank == 0) p.new_lens[b] = K;
  for (int i = rank * kSelectThreads + tid; i < lo; i += ctas * kSelectThreads) kept[i] = i;
  for (int i = rank * kSelectThreads + tid; i < tail; i += ctas * kSelectThreads) kept[K - tail + i] = hi + i;
  if (m == 0) return;
  const int share = share_of(hi - lo, ctas);
  const int first = lo + static_cast<int>(min(static_cast<int64_t>(rank) * share, static_cast<int64_t>(hi - lo)));
  const int n = min(share, hi - first);
  const float* mass = p.mass + static_cast<int64_t>(b) * p.mass_stride + first;
  const bool cached = share <= p.cached;
  auto image = [&](int i) -> uint32_t { return cached ? images[i] : mass_key(mass[i]); };

  // threshold: the m-th largest image; `need` of the images equal to it are kept
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  uint32_t prefix = 0;
  int need = m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    if (pass == 0) {
#pragma unroll 8
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t k = mass_key(mass[i]);
        if (cached) images[i] = k;
        atomicAdd(&hist[0][k >> 21], 1);
      }
    } else {
      const int known = pass == 1 ? 21 : 10;  // the bits above are the prefix
      const uint32_t mask = pass == 1 ? kBins - 1 : 1023;
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t k = image(i);
        if (((k ^ prefix) >> known) == 0) atomicAdd(&hist[pass][(k >> shift) & mask], 1);
      }
    }
    cluster.sync();
    // every CTA sums the cluster's counts and scans them from the largest digit down
    int c[2] = {0, 0};
    const int bin = kBins - 1 - 2 * tid;  // this thread: bins bin and bin - 1
    for (int r = 0; r < ctas; ++r) {
      const int* h = cluster.map_shared_rank(&hist[pass][0], r);
      c[0] += h[bin];
      c[1] += h[bin - 1];
    }
    int incl = c[0] + c[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - c[0] - c[1];
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (before < need && need <= before + c[0] + c[1]) {  // (one thread)
      const bool up = need <= before + c[0];
      s_digit = up ? bin : bin - 1;
      s_need = up ? need - before : need - before - c[0];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_need;
  }
  // emission in order: heavier and equal keys before this warp, then round by round
  const int per_warp = share / kSelectWarps, w0 = warp * per_warp;
  int gt = 0, eq = 0;
  for (int i = w0 + lane; i < w0 + per_warp; i += 32) {
    const uint32_t k = i < n ? image(i) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < n && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < n && k == prefix));
  }
  if (lane == 0) warp_count[warp] = make_int2(gt, eq);
  __syncthreads();
  int2 at = make_int2(0, 0), all = make_int2(0, 0);
  for (int w = 0; w < kSelectWarps; ++w) {
    if (w == warp) at = all;
    all.x += warp_count[w].x;
    all.y += warp_count[w].y;
  }
  if (tid == 0) cta_count = all;
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const int2 v = *cluster.map_shared_rank(&cta_count, r);
    at.x += v.x;
    at.y += v.y;
  }
  for (int i = w0 + lane; i < w0 + per_warp; i += 32) {
    const uint32_t k = i < n ? image(i) : 0u;
    const bool g = i < n && k > prefix, e = i < n && k == prefix;
    const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    const unsigned below = (1u << lane) - 1u;
    const int gr = at.x + __popc(bg & below), er = at.y + __popc(be & below);
    if (g || (e && er < need)) kept[lo + gr + min(er, need)] = first + i;
    at.x += __popc(bg);
    at.y += __popc(be);
  }
  cluster.sync();  // no CTA leaves while another may read its counts
}

// kChunks: 16-byte pieces of a row (72 of bf16, 36 of 8-bit codes).
template <int kChunks>
__global__ void __launch_bounds__(32 * kCopyWarps) kv_copy_kernel(const EvictParams p) {
  constexpr int kRows = 288 / kChunks;  // rows a warp copies: 9 pieces a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kCopyWarps + (threadIdx.x >> 5)) * kRows;
  int L;
  const int K = keep_count(p, b, L);
  if (i0 >= K) return;
  // lanes 0 .. kRows-1: where a row comes from and goes to (in pieces; -1: nowhere)
  int64_t src = -1, dst = -1;
  const int i = i0 + lane, P = p.page_size;
  if (lane < kRows && i < K) {
    const int j = p.kept[static_cast<int64_t>(b) * p.kept_stride + i];
    const int64_t from = p.page_table[static_cast<int64_t>(b) * p.max_pages + j / P];
    const int64_t to = p.dst_page_table[static_cast<int64_t>(b) * p.max_dst_pages + i / P];
    p.mass_out[static_cast<int64_t>(b) * p.mass_out_stride + i] = p.mass[static_cast<int64_t>(b) * p.mass_stride + j];
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
      atomicOr(p.status, kStatusDeviceArg);
    } else {
      src = (from * P + j % P) * kChunks;
      dst = (to * P + i % P) * kChunks;
    }
  }
  uint4* pool = reinterpret_cast<uint4*>(p.kv_pages);
  uint4 v[9];
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int c = lane + 32 * k;
    const int64_t s = __shfl_sync(0xffffffffu, src, c / kChunks);
    if (s >= 0) v[k] = __ldcs(pool + s + c % kChunks);
  }
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int c = lane + 32 * k;
    const int64_t d = __shfl_sync(0xffffffffu, dst, c / kChunks);
    if (d >= 0) pool[d + c % kChunks] = v[k];
  }
}

template <typename K>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, int cluster, const EvictParams& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& params, cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  EvictParams p = params;
  // one CTA walks a short request faster than a cluster meets
  const int ctas = p.max_seq <= kOneCtaKeys ? 1 : kCluster;
  p.cached = std::min(share_of(std::max(p.max_seq, 1), ctas), kMaxCached);
  e = launch_dependent(kv_select_kernel, dim3(p.B * ctas), kSelectThreads, p.cached * 4, ctas, p, stream);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  const int rows = (p.row_bytes == 2 * kLatentDim ? 4 : 8) * kCopyWarps;
  const dim3 grid((p.max_keep + rows - 1) / rows, p.B);
  return p.row_bytes == 2 * kLatentDim ? launch_dependent(kv_copy_kernel<72>, grid, 32 * kCopyWarps, 0, 1, p, stream)
                                       : launch_dependent(kv_copy_kernel<36>, grid, 32 * kCopyWarps, 0, 1, p, stream);
}

}  // namespace mla
