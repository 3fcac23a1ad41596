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
// one warp of each reads the cluster's counts through distributed shared memory in two steps
// (64 sums of 32 bins, then the bins of one), one cluster barrier a pass.  The loops are left
// rolled: the kernel runs once through its code, and fully unrolled it waited 2,300 cycles
// a pass for instructions, whatever the number of keys.
// Copy: bound by memory.  A warp copies a few consecutive rows with all their loads in
// flight before the first store.
#include <cooperative_groups.h>

#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kCluster = 8;            // CTAs per request
constexpr int kCoarse = kBins / 32;    // sums of 32 bins
constexpr int kRound = 128;            // keys of a warp's round: four consecutive ones a lane
constexpr int kMaxCached = 48 * 1024;  // images a CTA keeps in shared memory; longer shares are read again
constexpr int kOneCtaKeys = 11264;      // up to this length a request has one CTA
constexpr int kCopyWarps = 8;
constexpr int kLanePieces = 9;         // 16-byte pieces a lane copies

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

// Keys of a CTA's share: whole rounds for each of its warps.
__host__ __device__ inline int share_of(int span, int ctas) {
  const int step = ctas * kSelectWarps * kRound;
  return (span + step - 1) / step * kSelectWarps * kRound;
}

// Sum over the warps before `warp` of one value per warp (in shared memory), and over all.
__device__ __forceinline__ int warps_before(const int* v, int warp, int lane, int& total) {
  const int own = v[lane];
  total = __reduce_add_sync(0xffffffffu, own);
  return __reduce_add_sync(0xffffffffu, lane < warp ? own : 0);
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int scan32(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// kCtas: CTAs per request (the cluster).
template <int kCtas>
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t images[];  // p.cached of them
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ __align__(16) int coarse[3][kCoarse];
  __shared__ int s_digit, s_need;
  __shared__ int warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  __shared__ int2 cta_count;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCtas == 1 ? 0 : static_cast<int>(cluster.block_rank());
  auto of = [&](int* x, int r) -> const int* { return kCtas == 1 ? x : cluster.map_shared_rank(x, r); };
  auto meet = [&]() {
    if (kCtas == 1) __syncthreads();
    else cluster.sync();
  };
  const int b = blockIdx.x / kCtas;
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
  for (int i = rank * kSelectThreads + tid; i < lo; i += kCtas * kSelectThreads) kept[i] = i;
  for (int i = rank * kSelectThreads + tid; i < tail; i += kCtas * kSelectThreads) kept[K - tail + i] = hi + i;
  if (m == 0) return;
  const int share = share_of(hi - lo, kCtas);
  const int first = lo + static_cast<int>(min(static_cast<int64_t>(rank) * share, static_cast<int64_t>(hi - lo)));
  const int n = min(share, hi - first);
  const float* mass = p.mass + static_cast<int64_t>(b) * p.mass_stride + first;
  const bool cached = share <= p.cached;
  const int rounds = share / (kSelectWarps * kRound);
  const int at0 = warp * rounds * kRound + 4 * lane;  // this lane's four keys of its warp's first round
  const int todo = min(rounds, max(0, (n - warp * rounds * kRound + kRound - 1) / kRound));  // rounds that hold keys
  auto fetch = [&](int i) -> uint4 {
    return make_uint4(i < n ? mass_key(mass[i]) : 0u, i + 1 < n ? mass_key(mass[i + 1]) : 0u,
                      i + 2 < n ? mass_key(mass[i + 2]) : 0u, i + 3 < n ? mass_key(mass[i + 3]) : 0u);
  };
  auto image4 = [&](int i) -> uint4 { return cached ? *reinterpret_cast<const uint4*>(images + i) : fetch(i); };

  for (int i = tid; i < 3 * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
  if (cached) {
#pragma unroll 4
    for (int r = 0; r < todo; ++r) *reinterpret_cast<uint4*>(images + at0 + r * kRound) = fetch(at0 + r * kRound);
  }
  __syncthreads();
  // threshold: the m-th largest image; `need` of the images equal to it are kept
  uint32_t prefix = 0;
  int need = m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit_mask = pass == 2 ? 1023 : kBins - 1;
    const uint32_t known = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);  // the bits of the prefix
    int* h = hist[pass];
#pragma unroll 1
    for (int r = 0; r < todo; ++r) {
      const int i = at0 + r * kRound;
      const uint4 k4 = image4(i);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < n && ((k[e] ^ prefix) & known) == 0) atomicAdd(&h[(k[e] >> shift) & digit_mask], 1);
    }
    __syncthreads();
    {
      const int2 two = *reinterpret_cast<const int2*>(h + 2 * tid);
      int s = two.x + two.y;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if ((lane & 15) == 0) coarse[pass][tid / 16] = s;
    }
    meet();
    if (warp == 0) {
      // from the largest digit down: the sum, then the bin, in which the m-th key falls
      const int c0 = kCoarse - 1 - 2 * lane;  // this lane's sums: c0 and c0 - 1
      int up = 0, down = 0;
#pragma unroll
      for (int r = 0; r < kCtas; ++r) {
        const int2 v = *reinterpret_cast<const int2*>(of(coarse[pass], r) + c0 - 1);
        up += v.y;
        down += v.x;
      }
      int before = scan32(up + down, lane) - up - down;
      bool mine = before < need && need <= before + up + down;
      int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      const bool first_of_two = need <= before + up;
      const int c = __shfl_sync(0xffffffffu, first_of_two ? c0 : c0 - 1, src);
      const int above = __shfl_sync(0xffffffffu, first_of_two ? before : before + up, src);
      const int bin = 32 * c + 31 - lane;
      int count = 0;
#pragma unroll
      for (int r = 0; r < kCtas; ++r) count += of(h, r)[bin];
      before = above + scan32(count, lane) - count;
      if (before < need && need <= before + count) {  // (one lane)
        s_digit = bin;
        s_need = need - before;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_need;
  }
  // emission in order: heavier and equal keys before this warp, then round by round
  int gt = 0, eq = 0;
#pragma unroll 1
  for (int r = 0; r < todo; ++r) {
    const int i = at0 + r * kRound;
    const uint4 k4 = image4(i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += i + e < n && k[e] > prefix;
      eq += i + e < n && k[e] == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  int all_gt, all_eq;
  gt = warps_before(warp_gt, warp, lane, all_gt);
  eq = warps_before(warp_eq, warp, lane, all_eq);
  if (kCtas > 1) {
    if (tid == 0) cta_count = make_int2(all_gt, all_eq);
    cluster.sync();
    const int2 v = lane < rank ? *cluster.map_shared_rank(&cta_count, lane) : make_int2(0, 0);
    gt += __reduce_add_sync(0xffffffffu, v.x);
    eq += __reduce_add_sync(0xffffffffu, v.y);
  }
#pragma unroll 1
  for (int r = 0; r < todo; ++r) {
    const int i = at0 + r * kRound;
    const uint4 k4 = image4(i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    int own = 0;  // heavier, and equal << 16, of this lane
#pragma unroll
    for (int e = 0; e < 4; ++e) own += i + e < n ? (k[e] > prefix ? 1 : k[e] == prefix ? 1 << 16 : 0) : 0;
    const int incl = scan32(own, lane), all = __shfl_sync(0xffffffffu, incl, 31);
    int g = gt + ((incl - own) & 0xffff), q = eq + ((incl - own) >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool heavy = i + e < n && k[e] > prefix, equal = i + e < n && k[e] == prefix;
      if (heavy || (equal && q < need)) kept[lo + g + min(q, need)] = first + i + e;
      g += heavy;
      q += equal;
    }
    gt += all & 0xffff;
    eq += all >> 16;
  }
  if (kCtas > 1) cluster.sync();  // no CTA leaves while another may read its counts
}

// kChunks: 16-byte pieces of a row (72 of bf16, 36 of 8-bit codes, 21 of a 4-bit row: 13 rows a warp).
template <int kChunks>
__global__ void __launch_bounds__(32 * kCopyWarps) kv_copy_kernel(const EvictParams p) {
  constexpr int kRows = 32 * kLanePieces / kChunks;  // rows a warp copies
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
  uint4 v[kLanePieces];
#pragma unroll
  for (int k = 0; k < kLanePieces; ++k) {
    const int c = lane + 32 * k;
    const int64_t s = __shfl_sync(0xffffffffu, src, c / kChunks);
    if (s >= 0) v[k] = __ldcs(pool + s + c % kChunks);
  }
#pragma unroll
  for (int k = 0; k < kLanePieces; ++k) {
    const int c = lane + 32 * k;
    const int64_t d = __shfl_sync(0xffffffffu, dst, c / kChunks);
    if (d >= 0) __stcs(pool + d + c % kChunks, v[k]);
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
    e = cudaFuncSetAttribute(kv_select_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv_select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  EvictParams p = params;
  // one CTA walks a short request faster than a cluster meets (four requests, whole call: of 8200
  // keys 12.0 us against 13.2, of 12000 15.5 against 15.1)
  const int ctas = p.max_seq <= kOneCtaKeys ? 1 : kCluster;
  const int share = share_of(p.max_seq > 0 ? p.max_seq : 1, ctas);
  p.cached = share < kMaxCached ? share : kMaxCached;
  e = ctas == 1 ? launch_dependent(kv_select_kernel<1>, dim3(p.B), kSelectThreads, p.cached * 4, 1, p, stream)
                : launch_dependent(kv_select_kernel<kCluster>, dim3(p.B * kCluster), kSelectThreads, p.cached * 4, kCluster,
                                   p, stream);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  const int rows = 32 * kLanePieces / (p.row_bytes / 16) * kCopyWarps;
  const dim3 grid((p.max_keep + rows - 1) / rows, p.B);
  auto copy = p.row_bytes == 2 * kLatentDim ? kv_copy_kernel<72> : p.row_bytes == kLatentDim ? kv_copy_kernel<36> : kv_copy_kernel<21>;
  return launch_dependent(copy, grid, 32 * kCopyWarps, 0, 1, p, stream);
}

}  // namespace mla
