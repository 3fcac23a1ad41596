// mla_pages_sm103a.cu -- the pages of a cache on the device: requests that fork share them, requests that shrink
// or end give them back, and a pool with holes is compacted.  A count per page says how many table entries
// refer to it (0: free).
//
// All of it is integer bookkeeping of some microseconds, bound by its chain of dependent loads and launches, around
// copies at memory speed:
//  * fork: a cluster of four CTAs per child copies the table row, counts up the shared pages and copies the
//    parent's partial last page.  The checks are made by each CTA for itself; what they read and the call writes
//    (the count of the new page) is written after a cluster barrier.  (4 children of 2000 tokens 2.7 us, 64 of up to
//    32768 3.4 us.)  Each CTA looks through the whole list for a slot or page named twice, so long lists take time with
//    the square of their length: calls of 1000, 4096, 16384 and 65535 children of one page 28, 105, 1080 and 15700 us, of
//    free 38, 63, 213 and 1740.
//  * free: counts go down in one grid, a cluster of four CTAs per slot (a page that nothing refers to any more is
//    marked in its count), and one cluster of eight CTAs then lists the marked pages in ascending order: each warp marks
//    in a range of its own, a scan over warps and CTAs places the ranges, and the warp writes what it marked.  No
//    atomics order anything.  (64 tokens of each of 16 requests, 88 thousand pages: 7.5 us; 256 of 512 requests, 345 thousand
//    pages: 16.0, the list 9.8 of them.  A cluster of 16, opt-in, listed these in 8.2, but took 0.6 to 3 us more on small
//    pools; one of four 15.1.  Both steps in one cluster saved a launch and took 8.9 and 38.8 us: eight SMs' atomics.)
//  * compact: the same scan over the counts pairs the k-th hole below the number of live pages with the k-th
//    live page above it; then a CTA an SM moves the pages by bulk copies through a ring in shared memory, while its other
//    warps rewrite the tables.  (412 MB read and written: 132 us with the scan, 6.2 TB/s; through registers 141; stages
//    of 16 KB 136, of 4 KB 214, half of the ring 142.)
#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

constexpr int kForkThreads = 256;
constexpr int kForkCluster = 4;
constexpr int kDropThreads = 256;
constexpr int kDropCluster = 4;
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanCluster = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 8192;  // of a page, a copy
constexpr int kMoveStages = 24;
constexpr int kMoveLag = 8;  // copies to global memory that may still read their stages
constexpr int kMoveSmem = kMoveStages * kMoveBytes;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The int at the same address of CTA `rank`'s shared memory.
__device__ __forceinline__ int read_cluster(const int* p, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Untiled bulk copy shared -> global (addresses 16-byte aligned, size a multiple of 16), a group of its own; its stage may
// be written again once all but the kPending newest groups have read theirs.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ----------------------------------------------------------------------------------------- fork
__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(const ForkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.y, t = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const int parent = __ldg(p.parents + i), child = __ldg(p.children + i), fresh = __ldg(p.new_pages + i);
  // another child of the same slot or new page goes first; a child that is some child's parent would be read
  // while it is written
  bool slot_taken = false, page_taken = false;
  for (int j = t; j < p.n; j += kForkThreads) {
    slot_taken |= __ldg(p.parents + j) == child || (j < i && __ldg(p.children + j) == child);
    page_taken |= j < i && __ldg(p.new_pages + j) == fresh;
  }
  slot_taken = __syncthreads_or(slot_taken);
  page_taken = __syncthreads_or(page_taken);
  bool ok = parent >= 0 && parent < p.slots && child >= 0 && child < p.slots && !slot_taken;
  int L = 0;
  if (ok) {
    L = p.seq_lens[parent];
    ok = L >= 0 && static_cast<int64_t>(L) <= static_cast<int64_t>(p.max_pages) * p.page_size;
  }
  const int full = L / p.page_size, rest = L % p.page_size;
  const int32_t* from = p.page_table + static_cast<int64_t>(ok ? parent : 0) * p.max_pages;
  int32_t* to = p.page_table + static_cast<int64_t>(ok ? child : 0) * p.max_pages;
  int last = -1;  // the parent's partial page
  if (ok && rest > 0) {
    last = from[full];
    ok = fresh >= 0 && fresh < p.num_pages && !page_taken && p.refs[fresh] == 0 && last >= 0 && last < p.num_pages;
  }
  cluster_sync();  // (every CTA of the child has read the new page's count)
  if (!ok) {  // (the same in the whole cluster)
    if (rank == 0 && t == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const int all = kForkCluster * kForkThreads;
  bool bad = false;
  for (int64_t j = rank * kForkThreads + t; j < full; j += all) {
    const int page = from[j];
    to[j] = page;
    if (page >= 0 && page < p.num_pages)
      atomicAdd(p.refs + page, 1);
    else
      bad = true;
  }
  if (bad) atomicOr(p.status, kStatusDeviceArg);
  if (rank == 0 && t == 0) {
    p.seq_lens[child] = L;
    if (rest > 0) {
      to[full] = fresh;
      p.refs[fresh] = 1;
      if (p.page_scales) p.page_scales[fresh] = p.page_scales[last];
    }
  }
  if (rest > 0) {
    const int64_t page_bytes = static_cast<int64_t>(p.page_size) * p.row_bytes;
    const uint4* src = reinterpret_cast<const uint4*>(p.kv_pages + last * page_bytes);
    uint4* dst = reinterpret_cast<uint4*>(p.kv_pages + fresh * page_bytes);
    const int pieces = rest * (p.row_bytes / 16);
    constexpr int kAtOnce = 4;
    for (int k0 = rank * kForkThreads + t; k0 < pieces; k0 += kAtOnce * all) {
      uint4 v[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (k0 + u * all < pieces) v[u] = src[k0 + u * all];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (k0 + u * all < pieces) dst[k0 + u * all] = v[u];
    }
  }
}

// ----------------------------------------------------------------------------------------- free
// Counts of pages that came free go down by kFreed more, so that the scan tells them from those that were free and
// still were dropped: both are below 0 until it sets them to 0.
constexpr int kFreed = 1 << 30;

__global__ void __launch_bounds__(kDropThreads) page_drop_kernel(const FreeParams p) {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  const int i = blockIdx.y, t = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const int slot = __ldg(p.list + i), keep = __ldg(p.keep_lens + i);
  bool again = false;
  for (int j = t; j < i; j += kDropThreads) again |= __ldg(p.list + j) == slot;
  again = __syncthreads_or(again);
  const bool known = !again && slot >= 0 && slot < p.slots;
  const int L = known ? p.seq_lens[slot] : 0;
  cluster_sync();  // (every CTA of the slot has read its length)
  if (!known || keep < 0 || keep > L || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_pages) * p.page_size) {
    if (rank == 0 && t == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  if (rank == 0 && t == 0) p.seq_lens[slot] = keep;
  const int32_t* row = p.page_table + static_cast<int64_t>(slot) * p.max_pages;
  const int last = (L - 1) / p.page_size;  // (L = 0 has keep = 0: first 0, last 0, and nothing below)
  const int first = keep > 0 ? (keep - 1) / p.page_size + 1 : 0;
  bool bad = false;
  for (int64_t j = static_cast<int64_t>(first) + rank * kDropThreads + t; L > 0 && j <= last; j += kDropCluster * kDropThreads) {
    const int page = row[j];
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      continue;
    }
    const int before = atomicSub(p.refs + page, 1);
    if (before == 1) atomicSub(p.refs + page, kFreed);
    bad |= before < 1;
  }
  if (bad) atomicOr(p.status, kStatusDeviceArg);
}

// Exclusive prefix over the cluster's warps of each warp's count, and the total.  `mine` may differ by warp, not by lane.
struct Scan {
  int warp[kScanWarps];
  int total;
};

__device__ __forceinline__ int cluster_prefix(Scan& s, int mine, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s.warp[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int v = s.warp[lane];
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    s.warp[lane] = sum - v;
    if (lane == 31) s.total = sum;
  }
  cluster_sync();
  int before = s.warp[warp];
  total = 0;
  const uint32_t rank = cluster_rank();
  for (uint32_t r = 0; r < kScanCluster; ++r) {
    const int n = read_cluster(&s.total, r);
    if (r < rank) before += n;
    total += n;
  }
  return before;
}

// Each warp's range of pages, a multiple of 32: [from, to).
__device__ __forceinline__ void scan_range(int num_pages, int& from, int& to) {
  const int warps = kScanCluster * kScanWarps;
  const int per = ((num_pages + warps - 1) / warps + 31) / 32 * 32;
  const int w = cluster_rank() * kScanWarps + (threadIdx.x >> 5);
  from = static_cast<int>(min(static_cast<int64_t>(num_pages), static_cast<int64_t>(w) * per));
  to = static_cast<int>(min(static_cast<int64_t>(num_pages), static_cast<int64_t>(w + 1) * per));
}

// Which of a warp's pages a predicate marks, 32 to a word.  The first kept words of a warp stay in shared memory; of
// larger pools the rest is read again.  (Reading everything again, 32 counts at a time, took 10 of 22 us for a third of a
// million pages.)
constexpr int kKept = 256;  // words: pools of 2 million pages
constexpr int kInFlight = 16;

struct Marks {
  uint32_t word[kScanWarps][kKept];
};

// Words of the pages [from, to) for which is(page, count) holds; f(index, word) of each.
template <typename Is, typename F>
__device__ __forceinline__ void each_word(const int32_t* refs, int from, int to, Is is, F f) {
  const int lane = threadIdx.x & 31;
  int x = from;
  for (; x + 32 * kInFlight <= to; x += 32 * kInFlight) {
    const int32_t* at = refs + x + lane;
    int v[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) v[k] = at[32 * k];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) f((x - from) / 32 + k, __ballot_sync(0xffffffffu, is(x + 32 * k + lane, v[k])));
  }
  for (; x < to; x += 32 * 4) {
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = x + 32 * k + lane < to ? refs[x + 32 * k + lane] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (x + 32 * k < to) f((x - from) / 32 + k, __ballot_sync(0xffffffffu, is(x + 32 * k + lane, v[k])));
  }
}

// How many there are; the words that fit are kept.
template <typename Is>
__device__ __forceinline__ int mark(Marks& marks, const int32_t* refs, int from, int to, Is is) {
  const int lane = threadIdx.x & 31;
  uint32_t* words = marks.word[threadIdx.x >> 5];
  int n = 0;
  const int kept = min(to, from + 32 * kKept);
  each_word(refs, from, kept, is, [&](int i, uint32_t m) {
    if (lane == 0) words[i] = m;
  });
  __syncwarp();
  for (int i = lane; from + 32 * i < kept; i += 32) n += __popc(words[i]);
  n = __reduce_add_sync(0xffffffffu, n);
  each_word(refs, kept, to, is, [&](int, uint32_t m) { n += __popc(m); });
  return n;
}

template <typename Is, typename F>
__device__ __forceinline__ void each_marked(const Marks& marks, const int32_t* refs, int from, int to, Is is, F f) {
  for (int i = 0; i < kKept && from + 32 * i < to; ++i) f(from + 32 * i, marks.word[threadIdx.x >> 5][i]);
  const int rest = from + 32 * kKept;
  if (rest < to) each_word(refs, rest, to, is, [&](int i, uint32_t m) { f(rest + 32 * i, m); });
}

__global__ void __launch_bounds__(kScanThreads) page_list_kernel(const FreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ Scan scan;
  __shared__ Marks marks;
  const int lane = threadIdx.x & 31;
  int from, to, total;
  scan_range(p.num_pages, from, to);
  // a count below 0 becomes 0 once it is not read again
  const auto freed = [&](int page, int v) {
    if (v < 0 && page - from < 32 * kKept) p.refs[page] = 0;
    return v <= -kFreed;
  };
  const auto freed_rest = [&](int page, int v) {
    if (v < 0) p.refs[page] = 0;
    return v <= -kFreed;
  };
  const int mine = mark(marks, p.refs, from, to, freed);
  int at = cluster_prefix(scan, mine, total);
  each_marked(marks, p.refs, from, to, freed_rest, [&](int x, uint32_t m) {
    if (m >> lane & 1) p.freed[at + __popc(m & ((1u << lane) - 1))] = x + lane;
    at += __popc(m);
  });
  if (cluster_rank() == 0 && threadIdx.x == 0) *p.num_freed = total;
  cluster_sync();  // (no CTA ends while another reads its total)
}

// ----------------------------------------------------------------------------------------- compact
__global__ void __launch_bounds__(kScanThreads) page_pair_kernel(const CompactParams p) {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Scan scan;
  __shared__ Marks marks;
  __shared__ int holes_here;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) holes_here = 0;
  int from, to, live;
  scan_range(p.num_pages, from, to);
  // live pages before each warp's range, and in all
  const auto used = [](int, int v) { return v > 0; };
  int at = cluster_prefix(scan, mark(marks, p.refs, from, to, used), live);
  // hole h < live is number h - (live pages before h); live page x >= live is number live - 1 - (live pages before x)
  // from the end
  int holes = 0;
  each_marked(marks, p.refs, from, to, used, [&](int x, uint32_t m) {
    const int page = x + lane, before = at + __popc(m & ((1u << lane) - 1));
    const bool in = page < to, here = m >> lane & 1, hole = in && !here && page < live;
    if (hole) p.holes[page - before] = page;
    if (in && page >= live) {
      if (here) p.movers[live - 1 - before] = page;
      p.remap[page] = -1;
    }
    holes += __popc(__ballot_sync(0xffffffffu, hole));
    at += __popc(m);
  });
  if (lane == 0) atomicAdd(&holes_here, holes);
  cluster_sync();
  int moves = 0;
  for (uint32_t r = 0; r < kScanCluster; ++r) moves += read_cluster(&holes_here, r);
  for (int k = cluster_rank() * kScanThreads + threadIdx.x; k < moves; k += kScanCluster * kScanThreads) {
    const int hole = p.holes[k], page = p.movers[moves - 1 - k];
    p.movers_up[k] = page;
    p.remap[page] = hole;
    p.refs[hole] = p.refs[page];
    p.refs[page] = 0;
    if (p.page_scales) p.page_scales[hole] = p.page_scales[page];
  }
  if (cluster_rank() == 0 && threadIdx.x == 0) {
    *p.num_live = live;
    p.head[0] = live;
    p.head[1] = moves;
  }
  cluster_sync();  // (no CTA ends while another reads its counts)
}

__global__ void __launch_bounds__(kMoveThreads) page_move_kernel(const CompactParams p) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ uint64_t full[kMoveStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x, lane = t & 31;
  if (t == 0) {
    abort_flag = 0;
    for (int s = 0; s < kMoveStages; ++s) mbar_init(full + s, 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int live = p.head[0], moves = p.head[1];
  if (t < 32) {
    // pages: a ring of slices through shared memory.  The lanes work out 32 slices at a time, ahead of their use (one
    // thread that did it slice by slice waited for their indexes: 196 us where plain copies took 142), and lane s knows
    // where the slice of stage s goes.
    const int64_t page_bytes = static_cast<int64_t>(p.page_size) * p.row_bytes;
    const int slices = static_cast<int>((page_bytes + kMoveBytes - 1) / kMoveBytes);
    const int64_t all = static_cast<int64_t>(moves) * slices;
    const int64_t mine = all > blockIdx.x ? (all - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    struct Slice {
      int64_t from, to;
      uint32_t bytes;
    };
    const auto slice = [&](int64_t i) {
      if (i >= mine) return Slice{0, 0, 0};
      const int64_t u = blockIdx.x + i * gridDim.x;
      const int k = static_cast<int>(u / slices), s = static_cast<int>(u % slices);
      const int64_t at = static_cast<int64_t>(s) * kMoveBytes;
      return Slice{p.movers_up[k] * page_bytes + at, p.holes[k] * page_bytes + at, static_cast<uint32_t>(min(static_cast<int64_t>(kMoveBytes), page_bytes - at))};
    };
    const uint64_t policy = policy_evict_first();
    Slice now = slice(lane), later = slice(32 + lane), held = {0, 0, 0};
    const auto load = [&](int64_t i) {  // (i one by one)
      const int r = static_cast<int>(i & 31), s = static_cast<int>(i % kMoveStages);
      if (r == 0 && i > 0) {
        now = later;
        later = slice(i + 32 + lane);
      }
      const Slice x = {__shfl_sync(0xffffffffu, now.from, r), __shfl_sync(0xffffffffu, now.to, r), __shfl_sync(0xffffffffu, now.bytes, r)};
      if (lane == s) {
        held = x;
        mbar_arrive_expect_tx(full + s, x.bytes);
        bulk_load(stages + s * kMoveBytes, p.kv_pages + x.from, x.bytes, full + s, policy);
      }
    };
    for (int64_t i = 0; i < min(mine, static_cast<int64_t>(kMoveStages)); ++i) load(i);
    for (int64_t i = 0; i < mine; ++i) {
      const int s = static_cast<int>(i % kMoveStages);
      const bool landed = mbar_wait(full + s, (i / kMoveStages) & 1, &abort_flag);
      if (!__all_sync(0xffffffffu, landed)) {
        if (lane == 0) atomicOr(p.status, kStatusTimeout);
        for (int64_t j = i + 1; j < min(mine, max(i - kMoveLag, int64_t(0)) + kMoveStages); ++j) {  // what is in flight lands first
          abort_flag = 0;
          if (!mbar_wait(full + j % kMoveStages, (j / kMoveStages) & 1, &abort_flag)) break;
        }
        break;
      }
      const int64_t to = __shfl_sync(0xffffffffu, held.to, s);
      const uint32_t bytes = __shfl_sync(0xffffffffu, held.bytes, s);
      if (lane == 0) bulk_store(p.kv_pages + to, stages + s * kMoveBytes, bytes);
      // the stage of the copy before the last kMoveLag takes a slice again
      const int64_t next = i - kMoveLag + kMoveStages;
      if (i >= kMoveLag && next < mine) {
        if (lane == 0) bulk_wait_read<kMoveLag>();
        __syncwarp();
        load(next);
      }
    }
    if (lane == 0) bulk_wait_all();
  } else {
    // tables: a warp a stretch of 32 x 8 entries
    const int64_t stretches = (p.max_pages + 255) / 256, units = stretches * p.slots;
    bool bad = false;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32 - 1) + (t >> 5) - 1; u < units; u += static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32 - 1)) {
      const int slot = static_cast<int>(u / stretches), j0 = static_cast<int>(u % stretches) * 256;
      const int L = __ldg(p.seq_lens + slot);
      if (L <= 0) continue;
      const int used = static_cast<int>(min(static_cast<int64_t>(p.max_pages), (static_cast<int64_t>(L) + p.page_size - 1) / p.page_size));
      if (lane == 0 && static_cast<int64_t>(L) > static_cast<int64_t>(p.max_pages) * p.page_size) bad = true;
      int32_t* row = p.page_table + static_cast<int64_t>(slot) * p.max_pages;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + 32 * k + lane;
        if (j >= used) continue;
        const int page = row[j];
        if (page < 0 || page >= p.num_pages) {
          bad = true;
        } else if (page >= live) {
          const int to = p.remap[page];
          if (to >= 0)
            row[j] = to;
          else
            bad = true;  // nothing referred to it
        }
      }
    }
    if (bad) atomicOr(p.status, kStatusDeviceArg);
  }
}

template <typename K, typename P>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int cluster, int smem, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_page_fork(const ForkParams& p, cudaStream_t stream) {
  return launch_dependent(page_fork_kernel, dim3(kForkCluster, p.n), kForkThreads, kForkCluster, 0, p, stream);
}

cudaError_t launch_page_free(const FreeParams& p, cudaStream_t stream) {
  if (p.n > 0) {
    const cudaError_t e = launch_dependent(page_drop_kernel, dim3(kDropCluster, p.n), kDropThreads, kDropCluster, 0, p, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(page_list_kernel, dim3(kScanCluster), kScanThreads, kScanCluster, 0, p, stream);
}

cudaError_t launch_page_compact(const CompactParams& p, int num_sms, cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(page_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  e = launch_dependent(page_pair_kernel, dim3(kScanCluster), kScanThreads, kScanCluster, 0, p, stream);
  if (e != cudaSuccess) return e;
  // a CTA an SM: which slices there are is known on the device alone
  return launch_dependent(page_move_kernel, dim3(num_sms), kMoveThreads, 1, kMoveSmem, p, stream);
}

}  // namespace mla
