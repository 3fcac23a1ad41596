// mla_decode_tree_sm103a.cu -- decode of a tree of drafted tokens over a paged bf16 latent
// cache for requests of more than 48 folded rows, sm_103a.
//
// What it computes (per request b, draft t, head h, folded row m = t*H + h):
//   out[b,t,h,:] = sum_j softmax_j(scale * q[b,t,h,:] . k_j) * k_j[:512]
// over the keys j < L - T and those drafts j = L - T + u whose bit u is set in the row's mask.
// (Fewer rows: decode_partial_narrow_kernel, which reads the cache faster, 214 us against 228 on 16
// requests of 8K-131K keys with 48 rows.  8-bit pools: the kernels of their formats.)
//
// Why a kernel of its own.  An output row takes 512 fp32 accumulators, so an SM's tensor memory
// (512 columns of 128 lanes) holds the output of 64 rows beside their scores.  One CTA with
// 64 rows multiplies at M = 64, half the tensor rate (such a kernel reached 0.37 of peak on wide
// trees, and 262 us where this takes 225 on those requests with 64 rows).  Here two CTAs of a
// cluster multiply as a pair (cta_group::2): M = 128 rows, 64 in each SM, runs at the full rate
// (measured: N = 64 / 128 / 256 in 24.8 / 31.9 / 63.9 cycles), and each SM fetches half of the B
// operand.  Bound by shared memory and the products on wide trees (0.71 of the bf16 peak in a burst of
// 279 us on 8 requests of 20K-65K keys with 32 x 16 rows; 0.65 sustained, where the board's power is
// the limit), by reading the cache with one pair a tile (0.80-0.84 of the copy rate at 64 rows).
//  * CTA r of a pair holds rows 64r .. 64r+63 of the group: their Q (shared memory), their S (two
//    buffers) and O (tensor memory; row i in lanes i and i + 64, which hold half of the
//    columns each), their softmax and their output.
//  * BMM1, S = Q . K^T (N = 64 keys, K = 576): CTA r holds keys 32r .. 32r+31 of the tile.
//  * BMM2, O += P . V (N = 256 twice, K = 64 keys): CTA r holds all 64 keys' columns 256r ..
//    256r+255.  (The operand of one MMA lies at one address in both CTAs, so K and V are two
//    copies: 68 KB a CTA and tile, the V one from L2.)  K and V have rings of their own.
//  * Warps: 0-7 softmax and epilogue, 8 and 9 load the K and the V ring, 10 and 11 issue BMM1 and
//    BMM2 (CTA 0's, for the pair).  Loads of both CTAs count on barriers of CTA 0; commits arrive in both.
//  * Softmax: TMEM lane l holds row l % 64, keys 0-31 (l < 64) or 32-63 of the tile; warps w and
//    w + 4 share a lane quadrant and take 16 of those keys each.  A row's four threads swap their
//    maxima through shared memory (one barrier a tile).  Lazy rescale as in the other kernels.
// Every wait is bounded; on expiry the CTA records a timeout, drains and returns.
#include "mla_internal.h"
#include "sm103a_ptx.cuh"
#include "tree_mask.cuh"

namespace mla {

int tree_pair_groups(int R) { return (R + 127) / 128; }

namespace {

constexpr int kDimBlocks = kLatentDim / 64;         // 9 blocks of 64 columns (128 bytes)
constexpr int kHalfKeys = kTileKeys / 2;            // keys of a tile that a CTA holds for BMM1
constexpr int kKBlock = kHalfKeys * 128;            // 4 KB
constexpr int kKBytes = kDimBlocks * kKBlock;       // 36 KB
constexpr int kVBlock = kTileKeys * 128;            // 8 KB
constexpr int kVBlocks = kValueDim / 64 / 2;        // 4: a CTA's half of the value columns
constexpr int kVBytes = kVBlocks * kVBlock;         // 32 KB
constexpr int kPBytes = 64 * 128;                   // 64 rows x 64 keys
constexpr int kKStages = 2;
constexpr int kVStages = 2;
constexpr int kRows = 64;                           // rows a CTA holds
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kLoadKWarp = kSoftmaxWarps, kLoadVWarp = kLoadKWarp + 1, kBmm1Warp = kLoadKWarp + 2, kBmm2Warp = kLoadKWarp + 3;
constexpr int kAhead = 2;  // tiles that the L2 prefetch runs ahead of the loads
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kArrivals = 2 * kSoftmaxWarps;        // softmax warps of the pair

struct PairCtrl {
  // counted in CTA 0 (loads and softmax warps of both CTAs)
  uint64_t q_full;
  uint64_t k_full[kKStages];
  uint64_t v_full[kVStages];
  uint64_t s_free[2];
  uint64_t p_full;
  uint64_t drain1, drain2;
  // in both CTAs (commits arrive in both)
  uint64_t v_here[2];  // V of the first or second tile that holds drafts has landed in both (BMM1's
                       // warp arrives, up to two tiles ahead of the softmax: one barrier each, used once)
  uint64_t k_empty[kKStages];
  uint64_t v_empty[kVStages];
  uint64_t s_full[2];
  uint64_t o_done;
  unsigned long long lost;  // drafts that some row sees with a score of -infinity
  uint32_t tmem_base;
  int abort_flag;
  float row_max[2][4][64];  // by tile parity: the four partial maxima of each row
  float row_sum[4][64];
};
constexpr int kCtrlBytes = 4096;
static_assert(sizeof(PairCtrl) <= kCtrlBytes, "control block");

// Shared memory map: Q | K ring | V ring | P | control
constexpr int kQBlock = kRows * 128;
constexpr int kQBytes = kDimBlocks * kQBlock;
constexpr int kOffK = kQBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;
constexpr int kOffP = kOffV + kVStages * kVBytes;
constexpr int kOffCtrl = kOffP + kPBytes;
constexpr int kSmemBytes = kOffCtrl + kCtrlBytes + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per block");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;  // O: columns 0-255; S: 32 columns per buffer
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// ----------------------------------------------------------------------------------------
// Pairs: cluster addresses, barriers across the two CTAs, cta_group::2 forms
// ----------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What one CTA hands the other crosses in shared memory (P, rewritten value rows) and tensor
// memory (scores read, outputs rescaled; tcgen05 fences on either side).  So an arrival at the other
// CTA releases, and a wait acquires, at cluster scope.  The release is a fence over the thread's
// own CTA's shared memory alone: one of all memory took 607-614 us where this takes 297-306 (8 requests
// of 20K-65K keys with 32 x 16 rows; without scopes 297-303).
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
      : "memory");
}
// The same, passing on what this thread has itself acquired (copies that landed in either CTA).
__device__ __forceinline__ void arrive_pair_all(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool try_wait_pair(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait for barriers that the other CTA, a copy or a commit of the pair arrives on.
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (try_wait_pair(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (true) {
    if (try_wait_pair(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      return false;
    }
  }
}
// TMA loads into this CTA's shared memory that count on a barrier of either CTA.
__device__ __forceinline__ void load_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                             uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this address in the CTAs of `mask` once this thread's MMAs are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
decode_tree_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const DecodeParams p, const int group_rows) {
  extern __shared__ uint8_t smem_raw[];
  // (the same offset in both CTAs: their dynamic shared memory starts at the same address)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PairCtrl* ctrl = reinterpret_cast<PairCtrl*>(smem + kOffCtrl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int group = blockIdx.x >> 1, groups = gridDim.x >> 1;
  const int b = p.split_major ? blockIdx.y : blockIdx.z;
  const int split = p.split_major ? blockIdx.z : blockIdx.y;

  if (threadIdx.x == 0) {
    mbar_init(&ctrl->q_full, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&ctrl->k_full[s], 1);
      mbar_init(&ctrl->k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&ctrl->v_full[s], 1);
      mbar_init(&ctrl->v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctrl->s_full[i], 1);
      mbar_init(&ctrl->s_free[i], kArrivals);
      mbar_init(&ctrl->v_here[i], 1);
    }
    mbar_init(&ctrl->p_full, kArrivals);
    mbar_init(&ctrl->o_done, 1);
    mbar_init(&ctrl->drain1, 1);
    mbar_init(&ctrl->drain2, 1);
    ctrl->abort_flag = 0;
    ctrl->lost = 0;
    fence_mbarrier_init();
  }
  if (warp == kBmm1Warp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctrl->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == kLoadKWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers exist
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto release_tmem = [&]() {
    if (warp == kBmm1Warp)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  };
  const int L = p.seq_lens[b];
  const bool bad_len = L < p.T || L > p.max_seq || L > static_cast<int64_t>(p.max_pages) * p.page_size;
  if (bad_len && threadIdx.x == 0 && split == 0 && blockIdx.x == 0) atomicOr(p.status, kStatusDeviceArg);
  const int kv_start = split * p.chunk;
  if (bad_len || kv_start >= L) {  // (uniform over the pair)
    release_tmem();
    return;
  }
  const int kv_end = min(L, kv_start + p.chunk);
  const int ntiles = (kv_end - kv_start + kTileKeys - 1) / kTileKeys;
  const int nsplit_b = (L + p.chunk - 1) / p.chunk;
  const int p0 = L - p.T;  // first draft
  // tiles from here on hold drafts (or the end), two at most (64 drafts): their V is touched by the softmax
  const int tail_tile = max(0, p0 - kv_start) / kTileKeys;
  const int half_rows = group_rows / 2;
  const int row0 = group * group_rows + static_cast<int>(rank) * half_rows;
  const int nrows = max(0, min(half_rows, p.R - row0));
  volatile int* abort_flag = &ctrl->abort_flag;
  // Shared memory of a tile: from a page of at least 64 keys [column block][key], else [8 keys][block]
  const bool whole = p.page_size >= kTileKeys;
  const uint32_t k_block = whole ? kKBlock : 1024, k_eight = whole ? 1024 : kDimBlocks * 1024;
  const uint32_t v_block = whole ? kVBlock : 1024, v_eight = whole ? 1024 : kVBlocks * 1024;

  if (warp == kLoadKWarp || warp == kLoadVWarp) {
    // ------------------------------------------------------------------ TMA producers, one per
    // ring (as two halves of one warp they held each other up: 304 against 268 us on 8 requests of
    // 20K-65K keys with 32 x 16 rows).  Pages of 64 keys or more: one box per operand and
    // tile; smaller pages: one box per 8 keys (a lane each).  A box past the request's end, and
    // a page id outside the pool (reported), lie before the first row, which TMA fills with zeros.
    const bool is_k = warp == kLoadKWarp;
    const int page_log2 = __ffs(p.page_size) - 1;  // (a power of two)
    const int keys = is_k ? kHalfKeys : kTileKeys;
    const int nbox = whole ? 1 : keys / 8;
    const int first_key = (is_k ? static_cast<int>(rank) * kHalfKeys : 0) + 8 * lane;
    const int first_blk = is_k ? 0 : static_cast<int>(rank) * kVBlocks;
    const int stages = is_k ? kKStages : kVStages;
    uint64_t* const full = is_k ? ctrl->k_full : ctrl->v_full;
    uint64_t* const empty = is_k ? ctrl->k_empty : ctrl->v_empty;
    const CUtensorMap* const map = is_k ? &tm_k : &tm_v;
    const uint32_t stage_bytes = is_k ? kKBytes : kVBytes;
    const uint32_t ring = smem_u32(smem + (is_k ? kOffK : kOffV)) + lane * (stage_bytes / (keys / 8));
    const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    const unsigned n_pages = static_cast<unsigned>(min(p.num_pages, static_cast<int64_t>(0x7fffffff)));
    const uint64_t pol = policy_evict_normal();  // (every byte of a value column is read by both CTAs)
    bool bad_pid = false;
    auto has_keys = [&](int j) { return lane < nbox && j < ntiles && kv_start + j * kTileKeys + first_key < L; };
    auto page_of = [&](int j) -> int {  // page of this lane's box of tile j (looked at tiles later)
      return has_keys(j) ? __ldg(pt + ((kv_start + j * kTileKeys + first_key) >> page_log2)) : 0;
    };
    auto row_of = [&](int j, int pid) -> int {  // and its pool row
      if (!has_keys(j)) return -kTileKeys;
      if (static_cast<unsigned>(pid) >= n_pages) {
        bad_pid = true;
        return -kTileKeys;
      }
      return (pid << page_log2) + ((kv_start + j * kTileKeys + first_key) & (p.page_size - 1));
    };
    if (is_k && lane == 0) {
      const uint32_t bar = map_rank(smem_u32(&ctrl->q_full), 0);
      if (rank == 0) mbar_arrive_expect_tx(&ctrl->q_full, 2 * kQBytes);
      load_pair_3d(smem_u32(smem), &tm_q, bar, 0, b * p.R + row0, 0, policy_evict_last());
    }
    int page[kAhead + 1];  // of the next tiles
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) page[i] = page_of(i);
    int slot = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      const int next = page_of(j + kAhead + 1);
      const int row = row_of(j, page[0]);
      if (j >= stages) {
        bool w = true;
        if (lane == 0) w = wait_pair(&empty[slot], phase ^ 1, abort_flag);
        ok = __shfl_sync(0xffffffffu, w, 0);
        if (!ok) break;
      }
      if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * stage_bytes);
      __syncwarp();
      if (lane < nbox)
        load_pair_3d(ring + slot * stage_bytes, map, map_rank(smem_u32(&full[slot]), 0), 0, row, first_blk, pol);
      // Each key goes to two copies, and several pairs may read a tile at about the same time: one
      // of them asks L2 for it ahead.  (Two tiles, against none: 304 -> 268 us with four pairs a
      // tile, 287 -> 234 with one on 16 requests of 8K-131K keys; six tiles ahead 273 and 264.)
      const int ahead = is_k && j % groups == group ? row_of(j + kAhead, page[kAhead]) : -1;
      if (ahead >= 0)
        asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                     "r"(0), "r"(ahead), "r"(0)
                     : "memory");
      ++issued;
      if (++slot == stages) {
        slot = 0;
        phase ^= 1;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) page[i] = page[i + 1];
      page[kAhead] = next;
    }
    if (__any_sync(0xffffffffu, bad_pid) && lane == 0) atomicOr(p.status, kStatusDeviceArg);
    if (!ok && lane == 0 && rank == 0) {
      // copies of the pair still in flight land before the CTAs leave
      if (is_k) drain_wait(&ctrl->q_full, 0);
      for (int u = max(0, issued - stages); u < issued; ++u) drain_wait(&full[u % stages], (u / stages) & 1);
    }
    __syncwarp();
  } else if (warp == kBmm1Warp) {
    // ------------------------------------------------------------------ BMM1 (CTA 0, for the pair)
    if (rank == 0) {
      const uint32_t idesc = make_idesc_bf16(128, kTileKeys, false, false);
      const uint64_t q_desc = make_smem_desc(smem_u32(smem), 16, 1024);
      bool ok = __all_sync(0xffffffffu, wait_pair(&ctrl->q_full, 0, abort_flag));
      int slot = 0, phase = 0;
      for (int j = 0; ok && j < ntiles; ++j) {
        const int sb = j & 1;
        bool w = wait_pair(&ctrl->k_full[slot], phase, abort_flag);
        if (w && j >= tail_tile) w = wait_pair(&ctrl->v_full[j % kVStages], (j / kVStages) & 1, abort_flag);
        if (w && j >= 2) w = wait_pair(&ctrl->s_free[sb], ((j - 2) >> 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, w);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k_desc = make_smem_desc(smem_u32(smem + kOffK + slot * kKBytes), 16, k_eight);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < kDimBlocks; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_pair(tmem + kTmemS + sb * 32, q_desc + static_cast<uint64_t>((c * kQBlock + k * 32) >> 4),
                        k_desc + static_cast<uint64_t>((c * k_block + k * 32) >> 4), idesc, (c | k) != 0);
          }
          commit_pair(&ctrl->s_full[sb], 3);
          commit_pair(&ctrl->k_empty[slot], 3);
        }
        __syncwarp();
        if (j >= tail_tile) {
          if (lane < 2) arrive_pair_all(map_rank(smem_u32(&ctrl->v_here[j - tail_tile]), lane));
          __syncwarp();
        }
        if (++slot == kKStages) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (elect_one()) {
        commit_pair(&ctrl->drain1, 1);
        drain_wait(&ctrl->drain1, 0);
      }
    }
    __syncwarp();
  } else if (warp == kBmm2Warp) {
    // ------------------------------------------------------------------ BMM2 (CTA 0, for the pair)
    if (rank == 0) {
      const uint32_t idesc = make_idesc_bf16(128, 256, false, true);
      const uint64_t p_desc = make_smem_desc(smem_u32(smem + kOffP), 16, 1024);
      bool ok = true;
      for (int j = 0; ok && j < ntiles; ++j) {
        const int s = j % kVStages;
        bool w = wait_pair(&ctrl->v_full[s], (j / kVStages) & 1, abort_flag);
        if (w) w = wait_pair(&ctrl->p_full, j & 1, abort_flag);
        ok = __all_sync(0xffffffffu, w);
        if (!ok) break;
        tc_fence_after();
        // V: 16 keys (two 8-key groups, SBO apart) x 128 of this CTA's value columns (two
        // 64-column blocks, LBO apart), MN-major
        const uint64_t v_desc = make_smem_desc(smem_u32(smem + kOffV + s * kVBytes), v_block, v_eight);
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_pair(tmem + q * 128, p_desc + static_cast<uint64_t>((kk * 32) >> 4),
                        v_desc + static_cast<uint64_t>((q * 2 * v_block + kk * 2 * v_eight) >> 4), idesc,
                        (j > 0 || kk > 0) ? 1u : 0u);
          }
          commit_pair(&ctrl->o_done, 3);
          commit_pair(&ctrl->v_empty[s], 3);
        }
        __syncwarp();
      }
      if (elect_one()) {
        commit_pair(&ctrl->drain2, 1);
        drain_wait(&ctrl->drain2, 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + epilogue (warps 0-7)
    const int quad = warp & 3, hf = warp >> 2;
    const int r = (quad & 1) * 32 + lane;  // row of this CTA
    const int hi = quad >> 1;              // keys 32 hi .. of the tile; output columns 256 hi ..
    const int kb = 32 * hi + 16 * hf;      // this thread's first key of a tile
    const int mine = 2 * hi + hf;          // its place among the row's four threads
    const bool row_active = r < nrows;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    uint64_t drafts = 0;  // the drafts this row sees
    if (row_active) drafts = p.tree_mask[static_cast<int64_t>(b) * p.T + (row0 + r) / p.H] & draft_bits(p.T);
    const uint32_t s_free0 = map_rank(smem_u32(&ctrl->s_free[0]), 0);
    const uint32_t p_full0 = map_rank(smem_u32(&ctrl->p_full), 0);
    const uint32_t p_row = smem_u32(smem + kOffP) + r * 128;
    float m_used = -INFINITY, l_sum = 0.f;
    bool failed = false, fail = false;
    for (int j = 0; j < ntiles; ++j) {
      const int sb = j & 1;
      const int k0 = kv_start + j * kTileKeys;
      uint32_t s[16];
      if (!fail) fail = __any_sync(0xffffffffu, !wait_pair(&ctrl->s_full[sb], (j >> 1) & 1, abort_flag));
      if (!fail) {
        tc_fence_after();
        tmem_ld16(tmem + lane_base + kTmemS + sb * 32 + 16 * hf, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(s_free0 + sb * 8);
        uint32_t seen = row_active ? 0xffffu : 0u;
        if (k0 + kTileKeys > p0) {
          seen = row_active ? static_cast<uint32_t>(tree_tile_bits(drafts, p0, k0) >> kb) & 0xffffu : 0u;
          uint32_t minus = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) minus |= (s[i] == 0xff800000u ? 1u : 0u) << i;
          if (minus & seen) atomicOr(&ctrl->lost, draft_word(minus & seen, k0 + kb, p0));
        }
        if (seen != 0xffffu) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!((seen >> i) & 1u)) s[i] = 0xff800000u;  // -inf: weight 0
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, __uint_as_float(s[i]));
        ctrl->row_max[sb][mine][r] = mx;
      }
      // every maximum of this tile is written (and every one of the tile before last read)
      if (bar_or(1, kSoftmaxThreads, fail || *abort_flag != 0)) {
        failed = true;
        break;
      }
      const float mx = fmaxf(fmaxf(ctrl->row_max[sb][0][r], ctrl->row_max[sb][1][r]),
                             fmaxf(ctrl->row_max[sb][2][r], ctrl->row_max[sb][3][r]));
      const float mt = mx * p.scale_log2;
      float alpha = 1.f;
      bool rescale = false;
      if (m_used == -INFINITY) {
        m_used = mt;  // nothing accumulated yet
      } else if (mt > m_used + kRescaleThreshold) {
        alpha = ex2_approx(m_used - mt);
        rescale = true;
        l_sum *= alpha;
        m_used = mt;
      }
      const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;
      uint32_t packed[8];
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float e0 = ex2_approx(fmaf(__uint_as_float(s[i]), p.scale_log2, neg_m));
        const float e1 = ex2_approx(fmaf(__uint_as_float(s[i + 1]), p.scale_log2, neg_m));
        l0 += e0;
        l1 += e1;
        packed[i >> 1] = pack_bf16x2(e0, e1);
      }
      l_sum += l0 + l1;
      if (j >= 1) {  // BMM2 of the tile before has read P and finished with O
        fail = __any_sync(0xffffffffu, !wait_pair(&ctrl->o_done, (j - 1) & 1, abort_flag));
        if (fail) continue;  // (reported at the next tile's barrier, or after the loop)
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        st_shared_v4(p_row + ((((kb >> 3) + c) ^ (r & 7)) << 4), packed[4 * c], packed[4 * c + 1], packed[4 * c + 2],
                     packed[4 * c + 3]);
      if (__any_sync(0xffffffffu, rescale) && j >= 1) {
        // O *= alpha for this lane's row: columns 128 hf .. 128 hf + 127 of the lane's 256
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          const uint32_t addr = tmem + lane_base + 128 * hf + 32 * c;
          tmem_ld32(addr, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st32(addr, v);
        }
        tmem_st_wait();
      }
      if (k0 + kTileKeys > p0) {
        // V's copies count on barriers of CTA 0, whose BMM1 warp passes their arrival on to both CTAs.
        // Rows past the request's end become zero, drafts' infinities and NaNs too: rows that do not
        // see them give them weight 0.
        fail = __any_sync(0xffffffffu, !wait_pair(&ctrl->v_here[j - tail_tile], 0, abort_flag));
        if (fail) continue;
        const uint32_t stage = smem_u32(smem + kOffV + (j % kVStages) * kVBytes);
        const int first = max(p0 - k0, 0), valid = min(L - k0, kTileKeys);
        for (int idx = threadIdx.x; idx < (kTileKeys - first) * 8 * kVBlocks; idx += kSoftmaxThreads) {
          const int row = first + idx / (8 * kVBlocks), rem = idx % (8 * kVBlocks);
          const uint32_t at = stage + (rem >> 3) * v_block + (row >> 3) * v_eight + (row & 7) * 128 + (rem & 7) * 16;
          if (row < valid)
            make_finite<false>(at);
          else
            st_shared_v4(at, 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair(p_full0);
    }
    if (!failed && !fail) fail = !wait_pair(&ctrl->o_done, (ntiles - 1) & 1, abort_flag);
    if (!failed) ctrl->row_sum[mine][r] = l_sum;
    if (!failed && !bar_or(1, kSoftmaxThreads, fail || *abort_flag != 0)) {
      tc_fence_after();
      const float l = (ctrl->row_sum[0][r] + ctrl->row_sum[1][r]) + (ctrl->row_sum[2][r] + ctrl->row_sum[3][r]);
      const bool some = l != 0.f;  // (0: the row sees nothing here; a NaN is passed on)
      const float inv = some ? 1.f / l : 0.f;
      const bool final_out = nsplit_b == 1;
      const int64_t grow = static_cast<int64_t>(b) * p.R + row0 + r;
      const int64_t prow = (static_cast<int64_t>(b) * p.max_splits + split) * p.R + row0 + r;
      if (row_active && mine == 0) {
        const float lse = some ? (m_used + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
        if (final_out)
          p.lse[grow] = lse;
        else
          p.ws_lse[prow] = lse;
      }
      // The row is staged in the (now free) rings, rows a padded pitch apart so that eight
      // lanes' 16-byte stores fall in all banks, and leaves in whole lines.  (Each thread storing
      // its own row's columns took 10,000 cycles for 64 fp32 rows: 14.7 against 12.1 us for a call
      // of 8 x 16 rows over 1000 keys.)
      const int dim = 256 * hi + 128 * hf;  // this thread's 128 output columns
      const int pitch = kValueDim * (final_out ? 2 : 4) + 16;
      static_assert(kRows * (kValueDim * 4 + 16) <= kKStages * kKBytes + kVStages * kVBytes, "output staging");
      const uint32_t stage = smem_u32(smem + kOffK);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + 128 * hf + 32 * c, v);
        tmem_ld_wait();
        if (!row_active) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv);
        const uint32_t at = stage + r * pitch + (dim + 32 * c) * (final_out ? 2 : 4);
        if (final_out) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]), __uint_as_float(v[8 * i + 2 * k + 1]));
            st_shared_v4(at + 16 * i, o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) st_shared_v4(at + 16 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      named_bar_sync(1, kSoftmaxThreads);
      if (ctrl->lost != 0) {  // (the same in every thread: last changed before the barriers above)
        pass_on_not_finite<kSoftmaxThreads>(ctrl->lost, p.kv_pool, p.num_pages, p.page_size,
                                            p.page_table + static_cast<int64_t>(b) * p.max_pages, p0,
                                            p.tree_mask + static_cast<int64_t>(b) * p.T, row0, nrows, p.H, stage, pitch, !final_out);
        named_bar_sync(1, kSoftmaxThreads);
      }
      const int pieces = final_out ? kValueDim * 2 / 16 : kValueDim * 4 / 16;  // per row
      uint4* const dst = final_out ? reinterpret_cast<uint4*>(p.out + (grow - r) * kValueDim)
                                   : reinterpret_cast<uint4*>(p.ws_of + (prow - r) * kValueDim);
#pragma unroll 4
      for (int i = threadIdx.x; i < nrows * pieces; i += kSoftmaxThreads)
        dst[i] = ld_shared_v4(stage + (i / pieces) * pitch + (i % pieces) * 16);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && ctrl->abort_flag) atomicOr(p.status, kStatusTimeout);
  // every store of this CTA is issued: the combine grid may be scheduled now
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cluster_sync_all();  // neither CTA leaves while the other may still signal it or use its tensor memory
  tc_fence_after();
  release_tmem();
}

}  // namespace

cudaError_t launch_decode_tree_pair(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(decode_tree_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const int groups = tree_pair_groups(p.R);
  const int group_rows = 2 * ((p.R + 2 * groups - 1) / (2 * groups));  // even groups, at most 128 rows
  const unsigned gx = static_cast<unsigned>(2 * groups);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.split_major ? dim3(gx, p.B, p.max_splits) : dim3(gx, p.max_splits, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, decode_tree_pair_kernel, tm_q, tm_k, tm_v, p, group_rows);
}

}  // namespace mla
