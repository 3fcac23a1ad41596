// mla_key_mass_sm103a.cu -- the attention weight that each cached key received in a decode
// step, accumulated over steps, sm_103a.
//
// What it computes, per request b and key j < L_b:
//   mass[b, j] = decay * mass[b, j] + sum over the rows (t, h) that see key j of
//                exp(scale * q[b,t,h] . k_j - lse[b,t,h])
// with the visibility of mla_decode (draft t sees keys 0 .. L_b - T + t) or, with tree masks,
// of mla_decode_tree.  A row whose lse is not finite adds nothing.
//
// What has to be read is the keys, once; so it is bound by memory while a request has few rows,
// and by the product with many.
//  * S^T = K . Q^T on the tensor cores (tcgen05, M = 128 keys, N = up to 128 query rows): a
//    key is a TMEM lane, so its weights lie in one thread's columns and their sum needs no
//    exchange between threads; the result is stored without atomics, in a fixed order.
//  * K streams by TMA (128 keys x 64 columns a piece) through a ring that takes what shared
//    memory the resident Q leaves.  An e4m3 pool is multiplied as its raw codes (kind::f8f6f4)
//    with Q split in two e4m3 parts (as mla_decode_e4m3_sm103a.cu), the two parts side by
//    side along N.
//  * The grid is one CTA per SM; every CTA takes an equal run of the batch's 128-key tiles,
//    across requests (keys are independent, so nothing is joined afterwards).  Requests of
//    more than 128 rows run in row groups side by side, whose sums a second kernel adds up.
//  * Two groups of four warps take alternate tiles from two S buffers, so exponentials
//    (R per key) run beside the next tile's product.
//  * int8 pools: the codes arrive by TMA in a ring of their own; six warps write them into the
//    K ring as f16, exactly; Q is converted to f16.  A page's scale multiplies its keys' scores;
//    keys of a page whose scale is out of range (reported) get no weight.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kv8_decode.cuh"
#include "mla_internal.h"
#include "sm103a_ptx.cuh"
#include "tree_mask.cuh"

namespace mla {
namespace {

constexpr int kTile = 128;                        // keys per tile (MMA M, TMEM lanes)
constexpr int kDimBlocks = kLatentDim / 64;       // 9 blocks of 64 columns
constexpr int kMaxRows = 128;                     // query rows a CTA holds (MMA N; e4m3: 2 x)
constexpr int kMaxStages = 12;
constexpr int kGroupWarps = 4;                    // warps that read one S buffer
constexpr int kEpiWarps = 2 * kGroupWarps;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kLoadWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kDecodeWarps = 6;                   // int8: the warps after kMmaWarp
constexpr int threads_for(int kv) { return 32 * (kEpiWarps + 2 + (kv >= kKvInt8 ? kDecodeWarps : 0)); }
constexpr int kRawBytes = kTile * 64;             // int8: one column block of a tile as codes
constexpr uint32_t kTmemCols = 512;               // two S buffers of up to 256 columns

// Column blocks per ring stage: a 16-bit block is 16 KB; e4m3 blocks are 8 KB and two MMAs
// each, so three share a barrier.
template <int kKv>
constexpr int kStageBlocks = kKv == kKvE4m3 ? 3 : 1;
template <int kKv>
constexpr int kStageBytes = kTile * 64 * (kKv == kKvE4m3 ? 1 : 2) * kStageBlocks<kKv>;

struct MassCtrl {
  uint64_t q_full;
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t raw_full[kMaxStages];   // int8: codes landed
  uint64_t raw_empty[kMaxStages];  // int8: codes written to the K ring
  uint64_t s_full[2];
  uint64_t s_free[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int first_b, first_tile;   // where this CTA's run of tiles begins
  int tiles;                 // and its length
  alignas(16) float2 row[kMaxRows];      // scale of the row's scores and its -lse, log2 domain
  uint64_t mask[kMaxTreeDrafts];         // trees: what each of the group's drafts sees
  alignas(16) int draft[kMaxRows];       // the row's draft (trees: from the group's first on)
  uint32_t live[kMaxRows / 32];          // a bit per row that adds something
};
constexpr int kCtrlBytes = 4096;
static_assert(sizeof(MassCtrl) <= kCtrlBytes, "control block");
constexpr int kMaxSmem = 232448;

// The shared memory a launch takes: alignment slack, control, Q (N rows x 1152 bytes in either
// format), and as many ring stages as fit.
struct MassShape {
  int rows, groups, stages, raw_stages, smem;
};
template <int kKv>
MassShape mass_shape(int R) {
  MassShape s;
  s.groups = (R + kMaxRows - 1) / kMaxRows;
  s.rows = ((R + s.groups - 1) / s.groups + 15) / 16 * 16;  // even groups, a multiple of the MMA's N step
  s.groups = (R + s.rows - 1) / s.rows;
  const int left = kMaxSmem - 1024 - kCtrlBytes - s.rows * kLatentDim * 2;
  s.raw_stages = 0;
  if (kKv >= kKvInt8) {  // of what is left, somewhat less than half for the K ring
    s.stages = std::min(6, left / (kStageBytes<kKv> + 5 * kRawBytes / 2));
    s.raw_stages = std::min(kMaxStages, (left - s.stages * kStageBytes<kKv>) / kRawBytes);
  } else {
    s.stages = std::min(kMaxStages, left / kStageBytes<kKv>);
  }
  s.smem = 1024 + kCtrlBytes + s.rows * kLatentDim * 2 + s.stages * kStageBytes<kKv> + s.raw_stages * kRawBytes;
  return s;
}

// Query rows of an e4m3 launch: q 2^s = hi + lo with each row's largest element in [128, 256),
// as K-major 64-byte-swizzled rows r (hi) and r + rows (lo) of nine blocks of 2 x rows rows.
// Eight lanes take a row, a chunk of eight columns of every block each, so a warp takes four rows
// and no lane idles: it is bound by its instructions (a row at a time, 72 chunks in three turns of
// 32 lanes, took 17.7 us for 8 requests of 2K-16K keys and 80 rows where this takes 16.6; the next
// four rows' loads in flight meanwhile changed nothing).  Rows past `real` repeat the last one.
// scale[r] becomes scale_log2 2^-s.
__device__ __forceinline__ void split_rows(const __nv_bfloat16* q, uint32_t q_smem, int rows, int real, int warp, int lane,
                                           float scale_log2, float2* scale) {
  const int l = lane & 7;
  // (rows is a multiple of 16: a warp's four rows exist or do not)
#pragma unroll 1
  for (int r = 4 * warp + (lane >> 3); r < rows; r += 4 * kEpiWarps) {
    const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<int64_t>(min(r, real - 1)) * kLatentDim) + l;
    uint4 w[kDimBlocks];
#pragma unroll
    for (int i = 0; i < kDimBlocks; ++i) w[i] = __ldg(src + 8 * i);
    __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < kDimBlocks; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[k])));
    }
    float mx = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^s from the exponent field, kept where both 2^s and 2^-s are normal numbers
    const int e = max(-110, min(static_cast<int>(__float_as_uint(mx) >> 23) - 127, 120));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
    if (l == 0) scale[r].x = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
#pragma unroll
    for (int i = 0; i < kDimBlocks; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t h[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // (8 significant bits below 256: exact in f16, and the residual too)
        const uint32_t x = pack_f16x2(__uint_as_float(u[k] << 16) * up, __uint_as_float(u[k] & 0xFFFF0000u) * up);
        const __half2 xh = *reinterpret_cast<const __half2*>(&x);
        const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(xh), __NV_SATFINITE, __NV_E4M3);
        const __half2 d = __hsub2(xh, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
        h[k] = c;
        lo[k] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(d), __NV_SATFINITE, __NV_E4M3);
      }
      auto put = [&](int row, const uint32_t (&c)[4]) {  // eight codes at byte 8 l of the block's 64-byte row
        const uint32_t at = q_smem + i * (2 * rows * 64) + row * 64 + ((((l >> 1) ^ (row >> 1)) & 3) << 4) + ((l & 1) << 3);
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(__byte_perm(c[0], c[1], 0x5410)),
                     "r"(__byte_perm(c[2], c[3], 0x5410))
                     : "memory");
      };
      put(r, h);
      put(r + rows, lo);
    }
  }
}

// Query rows of an int8 launch as f16 (rows past `real` repeat the last one).
__device__ __forceinline__ void half_rows(const __nv_bfloat16* q, uint32_t q_smem, int rows, int real, int warp, int lane) {
  for (int r = warp; r < rows; r += kEpiWarps) {
    const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<int64_t>(min(r, real - 1)) * kLatentDim);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = lane + 32 * i;  // chunk of eight columns, 72 in all
      if (c >= kLatentDim / 8) break;
      const uint4 w = __ldg(src + c);
      st_shared_v4(q_smem + (c >> 3) * (rows * 128) + r * 128 + (((c ^ r) & 7) << 4), bf16x2_to_f16x2(w.x),
                   bf16x2_to_f16x2(w.y), bf16x2_to_f16x2(w.z), bf16x2_to_f16x2(w.w));
    }
  }
}

template <int kKv>
__global__ void __launch_bounds__(threads_for(kKv), 1)
key_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                const KeyMassParams p) {
  constexpr bool kE4m3 = kKv == kKvE4m3, kInt8 = kKv == kKvInt8 || kKv == kKvInt8Page, kBf16 = kKv == kKvBf16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int N = p.group_rows;
  MassCtrl* ctrl = reinterpret_cast<MassCtrl*>(smem);
  uint8_t* q_s = smem + kCtrlBytes;                    // [9][N (e4m3: 2 N)][128 (64) bytes]
  uint8_t* ring = q_s + N * kLatentDim * 2;
  uint8_t* raw = ring + p.stages * kStageBytes<kKv>;   // int8: codes, [128][64] a slot
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % p.groups, set = blockIdx.x / p.groups;
  const int row0 = group * N, nrows = min(N, p.R - row0);

  if (threadIdx.x == 0) {
    mbar_init(&ctrl->q_full, kBf16 ? 1 : kEpiWarps);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int s = 0; s < p.raw_stages; ++s) {
      mbar_init(&ctrl->raw_full[s], 1);
      mbar_init(&ctrl->raw_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctrl->s_full[i], 1);
      mbar_init(&ctrl->s_free[i], kGroupWarps);
    }
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctrl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    if (kBf16) tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kv);
  }
  // programmatic dependent launch: no input is read before the previous kernel has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto bad_len = [&](int L) {
    return L < p.T || L > p.max_seq || L > static_cast<int64_t>(p.max_pages) * p.page_size;
  };
  auto tiles_of = [&](int b) -> int {
    const int L = p.seq_lens[b];
    return bad_len(L) ? 0 : (L + kTile - 1) / kTile;
  };
  if (warp == 0) {
    // This CTA's run.  Equal runs, tiles [total set / sets, total (set + 1) / sets) of the batch,
    // may cross from one request into the next, which costs a CTA the new queries and a drained
    // pipe: about a tile's time, on an e4m3 pool, whose queries are split, three.  Runs of whole
    // shares of one request, c tiles each, are taken instead where they are no longer than that
    // (8 requests of 2K-16K e4m3 keys: 24.7 -> 19.0 us; on 16 of 8K-131K bf16 keys neither is
    // better by more than the runs' scatter).
    const int mine = lane < p.B ? tiles_of(lane) : 0;  // (the first 32 requests stay in registers)
    auto tiles = [&](int b0) { return b0 == 0 ? mine : (b0 + lane < p.B ? tiles_of(b0 + lane) : 0); };
    auto sum_of = [&](auto&& f) {
      int s = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) s += f(tiles(b0));
      return __reduce_add_sync(0xffffffffu, s);
    };
    if (blockIdx.x == 0)
      for (int b = lane; b < p.B; b += 32)
        if (bad_len(p.seq_lens[b])) atomicOr(p.status, kStatusDeviceArg);
    const int total = sum_of([](int n) { return n; });
    const int even = (total + p.sets - 1) / p.sets;
    int share = 0;  // tiles of a whole share, or 0: equal runs
    for (int c = even; c > 0 && c <= even + (kE4m3 ? 3 : 1); ++c)
      if (sum_of([c](int n) { return (n + c - 1) / c; }) <= p.sets) {
        share = c;
        break;
      }
    // units (tiles or shares) before each request locate this CTA's first one
    auto units = [&](int n) { return share ? (n + share - 1) / share : n; };
    auto cut = [&](int s) { return static_cast<int>(static_cast<int64_t>(total) * s / p.sets); };
    const int begin = share ? set : cut(set);
    int fb = 0, ft = 0, count = share ? 0 : cut(set + 1) - begin, before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int nt = tiles(b0), n = units(nt);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > begin);
      if (hit) {
        const int l = __ffs(hit) - 1;
        const int at = __shfl_sync(0xffffffffu, before + incl - n, l);
        const int its = __shfl_sync(0xffffffffu, nt, l);
        fb = b0 + l;
        ft = (begin - at) * (share ? share : 1);
        if (share) count = min(share, its - ft);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      ctrl->first_b = fb;
      ctrl->first_tile = ft;
      ctrl->tiles = count;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  volatile int* abort_flag = &ctrl->abort_flag;
  constexpr int kBlocksPerStage = kStageBlocks<kKv>;
  constexpr int kStageB = kStageBytes<kKv>;
  constexpr int kBlockB = kStageB / kBlocksPerStage;
  const uint32_t s_cols = kE4m3 ? 2 * N : N;

  // Every role walks the same segments: the run's tiles of one request.
  int b = ctrl->first_b, it = ctrl->first_tile;
  int left = ctrl->tiles;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ TMA producer: lanes
    // share the pieces (page part, column block) of a stage
    uint64_t* const full = kInt8 ? ctrl->raw_full : ctrl->full;
    uint64_t* const empty = kInt8 ? ctrl->raw_empty : ctrl->empty;
    uint8_t* const into = kInt8 ? raw : ring;
    const int stages = kInt8 ? p.raw_stages : p.stages;
    constexpr int kLoadB = kInt8 ? kRawBytes : kStageB, kPieceB = kLoadB / kBlocksPerStage;
    const int P = p.page_size;
    const int parts = P >= kTile ? 1 : kTile / P, part_rows = kTile / parts;
    const uint64_t pol = p.groups == 1 ? policy_evict_first() : policy_evict_normal();
    const unsigned n_pages = static_cast<unsigned>(min(p.num_pages, static_cast<int64_t>(0x7fffffff)));
    bool bad_pid = false, ok = true;
    int slot = 0, phase = 0, issued = 0;
    while (ok && left > 0) {
      const int nt = tiles_of(b);
      if (it >= nt) {
        ++b;
        it = 0;
        continue;
      }
      const int n = min(nt - it, left);
      const int L = p.seq_lens[b];
      const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.max_pages;
      // pool row of this lane's page part of tile i; a part past the end, and an id outside the
      // pool (reported), lie before the first row, which TMA fills with zeros
      auto part_row = [&](int i) -> int {
        const int k = i * kTile + lane * part_rows;
        if (lane >= parts || k >= L) return -part_rows;
        const int pid = __ldg(pt + k / P);
        if (static_cast<unsigned>(pid) >= n_pages) {
          bad_pid = true;
          return -part_rows;
        }
        return pid * P + k % P;
      };
      int row = part_row(it);
      for (int i = 0; ok && i < n; ++i) {
        const int next = i + 1 < n ? part_row(it + i + 1) : 0;
#pragma unroll 1
        for (int c = 0; c < kDimBlocks; c += kBlocksPerStage) {
          bool w = true;
          if (lane == 0 && issued >= stages) w = mbar_wait(&empty[slot], phase ^ 1, abort_flag);
          ok = __shfl_sync(0xffffffffu, w, 0);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], kLoadB);
          __syncwarp();
          if (lane < parts) {
            uint8_t* dst = into + slot * kLoadB + lane * part_rows * (kPieceB / kTile);
#pragma unroll
            for (int k = 0; k < kBlocksPerStage; ++k)
              tma_load_2d(dst + k * kPieceB, &tm_kv, &full[slot], (c + k) * 64, row, pol);
          }
          ++issued;
          if (++slot == stages) {
            slot = 0;
            phase ^= 1;
          }
        }
        row = next;
      }
      left -= n;
      it += n;
    }
    if (__any_sync(0xffffffffu, bad_pid) && lane == 0) atomicOr(p.status, kStatusDeviceArg);
    if (!ok && lane == 0) {
      // copies still in flight land before the CTA exits: the last use of every stage
      for (int u = max(0, issued - stages); u < issued; ++u) drain_wait(&full[u % stages], (u / stages) & 1);
    }
    __syncwarp();
  } else if (kInt8 && warp > kMmaWarp) {
    // ------------------------------------------------------------------ int8 codes into the K ring as
    // f16: each warp takes every sixth (tile, column block).  (Reading the codes with loads
    // instead, whole sectors from 64-byte pieces of rows, held the in-flight bytes to what L1
    // can allocate: 313 us for 16 requests of 65536 keys and 32 rows where this takes 175.)
    // No more warps than stages of either ring: a warp that starts block u has seen block u -
    // warps filled and u - warps - stages consumed, so the parities it waits for are the right
    // ones.
    const int warps = min(kDecodeWarps, min(p.stages, p.raw_stages)), dw = warp - kMmaWarp - 1;
    const int blocks = left * kDimBlocks;
    bool ok = true;
    for (int u = dw; ok && dw < warps && u < blocks; u += warps) {
      const int rs = u % p.raw_stages, slot = u % p.stages, use = u / p.stages;
      bool go = true;
      if (lane == 0) {
        go = mbar_wait(&ctrl->raw_full[rs], (u / p.raw_stages) & 1, abort_flag);
        if (go && use > 0) go = mbar_wait(&ctrl->empty[slot], (use - 1) & 1, abort_flag);
      }
      ok = __shfl_sync(0xffffffffu, go, 0);
      if (!ok) break;
      // lane l: 16 codes, chunk l % 4 of rows l / 4 + 8 k
      const uint32_t from = smem_u32(raw) + rs * kRawBytes + lane * 16;
      const uint32_t to = smem_u32(ring) + slot * kStageB + (lane >> 2) * 128 + (lane & 3) * 32;
      const int sw = (lane >> 2) << 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = ld_shared_v4(from + (8 * h + k) * 512);
#pragma unroll
        for (int k = 0; k < 8; ++k) store_f16_chunk_int8(to + (8 * h + k) * 1024, sw, w[k]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctrl->full[slot]);
        mbar_arrive(&ctrl->raw_empty[rs]);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t idesc = kE4m3   ? make_idesc_e4m3(kTile, 2 * N)
                           : kInt8 ? make_idesc_f16(kTile, N, false, false)
                                   : make_idesc_bf16(kTile, N, false, false);
    const uint32_t q_block = N * 128;  // bytes of a column block of Q in either format
    bool ok = true;
    int slot = 0, phase = 0, t = 0, seg = 0;
    while (ok && left > 0) {
      const int nt = tiles_of(b);
      if (it >= nt) {
        ++b;
        it = 0;
        continue;
      }
      const int n = min(nt - it, left);
      ok = __all_sync(0xffffffffu, mbar_wait(&ctrl->q_full, seg & 1, abort_flag));
      for (int i = 0; ok && i < n; ++i, ++t) {
        const int buf = t & 1;
        if (t >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&ctrl->s_free[buf], ((t >> 1) - 1) & 1, abort_flag));
        const uint32_t d = tmem + buf * s_cols;
#pragma unroll 1
        for (int c = 0; ok && c < kDimBlocks; c += kBlocksPerStage) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ctrl->full[slot], phase, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kBlocksPerStage; ++k) {
              const uint32_t ka = smem_u32(ring + slot * kStageB + k * kBlockB), qa = smem_u32(q_s) + (c + k) * q_block;
              if constexpr (kE4m3) {
                const uint64_t kd = make_smem_desc_sw64(ka), qd = make_smem_desc_sw64(qa);
#pragma unroll
                for (int x = 0; x < 2; ++x) umma_f8(d, kd + 2 * x, qd + 2 * x, idesc, (c | k | x) != 0);
              } else {
                const uint64_t kd = make_smem_desc(ka, 16, 1024), qd = make_smem_desc(qa, 16, 1024);
#pragma unroll
                for (int x = 0; x < 4; ++x) umma_bf16(d, kd + 2 * x, qd + 2 * x, idesc, (c | k | x) != 0);
              }
            }
            umma_commit(&ctrl->empty[slot]);
            if (c + kBlocksPerStage >= kDimBlocks) umma_commit(&ctrl->s_full[buf]);
          }
          __syncwarp();
          if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      left -= n;
      it += n;
      ++seg;
    }
    if (elect_one()) {
      umma_commit(&ctrl->drain);
      drain_wait(&ctrl->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ weights and sums (warps
    // 0-7): warps 0-3 take even tiles, 4-7 odd ones; a thread owns the key of its TMEM lane
    const int mine = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int key_in_tile = 32 * (warp & 3) + lane;
    bool fail = false;
    int t = 0, seg = 0;
    while (left > 0) {
      const int nt = tiles_of(b);
      if (it >= nt) {
        ++b;
        it = 0;
        continue;
      }
      const int n = min(nt - it, left);
      const int L = p.seq_lens[b];
      const int p0 = L - p.T;
      // both groups have read every S of the segment before: its products are complete, and
      // Q and the rows' data may be replaced
      if (bar_or(1, kEpiThreads, fail || *abort_flag != 0)) break;
      if (kBf16 && threadIdx.x == 0) {
        mbar_arrive_expect_tx(&ctrl->q_full, N * kLatentDim * 2);
        tma_load_3d(q_s, &tm_q, &ctrl->q_full, 0, b * p.R + row0, 0, policy_evict_last());
      }
      if (warp < kMaxRows / 32) {  // a thread per row
        const int r = threadIdx.x;
        const float lse = r < nrows ? p.lse[static_cast<int64_t>(b) * p.R + row0 + r] : INFINITY;
        const bool live = fabsf(lse) < INFINITY;  // (false for NaN)
        const unsigned word = __ballot_sync(0xffffffffu, live);
        if (lane == 0) ctrl->live[warp] = word;
        ctrl->draft[r] = (row0 + r) / p.H - (p.tree_mask ? row0 / p.H : 0);
        const float neg_lse = live ? -lse * 1.4426950408889634f : 0.f;
        if (kE4m3) ctrl->row[r].y = neg_lse;
        else ctrl->row[r] = make_float2(p.scale_log2, neg_lse);
      } else if (p.tree_mask) {  // a thread per draft of the group
        const int t = row0 / p.H + threadIdx.x - kMaxRows;
        if (t * p.H < row0 + nrows) ctrl->mask[t - row0 / p.H] = p.tree_mask[static_cast<int64_t>(b) * p.T + t] & draft_bits(p.T);
      }
      if (kInt8) {
        half_rows(p.q + (static_cast<int64_t>(b) * p.R + row0) * kLatentDim, smem_u32(q_s), N, nrows, warp, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->q_full);
      }
      if (kE4m3) {
        split_rows(p.q + (static_cast<int64_t>(b) * p.R + row0) * kLatentDim, smem_u32(q_s), N, nrows, warp, lane,
                   p.scale_log2, ctrl->row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->q_full);
      }
      named_bar_sync(1, kEpiThreads);
      bool all_live = true;
      for (int r = 0; r < N; r += 16) all_live &= ((ctrl->live[r >> 5] >> (r & 31)) & 0xffffu) == 0xffffu;
      for (int i = 0; i < n; ++i, ++t) {
        if ((t & 1) != mine || fail) continue;
        const int k0 = (it + i) * kTile;
        const int key = k0 + key_in_tile;
        float* out = p.groups == 1 ? p.mass + static_cast<int64_t>(b) * p.mass_stride + key
                                   : p.part + (static_cast<int64_t>(group) * p.B + b) * p.max_seq + key;
        const bool accumulate = p.groups == 1 && p.decay != 0.f && key < L;
        const float old = accumulate ? *out : 0.f;
        float rel = 1.f;  // the scale of the key's page, relative to kv_scale
        bool bad_scale = false;
        if (kKv == kKvInt8Page && key < L) {
          const int pid = __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + key / p.page_size);
          rel = pid >= 0 && pid < p.num_pages ? __ldg(p.page_scales + pid) * p.inv_ref_scale : 0.f;
          // the decode's range; beyond it (or NaN) the key's weight would stay in the mass for good
          bad_scale = !(rel >= 0.f && rel <= 255.f);
          if (bad_scale) atomicOr(p.status, kStatusDeviceArg);
        }
        fail = __any_sync(0xffffffffu, !mbar_wait(&ctrl->s_full[mine], (t >> 1) & 1, abort_flag));
        if (fail) continue;
        tc_fence_after();
        const uint32_t s_tmem = tmem + lane_base + mine * s_cols;
        const int u = key - p0;  // draft index of this key (negative: prefix)
        const bool all = all_live && k0 + kTile <= p0;
        // trees: the group's drafts that see this key, a bit each
        uint64_t seers = ~0ull;
        if (!all && p.tree_mask && u >= 0) {
          seers = 0;
          const int drafts = (row0 + nrows - 1) / p.H - row0 / p.H + 1;
          if (u < p.T)
            for (int d = 0; d < drafts; ++d) seers |= ((ctrl->mask[d] >> u) & 1ull) << d;
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        auto add16 = [&](int c, const uint32_t(&v)[16], const uint32_t(&w)[16]) {
          auto weights = [&](int k, float& e0, float& e1) {
            const float4 rc = *reinterpret_cast<const float4*>(&ctrl->row[c + k]);
            float s0 = __uint_as_float(v[k]), s1 = __uint_as_float(v[k + 1]);
            if (kE4m3) {
              s0 += __uint_as_float(w[k]);
              s1 += __uint_as_float(w[k + 1]);
            }
            if (kKv == kKvInt8Page) {
              s0 *= rel;
              s1 *= rel;
            }
            e0 = ex2_approx(fmaf(s0, rc.x, rc.y));
            e1 = ex2_approx(fmaf(s1, rc.z, rc.w));
          };
          if (all) {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float e0, e1;
              weights(k, e0, e1);
              acc[(k >> 1) & 1] += e0;
              acc[2 + ((k >> 1) & 1)] += e1;
            }
          } else {
            const uint32_t live = ctrl->live[c >> 5] >> (c & 31);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float e0, e1;
              weights(k, e0, e1);
              const int2 d = *reinterpret_cast<const int2*>(&ctrl->draft[c + k]);
              const bool see0 = p.tree_mask ? (seers >> (d.x & 63)) & 1 : u <= d.x;
              const bool see1 = p.tree_mask ? (seers >> (d.y & 63)) & 1 : u <= d.y;
              acc[(k >> 1) & 1] += see0 && ((live >> k) & 1) ? e0 : 0.f;
              acc[2 + ((k >> 1) & 1)] += see1 && ((live >> (k + 1)) & 1) ? e1 : 0.f;
            }
          }
        };
#pragma unroll 1
        for (int c = 0; c < N; c += 32) {  // two loads of 16 columns a wait
          uint32_t v[2][16], w[2][16];
          const bool two = c + 16 < N;
          tmem_ld16(s_tmem + c, v[0]);
          if (kE4m3) tmem_ld16(s_tmem + N + c, w[0]);
          if (two) tmem_ld16(s_tmem + c + 16, v[1]);
          if (kE4m3 && two) tmem_ld16(s_tmem + N + c + 16, w[1]);
          tmem_ld_wait();
          add16(c, v[0], w[0]);
          if (two) add16(c + 16, v[1], w[1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->s_free[mine]);
        const float sum = bad_scale ? 0.f : (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if (key < L) *out = accumulate ? fmaf(p.decay, old, sum) : sum;
      }
      left -= n;
      it += n;
      ++seg;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && ctrl->abort_flag) atomicOr(p.status, kStatusTimeout);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Row groups' sums into the mass, in the groups' order.
__global__ void __launch_bounds__(256) key_mass_join_kernel(const KeyMassParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y, key = blockIdx.x * 256 + threadIdx.x;
  const int L = p.seq_lens[b];
  if (L < p.T || L > p.max_seq || L > static_cast<int64_t>(p.max_pages) * p.page_size || key >= L) return;
  float sum = 0.f;
  for (int g = 0; g < p.groups; ++g) sum += p.part[(static_cast<int64_t>(g) * p.B + b) * p.max_seq + key];
  float* m = p.mass + static_cast<int64_t>(b) * p.mass_stride + key;
  *m = p.decay == 0.f ? sum : fmaf(p.decay, *m, sum);
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kKv>
cudaError_t launch(KeyMassParams p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv, int num_sms, cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(key_mass_kernel<kKv>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const MassShape s = mass_shape<kKv>(p.R);
  p.group_rows = s.rows;
  p.groups = s.groups;
  p.stages = s.stages;
  p.raw_stages = s.raw_stages;
  // one CTA per SM, and no more sets than tiles
  const int64_t tiles = static_cast<int64_t>(p.B) * ((p.max_seq + kTile - 1) / kTile);  // (below 2^31: the caller)
  p.sets = static_cast<int>(std::min(static_cast<int64_t>(std::max(1, num_sms / s.groups)), tiles));
  e = launch_dependent(key_mass_kernel<kKv>, dim3(p.sets * s.groups), threads_for(kKv), s.smem, stream, tm_q, tm_kv, p);
  if (e != cudaSuccess || s.groups == 1) return e;
  return launch_dependent(key_mass_join_kernel, dim3((p.max_seq + 255) / 256, p.B), 256, 0, stream, p);
}

}  // namespace

int key_mass_group_rows(int R) { return mass_shape<kKvBf16>(R).rows; }

size_t key_mass_part_bytes(int B, int R, int max_seq) {
  const int groups = mass_shape<kKvBf16>(R).groups;
  return groups == 1 ? 0 : static_cast<size_t>(groups) * B * max_seq * sizeof(float);
}

cudaError_t launch_key_mass(const KeyMassParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_kv, int num_sms,
                            cudaStream_t stream) {
  switch (p.kv_dtype) {
    case kKvE4m3: return launch<kKvE4m3>(p, tm_q, tm_kv, num_sms, stream);
    case kKvInt8: return launch<kKvInt8>(p, tm_q, tm_kv, num_sms, stream);
    case kKvInt8Page: return launch<kKvInt8Page>(p, tm_q, tm_kv, num_sms, stream);
    default: return launch<kKvBf16>(p, tm_q, tm_kv, num_sms, stream);
  }
}

}  // namespace mla
