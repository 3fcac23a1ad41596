// mla_decode_fp4_sm103a.cu -- absorbed MLA decode over a 4-bit paged latent KV cache, sm_103a.
//
// What it computes: out[b,t,h] = sum_j softmax_j(scale q.k_j) k_j[:512] over the keys that draft t sees
// (0 .. L - T + t, or a tree's mask), with the latent rows stored as e2m1 codes under a power of two per
// 16 columns and the rotated columns as e4m3 codes (include/mla.h, MLA_KV_FP4), all times kv_scale.
//
// Every value of a row in units of kv_scale is an e4m3 number exactly: magnitude (2 bits of significand)
// times 2^(e-5), e = 0..11, lies in 2^-6 .. 384.  So a tile is decoded to e4m3 codes, once, and both
// products run on 8-bit tensor-core operands:
//  * BMM1: S^T[key, row] = K Q^T, M = 128 keys, A = K from tensor memory (a key is a lane), B = the query
//    rows, each bf16 row scaled by a power of two and split into q_hi = e4m3(q) and q_lo = e4m3(q - q_hi)
//    (8 bits of significand: exact down to 2^-9 of the row's largest |q|), one product after the other
//    into the same accumulator.  A from tensor memory keeps 72 KB a tile of operand reads off shared
//    memory.
//  * BMM2: O^T[value column, row] += V^T P^T, A = V^T, MN-major out of shared memory, B = the weights,
//    P 2^6 split into p_hi = e4m3(P) and p_lo = e4m3(28 (P - p_hi)), stacked as 2 x NR columns so that V
//    is read once; the epilogue adds O_hi + O_lo / 28.  (P 2^6 <= 448, its residual at most 16: kept to 2^-9
//    relative where P 2^6 >= 2^-6, to 2^-14.8 absolute below.)
//  * A key is one thread's in the softmax, so a row's sum is kept per thread and its reference, which takes the
//    place of a running maximum, moves only when some score exceeds it by more than 2.8 (log2): ordinary tiles
//    reduce nothing across threads but one vote and a word of marks.
//  * A reference also goes down.  Behind a key that dominates its row (an attention sink) every other weight would
//    fall below what hi + lo hold: of 20000 even keys behind one of 99 % nothing or twice their weight was left, by
//    chance.  O and the sums are fp32 and have room above: where no weight reaches 2^-5 in two tiles on end, the row's
//    reference is lowered by 2^8 and what it has accumulated multiplied by as much.  Warps mark such rows after their
//    weights are written, read all marks after the next vote and move at the tile after it, so no wait is added: three
//    tiles go by.  A first key that stands alone in its tile, or one 2^8 above the reference, gets 448 and the keys beside
//    it the whole range below.  (16 requests of 8K-131K keys: 99.2 -> 101.0 us at 32 rows of flat scores, 86.0 -> 89.9
//    at 16.  Deciding in the same tile took 104.7 and 91.5; a vote on each warp's own marks 132 at 32 rows of normal scores,
//    111 here.)
//    Very uneven scores lower references that soon rise again, two waits for BMM2 where there was one: with deviations
//    of 2.6, 3.5 and 5.2 (nats) 32 rows take 119.6, 125.3 and 144.9 us, without 115.5, 118.3 and 122.6.  So a row that
//    has risen again waits for twice as many low tiles, up to eight.  (2^-5 is the least that leaves hi normal; lowered
//    from 2^-2, after one tile, 128, 143 and 158.)
// One CTA per (group of NR rows, split, request), 128 keys a tile, 576 threads: softmax warps 0-7 (32 keys
// and half of the rows each), decoding warps 8-15 (32 keys and half of the columns each; a row's codes go
// to registers at once and free their stage), producer 16 (boxes of up to 64 rows), MMA 17.
// What bounds it: shared memory, and a tile's chain of decoding, BMM1, softmax and BMM2.  A tile takes 2.6k cycles at 16 rows
// and 2.95k at 32 (its 43 KB 1.85k at the copy rate), of which shared memory is busy 2.0k and 2.4k: rows in and out 0.34k
// each, V in 0.5k, V and P as BMM2's operands 0.6-0.8k, queries 0.15-0.3k, P.  One thread issues 52 small products beside
// four busy warps for 2.1k of the 2.95k (1.4k alone on an SM), decoding takes half the integer pipe, and one or two tiles fit
// in tensor memory to overlap them.
// 16 requests of 8K-131K keys (375 MB, 55 us of bytes): 90 us at 16 rows; at 32 rows 111, of which 10 are references that
// move (101 with scores that move none): the next tile then waits for BMM2 of the last.
// Every wait is bounded; on expiry the CTA records a timeout, drains its copies and MMAs, frees tensor
// memory and returns.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fp4_rows.cuh"
#include "mla_internal.h"
#include "sm103a_ptx.cuh"
#include "tree_mask.cuh"

namespace mla {
namespace {

constexpr int kTile = kFp4TileKeys;               // keys per tile
constexpr int kSub = 64;                          // keys per raw stage (half a tile)
constexpr int kRawStage = kSub * kFp4RowBytes;    // 21504
constexpr int kVBlock = kTile * 64;               // 128 keys x 64 codes (64-byte swizzle)
constexpr int kVTile = (kValueDim / 64) * kVBlock;
constexpr int kKCols = kLatentDim / 4;            // tensor-memory columns of a decoded tile
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kDecodeWarps = 8;
constexpr int kDecodeThreads = 32 * kDecodeWarps;
constexpr int kWorkers = kSoftmaxThreads + kDecodeThreads;
constexpr int kProducerWarp = 16, kMmaWarp = 17;
constexpr int kThreads = 576;
constexpr int kMaxRaw = 3;
constexpr int kMaxFull = 6;
constexpr int kMaxRows = 32;
constexpr int kCtrlBytes = 4096;
constexpr int kAbortTimeout = 1;
constexpr int64_t kMostEmpty = 304;  // CTAs without a split that a grid may have: two for each of the GPU's 152 SMs, however
                                     // many of them the plan was made for
constexpr uint32_t kTmemCols = 512;
constexpr float kPShift = 6.0f;    // P is formed times 2^6 ...
constexpr float kThreshold = 2.8f; // ... and at most 2^8.8: the reference moves when a score exceeds it by more than this,
constexpr float kMargin = 0.6780719f;  // to so much above the score, whose weight is then 40, an e4m3 number: a weight that
                                   // dominates its row has no error
constexpr float kFar = 8.f;        // A first key, or one so far above the reference, whose weight may be all that counts of its
constexpr float kFarMargin = -2.8073549f;  // tile, gets 448, the largest weight: the keys beside it keep the most bits
constexpr uint32_t kLowCodes = 0x70707070u;  // brings the e4m3 code of 2^-5, 0x10, to a byte's top bit, and of 448 not past it
constexpr float kDrop = 8.f;       // a reference goes down so far where a row's tiles weigh less than 2^-5 ...
constexpr float kDropFactor = 256.f;
constexpr int kLowTiles = 2, kMostLowTiles = 8;  // ... so many on end, at first and after it came up again ...
constexpr float kDepth = 40.f;     // ... until it is this far below the highest that it has been
constexpr int kNoScore = static_cast<int>(0x807fffffu);  // -infinity as an ordered integer
constexpr float kLoScale = 28.0f;  // p_lo carries 28 times the residual (at most 16).  With 32, 2 and 1 in these places, the same
                                   // error below, references moved more often: 112.4 us on 32 rows

template <int NR>
struct Map {
  static constexpr int kRaw = NR == 16 ? 3 : 2;        // raw stages
  static constexpr int kFull = NR == 16 ? 6 : 2;       // least common multiple of the stages and a tile's two
  static constexpr int kKBufs = NR == 16 ? 2 : 1;      // decoded K tiles in tensor memory
  static constexpr bool kHalves = NR == 32;            // one tile: handed over and freed in two halves
  static constexpr int kQBlock = NR * 64;
  static constexpr int kQPart = 9 * kQBlock;           // q_hi or q_lo
  static constexpr int kPBuf = 2 * NR * kTile;
  static constexpr int kOffV = 0;
  static constexpr int kOffQ = kOffV + 2 * kVTile;
  static constexpr int kOffP = kOffQ + 2 * kQPart;
  static constexpr int kOffRaw = kOffP + 2 * kPBuf;
  static constexpr int kOffCtrl = kOffRaw + kRaw * kRawStage;
  static constexpr int kSmem = kOffCtrl + kCtrlBytes + 1024;
  // tensor memory: O^T (4 chunks of hi | lo columns), S^T (2 buffers), K
  static constexpr uint32_t kO = 0;
  static constexpr uint32_t kS = 8 * NR;
  static constexpr uint32_t kK = kS + 2 * NR;
  static_assert(kK + kKBufs * kKCols <= kTmemCols, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory per block");
  static_assert(kOffP % 1024 == 0 && kOffQ % 512 == 0 && kOffRaw % 16 == 0 && kOffCtrl % 16 == 0, "alignment");
};

struct Ctrl {
  // Copies landed.  A wait by parity has to see every phase of its barrier, and a decoding warp reads every other
  // stage only: so a barrier of its own for each stage and half of a tile.
  uint64_t raw_full[kMaxFull];
  uint64_t raw_empty[kMaxRaw];  // the four warps of the stage's keys have it in registers
  uint64_t q_ready;             // split queries written
  uint64_t k_full[2];           // tile decoded into tensor memory (tile parity)
  uint64_t v_full[2];           // and copied into its V buffer
  uint64_t k_free[2];           // BMM1 of the tile done
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2];
  uint64_t o_done[2];           // BMM2 of the tile done
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int item[4];                  // request (-1: none), split and length; all splits
  int2 found[kThreads / 32];    // whole splits and remainders of 32 requests
  alignas(16) float mult[kMaxRows];   // scale_log2 2^-s of the row's split; 0: no such row
  alignas(16) float off[kSoftmaxWarps][kMaxRows];  // kPShift - reference maximum, a copy for each warp
  alignas(16) int top[3][kMaxRows];   // largest score (ordered as an integer) of the rows that outgrew their reference, by
                                      // tile: written before a tile's vote, read after it, cleared after the next one
  alignas(16) uint32_t low[2][kSoftmaxWarps];  // rows (row_mark) of which a warp's keys all weigh less than 2^-5, by tile parity
  alignas(16) uint32_t alone[kSoftmaxWarps];   // and less than 2^-2, where first keys are
  alignas(16) float row_scale[kMaxRows];
  alignas(16) float lse[kMaxRows];
  alignas(16) int lim[kMaxRows];      // last key that the row sees; -1: none
  alignas(16) uint64_t drafts[kMaxRows];
  alignas(16) float sums[4][kMaxRows];
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t h2;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h2) : "r"(codes));
  return h2;
}

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

__device__ __forceinline__ void st_shared_v2(uint32_t saddr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(saddr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
}

__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// P as BMM2's B operand, MN-major: 2 NR bytes a key (hi of the NR rows, then lo), so that a thread stores its
// key's rows whole.  32-byte rows are swizzled by 32 bytes (code 6: the 16-byte chunk's bit XORed with bit 2 of
// the key), 64-byte rows by 64 (code 4: two bits with bits 1-2); groups of eight keys follow one another.
template <int NR>
__device__ __forceinline__ uint64_t p_smem_desc(uint32_t saddr) {
  constexpr uint64_t kSwizzle = NR == 16 ? 6 : kSwizzle64B;
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16 * NR >> 4) << 16) |
         (static_cast<uint64_t>(16 * NR >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (kSwizzle << 61);
}

// A warp's arrival once its loads from a stage are in registers.
__device__ __forceinline__ void release_stage(uint64_t* bar, int lane) {
  __threadfence_block();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Sum (or largest) of v[r] over the warp's lanes, value r left in the lanes with lane / (32 / NR) == r.
template <int NR, bool kMax = false>
__device__ __forceinline__ float lanes_reduce(float (&v)[NR], int lane) {
  const auto both = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int n = NR / 2, o = 16; o > 0; n >>= 1, o >>= 1) {
    if (n >= 1) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool up = (lane & o) != 0;
        const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
        v[i] = both(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    } else {
      v[0] = both(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

// The item-th split of the batch in the order "whole splits, then remainders", by the whole CTA, a thread a request:
// request, split and the request's length to ctrl->item[0 .. 2] (request -1 past the last), the number of splits to
// item[3].  A bad length counts as none (the first CTA reports it).
__device__ __forceinline__ void find_split(const DecodeParams& p, int item, bool report, Ctrl* ctrl) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int L = t < p.B ? __ldg(p.seq_lens + t) : 0;
  const bool bad = t < p.B && (L < p.T || L > p.max_seq || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_pages) * p.page_size);
  if (bad) {
    L = 0;
    if (report) atomicOr(p.status, kStatusDeviceArg);
  }
  const int whole = L / p.chunk;
  const uint32_t rest = __ballot_sync(0xffffffffu, L > whole * p.chunk);
  int sum = whole;  // inclusive, over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) ctrl->found[warp] = make_int2(sum, __popc(rest));
  if (t == 0) ctrl->item[0] = -1;
  __syncthreads();
  int wholes = 0, rests = 0, at = sum - whole, rest_at = __popc(rest & ((1u << lane) - 1));
  for (int w = 0; 32 * w < p.B; ++w) {
    const int2 n = ctrl->found[w];
    if (w < warp) at += n.x, rest_at += n.y;
    wholes += n.x, rests += n.y;
  }
  if (item >= at && item < at + whole) ctrl->item[0] = t, ctrl->item[1] = item - at, ctrl->item[2] = L;
  if ((rest >> lane & 1) && item - wholes == rest_at) ctrl->item[0] = t, ctrl->item[1] = whole, ctrl->item[2] = L;
  if (t == 0) ctrl->item[3] = wholes + rests;
  __syncthreads();
}

// Where a warp's marks hold its row r.
__device__ __forceinline__ uint32_t row_mark(int r) { return 0x80u << 8 * (r & 3) >> (r >> 2); }

// The rows of which no lane has a weight of 2^-5 or more: hi4 holds their e4m3 codes, four rows a word.
template <int N>
__device__ __forceinline__ uint32_t low_rows(const uint32_t (&hi4)[N]) {
  uint32_t some = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) some |= ((hi4[k] + kLowCodes) & 0x80808080u) >> k;
  return ~__reduce_or_sync(0xffffffffu, some);
}

template <int NR>
__device__ __forceinline__ void load_s(uint32_t addr, uint32_t (&s)[NR]) {
  if constexpr (NR == 8) tmem_ld8(addr, s);
  if constexpr (NR == 16) tmem_ld16(addr, s);
  tmem_ld_wait();
}

template <int NR>
__device__ __forceinline__ void init_barriers(Ctrl* ctrl) {
  for (int s = 0; s < kMaxFull; ++s) mbar_init(&ctrl->raw_full[s], 1);
  for (int s = 0; s < kMaxRaw; ++s) mbar_init(&ctrl->raw_empty[s], 4);
  mbar_init(&ctrl->q_ready, kDecodeWarps);
  for (int s = 0; s < 2; ++s) {
    mbar_init(&ctrl->k_full[s], kDecodeWarps);
    mbar_init(&ctrl->v_full[s], kDecodeWarps);
    mbar_init(&ctrl->k_free[s], 1);
    mbar_init(&ctrl->s_full[s], 1);
    mbar_init(&ctrl->s_free[s], kSoftmaxWarps);
    mbar_init(&ctrl->p_full[s], kSoftmaxWarps);
    mbar_init(&ctrl->o_done[s], 1);
  }
  mbar_init(&ctrl->drain, 1);
  fence_mbarrier_init();
}

// One split (keys kv_start and on of request b) for the rows of a group, by the whole CTA; ends with all roles in step.
// kTree: drafts see each other by p.tree_mask instead of in order.
template <int NR, bool kTree>
__device__ __forceinline__ void take_split(const CUtensorMap& tm_kv, const DecodeParams& p, uint8_t* smem, int group, int b, int split, int L) {
  using M = Map<NR>;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + M::kOffCtrl);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t tmem = ctrl->tmem_base;
  const int kv_start = split * p.chunk;
  const int kv_end = min(L, kv_start + p.chunk);
  const int ntiles = (kv_end - kv_start + kTile - 1) / kTile;
  const int nsplit_b = (L + p.chunk - 1) / p.chunk;
  const int row0 = group * NR;
  const int nrows = min(NR, p.R - row0);
  volatile int* abort_flag = &ctrl->abort_flag;
  const bool final_out = nsplit_b == 1;
  bool worker_failed = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer: raw rows, 64 keys a stage
    const int lg = __ffs(p.page_size) - 1;          // (a power of two)
    const int per = max(1, kSub >> lg);             // pages per stage
    const int box_bytes = min(p.page_size, kSub) * kFp4RowBytes;
    const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    const int last_page = (kv_end - 1) >> lg;
    int base = kv_start >> lg;
    int cur = base + lane <= last_page ? __ldg(pt + base + lane) : 0;
    int nxt = base + 32 + lane <= last_page ? __ldg(pt + base + 32 + lane) : 0;
    const uint64_t policy = policy_evict_first();
    const unsigned n_pages = static_cast<unsigned>(min(p.num_pages, static_cast<int64_t>(0x7fffffff)));
    bool bad_pid = false, ok = true;
    int issued = 0;
    int s = 0;
    uint32_t parity = 1;  // of the stage's previous release (none to wait for in the first round)
    for (int i = 0; i < 2 * ntiles; ++i) {
      const int k0 = kv_start + i * kSub, pg0 = k0 >> lg;
      const int npg = k0 < kv_end ? min(per, last_page - pg0 + 1) : 0;  // (none: past the end of the last tile)
      if (pg0 - base >= 32) {  // advance the window of page ids (warp-uniform; a stage's pages lie in one half: both
        base += 32;            // start at a multiple of `per` pages)
        cur = nxt;
        const int nb = base + 32 + lane;
        nxt = nb <= last_page ? __ldg(pt + nb) : 0;
      }
      // (everything but the copies is done before the wait)
      const int pid = __shfl_sync(0xffffffffu, cur, (pg0 + lane - base) & 31);  // lane k: the stage's k-th page
      // a page id outside the pool: a box wholly before the first row, which arrives as zeros
      const bool outside = static_cast<unsigned>(pid) >= n_pages;
      bad_pid |= outside && lane < npg;
      const int y = outside ? -kSub : (pid << lg) + (k0 & (p.page_size - 1));
      uint8_t* dst = smem + M::kOffRaw + s * kRawStage;
      ok = mbar_wait(&ctrl->raw_empty[s], parity, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint64_t* full = &ctrl->raw_full[i % M::kFull];
      if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(npg * box_bytes));
      __syncwarp();
      if (lane < npg) tma_load_2d(dst + lane * box_bytes, &tm_kv, full, 0, y, policy);
      issued = i + 1;
      if (++s == M::kRaw) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (bad_pid) atomicOr(p.status, kStatusDeviceArg);
    // copies still in flight (their readers may have given up) land before the CTA exits
    for (int k = max(0, issued - M::kRaw); k < issued; ++k) drain_wait(&ctrl->raw_full[k % M::kFull], (k / M::kFull) & 1);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer: BMM1 of a tile goes before BMM2 of
    // the last one, so that its K columns and the next softmax wait for one product, not two.  (Issuing whichever was
    // ready first, by polling: 135 us where this takes 107.)
    const uint32_t idesc1 = make_idesc_e4m3(128, NR);
    const uint32_t idesc2 = make_idesc_e4m3(128, 2 * NR, true, true);
    const uint64_t hi_desc = make_smem_desc_sw64(smem_u32(smem + M::kOffQ));
    const uint64_t lo_desc = make_smem_desc_sw64(smem_u32(smem + M::kOffQ + M::kQPart));
    bool ok = mbar_wait(&ctrl->q_ready, 0, abort_flag);
    for (int j = 0; j <= ntiles; ++j) {
      if (j < ntiles) {
        const int sb = j & 1, kb = j % M::kKBufs;
        const uint32_t d = tmem + M::kS + sb * NR;
        const uint32_t a = tmem + M::kK + kb * kKCols;
        if (ok && j >= 2) ok = mbar_wait(&ctrl->s_free[sb], ((j - 2) >> 1) & 1, abort_flag);
        if (ok) ok = M::kHalves ? mbar_wait(&ctrl->k_full[0], j & 1, abort_flag) : mbar_wait(&ctrl->k_full[sb], (j >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const auto block = [&](int c, bool more) {  // 64 columns
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint64_t off = static_cast<uint64_t>((c * M::kQBlock + k * 32) >> 4);
            umma_f8_ts(d, a + c * 16 + k * 8, hi_desc + off, idesc1, more || k != 0 ? 1u : 0u);
            umma_f8_ts(d, a + c * 16 + k * 8, lo_desc + off, idesc1, 1u);
          }
        };
        // (unrolled, the descriptors of all 36 products would be kept in registers, or spilled)
        if constexpr (M::kHalves) {
          if (elect_one()) {
#pragma unroll 1
            for (int c = 0; c < 6; c += c == 1 ? 3 : 1) block(c, c != 0);  // columns 0-127, 256-383
            umma_commit(&ctrl->k_free[0]);
          }
          __syncwarp();
          ok = mbar_wait(&ctrl->k_full[1], j & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 1
            for (int c = 2; c < 9; c += c == 3 ? 3 : 1) block(c, true);
            umma_commit(&ctrl->s_full[sb]);
            umma_commit(&ctrl->k_free[1]);
          }
        } else if (elect_one()) {
#pragma unroll 1
          for (int c = 0; c < 9; ++c) block(c, c != 0);
          umma_commit(&ctrl->s_full[sb]);
          umma_commit(&ctrl->k_free[kb]);
        }
        __syncwarp();
      }
      if (j > 0) {
        const int jv = j - 1, pb = jv & 1;
        if (ok) ok = mbar_wait(&ctrl->v_full[pb], (jv >> 1) & 1, abort_flag);
        if (ok) ok = mbar_wait(&ctrl->p_full[pb], (jv >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint64_t v_desc = make_smem_desc_sw64(smem_u32(smem + M::kOffV + pb * kVTile), kVBlock, 512);
        const uint64_t p_desc = p_smem_desc<NR>(smem_u32(smem + M::kOffP + pb * M::kPBuf));
        if (elect_one()) {
#pragma unroll 1
          for (int qc = 0; qc < 4; ++qc) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f8(tmem + M::kO + qc * 2 * NR, v_desc + static_cast<uint64_t>((2 * qc * kVBlock + kk * 2048) >> 4),
                      p_desc + static_cast<uint64_t>((kk * 32 * 2 * NR) >> 4), idesc2, (jv > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&ctrl->o_done[pb]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {  // every MMA completes before tensor memory is released
      umma_commit(&ctrl->drain);
      drain_wait(&ctrl->drain, 0);
      // and every arrival that no other warp waits for lands before the barriers serve another split
      for (int j = max(0, ntiles - 2); ok && j < ntiles; ++j) {
        drain_wait(&ctrl->o_done[j & 1], (j >> 1) & 1);
        if (!M::kHalves) drain_wait(&ctrl->k_free[j & 1], (j >> 1) & 1);
      }
      for (int h = 0; M::kHalves && ok && h < 2; ++h) drain_wait(&ctrl->k_free[h], (ntiles - 1) & 1);
    }
    __syncwarp();
  } else if (warp >= kSoftmaxWarps) {
    // ------------------------------------------------------------------ decoding warps
    const int dw = warp - kSoftmaxWarps, quad = dw & 3, half = dw >> 2;
    bool failed = false;
    {
      // Split of the queries: kPer adjacent threads a row, 16-byte chunks t, t + kPer, ...
      constexpr int kPer = kDecodeThreads / NR, kChunks = (72 + kPer - 1) / kPer;
      const int t = (threadIdx.x - kSoftmaxThreads) % kPer, r = (threadIdx.x - kSoftmaxThreads) / kPer;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(b) * p.R + row0 + r) * kLatentDim);
      uint4 w[kChunks];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = t + kPer * i;
        w[i] = r < nrows && c < 72 ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
      }
#pragma unroll
      for (int o = kPer / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      int sh = 0;  // the row's power of two: its largest |q| lands in [128, 256)
      if (mx > 0.f) sh = min(126, max(-120, 7 - (static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu) - 127)));
      const float mul = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = t + kPer * i;
        if (c >= 72) continue;
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[2], l[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x0 = __uint_as_float(u[2 * k + e] << 16) * mul, x1 = __uint_as_float(u[2 * k + e] & 0xFFFF0000u) * mul;
            h[e] = f32x2_to_e4m3x2(x0, x1);
            const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2(h[e]));
            l[e] = f32x2_to_e4m3x2(x0 - v.x, x1 - v.y);
          }
          hi[k] = h[0] | (h[1] << 16);
          lo[k] = l[0] | (l[1] << 16);
        }
        const uint32_t at = smem_u32(smem + M::kOffQ) + (c >> 3) * M::kQBlock + r * 64 + ((((c >> 1) & 3) ^ ((r >> 1) & 3)) << 4) + (c & 1) * 8;
        st_shared_v2(at, hi[0], hi[1]);
        st_shared_v2(at + M::kQPart, lo[0], lo[1]);
      }
      if (t == 0) {
        const bool real = r < nrows;
        // (an infinite query has no finite score: its row becomes NaN)
        ctrl->mult[r] = !real ? 0.f : mx == INFINITY ? NAN : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
        // (no such row: -infinity; a row that has seen nothing: +infinity, so that its first key shows)
        for (int w = 0; w < kSoftmaxWarps; ++w) ctrl->off[w][r] = real ? INFINITY : -INFINITY;
        for (int k = 0; k < 3; ++k) ctrl->top[k][r] = kNoScore;
        const int draft = (row0 + r) / p.H;
        ctrl->lim[r] = real ? L - p.T + draft : -1;
        if (kTree) ctrl->drafts[r] = real ? p.tree_mask[static_cast<int64_t>(b) * p.T + draft] & draft_bits(p.T) : 0ull;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->q_ready);
    }
    // A tile's codes go to tensor memory first (K) and from there to shared memory (V), one tile later where two K
    // tiles fit: BMM1 and the softmax then need not wait for a V buffer, nor the next tile's decoding.
    const int row = quad * 32 + lane;  // this thread's key of a tile
    const uint32_t v_row = smem_u32(smem + M::kOffV) + row * 64 + half * 4 * kVBlock;
    const uint32_t sw = ((row >> 1) & 3) << 4;
    const uint32_t k_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + M::kK + half * 64;
    const uint32_t raw_at = ((quad & 1) * 32 + lane) * kFp4RowBytes;
    constexpr int kLag = M::kKBufs - 1;  // with two K tiles, the V copy runs a tile behind
    for (int j = 0; j < ntiles + kLag; ++j) {
      bool ok = true;
      if (j < ntiles) {
        uint4 w[8], rope[2];
        uint32_t ex[2];
        const int i = 2 * j + (quad >> 1), s = i % M::kRaw;
        ok = mbar_wait(&ctrl->raw_full[i % M::kFull], (i / M::kFull) & 1, abort_flag);
        const uint32_t raw = smem_u32(smem + M::kOffRaw + s * kRawStage) + raw_at;
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = ld_shared_v4(raw + half * 128 + k * 16);
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(ex[0]), "=r"(ex[1]) : "r"(raw + 256 + half * 8));
#pragma unroll
        for (int k = 0; k < 2; ++k) rope[k] = ld_shared_v4(raw + 272 + half * 32 + k * 16);
        const int kb = j % M::kKBufs;
        // The stage may be overwritten as soon as it is released, and an arrival does not wait for loads on their way to
        // registers (measured: rows of the next tile in one of 20 calls): the fence does.  With two K tiles the release
        // comes after the first columns, the loads spread over the decoding: 89 us on 16 requests of 8K-131K keys, one
        // token, where the loads all at once took 95; with one K tile they fill the wait for it (106 against 121).
        constexpr int kRelease = M::kKBufs == 2 ? 0 : -1;
        if (kRelease < 0) release_stage(&ctrl->raw_empty[s], lane);
        // the K columns are free once BMM1 of their last tile has completed (this warp's own reads have)
        if (ok && j >= M::kKBufs) ok = mbar_wait(&ctrl->k_free[M::kHalves ? 0 : kb], ((j / M::kKBufs) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t kcol = k_lane + kb * kKCols;
        const uint32_t nibble[2][2] = {{ex[0] & 0x0F0F0F0Fu, ex[1] & 0x0F0F0F0Fu}, {(ex[0] >> 4) & 0x0F0F0F0Fu, (ex[1] >> 4) & 0x0F0F0F0Fu}};
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {  // 64 columns: 16 columns of tensor memory
          uint32_t o[16];
#pragma unroll
          for (int k1 = 0; k1 < 2; ++k1) {
            const int k = 2 * k2 + k1;
            const uint32_t word[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // 16 columns under one power of two
              const uint32_t e = __byte_perm(nibble[g][k >> 2], 0u, 0x4440u | (k & 3));
              uint32_t lo, hi;
              fp4_table(e, lo, hi);
              fp4_to_e4m3(word[2 * g], lo, hi, o[8 * k1 + 4 * g], o[8 * k1 + 4 * g + 1]);
              fp4_to_e4m3(word[2 * g + 1], lo, hi, o[8 * k1 + 4 * g + 2], o[8 * k1 + 4 * g + 3]);
            }
          }
          tmem_st16(kcol + k2 * 16, o);
          if (k2 == kRelease) release_stage(&ctrl->raw_empty[s], lane);
          if (M::kHalves && k2 == 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctrl->k_full[0]);
            if (j >= 1) ok = mbar_wait(&ctrl->k_free[1], (j - 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);  // (what follows the loop asks it again)
            if (!ok) break;
            tc_fence_after();
          }
        }
        if (!ok) {
          failed = true;
          break;
        }
        const uint32_t ro[8] = {rope[0].x, rope[0].y, rope[0].z, rope[0].w, rope[1].x, rope[1].y, rope[1].z, rope[1].w};
        tmem_st8(kcol + 128 - half * 56, ro);  // (columns 128 + 8 half of the tile)
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->k_full[M::kHalves ? 1 : j & 1]);
      }
      const int jv = j - kLag;
      if (jv < 0) continue;
      // the V buffer is free once BMM2 of its last tile has completed
      if (jv >= 2) ok = mbar_wait(&ctrl->o_done[jv & 1], ((jv >> 1) - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        failed = true;
        break;
      }
      const uint32_t vrow = v_row + (jv & 1) * kVTile;
      const uint32_t from = k_lane + (jv % M::kKBufs) * kKCols;
      uint32_t o[2][32];
      tmem_ld32(from, o[0]);
      tmem_ld32(from + 32, o[1]);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const uint32_t* c = &o[q >> 3][4 * (q & 7)];
        st_shared_v4(vrow + (q >> 2) * kVBlock + (((q & 3) << 4) ^ sw), c[0], c[1], c[2], c[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->v_full[jv & 1]);
    }
    worker_failed = failed;
  } else {
    // ------------------------------------------------------------------ softmax: a key and RW rows per thread
    constexpr int RW = NR / 2;
    const int quad = warp & 3, r0 = (warp >> 2) * RW;  // rows r0 .. r0 + RW - 1 of the group
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int key_in = quad * 32 + lane;
    const int p0 = L - p.T;  // first draft
    float l_sum[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) l_sum[r] = 0.f;
    // this thread's bytes of P: hi of its RW rows, lo of them NR bytes further (under the key's swizzle)
    const uint32_t p_sw = NR == 16 ? ((key_in >> 2) & 1) << 4 : ((key_in >> 1) & 3) << 4;
    const uint32_t p_hi = smem_u32(smem + M::kOffP) + key_in * 2 * NR + (static_cast<uint32_t>(r0) ^ p_sw);
    const uint32_t p_lo = smem_u32(smem + M::kOffP) + key_in * 2 * NR + (static_cast<uint32_t>(NR + r0) ^ p_sw);
    bool failed = !mbar_wait(&ctrl->q_ready, 0, abort_flag);  // (the rows' factors and limits)
    float m = -INFINITY;  // reference maximum (log2 of the scaled score) of row `lane`, the same in every warp
    float peak = -INFINITY;  // the largest it has been
    int low_for = 0, low_needed = kLowTiles;  // tiles on end that row `lane` has been low for; as many as lower its reference
    const int half = lane < RW ? 0 : 1;  // of the rows
    const uint32_t mark = lane < NR ? row_mark(lane % RW) : 0u;
    const auto marks = [&](bool of_row) { return __reduce_or_sync(0xffffffffu, half == r0 / RW && of_row ? mark : 0u); };
    if (lane == 0) ctrl->low[1][warp] = 0;
    uint32_t sunk = 0;       // rows whose reference goes down at the next tile
    int third = 0;        // j % 3
    for (int j = 0; j < ntiles; ++j) {
      const int sb = j & 1;
      const int k0 = kv_start + j * kTile, key = k0 + key_in;
      const bool edge = k0 + kTile > min(kv_end, kTree ? p0 : p0 + 1);  // some key here is not every row's
      const uint32_t s_addr = tmem + lane_base + M::kS + sb * NR + r0;
      bool fail = failed || !mbar_wait(&ctrl->s_full[sb], (j >> 1) & 1, abort_flag);
      fail = __any_sync(0xffffffffu, fail);
      float x[RW];
      float alpha = 1.f;
      if (sunk != 0) {
        if ((sunk >> lane) & 1) {
          m -= kDrop;
          alpha = kDropFactor;
          ctrl->off[warp][lane] = kPShift - m;
        }
        __syncwarp();
      }
      auto sees = [&](int r) -> bool {  // (r within the group)
        if (key >= kv_end) return false;
        if (!kTree) return key <= ctrl->lim[r];
        const int u = key - p0;
        return ctrl->lim[r] >= 0 && (u < 0 || ((ctrl->drafts[r] >> u) & 1));
      };
      // x = score - reference + kPShift (log2); -infinity where a row does not see the key
      auto scores = [&]() {
        uint32_t s[RW];
        load_s<RW>(s_addr, s);
#pragma unroll
        for (int r = 0; r < RW; r += 4) {
          const float4 mu = *reinterpret_cast<const float4*>(&ctrl->mult[r0 + r]), of = *reinterpret_cast<const float4*>(&ctrl->off[warp][r0 + r]);
          x[r] = fmaf(__uint_as_float(s[r]), mu.x, of.x);
          x[r + 1] = fmaf(__uint_as_float(s[r + 1]), mu.y, of.y);
          x[r + 2] = fmaf(__uint_as_float(s[r + 2]), mu.z, of.z);
          x[r + 3] = fmaf(__uint_as_float(s[r + 3]), mu.w, of.w);
        }
        if (edge) {
#pragma unroll
          for (int r = 0; r < RW; ++r)
            if (!sees(r0 + r)) x[r] = -INFINITY;
        }
      };
      // every row's largest score here into top[third]: all rows at once, by halves (0.2 us where a reduction for each row that
      // needs it took 1.0 for the first tile's 16)
      auto tops = [&]() {
        uint32_t s[RW];
        load_s<RW>(s_addr, s);
        float top_of[RW];
#pragma unroll
        for (int r = 0; r < RW; r += 4) {
          const float4 mu = *reinterpret_cast<const float4*>(&ctrl->mult[r0 + r]);
          top_of[r] = x[r] == -INFINITY ? -INFINITY : __uint_as_float(s[r]) * mu.x;
          top_of[r + 1] = x[r + 1] == -INFINITY ? -INFINITY : __uint_as_float(s[r + 1]) * mu.y;
          top_of[r + 2] = x[r + 2] == -INFINITY ? -INFINITY : __uint_as_float(s[r + 2]) * mu.z;
          top_of[r + 3] = x[r + 3] == -INFINITY ? -INFINITY : __uint_as_float(s[r + 3]) * mu.w;
        }
        const int i = __float_as_int(lanes_reduce<RW, true>(top_of, lane));
        if (lane % (32 / RW) == 0) atomicMax(&ctrl->top[third][r0 + lane / (32 / RW)], i ^ ((i >> 31) & 0x7fffffff));
      };
      bool over = false;  // (warp-uniform) some row outgrew its reference here
      if (!fail) {
        tc_fence_after();
        scores();
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < RW; ++r) top = fmaxf(top, x[r]);
        over = __any_sync(0xffffffffu, top > kPShift + kThreshold);
        if (over) {
          tops();
        }
      }
      // one vote a tile; ordinary tiles reduce nothing else across threads
      uint32_t moved = sunk;
      if (bar_or(1, kSoftmaxThreads, fail || over || *abort_flag != 0)) {
        if (bar_or(1, kSoftmaxThreads, fail || *abort_flag != 0)) {
          failed = true;
          break;
        }
        // ---------------------------------------------------------------- some rows' references move
        bool first = false;  // the row's first keys
        if (lane < NR) {
          int i = ctrl->top[third][lane];
          i ^= (i >> 31) & 0x7fffffff;
          const float best = __int_as_float(i);
          float to = m;
          first = m == -INFINITY && best != -INFINITY;
          if (m == -INFINITY)
            to = best + kMargin;
          else if (best > m)  // (where one row has to move, those that need not yet go along: 114.0 -> 112.4 us)
            to = best + (best > m + kFar ? kFarMargin : kMargin);
          if (to > m && m < peak) low_needed = min(2 * low_needed, kMostLowTiles);
          if (m != -INFINITY && to != m) alpha *= ex2_approx(m - to);
          m = to;
          peak = fmaxf(peak, m);
          if (i != __float_as_int(-INFINITY)) ctrl->off[warp][lane] = kPShift - m;
        }
        moved = __ballot_sync(0xffffffffu, alpha != 1.f);
        __syncwarp();
        scores();
        // First keys of which one stands alone: so far above 32 others, one warp's, that its weight may go up to the largest
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        if (firsts != 0) {  // (the same in all warps)
          uint32_t far = 0, seen = 0;
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            far |= x[r] >= -2.f ? row_mark(r) : 0u;
            seen |= x[r] != -INFINITY ? row_mark(r) : 0u;  // (keys that a row does not see leave none alone)
          }
          far = __reduce_or_sync(0xffffffffu, far), seen = __reduce_or_sync(0xffffffffu, seen);
          if (lane == 0) ctrl->alone[warp] = seen & ~far;
          named_bar_sync(1, kSoftmaxThreads);
          const uint4 by = *reinterpret_cast<const uint4*>(&ctrl->alone[4 * half]);
          const bool alone = first && ((by.x | by.y | by.z | by.w) & mark) != 0;
          if (__any_sync(0xffffffffu, alone)) {  // (the same in all warps)
            if (alone) {
              m += kFarMargin - kMargin;
              peak = m;
              ctrl->off[warp][lane] = kPShift - m;
            }
            __syncwarp();
            scores();
          }
        }
      }
      // the rows that lay far below their reference throughout the last tile: all warps' marks are there since the vote, and all
      // warps find the same
      const uint4 low_by = *reinterpret_cast<const uint4*>(&ctrl->low[sb ^ 1][4 * half]);
      if (warp == 0 && lane < NR) ctrl->top[third == 0 ? 2 : third - 1][lane] = kNoScore;  // (the last tile's: all have read it)
      third = third == 2 ? 0 : third + 1;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->s_free[sb]);
      if (moved != 0) {
        // what the moved rows have accumulated, once BMM2 of the last tile has completed: their sums, and their columns of
        // O, hi and lo of two chunks a warp
#pragma unroll
        for (int r = 0; r < RW; ++r)
          if ((moved >> (r0 + r)) & 1) l_sum[r] *= __shfl_sync(0xffffffffu, alpha, r0 + r);
        const bool ok = mbar_wait(&ctrl->o_done[sb ^ 1], ((j - 1) >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) failed = true;  // (the others learn of it at the next vote)
        tc_fence_after();
        for (uint32_t left = failed ? 0u : moved; left != 0; left &= left - 1) {
          const int r = __ffs(left) - 1;
          const float f = __shfl_sync(0xffffffffu, alpha, r);
          const uint32_t at = tmem + lane_base + M::kO + (warp >> 2) * 4 * NR + r;
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld1(at + k * NR, v[k]);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_st1(at + k * NR, __float_as_uint(__uint_as_float(v[k]) * f));
        }
        tmem_st_wait();
      }
      if (j >= 2) {  // this P buffer's last reader
        const bool ok = mbar_wait(&ctrl->o_done[sb], ((j >> 1) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) failed = true;  // (the others learn of it at the next vote)
      }
      uint32_t hi4[RW / 4], lo4[RW / 4];
#pragma unroll
      for (int r = 0; r < RW; r += 2) {
        const float a = ex2_approx(x[r]), c = ex2_approx(x[r + 1]);
        l_sum[r] += a;
        l_sum[r + 1] += c;
        const uint32_t ph = pack_f16x2(a, c);
        const uint32_t hi = f16x2_to_e4m3x2(ph);
        const uint32_t hb = e4m3x2_to_f16x2(hi);
        uint32_t d;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(ph), "r"(hb));  // (exact)
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(d), "r"(0x4F004F00u));  // times 28
        const uint32_t lo = f16x2_to_e4m3x2(d);
        hi4[r >> 2] = (r & 2) ? __byte_perm(hi4[r >> 2], hi, 0x5410) : hi;
        lo4[r >> 2] = (r & 2) ? __byte_perm(lo4[r >> 2], lo, 0x5410) : lo;
      }
      const uint32_t pb = sb * M::kPBuf;
      if constexpr (RW == 8) {
        st_shared_v2(p_hi + pb, hi4[0], hi4[1]);
        st_shared_v2(p_lo + pb, lo4[0], lo4[1]);
      } else {
        st_shared_v4(p_hi + pb, hi4[0], hi4[1], hi4[2], hi4[3]);
        st_shared_v4(p_lo + pb, lo4[0], lo4[1], lo4[2], lo4[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->p_full[sb]);
      uint32_t low = low_rows(hi4);
      if (edge && !kTree) low &= marks(ctrl->lim[lane % NR] >= k0);  // (rows that see none of these keys stay)
      if (lane == 0) ctrl->low[sb][warp] = low;
      low_for = (low_by.x & low_by.y & low_by.z & low_by.w & mark) != 0 && !((moved >> lane) & 1) ? low_for + 1 : 0;
      sunk = __ballot_sync(0xffffffffu, low_for >= low_needed && m > peak - kDepth);
    }
    const float ls = lanes_reduce<RW>(l_sum, lane);
    if (lane % (32 / RW) == 0) ctrl->sums[quad][r0 + lane / (32 / RW)] = ls;
    named_bar_sync(1, kSoftmaxThreads);
    if (warp == 0 && lane < NR) {
      const float s = (ctrl->sums[0][lane] + ctrl->sums[1][lane]) + (ctrl->sums[2][lane] + ctrl->sums[3][lane]);
      // (a row that sees nothing has a sum of 0; a NaN goes on)
      ctrl->row_scale[lane] = s != 0.f ? (final_out ? p.v_scale : 1.f) / s : 0.f;
      ctrl->lse[lane] = s != 0.f ? (m + __log2f(s) - kPShift) * 0.69314718055994530942f : -INFINITY;
    }
    if (!failed) failed = !mbar_wait(&ctrl->o_done[(ntiles - 1) & 1], ((ntiles - 1) >> 1) & 1, abort_flag);
    worker_failed = failed;
  }
  if (warp < kSoftmaxWarps + kDecodeWarps) {
    // ------------------------------------------------------------------ output: a chunk of 128 value columns a warp
    if (!bar_or(2, kWorkers, worker_failed || *abort_flag != 0)) {
      tc_fence_after();
      const int quad = warp & 3, qc = warp >> 2, col = qc * 128 + quad * 32 + lane;
      uint16_t* dst = reinterpret_cast<uint16_t*>(
          final_out ? p.out + (static_cast<int64_t>(b) * p.R + row0) * kValueDim
                    : p.ws_o + ((static_cast<int64_t>(b) * p.max_splits + split) * p.R + row0) * kValueDim);
      const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + M::kO + qc * 2 * NR;
      const bool odd = lane & 1;
      const auto store = [&](auto final_rows) {
        uint32_t hi[NR], lo[NR];
        if constexpr (NR == 16) {
          tmem_ld16(at, hi);
          tmem_ld16(at + NR, lo);
        } else {
          tmem_ld32(at, hi);
          tmem_ld32(at + NR, lo);
        }
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          // two rows: even lanes store two columns of the first, odd lanes of the second (through shared memory in rows,
          // this took 0.9 us more at 32 rows)
          // (a split's partial is f16 in units of the codes, at most 384; the combine scales it)
          const float2 scale = *reinterpret_cast<const float2*>(&ctrl->row_scale[r]);
          const float v0 = (__uint_as_float(hi[r]) + __uint_as_float(lo[r]) * (1.f / kLoScale)) * scale.x;
          const float v1 = (__uint_as_float(hi[r + 1]) + __uint_as_float(lo[r + 1]) * (1.f / kLoScale)) * scale.y;
          const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
          const float left = odd ? other : v0, right = odd ? v1 : other;
          const int row = r + (odd ? 1 : 0);
          if (row < nrows)
            *reinterpret_cast<uint32_t*>(dst + row * kValueDim + (col & ~1)) = final_rows.value ? pack_bf16x2(left, right) : pack_f16x2(left, right);
        }
      };
      if (final_out)
        store(std::true_type{});
      else
        store(std::false_type{});
      if (warp == 0 && lane < nrows) {
        if (final_out)
          p.lse[static_cast<int64_t>(b) * p.R + row0 + lane] = ctrl->lse[lane];
        else
          p.ws_lse[(static_cast<int64_t>(b) * p.max_splits + split) * p.R + row0 + lane] = ctrl->lse[lane];
      }
    }
  }

  tc_fence_before();
  __syncthreads();
}

// The splits item, item + stride, ... of a batch that has more of them than the grid has CTAs: rare, and out of line so that
// the first split is not compiled into a loop (7 % of a long call, as a call 4 %).
template <int NR, bool kTree>
__device__ __noinline__ void take_more_splits(const CUtensorMap* tm_kv, const DecodeParams* p, uint8_t* smem, int group, int item, int stride) {
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + Map<NR>::kOffCtrl);
  for (; item < ctrl->item[3] && !*static_cast<volatile int*>(&ctrl->abort_flag); item += stride) {  // (the same for all threads)
    __syncthreads();  // (item[3] and the flag are read)
    if (threadIdx.x == 0) {
      for (uint64_t* bar = ctrl->raw_full; bar <= &ctrl->drain; ++bar) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
      init_barriers<NR>(ctrl);
    }
    find_split(*p, item, false, ctrl);
    tc_fence_after();
    take_split<NR, kTree>(*tm_kv, *p, smem, group, ctrl->item[0], ctrl->item[1], ctrl->item[2]);
  }
}

// kMore: the grid has a CTA for each planned split, and should the lengths give more, CTAs take several; else it has one for
// each split that the lengths can give.
template <int NR, bool kTree, bool kMore>
__global__ void __launch_bounds__(kThreads, 1) decode_partial_fp4_kernel(const __grid_constant__ CUtensorMap tm_kv,
                                                                         const __grid_constant__ DecodeParams p) {
  using M = Map<NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + M::kOffCtrl);
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    init_barriers<NR>(ctrl);
    ctrl->abort_flag = 0;
  }
  if (threadIdx.x == 32 * kProducerWarp) tma_prefetch_desc(&tm_kv);
  if (warp == kMmaWarp) {
    tmem_alloc(&ctrl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // programmatic dependent launch: no input is read before the previous kernel has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (p.part_scale && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) *p.part_scale = p.v_scale;
  // Which split this CTA takes: whole splits first, then the remainders (split_major 2), split by split (1) or
  // request by request (0).  Splits that a request does not have come last in the first order and end at once: in
  // the others they hold up the CTAs behind them, which measured 24 us on 16 requests of 8K-131K keys.
  const int groups = (p.R + NR - 1) / NR;
  const bool listed = p.split_major == 2;
  int group = blockIdx.x, b = p.split_major ? blockIdx.y : blockIdx.z, split = p.split_major ? blockIdx.z : blockIdx.y;
  if (listed) {
    group = blockIdx.x % groups;
    find_split(p, blockIdx.x / groups, blockIdx.x == 0, ctrl);
    b = ctrl->item[0], split = ctrl->item[1];
  }
  const int L = b < 0 ? 0 : listed ? ctrl->item[2] : p.seq_lens[b];
  const bool bad_len = L < p.T || L > p.max_seq || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_pages) * p.page_size;
  if (!listed && bad_len && threadIdx.x == 0 && split == 0 && group == 0) atomicOr(p.status, kStatusDeviceArg);
  if (b >= 0 && !bad_len && split * p.chunk < L) {  // (CTA-uniform) else there is no such split
    take_split<NR, kTree>(tm_kv, p, smem, group, b, split, L);
    if (kMore && listed && ctrl->item[3] > static_cast<int>(gridDim.x) / groups)
      take_more_splits<NR, kTree>(&tm_kv, &p, smem, group, (blockIdx.x + gridDim.x) / groups, gridDim.x / groups);
    if (threadIdx.x == 0 && *static_cast<volatile int*>(&ctrl->abort_flag) == kAbortTimeout) atomicOr(p.status, kStatusTimeout);
    // every store of this CTA is issued: the combine grid may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(ctrl->tmem_base, kTmemCols);
  }
}

}  // namespace

int fp4_group_rows(int R) { return R <= 16 ? 16 : 32; }

cudaError_t launch_decode_partial_fp4(const DecodeParams& p, const CUtensorMap& tm_kv, cudaStream_t stream) {
  // [32 rows][tree][more]
  static constexpr decltype(&decode_partial_fp4_kernel<16, false, false>) kernels[8] = {
      decode_partial_fp4_kernel<16, false, false>, decode_partial_fp4_kernel<16, false, true>,
      decode_partial_fp4_kernel<16, true, false>,  decode_partial_fp4_kernel<16, true, true>,
      decode_partial_fp4_kernel<32, false, false>, decode_partial_fp4_kernel<32, false, true>,
      decode_partial_fp4_kernel<32, true, false>,  decode_partial_fp4_kernel<32, true, true>};
  static constexpr int smem[2] = {Map<16>::kSmem, Map<32>::kSmem};
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    for (int i = 0; i < 8; ++i) {
      e = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem[i / 4]);
      if (e != cudaSuccess) return e;
    }
    configured_device = dev;
  }
  const int rows = fp4_group_rows(p.R), wide = rows == 32 ? 1 : 0;
  const int groups = (p.R + rows - 1) / rows;
  cudaLaunchConfig_t cfg = {};
  // A CTA for every split that the lengths can give, or, where that is many more than were planned, for the planned ones.
  // An empty CTA takes an SM 1-3 us: one request of 131K keys and 127 of 500 took 256 us with 9472 CTAs, 35 with the
  // planned 201; but a kernel that takes several splits is 4 % slower (88.0 against 91.7 us on 16 requests of 8K-131K keys,
  // 288 CTAs of which 160 are planned).
  const int64_t most = static_cast<int64_t>(p.B) * p.max_splits;
  const bool more = p.split_major == 2 && p.num_splits > 0 && groups * (most - p.num_splits) > kMostEmpty;
  const int64_t listed = more ? std::min<int64_t>(p.num_splits, 0x7fffffff / groups) : most;
  if (p.split_major == 2 && (groups * listed > 0x7fffffff || p.B > kThreads)) return cudaErrorInvalidConfiguration;
  cfg.gridDim = p.split_major == 2   ? dim3(static_cast<unsigned>(groups * listed))
                : p.split_major == 1 ? dim3(groups, p.B, p.max_splits)
                                     : dim3(groups, p.max_splits, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem[wide];
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernels[4 * wide + (p.tree_mask ? 2 : 0) + (more ? 1 : 0)], tm_kv, p);
}

}  // namespace mla
