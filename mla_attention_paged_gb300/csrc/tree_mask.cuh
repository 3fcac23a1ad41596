// tree_mask.cuh -- what the decode kernels share for trees of drafted tokens: which keys of a
// 64-key tile a row sees, and draft rows made safe to multiply by a zero weight.
#pragma once

#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {

// Keys of the tile k0 .. k0 + 63 that a row sees, as a bit per key: every key before the
// first draft (position p0), and draft u where bit u of `mask` (cut to the T drafts) is set.
__device__ __forceinline__ uint64_t tree_tile_bits(uint64_t mask, int p0, int k0) {
  const int d = p0 - k0;  // prefix keys in (or past) this tile
  if (d >= 64) return ~0ull;
  if (d > 0) return ((1ull << d) - 1) | (mask << d);
  return d > -64 ? mask >> (-d) : 0ull;
}

// The T low bits.
__device__ __forceinline__ uint64_t draft_bits(int T) { return T >= 64 ? ~0ull : (1ull << T) - 1; }

// An output value as the bits it is staged in: bf16, or f16 for a split partial of a tree
// (an 8-bit pool's, in units of its codes).
template <bool kTree>
__device__ __forceinline__ uint32_t out_bits(float v, bool final_out) {
  if (kTree && !final_out) return __half_as_ushort(__float2half_rn(v));
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// bf16 pairs with infinities and NaNs replaced by zero.  A draft that a row does not see
// has weight 0 there, but 0 times an infinity or NaN is NaN.  Rows that do see it have a score
// that is not finite: NaN or +infinity makes the whole row NaN without its values; -infinity
// is a weight of 0, and pass_on_not_finite gives such rows the NaNs of 0 times infinity.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

// e4m3 codes (four in a word) with the NaN codes 0x7F and 0xFF replaced by zero.
__device__ __forceinline__ uint32_t finite_e4m3x4(uint32_t w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((w >> (8 * i)) & 0x7Fu) == 0x7Fu) w &= ~(0xFFu << (8 * i));
  return w;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(saddr));
  return v;
}

// Rewrite a 16-byte piece of a draft's value row without infinities or NaNs.
template <bool kE4m3>
__device__ __forceinline__ void make_finite(uint32_t saddr) {
  const uint4 v = ld_shared_v4(saddr);
  uint4 f;
  f.x = kE4m3 ? finite_e4m3x4(v.x) : finite_bf16x2(v.x);
  f.y = kE4m3 ? finite_e4m3x4(v.y) : finite_bf16x2(v.y);
  f.z = kE4m3 ? finite_e4m3x4(v.z) : finite_bf16x2(v.z);
  f.w = kE4m3 ? finite_e4m3x4(v.w) : finite_bf16x2(v.w);
  if ((f.x ^ v.x) | (f.y ^ v.y) | (f.z ^ v.z) | (f.w ^ v.w)) st_shared_v4(saddr, f.x, f.y, f.z, f.w);
}

// A 32-bit word of keys first .. first + 31 of a request as a word of its drafts (p0: the first one).
__device__ __forceinline__ uint64_t draft_word(uint32_t keys, int first, int p0) {
  const int d = p0 - first;  // (below 64 for keys that may be drafts)
  return d >= 0 ? static_cast<uint64_t>(keys) >> d : static_cast<uint64_t>(keys) << -d;
}

// Staged output rows (a row's 512 columns `pitch` bytes from the last one's, fp32 or bf16) become
// NaN in the columns in which a draft of `lost` that they see holds an infinity or NaN in the
// bf16 pool.  lost: the drafts that some row sees with a score of -infinity.  For all threads
// 0 .. kThreads - 1, between barriers.
template <int kThreads>
__device__ __noinline__ void pass_on_not_finite(uint64_t lost, const uint8_t* pool, int64_t num_pages, int page_size,
                                                const int32_t* pages, int p0, const uint64_t* masks, int row0, int nrows,
                                                int heads, uint32_t stage, int pitch, bool fp32) {
  for (; lost != 0; lost &= lost - 1) {
    const int u = __ffsll(static_cast<long long>(lost)) - 1, j = p0 + u;
    const int64_t pid = __ldg(pages + j / page_size);
    if (pid < 0 || pid >= num_pages) continue;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(pool) + (pid * page_size + j % page_size) * (kLatentDim / 2);
    for (int c = threadIdx.x; c < kValueDim / 2; c += kThreads) {
      const uint32_t w = __ldg(row + c), gone = w ^ finite_bf16x2(w);
      if (gone == 0) continue;
      for (int r = 0; r < nrows; ++r) {
        if (!((masks[(row0 + r) / heads] >> u) & 1)) continue;
        const uint32_t at = stage + r * pitch + c * (fp32 ? 8 : 4);
        if (gone & 0xFFFFu) fp32 ? st_shared_f32(at, NAN) : st_shared_u16(at, 0x7FFFu);
        if (gone >> 16) fp32 ? st_shared_f32(at + 4, NAN) : st_shared_u16(at + 2, 0x7FFFu);
      }
    }
  }
}

}  // namespace mla
