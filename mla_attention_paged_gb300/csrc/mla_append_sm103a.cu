// mla_append_sm103a.cu -- one pass that prepares a step's queries and latent keys and writes
// the keys into the paged latent cache, sm_103a.
//
// What it computes, per token n with position x = positions[n]:
//   key:   c = kv[n, :512];  c' = c / sqrt(mean(c^2) + eps) * kv_weight   (no weight: c' = c)
//          r' = rot(kv[n, 512:576], x);  row = [c', r'] into slot slots[n] of the pool
//   query: every head h: v = q[n, h, :];  v' = v / sqrt(mean(v^2) + eps) * q_weight (no
//          weight: v' = v), then the last 64 columns rotated: q_out[n, h, :]
//   rot: pair i of 32 is (2i, 2i+1) interleaved or (i, i+32) half-split;
//        (a, b) -> (a cos - b sin, b cos + a sin) with cos/sin of row x of the table.
// Everything is held in fp32 from the load to the one rounding at the store (bf16, or the
// value over kv_scale rounded to the nearest e4m3 or int8 code, saturated).
//
// Bound by memory: each input is read once and each output written once.  Eight lanes share a
// row (a head's query or a token's key) and hold it in registers, 16-byte chunk l, l + 8, ... in
// lane l, so the norm is three shuffles and nothing passes through shared memory.  The 64
// rotated columns are one chunk per lane, which puts the two chunks of a half-split pair in
// lanes that differ in bit 2.  A warp takes four rows at a time: for queries four heads of one
// token, kSteps times with all loads in flight, so positions, cosines and weights are read once
// per warp; keys 16 lanes a row.  (A warp per row, two loads in flight, took 72 us where this
// takes 22.8 for 8191 tokens of 16 normed 192-wide heads and their keys: 5.3 TB/s.)
#include <cuda_fp8.h>

#include <type_traits>

#include "fp4_rows.cuh"
#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

constexpr int kRope = 64;
constexpr int kWarps = 4;
constexpr int kManySteps = 2;
constexpr int kManySteps64 = 4;  // heads of the 64 rotated columns alone: 128 bytes a step
constexpr int kManyKeyLanes = 16;
constexpr int64_t kFewRows = 12288;
constexpr int64_t kOneWave = 152 * 28;  // warps of two steps: seven CTAs an SM

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float sum_sq(const float (&f)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  return s;
}

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A lane's cosines and sines: interleaved, pairs 4l .. 4l+3 of its chunk l; half-split, pairs
// 8 (l % 4) .. + 7.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void load_turn(Turn& t, const float* cs, int l, bool interleaved) {
  const float4* cp = reinterpret_cast<const float4*>(cs) + (interleaved ? l : 2 * (l & 3));
  const float4 c0 = __ldg(cp), s0 = __ldg(cp + 8);
  const float4 c1 = interleaved ? c0 : __ldg(cp + 1), s1 = interleaved ? s0 : __ldg(cp + 9);
  t.c[0] = c0.x, t.c[1] = c0.y, t.c[2] = c0.z, t.c[3] = c0.w, t.c[4] = c1.x, t.c[5] = c1.y, t.c[6] = c1.z, t.c[7] = c1.w;
  t.s[0] = s0.x, t.s[1] = s0.y, t.s[2] = s0.z, t.s[3] = s0.w, t.s[4] = s1.x, t.s[5] = s1.y, t.s[6] = s1.z, t.s[7] = s1.w;
}

__device__ __forceinline__ void rotate(float (&f)[8], const Turn& t, int l, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = a * t.c[i] - b * t.s[i];
      f[2 * i + 1] = b * t.c[i] + a * t.s[i];
    }
  } else {
    const float sign = l < 4 ? -1.f : 1.f;  // first half: a cos - b sin; second: b cos + a sin
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
      f[i] = f[i] * t.c[i] + sign * (other * t.s[i]);
    }
  }
}

// rotate, each product and sum rounded by itself.
__device__ __forceinline__ void rotate_exact(float (&f)[8], const Turn& t, int l, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
      f[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
      const float x = __fmul_rn(f[i], t.c[i]), y = __fmul_rn(other, t.s[i]);
      f[i] = l < 4 ? __fsub_rn(x, y) : __fadd_rn(x, y);
    }
  }
}

// A sum and the error of its rounding (exact after each addition: the two-sum of Knuth, The Art of Computer
// Programming, volume 2, 4.2.2; errors themselves are summed plainly).
struct Sum {
  float hi, lo;
};

__device__ __forceinline__ Sum add(const Sum& s, float x) {
  const float t = __fadd_rn(s.hi, x), u = __fsub_rn(t, s.hi);
  const float err = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, u)), __fsub_rn(x, u));
  return {t, __fadd_rn(s.lo, err)};
}

__device__ __forceinline__ void scale8(float (&f)[8], float inv, const uint4& w) {
  float g[8];
  unpack8(w, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * g[i];
}

// Eight values as 8-bit codes of x / scale.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale, bool int8) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u = 0;
    if (int8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = __fdiv_rn(f[4 * h + i], scale);
        // NaN encodes as 0 (int8 has no code for it)
        const int c = x != x ? 0 : static_cast<int>(rintf(fminf(fmaxf(x, -127.f), 127.f)));
        u |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = make_float2(__fdiv_rn(f[4 * h + 2 * i], scale), __fdiv_rn(f[4 * h + 2 * i + 1], scale));
        u |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) << (16 * i);
      }
    }
    w[h] = u;
  }
  return make_uint2(w[0], w[1]);
}

// kChunks: most chunks of a query lane that are not rotated, ceil((q_dim - 64) / 64).
// kSteps: four heads a step.  kKeyLanes: lanes that share a key's row.  Five CTAs an SM (96
// registers) measured 22.8 us on 8191 tokens of 16 normed 192-wide heads against 25.0 at four and
// 29 spilling at six; streaming loads and stores (nothing is read again) 24.6 against 26.8.
// The first k_warps warps of the grid take keys, the others queries.
// A 4-bit row (kFp4) is written to the bit of the plain formula, since a code of four bits may hang on the last bit of
// the norm: the squares (exact) are summed with their rounding errors, and the rotation uses no fused multiply-adds.
template <int kChunks, int kSteps, int kKeyLanes, bool kFp4>
__global__ void __launch_bounds__(32 * kWarps, kChunks == 0 && kSteps > 1 ? 6 : kChunks <= 2 ? 5 : 1) kv_append_kernel(const AppendParams p, int64_t k_warps, int warps_per_token) {
  // programmatic dependent launch: no input is read before the previous kernel has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, sub = lane >> 3, l = lane & 7;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const bool inter = p.interleaved != 0;
  if (unit >= k_warps) {
    // ------------------------------------------------------------------ queries of one token
    if (unit - k_warps >= static_cast<int64_t>(p.tokens) * warps_per_token) return;
    const int n = static_cast<int>((unit - k_warps) / warps_per_token);
    const int h0 = static_cast<int>((unit - k_warps) % warps_per_token) * 4 * kSteps + sub;
    const int pos = __ldg(p.positions + n);  // (checked once the rows' loads are in flight)
    const int chunks = (p.q_dim - kRope) / 8;
    const __nv_bfloat16* src = p.q_in + static_cast<int64_t>(n) * p.q_in_token;
    __nv_bfloat16* dst = p.q_out + static_cast<int64_t>(n) * p.q_out_token;
    // (wide rows go one step at a time: their chunks fill the registers)
    constexpr int kTogether = kChunks <= 2 ? kSteps : 1;
    Turn turn;
    uint4 wt[kChunks + 1];
#pragma unroll 1
    for (int s0 = 0; s0 < kSteps; s0 += kTogether) {
      uint4 w[kTogether][kChunks + 1];
#pragma unroll
      for (int s = 0; s < kTogether; ++s) {
        const int h = h0 + 4 * (s0 + s);
        const uint4* row = reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * p.q_in_head);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          w[s][i] = h < p.heads && l + 8 * i < chunks ? __ldcs(row + l + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        w[s][kChunks] = h < p.heads ? __ldcs(row + chunks + l) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (s0 == 0) {
        if (static_cast<unsigned>(pos) >= static_cast<unsigned>(p.max_positions)) {
          if (lane == 0) atomicOr(p.status, kStatusDeviceArg);
          return;
        }
        load_turn(turn, p.cos_sin + static_cast<int64_t>(pos) * kRope, l, inter);
        if (p.q_weight) {
          const uint4* g = reinterpret_cast<const uint4*>(p.q_weight);
#pragma unroll
          for (int i = 0; i < kChunks; ++i) wt[i] = l + 8 * i < chunks ? __ldg(g + l + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
          wt[kChunks] = __ldg(g + chunks + l);
        }
      }
#pragma unroll
      for (int s = 0; s < kTogether; ++s) {
        const int h = h0 + 4 * (s0 + s);
        float f[kChunks + 1][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i <= kChunks; ++i) {
          unpack8(w[s][i], f[i]);
          ss += sum_sq(f[i]);
        }
        if (p.q_weight) {
          const float inv = 1.f / sqrtf(row_sum<8>(ss) / static_cast<float>(p.q_dim) + p.eps);
#pragma unroll
          for (int i = 0; i <= kChunks; ++i) scale8(f[i], inv, wt[i]);
        }
        rotate(f[kChunks], turn, l, inter);
        if (h < p.heads) {
          uint4* out = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(h) * p.q_out_head);
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            if (l + 8 * i < chunks) __stcs(out + l + 8 * i, pack8(f[i]));
          __stcs(out + chunks + l, pack8(f[kChunks]));
        }
      }
    }
    return;
  }
  // -------------------------------------------------------------------- keys, kKeyLanes a row
  constexpr int kLatentChunks = kValueDim / 8 / kKeyLanes;  // per lane; lanes 0-7 also rotate one
  const int kl = lane % kKeyLanes;
  const int64_t n = unit * (32 / kKeyLanes) + lane / kKeyLanes;
  const bool real = n < p.tokens;
  int64_t slot = real ? __ldg(p.slots + n) : -1;  // (negative: a padded token has no place in the cache)
  const int pos = real ? __ldg(p.positions + n) : 0;
  uint4 w[kLatentChunks + 1];
  const uint4* row = reinterpret_cast<const uint4*>(p.kv_in + n * p.kv_in_token);
#pragma unroll
  for (int i = 0; i < kLatentChunks; ++i) w[i] = real ? __ldcs(row + kl + kKeyLanes * i) : make_uint4(0u, 0u, 0u, 0u);
  w[kLatentChunks] = real && kl < 8 ? __ldcs(row + kValueDim / 8 + kl) : make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0 && (slot >= p.num_slots || static_cast<unsigned>(pos) >= static_cast<unsigned>(p.max_positions))) {
    if (kl == 0) atomicOr(p.status, kStatusDeviceArg);
    slot = -1;
  }
  const bool live = slot >= 0;  // (the others still take part in the shuffles)
  Turn turn;
  load_turn(turn, p.cos_sin + (live ? static_cast<int64_t>(pos) * kRope : 0), l, inter);
  float inv = 1.f;
  if (kFp4 && p.kv_weight) {
    // (a chain of its own for every chunk: each addition waits for the one before it)
    Sum part[kLatentChunks];
#pragma unroll
    for (int i = 0; i < kLatentChunks; ++i) {
      float f[8];
      unpack8(w[i], f);
      part[i] = {f[0] * f[0], 0.f};
#pragma unroll
      for (int k = 1; k < 8; ++k) part[i] = add(part[i], f[k] * f[k]);
    }
    Sum ss = part[0];
#pragma unroll
    for (int i = 1; i < kLatentChunks; ++i) {
      ss = add(ss, part[i].hi);
      ss.lo += part[i].lo;
    }
#pragma unroll
    for (int o = kKeyLanes / 2; o > 0; o >>= 1) {
      const Sum other = {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)};
      ss = add(ss, other.hi);
      ss.lo += other.lo;
    }
    inv = 1.f / sqrtf((ss.hi + ss.lo) / static_cast<float>(kValueDim) + p.eps);
    inv = __shfl_sync(0xffffffffu, inv, 0, kKeyLanes);  // (one lane's, whatever the order of the errors' sum)
  } else if (p.kv_weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kLatentChunks; ++i) {
      float f[8];
      unpack8(w[i], f);
      ss += sum_sq(f);
    }
    inv = 1.f / sqrtf(row_sum<kKeyLanes>(ss) / static_cast<float>(kValueDim) + p.eps);
  }
#pragma unroll
  for (int i = 0; i <= kLatentChunks; ++i) {
    const int c = i < kLatentChunks ? kl + kKeyLanes * i : kValueDim / 8 + kl;
    float f[8];
    unpack8(w[i], f);
    if (i == kLatentChunks) {
      if (kFp4)
        rotate_exact(f, turn, l, inter);
      else
        rotate(f, turn, l, inter);
    } else if (p.kv_weight) {
      scale8(f, inv, __ldg(reinterpret_cast<const uint4*>(p.kv_weight) + c));
    }
    if constexpr (kFp4) {
      // values over kv_scale; 16 columns, two lanes', share an exponent, and four lanes' two exponents a byte
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] *= p.kv_scale;  // (1 / kv_scale)
        if (i < kLatentChunks && f[k] != f[k]) f[k] = 0.f;  // (no code for a NaN)
        top = fmaxf(top, fabsf(f[k]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const int e = fp4_exponent(top), next = __shfl_xor_sync(0xffffffffu, e, 2);
      if (!live) continue;
      uint8_t* at = p.kv_pages + slot * kFp4RowBytes;
      if (i < kLatentChunks) {
        reinterpret_cast<uint32_t*>(at)[c] = fp4_encode8(f, e);
        if ((c & 3) == 0) at[kFp4ExpAt + c / 4] = static_cast<uint8_t>(e | (next << 4));
      } else if (kl < 8) {
        reinterpret_cast<uint2*>(at + kFp4RopeAt)[kl] = codes8(f, 1.f, false);
      }
      continue;
    }
    if (!live || (i == kLatentChunks && kl >= 8)) continue;
    const int64_t at = slot * (kLatentDim / 8) + c;
    if (p.kv_dtype == kKvBf16)
      reinterpret_cast<uint4*>(p.kv_pages)[at] = pack8(f);
    else
      reinterpret_cast<uint2*>(p.kv_pages)[at] = codes8(f, p.kv_scale, p.kv_dtype == kKvInt8);
  }
}

template <int kChunks>
cudaError_t launch_chunks(const AppendParams& p, cudaStream_t stream) {
  // Few rows: one step and a warp per key, for the shortest chain; many: more bytes in flight per
  // warp.  GPU us, few against many, by tokens x heads: 16 heads of 192 normed columns 2.8 / 3.1 at
  // 8192, 4.2 / 3.6 at 12288, 4.7 / 4.3 at 16384, 11.6 / 10.1 at 49152; 64 columns 2.4 / 2.8, 2.5 / 2.9,
  // 2.6 / 3.1, 6.1 / 5.3; 8 heads of 576 normed 7.9 / 6.9, 10.7 / 8.9, 13.0 / 11.2, 36.7 / 27.4.  (Wide
  // rows cross at about 9000, 64 columns at about 20000: one border between them for all.)
  const bool few = static_cast<int64_t>(p.tokens) * (p.heads > 0 ? p.heads : 16) <= kFewRows;
  const int key_rows = few ? 1 : 32 / kManyKeyLanes;
  const int64_t k_warps = p.kv_in ? (p.tokens + key_rows - 1) / key_rows : 0;
  // Rows of 64 columns alone take four steps where two would be more than one wave of warps, and where four leave no more
  // places of a token's last warp idle.  GPU us at two steps / four: 16 heads 1.96 / 2.07 at 1125 tokens, 2.33 / 2.32 at 1875,
  // 2.34 / 2.38 at 2125, 2.82 / 2.38 at 2375, 6.0 / 5.1 at 8192; 9 heads 2.07 / 2.08 at 2000, 2.68 / 2.17 at 2444; 20 heads
  // (24 places or 32) 2.33 / 2.46 at 1300, 3.89 / 3.82 at 3000; 16 heads with their keys 2.98 / 2.98 at 1625 tokens, 3.13 /
  // 3.06 at 1875, 8.6 / 7.7 at 8192.
  const int warps2 = (p.heads + 4 * kManySteps - 1) / (4 * kManySteps), warps4 = (p.heads + 4 * kManySteps64 - 1) / (4 * kManySteps64);
  const bool four = kChunks == 0 && p.heads > 4 * kManySteps && warps4 * kManySteps64 == warps2 * kManySteps &&
                    k_warps + static_cast<int64_t>(p.tokens) * warps2 > kOneWave;
  const int steps = few ? 1 : four ? kManySteps64 : kManySteps;
  const int per_token = (p.heads + 4 * steps - 1) / (4 * steps);
  const int64_t warps = k_warps + static_cast<int64_t>(p.tokens) * per_token;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  AppendParams q = p;
  if (p.kv_dtype == kKvFp4) q.kv_scale = 1.f / p.kv_scale;
  const auto go = [&](auto fp4) {
    if (few) return cudaLaunchKernelEx(&cfg, kv_append_kernel<kChunks, 1, 32, fp4.value>, q, k_warps, per_token);
    if constexpr (kChunks == 0)
      if (four) return cudaLaunchKernelEx(&cfg, kv_append_kernel<kChunks, kManySteps64, kManyKeyLanes, fp4.value>, q, k_warps, per_token);
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<kChunks, kManySteps, kManyKeyLanes, fp4.value>, q, k_warps, per_token);
  };
  return p.kv_dtype == kKvFp4 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const int chunks = p.q_in ? (p.q_dim - kRope + 63) / 64 : 0;
  if (chunks == 0) return launch_chunks<0>(p, stream);
  if (chunks <= 2) return launch_chunks<2>(p, stream);
  return launch_chunks<8>(p, stream);
}

}  // namespace mla
