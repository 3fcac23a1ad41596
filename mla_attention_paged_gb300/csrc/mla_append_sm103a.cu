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
// Bound by memory: each input is read once and each output written once.  One warp per
// (token, head) or per token's key; a lane holds 16-byte chunks (8 columns) in registers, so
// the norm is one shuffle reduction and nothing passes through shared memory.  The 64
// rotated columns always sit in lanes 24-31 (chunk k of 8 in lane 24 + k), which puts a
// half-split pair's two chunks in lanes that differ in bit 2.
#include <cuda_fp8.h>

#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

constexpr int kRope = 64;
constexpr int kWarps = 4;
constexpr int kRopeLane = 24;  // lanes 24-31 hold the rotated columns' eight chunks

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

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ void scale8(float (&f)[8], float inv, const __nv_bfloat16* w) {
  float g[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(w)), g);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * g[i];
}

// Rotate this lane's chunk k = lane - 24 (lanes 24-31; the others take part in the shuffles).
__device__ __forceinline__ void rotate(float (&f)[8], const float* cs, int lane, bool interleaved) {
  const int k = lane & 7;
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + k);
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + 32) + k);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = a * cc[i] - b * ss[i];
      f[2 * i + 1] = b * cc[i] + a * ss[i];
    }
  } else {
    const float4* cp = reinterpret_cast<const float4*>(cs) + 2 * (k & 3);
    const float4* sp = reinterpret_cast<const float4*>(cs + 32) + 2 * (k & 3);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    const float sign = k < 4 ? -1.f : 1.f;  // first half: a cos - b sin; second: b cos + a sin
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
      f[i] = f[i] * cc[i] + sign * (other * ss[i]);
    }
  }
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

__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const AppendParams p) {
  // programmatic dependent launch: no input is read before the previous kernel has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int per_token = p.heads + (p.kv_in ? 1 : 0);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= static_cast<int64_t>(p.tokens) * per_token) return;
  const int n = static_cast<int>(unit / per_token);
  const int h = static_cast<int>(unit % per_token);  // == heads: the token's key
  const int pos = __ldg(p.positions + n);
  const bool is_key = h == p.heads;
  int64_t slot = 0;
  if (is_key) {
    slot = __ldg(p.slots + n);
    if (slot < 0) return;  // a padded token has no place in the cache
  }
  if (static_cast<unsigned>(pos) >= static_cast<unsigned>(p.max_positions) || (is_key && slot >= p.num_slots)) {
    if (lane == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const float* cs = p.cos_sin + static_cast<int64_t>(pos) * kRope;
  const __nv_bfloat16* src = is_key ? p.kv_in + static_cast<int64_t>(n) * p.kv_in_token
                                    : p.q_in + static_cast<int64_t>(n) * p.q_in_token + static_cast<int64_t>(h) * p.q_in_head;
  const int plain = (is_key ? kLatentDim : p.q_dim) - kRope;  // columns that are not rotated
  const __nv_bfloat16* weight = is_key ? p.kv_weight : p.q_weight;
  const int chunks = plain / 8;                               // at most 64: two per lane
  const bool has0 = lane < chunks, has1 = lane + 32 < chunks, has_r = lane >= kRopeLane;
  float f0[8] = {}, f1[8] = {}, fr[8] = {};
  {
    const uint4* s4 = reinterpret_cast<const uint4*>(src);
    uint4 w0 = {}, w1 = {}, wr = {};
    if (has0) w0 = s4[lane];
    if (has1) w1 = s4[lane + 32];
    if (has_r) wr = s4[chunks + lane - kRopeLane];
    unpack8(w0, f0);
    unpack8(w1, f1);
    unpack8(wr, fr);
  }
  if (weight) {
    // a key's norm covers its 512 latent columns, a query's its whole width
    const float ss = warp_sum(sum_sq(f0) + sum_sq(f1) + (is_key ? 0.f : sum_sq(fr)));
    const int width = is_key ? kValueDim : p.q_dim;
    const float inv = 1.f / sqrtf(ss / static_cast<float>(width) + p.eps);
    if (has0) scale8(f0, inv, weight + lane * 8);
    if (has1) scale8(f1, inv, weight + (lane + 32) * 8);
    if (has_r && !is_key) scale8(fr, inv, weight + plain + (lane - kRopeLane) * 8);
  }
  rotate(fr, cs, lane, p.interleaved != 0);
  if (!is_key || p.kv_dtype == kKvBf16) {
    uint4* dst = reinterpret_cast<uint4*>(
        is_key ? reinterpret_cast<__nv_bfloat16*>(p.kv_pages) + slot * kLatentDim
               : p.q_out + static_cast<int64_t>(n) * p.q_out_token + static_cast<int64_t>(h) * p.q_out_head);
    if (has0) dst[lane] = pack8(f0);
    if (has1) dst[lane + 32] = pack8(f1);
    if (has_r) dst[chunks + lane - kRopeLane] = pack8(fr);
  } else {
    const bool int8 = p.kv_dtype == kKvInt8;
    uint2* dst = reinterpret_cast<uint2*>(p.kv_pages + slot * kLatentDim);
    if (has0) dst[lane] = codes8(f0, p.kv_scale, int8);
    if (has1) dst[lane + 32] = codes8(f1, p.kv_scale, int8);
    if (has_r) dst[chunks + lane - kRopeLane] = codes8(fr, p.kv_scale, int8);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.tokens) * (p.heads + (p.kv_in ? 1 : 0));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append_kernel, p);
}

}  // namespace mla
