// mla_key_mass_sm103a.cu -- the attention weight that each cached key received in a decode
// step, accumulated over steps, sm_103a.
//
// What it computes, per request b and key j < L_b:
//   mass[b, j] = decay * mass[b, j] + sum over the rows (t, h) that see key j of
//                exp(scale * q[b,t,h] . k_j - lse[b,t,h])
// with the visibility of mla_decode (draft t sees keys 0 .. L_b - T + t) or, with tree masks,
// of mla_decode_tree.  A row whose lse is not finite adds nothing.
//
// This kernel: one CTA per (32 keys, request), the keys decoded to fp32 in shared memory,
// 16 query rows at a time beside them; a thread owns one key and every fourth row, and the
// four threads of a key add their sums in a fixed order.
#include <cuda_fp8.h>

#include "mla_internal.h"
#include "sm103a_ptx.cuh"
#include "tree_mask.cuh"

namespace mla {
namespace {

constexpr int kKeys = 32;
constexpr int kRows = 16;
constexpr int kThreads = 128;
constexpr int kPitch = kLatentDim + 1;  // odd: a warp's 32 keys fall in 32 banks
constexpr int kSmemBytes = (kKeys * kPitch + kRows * kLatentDim + kThreads) * 4;

template <int kKv>
__device__ __forceinline__ float element(const uint8_t* row, int c) {
  if constexpr (kKv == kKvBf16) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c]);
  } else if constexpr (kKv == kKvE4m3) {
    return static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(row)[c]);
  } else {
    return static_cast<float>(reinterpret_cast<const int8_t*>(row)[c]);
  }
}

template <int kKv>
__global__ void __launch_bounds__(kThreads) key_mass_kernel(const KeyMassParams p) {
  extern __shared__ float sm[];
  float* ks = sm;                       // [32][577]
  float* qs = ks + kKeys * kPitch;      // [16][576]
  float* part = qs + kRows * kLatentDim;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int L = p.seq_lens[b];
  const int k0 = blockIdx.x * kKeys;
  if (L < p.T || L > p.max_seq || L > static_cast<int64_t>(p.max_pages) * p.page_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  if (k0 >= L) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int elem = kKv == kKvBf16 ? 2 : 1;
  for (int i = warp; i < kKeys; i += kThreads / 32) {
    const int j = k0 + i;
    const uint8_t* row = nullptr;
    float mult = 1.f;
    if (j < L) {
      const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, kStatusDeviceArg);
      } else {
        row = p.kv_pool + (page * p.page_size + j % p.page_size) * kLatentDim * elem;
        if (kKv == kKvInt8Page) mult = p.page_scales[page] * p.inv_ref_scale;
      }
    }
    for (int c = lane; c < kLatentDim; c += 32) ks[i * kPitch + c] = row ? element<kKv>(row, c) * mult : 0.f;
  }
  const int key = k0 + lane;
  const int u = key - (L - p.T);  // draft index of this key (negative: prefix)
  float total = 0.f;
  for (int r0 = 0; r0 < p.R; r0 += kRows) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kLatentDim; i += kThreads) {
      const int r = r0 + i / kLatentDim;
      qs[i] = r < p.R ? __bfloat162float(p.q[(static_cast<int64_t>(b) * p.R + r) * kLatentDim + i % kLatentDim]) : 0.f;
    }
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const float* kr = ks + lane * kPitch;
    for (int c = 0; c < kLatentDim; ++c) {
      const float k = kr[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fmaf(k, qs[(warp + 4 * i) * kLatentDim + c], s[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + warp + 4 * i;
      if (r >= p.R) continue;
      const int t = r / p.H;
      const bool seen = u < 0 || (p.tree_mask ? (u < p.T && ((p.tree_mask[static_cast<int64_t>(b) * p.T + t] >> u) & 1))
                                              : u <= t);
      const float lse = p.lse[static_cast<int64_t>(b) * p.R + r];
      if (seen && fabsf(lse) < INFINITY) total += ex2_approx(fmaf(s[i], p.scale_log2, -lse * 1.4426950408889634f));
    }
  }
  part[threadIdx.x] = total;
  __syncthreads();
  if (warp == 0 && key < L) {
    const float sum = (part[lane] + part[32 + lane]) + (part[64 + lane] + part[96 + lane]);
    float* m = p.mass + static_cast<int64_t>(b) * p.mass_stride + key;
    *m = p.decay == 0.f ? sum : fmaf(p.decay, *m, sum);
  }
}

template <int kKv>
cudaError_t launch(const KeyMassParams& p, cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(key_mass_kernel<kKv>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.max_seq + kKeys - 1) / kKeys, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_mass_kernel<kKv>, p);
}

}  // namespace

cudaError_t launch_key_mass(const KeyMassParams& p, cudaStream_t stream) {
  switch (p.kv_dtype) {
    case kKvE4m3: return launch<kKvE4m3>(p, stream);
    case kKvInt8: return launch<kKvInt8>(p, stream);
    case kKvInt8Page: return launch<kKvInt8Page>(p, stream);
    default: return launch<kKvBf16>(p, stream);
  }
}

}  // namespace mla
