// mla_gather_sm103a.cu -- latent rows of requests, out of the pages of any pool format, as contiguous bf16 rows:
// what a prefill needs that projects a cached prefix up again (its k and v are functions of these rows).
//
// out[r] = value(row r - cu_rows[b] of request b), r in cu_rows[b] .. cu_rows[b+1] - 1; a value is its code times
// the scale, in fp32, rounded once.
//
// Bound by memory: each row is read once and 1152 bytes are written.  A row is 72 chunks of eight columns, a
// lane takes three; a warp has the loads of two rows in flight (336-byte rows are three loads of 4, 4 and 8 bytes a
// lane and the exponents).  64192 rows of 4-bit pages: 15.0 us, 6.3 TB/s; one row a warp 17.5, four 16.0 (65536 bf16
// rows 21.4, 22.3, 22.3); with codes decoded to e4m3, converted and multiplied 17.3 at four, the issue slots 72 % busy.
#include <cuda_fp8.h>

#include "fp4_rows.cuh"
#include "mla_internal.h"
#include "sm103a_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 2;  // rows a warp takes
constexpr int kChunks = kLatentDim / 8;

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t codes) {
  uint32_t h2;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h2) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// Four codes times the scale as two bf16 pairs.
__device__ __forceinline__ uint2 scaled4(uint32_t w, float scale, bool int8) {
  float2 x, y;
  if (int8) {
    x = make_float2(static_cast<float>(static_cast<int8_t>(w)), static_cast<float>(static_cast<int8_t>(w >> 8)));
    y = make_float2(static_cast<float>(static_cast<int8_t>(w >> 16)), static_cast<float>(static_cast<int8_t>(w >> 24)));
  } else {
    x = e4m3x2_to_f32x2(w & 0xFFFFu);
    y = e4m3x2_to_f32x2(w >> 16);
  }
  return make_uint2(pack_bf16x2(x.x * scale, x.y * scale), pack_bf16x2(y.x * scale, y.y * scale));
}

// Eight 4-bit columns as bf16: low and high bytes of each value are looked up in their group's table (a value is
// one of eight magnitudes, whose products with the scale are the table, and a sign).
__device__ __forceinline__ uint4 fp4_to_bf16(uint32_t w, const uint4& table) {
  const uint32_t m = w & 0x77777777u;
  const uint32_t la = __byte_perm(table.x, table.y, m), ha = __byte_perm(table.z, table.w, m) | (w & 0x80808080u);
  const uint32_t lb = __byte_perm(table.x, table.y, m >> 16), hb = __byte_perm(table.z, table.w, m >> 16) | ((w << 4) & 0x80808080u);
  return make_uint4(__byte_perm(la, ha, 0x5140), __byte_perm(la, ha, 0x7362), __byte_perm(lb, hb, 0x5140), __byte_perm(lb, hb, 0x7362));
}

template <int kKv>
__global__ void __launch_bounds__(32 * kWarps) kv_gather_kernel(const GatherParams p) {
  __shared__ uint4 tables[16];  // kKvFp4: by exponent, low bytes of the eight magnitudes, then high bytes
  if constexpr (kKv == kKvFp4) {
    static_assert(32 * kWarps == 16 * 8, "a thread for each entry");
    const int e = threadIdx.x >> 3, i = threadIdx.x & 7;
    const float magnitude = i < 2 ? 0.5f * i : __uint_as_float(static_cast<uint32_t>(127 + (i >> 1) - 1) << 23 | (i & 1) << 22);
    const uint32_t v = pack_bf16x2(magnitude * __uint_as_float(static_cast<uint32_t>(127 + e - kFp4ExpBias) << 23) * p.kv_scale, 0.f);
    uint8_t* bytes = reinterpret_cast<uint8_t*>(tables + e);
    bytes[i] = static_cast<uint8_t>(v);
    bytes[8 + i] = static_cast<uint8_t>(v >> 8);
    __syncthreads();
  }
  // programmatic dependent launch: no input is read before the previous kernel has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRows;
  // the last request that starts at or before the first row (a lane for each of 32 candidates at a time)
  int lo = 0, hi = p.B;  // cu_rows[lo] <= first (if any is), cu_rows[hi] > first (if any is)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool below = at < hi && __ldg(p.cu_rows + at) <= first;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    hi = min(hi, lo + (n + 1) * step);
    lo += n * step;
  }
  int b = lo;
  const int page_bits = 31 - __clz(p.page_size);  // (dividing cost 2.8 of 20.4 us)
  const int end = __ldg(p.cu_rows + p.B);
  if (blockIdx.x == 0 && threadIdx.x == 0 && (end > p.total || __ldg(p.cu_rows) < 0)) atomicOr(p.status, kStatusDeviceArg);
  int64_t src[kRows];
  float scale[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t r = first + k;
    src[k] = -2;  // not a row of any request: left alone
    scale[k] = p.kv_scale;
    if (r >= p.total || r >= end) continue;
    while (b + 1 < p.B && __ldg(p.cu_rows + b + 1) <= r) ++b;
    const int j = static_cast<int>(r) - __ldg(p.cu_rows + b);
    if (j < 0) continue;
    if (j >> page_bits >= p.max_pages) {
      if (lane == 0) atomicOr(p.status, kStatusDeviceArg);
      continue;
    }
    const int64_t page = __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + (j >> page_bits));
    src[k] = -1;  // (a page outside the pool reads as zeros)
    if (page >= 0 && page < p.num_pages) {
      src[k] = (page << page_bits) + (j & (p.page_size - 1));
      if (kKv == kKvInt8Page) scale[k] = __ldg(p.page_scales + page);
    } else if (lane == 0) {
      atomicOr(p.status, kStatusDeviceArg);
    }
  }
  constexpr int kRowBytes = kKv == kKvBf16 ? 2 * kLatentDim : kKv == kKvFp4 ? kFp4RowBytes : kLatentDim;
  uint4 v[kRows][3];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const uint8_t* row = p.kv_pages + src[k] * kRowBytes;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = lane + 32 * i;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (src[k] >= 0 && c < kChunks) {
        if constexpr (kKv == kKvBf16) {
          x = __ldcs(reinterpret_cast<const uint4*>(row) + c);
        } else if constexpr (kKv == kKvFp4) {
          if (i < 2) {
            x.x = __ldcs(reinterpret_cast<const unsigned*>(row) + c);
            x.y = __ldcs(row + kFp4ExpAt + c / 4) >> (c & 2 ? 4 : 0) & 15;
          } else {
            const uint2 t = __ldcs(reinterpret_cast<const uint2*>(row + kFp4RopeAt) + (c - 64));
            x.x = t.x, x.y = t.y;
          }
        } else {
          const uint2 t = __ldcs(reinterpret_cast<const uint2*>(row) + c);
          x.x = t.x, x.y = t.y;
        }
      }
      v[k][i] = x;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (src[k] < -1) continue;
    uint4* out = reinterpret_cast<uint4*>(p.out + (first + k) * p.out_stride);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = lane + 32 * i;
      if (c >= kChunks) continue;
      uint4 x = v[k][i];
      if constexpr (kKv != kKvBf16) {
        if (kKv == kKvFp4 && i < 2) {
          x = fp4_to_bf16(x.x, tables[x.y]);
        } else {
          constexpr bool kInt8 = kKv == kKvInt8 || kKv == kKvInt8Page;
          const uint2 l = scaled4(x.x, scale[k], kInt8), h = scaled4(x.y, scale[k], kInt8);
          x = make_uint4(l.x, l.y, h.x, h.y);
        }
      }
      out[c] = x;
    }
  }
}

}  // namespace

cudaError_t launch_kv_gather(const GatherParams& p, cudaStream_t stream) {
  static constexpr decltype(&kv_gather_kernel<kKvBf16>) kernels[5] = {
      kv_gather_kernel<kKvBf16>, kv_gather_kernel<kKvE4m3>, kv_gather_kernel<kKvInt8>, kv_gather_kernel<kKvInt8Page>,
      kv_gather_kernel<kKvFp4>};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.total) + kWarps * kRows - 1) / (kWarps * kRows)));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernels[p.kv_dtype], p);
}

}  // namespace mla
