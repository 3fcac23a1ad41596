// fp4_rows.cuh -- the 4-bit latent row of include/mla.h (MLA_KV_FP4): decoding to e4m3 codes and encoding.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace mla {

constexpr int kFp4ExpAt = 256;   // bytes of a row: codes, exponents, rotated columns
constexpr int kFp4RopeAt = 272;
constexpr int kFp4MaxExp = 11;
constexpr int kFp4ExpBias = 5;   // value = magnitude 2^(e - 5)

// The e4m3 codes of a group's eight magnitudes under exponent e, 0-3 in lo and 4-7 in hi.  Magnitude m >= 1 is
// 2^(m / 2 - 1) (1 + (m % 2) / 2) (1/2 for m = 1), so each code is a constant plus 8 e, and 0 stays 0.
__device__ __forceinline__ void fp4_table(uint32_t e, uint32_t& lo, uint32_t& hi) {
  lo = e * 0x08080800u + 0x14100800u;
  hi = e * 0x08080808u + 0x24201C18u;
}

// Eight columns (a word of the row) as e4m3 codes: the magnitude's code is looked up by a byte permute in its
// group's table; the signs lie where one mask (columns 0-3) or a shift by four (4-7) brings them to each byte's
// top bit.  (Seven instructions for eight columns; with the sign beside each magnitude, as the type's own nibbles
// have it, they would be eleven.)
__device__ __forceinline__ void fp4_to_e4m3(uint32_t w, uint32_t lo, uint32_t hi, uint32_t& a, uint32_t& b) {
  const uint32_t m = w & 0x77777777u;
  a = __byte_perm(lo, hi, m) | (w & 0x80808080u);
  b = __byte_perm(lo, hi, m >> 16) | ((w << 4) & 0x80808080u);
}

// The exponent for a group whose largest magnitude (in units of kv_scale) is top: the smallest whose last step still
// rounds it by at most half a step, top <= 7 2^(e - 5), within 0 .. 11.
__device__ __forceinline__ int fp4_exponent(float top) {
  const uint32_t bits = __float_as_uint(top);
  // top = m 2^E; top / 7 <= 2^(E - 2) for m <= 1.75, else <= 2^(E - 1)
  const int k = static_cast<int>(bits >> 23) - 127 - 2 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(kFp4MaxExp, max(0, k + kFp4ExpBias));
}

// Eight columns (in units of kv_scale, no NaN) as a word of codes under exponent e: nearest, ties to even, saturated.
__device__ __forceinline__ uint32_t fp4_encode8(const float (&f)[8], int e) {
  const float scale = __uint_as_float(static_cast<uint32_t>(127 + kFp4ExpBias - e) << 23);
  uint32_t n = 0;  // eight nibbles, sign above magnitude
#pragma unroll
  for (int i = 0; i < 4; ++i)
    n |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(f[2 * i] * scale, f[2 * i + 1] * scale), __NV_E2M1, cudaRoundNearest)) << (8 * i);
  // signs: columns 0-3 to the bytes' top bits, 4-7 to their bits 3
  const uint32_t s = n & 0x88888888u, x = __byte_perm(s, 0, 0x1100), y = __byte_perm(s, 0, 0x3322);
  const uint32_t w = (n & 0x77777777u) | ((x << 4) & 0x00800080u) | (x & 0x80008000u) | (y & 0x00080008u) | ((y >> 4) & 0x08000800u);
  return w;
}

}  // namespace mla
