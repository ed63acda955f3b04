// Rows of a cache in 4 bits, shared by the kernel that writes them (norm_rope.cu) and those that read them
// (q4.cu).
//
// A row x of 128 values is kept as  x[i] ~ 2^e s[i / 16] c[i]:
//   c  sign, two exponent bits, one of mantissa (0, 1/2, 1, 3/2, 2, 3, 4, 6), low nibble first
//   s  sign, four exponent bits, three of mantissa, one scale for 16 values: their largest over 6, rounded
//   e  one power of two for the row, such that its largest scale lies in [128, 256] (-100 .. 90): scales
//      down to 2^-13 of the row's largest then have all their bits, whatever the row's magnitude (values,
//      unlike keys, come without a norm).
// The value of a code times its scale has at most six significant bits, so 16-bit floats hold it exactly.
// Every rounding is to nearest, ties to even.  A row with an infinity or NaN is NaN throughout (its scales are).
// A cache is [B][heads][capacity / 128] blocks of 128 rows of one head, which the decode kernels copy whole:
// 128 x 64 bytes of codes, 128 x 8 scales, 128 bytes e + 127.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace msa {

constexpr int kQ4Codes = kD / 2, kQ4Scales = kD / 16;          // bytes of a row
constexpr int kQ4ScaleAt = kBlock * kQ4Codes;                  // offsets in a block
constexpr int kQ4ExpAt = kQ4ScaleAt + kBlock * kQ4Scales;
constexpr int kQ4Block = kQ4ExpAt + kBlock;                    // 9344 bytes
constexpr int kQ4MinExp = -100, kQ4MaxExp = 90;
constexpr int kQ4NaN = 0x7f;  // scale byte

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Eight codes as fp16 pairs (the bytes are taken inside the conversions: no shifts and masks), and two scales.
__device__ __forceinline__ void q4_codes(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\ncvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t q4_scales(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}

// One row held by 16 lanes, eight bf16 each (v), to `row` of a block.  All lanes of the warp take part;
// those whose row is not wanted pass store = false.
__device__ __forceinline__ void q4_store_row(uint4 v, uint8_t* block, int row, int l, bool store) {
  constexpr uint32_t kFull = 0xffffffffu;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // magnitudes of bf16 compare as integers, infinities and NaN above the rest
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  m = max(m & 0xffffu, m >> 16);
  const uint32_t top16 = max(m, __shfl_xor_sync(kFull, m, 1));
  uint32_t top = max(top16, __shfl_xor_sync(kFull, top16, 2));
  top = max(top, __shfl_xor_sync(kFull, top, 4));
  top = max(top, __shfl_xor_sync(kFull, top, 8));
  const bool finite = top < 0x7f80u;
  const int p = (int)(__float_as_uint(__fdiv_rn(__uint_as_float(top << 16), 6.f)) >> 23) - 127;  // floor of log2
  const int e = finite ? min(max(p - 7, kQ4MinExp), kQ4MaxExp) : 0;
  const float down = pow2f(-e);
  const float want = __fdiv_rn(__uint_as_float(top16 << 16) * down, 6.f);
  uint32_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  if (!finite) sb = kQ4NaN;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)sb, __NV_E4M3)));
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = make_float2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
    // x / s: the product with the rounded reciprocal corrected by its remainder.  Exact wherever the quotient
    // lies on a border between two codes (x has 8 bits, a border times s at most 7); elsewhere it is 2^-12 away
    // from one.
    const float a = x.x * r, b = x.y * r;
    x.x = fmaf(fmaf(-a, s, x.x), r, a);
    x.y = fmaf(fmaf(-b, s, x.y), r, b);
    code |= (uint32_t)__nv_cvt_float2_to_fp4x2(x, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  if (!finite) code = 0;
  sb <<= 8 * ((l >> 1) & 3);
  sb |= __shfl_xor_sync(kFull, sb, 2);
  sb |= __shfl_xor_sync(kFull, sb, 4);
  if (!store) return;
  *reinterpret_cast<uint32_t*>(block + row * kQ4Codes + 4 * l) = code;
  if ((l & 7) == 0) *reinterpret_cast<uint32_t*>(block + kQ4ScaleAt + row * kQ4Scales + (l >> 1)) = sb;
  if (l == 0) block[kQ4ExpAt + row] = (uint8_t)(e + 127);
}

}  // namespace msa
