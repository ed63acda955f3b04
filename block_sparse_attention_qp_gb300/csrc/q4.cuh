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

// a / b in a few instructions, with c within 2^-22 of 1 / b: the product corrected by its remainder (exact in a fused
// multiply-add).  Wherever the quotient is a number of few bits, as the borders between two members of the grids below are, it
// is found exactly; the quotients here (a of 8 bits, b of 4 or 6) are 2^-12 away from any border that they do not lie on.
__device__ __forceinline__ float quotient(float a, float b, float c) {
  const float q = a * c;
  return fmaf(fmaf(-q, b, a), c, q);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row's largest magnitude (bf16 bits; they compare as integers, infinities and NaN above the rest) makes of it:
// the exponent, and with a run's largest magnitude the scale's byte, the scale times 2^e and its reciprocal (0 for a
// scale of 0).
struct Q4Row {
  int e;
  bool finite;
};
__device__ __forceinline__ Q4Row q4_row(uint32_t top) {
  Q4Row r;
  r.finite = top < 0x7f80u;
  // floor(log2(top / 6)): 6 is 3/2 4, so a mantissa from 3/2 on loses two, a smaller one three (subnormal ones are far
  // below the least exponent)
  const int p = (int)(top >> 7) - 127 - ((top & 0x7f) >= 64 ? 2 : 3);
  r.e = r.finite ? min(max(p - 7, kQ4MinExp), kQ4MaxExp) : 0;
  return r;
}
__device__ __forceinline__ uint32_t q4_scale(const Q4Row& r, uint32_t top16, float& s, float& inv) {
  const float want = quotient(__uint_as_float(top16 << 16) * pow2f(-r.e), 6.f, 1.f / 6.f);
  const uint32_t sb = r.finite ? __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3) : kQ4NaN;
  const uint32_t h = q4_scales(sb);
  s = __half2float(*reinterpret_cast<const __half*>(&h)) * pow2f(r.e);
  inv = sb != 0 ? rcp_approx(s) : 0.f;
  return sb;
}
// Codes of eight bf16.
__device__ __forceinline__ uint32_t q4_encode(const Q4Row& r, uint4 v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = quotient(__uint_as_float(w[i] << 16), s, inv);
    x[2 * i + 1] = quotient(__uint_as_float(w[i] & 0xffff0000u), s, inv);
  }
  uint32_t code;
  asm("{\n.reg .b8 a, b, c, d;\ncvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\nmov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(code)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r.finite ? code : 0u;
}
__device__ __forceinline__ uint32_t q4_top(uint4 v) {  // two bf16 magnitudes whose larger is the largest of the eight
  return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}

// One row held by 16 lanes, eight bf16 each, to `row` of a block.  All lanes of the warp take part; those whose row is
// not wanted pass store = false.
__device__ __forceinline__ void q4_store_row(uint4 v, uint8_t* block, int row, int l, bool store) {
  constexpr uint32_t kFull = 0xffffffffu;
  uint32_t m = q4_top(v);
  m = max(m & 0xffffu, m >> 16);
  const uint32_t top16 = max(m, __shfl_xor_sync(kFull, m, 1));
  uint32_t top = max(top16, __shfl_xor_sync(kFull, top16, 2));
  top = max(top, __shfl_xor_sync(kFull, top, 4));
  top = max(top, __shfl_xor_sync(kFull, top, 8));
  const Q4Row r = q4_row(top);
  float s, inv;
  const uint32_t sb = q4_scale(r, top16, s, inv);
  const uint32_t code = q4_encode(r, v, s, inv);
  if (!store) return;
  *reinterpret_cast<uint32_t*>(block + row * kQ4Codes + 4 * l) = code;
  if (!(l & 1)) block[kQ4ScaleAt + row * kQ4Scales + (l >> 1)] = (uint8_t)sb;
  if (l == 0) block[kQ4ExpAt + row] = (uint8_t)(r.e + 127);
}

// The same for a row held by 8 lanes, the 16 bf16 of one scale each: rows that are stored as they are.
__device__ __forceinline__ void q4_store_row8(uint4 a, uint4 b, uint8_t* block, int row, int l8, bool store) {
  constexpr uint32_t kFull = 0xffffffffu;
  uint32_t m = __vmaxu2(q4_top(a), q4_top(b));
  const uint32_t top16 = max(m & 0xffffu, m >> 16);
  uint32_t top = max(top16, __shfl_xor_sync(kFull, top16, 1));
  top = max(top, __shfl_xor_sync(kFull, top, 2));
  top = max(top, __shfl_xor_sync(kFull, top, 4));
  const Q4Row r = q4_row(top);
  float s, inv;
  const uint32_t sb = q4_scale(r, top16, s, inv);
  const uint2 code = make_uint2(q4_encode(r, a, s, inv), q4_encode(r, b, s, inv));
  if (!store) return;
  *reinterpret_cast<uint2*>(block + row * kQ4Codes + 8 * l8) = code;
  block[kQ4ScaleAt + row * kQ4Scales + l8] = (uint8_t)sb;
  if (l8 == 0) block[kQ4ExpAt + row] = (uint8_t)(r.e + 127);
}

}  // namespace msa
