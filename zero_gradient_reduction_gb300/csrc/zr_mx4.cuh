// The microscaled 4-bit matrix (MX4) as the kernels see it: E2M1 codes, one E8M0 scale for
// each 32 neighbours of a row, in tiles that a block copies to shared memory as they stand.
//
// A tile is 128 rows x 256 columns, 17,408 contiguous bytes (a multiple of 1024):
//   codes   128 rows of 128 bytes; the 16-byte chunk j (columns 32j .. 32j+31) of row r lies
//           at chunk j ^ (r % 8), which is the 128-byte swizzle that the tensor cores read,
//           the lower column of a byte in its lower half;
//   scales  for each half of 128 columns 512 bytes, [r % 32][r / 32][column / 32 % 4]: the
//           order in which one copy brings 128 rows' scales to tensor memory.
// Tiles of one row of tiles follow each other along the columns. Rows and columns past the
// matrix hold zero codes and finite scales, so products over whole tiles need no masks.
//
// A block's scale byte is clamp(e - 2, 0, 254) for the biased exponent e of its largest
// magnitude (2 = the exponent of 4, E2M1's largest power of two), and 255, not a number, if
// a value is not finite; the block's codes are zero then. Values are code * 2^(byte - 127).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_device.cuh"

namespace zr {

constexpr int kMxRows = 128, kMxCols = 256, kMxBlock = 32;
constexpr int kMxCodeBytes = kMxRows * kMxCols / 2;      // 16384
constexpr int kMxScaleBytes = kMxRows * kMxCols / 32;    // 1024
constexpr int kMxTileBytes = kMxCodeBytes + kMxScaleBytes;

// (No sum that could pass 63 bits.)
__host__ __device__ inline int64_t mx_tiles(int64_t n, int per) { return n / per + (n % per != 0); }

// Offset of the 16-byte chunk of (row in tile, block of 32 columns in tile) in its tile.
__device__ __forceinline__ int mx_chunk_at(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }
// Offset of its scale byte.
__device__ __forceinline__ int mx_scale_at(int r, int j) {
  return kMxCodeBytes + (j >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3);
}

// 2^(127 - byte) for byte <= 253: what a block's values are multiplied by before rounding.
__device__ __forceinline__ float mx_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// 2^(byte - 127), a subnormal for byte 0, NaN for byte 255.
__device__ __forceinline__ float mx_scale_value(int byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : (uint32_t)byte << 23);
}

// Eight values to eight codes, to nearest with ties to the even code, magnitudes over 6 to 6.
__device__ __forceinline__ uint32_t mx_codes8(const float t[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return r;
}

// Eight values to codes, rounded by chance; quarter: a quarter of 2^(127 - byte). With the neighbours
// low <= t < high of the magnitude t <= 6 under its scale and f = (t - low) / (high - low), to high iff
// f > (255.5 - r) / 256. From 1 on the neighbours are a value's leading two significand bits and the
// next, so with b the 22 bits below them the condition is b > (255.5 - r) 2^14: b + 2^14 r + 2^13 - 1
// carries, or, moved up by two bits, where the byte r lies in byte 2, 4 b + 2^16 r + 2^15 - 4. Below 1
// the spacing is 1/2, which is what t/2 + 1/2 has in its leading two bits, with the exponents that
// continue the others'; that sum is the larger of the two exactly there, and it is rounded up, which
// keeps the condition's sign because the thresholds are representable. On t/4 the leading bits run
// from 248 (for 0) to 255 (for 6), so the code is the upper byte's lower three bits.
__device__ __forceinline__ uint32_t mx_codes8_by_chance(const float x[8], float quarter, const uint32_t dither[8]) {
  uint32_t four, s[8], bits[8];
  asm("mov.u32 %0, 4;" : "=r"(four));  // unknown to the compiler: a multiply-add, off the busier pipe
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = __fmul_rn(fabsf(x[j]), quarter);
    s[j] = __float_as_uint(fmaxf(t, __fmaf_ru(t, 0.5f, 0.125f))) * four + dither[j];
    bits[j] = __float_as_uint(x[j]);
  }
  // the upper bytes of the even words, or of the odd ones: a byte to each pair of codes
  auto upper = [](const uint32_t* w) {
    return __byte_perm(__byte_perm(w[0], w[2], 0x0073), __byte_perm(w[4], w[6], 0x7300), 0x7610);
  };
  return (upper(s) & 0x07070707u) | (upper(s + 1) << 4 & 0x70707070u) | (upper(bits) >> 4 & 0x08080808u) |
         (upper(bits + 1) & 0x80808080u);
}
// 2^16 r + 2^15 - 4 for r = byte k of w.
__device__ __forceinline__ uint32_t mx_dither(uint32_t w, int k) { return __byte_perm(w, 0x7FFCu, 0x6054 | k << 8); }

// The scale byte of a block from the bits of its largest magnitude. By chance nothing may be
// clipped, or the rounding would lose its mean: a block whose largest value would lie over 6
// takes the next power of two.
template <bool CHANCE>
__device__ __forceinline__ int mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  if (e == 255) return 255;
  int byte = e > 2 ? e - 2 : 0;
  if (CHANCE && __uint_as_float(amax_bits) * mx_inverse(byte) > 6.0f) ++byte;
  return byte;
}

// Eight codes (a 32-bit word) to the values they stand for before the scale, exact in fp16.
__device__ __forceinline__ void mx_decode8(uint32_t w, float v[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// Bytes sh .. sh + 15 of the 32 bytes lo, hi (sh 0 to 15).
__device__ __forceinline__ uint4 shift16(uint4 lo, uint4 hi, uint32_t sh) {
  uint32_t v[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  if (sh & 8) {
    v[0] = v[2]; v[1] = v[3]; v[2] = v[4]; v[3] = v[5]; v[4] = v[6]; v[5] = hi.w;
  }
  if (sh & 4) {
    v[0] = v[1]; v[1] = v[2]; v[2] = v[3]; v[3] = v[4]; v[4] = v[5];
  }
  const uint32_t bits = (sh & 3u) * 8u;
  return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                    __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
}

// 16 bytes at any address, out of the one or two aligned words that hold them; no word is read
// that holds none of the 16 bytes.
__device__ __forceinline__ uint4 load16(const char* p) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  const uint32_t sh = (uint32_t)a & 15u;
  const uint4* w = reinterpret_cast<const uint4*>(a - sh);
  if (sh == 0) return ld_once(w);
  return shift16(__ldg(w), __ldg(w + 1), sh);  // (the next lane's first word: from the nearest cache)
}

}  // namespace zr
