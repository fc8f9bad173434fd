// The form of an 8-bit activation checkpoint.  The columns of a row are taken in blocks of
// 32, the last padded with zeros; a block's values are q 2^(b - 133), q a signed byte in
// -127 .. 127 and b a byte:
//   b = 255      an infinity or NaN in the block: every value of it reads back as NaN
//   b = 7 .. 254 2^(b - 133) is the smallest power of two (no smaller than 2^-126) for which
//                the block's largest magnitude rounds to 127 steps or fewer
// A value is thus off by half a step at most, which is 2^-127 or up to 1/127.5 of the block's largest
// magnitude; only magnitudes above 127.5 2^121 are cut to 127 2^121.  Steps are powers of two so
// that a value, of 7 significant bits, is a bf16 number: products on the tensor cores take
// it as it is.
#pragma once

#include <stdint.h>

namespace muon {
namespace {

constexpr int kBlockCols = 32;

struct CheckpointView {
  int8_t* q;     // [rows][blocks * 32]
  uint8_t* b;    // [rows][blocks]
  int64_t rows;
  int32_t cols, blocks;
};

// The byte of a block whose largest magnitude has these fp32 bits (NaN above infinity).
__device__ __forceinline__ int block_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return 255;
  const int b = (int)((bits + 0x10000u) >> 23);  // from 127.5 / 64 2^k on: the next power
  return min(max(b, 7), 254);
}
// 2^(133 - b): values to steps.
__device__ __forceinline__ float steps_per_unit(int b) { return __uint_as_float((uint32_t)max(260 - b, 1) << 23); }
// 2^(b - 133), NaN for 255.
__device__ __forceinline__ float step_of(int b) {
  return b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)max(b - 6, 1) << 23);
}

// Four values in steps, rounded to even, as bytes: adding 3 2^22 leaves the integer in the
// sum's low bits.
__device__ __forceinline__ uint32_t quantize4(float x0, float x1, float x2, float x3, float scale) {
  const float big = 12582912.f;
  const uint32_t a = __float_as_uint(__fmaf_rn(x0, scale, big)), b = __float_as_uint(__fmaf_rn(x1, scale, big));
  const uint32_t c = __float_as_uint(__fmaf_rn(x2, scale, big)), d = __float_as_uint(__fmaf_rn(x3, scale, big));
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace
}  // namespace muon
