// Device helpers of the 4-bit merged weight: the code words, the decisions of the quantiser
// and the warp-level bf16 MMA that the few-token products run on.
//
// Layout.  The weight is cut into blocks of 128 columns.  codes: uint8 [n/128][m][64], scales:
// bf16 [n/128][m][128/group], so every tile of R consecutive rows of a block is one contiguous
// run of R * 64 (and R * 256/group) bytes, whichever way the product walks.  A row's 64 bytes
// are four 16-byte chunks t of four words w; word (t, w) holds columns 32 w + 8 t + e, e < 8,
// as q + 8: column e sits at nibble e/2 + 4 (e % 2).  Chunk t is then what lane t of a
// four-lane MMA fragment group needs of the block (8 columns of each 32-column group), and a
// pair of columns (2p, 2p + 1) is the two 16-bit halves of (word >> 4p) & 0x000f000f.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace poetx {
namespace {

// columns (2p, 2p + 1) of a code word as two bf16 integers q: 0x4300 | u is the bf16 128 + u
// (one unit in the last place is 1), and subtracting 136 leaves q = u - 8 exactly
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int p) {
  const uint32_t v = ((word >> (4 * p)) & 0x000f000fu) | 0x43004300u;
  const uint32_t off = 0x43084308u;  // 136, 136
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                             *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                             *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 accumulation
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scale of a group whose largest magnitude has the fp32 bits `amax_bits`: amax / 7 (IEEE
// division) rounded to 5 significant bits, nearest even.  With 5 bits in the scale and at most
// 3 in the code, s q is a bf16 number: no path of the library rounds the dequantised weight.
// (amax / s <= 7 / (1 - 2^-5) < 7.5, so the largest value still rounds to code 7.)  A group
// holding an infinity or a NaN gets the scale NaN.
__device__ __forceinline__ uint32_t q4_scale_bits(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 0x7fc00000u;
  const uint32_t b = __float_as_uint(__fdiv_rn(__uint_as_float(amax_bits), 7.0f));
  return (b + 0x3ffffu + ((b >> 19) & 1u)) & 0xfff80000u;
}

// q = the integer nearest to w / s (ties to even), in [-7, 7]; inv = 1 / s rounded.  w * inv is
// within 2^-22 of w / s, so its rounding can only be off where w / s lies next to a half; the
// residual w - q s is exact in fp32 (both are multiples of the finer unit and it is below s),
// and it decides those cases.
__device__ __forceinline__ int q4_code(float w, float s, float inv, float half_s) {
  float q = rintf(w * inv);
  const float r = fmaf(-q, s, w);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r > half_s || (r == half_s && odd)) q += 1.f;
  else if (r < -half_s || (r == -half_s && odd)) q -= 1.f;
  return static_cast<int>(fminf(fmaxf(q, -7.f), 7.f));
}

}  // namespace
}  // namespace poetx
