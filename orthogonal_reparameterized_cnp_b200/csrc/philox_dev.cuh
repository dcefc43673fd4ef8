// Counter-based random numbers for dropout: Philox4x32 with 10 rounds (Salmon, Moraes, Dror,
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), written from the paper's
// definition: each round multiplies words 0 and 2 of the counter by the constants M0, M1 and
// exchanges the halves of the products with words 1 and 3 and the round key; the key advances
// by the Weyl constants.
//
// One call serves 8 columns: counter = (column / 8, row, site, step), key = seed, and column
// lane l takes 16 of the 128 bits (word l / 2, low half first).  A value is kept when its 16
// bits are >= thr, so the probability of keeping is exactly (65536 - thr) / 65536 and the kept
// values are multiplied by its inverse; a dropped value becomes zero whatever it was.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace poetx {

// kernel-side form of poetx_dropout_desc
struct DropArgs {
  uint32_t rk0[10], rk1[10];  // round keys (the seed, advanced)
  uint32_t row0, site;
  uint32_t thr_hi;      // thr << 16
  float scale;          // 65536 / (65536 - thr)
  const unsigned long long* step;  // device counter, or nullptr for step 0
};

inline void drop_keys(DropArgs* d, uint64_t seed) {
  for (uint32_t i = 0; i < 10; ++i) {
    d->rk0[i] = (uint32_t)seed + i * 0x9E3779B9u;
    d->rk1[i] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
  }
}

namespace {

// (the round keys are kernel parameters: operands of the exclusive-ors as they stand)
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                          const DropArgs& d) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ d.rk0[i];
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ d.rk1[i];
    c3 = (uint32_t)p0;
  }
  return make_uint4(c0, c1, c2, c3);
}

// (The low half of the counter; a volatile load stays behind the wait for the previous kernel,
// which may have moved the counter.)
__device__ __forceinline__ uint32_t drop_step(const DropArgs& d) {
  uint32_t v = 0;
  if (d.step) asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(d.step) : "memory");
  return v;
}
__device__ __forceinline__ uint4 drop_words(const DropArgs& d, uint32_t step, uint32_t row,
                                            uint32_t col8) {
  return philox10(col8, d.row0 + row, d.site, step, d);
}
// bit l set: column 8 * col8 + l is kept
__device__ __forceinline__ uint32_t drop_bits(const DropArgs& d, const uint4& w) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b |= ((ww[i] << 16) >= d.thr_hi ? 1u : 0u) << (2 * i);
    b |= (ww[i] >= d.thr_hi ? 1u : 0u) << (2 * i + 1);
  }
  return b;
}

// dropout of two bf16 values (lo, hi) whose 16-bit draws are the halves of `word`
__device__ __forceinline__ uint32_t drop_bf16x2(const DropArgs& d, uint32_t v, uint32_t word) {
  const float lo = (word << 16) >= d.thr_hi ? __uint_as_float(v << 16) * d.scale : 0.f;
  const float hi = word >= d.thr_hi ? __uint_as_float(v & 0xffff0000u) * d.scale : 0.f;
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 8 bf16 columns of one call
__device__ __forceinline__ uint4 drop_bf16x8(const DropArgs& d, const uint4& v, const uint4& w) {
  return make_uint4(drop_bf16x2(d, v.x, w.x), drop_bf16x2(d, v.y, w.y), drop_bf16x2(d, v.z, w.z),
                    drop_bf16x2(d, v.w, w.w));
}
// 4 fp32 columns: the draws in words wa (columns 0, 1) and wb (columns 2, 3)
__device__ __forceinline__ uint4 drop_f32x4(const DropArgs& d, const uint4& v, uint32_t wa,
                                            uint32_t wb) {
  const float a = (wa << 16) >= d.thr_hi ? __uint_as_float(v.x) * d.scale : 0.f;
  const float b = wa >= d.thr_hi ? __uint_as_float(v.y) * d.scale : 0.f;
  const float c = (wb << 16) >= d.thr_hi ? __uint_as_float(v.z) * d.scale : 0.f;
  const float e = wb >= d.thr_hi ? __uint_as_float(v.w) * d.scale : 0.f;
  return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                    __float_as_uint(e));
}
// one 16-byte vector (8 bf16 or 4 fp32) starting at column `col` (a multiple of its length)
template <int ELEM>
__device__ __forceinline__ uint4 drop_vec(const DropArgs& d, uint32_t step, uint32_t row,
                                          uint32_t col, const uint4& v) {
  const uint4 w = drop_words(d, step, row, col >> 3);
  if (ELEM == 2) return drop_bf16x8(d, v, w);
  return (col & 4u) ? drop_f32x4(d, v, w.z, w.w) : drop_f32x4(d, v, w.x, w.y);
}
// one value
template <typename E>
__device__ __forceinline__ E drop_one(const DropArgs& d, bool keep, E v);
template <>
__device__ __forceinline__ uint16_t drop_one<uint16_t>(const DropArgs& d, bool keep, uint16_t v) {
  if (!keep) return 0;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float((uint32_t)v << 16) * d.scale));
}
template <>
__device__ __forceinline__ uint32_t drop_one<uint32_t>(const DropArgs& d, bool keep, uint32_t v) {
  return keep ? __float_as_uint(__uint_as_float(v) * d.scale) : 0u;
}
__device__ __forceinline__ bool drop_keep(const DropArgs& d, uint32_t step, uint32_t row,
                                          uint32_t col) {
  const uint4 w = drop_words(d, step, row, col >> 3);
  const uint32_t l = col & 7u, i = l >> 1;
  const uint32_t word = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
  return ((l & 1u) ? word : word << 16) >= d.thr_hi;
}

}  // namespace
}  // namespace poetx
