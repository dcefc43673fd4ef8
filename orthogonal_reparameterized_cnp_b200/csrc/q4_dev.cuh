// Device helpers of the 4-bit merged weight: the code words, the decisions of the quantiser
// and the warp-level bf16 MMA that the few-token products run on.
//
// Layout.  The weight is cut into blocks of 128 columns.  codes: uint8 [n/128][m][64], scales:
// bf16 [n/128][m][128/group], so every tile of R consecutive rows of a block is one contiguous
// run of R * 64 (and R * 256/group) bytes, whichever way the product walks.  A row's 64 bytes
// are four 16-byte chunks t of four words w; word (t, w) holds columns 32 w + 8 t + e, e < 8,
// as q + 8: column e sits at nibble e/2 + 4 (e % 2).  Chunk t is then what lane t of a
// four-lane MMA fragment group needs of the block (8 columns of each 32-column group), and a
// pair of columns (2p, 2p + 1) is nibble p of the word's two 16-bit halves.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace poetx {
namespace {

// Loads that stay where they are written: after the wait of a kernel that was launched early
// (__ldg may be moved ahead of it, and the read-only path may hold lines from before it).  The
// predicate is the instruction's own, with no branch around it: a load inside a branch is waited
// for where the paths meet, which undoes a prefetch.  Registers keep their values when `on` is
// false.
__device__ __forceinline__ void ld_u4_if(uint4& v, const void* p, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "l"(p), "r"((int)on));
}
// (codes: each line is read once)
__device__ __forceinline__ void ld_u4_stream_if(uint4& v, const void* p, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void ld_u2_if(uint2& v, const void* p, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t"
      "@q ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
      : "+r"(v.x), "+r"(v.y)
      : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void ld_u32_if(uint32_t& v, const void* p, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q ld.global.u32 %0, [%1];\n\t}"
      : "+r"(v)
      : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void ld_u16_if(uint32_t& v, const void* p, bool on) {  // zero-extended
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q ld.global.u16 %0, [%1];\n\t}"
      : "+r"(v)
      : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void cp_async16_cg(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_u4(const void* p) {
  uint4 v = make_uint4(0, 0, 0, 0);
  ld_u4_if(v, p, true);
  return v;
}
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t v = 0;
  ld_u32_if(v, p, true);
  return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
  uint32_t v = 0;
  ld_u16_if(v, p, true);
  return v;
}

// The 8 columns of a code word as four bf16 pairs (columns 2p, 2p + 1) of (code - 8) / 4,
// exactly.  Even pairs sit in bits 0-3 of the halves: 0x4300 | u is the bf16 128 + u, and one
// fused multiply-add gives (128 + u) / 4 - 34.  Odd pairs sit in bits 4-7: alone there, they are
// the bf16 number u 2^-129 (exponent fields 0 and 1 share one spacing), and u 2^-129 2^127 - 2 is
// the same (u - 8) / 4.  So a word costs one byte permutation, four masks and four
// multiply-adds; the shifts of the direct way (3 more instructions on the half-rate integer
// pipe) made the few-token products 1.2 times slower.  The factor 4 goes to a scale or a sum.
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ void q4_unpack(uint32_t word, uint32_t (&q)[4]) {
  const uint32_t hi = __byte_perm(word, 0, 0x4341);  // the halves' upper bytes
  q[0] = bf2_fma((word & 0x000f000fu) | 0x43004300u, 0x3e803e80u, 0xc208c208u);
  q[1] = bf2_fma(word & 0x00f000f0u, 0x7f007f00u, 0xc000c000u);
  q[2] = bf2_fma((hi & 0x000f000fu) | 0x43004300u, 0x3e803e80u, 0xc208c208u);
  q[3] = bf2_fma(hi & 0x00f000f0u, 0x7f007f00u, 0xc000c000u);
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                             *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// One K chunk of the tensor-core operand from a staged tile of codes: bf16 s (code - 8) / 4 (the
// caller's sums are 4 times too small), written in the 128-byte-swizzled layout that the MMA reads.
// GT threads; 512 units of two code words (16 codes): row r of the tile, 16-byte chunk t, columns
// 64 h + 8 t .. and 64 h + 32 + 8 t .., which are the 16-byte chunks t and 4 + t of the row's 64
// columns in the operand.
//   ROWS = 128 (K-major operand): tile of 128 rows; h = `half` of its columns; row r of the stage.
//   ROWS = 64 (MN-major operand): tile of 64 rows; row r of box h of the stage.
// A thread's rows are r0, r0 + GT / 4, .., which share the swizzle and the parity: odd rows store
// their second word first, so that 8 lanes (two rows) write 8 different bank groups.
//   FULL: every row is in the tile, and its scales are staged behind the codes at `ssrc`; else
//   rows from `rows` on give zeros, and scales come from `gs` (global, row 0 of the tile) if given.
template <int ROWS, int GT, bool FULL>
__device__ __forceinline__ void q4_convert(uint32_t src, uint32_t ssrc, uint32_t dst, int gt,
                                           uint32_t half, uint32_t sg, int rows,
                                           const uint16_t* gs) {
  constexpr uint32_t RSTEP = GT / 4;
  static_assert(RSTEP % 8 == 0, "one swizzle a thread");
  const uint32_t t = (uint32_t)gt & 3u, r0 = (uint32_t)gt >> 2;
  const bool odd = (r0 & 1u) != 0;
  const uint32_t c0 = ((((odd ? 4u : 0u) + t) ^ (r0 & 7u)) << 4) + r0 * 128u + dst;
  const uint32_t c1 = ((((odd ? 0u : 4u) + t) ^ (r0 & 7u)) << 4) + r0 * 128u + dst;
#pragma unroll
  for (int jj = 0; jj < 512 / GT; ++jj) {
    const uint32_t unit_rows = ROWS / RSTEP;                       // units before the next box
    const uint32_t h = ROWS == 64 ? (uint32_t)jj / unit_rows : half;
    const uint32_t dr = ((uint32_t)jj % unit_rows) * RSTEP, r = r0 + dr;
    uint2 wd;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(wd.x), "=r"(wd.y)
                 : "r"(src + r0 * 64u + t * 16u + h * 8u + dr * 64u)
                 : "memory");
    // scales of the unit's words (32-column groups 2 h and 2 h + 1)
    const uint32_t i0 = (2u * h * sg) >> 2, i1 = ((2u * h + 1u) * sg) >> 2;
    uint32_t s0, s1;
    if (FULL || !gs) {
      uint16_t a, b;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(ssrc + (r * sg + i0) * 2u) : "memory");
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(ssrc + (r * sg + i1) * 2u) : "memory");
      s0 = a;
      s1 = b;
    } else {
      const uint16_t* g = gs + (int64_t)min((int)r, max(rows - 1, 0)) * sg;
      s0 = ld_u16(g + i0);
      s1 = ld_u16(g + i1);
    }
    const uint32_t sa = (odd ? s1 : s0) * 0x10001u, sb = (odd ? s0 : s1) * 0x10001u;
    uint32_t a[4], b[4];
    q4_unpack(odd ? wd.y : wd.x, a);
    q4_unpack(odd ? wd.x : wd.y, b);
    const bool live = FULL || (int)r < rows;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = live ? bf2_mul(a[e], sa) : 0u;
      b[e] = live ? bf2_mul(b[e], sb) : 0u;
    }
    const uint32_t off = dr * 128u + (ROWS == 64 ? h * 8192u : 0u);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(c0 + off), "r"(a[0]), "r"(a[1]),
                 "r"(a[2]), "r"(a[3])
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(c1 + off), "r"(b[0]), "r"(b[1]),
                 "r"(b[2]), "r"(b[3])
                 : "memory");
  }
}

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 accumulation
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Scale of a group whose largest magnitude has the fp32 bits `amax_bits`: amax / 7 (IEEE
// division) rounded to 5 significant bits, nearest even.  With 5 bits in the scale and at most
// 3 in the code, s q is a bf16 number: no path of the library rounds the dequantised weight.
// (amax / s <= 7 / (1 - 2^-5) < 7.5, so the largest value still rounds to code 7.)  A group
// holding an infinity or a NaN gets the scale NaN.
// The quotient: q0 = a c with c = 1/7 rounded, then q0 + (a - 7 q0) c in fused multiply-adds,
// which is a / 7 correctly rounded (Markstein 1990; checked for every mantissa), except where the
// residual could be subnormal.
__device__ __forceinline__ uint32_t q4_scale_bits(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 0x7fc00000u;
  const float a = __uint_as_float(amax_bits), c = 0x1.24924ap-3f;
  const float q0 = a * c;
  float q = fmaf(fmaf(-7.f, q0, a), c, q0);
  if (a < 0x1p-90f) q = __fdiv_rn(a, 7.f);
  const uint32_t b = __float_as_uint(q);
  return (b + 0x3ffffu + ((b >> 19) & 1u)) & 0xfff80000u;
}

// q = the integer nearest to w / s (ties to even), in [-7, 7]; inv = 1 / s within two units in
// the last place.  w * inv is within 2^-19 of w / s, so its rounding can only be off where w / s
// lies next to a half; the residual w - q s is exact in fp32 (both are multiples of the finer unit and it is below s),
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
