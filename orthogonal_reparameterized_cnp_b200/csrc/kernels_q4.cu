// 4-bit merged weight with group scales (POET-X technical summary section 2.6, POET-XQ: the
// low-bit base weight; format and quantiser in q4_dev.cuh): quantisation fused with the
// permutation reduction, reading back, the products with it for few tokens, and the
// block-diagonal products of a few tokens fused with their index maps.
#include <cuda_bf16.h>

#include "poetx_internal.h"
#include "q4_dev.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRowBytes = 200 * 1024;

template <typename E>
__device__ __forceinline__ float q4_f32(E v);
template <>
__device__ __forceinline__ float q4_f32<uint32_t>(uint32_t v) { return __uint_as_float(v); }
template <>
__device__ __forceinline__ float q4_f32<uint16_t>(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}

// Codes and scales of W0[perm_R][:, perm_P] (NULL maps: identity).  Two rows at a time.  bf16: they
// come in with cp.async while the pair before them is quantised, and are then interleaved in shared
// memory, so that one access gathers a column of both.  fp32: they come in between two pairs and
// stay as they are; the smaller buffer lets a third CTA run on an SM, whose work hides the loads
// (13824 x 5120: 96 us interleaved, 81 so).  Thread t owns the
// code words t, t + threads, .. (8 columns each) of every row, with their index map in registers
// (16 bits a column); the group maximum is taken over the 4, 8 or 16 threads of a group by
// shuffles, for bf16 both rows in one register.
//
// The code.  A bf16 w (8 bits) over a scale of 5 bits is a half or at least 2^-10 away from one,
// so w inv rounded to multiples of 2^-11 (one fused multiply-add) is the half exactly or on the
// right side of it, and adding 1.5 2^23 rounds to the nearest integer, ties to even: checked for
// every mantissa of w and s.  An fp32 w can lie closer: t = w inv + 1.5 2^23 rounds at once, and
// the residual w - q s sends the elements next to a half through the exact decision of q4_code.
// Codes are put together as fp32 sums (16 u1 + u0 ...), which keeps the work on the multiply-add
// pipe.
//
// More than 8192 columns: four words a thread (MAXW = 4), held to 64 registers so that two CTAs run
// on an SM (128 and one CTA otherwise; 8 spilled bytes in the bf16 forms, 84 in the fp32 ones).
// 5120 x 13824, groups of 64: bf16 77 -> 65 us, fp32 111 -> 91.
template <typename E>
struct Pair;  // a column of two rows
template <>
struct Pair<uint16_t> {
  using T = uint32_t;
  // the largest magnitudes of both rows, 16 bits each
  uint32_t m = 0;
  __device__ __forceinline__ void see(T v) { m = __vmaxu2(m, v & 0x7fff7fffu); }
  __device__ __forceinline__ void meet(int o) { m = __vmaxu2(m, __shfl_xor_sync(~0u, m, o)); }
  __device__ __forceinline__ uint32_t a() const { return m << 16; }
  __device__ __forceinline__ uint32_t b() const { return m & 0xffff0000u; }
  static __device__ __forceinline__ void split(T v, float& a, float& b) {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xffff0000u);
  }
};
template <>
struct Pair<uint32_t> {
  using T = uint2;
  uint32_t ma = 0, mb = 0;
  __device__ __forceinline__ void see(T v) {
    ma = max(ma, v.x & 0x7fffffffu);
    mb = max(mb, v.y & 0x7fffffffu);
  }
  __device__ __forceinline__ void meet(int o) {
    ma = max(ma, __shfl_xor_sync(~0u, ma, o));
    mb = max(mb, __shfl_xor_sync(~0u, mb, o));
  }
  __device__ __forceinline__ uint32_t a() const { return ma; }
  __device__ __forceinline__ uint32_t b() const { return mb; }
  static __device__ __forceinline__ void split(T v, float& a, float& b) {
    a = __uint_as_float(v.x);
    b = __uint_as_float(v.y);
  }
};
// row a's and row b's 16-byte vectors, columns interleaved
__device__ __forceinline__ void put_pair(uint32_t* dst, const uint4& a, const uint4& b) {  // bf16
  uint4* d = reinterpret_cast<uint4*>(dst);
  d[0] = make_uint4(__byte_perm(a.x, b.x, 0x5410), __byte_perm(a.x, b.x, 0x7632),
                    __byte_perm(a.y, b.y, 0x5410), __byte_perm(a.y, b.y, 0x7632));
  d[1] = make_uint4(__byte_perm(a.z, b.z, 0x5410), __byte_perm(a.z, b.z, 0x7632),
                    __byte_perm(a.w, b.w, 0x5410), __byte_perm(a.w, b.w, 0x7632));
}

// the code word of 8 columns with scale s (bits sb)
template <bool BF16>
__device__ __forceinline__ uint32_t q4_word(const float (&w)[8], uint32_t sb) {
  float s = __uint_as_float(sb);
  if (!(s > 0.f)) return 0x88888888u;  // zero or NaN scale
  // tiny scales go through the exact decision with both sides times 2^100 (exact), so that 1 / s
  // stays finite
  const bool tiny = s < 0x1p-100f;
  const float up = tiny ? 0x1p100f : 1.f;
  s *= up;
  float inv;  // (both uses below bear an error of some units in the last place)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float half = 0.5f * s, near = half * 0.9999f;
  const float magic = 12582920.f;  // 1.5 2^23 + 8: t - 1.5 2^23 is q + 8
  float u[8];
  bool exact = tiny;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (BF16) {
      u[e] = (fmaf(w[e], inv, 6144.f) + (magic - 6144.f)) - 12582912.f;
    } else {
      u[e] = fmaf(w[e], inv, magic) - 12582912.f;
      const float r = fmaf(8.f - u[e], s, w[e]);
      exact |= !(fabsf(r) < near);
    }
  }
  if (exact) {
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = (float)(q4_code(w[e] * up, s, inv, half) + 8);
  }
  // nibble p of the lower half: columns 0, 2, 4, 6; of the upper half: 1, 3, 5, 7
  const float lo = fmaf(u[6], 4096.f, fmaf(u[4], 256.f, fmaf(u[2], 16.f, u[0])));
  const float hi = fmaf(u[7], 4096.f, fmaf(u[5], 256.f, fmaf(u[3], 16.f, u[1])));
  return __byte_perm(__float_as_uint(lo + 8388608.f), __float_as_uint(hi + 8388608.f), 0x5410);
}

template <typename E, int GS, int MAXW>
__global__ void __launch_bounds__(512, MAXW == 4 ? 2 : 0)  // (0: not given)
    k_merge_q4_pairs(const E* __restrict__ W0, const int32_t* __restrict__ perm_R,
                     const int32_t* __restrict__ perm_P, uint8_t* __restrict__ codes,
                     __nv_bfloat16* __restrict__ scales, int m, int n) {
  extern __shared__ __align__(16) unsigned char row_raw[];
  using P = Pair<E>;
  using T = typename P::T;
  constexpr int V = 16 / sizeof(E);
  constexpr bool MIX = sizeof(E) == 2;  // interleave
  T* pair = reinterpret_cast<T*>(row_raw);                                    // [n] (MIX)
  const unsigned char* stage = row_raw + (MIX ? (size_t)n * sizeof(T) : 0);  // [2][n] elements
  const uint32_t stage_s = (uint32_t)__cvta_generic_to_shared(stage);
  const int threads = blockDim.x, tid = threadIdx.x;
  const int words = n / 8, vecs = n / V;
  uint32_t idx[MAXW][4];  // byte offset of a column in 4-byte columns, 16 bits (n <= 16384)
#pragma unroll
  for (int j = 0; j < MAXW; ++j) {
    const int c = min(tid + j * threads, words - 1);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      unsigned c0 = 8u * c + e, c1 = c0 + 1;
      if (perm_P) {
        c0 = (unsigned)__ldg(perm_P + c0);
        c1 = (unsigned)__ldg(perm_P + c1);
      }
      c0 = c0 < (unsigned)n ? c0 : (unsigned)n - 1;
      c1 = c1 < (unsigned)n ? c1 : (unsigned)n - 1;
      idx[j][e / 2] = (4u * c0) | (c1 << 18);
    }
  }
  const int npair = (m + 1) / 2;
  auto fetch = [&](int pr) {
    if (pr < npair) {
      const int i0 = 2 * pr, i1 = min(2 * pr + 1, m - 1);
      unsigned s0 = perm_R ? (unsigned)__ldg(perm_R + i0) : (unsigned)i0;
      unsigned s1 = perm_R ? (unsigned)__ldg(perm_R + i1) : (unsigned)i1;
      s0 = s0 < (unsigned)m ? s0 : (unsigned)m - 1;  // keep the reads inside the matrix
      s1 = s1 < (unsigned)m ? s1 : (unsigned)m - 1;
      const uint4* a = reinterpret_cast<const uint4*>(W0 + (int64_t)s0 * n);
      const uint4* b = reinterpret_cast<const uint4*>(W0 + (int64_t)s1 * n);
      for (int v = tid; v < vecs; v += threads) {
        cp_async16_cg(stage_s + 16u * v, a + v);
        cp_async16_cg(stage_s + 16u * (vecs + v), b + v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int pr = blockIdx.x;
  fetch(pr);
  for (; pr < npair; pr += gridDim.x) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (MIX) {
      // each thread interleaves the vectors it fetched itself (the gathers of the pair before
      // ended at the barrier below)
      for (int v = tid; v < vecs; v += threads)
        put_pair(pair + v * V, lds_u4(stage_s + 16u * v), lds_u4(stage_s + 16u * (vecs + v)));
      __syncthreads();
      fetch(pr + gridDim.x);
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < MAXW; ++j) {
      const int c = tid + j * threads;
      if (c - (tid & 31) >= words) break;  // (whole warps)
      float a[8], b[8];
      P most;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t off = (e & 1) ? idx[j][e / 2] >> 16 : idx[j][e / 2] & 0xffffu;
        T v;
        if constexpr (MIX)
          v = *reinterpret_cast<const T*>(row_raw + off);
        else
          v = make_uint2(*reinterpret_cast<const uint32_t*>(row_raw + off),
                         *reinterpret_cast<const uint32_t*>(row_raw + (size_t)n * 4 + off));
        most.see(v);
        P::split(v, a[e], b[e]);
      }
#pragma unroll
      for (int o = 1; o < GS / 8; o <<= 1) most.meet(o);
      const uint32_t sa = q4_scale_bits(most.a()), sb = q4_scale_bits(most.b());
      const uint32_t wa = q4_word<sizeof(E) == 2>(a, sa), wb = q4_word<sizeof(E) == 2>(b, sb);
      if (c < words) {
        const int blk = c >> 4, l = c & 15;  // columns 8 l: word w = l / 4 of chunk t = l % 4
        const int64_t r = (int64_t)blk * m + 2 * pr;
        const bool both = 2 * pr + 1 < m;
        uint32_t* cw = reinterpret_cast<uint32_t*>(codes + r * 64) + 4 * (l & 3) + (l >> 2);
        cw[0] = wa;
        if (both) cw[16] = wb;
        if ((l & (GS / 8 - 1)) == 0) {
          uint16_t* sw = reinterpret_cast<uint16_t*>(scales) + r * (128 / GS) + l / (GS / 8);
          sw[0] = (uint16_t)(sa >> 16);
          if (both) sw[128 / GS] = (uint16_t)(sb >> 16);
        }
      }
    }
    __syncthreads();
    if constexpr (!MIX) fetch(pr + gridDim.x);
  }
}

// Rows too wide for the pairs (index map or shared memory): one CTA per row; the source row is
// staged in shared memory, thread c owns the 8 columns of code word c.
template <typename E, int GS>
__global__ void __launch_bounds__(kThreads)
    k_merge_q4(const E* __restrict__ W0, const int32_t* __restrict__ perm_R,
               const int32_t* __restrict__ perm_P, uint8_t* __restrict__ codes,
               __nv_bfloat16* __restrict__ scales, int m, int n) {
  extern __shared__ __align__(16) unsigned char row_raw[];
  E* row = reinterpret_cast<E*>(row_raw);
  constexpr int V = 16 / sizeof(E);
  const int words = n / 8;
  for (int i = blockIdx.x; i < m; i += gridDim.x) {
    unsigned sr = perm_R ? (unsigned)__ldg(perm_R + i) : (unsigned)i;
    sr = sr < (unsigned)m ? sr : (unsigned)m - 1;  // keep the read inside the matrix
    const uint4* src = reinterpret_cast<const uint4*>(W0 + (int64_t)sr * n);
    for (int v = threadIdx.x; v < n / V; v += kThreads)
      reinterpret_cast<uint4*>(row)[v] = __ldg(src + v);
    __syncthreads();
    for (int c0 = 0; c0 < words; c0 += kThreads) {  // whole warps: words % 16 == 0
      const int c = c0 + threadIdx.x;
      const bool on = c < words;
      float w[8];
      uint32_t amax = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        unsigned col = on ? 8 * c + e : 0;
        if (perm_P) col = (unsigned)__ldg(perm_P + col);
        col = col < (unsigned)n ? col : (unsigned)n - 1;
        w[e] = q4_f32<E>(row[col]);
        amax = max(amax, __float_as_uint(w[e]) & 0x7fffffffu);
      }
#pragma unroll
      for (int o = 1; o < GS / 8; o <<= 1) amax = max(amax, __shfl_xor_sync(~0u, amax, o));
      const uint32_t sb = q4_scale_bits(amax);
      float s = __uint_as_float(sb);
      // tiny scales: both sides times 2^100 (exact), so that 1 / s stays finite
      const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
      s *= up;
      const bool live = s > 0.f;  // false for 0 and NaN: codes 0
      const float inv = live ? __fdiv_rn(1.f, s) : 0.f;
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int q = live ? q4_code(w[e] * up, s, inv, 0.5f * s) : 0;
        word |= (uint32_t)(q + 8) << (4 * (e / 2 + 4 * (e & 1)));
      }
      if (on) {
        const int blk = c >> 4, l = c & 15;  // columns 8 l: word w = l / 4 of chunk t = l % 4
        const int64_t r = (int64_t)blk * m + i;
        reinterpret_cast<uint32_t*>(codes + r * 64)[4 * (l & 3) + (l >> 2)] = word;
        if ((l & (GS / 8 - 1)) == 0)
          reinterpret_cast<uint16_t*>(scales)[r * (128 / GS) + l / (GS / 8)] =
              (uint16_t)(sb >> 16);
      }
    }
    __syncthreads();
  }
}

// out[i, j] = s q (fp32 product, rounded once to the output type; exact for the quantiser's
// scales).  Thread per 16-byte chunk: four consecutive threads hold a row's block, and write it as
// four runs of 32 columns.
template <typename E, int GS>
__global__ void __launch_bounds__(kThreads)
    k_dequant_q4(const uint8_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                 E* __restrict__ out, int m, int n) {
  const int64_t v = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  const int t = (int)(v & 3);
  const int64_t i = v >> 2;
  if (i >= m) return;
  for (int blk = blockIdx.y; blk < n / 128; blk += gridDim.y) {
    const int64_t r = (int64_t)blk * m + i;
    const uint4 cd = __ldg(reinterpret_cast<const uint4*>(codes + r * 64) + t);
    const uint32_t words[4] = {cd.x, cd.y, cd.z, cd.w};
    E* o = out + i * n + blk * 128 + 8 * t;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float s = __bfloat162float(scales[r * (128 / GS) + w / (GS / 32)]);
      uint32_t q[4];
      q4_unpack(words[w], q);
      float f[8];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f[2 * p] = s * (4.f * bf_lo(q[p]));
        f[2 * p + 1] = s * (4.f * bf_hi(q[p]));
      }
      if constexpr (sizeof(E) == 2) {
        uint32_t h[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * p], f[2 * p + 1]);
          h[p] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(o + 32 * w) = make_uint4(h[0], h[1], h[2], h[3]);
      } else {
        reinterpret_cast<float4*>(o + 32 * w)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(o + 32 * w)[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// y[t, i] = sum_j W[i, j] x[t, j], up to 8 tokens (NT = 1) or 16 (NT = 2: each code is unpacked
// once for two MMAs).  One CTA: 16 rows of W; the K blocks are
// dealt to its warps.  Lane (g, t) loads chunk t of rows g and g + 8 (1 KB a warp and block,
// contiguous), which is its A fragment of 8 MMAs once the nibbles are bf16 integers; the
// integers are multiplied exactly, and the group's sum is scaled in fp32.  Lanes of tokens past
// T read the last token's row: a column of the MMA is one token's alone, and theirs is not
// stored.
// Small CTAs (four warps) spread evenly over the SMs.  Each lane's codes of the next kRowD
// blocks are on their way into its own slots of shared memory (cp.async; nothing is shared, so
// nothing is synchronised).  Offsets count 16-byte chunks in 32 bits: one wide multiply-add an
// address.
//
// Bound: codes and scales at HBM rate (5.6 us at 13824 x 5120); the conversion's masks on the
// half-rate integer pipe come next (about 3 us there, overlapped in part).  Measured, T = 1, group
// 128: 6.6 us at 5120 x 5120, 11.5 at 13824 x 5120, 13.6 at 5120 x 13824 (loads alone: 7.0 at
// 13824 x 5120).  16 tokens: 11.3, 22.1, 25.6, and 6.4 at 4096 x 4096 (with the weight as the M
// operand of tcgen05: 13.8, 28, 27.2, 11.8; 128-row tiles whose tokens pass through shared memory:
// 21 at 13824 x 5120).  One load a block without the ring: 8.5, 16.4, 20.4; a persistent grid with
// the ring in registers: 9.4, 15.4, 22.5 (320 row tiles do not divide evenly).
constexpr int kRowD = 4;

// a row's scales in a block as one load
template <int SG>
struct RowScales;
template <>
struct RowScales<1> {
  uint32_t v = 0;
  __device__ __forceinline__ void load(const uint16_t* p, bool on) { ld_u16_if(v, p, on); }
  __device__ __forceinline__ float at(int) const { return __uint_as_float(v << 16); }
};
template <>
struct RowScales<2> {
  uint32_t v = 0;
  __device__ __forceinline__ void load(const uint16_t* p, bool on) { ld_u32_if(v, p, on); }
  __device__ __forceinline__ float at(int h) const {
    return __uint_as_float(h ? v & 0xffff0000u : v << 16);
  }
};
template <>
struct RowScales<4> {
  uint2 v = {0, 0};
  __device__ __forceinline__ void load(const uint16_t* p, bool on) { ld_u2_if(v, p, on); }
  __device__ __forceinline__ float at(int h) const {
    const uint32_t w = h & 2 ? v.y : v.x;
    return __uint_as_float(h & 1 ? w & 0xffff0000u : w << 16);
  }
};

// what hi leaves of v (nothing of an infinity: the sum stays one)
__device__ __forceinline__ __nv_bfloat16 lo_part(float v, __nv_bfloat16 hi) {
  const float h = __bfloat162float(hi);
  return __float2bfloat16_rn(fabsf(h) < INFINITY ? v - h : 0.f);
}

// The row of column g of an MMA of up to 8 tokens: token g, or of up to 4 tokens (hi + lo) token
// g % 4 of hi (g < 4) or lo; behind the last token, that one again.
__device__ __forceinline__ const __nv_bfloat16* few_row(const __nv_bfloat16* hi,
                                                        const __nv_bfloat16* lo, int g, int T,
                                                        int width) {
  if (T > 4) return hi + (int64_t)min(g, T - 1) * width;
  return (g < 4 ? hi : lo) + (int64_t)min(g & 3, T - 1) * width;
}

// In the layer (LAYER) up to 4 tokens come and go as sums of two bf16 numbers, hi + lo (16
// significant bits): lo takes the MMAs' columns 4 to 7, which are idle then, so that the
// intermediates of so few tokens are not rounded to bf16 at no cost.  (A form with MMAs of their
// own for lo, up to 8 tokens, read x twice as often as the codes: 5120 x 13824, 8 tokens, layer
// 36 us against 29.)
template <int GS, int WARPS, int NT, bool LAYER>
__global__ void __launch_bounds__(32 * WARPS, (NT == 1 ? 24 : 16) / WARPS)
    k_q4_rows(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
              const __nv_bfloat16* __restrict__ x, __nv_bfloat16* __restrict__ y,
              const __nv_bfloat16* __restrict__ x_lo, __nv_bfloat16* __restrict__ y_lo, int T,
              int m, int n) {
  constexpr int SG = 128 / GS, D = kRowD;  // SG: scales per row and block
  extern __shared__ __align__(16) unsigned char row_ring[];
  uint4 (*ring)[WARPS][64] = reinterpret_cast<uint4 (*)[WARPS][64]>(row_ring);  // [D]
  __shared__ float red[WARPS][8 * NT][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = blockIdx.x * 16;
  const int ra = min(row0 + g, m - 1), rb = min(row0 + g + 8, m - 1);
  const int cnt = (n / 128 - warp + WARPS - 1) / WARPS;  // blocks warp, warp + 4, ...
  const uint4* c16 = reinterpret_cast<const uint4*>(codes);
  uint32_t oc = ((uint32_t)warp * (uint32_t)m + (uint32_t)ra) * 4u + (uint32_t)t;
  uint32_t os = ((uint32_t)warp * (uint32_t)m + (uint32_t)ra) * SG;
  const uint32_t dc = (uint32_t)(rb - ra) * 4u, ds = (uint32_t)(rb - ra) * SG;
  const uint32_t step = (uint32_t)WARPS * (uint32_t)m;
  const uint4* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    xp[i] = reinterpret_cast<const uint4*>(
        (LAYER && NT == 1 ? few_row(x, x_lo, g, T, n) : x + (int64_t)min(8 * i + g, T - 1) * n) +
        warp * 128 + t * 8);
  RowScales<SG> sa[2], sb[2];
  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(&ring[0][warp][lane]);
  int left = cnt;  // blocks whose loads are to be issued
  auto load = [&](uint32_t slot) {
    if (left > 0) {  // (uniform; an empty group otherwise)
      cp_async16_cg(slot, c16 + oc);
      cp_async16_cg(slot + 512u, c16 + (oc + dc));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    --left;
    oc += step * 4u;
  };
  auto load_scales = [&](int b, bool on) {
    sa[b].load(scales + os, on);
    sb[b].load(scales + (os + ds), on);
    os += step * SG;
  };
  constexpr uint32_t kSlot = WARPS * 1024u;  // bytes of a ring stage
  if (!LAYER) {
    pdl_trigger();
    pdl_wait();
  }
#pragma unroll
  for (int d = 0; d < D; ++d) load(slot0 + d * kSlot);
  load_scales(0, cnt > 0);
  if (LAYER) {  // behind k_bd_rows, which lets this launch begin once all before it has ended
    pdl_wait();
    pdl_trigger();
  }
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
  uint32_t slot = slot0;
  auto compute = [&](int b) {
    uint4 xv[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int w = 0; w < 4; ++w) xv[i][w] = ld_u4(xp[i] + w * 4);
      xp[i] += WARPS * 16;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    const uint4 ca = lds_u4(slot), cb = lds_u4(slot + 512u);
    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
    float part[NT][4], odd[NT][4];  // two chains of MMAs
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t qa[4], qb[4];
      q4_unpack(wa[w], qa);
      q4_unpack(wb[w], qb);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = xv[i][w];
        if (w % (GS / 32) == 0) {
          mma16816_zero(part[i], qa[0], qb[0], qa[1], qb[1], v.x, v.y);
          mma16816_zero(odd[i], qa[2], qb[2], qa[3], qb[3], v.z, v.w);
        } else {
          mma16816(part[i], qa[0], qb[0], qa[1], qb[1], v.x, v.y);
          mma16816(odd[i], qa[2], qb[2], qa[3], qb[3], v.z, v.w);
        }
        if ((w + 1) % (GS / 32) == 0) {
          const float a = sa[b].at(w / (GS / 32)), c = sb[b].at(w / (GS / 32));
          acc[i][0] = fmaf(a, part[i][0] + odd[i][0], acc[i][0]);
          acc[i][1] = fmaf(a, part[i][1] + odd[i][1], acc[i][1]);
          acc[i][2] = fmaf(c, part[i][2] + odd[i][2], acc[i][2]);
          acc[i][3] = fmaf(c, part[i][3] + odd[i][3], acc[i][3]);
        }
      }
    }
    load(slot);  // (the slot's codes are in registers)
    slot = slot == slot0 + (D - 1) * kSlot ? slot0 : slot + kSlot;
  };
  int j = 0;
  for (; j + 2 <= cnt; j += 2) {
    load_scales(1, true);
    compute(0);
    load_scales(0, j + 2 < cnt);
    compute(1);
  }
  if (j < cnt) compute(0);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    red[warp][8 * i + 2 * t][g] = acc[i][0];
    red[warp][8 * i + 2 * t + 1][g] = acc[i][1];
    red[warp][8 * i + 2 * t][g + 8] = acc[i][2];
    red[warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
  }
  __syncthreads();
  const int r = threadIdx.x & 15;
  if (row0 + r >= m) return;
  for (int tok = threadIdx.x >> 4; tok < min(T, 8 * NT); tok += 2 * WARPS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += red[w][tok][r];  // fixed order
    if (LAYER && NT == 1 && T <= 4) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += red[w][tok + 4][r];
    }
    const int64_t o = (int64_t)tok * m + row0 + r;
    const __nv_bfloat16 hi = __float2bfloat16_rn(4.f * v);
    y[o] = hi;
    if (LAYER && NT == 1 && T <= 4) y_lo[o] = lo_part(4.f * v, hi);
  }
}

// ---------------------------------------------------------------------------------------
// dx[t, j] = sum_i W[i, j] dy[t, i], up to 8 tokens.  One CTA: one block of 128 columns; its
// share of the 16-row steps is dealt to 8 warps, and the shares of a block form a cluster.  Lane
// (g, t) loads two words (chunk g / 2, half g % 2) of rows 4 t .. 4 t + 3; halves of two rows'
// words side by side give bf16 pairs along the rows, which the MMA sums over.  The scale changes
// along the summed index, so it multiplies the bf16 integers (exact for scales of 5 significant
// bits).  Measured, T = 1, group 128: 7.8 us at 5120 x 5120, 14.9 at 13824 x 5120, 15.7 at 5120 x
// 13824; with loads inside branches (waited for where the paths meet) 10.7, 20.9, 21.5; adding the
// warps' sums in three halving rounds instead of one costs 1 us.
constexpr int kColWarps = 8;
constexpr int kColU = 3;  // steps in flight per warp

// WHOLE: m % 16 == 0
template <int GS, bool WHOLE>
__global__ void __launch_bounds__(32 * kColWarps, 2)
    k_q4_cols(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
              const __nv_bfloat16* __restrict__ dy, __nv_bfloat16* __restrict__ dx, int T, int m,
              int n, int steps_per_cta) {
  __shared__ __align__(16) float sums[kColWarps][8][132];
  constexpr int SG = 128 / GS, U = kColU;
  constexpr int NS = GS == 32 ? 2 : 1;  // scales per row for the lane's two words
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blk = blockIdx.x;
  const int nsteps = (m + 15) / 16;
  const int s_first = blockIdx.y * steps_per_cta;
  const int s_last = min(nsteps, s_first + steps_per_cta);
  const int64_t base = (int64_t)blk * m;
  // the warp's steps s_first + warp, s_first + warp + 8, ...: 16 rows, 4 of them the lane's
  const int cnt = max(0, (s_last - s_first - warp + kColWarps - 1) / kColWarps);
  const int i_first = (s_first + warp) * 16 + 4 * t;
  const uint2* c8 = reinterpret_cast<const uint2*>(codes);
  uint32_t oc = ((uint32_t)base + (uint32_t)i_first) * 8u + (uint32_t)g;  // 8 bytes x 8 a row
  uint32_t os = ((uint32_t)base + (uint32_t)i_first) * SG +
                (GS == 128 ? 0u : GS == 64 ? (uint32_t)(g & 1) : 2u * (uint32_t)(g & 1));
  const uint16_t* dp = reinterpret_cast<const uint16_t*>(dy) + (int64_t)min(g, T - 1) * m + i_first;
  int i0 = i_first;  // of the next load
  float acc[2][4][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][p][c] = 0.f;
  uint2 wd[U][4], dv[U];
  uint32_t sc[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    dv[u] = make_uint2(0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      wd[u][r] = make_uint2(0, 0);
      sc[u][r] = 0;
    }
  }
  auto load = [&](int u, bool on) {
    if (WHOLE) {
      ld_u2_if(dv[u], dp, on);
      const uint2* c = c8 + oc;
      const uint16_t* q = scales + os;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ld_u2_if(wd[u][r], c + 8 * r, on);
        if (NS == 2)
          ld_u32_if(sc[u][r], q + SG * r, on);
        else
          ld_u16_if(sc[u][r], q + SG * r, on);
      }
    } else if (on) {
      // rows past the end have zero dy, and the last row's word and scale again (its own group,
      // so nothing enters that is not there already)
      uint32_t d[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        d[r] = i0 + r < m ? ld_u16(dp + r) : 0u;
        const uint32_t back = (uint32_t)max(0, i0 + r - (m - 1));
        ld_u2_if(wd[u][r], c8 + (oc + 8u * (uint32_t)r - 8u * back), true);
        const uint16_t* q = scales + (os + SG * (uint32_t)r - SG * back);
        sc[u][r] = NS == 2 ? ld_u32(q) : ld_u16(q);
      }
      dv[u] = make_uint2(d[0] | (d[1] << 16), d[2] | (d[3] << 16));
    }
    oc += kColWarps * 16 * 8;
    os += kColWarps * 16 * SG;
    dp += kColWarps * 16;
    i0 += kColWarps * 16;
  };
  auto compute = [&](int u) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t sel = NS == 2 && j ? 0x7632u : 0x5410u;
      const uint32_t s01 = __byte_perm(sc[u][0], sc[u][1], sel);
      const uint32_t s23 = __byte_perm(sc[u][2], sc[u][3], sel);
      const uint32_t w0 = j ? wd[u][0].y : wd[u][0].x, w1 = j ? wd[u][1].y : wd[u][1].x;
      const uint32_t w2 = j ? wd[u][2].y : wd[u][2].x, w3 = j ? wd[u][3].y : wd[u][3].x;
      const uint32_t lo01 = __byte_perm(w0, w1, 0x5410), hi01 = __byte_perm(w0, w1, 0x7632);
      const uint32_t lo23 = __byte_perm(w2, w3, 0x5410), hi23 = __byte_perm(w2, w3, 0x7632);
      uint32_t a0[4], a1[4], a2[4], a3[4];
      q4_unpack(lo01, a0);
      q4_unpack(hi01, a1);
      q4_unpack(lo23, a2);
      q4_unpack(hi23, a3);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        mma16816(acc[j][p], bf2_mul(a0[p], s01), bf2_mul(a1[p], s01), bf2_mul(a2[p], s23),
                 bf2_mul(a3[p], s23), dv[u].x, dv[u].y);
    }
  };
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u < cnt);
  int k = 0;
  for (; k + U <= cnt; k += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      compute(u);
      load(u, k + u + U < cnt);
    }
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (k + u < cnt) compute(u);
  // lane's value (j, p, c): token 2 t + (c & 1), column 2 p + (c >> 1) of word (t' = g / 2,
  // w = 2 (g % 2) + j), i.e. column 32 w + 8 t' + ...  The warps' sums are added in warp order.
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (2 * t + (c & 1) < T)
          sums[warp][2 * t + (c & 1)]
              [32 * (2 * (g & 1) + j) + 8 * (g >> 1) + 2 * p + (c >> 1)] = acc[j][p][c];
  __syncthreads();
  for (int o = threadIdx.x; o < T * 128; o += 32 * kColWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kColWarps; ++w) v += sums[w][o >> 7][o & 127];
    sums[0][o >> 7][o & 127] = v;  // (this thread alone reads and writes the place)
  }
  const int splits = gridDim.y;
  auto store = [&](int tok, int c, float v) {
    dx[(int64_t)tok * n + blk * 128 + c] = __float2bfloat16_rn(4.f * v);
  };
  if (splits == 1) {
    __syncthreads();
    for (int o = threadIdx.x; o < T * 128; o += 32 * kColWarps)
      store(o >> 7, o & 127, sums[0][o >> 7][o & 127]);
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
  const uint32_t local = (uint32_t)__cvta_generic_to_shared(&sums[0][0][0]);
  for (int o = (int)blockIdx.y * 32 * kColWarps + threadIdx.x; o < T * 128;
       o += splits * 32 * kColWarps) {
    float v = 0.f;
    for (int q = 0; q < splits; ++q) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(addr)
                   : "r"(local + 4u * (uint32_t)((o >> 7) * 132 + (o & 127))), "r"(q));
      float f;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(addr) : "memory");
      v += f;
    }
    store(o >> 7, o & 127, v);
  }
  // no CTA leaves while another still reads its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// ---------------------------------------------------------------------------------------
// Block-diagonal product of a few tokens (8 a CTA) with its index map; V and W of up to 4 tokens
// are hi + lo (see k_q4_rows):
//   gather:  V_j = U_j G_P,j^T, U = X[:, p_P] (also written when `save` is given), V = out + lo;
//   scatter: Z_j = W_j G_R,j^T, W = in + lo, Y[:, p_R[i]] = Z[:, i].
// One CTA: 16 rows of one block; its four warps split k and add their sums in a fixed order.  A
// lane reads the operands of its MMAs straight from global memory - 8 columns of its token, for
// the gather by their indices - with everything of a warp in flight at once (KI = b / 128 steps).
// Bound by latency: the layer's three launches overlap by what each can read before its
// predecessor ends (G and the indices here, the codes in k_q4_rows).
constexpr int kBdWarps = 4;

template <int KI, int RT, bool GATHER>
__global__ void __launch_bounds__(32 * kBdWarps)
    k_bd_rows(const __nv_bfloat16* __restrict__ G, const __nv_bfloat16* __restrict__ in,
              __nv_bfloat16* __restrict__ out, __nv_bfloat16* __restrict__ lo,
              __nv_bfloat16* __restrict__ save, const int32_t* __restrict__ idx, int T,
              int width) {
  constexpr int b = 128 * KI, tiles = b / (16 * RT);
  __shared__ float red[RT][kBdWarps][8][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int j = blockIdx.x / tiles, i0 = (blockIdx.x - j * tiles) * (16 * RT);
  const int k0 = warp * (32 * KI) + 8 * t;  // columns k0 + 32 i .. + 7 of the block
  if (GATHER) {
    pdl_wait();
    pdl_trigger();  // after the wait: what the next launch reads early was there before this one
  }
  // tokens 8 blockIdx.y ..: `few` of them
  const int few = min(8, T - 8 * (int)blockIdx.y);
  const bool two = T <= 4;  // hi + lo
  in += (int64_t)blockIdx.y * 8 * width;
  out += (int64_t)blockIdx.y * 8 * width;
  if (save) save += (int64_t)blockIdx.y * 8 * width;
  uint4 ga[RT][KI], gb[RT][KI], xv[KI];
  const __nv_bfloat16* gp = G + ((int64_t)j * b + i0 + g) * b + k0;
  uint32_t c_out = 0;
  if (GATHER) {
    uint4 ci[KI][2];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      ci[i][0] = ld_u4(idx + j * b + k0 + 32 * i);
      ci[i][1] = ld_u4(idx + j * b + k0 + 32 * i + 4);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        ga[r][i] = ld_u4(gp + 16 * r * b + 32 * i);
        gb[r][i] = ld_u4(gp + (16 * r + 8) * b + 32 * i);
      }
    const __nv_bfloat16* x = in + (int64_t)min(g, few - 1) * width;
    uint32_t e[KI][8];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const uint32_t c[8] = {ci[i][0].x, ci[i][0].y, ci[i][0].z, ci[i][0].w,
                             ci[i][1].x, ci[i][1].y, ci[i][1].z, ci[i][1].w};
#pragma unroll
      for (int q = 0; q < 8; ++q) e[i][q] = ld_u16(x + min(c[q], (uint32_t)width - 1));
    }
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      xv[i] = make_uint4(e[i][0] | e[i][1] << 16, e[i][2] | e[i][3] << 16,
                         e[i][4] | e[i][5] << 16, e[i][6] | e[i][7] << 16);
      if (save && i0 == 0 && g < few)
        *reinterpret_cast<uint4*>(save + (int64_t)g * width + j * b + k0 + 32 * i) = xv[i];
    }
  } else {
    c_out = ld_u32(idx + j * b + i0 + (threadIdx.x & 15));
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        ga[r][i] = ld_u4(gp + 16 * r * b + 32 * i);
        gb[r][i] = ld_u4(gp + (16 * r + 8) * b + 32 * i);
      }
    pdl_trigger();
    pdl_wait();
    const __nv_bfloat16* w =
        (two ? few_row(in, lo, g, T, width) : in + (int64_t)min(g, few - 1) * width) + j * b + k0;
#pragma unroll
    for (int i = 0; i < KI; ++i) xv[i] = ld_u4(w + 32 * i);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const uint4 a = ga[r][i], c = gb[r][i];
      mma16816(acc, a.x, c.x, a.y, c.y, xv[i].x, xv[i].y);
      mma16816(acc, a.z, c.z, a.w, c.w, xv[i].z, xv[i].w);
    }
    red[r][warp][2 * t][g] = acc[0];
    red[r][warp][2 * t + 1][g] = acc[1];
    red[r][warp][2 * t][g + 8] = acc[2];
    red[r][warp][2 * t + 1][g + 8] = acc[3];
  }
  __syncthreads();
  const int ot = threadIdx.x >> 4, row = threadIdx.x & 15;  // an output of each row tile
  if (ot >= few) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kBdWarps; ++w) v += red[r][w][ot][row];
    if (!GATHER && two) {
#pragma unroll
      for (int w = 0; w < kBdWarps; ++w) v += red[r][w][ot + 4][row];
    }
    const uint32_t c =
        GATHER ? (uint32_t)(j * b + i0 + 16 * r + row) : min(c_out, (uint32_t)width - 1);
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    out[(int64_t)ot * width + c] = hi;
    if (GATHER && two)
      lo[(int64_t)ot * width + c] = lo_part(v, hi);
  }
}

template <typename E, int GS, int MAXW>
cudaError_t merge_pairs_t(const void* W0, const int32_t* pR, const int32_t* pP, uint8_t* codes,
                          void* scales, int m, int n, cudaStream_t s) {
  auto kern = k_merge_q4_pairs<E, GS, MAXW>;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  // two rows as they come, for bf16 interleaved as well
  const size_t smem = (sizeof(E) == 2 ? 4 : 2) * (size_t)n * sizeof(E);
  const int threads = (n / 8 + MAXW * 32 - 1) / (MAXW * 32) * 32;
  // as many CTAs as an SM holds, so that all run at once (one more a SM: 5120 x 5120 bf16 30.1 us
  // against 25.3)
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  per_sm = per_sm < 1 ? 1 : per_sm;
  int grid = num_sms() * per_sm;
  if (grid > (m + 1) / 2) grid = (m + 1) / 2;
  begin_launch("quant", s);
  kern<<<grid, threads, smem, s>>>(static_cast<const E*>(W0), pR, pP, codes,
                                   static_cast<__nv_bfloat16*>(scales), m, n);
  end_launch("quant", s);
  return cudaGetLastError();
}

template <typename E, int GS>
cudaError_t merge_t(const void* W0, const int32_t* pR, const int32_t* pP, uint8_t* codes,
                    void* scales, int m, int n, cudaStream_t s) {
  // pairs of rows: at most 4 code words a thread (n <= 16384)
  const int words = n / 8;
  if (words <= 4 * 512)
    return words <= 512    ? merge_pairs_t<E, GS, 1>(W0, pR, pP, codes, scales, m, n, s)
           : words <= 1024 ? merge_pairs_t<E, GS, 2>(W0, pR, pP, codes, scales, m, n, s)
                           : merge_pairs_t<E, GS, 4>(W0, pR, pP, codes, scales, m, n, s);
  const size_t smem = (size_t)n * sizeof(E);
  if (smem > (size_t)kMaxRowBytes) return cudaErrorInvalidValue;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_merge_q4<E, GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowBytes);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  int grid = num_sms() * 4;
  if (grid > m) grid = m;
  begin_launch("quant", s);
  k_merge_q4<E, GS><<<grid, kThreads, smem, s>>>(static_cast<const E*>(W0), pR, pP, codes,
                                                 static_cast<__nv_bfloat16*>(scales), m, n);
  end_launch("quant", s);
  return cudaGetLastError();
}

template <typename E, int GS>
cudaError_t dequant_t(const uint8_t* codes, const void* scales, void* out, int m, int n,
                      cudaStream_t s) {
  const dim3 grid((unsigned)((4ll * m + kThreads - 1) / kThreads),
                  (unsigned)(n / 128 < 65535 ? n / 128 : 65535));
  begin_launch("quant", s);
  k_dequant_q4<E, GS><<<grid, kThreads, 0, s>>>(
      codes, static_cast<const __nv_bfloat16*>(scales), static_cast<E*>(out), m, n);
  end_launch("quant", s);
  return cudaGetLastError();
}

template <int GS, int WARPS, int NT, bool LAYER>
cudaError_t rows_t(const Q4Weight& w, const void* x, void* y, const void* x_lo, void* y_lo, int T,
                   cudaStream_t s) {
  using B = __nv_bfloat16;
  begin_launch("gemm_w0", s);
  const cudaError_t e = launch_pdl(
      k_q4_rows<GS, WARPS, NT, LAYER>, dim3((w.m + 15) / 16), dim3(32 * WARPS),
      kRowD * WARPS * 1024, s, w.codes, static_cast<const uint16_t*>(w.scales),
      static_cast<const B*>(x), static_cast<B*>(y), static_cast<const B*>(x_lo),
      static_cast<B*>(y_lo), T, w.m, w.n);
  end_launch("gemm_w0", s);
  return e;
}
template <int GS, int NT, bool LAYER>
cudaError_t rows_layer(const Q4Weight& w, const void* x, void* y, const void* x_lo, void* y_lo,
                       int T, cudaStream_t s) {
  // Eight warps share a row tile where four would leave fewer than 16 warps on an SM (5120 x 5120:
  // 6.6 us against 9.4; 13824 x 5120: 12.6 against 11.6); with 16 tokens, at 128 registers a
  // thread, where two such CTAs an SM hold all tiles (5120 x 5120: 12.4 against 11.3 in two rounds;
  // 4096 x 4096: 6.4).
  if ((w.m + 15) / 16 <= (NT == 1 ? 4 * num_sms() - 1 : 2 * num_sms()))
    return rows_t<GS, 8, NT, LAYER>(w, x, y, x_lo, y_lo, T, s);
  return rows_t<GS, 4, NT, LAYER>(w, x, y, x_lo, y_lo, T, s);
}
template <int GS>
cudaError_t rows8(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  return rows_layer<GS, 1, false>(w, x, y, nullptr, nullptr, T, s);
}
template <int GS>
cudaError_t rows16(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  return rows_layer<GS, 2, false>(w, x, y, nullptr, nullptr, T, s);
}

template <int GS>
cudaError_t cols8(const Q4Weight& w, const void* dy, void* dx, int T, cudaStream_t s) {
  const int tiles = w.n / 128, nsteps = (w.m + 15) / 16;
  // shares: a grid within one wave of two CTAs an SM with a seventh of the places to spare (a
  // cluster needs all its places in one group of SMs; clusters of 7 pack worst).  5120 x 5120, T =
  // 1: 21.8 us with 1 share, 10.7 with 3, 9.2 with 6, 13.0 with 8 (two waves).
  int64_t splits = num_sms() * 17ll / (10ll * tiles);
  if (splits == 7) splits = 6;
  if (splits > nsteps / kColWarps) splits = nsteps / kColWarps;
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
  const int per = (int)((nsteps + splits - 1) / splits);
  splits = (nsteps + per - 1) / per;  // every share has a step
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, (unsigned)splits);
  cfg.blockDim = dim3(32 * kColWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)splits;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  begin_launch("gemm_w0", s);
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, w.m % 16 == 0 ? k_q4_cols<GS, true> : k_q4_cols<GS, false>, w.codes,
      static_cast<const uint16_t*>(w.scales), static_cast<const __nv_bfloat16*>(dy),
      static_cast<__nv_bfloat16*>(dx), T, w.m, w.n, per);
  end_launch("gemm_w0", s);
  return e;
}

template <int KI, int RT, bool GATHER>
cudaError_t bd_t(const void* G, const void* in, void* out, void* lo, void* save,
                 const int32_t* idx, int T, int width, cudaStream_t s) {
  using B = __nv_bfloat16;
  begin_launch("gemm_blockdiag", s);
  const cudaError_t e =
      launch_pdl(k_bd_rows<KI, RT, GATHER>, dim3(width / (16 * RT), (T + 7) / 8),
                 dim3(32 * kBdWarps), 0, s,
                 static_cast<const B*>(G), static_cast<const B*>(in), static_cast<B*>(out),
                 static_cast<B*>(lo), static_cast<B*>(save), idx, T, width);
  end_launch("gemm_blockdiag", s);
  return e;
}
template <bool GATHER>
cudaError_t bd(const void* G, const void* in, void* out, void* lo, void* save, const int32_t* idx,
               int T, int width, int b, cudaStream_t s) {
  // The gather takes two tiles of rows a CTA: half the 2-byte reads of x (8 tokens at 5120 x 5120,
  // b = 256: layer 18.8 us against 16.0; one token 12.4 against 12.6).
  constexpr int RT = GATHER ? 2 : 1;
  switch (b) {
    case 128: return bd_t<1, RT, GATHER>(G, in, out, lo, save, idx, T, width, s);
    case 256: return bd_t<2, RT, GATHER>(G, in, out, lo, save, idx, T, width, s);
    case 512: return bd_t<4, RT, GATHER>(G, in, out, lo, save, idx, T, width, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_merge_q4(const void* W0, const int32_t* perm_R, const int32_t* perm_P,
                            const Q4Weight& w, int elem_bytes, cudaStream_t s) {
  if (w.m <= 0 || w.n <= 0) return cudaSuccess;
  uint8_t* c = const_cast<uint8_t*>(w.codes);
  void* sc = const_cast<void*>(w.scales);
#define Q4_MERGE(E)                                                                        \
  (w.group == 32   ? merge_t<E, 32>(W0, perm_R, perm_P, c, sc, w.m, w.n, s)                \
   : w.group == 64 ? merge_t<E, 64>(W0, perm_R, perm_P, c, sc, w.m, w.n, s)                \
                   : merge_t<E, 128>(W0, perm_R, perm_P, c, sc, w.m, w.n, s))
  return elem_bytes == 2 ? Q4_MERGE(uint16_t) : Q4_MERGE(uint32_t);
#undef Q4_MERGE
}

cudaError_t launch_dequant_q4(const Q4Weight& w, void* out, int elem_bytes, cudaStream_t s) {
  if (w.m <= 0 || w.n <= 0) return cudaSuccess;
#define Q4_DEQ(E)                                                       \
  (w.group == 32   ? dequant_t<E, 32>(w.codes, w.scales, out, w.m, w.n, s)  \
   : w.group == 64 ? dequant_t<E, 64>(w.codes, w.scales, out, w.m, w.n, s)  \
                   : dequant_t<E, 128>(w.codes, w.scales, out, w.m, w.n, s))
  return elem_bytes == 2 ? Q4_DEQ(__nv_bfloat16) : Q4_DEQ(float);
#undef Q4_DEQ
}

#define Q4_BY_GROUP(f)                                                            \
  (w.group == 32 ? f<32>(w, x, y, T, s) : w.group == 64 ? f<64>(w, x, y, T, s) \
                                                        : f<128>(w, x, y, T, s))
cudaError_t launch_q4_product(const Q4Weight& w, const void* x, void* y, int T, bool transpose,
                              cudaStream_t s) {
  if (T <= 0 || w.m <= 0 || w.n <= 0) return cudaSuccess;
  if (T <= 8) return transpose ? Q4_BY_GROUP(cols8) : Q4_BY_GROUP(rows8);
  if (!transpose && T <= 16) return Q4_BY_GROUP(rows16);
  return launch_umma_q4(w, x, y, T, transpose, s);
}
#undef Q4_BY_GROUP

cudaError_t launch_q4_few(const void* G_P, const void* G_R, const Q4Weight& w, const void* x,
                             void* y, void* U, void* V, void* V_lo, void* W, void* W_lo,
                             const int32_t* perm_P, const int32_t* perm_R, int T, int b,
                             cudaStream_t s) {
  if (T <= 0) return cudaErrorInvalidValue;
  cudaError_t e = bd<true>(G_P, x, V, V_lo, U, perm_P, T, w.n, b, s);
  if (e != cudaSuccess) return e;
  if (T <= 8)
    e = w.group == 32   ? rows_layer<32, 1, true>(w, V, W, V_lo, W_lo, T, s)
        : w.group == 64 ? rows_layer<64, 1, true>(w, V, W, V_lo, W_lo, T, s)
                        : rows_layer<128, 1, true>(w, V, W, V_lo, W_lo, T, s);
  else if (T > 16)
    e = launch_q4_product(w, V, W, T, false, s);
  else
    e = w.group == 32   ? rows_layer<32, 2, true>(w, V, W, nullptr, nullptr, T, s)
        : w.group == 64 ? rows_layer<64, 2, true>(w, V, W, nullptr, nullptr, T, s)
                        : rows_layer<128, 2, true>(w, V, W, nullptr, nullptr, T, s);
  if (e != cudaSuccess || !y) return e;
  return bd<false>(G_R, W, y, W_lo, nullptr, perm_R, T, w.m, b, s);
}

}  // namespace poetx
