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

// Codes and scales of W0[perm_R][:, perm_P] (NULL maps: identity).  One CTA per row: the source
// row is staged in shared memory, thread c owns the 8 columns of code word c (16 words a
// block), the group maximum is taken over the 4, 8 or 16 threads of a group by shuffles.
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
// scales).  Thread per code word.
template <typename E, int GS>
__global__ void __launch_bounds__(kThreads)
    k_dequant_q4(const uint8_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                 E* __restrict__ out, int m, int n) {
  const int nb = n / 128;
  const int64_t total = (int64_t)m * nb * 16;
  for (int64_t v = blockIdx.x * (int64_t)kThreads + threadIdx.x; v < total;
       v += (int64_t)gridDim.x * kThreads) {
    // 16 consecutive threads take one row's block in column order
    const int l = (int)(v & 15);
    const int64_t rb = v >> 4;
    const int i = (int)(rb / nb), blk = (int)(rb - (int64_t)i * nb);
    const int64_t r = (int64_t)blk * m + i;
    const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(codes + r * 64) +
                                4 * (l & 3) + (l >> 2));
    const float s = __bfloat162float(scales[r * (128 / GS) + l / (GS / 8)]);
    float f[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t q2 = q4_pair(word, p);
      f[2 * p] = s * bf_lo(q2);
      f[2 * p + 1] = s * bf_hi(q2);
    }
    E* o = out + (int64_t)i * n + blk * 128 + 8 * l;
    if constexpr (sizeof(E) == 2) {
      uint32_t h[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * p], f[2 * p + 1]);
        h[p] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
      reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// ---------------------------------------------------------------------------------------
// y[t, i] = sum_j W[i, j] x[t, j], few tokens.  One CTA: 16 rows of W, 8 NT tokens; the K blocks
// are dealt to the 8 warps.  Lane (g, t) loads chunk t of rows g and g + 8 (1 KB a warp and
// block, contiguous), which is its A fragment of 8 MMAs once the nibbles are bf16 integers;
// the integers are multiplied exactly, and the group's sum is scaled in fp32.
constexpr int kRowWarps = 8;

template <int NT, int GS>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_q4_rows(const uint8_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
              const __nv_bfloat16* __restrict__ x, __nv_bfloat16* __restrict__ y, int T, int m,
              int n) {
  __shared__ float red[kRowWarps][NT * 8][17];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = blockIdx.x * 16, tok0 = blockIdx.y * (8 * NT);
  const int ra = min(row0 + g, m - 1), rb = min(row0 + g + 8, m - 1);
  const int nb = n / 128;
  constexpr int SG = 128 / GS;  // scales per row and block
  float acc[NT][4];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0.f;

  for (int kb = warp; kb < nb; kb += kRowWarps) {
    const int64_t base = (int64_t)kb * m;
    const uint4 ca = __ldg(reinterpret_cast<const uint4*>(codes + (base + ra) * 64) + t);
    const uint4 cb = __ldg(reinterpret_cast<const uint4*>(codes + (base + rb) * 64) + t);
    float sa[SG], sb[SG];
#pragma unroll
    for (int h = 0; h < SG; ++h) {
      sa[h] = __bfloat162float(scales[(base + ra) * SG + h]);
      sb[h] = __bfloat162float(scales[(base + rb) * SG + h]);
    }
    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
    float part[NT][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w % (GS / 32) == 0) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[a][c] = 0.f;
      }
      uint32_t pa[4], pb[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        pa[p] = q4_pair(wa[w], p);
        pb[p] = q4_pair(wb[w], p);
      }
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        const int tok = tok0 + a * 8 + g;
        uint4 xv = make_uint4(0, 0, 0, 0);
        if (tok < T)
          xv = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)tok * n + kb * 128 + w * 32) + t);
        mma16816(part[a], pa[0], pb[0], pa[1], pb[1], xv.x, xv.y);
        mma16816(part[a], pa[2], pb[2], pa[3], pb[3], xv.z, xv.w);
      }
      if ((w + 1) % (GS / 32) == 0) {
        const float fa = sa[w / (GS / 32)], fb = sb[w / (GS / 32)];
#pragma unroll
        for (int a = 0; a < NT; ++a) {
          acc[a][0] = fmaf(fa, part[a][0], acc[a][0]);
          acc[a][1] = fmaf(fa, part[a][1], acc[a][1]);
          acc[a][2] = fmaf(fb, part[a][2], acc[a][2]);
          acc[a][3] = fmaf(fb, part[a][3], acc[a][3]);
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    red[warp][a * 8 + 2 * t][g] = acc[a][0];
    red[warp][a * 8 + 2 * t + 1][g] = acc[a][1];
    red[warp][a * 8 + 2 * t][g + 8] = acc[a][2];
    red[warp][a * 8 + 2 * t + 1][g + 8] = acc[a][3];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < NT * 8 * 16; o += 32 * kRowWarps) {
    const int tok = o >> 4, r = o & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) v += red[w][tok][r];  // fixed order
    if (tok0 + tok < T && row0 + r < m)
      y[(int64_t)(tok0 + tok) * m + row0 + r] = __float2bfloat16_rn(v);
  }
}

// ---------------------------------------------------------------------------------------
// dx[t, j] = sum_i W[i, j] dy[t, i], few tokens.  One CTA: 64 JW columns (JW code words a lane),
// 8 NT tokens; the 16-row steps of its share of the rows are dealt to the 8 warps.  Lane (g, t)
// loads words g of rows 4 t .. 4 t + 3; halves of two rows' words side by side give bf16
// pairs along the rows, which the MMA sums over.  The scale changes along the summed index, so
// it multiplies the bf16 integers (exact for scales of 5 significant bits, else rounded to
// bf16 as in the tensor-core path).
template <int NT, int JW, int GS>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_q4_cols(const uint8_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
              const __nv_bfloat16* __restrict__ dy, __nv_bfloat16* __restrict__ dx, int T, int m,
              int n, int steps_per_cta) {
  extern __shared__ __align__(16) float redc[];  // [4][8 NT][64 JW]
  constexpr int COLS = 64 * JW, TOK = 8 * NT;
  constexpr int SG = 128 / GS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tok0 = blockIdx.z * TOK;
  const int splits = gridDim.y;
  const int L0 = blockIdx.x * (8 * JW) + g * JW;  // first code word of the lane in a row
  const int blk = min(L0 >> 4, n / 128 - 1), wi0 = L0 & 15;
  const int64_t base = (int64_t)blk * m;
  const int nsteps = (m + 15) / 16;
  const int s_first = blockIdx.y * steps_per_cta;
  const int s_last = min(nsteps, s_first + steps_per_cta);
  float acc[NT][JW][4][4];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int j = 0; j < JW; ++j)
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][j][p][c] = 0.f;

  for (int ks = s_first + warp; ks < s_last; ks += kRowWarps) {
    const int i0 = ks * 16 + 4 * t;
    uint32_t wd[4][JW];
    uint16_t sc[4][JW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = base + min(i0 + r, m - 1);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + row * 64) + wi0;
      if constexpr (JW == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
        wd[r][0] = v.x; wd[r][1] = v.y; wd[r][2] = v.z; wd[r][3] = v.w;
      } else if constexpr (JW == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        wd[r][0] = v.x; wd[r][1] = v.y;
      } else {
        wd[r][0] = __ldg(src);
      }
#pragma unroll
      for (int j = 0; j < JW; ++j)
        sc[r][j] = __ldg(reinterpret_cast<const uint16_t*>(scales) + row * SG +
                         ((wi0 + j) & 3) / (GS / 32));
    }
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int tok = tok0 + a * 8 + g;
      uint16_t d[4] = {0, 0, 0, 0};
      if (tok < T) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(dy) + (int64_t)tok * m + i0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (i0 + r < m) d[r] = __ldg(src + r);
      }
      b0[a] = d[0] | ((uint32_t)d[1] << 16);
      b1[a] = d[2] | ((uint32_t)d[3] << 16);
    }
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      // rows past the end have zero dy; their clamped scale must not bring in a NaN of its own
      const uint32_t s01 = sc[0][j] | ((uint32_t)sc[1][j] << 16);
      const uint32_t s23 = sc[2][j] | ((uint32_t)sc[3][j] << 16);
      const uint32_t lo01 = __byte_perm(wd[0][j], wd[1][j], 0x5410);
      const uint32_t hi01 = __byte_perm(wd[0][j], wd[1][j], 0x7632);
      const uint32_t lo23 = __byte_perm(wd[2][j], wd[3][j], 0x5410);
      const uint32_t hi23 = __byte_perm(wd[2][j], wd[3][j], 0x7632);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t a0 = bf2_mul(q4_pair(lo01, p), s01);
        const uint32_t a1 = bf2_mul(q4_pair(hi01, p), s01);
        const uint32_t a2 = bf2_mul(q4_pair(lo23, p), s23);
        const uint32_t a3 = bf2_mul(q4_pair(hi23, p), s23);
#pragma unroll
        for (int a = 0; a < NT; ++a) mma16816(acc[a][j][p], a0, a1, a2, a3, b0[a], b1[a]);
      }
    }
  }
  // the 8 warps' sums, halves added in a fixed order; then the splits, through the cluster
  auto at = [&](int slot, int tok, int col) -> float& {
    return redc[((size_t)slot * TOK + tok) * COLS + col];
  };
  // lane's value (a, j, p, c): token a * 8 + 2 t + (c & 1), column 8 (g JW + j) + 2 p + (c >> 1)
#pragma unroll
  for (int half = 4; half >= 1; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int j = 0; j < JW; ++j)
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              at(warp - half, a * 8 + 2 * t + (c & 1), 8 * (g * JW + j) + 2 * p + (c >> 1)) =
                  acc[a][j][p][c];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int j = 0; j < JW; ++j)
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[a][j][p][c] +=
                  at(warp, a * 8 + 2 * t + (c & 1), 8 * (g * JW + j) + 2 * p + (c >> 1));
    }
    __syncthreads();
  }
  if (warp == 0) {
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int j = 0; j < JW; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            at(0, a * 8 + 2 * t + (c & 1), 8 * (g * JW + j) + 2 * p + (c >> 1)) = acc[a][j][p][c];
  }
  // word L of the row holds columns 128 (L / 16) + 32 (L % 4) + 8 ((L / 4) % 4) ..
  auto store = [&](int o, float v) {
    const int tok = o / COLS, col = o - tok * COLS;
    const int L = blockIdx.x * (8 * JW) + col / 8;
    const int j = (L >> 4) * 128 + 32 * (L & 3) + 8 * ((L >> 2) & 3) + (col & 7);
    if (tok0 + tok < T && (L >> 4) < n / 128)
      dx[(int64_t)(tok0 + tok) * n + j] = __float2bfloat16_rn(v);
  };
  if (splits == 1) {
    __syncthreads();
    for (int o = threadIdx.x; o < TOK * COLS; o += 32 * kRowWarps) store(o, redc[o]);
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int per = TOK * COLS / splits;  // (splits divides 64)
  const uint32_t local = (uint32_t)__cvta_generic_to_shared(redc);
  for (int o = (int)rank * per + threadIdx.x; o < ((int)rank + 1) * per; o += 32 * kRowWarps) {
    float v = 0.f;
    for (int q = 0; q < splits; ++q) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(addr) : "r"(local + 4u * (uint32_t)o), "r"(q));
      float f;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(addr) : "memory");
      v += f;
    }
    store(o, v);
  }
  // no CTA leaves while another still reads its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// ---------------------------------------------------------------------------------------
// Block-diagonal product of a few tokens with its index map:
//   out[t, o(jb + i)] = sum_k G_j[i, k] in[t, c(jb + k)]
// gather: c = idx (U = X[:, p_P], V_j = U_j G_P,j^T; U is also written when `save` is given);
// scatter: o = idx (Z_j = W_j G_R,j^T, Y[:, p_R[i]] = Z[:, i]).  One CTA: 16 rows of one block,
// 8 NT tokens; its four warps split k and add their sums in a fixed order.
constexpr int kBdWarps = 4;

template <int NT, bool GATHER>
__global__ void __launch_bounds__(32 * kBdWarps)
    k_bd_rows(const __nv_bfloat16* __restrict__ G, const __nv_bfloat16* __restrict__ in,
              __nv_bfloat16* __restrict__ out, __nv_bfloat16* __restrict__ save,
              const int32_t* __restrict__ idx, int T, int width, int b) {
  extern __shared__ __align__(16) unsigned char bd_raw[];
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(bd_raw);  // [8 NT][b + 8]
  __shared__ float red[kBdWarps][NT * 8][17];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tiles = b / 16;
  const int j = blockIdx.x / tiles, i0 = (blockIdx.x - j * tiles) * 16;
  const int tok0 = blockIdx.y * (8 * NT);
  const int ld = b + 8;
  for (int e = threadIdx.x; e < NT * 8 * b; e += 32 * kBdWarps) {
    const int tok = e / b, k = e - tok * b;
    __nv_bfloat16 v = __ushort_as_bfloat16(0);
    if (tok0 + tok < T) {
      unsigned c = (unsigned)(j * b + k);
      if (GATHER) {
        c = (unsigned)__ldg(idx + c);
        c = c < (unsigned)width ? c : (unsigned)width - 1;
      }
      v = in[(int64_t)(tok0 + tok) * width + c];
      if (GATHER && save && i0 == 0) save[(int64_t)(tok0 + tok) * width + j * b + k] = v;
    }
    xs[tok * ld + k] = v;
  }
  __syncthreads();
  float acc[NT][4];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0.f;
  const __nv_bfloat16* ga = G + ((int64_t)j * b + i0 + g) * b;
  const __nv_bfloat16* gb = ga + 8 * (int64_t)b;
  const int kw = b / kBdWarps;  // 32, 64 or 128
  for (int k = warp * kw; k < (warp + 1) * kw; k += 32) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(ga + k) + t);
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(gb + k) + t);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const uint4 xv = *reinterpret_cast<const uint4*>(xs + (q * 8 + g) * ld + k + 8 * t);
      mma16816(acc[q], a.x, c.x, a.y, c.y, xv.x, xv.y);
      mma16816(acc[q], a.z, c.z, a.w, c.w, xv.z, xv.w);
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    red[warp][q * 8 + 2 * t][g] = acc[q][0];
    red[warp][q * 8 + 2 * t + 1][g] = acc[q][1];
    red[warp][q * 8 + 2 * t][g + 8] = acc[q][2];
    red[warp][q * 8 + 2 * t + 1][g + 8] = acc[q][3];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < NT * 8 * 16; o += 32 * kBdWarps) {
    const int tok = o >> 4, r = o & 15;
    if (tok0 + tok >= T) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kBdWarps; ++w) v += red[w][tok][r];
    unsigned c = (unsigned)(j * b + i0 + r);
    if (!GATHER) {
      c = (unsigned)__ldg(idx + c);
      c = c < (unsigned)width ? c : (unsigned)width - 1;
    }
    out[(int64_t)(tok0 + tok) * width + c] = __float2bfloat16_rn(v);
  }
}

template <typename E, int GS>
cudaError_t merge_t(const void* W0, const int32_t* pR, const int32_t* pP, uint8_t* codes,
                    void* scales, int m, int n, cudaStream_t s) {
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
  const int64_t blocks = ((int64_t)m * (n / 8) + kThreads - 1) / kThreads;
  int grid = num_sms() * 8;
  if (grid > blocks) grid = (int)blocks;
  begin_launch("quant", s);
  k_dequant_q4<E, GS><<<grid, kThreads, 0, s>>>(
      codes, static_cast<const __nv_bfloat16*>(scales), static_cast<E*>(out), m, n);
  end_launch("quant", s);
  return cudaGetLastError();
}

template <int NT, int GS>
cudaError_t rows_t(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  begin_launch("gemm_w0", s);
  const cudaError_t e =
      launch_pdl(k_q4_rows<NT, GS>, dim3((w.m + 15) / 16, (T + 8 * NT - 1) / (8 * NT)),
                 dim3(32 * kRowWarps), 0, s, w.codes, static_cast<const __nv_bfloat16*>(w.scales),
                 static_cast<const __nv_bfloat16*>(x), static_cast<__nv_bfloat16*>(y), T, w.m,
                 w.n);
  end_launch("gemm_w0", s);
  return e;
}
template <int GS>
cudaError_t rows_gs(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  if (T <= 8) return rows_t<1, GS>(w, x, y, T, s);
  if (T <= 16) return rows_t<2, GS>(w, x, y, T, s);
  if (T <= 32) return rows_t<4, GS>(w, x, y, T, s);
  return rows_t<8, GS>(w, x, y, T, s);
}

template <int NT, int JW, int GS>
cudaError_t cols_t(const Q4Weight& w, const void* dy, void* dx, int T, cudaStream_t s) {
  auto kern = k_q4_cols<NT, JW, GS>;
  constexpr int COLS = 64 * JW, TOK = 8 * NT;
  constexpr int smem = 4 * TOK * COLS * 4;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  const int tiles = (w.n + COLS - 1) / COLS, ztiles = (T + TOK - 1) / TOK;
  const int nsteps = (w.m + 15) / 16;
  // split the rows over a cluster while the grid is below two CTAs per SM and every warp
  // keeps a step
  int splits = 1;
  while (splits < 8 && tiles * ztiles * splits < 2 * num_sms() &&
         nsteps >= 2 * splits * kRowWarps)
    splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, splits, ztiles);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = splits;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  begin_launch("gemm_w0", s);
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, kern, w.codes, static_cast<const __nv_bfloat16*>(w.scales),
      static_cast<const __nv_bfloat16*>(dy), static_cast<__nv_bfloat16*>(dx), T, w.m, w.n,
      (nsteps + splits - 1) / splits);
  end_launch("gemm_w0", s);
  return e;
}
template <int GS>
cudaError_t cols_gs(const Q4Weight& w, const void* dy, void* dx, int T, cudaStream_t s) {
  if (T <= 8) return cols_t<1, 4, GS>(w, dy, dx, T, s);
  if (T <= 16) return cols_t<2, 2, GS>(w, dy, dx, T, s);
  if (T <= 32) return cols_t<4, 1, GS>(w, dy, dx, T, s);
  return cols_t<8, 1, GS>(w, dy, dx, T, s);
}

template <int NT, bool GATHER>
cudaError_t bd_t(const void* G, const void* in, void* out, void* save, const int32_t* idx, int T,
                 int width, int b, cudaStream_t s) {
  auto kern = k_bd_rows<NT, GATHER>;
  const size_t smem = (size_t)NT * 8 * (b + 8) * 2;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NT * 8 * (512 + 8) * 2);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  begin_launch("gemm_blockdiag", s);
  const cudaError_t e = launch_pdl(
      kern, dim3(width / 16, (T + 8 * NT - 1) / (8 * NT)), dim3(32 * kBdWarps), smem, s,
      static_cast<const __nv_bfloat16*>(G), static_cast<const __nv_bfloat16*>(in),
      static_cast<__nv_bfloat16*>(out), static_cast<__nv_bfloat16*>(save), idx, T, width, b);
  end_launch("gemm_blockdiag", s);
  return e;
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

cudaError_t launch_q4_product(const Q4Weight& w, const void* x, void* y, int T, bool transpose,
                              cudaStream_t s) {
  if (T <= 0 || w.m <= 0 || w.n <= 0) return cudaSuccess;
  if (!transpose)
    return w.group == 32   ? rows_gs<32>(w, x, y, T, s)
           : w.group == 64 ? rows_gs<64>(w, x, y, T, s)
                           : rows_gs<128>(w, x, y, T, s);
  return w.group == 32   ? cols_gs<32>(w, x, y, T, s)
         : w.group == 64 ? cols_gs<64>(w, x, y, T, s)
                         : cols_gs<128>(w, x, y, T, s);
}

cudaError_t launch_bd_gather(const void* G, const void* x, void* out, void* save_u,
                             const int32_t* idx, int T, int width, int b, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (T <= 8) return bd_t<1, true>(G, x, out, save_u, idx, T, width, b, s);
  if (T <= 16) return bd_t<2, true>(G, x, out, save_u, idx, T, width, b, s);
  return bd_t<4, true>(G, x, out, save_u, idx, T, width, b, s);
}
cudaError_t launch_bd_scatter(const void* G, const void* in, void* y, const int32_t* idx, int T,
                              int width, int b, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (T <= 8) return bd_t<1, false>(G, in, y, nullptr, idx, T, width, b, s);
  if (T <= 16) return bd_t<2, false>(G, in, y, nullptr, idx, T, width, b, s);
  return bd_t<4, false>(G, in, y, nullptr, idx, T, width, b, s);
}

}  // namespace poetx
