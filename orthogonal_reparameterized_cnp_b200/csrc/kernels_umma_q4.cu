// Products with the 4-bit weight for some tens to hundreds of tokens (format in q4_dev.cuh), on
// tcgen05 with the weight as the M operand:
//
//   forward      D[i, t] = sum_j W[i, j] x[t, j]        A = 128 rows of W, K-major
//   transposed   D[j, t] = sum_i W[i, j] dy[t, i]       A = 128 columns of W, MN-major
//
// One CTA: 128 outputs of the weight's free axis, up to NT tokens (N of the MMA), and its share of
// the summed axis in K chunks of 64; the shares of a tile are a cluster, whose fp32 sums are added
// in rank order through distributed shared memory.  Each code is converted once per token tile,
// into a bf16 operand in shared memory, whatever the number of tokens; the accumulator is in TMEM.
//
// Roles:
//   warp 0       bulk loads of codes and scales into slots (contiguous runs, see q4_dev.cuh)
//   warp 1       TMEM allocation, MMA issue
//   warps 2 ..   the tokens' operand: one thread's TMA loads, or, where rows are not whole 16-byte
//                vectors (transposed, up to 64 tokens a tile), words put together and stored by
//                four warps
//   then         G groups that convert every G-th chunk each; then the epilogue
// A stage holds two chunks, so that the MMA thread's wait and commit (about 0.2 us of the 0.34 us a
// chunk took with a commit each, conversion aside) come once for both.
// Bound by the latency of a chunk's way (below), not by a pipe: at 5120 x 5120, group 128, 16
// tokens (transposed) take 13.8 us, 64 15.4, 128 20.1, 256 24.2; at 13824 x 5120 64 take 29.1, 128
// 39.1, 256 42.9; 53 tokens of 4999 x 4096 transposed take 28 (35 with two warps of loaders), of
// 5000 x 4096 15.
// Every wait is bounded (Params::wait_ns); a role whose wait runs out records the timeout, leaves
// its loop, waits for its own copies and meets the others.
#include <cuda.h>
#include <cuda_bf16.h>

#include "poetx_internal.h"
#include "q4_dev.cuh"
#include "umma_ptx.cuh"

namespace poetx {

// (kernels_umma2.cu) load map of a row-major bf16 matrix, 128-byte swizzle
bool umma_load_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t ld,
                   uint32_t box_cols, uint32_t box_rows);

namespace {

constexpr int kABytes = 128 * 64 * 2;

// The way of a chunk (slot, conversion, fences and barriers, MMA, commit) takes 1 to 2 us, most
// of it waiting, so many chunks have to be on their way at once: as many groups and stages as
// shared memory holds.  Two groups of four warps with three stages, two CTAs an SM: 16.5 us at 16
// tokens, 5120 x 5120, of which 11.5 remain without any conversion.
//   G <= chunks in the stages, and SLOTS a multiple of G / 2 (a slot is visited by the same two
//   groups every time), so that no wait is two phases of its barrier ahead.
template <int NT, bool TR>
struct QCfg {
  static constexpr int B = NT * 128;                      // bytes of the tokens' operand a chunk
  static constexpr int STAGES = NT <= 32 ? 4 : NT <= 128 ? 3 : 2;  // of two chunks
  static constexpr int G = NT <= 32 ? 8 : NT == 64 ? 6 : NT == 128 ? 4 : 2;
  static constexpr int GT = NT <= 64 ? 64 : NT == 128 ? 128 : 256;  // threads of a group
  // token rows that are not whole vectors: only transposed (forward rows are n % 128 == 0 long),
  // and only in tiles of up to 64 tokens, whose threads have the registers for the words
  static constexpr bool words = TR && NT <= 64;
  // warps of token loaders (TMA needs one thread; with a second warp 128 tokens of 13824 x 5120
  // take 39.4 us, with one 39.1, but 256 tokens of 5120 x 5120 24.8 with one and 24.2 with two)
  static constexpr int TW = words ? 4 : NT == 128 ? 1 : 2;
  static constexpr int first = 64 + 32 * TW;      // thread of the first group
  static constexpr int threads = first + G * GT;
  // tiles of 128 rows x 128 columns: two chunks in either direction
  static constexpr int SLOTS = NT <= 32 ? 4 : NT == 64 ? 6 : 2;
  static constexpr int CODES = 8192;
  static constexpr int SLOT = CODES + 1024;
  static constexpr int smem = 1024 + 2 * STAGES * (kABytes + B) + SLOTS * SLOT + 512;
  static constexpr int sums = NT * 132 * 4;  // overlays the stages
  static constexpr uint32_t tmem_cols = NT < 32 ? 32 : NT;
  static_assert(G <= 2 * STAGES && SLOTS % (G / 2) == 0, "phases");
  static_assert(smem <= 227 * 1024 && threads <= 1024, "resources");
  static_assert(threads >= 512, "the epilogue's warps 8 .. 15");
  static_assert(sums <= 2 * STAGES * (kABytes + B), "sums fit the stages");
  static_assert(8 * (2 * STAGES + 2 * SLOTS + 2) <= 512, "barriers");
};

struct ParamsQ {
  const uint8_t* codes;
  const uint16_t* scales;
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  int T, m, n, sg;         // sg: scales per row and block
  int K, out;              // length of the summed axis, of the output rows
  int chunks, per_cta;     // K chunks in all, per CTA (even)
  int bulk_scales;         // the scales of a tile are whole 16-byte runs
  int vec;                 // rows of x are whole 16-byte vectors
  int* err;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void bulk_load_q(uint32_t dst, const void* src, uint32_t bytes,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr));
}
__device__ __forceinline__ void named_sync_q(int id, int count) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(count) : "memory");
}
template <int NT, bool TR>
__global__ void __launch_bounds__(QCfg<NT, TR>::threads, 1)
    k_umma_q4(const __grid_constant__ CUtensorMap tmX, const ParamsQ p) {
  using C = QCfg<NT, TR>;
  constexpr int RS = C::STAGES, G = C::G, GT = C::GT;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t sA = base, sB = sA + 2 * RS * kABytes, sQ = sB + 2 * RS * C::B;
  const uint32_t sBar = sQ + C::SLOTS * C::SLOT;
  auto full_bar = [&](int s) { return sBar + 8u * s; };
  auto empty_bar = [&](int s) { return sBar + 8u * (RS + s); };
  auto qfull_bar = [&](int j) { return sBar + 8u * (2 * RS + j); };
  auto qfree_bar = [&](int j) { return sBar + 8u * (2 * RS + C::SLOTS + j); };
  const uint32_t done_bar = sBar + 8u * (2 * RS + 2 * C::SLOTS);
  const uint32_t tmem_slot = done_bar + 8u;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * 128;  // forward: rows of W; transposed: columns
  const int tok0 = blockIdx.y * NT;
  const int c_first = blockIdx.z * p.per_cta;
  // K chunks of this CTA, a whole number of pairs (the last one may lie past the sum: zeros)
  const int cnt = min(p.per_cta, (p.chunks - c_first + 1) / 2 * 2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < RS; ++s) {
      // the converter groups of its chunks; the TMA thread (and its bytes), or the token loaders
      mbar_init(full_bar(s), 2 + (!C::words || p.vec ? 1 : 32 * C::TW));
      mbar_init(empty_bar(s), 1);
    }
    for (int j = 0; j < C::SLOTS; ++j) {
      mbar_init(qfull_bar(j), 1);
      mbar_init(qfree_bar(j), 2);  // the groups that read the slot
    }
    mbar_init(done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tmem_slot - base));
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ codes and scales
    if (lane == 0) {
      int tile = 0;
      bool ok = true;
      for (; tile < cnt / 2; ++tile) {
        const int slot = tile % C::SLOTS, use = tile / C::SLOTS;
        if (!mbar_wait(qfree_bar(slot), (use & 1) ^ 1, p.err, p.wait_ns)) {
          ok = false;
          break;
        }
        const int k = (c_first + 2 * tile) * 64;
        // forward: rows row0 .. of block k / 128; transposed: rows k .. of block row0 / 128
        const int64_t row = TR ? (int64_t)blockIdx.x * p.m + k : (int64_t)(k >> 7) * p.m + row0;
        const uint32_t rows = (uint32_t)min(128, p.m - (TR ? k : row0));
        const uint32_t sbytes = p.bulk_scales ? rows * 2u * (uint32_t)p.sg : 0u;
        mbar_expect_tx(qfull_bar(slot), rows * 64u + sbytes);
        const uint32_t dst = sQ + slot * C::SLOT;
        bulk_load_q(dst, p.codes + row * 64, rows * 64u, qfull_bar(slot));
        if (sbytes) bulk_load_q(dst + C::CODES, p.scales + row * p.sg, sbytes, qfull_bar(slot));
      }
      if (!ok)  // no load may still be in flight into this CTA's shared memory when it leaves
        for (int j = (tile > C::SLOTS ? tile - C::SLOTS : 0); j < tile; ++j)
          mbar_drain_wait(qfull_bar(j % C::SLOTS), (j / C::SLOTS) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((TR ? 1u : 0u) << 15) |
                             ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
      for (int it = 0; it < cnt / 2; ++it) {
        const int s = it % RS;
        if (!mbar_wait(full_bar(s), (it / RS) & 1, p.err, p.wait_ns)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t a = sA + (2 * s + kk / 4) * kABytes, b = sB + (2 * s + kk / 4) * C::B;
          const uint32_t k4 = kk & 3;
          umma_bf16(tmem, TR ? make_desc(a + k4 * 2048, 8192, 1024) : make_desc(a + k4 * 32, 16, 1024),
                    make_desc(b + k4 * 32, 16, 1024), idesc, (it > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(empty_bar(s));
      }
      // every MMA issued here completes before TMEM and the stages are used again
      umma_commit(done_bar);
    }
  } else if (warp < 2 + C::TW) {
    // ------------------------------------------------------------ tokens
    const int tid = threadIdx.x - 64;
    if (!C::words || p.vec) {
      if (tid == 0) {
        int it = 0;
        bool ok = true;
        for (; it < cnt / 2; ++it) {
          const int st = it % RS;
          if (!mbar_wait(empty_bar(st), ((it / RS) & 1) ^ 1, p.err, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_expect_tx(full_bar(st), 2u * (uint32_t)C::B);
          const int k = (c_first + 2 * it) * 64;
          tma_load_2d(sB + 2 * st * C::B, &tmX, k, tok0, full_bar(st));
          tma_load_2d(sB + (2 * st + 1) * C::B, &tmX, k + 64, tok0, full_bar(st));
        }
        if (!ok)  // no load may still be in flight into this CTA's shared memory when it leaves
          for (int j = (it > RS ? it - RS : 0); j < it; ++j)
            mbar_drain_wait(full_bar(j % RS), (j / RS) & 1);
      }
    } else if constexpr (C::words) {
      // 8 values from any 2-byte boundary: the five aligned words around them, shifted together;
      // a run of up to 8 such pieces a thread is loaded while the run before it is stored
      constexpr int TS = 4 * C::TW, PER = NT / TS;  // tokens apart, pieces of a thread and chunk
      constexpr int RUN = PER < 8 ? PER : 8, RUNS = PER / RUN;
      // The thread's pieces are column chunk c of tokens t0, t0 + TS, ..: whole words apart, so
      // they start on the same side of a word.
      const int t0 = tid >> 3, c = tid & 7;
      const int64_t total = (int64_t)p.T * p.K, whole = total >> 1;  // values; whole words
      const int64_t row = (int64_t)(tok0 + t0) * p.K;
      const uint32_t sh = ((uint32_t)row & 1u) * 16u;
      const uint32_t* x32 = reinterpret_cast<const uint32_t*>(p.x);
      auto load = [&](int n, uint32_t (&w)[RUN][5]) {
        const int k = (c_first + n / RUNS) * 64 + 8 * c;
        const int i0 = (n % RUNS) * RUN;
        int64_t word = ((row + k) >> 1) + (int64_t)i0 * (TS / 2) * p.K;
        const bool col_on = n < cnt * RUNS && k < p.K;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          const bool on = col_on && tok0 + t0 + TS * (i0 + i) < p.T;
          const int have = on ? (int)min((int64_t)5, whole - word) : 0;
#pragma unroll
          for (int j = 0; j < 5; ++j) {
            w[i][j] = 0;
            ld_u32_if(w[i][j], x32 + word + j, j < have);
          }
          // the last value of x alone when their count is odd
          if (on && have < 5 && (total & 1)) {
#pragma unroll
            for (int j = 0; j < 5; ++j) ld_u16_if(w[i][j], p.x + total - 1, word + j == whole);
          }
          word += TS / 2 * (int64_t)p.K;
        }
      };
      bool ok = true;
      auto put = [&](int n, const uint32_t (&w)[RUN][5]) {
        const int it = n / RUNS, st = (it >> 1) % RS;
        if (n % (2 * RUNS) == 0)
          ok = ok && mbar_wait(empty_bar(st), (((it >> 1) / RS) & 1) ^ 1, p.err, p.wait_ns);
        if (!ok) return;
        const uint32_t dst = sB + (2 * st + (it & 1)) * C::B;
        const int k0 = (c_first + it) * 64;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          const int tok = t0 + TS * ((n % RUNS) * RUN + i), k = k0 + 8 * c;
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = __funnelshift_r(w[i][j], w[i][j + 1], sh);
            // values past the end of the row
            if (k + 2 * j + 1 >= p.K) v[j] &= k + 2 * j < p.K ? 0xffffu : 0u;
          }
          sts128(dst + tok * 128 + ((c ^ (tok & 7)) << 4), v[0], v[1], v[2], v[3]);
        }
        if (n % (2 * RUNS) == 2 * RUNS - 1) {  // both chunks of the stage are written
          fence_async_smem();
          mbar_arrive(full_bar(st));
        }
      };
      uint32_t wa[RUN][5], wb[RUN][5];
      load(0, wa);
      for (int n = 0; n < cnt * RUNS; n += 2) {  // (cnt is even)
        load(n + 1, wb);
        put(n, wa);
        load(n + 2, wa);
        put(n + 1, wb);
      }
    }
  } else {
    // ------------------------------------------------------------ codes -> bf16 operand
    // group g converts chunks it = g, g + G, .. (q4_convert)
    const int grp = ((int)threadIdx.x - C::first) / GT;
    const int gt = ((int)threadIdx.x - C::first) % GT;
    const int bar_id = 1 + grp;
    const uint32_t sg = (uint32_t)p.sg;
    bool ok = true;
    for (int it = grp; it < cnt; it += G) {
      const int s = (it >> 1) % RS;
      const int tile = it >> 1, slot = tile % C::SLOTS, use = tile / C::SLOTS;
      const int k = (c_first + it) * 64;
      // (every thread of a group goes through every chunk, so that the group's barrier always
      // meets; once a wait has run out the others end at once, and nothing more is announced)
      ok = ok && mbar_wait(qfull_bar(slot), use & 1, p.err, p.wait_ns) &&
           mbar_wait(empty_bar(s), (((it >> 1) / RS) & 1) ^ 1, p.err, p.wait_ns);
      const uint32_t dst = sA + (2 * s + (it & 1)) * kABytes;
      // forward: the chunk is half of the tile's columns; rows past the weight's end give outputs
      // that are not stored.  transposed: it is half of the tile's rows; rows past the end of the
      // sum have to give zeros.
      const uint32_t first = TR ? 64u * ((uint32_t)it & 1u) : 0u;  // row of the tile
      const uint32_t src = sQ + slot * C::SLOT + first * 64u;
      const uint32_t ssrc = sQ + slot * C::SLOT + C::CODES + first * sg * 2u;
      const int rows = TR ? min(64, p.m - k) : min(128, p.m - row0);
      if (!ok) {
      } else if (p.bulk_scales && (!TR || rows == 64)) {
        q4_convert<TR ? 64 : 128, GT, true>(src, ssrc, dst, gt, (uint32_t)it & 1u, sg, rows,
                                            nullptr);
      } else {
        // (a chunk past the sum: rows <= 0, zeros; its scales' place is the last row's)
        const int64_t row = TR ? (int64_t)blockIdx.x * p.m + min(k, p.m - 1)
                               : (int64_t)(k >> 7) * p.m + row0;
        q4_convert<TR ? 64 : 128, GT, false>(src, ssrc, dst, gt, (uint32_t)it & 1u, sg, rows,
                                             p.bulk_scales ? nullptr : p.scales + row * p.sg);
      }
      fence_async_smem();  // the generic-proxy stores, then the tensor core's reads
      named_sync_q(bar_id, GT);
      if (gt == 0 && ok) {
        mbar_arrive(full_bar(s));
        mbar_arrive(qfree_bar(slot));
      }
    }
  }
  __syncthreads();  // every role has left; its copies have landed
  // ------------------------------------------------------------ sums
  // (without a timeout every MMA of this CTA completes; with one the sums mean nothing, and the
  // wait below covers the MMAs that were issued)
  int done = 0;
  if (warp >= 8 && warp < 16) {
    if (lane == 0) done = mbar_wait(done_bar, 0, p.err, p.wait_ns) ? 1 : 0;
    done = __shfl_sync(0xffffffffu, done, 0);
  }
  if (warp == 1 && lane == 0) mbar_drain_wait(done_bar, 0);
  __syncthreads();
  float* buf = reinterpret_cast<float*>(gbase);  // [NT][132]
  constexpr int LD = 132;
  if (done) {  // warps 8 .. 15
    tc_fence_after();
    const int q = warp & 3, half = (warp - 8) >> 2;
#pragma unroll
    for (int c = 0; c < NT / 2; c += 8) {
      const int col = half * (NT / 2) + c;
      uint32_t v[8];
      tmem_ld8(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)col, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 8; ++e) buf[(col + e) * LD + q * 32 + lane] = __uint_as_float(v[e]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::tmem_cols);
  }
  auto store = [&](int tok, int c, float v) {
    if (tok0 + tok < p.T && row0 + c < p.out)
      p.y[(int64_t)(tok0 + tok) * p.out + row0 + c] = __float2bfloat16_rn(4.f * v);
  };
  const int splits = gridDim.z;
  if (splits == 1) {
    for (int o = threadIdx.x; o < NT * 128; o += C::threads)
      store(o >> 7, o & 127, buf[(o >> 7) * LD + (o & 127)]);
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
  const uint32_t local = smem_u32(buf);
  const int toks = min(NT, p.T - tok0);
  for (int o = (int)blockIdx.z * C::threads + threadIdx.x; o < toks * 128; o += splits * C::threads) {
    float v = 0.f;
    for (int q = 0; q < splits; ++q) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(addr) : "r"(local + 4u * (uint32_t)((o >> 7) * LD + (o & 127))), "r"(q));
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

template <int NT, bool TR>
cudaError_t launch_q(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  using C = QCfg<NT, TR>;
  auto kern = k_umma_q4<NT, TR>;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  ParamsQ p;
  p.codes = w.codes;
  p.scales = static_cast<const uint16_t*>(w.scales);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.T = T;
  p.m = w.m;
  p.n = w.n;
  p.sg = 128 / w.group;
  p.K = TR ? w.m : w.n;
  p.out = TR ? w.n : w.m;
  p.chunks = (p.K + 63) / 64;
  p.bulk_scales = ((int64_t)w.m * p.sg) % 8 == 0;
  p.vec = p.K % 8 == 0;
  if (!p.vec && !C::words) return cudaErrorInvalidValue;
  p.err = device_error_flag();
  if (!p.err) return cudaErrorInvalidDevice;  // the bounded waits need the flag
  p.wait_ns = wait_limit_ns();
  const int tiles = (p.out + 127) / 128, ttiles = (T + NT - 1) / NT;
  // shares of the summed axis: a grid within one wave with a seventh of the places to spare (a
  // cluster needs all its places in one group of SMs), at least 4 chunks a share, at most 8
  const int units = (p.chunks + 1) / 2;  // pairs of chunks
  int64_t splits = (int64_t)num_sms() * 17 / 20 / ((int64_t)tiles * ttiles);
  if (splits > p.chunks / 4) splits = p.chunks / 4;
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
  if (splits == 7) splits = 6;
  const int per = (int)((units + splits - 1) / splits);
  splits = (units + per - 1) / per;  // every share has a chunk
  p.per_cta = per * 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, ttiles, (unsigned)splits);
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = (unsigned)splits;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  CUtensorMap mx = {};
  if (p.vec && !umma_load_map(&mx, x, T, p.K, p.K, 64u, (uint32_t)NT)) return cudaErrorInvalidValue;
  begin_launch("gemm_w0", s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mx, p);
  end_launch("gemm_w0", s);
  return e;
}

template <bool TR>
cudaError_t launch_tr(const Q4Weight& w, const void* x, void* y, int T, cudaStream_t s) {
  if constexpr (TR) {  // (forward, up to 16 tokens never come here)
    if (T <= 16) return launch_q<16, TR>(w, x, y, T, s);
  }
  if (T <= 32) return launch_q<32, TR>(w, x, y, T, s);
  // (rows that the loader threads put together: small token tiles)
  if (T <= 64 || (TR && w.m % 8 != 0)) return launch_q<64, TR>(w, x, y, T, s);
  if (T <= 128) return launch_q<128, TR>(w, x, y, T, s);
  return launch_q<256, TR>(w, x, y, T, s);
}

}  // namespace

cudaError_t launch_umma_q4(const Q4Weight& w, const void* x, void* y, int T, bool transpose,
                           cudaStream_t s) {
  // (gridDim.y counts tiles of 64 or more tokens: 2^21 tokens a launch)
  constexpr int kMost = 1 << 21;
  const int64_t in = transpose ? w.m : w.n, out = transpose ? w.n : w.m;
  for (int64_t t0 = 0; t0 < T; t0 += kMost) {
    const char* xs = static_cast<const char*>(x) + t0 * in * 2;
    char* ys = static_cast<char*>(y) + t0 * out * 2;
    const int now = T - t0 < kMost ? (int)(T - t0) : kMost;
    const cudaError_t e =
        transpose ? launch_tr<true>(w, xs, ys, now, s) : launch_tr<false>(w, xs, ys, now, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace poetx
