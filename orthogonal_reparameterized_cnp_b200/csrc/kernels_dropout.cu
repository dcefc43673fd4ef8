// Dropout with a mask that is never stored (philox_dev.cuh): out[r, c] = keep(r, c) ? in[r, c] *
// scale : 0.  The backward is the same call on the gradient.  (Dropout fused with an index map
// runs inside the gather kernels.)
//
// Rows of whole 8-column calls (k_dropout_vec): a thread takes one call's 16 or 32 bytes at a
// time.  Other rows start anywhere inside a 16-byte vector (k_dropout): a warp takes 31 calls of a
// row, each lane makes one call, 8 columns of mask bits; lane l works on the aligned window of 8
// columns that starts `a` columns before its own call's (a: the elements by which the row starts
// past a vector), taking the missing bits from the lane below (lane 0 only lends).
//
// Bound: HBM for fp32; for bf16 the generator and the selection come close to it (14
// instructions a value at 4 bytes a value).  Measured: 32.6 us at 8192 x 5120 bf16 (0.78 of the HBM
// copy rate; 52 with a division per call and the mask as bits), 31.5 at 4096 x 5120 fp32 (0.81),
// 22.5 at 3001 x 5003 fp32 (0.82).
#include <cuda_bf16.h>

#include "philox_dev.cuh"
#include "poetx_internal.h"

namespace poetx {
namespace {

constexpr int kDropThreads = 256;

template <typename E>
__device__ __forceinline__ void drop_call(const DropArgs& d, const uint4& w,
                                          uint4 (&v)[8 * sizeof(E) / 16]) {
  if constexpr (sizeof(E) == 2) {
    v[0] = drop_bf16x8(d, v[0], w);
  } else {
    v[0] = drop_f32x4(d, v[0], w.x, w.y);
    v[1] = drop_f32x4(d, v[1], w.z, w.w);
  }
}

// cols % 8 == 0; in == out allowed.  Each CTA walks a run of rows; two calls at a time.
template <typename E>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout_vec(const E* in, E* out, int rows, int cols, int rows_per_cta, const DropArgs d) {
  constexpr int NV = 8 * sizeof(E) / 16;  // 16-byte vectors a call
  const uint32_t step = drop_step(d);
  const int calls = cols / 8;
  const int r_first = blockIdx.x * rows_per_cta;
  const int r_last = min(rows, r_first + rows_per_cta);
  // (row, call) of the thread's next call, and the step to the one after, without divisions
  int r = r_first + threadIdx.x / calls, c = threadIdx.x % calls;
  const int dr = kDropThreads / calls, dc = kDropThreads - dr * calls;
  auto next = [&]() {
    r += dr;
    c += dc;
    if (c >= calls) {
      c -= calls;
      ++r;
    }
  };
  while (r < r_last) {
    const int ra = r, ca = c;
    next();
    const int rb = r, cb = c;
    const bool two = rb < r_last;
    next();
    const uint4* pa = reinterpret_cast<const uint4*>(in + (int64_t)ra * cols) + ca * NV;
    const uint4* pb = reinterpret_cast<const uint4*>(in + (int64_t)(two ? rb : ra) * cols) +
                      (two ? cb : ca) * NV;
    uint4 va[NV], vb[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      va[i] = pa[i];
      vb[i] = pb[i];
    }
    const uint4 wa = drop_words(d, step, (uint32_t)ra, ca);
    const uint4 wb = drop_words(d, step, (uint32_t)rb, cb);
    drop_call<E>(d, wa, va);
    drop_call<E>(d, wb, vb);
    uint4* qa = reinterpret_cast<uint4*>(out + (int64_t)ra * cols) + ca * NV;
    uint4* qb = reinterpret_cast<uint4*>(out + (int64_t)rb * cols) + cb * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      qa[i] = va[i];
      if (two) qb[i] = vb[i];
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const E* in, E* out, int rows, int cols, const DropArgs d) {  // in == out allowed
  const uint32_t step = drop_step(d);
  const int lane = threadIdx.x & 31;
  const int calls = (cols + 7) / 8;
  constexpr int V = 16 / sizeof(E);
  const int sg = blockIdx.x * (kDropThreads / 32) + (threadIdx.x >> 5);  // 31 windows of the row
  if (sg * 31 > calls) return;  // (whole warps)
  const int call = sg * 31 + lane - 1;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const int64_t row = (int64_t)r * cols;
    const int a = (int)(row & 7);  // elements past an 8-element boundary
    uint32_t bits = 0;
    if (call >= 0 && call < calls) bits = drop_bits(d, drop_words(d, step, (uint32_t)r, call));
    const uint32_t below = __shfl_up_sync(~0u, bits, 1);
    // bits of columns c0 .. c0 + 7, c0 = 8 call - a
    const uint32_t win = ((below | (bits << 8)) >> (8 - a)) & 0xffu;
    const int c0 = 8 * call - a;
    if (lane > 0 && c0 < cols) {
      const E* src = in + row + c0;
      E* dst = out + row + c0;
      if (c0 >= 0 && c0 + 8 <= cols) {
        E v[8];
#pragma unroll
        for (int i = 0; i < 8 / V; ++i)
          *reinterpret_cast<uint4*>(v + i * V) = reinterpret_cast<const uint4*>(src)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = drop_one<E>(d, (win >> i) & 1u, v[i]);
#pragma unroll
        for (int i = 0; i < 8 / V; ++i)
          reinterpret_cast<uint4*>(dst)[i] = *reinterpret_cast<const uint4*>(v + i * V);
      } else {
        for (int i = 0; i < 8; ++i)
          if (c0 + i >= 0 && c0 + i < cols) dst[i] = drop_one<E>(d, (win >> i) & 1u, src[i]);
      }
    }
    __syncwarp();
  }
}

template <typename E>
void dropout_t(const DropArgs& d, const void* in, void* out, int rows, int cols, cudaStream_t s) {
  const E* i = static_cast<const E*>(in);
  E* o = static_cast<E*>(out);
  const int calls = (cols + 7) / 8;
  if (cols % 8 == 0) {
    // about 16 calls a thread, at most 16 CTAs an SM at a time
    int64_t per = (16ll * kDropThreads + calls - 1) / calls;
    const int64_t even = (rows + 8ll * num_sms() - 1) / (8ll * num_sms());
    if (per > even) per = even;
    if (per < 1) per = 1;
    k_dropout_vec<E><<<(int)((rows + per - 1) / per), kDropThreads, 0, s>>>(i, o, rows, cols,
                                                                           (int)per, d);
    return;
  }
  // warps along a row: one more window than calls
  const int gx = (calls / 31 + 1 + kDropThreads / 32 - 1) / (kDropThreads / 32);
  int64_t gy = (16ll * num_sms() + gx - 1) / gx;
  if (gy > rows) gy = rows;
  if (gy > 65535) gy = 65535;
  k_dropout<E><<<dim3(gx, (unsigned)gy), kDropThreads, 0, s>>>(i, o, rows, cols, d);
}

}  // namespace

cudaError_t launch_dropout(const DropArgs& d, const void* in, void* out, int rows, int cols,
                           int elem_bytes, cudaStream_t s) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  begin_launch("dropout", s);
  if (elem_bytes == 2)
    dropout_t<uint16_t>(d, in, out, rows, cols, s);
  else
    dropout_t<uint32_t>(d, in, out, rows, cols, s);
  end_launch("dropout", s);
  return cudaGetLastError();
}

}  // namespace poetx
