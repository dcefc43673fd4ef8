// Dropout with a mask that is never stored (philox_dev.cuh): out[r, c] = keep(r, c) ? in[r, c] *
// scale : 0.  The backward is the same call on the gradient.  (Dropout fused with an index map
// runs inside the gather kernels.)
//
// A warp takes 32 (31) mask calls of a row at a time; each lane makes one call, 8 columns of
// mask bits.  Rows of any length start anywhere inside a 16-byte vector; where they start
// `a` elements past one, lane l works on the aligned window of 8 columns that starts a columns
// before its own call's, taking the missing bits from the lane below (lane 0 only lends).
#include <cuda_bf16.h>

#include "philox_dev.cuh"
#include "poetx_internal.h"

namespace poetx {
namespace {

constexpr int kDropThreads = 256;

template <typename E>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const E* in, E* out, int rows, int cols, const DropArgs d) {  // in == out allowed
  const uint32_t step = drop_step(d);
  const int lane = threadIdx.x & 31;
  const int calls = (cols + 7) / 8;
  // windows of a row: with an offset there is one more (its last columns), 31 a warp
  const int seg = (calls + 1 + 30) / 31;  // warp segments per row
  const int64_t total = (int64_t)rows * seg;
  const int64_t warps = (int64_t)gridDim.x * (kDropThreads / 32);
  constexpr int V = 16 / sizeof(E);
  for (int64_t w = blockIdx.x * (int64_t)(kDropThreads / 32) + (threadIdx.x >> 5); w < total;
       w += warps) {
    const int r = (int)(w / seg), sg = (int)(w - (int64_t)r * seg);
    const int64_t row = (int64_t)r * cols;
    const int a = (int)(row & 7);  // elements past an 8-element boundary
    const int call = sg * 31 + lane - 1;
    uint32_t bits = 0;
    if (call >= 0 && call < calls) bits = drop_bits(d, drop_words(d, step, (uint32_t)r, call));
    const uint32_t below = __shfl_up_sync(~0u, bits, 1);
    if (lane == 0) continue;
    // bits of columns c0 .. c0 + 7, c0 = 8 call - a
    const uint32_t win = ((below | (bits << 8)) >> (8 - a)) & 0xffu;
    const int c0 = 8 * call - a;
    if (c0 >= cols) continue;
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
}

}  // namespace

cudaError_t launch_dropout(const DropArgs& d, const void* in, void* out, int rows, int cols,
                           int elem_bytes, cudaStream_t s) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  const int64_t warps = (int64_t)rows * ((cols + 7) / 8 / 31 + 1);
  int64_t grid = (warps + kDropThreads / 32 - 1) / (kDropThreads / 32);
  if (grid > (int64_t)num_sms() * 8) grid = (int64_t)num_sms() * 8;
  begin_launch("dropout", s);
  if (elem_bytes == 2)
    k_dropout<uint16_t><<<(int)grid, kDropThreads, 0, s>>>(
        static_cast<const uint16_t*>(in), static_cast<uint16_t*>(out), rows, cols, d);
  else
    k_dropout<uint32_t><<<(int)grid, kDropThreads, 0, s>>>(
        static_cast<const uint32_t*>(in), static_cast<uint32_t*>(out), rows, cols, d);
  end_launch("dropout", s);
  return cudaGetLastError();
}

}  // namespace poetx
