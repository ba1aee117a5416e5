// k_tokens.cuh -- a bf16 row to int8 with one scale a token: the activations of a row-parallel
// product in 8-bit integers.
//
// A row is read once and stays in registers between its maximum and its codes, in the lanes of a part of a
// warp, of a warp or of a CTA, with up to 8 loads a lane in flight: a CTA a row with one load a thread
// reached half of the memory's rate, and a warp a row of 64 elements the rate of the launch.  HBM-bound: 2
// bytes read and 1 written an element, 4 bytes written a row; 65536 rows of 1024 take 31.8 us, 6.3 TB/s (a copy:
// 6.55), 8192 rows of 8192 36 us, 5.6 TB/s.  A few rows take 1.4 to 2.0 us, which is a launch and two round
// trips to memory.
#pragma once

#include "hq_rows.cuh"

namespace hq {

// kLanes: threads that share a row (8 or 32 lanes of a warp; 0: the CTA).
template <int NV, int kLanes>
__global__ void __launch_bounds__(kLanes ? 128 : kRowMaxThreads)
    quantize_tokens_kernel(const uint16_t* __restrict__ x, int ldx, long long rows, int K, int8_t* __restrict__ q,
                           int ldq, float* __restrict__ scale) {
  __shared__ float s_red[2 * kRowMaxWarps];
  grid_trigger();
  grid_wait();
  RowGroup<kLanes != 0> g{s_red, 0};
  const int i = kLanes ? threadIdx.x % (kLanes ? kLanes : 1) : threadIdx.x;
  const int nt = kLanes ? kLanes : blockDim.x;
  const long long row = kLanes ? (long long)blockIdx.x * (128 / (kLanes ? kLanes : 1)) + threadIdx.x / (kLanes ? kLanes : 1)
                               : blockIdx.x;
  const bool live = row < rows;
  if (kLanes == 32 && !live) return;  // the whole warp; the lanes of 8 stay for their warp's shuffles
  const uint16_t* xr = x + row * ldx;
  int8_t* qr = q + row * ldq;
  uint4 v[NV];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = i + c * nt;
    v[c] = live && 8 * j < K ? load_row8(xr, j, K) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) m = amax_bits(v[c], m);
  m = max(m & 0xFFFFu, m >> 16);
  if constexpr (kLanes == 8) {
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  } else {
    m = g.max_u32(m);
  }
  if (!live) return;
  const RowScale s = row_scale(m);
  if (i == 0) scale[row] = s.scale;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = i + c * nt;
    if (8 * j < K) store_codes8(qr, j, K, codes8(v[c], s.inv));
  }
}

}  // namespace hq
