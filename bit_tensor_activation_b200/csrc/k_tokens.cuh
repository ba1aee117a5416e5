// k_tokens.cuh -- a bf16 row to int8 with one scale a token: the activations of a row-parallel
// product in 8-bit integers.
//
// A row is read once and stays in registers between its maximum and its codes: up to 1024 elements in one
// warp (no barrier), longer ones in a CTA.  HBM-bound: 2 bytes read and 1 written an element, 4 bytes
// written a row; 65536 rows of 1024 take 31.6 us, 6.4 TB/s (a copy: 6.55).  A few rows take 1.4 to 2.0 us,
// which is a launch and two round trips to memory.
#pragma once

#include "hq_rows.cuh"

namespace hq {

template <int NV, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 128 : kRowMaxThreads)
    quantize_tokens_kernel(const uint16_t* __restrict__ x, int ldx, long long rows, int K, int8_t* __restrict__ q,
                           int ldq, float* __restrict__ scale) {
  __shared__ float s_red[2 * kRowMaxWarps];
  grid_trigger();
  grid_wait();
  RowGroup<kWarpRow> g{s_red, 0};
  const int i = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = kWarpRow ? 32 : blockDim.x;
  const long long row = kWarpRow ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && row >= rows) return;
  const uint16_t* xr = x + row * ldx;
  int8_t* qr = q + row * ldq;
  uint4 v[NV];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = i + c * nt;
    v[c] = 8 * j < K ? load_row8(xr, j, K) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) m = amax_bits(v[c], m);
  m = g.max_u32(max(m & 0xFFFFu, m >> 16));
  const RowScale s = row_scale(m);
  if (i == 0) scale[row] = s.scale;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = i + c * nt;
    if (8 * j < K) store_codes8(qr, j, K, codes8(v[c], s.inv));
  }
}

}  // namespace hq
