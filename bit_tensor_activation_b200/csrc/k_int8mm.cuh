// k_int8mm.cuh -- the row-parallel product in 8-bit integers, rank by rank: int8 activations with one
// scale a token times int8 weights with one scale a channel, leaving as the partial sum [P][T][H] or
// as the hybrid wire of that partial sum.
//
//   acc = sum_k a[r][t][k] * w[r][n][k]           exact: |acc| <= 128^2 K <= 2^30 for K <= 65536
//   v   = (float(acc) * a_scale[r][t]) * w_scale[r][n] (+ bias[r][n]), one rounding a step
#pragma once

#include "hq_common.cuh"

namespace hq {

struct MmArgs {
  const int8_t* a;
  const float* a_scale;
  int lda;
  const int8_t* w;
  const float* w_scale;
  int ldw;
  int P, T, H, K;
  // the partial sum
  const uint16_t* bias;
  void* out;
  int ldo;
  // the wire
  int k;
  const int32_t* rest_idx;
  const float* inv_scale;
  const uint8_t* zero;
  uint32_t* codes;
  uint16_t* side;
};

enum MmOut { kMmBf16 = 0, kMmF32 = 1, kMmWire = 2 };

// The wire's parameters of compact column c (feature rest_idx[c]) of rank r.
struct WireCol {
  float inv;
  int lo;  // -zero; the codes' range before the zero point is added is [lo, lo + 15]
};
__device__ __forceinline__ WireCol wire_col(const MmArgs& p, int r, int c) {
  const int h = checked_col(p.rest_idx, c, p.H);
  const size_t at = (size_t)r * p.H + h;
  return WireCol{__ldg(p.inv_scale + at), -(int)__ldg(p.zero + at)};
}
__device__ __forceinline__ uint32_t wire_code(float x, const WireCol& w) {
  const int c = __float2int_rn(__fmul_rn(x, w.inv));  // saturating; NaN -> 0
  return (uint32_t)(min(max(c, w.lo), w.lo + 15) - w.lo);
}

__device__ __forceinline__ float mm_value(int acc, float sa, float sw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), sa), sw);
}

constexpr int kMmSimpleTile = 64, kMmSimpleK = 64;

__device__ __forceinline__ uint32_t mm_load4(const int8_t* __restrict__ row, int k, int K) {
  if (k + 4 <= K) return *reinterpret_cast<const uint32_t*>(row + k);
  uint32_t w = 0;
  for (int i = 0; k + i < K; ++i) w |= (uint32_t)(uint8_t)row[k + i] << (8 * i);
  return w;
}

template <int kOut>
__global__ void __launch_bounds__(256) int8_matmul_simple_kernel(const MmArgs p) {
  __shared__ uint32_t sa[kMmSimpleTile][kMmSimpleK / 4 + 1], sb[kMmSimpleTile][kMmSimpleK / 4 + 1];
  const int n0 = blockIdx.x * kMmSimpleTile, t0 = blockIdx.y * kMmSimpleTile, r = blockIdx.z;
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;  // 8 x 32: 8 columns and 2 rows a thread
  int acc[2][8] = {};
  for (int k0 = 0; k0 < p.K; k0 += kMmSimpleK) {
    for (int i = threadIdx.x; i < kMmSimpleTile * kMmSimpleK / 4; i += 256) {
      const int row = i / (kMmSimpleK / 4), c = i % (kMmSimpleK / 4), k = k0 + 4 * c;
      sa[row][c] = t0 + row < p.T && k < p.K ? mm_load4(p.a + ((size_t)r * p.T + t0 + row) * p.lda, k, p.K) : 0u;
      sb[row][c] = n0 + row < p.H && k < p.K ? mm_load4(p.w + ((size_t)r * p.H + n0 + row) * p.ldw, k, p.K) : 0u;
    }
    __syncthreads();
    for (int c = 0; c < kMmSimpleK / 4; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[i][j] = __dp4a((int)sa[ty * 2 + i][c], (int)sb[tx * 8 + j][c], acc[i][j]);
    __syncthreads();
  }
  const int n = n0 + tx * 8;
  if (n >= p.H) return;
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + ty * 2 + i;
    if (t >= p.T) return;
    const size_t row = (size_t)r * p.T + t;
    const float s = __ldg(p.a_scale + row);
    float v[8];
    for (int j = 0; j < 8; ++j) {
      v[j] = mm_value(acc[i][j], s, __ldg(p.w_scale + (size_t)r * p.H + n + j));
      if (kOut != kMmWire && p.bias) v[j] = __fadd_rn(v[j], bf16_lo(__ldg(p.bias + (size_t)r * p.H + n + j)));
    }
    if (kOut == kMmF32) {
      for (int j = 0; j < 8; ++j) static_cast<float*>(p.out)[row * p.ldo + n + j] = v[j];
      continue;
    }
    uint32_t b[4];
    for (int j = 0; j < 4; ++j) b[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    if (kOut == kMmBf16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.ldo + n) = make_uint4(b[0], b[1], b[2], b[3]);
      continue;
    }
    const int Hr = p.H - p.k;
    if (n < Hr) {
      uint32_t word = 0;
      for (int j = 0; j < 8; ++j)
        word |= wire_code((j & 1) ? bf16_hi(b[j / 2]) : bf16_lo(b[j / 2]), wire_col(p, r, n + j)) << (4 * j);
      p.codes[row * (Hr / 8) + n / 8] = word;
    } else {
      for (int j = 0; j < 8; ++j)
        p.side[((size_t)r * p.k + (n - Hr) + j) * p.T + t] = (uint16_t)(b[j / 2] >> (16 * (j & 1)));
    }
  }
}

}  // namespace hq
