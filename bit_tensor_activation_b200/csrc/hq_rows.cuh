// hq_rows.cuh -- one row held in registers by a warp or by a whole CTA: loads, reductions, and the
// quantization of a row to int8 with one scale (sm_100a).
//
// A row of n elements is cut into vectors of 8; thread i of the row's threads holds vectors
// i, i + nt, i + 2 nt, ... (nt threads, at most NV vectors each), so that neighbouring threads load
// neighbouring 16-byte pieces.  Elements at or beyond n read as 0 and are not written.
#pragma once

#include "hq_common.cuh"

namespace hq {

constexpr int kRowMaxThreads = 1024;
constexpr int kRowMaxWarps = kRowMaxThreads / 32;

// The threads that share one row: one warp (kWarpRow) or the CTA.
template <bool kWarpRow>
struct RowGroup {
  float* red;  // kRowMaxWarps floats of shared memory for the CTA's reductions, two sets taken in turn
  int turn;

  // Both reductions return the same value to every thread, from one fixed order of operations.
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    if (kWarpRow) return v;
    float* r = red + (turn++ & 1) * kRowMaxWarps;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? r[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
  }
  __device__ __forceinline__ uint32_t max_u32(uint32_t v) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (kWarpRow) return v;
    uint32_t* r = reinterpret_cast<uint32_t*>(red + (turn++ & 1) * kRowMaxWarps);
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, lane < nw ? r[lane] : 0u);
  }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest |x| of eight bf16 values, as 15-bit patterns in both halves of a word (the order of
// non-negative bf16 patterns is the order of their values; 0x7F80 and above: infinity or NaN).
__device__ __forceinline__ uint32_t amax_bits(const uint4& v, uint32_t m) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  m = max_u16x2(max_u16x2(m, v.x & kAbs), v.y & kAbs);
  return max_u16x2(max_u16x2(m, v.z & kAbs), v.w & kAbs);
}

// Scale of a row whose largest |x| has the bf16 pattern `bits`, and the factor of its codes.
// Infinity or NaN in the row: scale NaN, codes 0, so that whatever the row is multiplied into is
// NaN.  A scale that would be zero or subnormal: scale 1, codes 0.
struct RowScale {
  float scale, inv;
};
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  if (bits >= 0x7F80u) return RowScale{__uint_as_float(0x7FC00000u), 0.0f};
  const float amax = __uint_as_float(bits << 16);
  const float s = __fdiv_rn(amax, 127.0f);
  if (s < 1.17549435e-38f) return RowScale{1.0f, 0.0f};
  return RowScale{s, __fdiv_rn(127.0f, amax)};
}

// rint(127 x / amax), half to even, of the exact quotient, as a number n + 1.5 * 2^23 whose low
// byte is n in two's complement.  t = x * inv is off from the quotient by at most 2^-23 of it (two
// roundings).  With x and amax bf16 (8-bit significands), a quotient that is not a half-integer is
// at least 1 / (254 * 255) > 2^-16 of itself away from every half-integer: 127 * 2 * x - (2h) * amax
// is a nonzero multiple of the two's smallest unit.  So t is first rounded to 20 significant bits
// (off by at most 2^-20 of it): that takes a t beside a half-integer onto it, and no other t onto or
// across one, and the rounding that follows ties where the exact quotient does.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  const uint32_t t = (__float_as_uint(__fmul_rn(x, inv)) + 8u) & ~15u;
  return __float_as_uint(__fadd_rn(__uint_as_float(t), 12582912.0f));
}
// Eight codes of a vector in two words.  A row of scale NaN or 1 has inv = 0: x * 0 is 0 or NaN, and
// `zero` clears it.
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  if (inv == 0.0f) return make_uint2(0u, 0u);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code_bits(bf16_at(v, i), inv);
  uint2 r;
  r.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return r;
}

// Vector j (elements 8j .. 8j+7) of a bf16 row of n elements; what lies at or beyond n reads as 0
// and is not touched in memory.
__device__ __forceinline__ uint4 load_row8(const uint16_t* __restrict__ row, int j, int n) {
  if (8 * j + 8 <= n) return ld_dep_stream16(row + 8 * j);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  for (int i = 0; 8 * j + i < n; ++i) w[i >> 1] |= ld_dep(row + 8 * j + i) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_codes8(int8_t* __restrict__ row, int j, int n, uint2 c) {
  if (8 * j + 8 <= n) {
    *reinterpret_cast<uint2*>(row + 8 * j) = c;
    return;
  }
  for (int i = 0; 8 * j + i < n; ++i) row[8 * j + i] = (int8_t)(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu);
}

}  // namespace hq
