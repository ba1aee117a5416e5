// k_norm.cuh -- the end of a block after its compressed sum: the block's output normalised and
// gated, added to the scaled residual, and the next block's norm of the new residual, as bf16 or as
// int8 with one scale a token.
//
//   u  = norm_post(y)                     (none, RMS or layer norm; weight, layer norm's bias)
//   r' = alpha * r + beta * gate * u      stored in the residual's type
//   h  = norm_pre(r')                     of the stored r', so a later reader of r' sees what was normed
//
// A row is read once: it stays in registers through both norms, with sums in fp32 and a layer norm's
// squares summed about the mean (no cancellation).  HBM-bound: y, r, r' and h, each once.
#pragma once

#include "hq_rows.cuh"

namespace hq {

struct NormArgs {
  const void* y;
  const void* res;
  void* res_out;
  int T, H;
  int post, pre;  // hq_norm_kind
  const float* post_w;
  const float* post_b;
  const uint16_t* gate;  // NULL: 1
  int gate_rows;
  float alpha, beta;
  const float* pre_w;
  const float* pre_b;
  float eps;
  uint16_t* h;
  int8_t* q;
  int ldq;
  float* q_scale;
};

template <typename T>
__device__ __forceinline__ void load_vec8(const void* base, size_t at, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = ld_stream16(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = bf16_at(v, i);
  } else {
    const uint4 a = ld_stream16(static_cast<const float*>(base) + at);
    const uint4 b = ld_stream16(static_cast<const float*>(base) + at + 4);
    f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
  }
}
__device__ __forceinline__ void load_param8(const float* __restrict__ p, int at, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + at) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The norm of the row in v, in place: kind is the same for all threads.
template <int NV, bool kWarpRow>
__device__ __forceinline__ void norm_row(RowGroup<kWarpRow>& g, float (&v)[NV][8], int kind, const float* w,
                                         const float* b, float eps, int H, int i, int nt) {
  const float inv_n = __fdiv_rn(1.0f, (float)H);
  float mean = 0.0f;
  if (kind == HQ_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fadd_rn(s, v[c][e]);
    mean = __fmul_rn(g.sum(s), inv_n);
  }
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    if (8 * (i + c * nt) >= H) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[c][e] = __fadd_rn(v[c][e], -mean);
      s = __fmaf_rn(v[c][e], v[c][e], s);
    }
  }
  const float rstd = __frsqrt_rn(__fmaf_rn(g.sum(s), inv_n, eps));
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int at = 8 * (i + c * nt);
    if (at >= H) continue;
    float f[8];
    if (w) {
      load_param8(w, at, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = __fmul_rn(__fmul_rn(v[c][e], rstd), f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = __fmul_rn(v[c][e], rstd);
    }
    if (b) {
      load_param8(b, at, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = __fadd_rn(v[c][e], f[e]);
    }
  }
}

template <typename Y, typename R, int NV, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 128 : kRowMaxThreads) residual_norm_kernel(const NormArgs a) {
  __shared__ float s_red[2 * kRowMaxWarps];
  RowGroup<kWarpRow> g{s_red, 0};
  const int i = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int row = kWarpRow ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && row >= a.T) return;
  const int H = a.H;
  const size_t base = (size_t)row * H;
  float v[NV][8], r[NV][8];
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int at = 8 * (i + c * nt);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = r[c][e] = 0.0f;
    if (at < H) {
      load_vec8<Y>(a.y, base + at, v[c]);
      load_vec8<R>(a.res, base + at, r[c]);
    }
  }
  if (a.post != HQ_NORM_NONE) norm_row<NV, kWarpRow>(g, v, a.post, a.post_w, a.post_b, a.eps, H, i, nt);
  const uint16_t* gate = a.gate ? a.gate + (size_t)(row / a.gate_rows) * H : nullptr;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int at = 8 * (i + c * nt);
    if (at >= H) continue;
    if (gate) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(gate + at));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = __fmul_rn(v[c][e], bf16_at(w, e));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = __fmaf_rn(a.alpha, r[c][e], __fmul_rn(a.beta, v[c][e]));
    if constexpr (sizeof(R) == 2) {
      const uint4 o = make_uint4(pack_bf16x2(v[c][0], v[c][1]), pack_bf16x2(v[c][2], v[c][3]),
                                 pack_bf16x2(v[c][4], v[c][5]), pack_bf16x2(v[c][6], v[c][7]));
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + base + at) = o;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = bf16_at(o, e);
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + base + at);
      o[0] = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
      o[1] = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
    }
  }
  if (a.pre == HQ_NORM_NONE) return;
  norm_row<NV, kWarpRow>(g, v, a.pre, a.pre_w, a.pre_b, a.eps, H, i, nt);
  // h as bf16, and its codes: exactly those of quantize_tokens on that bf16 row
  uint4 o[NV];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int at = 8 * (i + c * nt);
    o[c] = make_uint4(pack_bf16x2(v[c][0], v[c][1]), pack_bf16x2(v[c][2], v[c][3]), pack_bf16x2(v[c][4], v[c][5]),
                      pack_bf16x2(v[c][6], v[c][7]));
    if (at >= H) continue;
    m = amax_bits(o[c], m);
    if (a.h) *reinterpret_cast<uint4*>(a.h + base + at) = o[c];
  }
  if (!a.q) return;
  const RowScale s = row_scale(g.max_u32(max(m & 0xFFFFu, m >> 16)));
  if (i == 0) a.q_scale[row] = s.scale;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = i + c * nt;
    if (8 * j < H) store_codes8(a.q + (size_t)row * a.ldq, j, H, codes8(o[c], s.inv));
  }
}

}  // namespace hq
