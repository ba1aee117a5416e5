// k_norm.cuh -- the end of a block after its compressed sum: the block's output normalised and
// gated, added to the scaled residual, and the next block's norm of the new residual, as bf16 or as
// int8 with one scale a token.
//
//   u  = norm_post(y)                     (none, RMS or layer norm; weight, layer norm's bias)
//   r' = alpha * r + beta * gate * u      stored in the residual's type
//   h  = norm_pre(r')                     of the stored r', so a later reader of r' sees what was normed
//
// A row is read once: it stays in registers through both norms, with sums in fp32 and a layer norm's
// squares summed about the mean (no cancellation).  HBM-bound: y, r, r' and h, each once.  8192 x 8192 bf16
// with a gate and both weights: 98 us, 5.5 TB/s; 32 x 8192: 4.0 us, two block-wide reductions after a round
// trip to memory.  With int8 rows beside the bf16 ones 130 us (4.6 TB/s), in their place 127 (3.7): the row's
// maximum is a third reduction over the CTA, and its codes another pass over the registers.
#pragma once

#include "hq_rows.cuh"
#include "hq_tma.cuh"

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

// Eight values as they lie in memory, and as floats.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const void* base, size_t at) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
      v[i] = ld_dep_stream16(static_cast<const char*>(base) + at * sizeof(T) + 16 * i);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 2) return bf16_at(v[0], i);
    const uint4& q = v[i / 4];
    return __uint_as_float((i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w);
  }
};
// Pairs of neighbouring values throughout, for the instructions that take two at once: v[c][p] are
// elements 2p, 2p + 1 of vector c.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
template <typename T>
__device__ __forceinline__ float2 pair_of(const Raw8<T>& r, int p) { return make_float2(r.at(2 * p), r.at(2 * p + 1)); }
__device__ __forceinline__ Raw8<uint16_t> round_pairs(const float2 (&v)[4]) {
  return Raw8<uint16_t>{{make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                                    pack_bf16x2(v[3].x, v[3].y))}};
}

// The row in v less its mean (a layer norm's) and 1 / sqrt(mean square + eps) of what is then there.  Bit
// c of `in`: vector c lies within the row (kFull: all do); the others hold 0 and stay 0.
template <int NV, bool kFull, bool kWarpRow>
__device__ __forceinline__ float centre_row(RowGroup<kWarpRow>& g, float2 (&v)[NV][4], int kind, float eps, float inv_n,
                                            uint32_t in) {
  float2 s = both(0.0f);
  if (kind == HQ_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int p = 0; p < 4; ++p) s = __fadd2_rn(s, v[c][p]);
    const float mean = __fmul_rn(g.sum(__fadd_rn(s.x, s.y)), inv_n);
    s = both(0.0f);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const float2 m = both(kFull || ((in >> c) & 1u) ? -mean : 0.0f);
#pragma unroll
      for (int p = 0; p < 4; ++p) v[c][p] = __fadd2_rn(v[c][p], m);
    }
  }
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int p = 0; p < 4; ++p) s = __ffma2_rn(v[c][p], v[c][p], s);
  return __frsqrt_rn(__fmaf_rn(g.sum(__fadd_rn(s.x, s.y)), inv_n, eps));
}

// The norm of the row in v, in place, weight and bias from memory.  `at` are the places of the thread's
// vectors, moved back into the row where they lie past its end: what is computed there is finite work on
// nothing that is kept, and these loops have no condition in them.
template <int NV, bool kWarpRow>
__device__ __forceinline__ void norm_row(RowGroup<kWarpRow>& g, float2 (&v)[NV][4], int kind, const float* w,
                                         const float* b, float eps, int H, const int (&at)[NV], uint32_t in) {
  const float2 rstd = both(centre_row<NV, false, kWarpRow>(g, v, kind, eps, __fdiv_rn(1.0f, (float)H), in));
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int p = 0; p < 4; ++p) v[c][p] = __fmul2_rn(v[c][p], rstd);
  if (w) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int p = 0; p < 4; p += 2) {
        const float4 f = ld_dep(reinterpret_cast<const float4*>(w + at[c] + 2 * p));
        v[c][p] = __fmul2_rn(v[c][p], make_float2(f.x, f.y));
        v[c][p + 1] = __fmul2_rn(v[c][p + 1], make_float2(f.z, f.w));
      }
  }
  if (b) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int p = 0; p < 4; p += 2) {
        const float4 f = ld_dep(reinterpret_cast<const float4*>(b + at[c] + 2 * p));
        v[c][p] = __fadd2_rn(v[c][p], make_float2(f.x, f.y));
        v[c][p + 1] = __fadd2_rn(v[c][p + 1], make_float2(f.z, f.w));
      }
  }
}

// The new residual of one vector, stored if `here`, and back in v as it was stored (0 where it is another
// thread's).
template <typename R>
__device__ __forceinline__ void residual8(const NormArgs& a, const Raw8<R>& r, float2 (&v)[4], size_t at, bool in, bool here) {
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = __ffma2_rn(both(a.alpha), pair_of(r, p), __fmul2_rn(both(a.beta), v[p]));
  if constexpr (sizeof(R) == 2) {
    const Raw8<uint16_t> o = round_pairs(v);
    if (here) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + at) = o.v[0];
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = pair_of(o, p);
  } else if (here) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + at);
    o[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    o[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  if (!in) {
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = both(0.0f);
  }
}
__device__ __forceinline__ void gate8(const uint4& gate, float2 (&v)[4]) {
  const Raw8<uint16_t> w{{gate}};
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = __fmul2_rn(v[p], pair_of(w, p));
}

// The normed row out: as bf16, and its codes, which are those of quantize_tokens on that bf16 row.
template <int NV, bool kFull, bool kWarpRow>
__device__ __forceinline__ void store_row(RowGroup<kWarpRow>& g, const NormArgs& a, const float2 (&v)[NV][4], int row,
                                          const int (&at)[NV], uint32_t in, bool first, bool ok) {
  uint4 o[NV];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    o[c] = round_pairs(v[c]).v[0];
    if (!kFull && !((in >> c) & 1u)) continue;
    m = amax_bits(o[c], m);
    if (a.h && ok) *reinterpret_cast<uint4*>(a.h + (size_t)row * a.H + at[c]) = o[c];
  }
  if (!a.q) return;
  const RowScale s = row_scale(g.max_u32(max(m & 0xFFFFu, m >> 16)));
  if (first && ok) a.q_scale[row] = s.scale;
#pragma unroll
  for (int c = 0; c < NV; ++c)
    if ((kFull || ((in >> c) & 1u)) && ok)
      store_codes8(a.q + (size_t)row * a.ldq, at[c] / 8, a.H, codes8(o[c], s.inv));
}

template <typename Y, typename R, int NV, int kMaxThreads, bool kWarpRow>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_kernel(const NormArgs a) {
  __shared__ float s_red[2 * kRowMaxWarps];
  grid_trigger();
  grid_wait();
  RowGroup<kWarpRow> g{s_red, 0};
  const int i = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int row = kWarpRow ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && row >= a.T) return;
  const int H = a.H;
  const size_t base = (size_t)row * H;
  int at[NV];
  uint32_t in = 0;
  Raw8<Y> y[NV];
  Raw8<R> r[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    at[c] = 8 * (i + c * nt);
    y[c] = Raw8<Y>{};
    r[c] = Raw8<R>{};
    if (at[c] < H) {
      y[c].load(a.y, base + at[c]);
      r[c].load(a.res, base + at[c]);
      in |= 1u << c;
    }
    at[c] = min(at[c], H - 8);
  }
  float2 v[NV][4];
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int p = 0; p < 4; ++p) v[c][p] = pair_of(y[c], p);
  if (a.post != HQ_NORM_NONE) norm_row<NV, kWarpRow>(g, v, a.post, a.post_w, a.post_b, a.eps, H, at, in);
  if (a.gate) {
    const uint16_t* gate = a.gate + (size_t)(a.gate_rows >= a.T ? 0 : row / a.gate_rows) * H;
#pragma unroll
    for (int c = 0; c < NV; ++c) gate8(ld_dep(reinterpret_cast<const uint4*>(gate + at[c])), v[c]);
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) residual8(a, r[c], v[c], base + at[c], (in >> c) & 1u, (in >> c) & 1u);
  if (a.pre == HQ_NORM_NONE) return;
  norm_row<NV, kWarpRow>(g, v, a.pre, a.pre_w, a.pre_b, a.eps, H, at, in);
  store_row<NV, false, kWarpRow>(g, a, v, row, at, in, i == 0, true);
}

// ------------------------------------------------------------------------------------------------
// Many rows: one CTA an SM walks the rows, a ring of whole rows ahead of it.
//
// A thread keeps its 16 columns (two vectors) of the weights and of the gate in registers from row to
// row: at H = 8192 a row's weights and gate are 80 KB beside its 64 KB of data, and reading them from L1
// for every row, with a row's loads waited for at its start, holds the one-CTA-a-row kernel above to two
// thirds of the memory's rate (120 us where this one takes 98).  The rows come by bulk copies of H elements, counted by an mbarrier a stage; a
// stage is refilled once every thread has taken its part of it (the first barrier of its row).
constexpr int kRowsVec = 2;
constexpr int kRowsThreads = 512;
constexpr int kRowsMaxStages = 8;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, unsigned bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// The norm of the row in v with the weights in registers (w: all ones where there is none, no bias).
template <bool kFull>
__device__ __forceinline__ void norm_row_reg(RowGroup<false>& g, float2 (&v)[kRowsVec][4], int kind,
                                             const float2 (&w)[kRowsVec][4], float eps, float inv_n, uint32_t in) {
  const float2 rstd = both(centre_row<kRowsVec, kFull, false>(g, v, kind, eps, inv_n, in));
#pragma unroll
  for (int c = 0; c < kRowsVec; ++c)
#pragma unroll
    for (int p = 0; p < 4; ++p) v[c][p] = __fmul2_rn(__fmul2_rn(v[c][p], rstd), w[c][p]);
}

template <typename T>
__device__ __forceinline__ Raw8<T> raw_from_shared(uint32_t at) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.v[i].x), "=r"(r.v[i].y), "=r"(r.v[i].z), "=r"(r.v[i].w)
                 : "r"(at + 16 * i));
  return r;
}

template <typename Y, typename R, bool kFull>
__global__ void __launch_bounds__(kRowsThreads, 1) residual_norm_rows_kernel(const NormArgs a, int stages, WaitLimits lim) {
  extern __shared__ __align__(128) unsigned char s_rows[];
  __shared__ float s_red[2 * kRowMaxWarps];
  __shared__ uint64_t s_full[kRowsMaxStages];
  __shared__ int s_abort;
  RowGroup<false> g{s_red, 0};
  const int i = threadIdx.x, nt = blockDim.x, H = a.H;
  const unsigned y_bytes = H * sizeof(Y), r_bytes = H * sizeof(R), stage_bytes = y_bytes + r_bytes;
  const uint32_t ring = smem_addr(s_rows);
  volatile int* abort = &s_abort;
  if (i == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&s_full[s], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_trigger();
  grid_wait();
  // thread 0 loads row `row` into stage s
  int issued = 0;
  auto load = [&](int row, int s) {
    ++issued;
    mbar_arrive_expect_tx(&s_full[s], stage_bytes);
    bulk_load(ring + s * stage_bytes, static_cast<const Y*>(a.y) + (size_t)row * H, y_bytes, &s_full[s]);
    bulk_load(ring + s * stage_bytes + y_bytes, static_cast<const R*>(a.res) + (size_t)row * H, r_bytes, &s_full[s]);
  };
  if (i == 0) {
    producer_start_delay(lim.start_delay);
    for (int s = 0, row = blockIdx.x; s < stages && row < a.T; ++s, row += gridDim.x) load(row, s);
  }
  int at[kRowsVec];
  uint32_t in = 0;
  float2 pw[kRowsVec][4], qw[kRowsVec][4];
  uint4 gate[kRowsVec];
#pragma unroll
  for (int c = 0; c < kRowsVec; ++c) {
    at[c] = 8 * (i + c * nt);
    if (at[c] < H) in |= 1u << c;
    at[c] = min(at[c], H - 8);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      pw[c][p] = a.post_w ? ld_dep(reinterpret_cast<const float2*>(a.post_w + at[c]) + p) : both(1.0f);
      qw[c][p] = a.pre_w ? ld_dep(reinterpret_cast<const float2*>(a.pre_w + at[c]) + p) : both(1.0f);
    }
  }
  const float inv_n = __fdiv_rn(1.0f, (float)H);
  int gate_row = -1, n = 0, s = 0, phase = 0;
  bool ok = true;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, ++n) {
    if (a.gate) {
      const int gr = a.gate_rows >= a.T ? 0 : row / a.gate_rows;
      if (gr != gate_row) {
        gate_row = gr;
#pragma unroll
        for (int c = 0; c < kRowsVec; ++c) gate[c] = ld_dep(reinterpret_cast<const uint4*>(a.gate + (size_t)gr * H + at[c]));
      }
    }
    // a wait that gives up leaves the barriers of the rows to come in step: nothing more is written
    ok = mbar_wait(&s_full[s], phase, abort, lim.consumer) && ok;
    Raw8<R> r[kRowsVec];
    float2 v[kRowsVec][4];
#pragma unroll
    for (int c = 0; c < kRowsVec; ++c) {
      const Raw8<Y> y = raw_from_shared<Y>(ring + s * stage_bytes + at[c] * (unsigned)sizeof(Y));
      r[c] = raw_from_shared<R>(ring + s * stage_bytes + y_bytes + at[c] * (unsigned)sizeof(R));
#pragma unroll
      for (int p = 0; p < 4; ++p) v[c][p] = kFull || ((in >> c) & 1u) ? pair_of(y, p) : both(0.0f);
    }
    if (a.post != HQ_NORM_NONE) norm_row_reg<kFull>(g, v, a.post, pw, a.eps, inv_n, in);
    else __syncthreads();
    if (i == 0 && ok) {  // every thread has its part of the stage
      const long long ahead = (long long)row + (long long)stages * gridDim.x;
      if (ahead < a.T) load((int)ahead, s);
    }
    if (++s == stages) s = 0, phase ^= 1;
    const size_t base = (size_t)row * H;
#pragma unroll
    for (int c = 0; c < kRowsVec; ++c) {
      if (a.gate) gate8(gate[c], v[c]);
      const bool mine = kFull || ((in >> c) & 1u);
      residual8(a, r[c], v[c], base + at[c], mine, mine && ok);
    }
    if (a.pre == HQ_NORM_NONE) continue;
    norm_row_reg<kFull>(g, v, a.pre, qw, a.eps, inv_n, in);
    store_row<kRowsVec, kFull, false>(g, a, v, row, at, in, i == 0, ok);
  }
  if (i == 0 && *abort) {  // the copies in flight have landed before the CTA leaves
    int ignore = 0;
    for (int q = max(0, issued - stages); q < issued; ++q)
      mbar_wait(&s_full[q % stages], (q / stages) & 1, &ignore, lim.producer);
  }
}

}  // namespace hq
