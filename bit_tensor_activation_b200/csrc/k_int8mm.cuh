// k_int8mm.cuh -- the row-parallel product in 8-bit integers, rank by rank: int8 activations with one
// scale a token times int8 weights with one scale a channel, leaving as the partial sum [P][T][H] or
// as the hybrid wire of that partial sum.
//
//   acc = sum_k a[r][t][k] * w[r][n][k]           exact: |acc| <= 128^2 K <= 2^30 for K <= 65536
//   v   = (float(acc) * a_scale[r][t]) * w_scale[r][n] (+ bias[r][n]), one rounding a step
#pragma once

#include "hq_tc.cuh"

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

// ------------------------------------------------------------------------------------------------
// Many tokens: a pair of CTAs to a tile of 256 tokens x 256 features.
//
// tcgen05.mma with cta_group::2 takes M = 256, N = 256: each CTA of the pair loads its own 128 tokens
// and its own 128 features (32 KB a step of K = 128 bytes) and holds the accumulators of its 128
// tokens x 256 features, so an operand byte is read from L2 once for 256 rows of the other operand.
// A 256 x 256 tile of int32 is half of tensor memory: two tiles take turns, and the epilogue of one
// runs under the products of the next.  One cluster a pair of SMs walks the tiles, rank by rank.
//
// Warps 0-7 are the epilogue (warp w: lanes of tensor memory 32 (w % 4) .., columns 128 (w / 4) ..),
// warp 8 loads, warp 9 of the first CTA issues the products.  Every wait is bounded (hq_tma.cuh).
constexpr int kMmTile = 256;                                   // tokens and features of a pair's tile
constexpr int kMmHalf = 128;                                   // of one CTA
constexpr int kMmK = 128;                                      // bytes of K a step
constexpr int kMmStages = 5;
constexpr int kMmEpiWarps = 8;
constexpr int kMmThreads = 32 * (kMmEpiWarps + 2);
constexpr unsigned kMmStageBytes = 2 * kMmHalf * kMmK;         // one CTA's part of a step
constexpr int kMmGroupM = 8;                                   // token tiles that share a sweep over the features

// The parameters of a warp's 128 columns.
struct MmCols {
  alignas(16) float scale[kMmHalf];
  alignas(16) float second[kMmHalf];  // bias, or the wire's inv_scale
  alignas(16) float lo[kMmHalf];      // -zero
  uint32_t zeros[kMmHalf / 8];        // the zero points of 8 columns as one word of codes
};

struct MmSmem {
  alignas(1024) unsigned char a[kMmStages][kMmHalf * kMmK];
  alignas(1024) unsigned char b[kMmStages][kMmHalf * kMmK];
  alignas(1024) unsigned char out[kMmEpiWarps][32 * 128];      // a warp's 32 rows of 128 bytes on their way out
  MmCols col[kMmEpiWarps];
  uint64_t full[kMmStages], empty[kMmStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
};

static_assert(sizeof(MmSmem) + 1024 <= 227 * 1024, "shared memory of one CTA");

// Tile i of the walk: rank, token tile, feature tile.  Within a rank, groups of kMmGroupM token tiles
// sweep all features, so that a wave of tiles shares its operands in L2.
struct MmTileAt {
  int r, t0, n0;
};
__device__ __forceinline__ MmTileAt mm_tile(int i, int mt, int nt) {
  const int r = i / (mt * nt);
  int j = i - r * mt * nt;
  const int g = j / (kMmGroupM * nt);
  const int rows = min(kMmGroupM, mt - g * kMmGroupM);
  j -= g * kMmGroupM * nt;
  const int n = j / rows;
  return MmTileAt{r, (g * kMmGroupM + j - n * rows) * kMmTile, n * kMmTile};
}

// Eight bf16 values (w: four words) of one token as one word of codes, the columns' parameters at
// inv and lo.  clamp(rint(t) + zero, 0, 15) = zero + rint(clamp(t, -zero, 15 - zero)), the bounds being
// integers; adding 1.5 * 2^23 rounds to an integer, half to even, and leaves it in the low bits.  A NaN
// (code: the zero point) shows in the sum of the products, and that word is made one code at a time.
__device__ __forceinline__ uint32_t wire_word(const uint32_t* w, const float* inv, const float* lo, uint32_t zeros) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 i4 = *reinterpret_cast<const float4*>(inv + j);
    fmul2(t[j], t[j + 1], bf16_lo(w[j / 2]), bf16_hi(w[j / 2]), i4.x, i4.y);
    fmul2(t[j + 2], t[j + 3], bf16_lo(w[j / 2 + 1]), bf16_hi(w[j / 2 + 1]), i4.z, i4.w);
  }
  float s0, s1, s2, s3;
  fadd2(s0, s1, t[0], t[1], t[2], t[3]);
  fadd2(s2, s3, t[4], t[5], t[6], t[7]);
  fadd2(s0, s1, s0, s1, s2, s3);
  s0 = __fadd_rn(s0, s1);
  if (s0 != s0) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int l = (int)lo[j], c = __float2int_rn(t[j]);  // saturating; NaN -> 0
      word |= (uint32_t)(min(max(c, l), l + 15) - l) << (4 * j);
    }
    return word;
  }
  constexpr uint32_t kOnes = 0x11111111u;
  uint32_t word = zeros - 0x4B400000u * kOnes;  // the constant's share of the sum below, modulo 2^32
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 l4 = *reinterpret_cast<const float4*>(lo + j);
    const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float a = fminf(fmaxf(t[j + i], l[i]), __fadd_rn(l[i], 15.0f));
      float b = fminf(fmaxf(t[j + i + 1], l[i + 1]), __fadd_rn(l[i + 1], 15.0f));
      fadd2(a, b, a, b, 12582912.0f, 12582912.0f);
      word += (__float_as_uint(a) << (4 * (j + i))) + (__float_as_uint(b) << (4 * (j + i + 1)));
    }
  }
  return word;
}

// A lane's four columns' parameters on their way to shared memory: fetched a tile ahead.
template <int kOut>
struct MmFetch {
  float4 scale, second;
  int4 rest;
  uint32_t zero;  // four bytes

  __device__ __forceinline__ void start(const MmArgs& p, int r, int c) {
    scale = second = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    rest = make_int4(0, 0, 0, 0);
    zero = 0;
    if (c < p.H) {
      const size_t g = (size_t)r * p.H + c;
      scale = __ldg(reinterpret_cast<const float4*>(p.w_scale + g));
      if (kOut != kMmWire && p.bias) {
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(p.bias + g));
        second = make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
      }
    }
    if (kOut == kMmWire && c < p.H - p.k)
      rest = make_int4(__ldg(p.rest_idx + c), __ldg(p.rest_idx + c + 1), __ldg(p.rest_idx + c + 2),
                       __ldg(p.rest_idx + c + 3));
  }
  // The wire's grids, once the features are known.
  __device__ __forceinline__ void grids(const MmArgs& p, int r, int c) {
    if (kOut != kMmWire || c >= p.H - p.k) return;
    rest = make_int4(checked_index(rest.x, p.H), checked_index(rest.y, p.H), checked_index(rest.z, p.H),
                     checked_index(rest.w, p.H));
    const float* inv = p.inv_scale + (size_t)r * p.H;
    const uint8_t* z = p.zero + (size_t)r * p.H;
    second = make_float4(__ldg(inv + rest.x), __ldg(inv + rest.y), __ldg(inv + rest.z), __ldg(inv + rest.w));
    zero = (uint32_t)__ldg(z + rest.x) | (uint32_t)__ldg(z + rest.y) << 8 | (uint32_t)__ldg(z + rest.z) << 16 |
           (uint32_t)__ldg(z + rest.w) << 24;
  }
  __device__ __forceinline__ void store(MmCols& s, int lane) const {
    *reinterpret_cast<float4*>(s.scale + 4 * lane) = scale;
    *reinterpret_cast<float4*>(s.second + 4 * lane) = second;
    if (kOut == kMmWire) {
      const uint32_t z0 = zero & 0xFFu, z1 = (zero >> 8) & 0xFFu, z2 = (zero >> 16) & 0xFFu, z3 = zero >> 24;
      *reinterpret_cast<float4*>(s.lo + 4 * lane) = make_float4(-(float)z0, -(float)z1, -(float)z2, -(float)z3);
      uint32_t w = (z0 + (z1 << 4) + (z2 << 8) + (z3 << 12)) << (16 * (lane & 1));
      w += __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      if ((lane & 1) == 0) s.zeros[lane >> 1] = w;
    }
  }
};

// `n` words of one token's codes, as widely as their address allows.
__device__ __forceinline__ void store_words8(uint32_t* p, const uint32_t* w, int n, int align) {
  if (n == 8 && align == 32) {
    st_global32(p, w);
  } else if (n == 8 && align == 16) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = w[i];
  }
}

template <int kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
    int8_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                            const __grid_constant__ CUtensorMap map_out, const MmArgs p, WaitLimits lim) {
  extern __shared__ unsigned char s_raw[];
  MmSmem& sm = *reinterpret_cast<MmSmem*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_ctarank();
  const int mt = (p.T + kMmTile - 1) / kMmTile, nt = (p.H + kMmTile - 1) / kMmTile;
  const int tiles = p.P * mt * nt, step = gridDim.x / 2, first = blockIdx.x / 2;
  const int kc = (p.K + kMmK - 1) / kMmK;
  volatile int* abort = &sm.abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMmStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * kMmEpiWarps);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmEpiWarps + 1) tc_alloc<2>(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp == kMmEpiWarps) {  // ---------------------------------------------- loads
    if (lane == 0) {
      prefetch_tensor_map(&map_a);
      prefetch_tensor_map(&map_w);
      producer_start_delay(lim.start_delay);
      int i = 0;
      bool go = true;
      for (int t = first; t < tiles && go; t += step) {
        const MmTileAt at = mm_tile(t, mt, nt);
        for (int c = 0; c < kc; ++c, ++i) {
          const int s = i % kMmStages;
          if (i >= kMmStages && !mbar_wait(&sm.empty[s], ((i / kMmStages) - 1) & 1, abort, lim.producer)) {
            go = false;
            break;
          }
          if (cta == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kMmStageBytes);
          const uint32_t bar = cluster_addr(smem_addr(&sm.full[s]), 0);
          tma_load_3d_pair(smem_addr(sm.a[s]), &map_a, c * kMmK, at.t0 + (int)cta * kMmHalf, at.r, bar);
          tma_load_3d_pair(smem_addr(sm.b[s]), &map_w, c * kMmK, at.n0 + (int)cta * kMmHalf, at.r, bar);
        }
      }
      // after an abort: the pair's loads have landed before either CTA leaves (the first CTA counts both)
      if (*abort && cta == 0) {
        int ignore = 0;
        for (int j = max(0, i - kMmStages); j < i; ++j)
          mbar_wait(&sm.full[j % kMmStages], (j / kMmStages) & 1, &ignore, lim.producer);
      }
    }
  } else if (warp == kMmEpiWarps + 1) {  // ---------------------------------- products
    if (cta == 0 && lane == 0) {
      constexpr uint32_t idesc = tc_idesc(kMmTile, kMmTile);
      int i = 0, n = 0;
      bool go = true;
      for (int t = first; t < tiles && go; t += step, ++n) {
        const int b = n & 1;
        if (n >= 2 && !mbar_wait(&sm.acc_empty[b], ((n >> 1) - 1) & 1, abort, lim.producer)) break;
        tc_fence_after();
        const uint32_t d = tmem + b * kMmTile;
        for (int c = 0; c < kc; ++c, ++i) {
          const int s = i % kMmStages;
          if (!mbar_wait(&sm.full[s], (i / kMmStages) & 1, abort, lim.consumer)) {
            go = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = tc_desc(smem_addr(sm.a[s])), db = tc_desc(smem_addr(sm.b[s]));
#pragma unroll
          for (int k = 0; k < kMmK / 32; ++k) tc_mma<2>(d, da + 2 * k, db + 2 * k, idesc, c > 0 || k > 0);
          tc_commit<2>(&sm.empty[s]);
        }
        if (go) tc_commit<2>(&sm.acc_full[b]);
      }
      if (*abort) {  // the products in flight are done before tensor memory is freed
        int ignore = 0;
        tc_commit<2>(&sm.drain);
        mbar_wait(&sm.drain, 0, &ignore, lim.producer);
      }
    }
  } else {  // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3, side = warp >> 2;  // lanes 32 quad .., columns 128 side ..
    const uint32_t stage = smem_addr(sm.out[warp]);
    MmCols& cols = sm.col[warp];
    const int Hr = p.H - p.k;
    const int word_align = Hr % 64 == 0 && ((uintptr_t)p.codes & 31) == 0 ? 32 : Hr % 32 == 0 && ((uintptr_t)p.codes & 15) == 0 ? 16 : 4;
    MmFetch<kOut> next;
    float next_sa = 0.0f;
    auto fetch = [&](int t) {
      if (t >= tiles) return;
      const MmTileAt at = mm_tile(t, mt, nt);
      const int row = at.t0 + (int)cta * kMmHalf + 32 * quad + lane;
      next_sa = row < p.T ? __ldg(p.a_scale + (size_t)at.r * p.T + row) : 0.0f;
      next.start(p, at.r, at.n0 + kMmHalf * side + 4 * lane);
    };
    auto fetch_grids = [&](int t) {
      if (kOut != kMmWire || t >= tiles) return;
      const MmTileAt at = mm_tile(t, mt, nt);
      next.grids(p, at.r, at.n0 + kMmHalf * side + 4 * lane);
    };
    fetch(first);
    fetch_grids(first);
    int n = 0;
    for (int t = first; t < tiles; t += step, ++n) {
      const int b = n & 1;
      const MmTileAt at = mm_tile(t, mt, nt);
      const int row = at.t0 + (int)cta * kMmHalf + 32 * quad;  // the warp's first token
      const float sa = next_sa;
      __syncwarp();
      next.store(cols, lane);
      __syncwarp();
      fetch(t + step);
      // every lane of the warp, or none
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.acc_full[b], (n >> 1) & 1, abort, lim.consumer))) break;
      tc_fence_after();
      fetch_grids(t + step);
      const uint32_t acc = tmem + b * kMmTile + ((uint32_t)(32 * quad) << 16) + kMmHalf * side;
      const float* col = cols.scale;
      const float* col2 = cols.second;
      uint32_t words[8];
      uint32_t ld[2][32];
      tc_load32(acc, ld[0]);
#pragma unroll
      for (int c = 0; c < kMmHalf; c += 32) {
        uint32_t(&v)[32] = ld[(c >> 5) & 1];
        tc_load_wait(v);
        if (c + 32 < kMmHalf) {  // the next columns come while these are worked on
          tc_load32(acc + c + 32, ld[((c >> 5) + 1) & 1]);
        } else {  // the tile's last read: its columns may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&sm.acc_empty[b]), 0));
        }
        const int n0 = at.n0 + kMmHalf * side + c;
        if (n0 >= p.H || row >= p.T) continue;
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(col + c + j);
          fmul2(f[j], f[j + 1], __int2float_rn((int)v[j]), __int2float_rn((int)v[j + 1]), sa, sa);
          fmul2(f[j + 2], f[j + 3], __int2float_rn((int)v[j + 2]), __int2float_rn((int)v[j + 3]), sa, sa);
          fmul2(f[j], f[j + 1], f[j], f[j + 1], w.x, w.y);
          fmul2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], w.z, w.w);
        }
        if (kOut != kMmWire && p.bias) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(col2 + c + j);
            fadd2(f[j], f[j + 1], f[j], f[j + 1], w.x, w.y);
            fadd2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], w.z, w.w);
          }
        }
        // 16-byte piece q of row `lane` lies at piece q ^ (lane % 8): the store's 128-byte swizzle
        if (kOut == kMmF32) {
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared16(stage + lane * 128 + ((q ^ (lane & 7)) << 4), __float_as_uint(f[4 * q]),
                        __float_as_uint(f[4 * q + 1]), __float_as_uint(f[4 * q + 2]), __float_as_uint(f[4 * q + 3]));
          fence_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_3d(&map_out, stage, n0, row, at.r);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = kOut == kMmBf16 ? pack_bf16x2(f[2 * j], f[2 * j + 1]) : round_bf16x2(f[2 * j], f[2 * j + 1]);
          if (kOut == kMmBf16) {
            const int half = (c >> 5) & 1;  // 64 columns to a store
            if (half == 0) {
              if (lane == 0) tma_store_wait_read<0>();
              __syncwarp();
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared16(stage + lane * 128 + (((4 * half + q) ^ (lane & 7)) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2],
                          w[4 * q + 3]);
            if (half == 1 || n0 + 32 >= p.H) {
              fence_async_smem();
              __syncwarp();
              if (lane == 0) tma_store_3d(&map_out, stage, n0 - 32 * half, row, at.r);
            }
          } else {
            const int half = (c >> 5) & 1;  // 64 columns are 8 words
            const size_t tok = (size_t)at.r * p.T + row + lane;
            const bool live = row + lane < p.T;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              words[4 * half + q] = wire_word(w + 4 * q, col2 + c + 8 * q, cols.lo + c + 8 * q, cols.zeros[c / 8 + q]);
            const int first_col = n0 - 32 * half;
            if (live && first_col < Hr && (half == 1 || n0 + 32 >= Hr))
              store_words8(p.codes + tok * (Hr / 8) + first_col / 8, words, min(8, (Hr - first_col) / 8), word_align);
            if (live && n0 + 32 > Hr) {  // kept features, 32 tokens of one beside one another
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int f0 = n0 + j - Hr;
                const uint32_t x = (w[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
                if (f0 >= 0 && n0 + j < p.H)
                  p.side[((size_t)at.r * p.k + f0) * p.T + row + lane] = (uint16_t)((x & 0x7FFFu) > 0x7F80u ? 0x7FC0u : x);
              }
            }
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_read<0>();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memory goes while the other still counts on it
  tc_fence_after();
  if (warp == kMmEpiWarps + 1) tc_dealloc<2>(tmem, 512);
}

}  // namespace hq
