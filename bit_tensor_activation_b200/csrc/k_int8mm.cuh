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
  const int32_t* keep_idx;
  const int32_t* rest_idx;
  const float* inv_scale;
  const uint8_t* zero;
  uint32_t* codes;
  uint16_t* side;
};

enum MmOut { kMmBf16 = 0, kMmF32 = 1, kMmWire = 2 };

// The feature, in their own order, of compact position c of the wire.
__device__ __forceinline__ int wire_feature(const MmArgs& p, int c) {
  const int Hr = p.H - p.k;
  return ld_dep(c < Hr ? p.rest_idx + c : p.keep_idx + (c - Hr));
}

// ------------------------------------------------------------------------------------------------
// Many tokens: a pair of CTAs to a tile of 256 tokens x kN features.
//
// tcgen05.mma with cta_group::2 takes M = 256, N = 256: each CTA of the pair loads its own 128 tokens
// and its own 128 features (32 KB a step of K = 128 bytes) and holds the accumulators of its 128
// tokens x 256 features, so an operand byte is read from L2 once for 256 rows of the other operand.
// A 256 x 256 tile of int32 is half of tensor memory: two tiles take turns, and the epilogue of one
// runs under the products of the next.  One cluster a pair of SMs walks the tiles, rank by rank.
//
// What bounds it.  With long K the tensor cores under the power limit: 8 ranks, 4096 tokens, H = 4096, K = 2048
// take 182 us from cold, 3.0 POP/s, and 208 to 221 us back to back at 1000 W; the products alone, on operands
// that stay in shared memory, reach 4.2 POP/s, 4.4 on zeros.  With K = 1024 and below the epilogue: 32768 values
// a CTA and tile take 2.5 us as bf16 and 3.9 as the wire; K = 512, H = 4096 takes 71 and 109 us.  It is latency
// more than instructions: their 7 and 14 a value are 0.9 and 1.8 us of issue slots, and with K = 1024 the
// wire uses 41% of the slots, 40% of the ALU and 48% of shared memory's.  A warp waits for its chunk's load
// from tensor memory before the chunk's arithmetic, and three such warps a scheduler do not hide that.
// What helped: codes without conversions (wire_word), stores by TMA from 2 KB a warp (32-byte stores
// straight from registers: 10% more time), a body small enough to stay in the instruction cache (unrolled over
// a tile's columns: 20% more), and twelve warps (eight: 5% more for the wire; sixteen: spills).
//
// Warps 0-11 are the epilogue: three warps share the 32 lanes (tokens) of tensor memory that a warp can
// read and take its chunks of 32 columns in turn, from one tile to the next.  Warp 12 loads, warp 13 of
// the first CTA issues the products.  Every wait is bounded (hq_tma.cuh).
//
// kN, a tile's features, is 256 where there are tiles enough; with fewer, tiles of 128 features spread over
// more SMs and leave half the epilogue at the end, for half as many more operand bytes a product.
constexpr int kMmTile = 256;                              // tokens of a pair's tile
constexpr int kMmHalf = 128;                              // of one CTA
constexpr int kMmK = 128;                                 // bytes of K a step
constexpr int kMmStages = 5;
constexpr int kMmEpiWarps = 12;
constexpr int kMmSides = kMmEpiWarps / 4;                 // epilogue warps that share 32 lanes of tensor memory
constexpr int kMmThreads = 32 * (kMmEpiWarps + 2);
constexpr int kMmGroupM = 8;                              // token tiles that share a sweep over the features
template <int kN>
struct MmShape {
  static_assert(kN == 128 || kN == 256, "every epilogue warp has a chunk of every tile");
  static constexpr int kChunks = kN / 32;                 // 32 columns at a time
  static constexpr int kWarpChunks = (kChunks + kMmSides - 1) / kMmSides;
  static constexpr unsigned kStageBytes = (kMmHalf + kN / 2) * kMmK;  // one CTA's part of a step
};

// The parameters of 32 columns.
struct MmCols {
  alignas(16) float scale[32];
  alignas(16) float second[32];  // bias, or the wire's inv_scale
  alignas(16) int zero[32];      // the wire's zero point - kMagicBits
};

template <int kN>
struct MmSmem {
  alignas(1024) unsigned char a[kMmStages][kMmHalf * kMmK];
  alignas(1024) unsigned char b[kMmStages][kN / 2 * kMmK];
  alignas(1024) unsigned char out[kMmEpiWarps][32 * 64];       // a warp's 32 rows of 64 bytes on their way out
  MmCols col[kMmEpiWarps][MmShape<kN>::kWarpChunks];
  uint64_t full[kMmStages], empty[kMmStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
  uint32_t gave_up[2];                                         // of both CTAs, once their roles are done
  uint32_t issued[2];                                          // and the steps each of them has loaded
};
static_assert(sizeof(MmSmem<256>) + 1024 <= 227 * 1024, "shared memory of one CTA");

// The walk over the tiles, rank by rank.  Within a rank, groups of kMmGroupM token tiles sweep all
// features, so that a wave of tiles shares its operands in L2.  Quotients come from fp32 reciprocals and
// one correction: they are below 2^20 (2^31 tokens are 2^20 groups), so the estimate is off by at most one.
struct MmTileAt {
  int r, t0, n0;
};
template <int kN>
struct MmWalk {
  int mt, nt, per_rank, r, j;
  float inv_group;

  __device__ __forceinline__ MmWalk(const MmArgs& p, int i) {
    mt = (p.T - 1) / kMmTile + 1;  // T >= 1; T + 255 may pass 2^31
    nt = (p.H + kN - 1) / kN;
    per_rank = mt * nt;
    r = i / per_rank;
    j = i - r * per_rank;
    inv_group = __frcp_rn((float)(kMmGroupM * nt));
  }
  __device__ __forceinline__ void advance(int step) {
    for (j += step; j >= per_rank; j -= per_rank) ++r;
  }
  __device__ __forceinline__ MmTileAt at() const {
    int g = __float2int_rz(__fmul_rn((float)j, inv_group));
    int rem = j - g * kMmGroupM * nt;
    if (rem < 0) --g, rem += kMmGroupM * nt;
    if (rem >= kMmGroupM * nt) ++g, rem -= kMmGroupM * nt;
    const int rows = min(kMmGroupM, mt - g * kMmGroupM);
    const int n = rows == kMmGroupM ? rem / kMmGroupM : rem / rows;
    return MmTileAt{r, (g * kMmGroupM + rem - n * rows) * kMmTile, n * kN};
  }
};

// Eight bf16 values (w: four words) of one token as one word of codes: clamp(rint(x * inv) + zero, 0, 15).
// Adding 1.5 * 2^23 rounds a product below 2^22 to an integer, half to even, in the low bits of the sum;
// with the zero point less the constant's bits that is rint + zero, which cvt.pack saturates to 0 .. 15
// and puts beside the others.  Eight products with a larger one or a NaN among them are taken one by one
// (their largest magnitude costs half an instruction each; clamping every one of them would cost two).
constexpr int kMagicBits = 0x4B400000;  // 12582912.0f
__device__ __noinline__ uint32_t wire_word_slow(float4 ta, float4 tb, const int* zero) {
  const float t[8] = {ta.x, ta.y, ta.z, ta.w, tb.x, tb.y, tb.z, tb.w};
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int z = zero[j] + kMagicBits, c = __float2int_rn(t[j]);  // saturating; NaN -> 0
    word |= (uint32_t)(min(max(c, -z), 15 - z) + z) << (4 * j);
  }
  return word;
}
__device__ __forceinline__ uint32_t wire_word(const uint32_t* w, const MmCols& cols, int c) {
  float t[8];
  int q[8];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 i = *reinterpret_cast<const float4*>(cols.second + c + j);
    fmul2(t[j], t[j + 1], bf16_lo(w[j / 2]), bf16_hi(w[j / 2]), i.x, i.y);
    fmul2(t[j + 2], t[j + 3], bf16_lo(w[j / 2 + 1]), bf16_hi(w[j / 2 + 1]), i.z, i.w);
    const int4 z = *reinterpret_cast<const int4*>(cols.zero + c + j);
    float a0, a1, a2, a3;
    fadd2(a0, a1, t[j], t[j + 1], 12582912.0f, 12582912.0f);
    fadd2(a2, a3, t[j + 2], t[j + 3], 12582912.0f, 12582912.0f);
    q[j] = __float_as_int(a0) + z.x, q[j + 1] = __float_as_int(a1) + z.y;
    q[j + 2] = __float_as_int(a2) + z.z, q[j + 3] = __float_as_int(a3) + z.w;
  }
  float top;  // the largest |t|, or NaN
  asm("{.reg .f32 a, b;\n\tmax.NaN.abs.f32 a, %1, %2, %3;\n\tmax.NaN.abs.f32 b, %4, %5, %6;\n\t"
      "max.NaN.abs.f32 a, a, %7, %8;\n\tmax.NaN.abs.f32 %0, a, b, b;}"
      : "=f"(top)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  uint32_t word = 0;
#pragma unroll
  for (int j = 6; j >= 0; j -= 2)
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %0;" : "+r"(word) : "r"(q[j + 1]), "r"(q[j]));
  if (!(top < 2097152.0f))
    word = wire_word_slow(make_float4(t[0], t[1], t[2], t[3]), make_float4(t[4], t[5], t[6], t[7]), cols.zero + c);
  return word;
}

// A lane's column of each of its warp's chunks, fetched a tile ahead of its use: chunk j0 + kMmSides i
// of the 32 columns each from feature n0.
template <int kOut, int kN>
struct MmFetch {
  static constexpr int kWarpChunks = MmShape<kN>::kWarpChunks, kChunks = MmShape<kN>::kChunks;
  float scale[kWarpChunks], second[kWarpChunks];
  int feature[kWarpChunks];
  uint32_t zero[kWarpChunks];

  __device__ __forceinline__ static int column(int n0, int j0, int i, int lane) { return n0 + 32 * (j0 + kMmSides * i) + lane; }

  __device__ __forceinline__ void start(const MmArgs& p, int r, int n0, int j0, int lane) {
#pragma unroll
    for (int i = 0; i < kWarpChunks; ++i) {
      const int c = column(n0, j0, i, lane);
      const size_t g = (size_t)r * p.H + c;
      const bool on = j0 + kMmSides * i < kChunks && c < p.H;
      scale[i] = on ? ld_dep(p.w_scale + g) : 0.0f;
      second[i] = kOut != kMmWire && p.bias && on ? bf16_lo(ld_dep(p.bias + g)) : 0.0f;
      feature[i] = kOut == kMmWire && on ? wire_feature(p, c) : 0;
      zero[i] = 0;
    }
  }
  // The wire's grids, once the features are known.  A kept one has none: its index is checked.
  __device__ __forceinline__ void grids(const MmArgs& p, int r, int n0, int j0, int lane) {
#pragma unroll
    for (int i = 0; i < kWarpChunks; ++i) {
      const size_t g = (size_t)r * p.H + checked_index(feature[i], p.H);
      if (j0 + kMmSides * i >= kChunks || column(n0, j0, i, lane) >= p.H - p.k) continue;
      second[i] = ld_dep(p.inv_scale + g);
      zero[i] = ld_dep(p.zero + g);
    }
  }
  __device__ __forceinline__ void store(MmCols* s, int lane) const {
#pragma unroll
    for (int i = 0; i < kWarpChunks; ++i) {
      s[i].scale[lane] = scale[i];
      s[i].second[lane] = second[i];
      if (kOut == kMmWire) s[i].zero[lane] = (int)zero[i] - kMagicBits;
    }
  }
};

// A warp's 32 tokens' four words of codes each (x: the lane's token's, at words): `n` words of `rows` tokens,
// `pitch` words apart.  kWide (a token's words start and end on 16 bytes: n is 4): one store a token.  Else through 512 bytes
// at `stage`, four lanes to a token, since single words straight from the lanes that hold them touch 32 lines
// with every store (8 ranks, 4096 tokens, H = 4104, K = 512: 121 us, 147 so; kWide, H = 4096: 105).
template <bool kWide>
__device__ __forceinline__ void store_words(uint32_t* words, int pitch, const uint32_t (&x)[4], int n, int rows,
                                            uint32_t stage, int lane) {
  if constexpr (kWide) {
    if (lane < rows) *reinterpret_cast<uint4*>(words) = make_uint4(x[0], x[1], x[2], x[3]);
  } else {
    __syncwarp();
    st_shared16(stage + 16 * lane, x[0], x[1], x[2], x[3]);
    __syncwarp();
    const int w = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint32_t v = ld_shared(stage + 16 * r + 4 * w);
      if (r < rows && w < n) words[(long long)(r - lane) * pitch + w] = v;
    }
  }
}

// After a wait that gave up, in either CTA: what is in flight is done before either of them leaves.  Loads are
// counted on the first CTA's barriers, both CTAs' parts of a step together.  A step that only one CTA has loaded
// (they give up apart by a few steps, never by more than the ring) is made up to its whole count here: the
// first CTA has announced both parts, the second none.  Only the last step of each stage can be under way, since a
// stage is loaded anew once its products are done.
template <int kN>
__device__ __noinline__ void mm_pair_drain(MmSmem<kN>& sm, int warp, int lane, uint32_t cta, WaitLimits lim) {
  if (cta != 0 || lane != 0) return;
  int ignore = 0;
  if (warp == kMmEpiWarps) {
    const int mine = (int)sm.issued[0], other = (int)sm.issued[1], most = max(mine, other);
    for (int j = max(0, most - kMmStages); j < most; ++j) {
      uint64_t* const full = &sm.full[j % kMmStages];
      if (j >= mine) mbar_arrive_expect_tx(full, MmShape<kN>::kStageBytes);
      if (j >= other) mbar_complete_tx(full, MmShape<kN>::kStageBytes);
      mbar_wait(full, (j / kMmStages) & 1, &ignore, lim.producer);
    }
  }
  if (warp == kMmEpiWarps + 1) {  // the lane that issued the products
    tc_commit<2>(&sm.drain);
    mbar_wait(&sm.drain, 0, &ignore, lim.producer);
  }
}

template <int kOut, int kN, bool kWide>
__global__ void __launch_bounds__(kMmThreads, 1)
    int8_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                            const __grid_constant__ CUtensorMap map_out, const MmArgs p, WaitLimits lim) {
  extern __shared__ unsigned char s_raw[];
  constexpr int kChunks = MmShape<kN>::kChunks;
  MmSmem<kN>& sm = *reinterpret_cast<MmSmem<kN>*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_ctarank();
  const int step = gridDim.x / 2, first = blockIdx.x / 2;
  MmWalk<kN> walk(p, first);
  const int tiles = p.P * walk.per_rank;
  const int kc = (p.K + kMmK - 1) / kMmK;
  volatile int* abort = &sm.abort;
  int issued = 0;  // the load lane's steps

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
  if (warp == kMmEpiWarps + 1) tc_alloc<2>(&sm.tmem, 2 * kN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  grid_trigger();
  grid_wait();

  if (warp == kMmEpiWarps) {  // ---------------------------------------------- loads
    if (lane == 0) {
      prefetch_tensor_map(&map_a);
      prefetch_tensor_map(&map_w);
      producer_start_delay(lim.start_delay);
      bool go = true;
      for (int t = first; t < tiles && go; t += step, walk.advance(step)) {
        const MmTileAt at = walk.at();
        for (int c = 0; c < kc; ++c, ++issued) {
          const int s = issued % kMmStages;
          if (issued >= kMmStages && !mbar_wait(&sm.empty[s], ((issued / kMmStages) - 1) & 1, abort, lim.producer)) {
            go = false;
            break;
          }
          if (cta == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * MmShape<kN>::kStageBytes);
          const uint32_t bar = cluster_addr(smem_addr(&sm.full[s]), 0);
          tma_load_3d_pair(smem_addr(sm.a[s]), &map_a, c * kMmK, at.t0 + (int)cta * kMmHalf, at.r, bar);
          tma_load_3d_pair(smem_addr(sm.b[s]), &map_w, c * kMmK, at.n0 + (int)cta * (kN / 2), at.r, bar);
        }
      }
    }
  } else if (warp == kMmEpiWarps + 1) {  // ---------------------------------- products
    if (cta == 0 && lane == 0) {
      constexpr uint32_t idesc = tc_idesc(kMmTile, kN);
      int i = 0, n = 0;
      bool go = true;
      for (int t = first; t < tiles && go; t += step, ++n) {
        const int b = n & 1;
        if (n >= 2 && !mbar_wait(&sm.acc_empty[b], ((n >> 1) - 1) & 1, abort, lim.producer)) break;
        tc_fence_after();
        const uint32_t d = tmem + b * kN;
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
    }
  } else {  // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3, side = warp >> 2;
    const uint32_t stage = smem_addr(sm.out[warp]);
    MmCols* const cols_of = sm.col[warp];
    const int Hr = p.H - p.k, Wr = Hr >> 3;
    MmFetch<kOut, kN> next;
    float next_sa = 0.0f;
    // the warp's first chunk of its n-th tile: chunks 0, 1, .. of tile after tile go round the sides
    auto first_chunk = [&](int n) { return (side + (kMmSides - kChunks % kMmSides) * n) % kMmSides; };
    auto fetch = [&](const MmTileAt& at, int n) {
      const int row = at.t0 + (int)cta * kMmHalf + 32 * quad + lane;
      next_sa = row < p.T ? ld_dep(p.a_scale + (size_t)at.r * p.T + row) : 0.0f;
      next.start(p, at.r, at.n0, first_chunk(n), lane);
    };
    int n = 0;
    MmTileAt at = walk.at();
    fetch(at, 0);
    if (kOut == kMmWire) next.grids(p, at.r, at.n0, first_chunk(0), lane);
    for (int t = first; t < tiles; t += step, ++n) {
      const int b = n & 1;
      const int row = at.t0 + (int)cta * kMmHalf + 32 * quad;  // the warp's first token
      const float sa = next_sa;
      __syncwarp();
      next.store(cols_of, lane);
      __syncwarp();
      const MmTileAt cur = at;
      const bool more = t + step < tiles;
      if (more) {
        walk.advance(step);
        at = walk.at();
        fetch(at, n + 1);
      }
      // every lane of the warp, or none
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.acc_full[b], (n >> 1) & 1, abort, lim.consumer))) break;
      tc_fence_after();
      const uint32_t acc = tmem + b * kN + ((uint32_t)(32 * quad) << 16);
      const bool live = row + lane < p.T;
      uint32_t* const words =
          kOut == kMmWire ? p.codes + ((size_t)cur.r * p.T + row + lane) * Wr + (cur.n0 >> 3) : nullptr;
      int i = 0;
#pragma unroll 1
      for (int chunk = first_chunk(n); chunk < kChunks; chunk += kMmSides, ++i) {
        const MmCols& cols = cols_of[i];
        uint32_t v[32];
        __syncwarp();  // a chunk ends in work of single lanes, tc_load takes the whole warp
        tc_load(acc + 32 * chunk, v);
        if (chunk + kMmSides >= kChunks) {  // the warp's last read of the tile: its columns may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&sm.acc_empty[b]), 0));
        }
        if (kOut == kMmWire && kChunks > 4 && i == 1 && more) next.grids(p, at.r, at.n0, first_chunk(n + 1), lane);
        const int n0 = cur.n0 + 32 * chunk;
        if (n0 >= p.H || row >= p.T) continue;
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(cols.scale + j);
          fmul2(f[j], f[j + 1], __int2float_rn((int)v[j]), __int2float_rn((int)v[j + 1]), sa, sa);
          fmul2(f[j + 2], f[j + 3], __int2float_rn((int)v[j + 2]), __int2float_rn((int)v[j + 3]), sa, sa);
          fmul2(f[j], f[j + 1], f[j], f[j + 1], w.x, w.y);
          fmul2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], w.z, w.w);
        }
        if (kOut != kMmWire && p.bias) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(cols.second + j);
            fadd2(f[j], f[j + 1], f[j], f[j + 1], w.x, w.y);
            fadd2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], w.z, w.w);
          }
        }
        // a store's 32 rows of 64 bytes: 16-byte piece q of row `lane` lies at piece q ^ (lane / 2 % 4)
        auto send = [&](int at_col, const uint32_t* x) {
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_shared16(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_3d(&map_out, stage, at_col, row, cur.r);
        };
        if constexpr (kOut == kMmF32) {
          uint32_t x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(f[j]);
          send(n0, x);
          if (n0 + 16 < p.H) send(n0 + 16, x + 16);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = kOut == kMmBf16 ? pack_bf16x2(f[2 * j], f[2 * j + 1]) : round_bf16x2(f[2 * j], f[2 * j + 1]);
          if (kOut == kMmBf16) send(n0, w);
          if (kOut == kMmWire && n0 < Hr) {
            uint32_t x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = wire_word(w + 4 * q, cols, 8 * q);
            store_words<kWide>(words + 4 * chunk, Wr, x, min(4, (Hr - n0) >> 3), p.T - row, stage, lane);
          }
          if (kOut == kMmWire && live && n0 + 32 > Hr) {  // kept features: 32 tokens of one lie beside one another
            uint16_t* s = p.side + (size_t)cur.r * p.k * p.T + row + lane;
            const int c0 = max(Hr - n0, 0), c1 = min(p.H - n0, 32);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const uint32_t x = (w[c / 2] >> (16 * (c & 1))) & 0xFFFFu;
              if (c >= c0 && c < c1) s[(size_t)(n0 + c - Hr) * p.T] = (uint16_t)((x & 0x7FFFu) > 0x7F80u ? 0x7FC0u : x);
            }
          }
        }
      }
      if (kOut == kMmWire && kChunks <= 4 && more) next.grids(p, at.r, at.n0, first_chunk(n + 1), lane);
    }
    if (kOut != kMmWire && lane == 0) tma_store_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // All roles are done and the CTA's own abort flag is final; both CTAs learn both flags and counts.
  if (warp == kMmEpiWarps && lane == 0) {
    const uint32_t gave_up = *abort != 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      st_cluster(cluster_addr(smem_addr(&sm.gave_up[cta]), q), gave_up);
      st_cluster(cluster_addr(smem_addr(&sm.issued[cta]), q), (uint32_t)issued);
    }
  }
  __syncwarp();
  cluster_sync();  // neither CTA's memory goes while the other still counts on it
  if (sm.gave_up[0] | sm.gave_up[1]) {  // in both CTAs or in none
    mm_pair_drain(sm, warp, lane, cta, lim);
    __syncwarp();
    cluster_sync();
  }
  tc_fence_after();
  if (warp == kMmEpiWarps + 1) tc_dealloc<2>(tmem, 2 * kN);
}

// ------------------------------------------------------------------------------------------------
// Few tokens: a CTA, or a cluster of CTAs that share K, to 128 features and all tokens.
//
// With few tokens the product is bound by reading the weights once, so the weights are the M operand
// (128 features a tile) and the tokens, padded to kTokens, the N operand: the accumulator's lane is a
// feature and its column a token, and only as many columns as there are tokens are computed, loaded and
// converted.  Where the feature tiles alone do not fill the GPU, the cluster's CTAs take a share of K
// each and their int32 sums meet in distributed shared memory: CTA q adds up the columns q kTokens / S ..
// of all S of them.  Sums of integers do not depend on the order.
//
// Weights from memory, 8 ranks, H = 8192, K = 1024: 12.8 us with one token and 13.6 with 32, 5.2 and 4.9 TB/s
// of weights; one rank, H = 4096, K = 512, one token: 3.1 us, of which the weights' bytes are 0.3.  As a wire, 4
// ranks, 32 tokens, H = 4096, K = 1024: 7.6 us, of which the weights' bytes are 2.6; the rest is set-up, eight steps
// in a row on one CTA an SM, and an epilogue that nothing runs beside.
//
// Warps 0-3 are the epilogue, warp 4 loads, warp 5 issues the products.
constexpr int kFewFeatures = 128;
constexpr int kFewThreads = 192;
constexpr int kFewMaxStages = 8;
constexpr int kFewMaxSplit = 8;

__host__ __device__ constexpr unsigned few_stage_bytes(int tokens) { return kFewFeatures * kMmK + tokens * kMmK; }
__host__ __device__ constexpr unsigned few_red_bytes(int tokens) { return kFewFeatures * tokens * 4; }

// A lane's feature: its parameters, and where its results go.
template <int kOut>
struct FewFeature {
  const MmArgs& p;
  int r, n;  // rank, feature (compact position in the wire's order)
  bool on;
  float scale = 0.0f, second = 0.0f;
  int zero = 0;

  __device__ __forceinline__ FewFeature(const MmArgs& p, int r, int n) : p(p), r(r), n(n), on(n < p.H) {
    if (!on) return;
    const size_t g = (size_t)r * p.H + n;
    scale = ld_dep(p.w_scale + g);
    if (kOut != kMmWire && p.bias) second = bf16_lo(ld_dep(p.bias + g));
    if (kOut == kMmWire) {
      const size_t h = (size_t)r * p.H + checked_index(wire_feature(p, n), p.H);
      if (n < p.H - p.k) {  // a kept feature has no grid
        second = ld_dep(p.inv_scale + h);
        zero = ld_dep(p.zero + h);
      }
    }
  }

  // `count` (at most N) tokens from t on, whose sums are acc and whose scales lie at sa.  All lanes of a
  // warp hold neighbouring features and call together.  The values are independent of one another: with 32
  // at a time the latencies of a conversion, a shuffle and a store are those of one, not of four groups.
  template <int N>
  __device__ __forceinline__ void emit(const uint32_t (&acc)[N], int t, int count, uint32_t sa) {
    const int lane = threadIdx.x & 31, Hr = p.H - p.k;
    count = min(count, p.T - t);
    if (count <= 0) return;
    float v[N];
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 s = ld_shared_float4(sa + 4 * j);
      fmul2(v[j], v[j + 1], __int2float_rn((int)acc[j]), __int2float_rn((int)acc[j + 1]), s.x, s.y);
      fmul2(v[j + 2], v[j + 3], __int2float_rn((int)acc[j + 2]), __int2float_rn((int)acc[j + 3]), s.z, s.w);
      fmul2(v[j], v[j + 1], v[j], v[j + 1], scale, scale);
      fmul2(v[j + 2], v[j + 3], v[j + 2], v[j + 3], scale, scale);
    }
    if (kOut != kMmWire && p.bias) {
#pragma unroll
      for (int j = 0; j < N; j += 2) fadd2(v[j], v[j + 1], v[j], v[j + 1], second, second);
    }
    if (kOut == kMmF32) {
      float* o = static_cast<float*>(p.out) + ((size_t)r * p.T + t) * p.ldo + n;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (on && j < count) o[(size_t)j * p.ldo] = v[j];
    } else if (kOut == kMmBf16) {
      // two tokens at a time: an even lane takes the first token's features n, n + 1, an odd lane the
      // second token's n - 1, n (H is a multiple of 8, so both are features or neither)
      const bool odd = lane & 1;
      uint16_t* o = static_cast<uint16_t*>(p.out) + ((size_t)r * p.T + t + odd) * p.ldo + (n - odd);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
        const uint32_t w = odd ? pack_bf16x2(other, v[j + 1]) : pack_bf16x2(v[j], other);
        if (on && j + odd < count) *reinterpret_cast<uint32_t*>(o + (size_t)j * p.ldo) = w;
      }
    } else {
      // a token's code of this feature to nibble lane % 8, then 8 tokens x 8 lanes are exchanged so that
      // lane i of 8 holds the whole word of token t + i
      const int i = lane & 7;
#pragma unroll
      for (int j0 = 0; j0 < N; j0 += 8) {
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float b = bf16_lo(round_bf16x2(v[j0 + j], 0.0f));
          const int c = __float2int_rn(__fmul_rn(b, second));  // saturating; NaN -> 0
          x[j] = (uint32_t)(min(max(c, -zero), 15 - zero) + zero) << (4 * i);
        }
#pragma unroll
        for (int step = 0; step < 3; ++step) {
          const bool up = (i >> step) & 1;
#pragma unroll
          for (int j = 0; j < (4 >> step); ++j) {
            const uint32_t keep = up ? x[2 * j + 1] : x[2 * j], give = up ? x[2 * j] : x[2 * j + 1];
            x[j] = keep | __shfl_xor_sync(0xFFFFFFFFu, give, 1 << step);
          }
        }
        if (n < Hr && j0 + i < count) p.codes[((size_t)r * p.T + t + j0 + i) * (Hr / 8) + (n >> 3)] = x[0];
      }
      if (on && n >= Hr) {
        uint16_t* s = p.side + ((size_t)r * p.k + (n - Hr)) * p.T + t;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j < count) s[j] = (uint16_t)pack_bf16x2(v[j], 0.0f);
      }
    }
  }
};

// At most kTokens tokens.
template <int kOut, int kTokens>
__global__ void __launch_bounds__(kFewThreads)
    int8_matmul_few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                           const MmArgs p, int split_log2, int stages, WaitLimits lim) {
  extern __shared__ unsigned char s_raw[];
  __shared__ uint64_t s_full[kFewMaxStages], s_empty[kFewMaxStages], s_acc;
  __shared__ __align__(16) float s_scale[kTokens + 32];  // the last group's loads may go past the tokens
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  unsigned char* const base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  int* const red = reinterpret_cast<int*>(base + stages * few_stage_bytes(kTokens));  // [split][kTokens / split][128]
  constexpr uint32_t kColumns = kTokens < 32 ? 32 : kTokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = 1 << split_log2;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = (int)(blockIdx.x >> split_log2) * kFewFeatures, r = blockIdx.y;
  const int kc = (p.K + kMmK - 1) / kMmK;
  const int c0 = (kc * rank) >> split_log2, c1 = (kc * (rank + 1)) >> split_log2;
  volatile int* abort = &s_abort;
  int issued = 0;  // the load lane's steps

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 1);
    }
    mbar_init(&s_acc, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 5) tc_alloc<1>(&s_tmem, kColumns);
  if (warp == 4 && lane == 0) {
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_w);
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_arrive();  // here: this CTA's memory may be written
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_trigger();
  grid_wait();

  if (warp == 4) {  // ---------------------------------------------------------- loads
    if (lane == 0) {
      producer_start_delay(lim.start_delay);
      int s = 0, phase = 1;
      for (int c = c0; c < c1; ++c, ++issued) {
        if (issued >= stages && !mbar_wait(&s_empty[s], phase, abort, lim.producer)) break;
        unsigned char* at = base + s * few_stage_bytes(kTokens);
        mbar_arrive_expect_tx(&s_full[s], few_stage_bytes(kTokens));
        tma_load_3d(smem_addr(at), &map_w, c * kMmK, n0, r, smem_addr(&s_full[s]));
        tma_load_3d(smem_addr(at + kFewFeatures * kMmK), &map_a, c * kMmK, 0, r, smem_addr(&s_full[s]));
        if (++s == stages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 5) {  // ---------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t idesc = tc_idesc(kFewFeatures, kTokens);
      int s = 0, phase = 0;
      for (int c = c0; c < c1; ++c) {
        if (!mbar_wait(&s_full[s], phase, abort, lim.consumer)) break;
        tc_fence_after();
        const uint32_t at = smem_addr(base + s * few_stage_bytes(kTokens));
        const uint64_t dw = tc_desc(at), da = tc_desc(at + kFewFeatures * kMmK);
#pragma unroll
        for (int k = 0; k < kMmK / 32; ++k) tc_mma<1>(tmem, dw + 2 * k, da + 2 * k, idesc, c > c0 || k > 0);
        tc_commit<1>(&s_empty[s]);
        if (++s == stages) s = 0, phase ^= 1;
      }
      tc_commit<1>(&s_acc);  // also after an abort
    }
  }
  FewFeature<kOut> feature(p, r, warp < 4 ? n0 + 32 * warp + lane : p.H);
  const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  bool ok = true;
  if (warp < 4) {  // ------------------------------------------------------------ epilogue
    for (int j = threadIdx.x; j < kTokens; j += 128)
      s_scale[j] = j < p.T ? ld_dep(p.a_scale + (size_t)r * p.T + j) : 0.0f;
    __syncwarp();
    named_barrier_sync(128);
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_acc, 0, abort, lim.consumer)) && !*abort;
    ok = __all_sync(0xFFFFFFFFu, ok);
    tc_fence_after();
    if (ok && split == 1) {
      constexpr int kGroup = kTokens < 32 ? 8 : 32;
#pragma unroll 1
      for (int j = 0; j < p.T; j += kGroup) {
        uint32_t v[kGroup];
        __syncwarp();  // emit's stores are those of single lanes, tc_load takes the whole warp
        tc_load(acc + j, v);
        feature.emit(v, j, kGroup, smem_addr(s_scale + j));
      }
    } else if (ok) {
      // the columns go to the CTAs that add them up
      constexpr int kTokensLog2 = kTokens == 16 ? 4 : kTokens == 32 ? 5 : 6;
      const int width_log2 = kTokensLog2 - split_log2;
      const uint32_t mine = smem_addr(red + ((rank << width_log2) * kFewFeatures + threadIdx.x));
#pragma unroll 1
      for (int j = 0; j < kTokens; j += 8) {
        uint32_t v[8];
        tc_load(acc + j, v);
        if (j == 0) cluster_wait();  // every CTA of the cluster is there
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = (j + i) >> width_log2, c = (j + i) & ((1 << width_log2) - 1);
          st_cluster(cluster_addr(mine + c * kFewFeatures * 4, q), v[i]);
        }
      }
    }
  }
  __syncwarp();  // the roles of warps 4 and 5 are one lane's, the barrier is the whole warp's
  if (split > 1 && (warp >= 4 || !ok)) cluster_wait();
  tc_fence_before();
  __syncthreads();
  // All roles are done and the abort flag is final.  After a wait that gave up: the loads in flight have landed
  // before the CTA leaves, and the products are done before tensor memory is freed.
  if (*abort && lane == 0) {
    int ignore = 0;
    if (warp == 4)
      for (int j = max(0, issued - stages); j < issued; ++j)
        mbar_wait(&s_full[j % stages], (j / stages) & 1, &ignore, lim.producer);
    if (warp == 5) mbar_wait(&s_acc, 0, &ignore, lim.producer);
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();  // all parts of this CTA's columns are here
    if (warp < 4 && ok) {
      const int width = kTokens >> split_log2;
#pragma unroll 1
      for (int c = 0; c < width; c += 8) {
        uint32_t v[8] = {};
#pragma unroll 2
        for (int q = 0; q < split; ++q) {
          const uint32_t at = smem_addr(red) + 4 * ((q * width + c) * kFewFeatures + threadIdx.x);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < width) v[i] += ld_shared(at + 4 * i * kFewFeatures);
        }
        feature.emit(v, rank * width + c, min(width - c, 8), smem_addr(s_scale) + 4 * (rank * width + c));
      }
    }
  }
  tc_fence_after();
  if (warp == 5) tc_dealloc<1>(tmem, kColumns);
}

}  // namespace hq
