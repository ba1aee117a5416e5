// hq_api.cu -- the C ABI of libhq.so (declared in include/hq.h).
//
// One translation unit holds every kernel (so the device error word is a single symbol).  Each
// entry point checks its arguments on the host, picks a launch shape, enqueues one kernel on the
// caller's stream and returns; nothing is allocated and nothing waits, except
// hq_read_device_error, which synchronises the stream it is given.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <mutex>

#include "hq.h"
#include "hq_common.cuh"
#include "hq_tma.cuh"
#include "k_calibrate.cuh"
#include "k_dequant.cuh"
#include "k_fused.cuh"
#include "k_int8mm.cuh"
#include "k_norm.cuh"
#include "k_quantize.cuh"
#include "k_select.cuh"
#include "k_tokens.cuh"

namespace {

constexpr int kMaxRanks = 64;
static_assert(kMaxRanks <= hq::kSelMaxRanks, "the parameter kernel stages one range per rank");
constexpr int kMaxDevices = 64;
constexpr long long kMaxStallDelayCycles = 1LL << 31;  // about a second

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hq_status check_shape(int P, int H, int k) {
  if (P < 1 || P > kMaxRanks) return HQ_ERR_INVALID_ARG;
  if (H < 8 || H > hq::kMaxH || (H % 8) != 0) return HQ_ERR_INVALID_ARG;
  if (k < 0 || k > H || (k % 8) != 0) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

// Resident CTAs per SM of one kernel for each rank count P (its shared memory grows with P),
// queried once per device; the kernel's dynamic shared-memory limit is raised to the largest size
// requested so far.
struct OccupancyCache {
  int smem_set = 0;
  int per_sm[kMaxRanks + 1] = {};
};

// Launch-shape facts cached per device: SM count and resident CTAs per SM of each kernel.
struct DeviceInfo {
  int sms = 0;
  int qt_blocks = 0;
  bool select_smem_set = false;
  bool pair_smem_set[3][2][2] = {};  // [output][features 128, 256][wide codes]
  bool norm_smem_set[2][2][2] = {};  // [fp32 y][fp32 residual][threads all full]
  bool few_smem_set[3][3] = {};      // [output][tokens 16, 32, 64]
  OccupancyCache dequant_tma[2][2];  // [fp32 out][bf16 shards]
  OccupancyCache dequant_cp[2][2];
  OccupancyCache fused[2];           // [fp32 out]
};

// cuTensorMapEncodeTiled, fetched once through the runtime (no link-time libcuda dependency).
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::mutex g_encode_mu;

bool get_encode() {
  std::lock_guard<std::mutex> lock(g_encode_mu);
  if (g_encode) return true;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return false;
  g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return true;
}

// Row-major 2-D tensor [rows][cols] of `elem`-byte elements (row pitch `pitch` bytes, cols*elem
// when 0; a multiple of 16) read in boxes of box_rows x box_cols; out-of-range box elements read as 0.
bool encode_2d(CUtensorMap* map, const void* base, CUtensorMapDataType type, size_t elem, uint64_t cols,
               uint64_t rows, uint32_t box_cols, uint32_t box_rows,
               CUtensorMapL2promotion promo = CU_TENSOR_MAP_L2_PROMOTION_L2_256B, uint64_t pitch = 0) {
  if (!get_encode()) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch ? pitch : cols * elem};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return g_encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

hq_status device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return HQ_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (d.sms == 0) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return HQ_ERR_CUDA;
    const int qt_smem = (int)(sizeof(hq::QtSmem) + 128);
    if (cudaFuncSetAttribute(hq::quantize_pack_tma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             qt_smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.qt_blocks, hq::quantize_pack_tma_kernel,
                                                      hq::kQtThreads, qt_smem) != cudaSuccess)
      return HQ_ERR_CUDA;
    if (d.qt_blocks < 1) d.qt_blocks = 1;
  }
  *out = &d;
  return HQ_OK;
}

hq_status launched() { return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA; }

// CTAs of `kern` resident per SM with `smem` bytes of dynamic shared memory (at least 1), from the
// device's cache; the first use for a P sets the shared-memory limit and runs the query.
template <typename Kernel>
hq_status occupancy(OccupancyCache& c, Kernel kern, int threads, size_t smem, int P, int* per_sm) {
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (c.per_sm[P] == 0) {
    if ((int)smem > c.smem_set) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return HQ_ERR_CUDA;
      c.smem_set = (int)smem;
    }
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess) return HQ_ERR_CUDA;
    c.per_sm[P] = n < 1 ? 1 : n;
  }
  *per_sm = c.per_sm[P];
  return HQ_OK;
}

// Wait bounds of the pipeline kernels.  Normal launches use the long default everywhere; the
// abort self-test (hq_selftest_set_pipeline_stall) shortens the consumers' bound and delays the
// producers' first loads.
std::atomic<long long> g_stall_consumer_limit{0};
std::atomic<long long> g_stall_producer_delay{0};

hq::WaitLimits wait_limits() {
  const long long c = g_stall_consumer_limit.load(), d = g_stall_producer_delay.load();
  if (c == 0 && d == 0) return hq::WaitLimits{hq::kWaitLimitCycles, hq::kWaitLimitCycles, 0};
  return hq::WaitLimits{c, hq::kWaitLimitCycles, d};
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// A launch that may begin under the kernel ahead of it in the stream; the kernel waits for that one
// (grid_wait) before it touches global memory.  cluster > 1: in clusters of that many CTAs.
template <typename Kernel, typename... Args>
hq_status launch_dependent(Kernel kern, dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                           const Args&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return HQ_OK;
  cudaGetLastError();
  return HQ_ERR_CUDA;
}

// One wave of `resident` CTAs over S slices of nb_all row blocks each: every slice gets `base`
// row chunks and slices 0..extra-1 one more; never more chunks than blocks, at least one.
struct WaveChunks {
  int base, extra;
};
WaveChunks wave_chunks(long long resident, int S, long long nb_all) {
  long long base = resident / S, extra = resident - base * S;
  if (base < 1) base = 1, extra = 0;
  if (base >= nb_all) base = std::max(nb_all, 1LL), extra = 0;
  return WaveChunks{(int)base, (int)extra};
}

// Slices x row chunks of the cp.async dequant-reduce kernel: one wave of CTAs at most.
void slice_chunks(int T, int S, long long resident, int rows_per_block, int* chunks, int* rows_per_chunk) {
  long long c = resident / S;
  if (c < 1) c = 1;
  const long long max_c = ceil_div(T, rows_per_block);
  if (c > max_c) c = max_c;
  long long rpc = ceil_div(ceil_div(T, c), rows_per_block) * rows_per_block;
  *rows_per_chunk = (int)rpc;
  *chunks = (int)ceil_div(T, rpc);
}

// Where dequant-reduce reads the P ranks' wires: one stacked buffer [P][T][W] / [P][k][T], or one
// buffer per rank (host arrays of P device pointers; each may be a peer GPU's memory).
struct WireSrc {
  const uint32_t* codes = nullptr;
  const uint16_t* side = nullptr;
  const uint32_t* const* codes_r = nullptr;
  const uint16_t* const* side_r = nullptr;
  bool per_rank = false;
};

// nbatch > 1: nbatch independent problems of P ranks each, stacked (problem b: ranks b*P .. b*P+P-1
// of the wire and the parameters, output rows b*T .. b*T+T-1); one launch when TMA can stage them.
template <typename OutT, bool kShard>
hq_status launch_dequant(const WireSrc& src, int P, int T, int H, int k, const int32_t* keep_idx, const float* scale,
                         const uint8_t* zero, void* out, int ldo, cudaStream_t st, DeviceInfo& d, int nbatch = 1) {
  const int S = (H + 8 * hq::kDqSliceGroups - 1) / (8 * hq::kDqSliceGroups);
  const int Wr = (H - k) / 8;
  hq::DqWire wire;
  memset(&wire, 0, sizeof wire);
  wire.per_rank = src.per_rank ? 1 : 0;
  bool tma = Wr >= 4 && Wr % 4 == 0;
  // side[r][j][t] as [k][T] rows: boxes of 32 rows (inner) x 32 kept features; needs rows of a
  // multiple of 16 bytes (T % 8 == 0), else the kept sums read the side buffer directly
  bool side_tma = k > 0 && T % 8 == 0;
  if (!src.per_rank) {
    tma = tma && aligned(src.codes, 16) &&
          encode_2d(&wire.code[0], src.codes, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)Wr,
                    (uint64_t)nbatch * P * T, hq::kDtWords, hq::kDtTileRows);
    side_tma = tma && side_tma &&
               encode_2d(&wire.side[0], src.side, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, (uint64_t)T,
                         (uint64_t)nbatch * P * k, hq::kDtTileRows, hq::kDtSideCols, CU_TENSOR_MAP_L2_PROMOTION_NONE);
  } else {
    for (int r = 0; r < P && tma; ++r)
      tma = encode_2d(&wire.code[r], src.codes_r[r], CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)Wr, (uint64_t)T,
                      hq::kDtWords, hq::kDtTileRows);
    for (int r = 0; r < P && side_tma; ++r)
      side_tma = encode_2d(&wire.side[r], src.side_r[r], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, (uint64_t)T, (uint64_t)k,
                           hq::kDtTileRows, hq::kDtSideCols, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    for (int r = 0; r < P; ++r) wire.side_ptr[r] = k > 0 ? src.side_r[r] : nullptr;
    if (!tma || nbatch != 1) return HQ_ERR_INVALID_ARG;  // per-rank buffers: TMA kernel, one problem
    side_tma = side_tma && tma;
  }
  constexpr int kF32 = std::is_same<OutT, float>::value ? 1 : 0;
  if (tma) {
    const size_t smem = hq::dt_smem_bytes(P);
    auto kern = hq::dequant_reduce_tma_kernel<OutT, kShard>;
    int per_sm = 0;
    if (occupancy(d.dequant_tma[kF32][kShard], kern, hq::kDtThreads, smem, P, &per_sm) != HQ_OK) return HQ_ERR_CUDA;
    // one wave that fills every resident CTA slot (wave_chunks)
    const long long nb_all = ceil_div(T, hq::kDtTileRows);
    const WaveChunks wc = wave_chunks((long long)d.sms * per_sm / nbatch, S, nb_all);
    const dim3 grid((unsigned)(S * wc.base + wc.extra), (unsigned)nbatch);
    kern<<<grid, hq::kDtThreads, smem, st>>>(wire, side_tma ? 1 : 0, src.side, P, T, H, k, keep_idx, scale, zero,
                                             static_cast<OutT*>(out), ldo, S, wc.base, wc.extra, wait_limits());
    return launched();
  }
  if (nbatch > 1) {  // the cp.async kernel takes one problem per launch
    const int Wr2 = (H - k) / 8;
    for (int b = 0; b < nbatch; ++b) {
      WireSrc one;
      one.codes = src.codes ? src.codes + (size_t)b * P * T * Wr2 : nullptr;
      one.side = src.side ? src.side + (size_t)b * P * k * T : nullptr;
      const hq_status r = launch_dequant<OutT, kShard>(one, P, T, H, k, keep_idx, scale + (size_t)b * P * H,
                                                       zero + (size_t)b * P * H,
                                                       static_cast<OutT*>(out) + (size_t)b * T * ldo, ldo, st, d, 1);
      if (r != HQ_OK) return r;
    }
    return HQ_OK;
  }
  const size_t smem = hq::dq_smem_bytes(P);
  auto kern = hq::dequant_reduce_kernel<OutT, kShard>;
  int per_sm = 0;
  if (occupancy(d.dequant_cp[kF32][kShard], kern, hq::kDqThreads, smem, P, &per_sm) != HQ_OK) return HQ_ERR_CUDA;
  int chunks, rpc;
  slice_chunks(T, S, (long long)d.sms * per_sm, hq::kDqR, &chunks, &rpc);
  kern<<<(unsigned)(S * chunks), hq::kDqThreads, smem, st>>>(src.codes, src.side, P, T, H, k, keep_idx, scale,
                                                              zero, static_cast<OutT*>(out), ldo, S, chunks, rpc);
  return launched();
}

template <typename OutT>
hq_status launch_fused(const uint16_t* x, int ldx, int P, int T, int H, int k, const int32_t* keep_idx,
                       const float* scale, const float* inv_scale, const uint8_t* zero, void* out, int ldo,
                       cudaStream_t st, DeviceInfo& d) {
  const int S = (H + hq::kFuSlice - 1) / hq::kFuSlice;
  CUtensorMap map;
  if (!encode_2d(&map, x, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, (uint64_t)H, (uint64_t)P * T, hq::kFuSlice,
                 hq::kFuTileRows, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, (uint64_t)ldx * 2))
    return HQ_ERR_CUDA;
  const size_t smem = hq::fu_smem_bytes(P);
  auto kern = hq::compress_reduce_kernel<OutT>;
  int per_sm = 0;
  if (occupancy(d.fused[std::is_same<OutT, float>::value ? 1 : 0], kern, hq::kFuThreads, smem, P, &per_sm) != HQ_OK)
    return HQ_ERR_CUDA;
  // one wave that fills every resident CTA slot (wave_chunks)
  const WaveChunks wc = wave_chunks((long long)d.sms * per_sm, S, (T + hq::kFuTileRows - 1) / hq::kFuTileRows);
  kern<<<(unsigned)(S * wc.base + wc.extra), hq::kFuThreads, smem, st>>>(map, P, T, H, k, keep_idx, scale, inv_scale,
                                                                          zero, static_cast<OutT*>(out), ldo, S,
                                                                          wc.base, wc.extra, wait_limits());
  return launched();
}

// hq_read_device_error: the error word is taken and cleared in one atomic exchange, so an error a
// kernel on another stream records at the same moment lands either in this read or in the word
// for the next one; the value goes through a second device word to the host.
__device__ unsigned int g_error_taken = 0;
__global__ void take_error_kernel() { g_error_taken = atomicExch(&hq::g_error_word, 0u); }
std::mutex g_error_mu;  // one read at a time per process (they share g_error_taken)

// Bounded-wait self-test: one thread waits on an mbarrier that nothing arrives on.
__global__ void selftest_wait_kernel(long long limit) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  hq::mbar_init(&bar, 1);
  abort = 0;
  hq::fence_barrier_init();
  hq::mbar_wait(&bar, 0, &abort, limit);
}

// A leading dimension: at least the width, and rows of a multiple of 16 bytes.
bool ld_ok(int ld, int H) { return ld >= H && ld % 8 == 0; }

// Argument checks and launch shared by the two reductions (kShard: each rank's value rounded to
// bf16 before it is added); the output has a row pitch of ldo elements.
template <bool kShard>
hq_status dequant_entry(const uint32_t* codes, const uint16_t* side, int P, int T, int H, int k,
                        const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                        const uint8_t* zero, void* out, int ldo, hq_out_dtype out_dtype, void* stream) {
  if (check_shape(P, H, k) != HQ_OK || T < 0 || !ld_ok(ldo, H)) return HQ_ERR_INVALID_ARG;
  if (out_dtype != HQ_OUT_BF16 && out_dtype != HQ_OUT_F32) return HQ_ERR_INVALID_ARG;
  if (!scale || !zero) return HQ_ERR_INVALID_ARG;
  if ((k > 0 && !keep_idx) || (k < H && !rest_idx)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && (!out || (k > 0 && !side) || (k < H && !codes))) return HQ_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(side, 16) || !aligned(codes, 4) || !aligned(scale, 16) ||
      !aligned(zero, 16) || !aligned(keep_idx, 4) || !aligned(rest_idx, 4))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  WireSrc src;
  src.codes = codes;
  src.side = side;
  if (out_dtype == HQ_OUT_BF16)
    return launch_dequant<uint16_t, kShard>(src, P, T, H, k, keep_idx, scale, zero, out, ldo, st, *d);
  return launch_dequant<float, kShard>(src, P, T, H, k, keep_idx, scale, zero, out, ldo, st, *d);
}

// The wires of the P ranks in P separate buffers (each possibly a peer GPU's memory).
hq_status dequant_ranks_entry(const uint32_t* const* codes, const uint16_t* const* side, int P, int T, int H, int k,
                              const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                              const uint8_t* zero, void* out, hq_out_dtype out_dtype, void* stream) {
  if (check_shape(P, H, k) != HQ_OK || P > hq::kMaxRankMaps || T < 0) return HQ_ERR_INVALID_ARG;
  if (H - k < 32 || (H - k) % 32 != 0) return HQ_ERR_INVALID_ARG;  // code rows staged by TMA
  if (out_dtype != HQ_OUT_BF16 && out_dtype != HQ_OUT_F32) return HQ_ERR_INVALID_ARG;
  if (!scale || !zero || !rest_idx || (k > 0 && !keep_idx)) return HQ_ERR_INVALID_ARG;
  if (T > 0) {
    if (!out || !codes || (k > 0 && !side)) return HQ_ERR_INVALID_ARG;
    for (int r = 0; r < P; ++r) {
      if (!codes[r] || (k > 0 && !side[r])) return HQ_ERR_INVALID_ARG;
      if (!aligned(codes[r], 16) || (k > 0 && !aligned(side[r], 16))) return HQ_ERR_MISALIGNED;
    }
  }
  if (!aligned(out, 16) || !aligned(scale, 16) || !aligned(zero, 16) || !aligned(keep_idx, 4) ||
      !aligned(rest_idx, 4))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  WireSrc src;
  src.codes_r = codes;
  src.side_r = k > 0 ? side : nullptr;
  src.per_rank = true;
  if (k == 0) {
    static const uint16_t* const kNone[hq::kMaxRankMaps] = {};
    src.side_r = kNone;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (out_dtype == HQ_OUT_BF16)
    return launch_dequant<uint16_t, false>(src, P, T, H, k, keep_idx, scale, zero, out, H, st, *d);
  return launch_dequant<float, false>(src, P, T, H, k, keep_idx, scale, zero, out, H, st, *d);
}

hq_status calibrate_entry(const uint16_t* x, int ldx, int P, int T, int H, float beta, int first_batch,
                          float* ema_min, float* ema_max, void* stream) {
  if (check_shape(P, H, 0) != HQ_OK || T < 1 || !ld_ok(ldx, H)) return HQ_ERR_INVALID_ARG;
  if (!(beta >= 0.0f && beta < 1.0f)) return HQ_ERR_INVALID_ARG;
  if (!x || !ema_min || !ema_max) return HQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(ema_min, 16) || !aligned(ema_max, 16)) return HQ_ERR_MISALIGNED;
  const float one_minus_beta = 1.0f - beta;
  dim3 grid((unsigned)((H + hq::kCalCols - 1) / hq::kCalCols), (unsigned)P);
  hq::calibrate_kernel<<<grid, hq::kCalThreads, 0, (cudaStream_t)stream>>>(
      x, ldx, T, H, beta, one_minus_beta, first_batch ? 1 : 0, ema_min, ema_max);
  return launched();
}

hq_status quantize_entry(const uint16_t* x, int ldx, int P, int T, int H, int k, const int32_t* keep_idx,
                         const int32_t* rest_idx, const float* inv_scale, const uint8_t* zero, uint32_t* codes,
                         uint16_t* side, void* stream) {
  if (check_shape(P, H, k) != HQ_OK || T < 0 || !ld_ok(ldx, H)) return HQ_ERR_INVALID_ARG;
  if (!inv_scale || !zero) return HQ_ERR_INVALID_ARG;
  if ((k > 0 && !keep_idx) || (k < H && !rest_idx)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && (!x || (k > 0 && !side) || (k < H && !codes))) return HQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(side, 16) || !aligned(codes, 4) || !aligned(inv_scale, 16) ||
      !aligned(zero, 16) || !aligned(keep_idx, 4) || !aligned(rest_idx, 4))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  const int S = (H + hq::kQtSlice - 1) / hq::kQtSlice;
  CUtensorMap map_x;  // x as 32-bit pairs of bf16: the box is 132 pairs = 264 features wide
  if (!encode_2d(&map_x, x, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)H / 2, (uint64_t)P * T, hq::kQtBoxU32,
                 hq::kQtTileRows, CU_TENSOR_MAP_L2_PROMOTION_NONE,  // 528-byte rows: no 256-byte over-fetch
                 (uint64_t)ldx * 2))
    return HQ_ERR_CUDA;
  // J CTAs per slice, one wave; each takes a balanced contiguous range of (rank, 64-row block) units
  const long long units = (long long)P * ceil_div(T, hq::kQtTileRows);
  long long J = (long long)d->sms * d->qt_blocks / S;
  if (J < 1) J = 1;
  if (J > units) J = units;
  hq::quantize_pack_tma_kernel<<<(unsigned)(S * J), hq::kQtThreads, sizeof(hq::QtSmem) + 128,
                                 (cudaStream_t)stream>>>(map_x, x, ldx, P, T, H, k, keep_idx, rest_idx,
                                                         inv_scale, zero, codes, side, S, (int)J,
                                                         wait_limits());
  return launched();
}

hq_status compress_entry(const uint16_t* x, int ldx, int P, int T, int H, int k, const int32_t* keep_idx,
                         const int32_t* rest_idx, const float* scale, const float* inv_scale, const uint8_t* zero,
                         void* out, int ldo, hq_out_dtype out_dtype, uint32_t* codes_or_null,
                         uint16_t* side_or_null, void* stream) {
  if (check_shape(P, H, k) != HQ_OK || T < 0 || !ld_ok(ldx, H) || !ld_ok(ldo, H)) return HQ_ERR_INVALID_ARG;
  if (out_dtype != HQ_OUT_BF16 && out_dtype != HQ_OUT_F32) return HQ_ERR_INVALID_ARG;
  if (!scale || !inv_scale || !zero) return HQ_ERR_INVALID_ARG;
  if ((k > 0 && !keep_idx) || (k < H && !rest_idx)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && (!x || !out)) return HQ_ERR_INVALID_ARG;
  const bool wire = codes_or_null || side_or_null;
  if (T > 0 && wire && ((k > 0 && !side_or_null) || (k < H && !codes_or_null))) return HQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(scale, 16) || !aligned(inv_scale, 16) ||
      !aligned(zero, 16) || !aligned(keep_idx, 4) || !aligned(rest_idx, 4) ||
      !aligned(codes_or_null, 4) || !aligned(side_or_null, 16))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  if (wire) {
    const hq_status q = quantize_entry(x, ldx, P, T, H, k, keep_idx, rest_idx, inv_scale, zero, codes_or_null,
                                       side_or_null, stream);
    if (q != HQ_OK) return q;
  }
  if (out_dtype == HQ_OUT_BF16)
    return launch_fused<uint16_t>(x, ldx, P, T, H, k, keep_idx, scale, inv_scale, zero, out, ldo, st, *d);
  return launch_fused<float>(x, ldx, P, T, H, k, keep_idx, scale, inv_scale, zero, out, ldo, st, *d);
}

// The two-step all-reduce's workspace: step-1 wire (codes, side), the reduced tensor, and the P
// reducers' step-2 wires, each region 256-byte aligned.
struct TwoStepLayout {
  size_t codes, side, red, codes2, side2, total;
};
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
TwoStepLayout two_step_layout(int P, int T, int H, int k, int k2) {
  TwoStepLayout L;
  size_t off = 0;
  L.codes = off;
  off += round256((size_t)P * T * (H - k) / 2);
  L.side = off;
  off += round256((size_t)P * k * T * 2);
  L.red = off;
  off += round256((size_t)T * H * 2);
  L.codes2 = off;
  off += round256((size_t)T * (H - k2) / 2);  // P blocks of T/P rows
  L.side2 = off;
  off += round256((size_t)k2 * T * 2);
  L.total = off;
  return L;
}

hq_status two_step_entry(const uint16_t* x, int P, int T, int H, int k, const int32_t* keep_idx,
                         const int32_t* rest_idx, const float* scale, const float* inv_scale, const uint8_t* zero,
                         int k2, const int32_t* keep2, const int32_t* rest2, const float* scale2,
                         const float* inv_scale2, const uint8_t* zero2, void* workspace, size_t workspace_bytes,
                         void* out, hq_out_dtype out_dtype, void* stream) {
  if (check_shape(P, H, k) != HQ_OK || check_shape(P, H, k2) != HQ_OK || T < 0 || T % P != 0 || H % 16 != 0)
    return HQ_ERR_INVALID_ARG;  // H % 16: every reducer's row of zero2 starts on a 16-byte boundary
  if (out_dtype != HQ_OUT_BF16 && out_dtype != HQ_OUT_F32) return HQ_ERR_INVALID_ARG;
  if (!scale2 || !inv_scale2 || !zero2 || (k2 > 0 && !keep2) || (k2 < H && !rest2)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && !out) return HQ_ERR_INVALID_ARG;
  if (!aligned(scale2, 16) || !aligned(inv_scale2, 16) || !aligned(zero2, 16) || !aligned(keep2, 4) ||
      !aligned(rest2, 4) || !aligned(out, 16))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  const TwoStepLayout L = two_step_layout(P, T, H, k, k2);
  if (!workspace || workspace_bytes < L.total) return HQ_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return HQ_ERR_MISALIGNED;
  char* ws = static_cast<char*>(workspace);
  uint32_t* codes = reinterpret_cast<uint32_t*>(ws + L.codes);
  uint16_t* side = reinterpret_cast<uint16_t*>(ws + L.side);
  uint16_t* red = reinterpret_cast<uint16_t*>(ws + L.red);
  uint32_t* codes2 = reinterpret_cast<uint32_t*>(ws + L.codes2);
  uint16_t* side2 = reinterpret_cast<uint16_t*>(ws + L.side2);
  // step 1: every rank's wire, the rank-ordered reduction into the reduced tensor (bf16)
  hq_status st = quantize_entry(x, H, P, T, H, k, keep_idx, rest_idx, inv_scale, zero, codes, side, stream);
  if (st != HQ_OK) return st;
  st = dequant_entry<false>(codes, side, P, T, H, k, keep_idx, rest_idx, scale, zero, red, H, HQ_OUT_BF16, stream);
  if (st != HQ_OK) return st;
  // step 2: reducer j re-quantizes its row block with grid row j, and the block is dequantized
  // with it.  The reduced tensor [T][H] is [P][T/P][H]: reducer j's block is "rank" j of one
  // quantize-pack call (whose output layout is exactly the P step-2 wires, block after block),
  // and the P blocks are P independent one-rank problems of one batched dequant-reduce launch.
  const int Tb = T / P;
  st = quantize_entry(red, H, P, Tb, H, k2, keep2, rest2, inv_scale2, zero2, codes2, side2, stream);
  if (st != HQ_OK) return st;
  if (Tb == 0) return HQ_OK;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  WireSrc src;
  src.codes = codes2;
  src.side = side2;
  if (out_dtype == HQ_OUT_BF16)
    return launch_dequant<uint16_t, false>(src, 1, Tb, H, k2, keep2, scale2, zero2, out, H, (cudaStream_t)stream, *d, P);
  return launch_dequant<float, false>(src, 1, Tb, H, k2, keep2, scale2, zero2, out, H, (cudaStream_t)stream, *d, P);
}

hq_status quantize_tokens_entry(const uint16_t* x, int ldx, int64_t rows, int K, int8_t* q, int ldq, float* scale,
                                void* stream) {
  if (rows < 0 || K < 1 || K > HQ_INT8_MAX_K || !ld_ok(ldx, K) || ldq < K || ldq % 16 != 0) return HQ_ERR_INVALID_ARG;
  if (rows > 0x7FFFFFFFLL) return HQ_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !q || !scale)) return HQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return HQ_ERR_MISALIGNED;
  if (rows == 0) return HQ_OK;
  const long long n = rows;
  const int nvec = (int)ceil_div(K, 8);
  cudaStream_t st = (cudaStream_t)stream;
  auto go = [&](auto kern, long long ctas, int threads) {
    return launch_dependent(kern, dim3((unsigned)ctas), threads, 0, st, 1, x, ldx, n, K, q, ldq, scale);
  };
  auto cta = [&](int nv) { return (int)(32 * ceil_div(ceil_div(nvec, nv), 32)); };
  if (nvec <= 8) return go(hq::quantize_tokens_kernel<1, 8>, ceil_div(n, 16), 128);
  if (nvec <= 16) return go(hq::quantize_tokens_kernel<2, 8>, ceil_div(n, 16), 128);
  if (nvec <= 32) return go(hq::quantize_tokens_kernel<4, 8>, ceil_div(n, 16), 128);
  if (nvec <= 64) return go(hq::quantize_tokens_kernel<2, 32>, ceil_div(n, 4), 128);
  if (nvec <= 128) return go(hq::quantize_tokens_kernel<4, 32>, ceil_div(n, 4), 128);
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  // Longer rows: one load a thread where rows are few, for the shortest chain; with more rows a warp holds up
  // to 2048 elements (32768 rows: 31.5 us, a CTA with one load a thread 49), and a CTA has four loads a thread
  // (8192 rows of 8192: 36 us, 59 with one) and above 8192 elements eight (8192 rows of 14336: 61 us, 75 with four).
  if (n < 4LL * d->sms && nvec <= hq::kRowMaxThreads) return go(hq::quantize_tokens_kernel<1, 0>, n, cta(1));
  if (nvec <= 256) return go(hq::quantize_tokens_kernel<8, 32>, ceil_div(n, 4), 128);
  if (nvec <= 1024) return go(hq::quantize_tokens_kernel<4, 0>, n, cta(4));
  return go(hq::quantize_tokens_kernel<8, 0>, n, cta(8));
}

// The checks that the two products share.
hq_status matmul_check(const int8_t* a, int lda, const float* a_scale, const int8_t* w, int ldw, const float* w_scale,
                       int P, int T, int H, int max_h, int K) {
  if (P < 1 || P > kMaxRanks || T < 0 || H < 8 || H > max_h || H % 8 != 0) return HQ_ERR_INVALID_ARG;
  if (K < 1 || K > HQ_INT8_MAX_K || lda < K || lda % 16 != 0 || ldw < K || ldw % 16 != 0) return HQ_ERR_INVALID_ARG;
  if (!w || !w_scale || (T > 0 && (!a || !a_scale))) return HQ_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(w_scale, 16) || !aligned(a_scale, 4)) return HQ_ERR_MISALIGNED;
  return HQ_OK;
}

// [ranks][rows][cols] of `elem`-byte elements, rows `pitch` bytes apart and the ranks' rows back to
// back, in boxes of box_rows x box_bytes (128 or 64) with the swizzle of that width.
bool encode_3d(CUtensorMap* map, const void* base, CUtensorMapDataType type, uint64_t elem, uint64_t cols, uint64_t rows,
               uint64_t ranks, uint64_t pitch, uint32_t box_rows, uint32_t box_bytes) {
  if (!get_encode()) return false;
  cuuint64_t dims[3] = {cols, rows, ranks};
  cuuint64_t strides[2] = {pitch, pitch * rows};
  cuuint32_t box[3] = {(cuuint32_t)(box_bytes / elem), box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The dynamic shared memory of a kernel is raised to `bytes` once per device.
template <typename Kernel>
hq_status raise_smem(bool& done, Kernel kern, size_t bytes) {
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!done && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return HQ_ERR_CUDA;
  done = true;
  return HQ_OK;
}

constexpr size_t kSmemPerSm = 227 * 1024;

template <int kOut, int kTokens>
hq_status launch_few(const hq::MmArgs& p, DeviceInfo& d, cudaStream_t st) {
  CUtensorMap map_a, map_w;
  if (!encode_3d(&map_a, p.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.T, p.P, p.lda, kTokens, 128) ||
      !encode_3d(&map_w, p.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.H, p.P, p.ldw, hq::kFewFeatures, 128))
    return HQ_ERR_CUDA;
  auto kern = hq::int8_matmul_few_kernel<kOut, kTokens>;
  constexpr int kIdx = kTokens == 16 ? 0 : kTokens == 32 ? 1 : 2;
  if (raise_smem(d.few_smem_set[kOut][kIdx], kern, kSmemPerSm - 1024) != HQ_OK) return HQ_ERR_CUDA;
  // K is shared by a cluster of CTAs until they are one to an SM (4 ranks, 32 tokens, H = 4096, K = 1024 as a
  // wire: 7.3 us with 128 CTAs, 7.7 with 256), or two with at least eight steps each (64 tokens, 8192 x 8192:
  // 15.7 us with 256 CTAs, 15.8 with 128), and as long as each has four steps (one token, H = 4096, K = 512:
  // alone 3.0 us, two to a cluster 3.4, four 3.7) or, with 17 to 32 tokens, two (measured at one shape: H = 2048,
  // K = 1024 4.1 us, with four 4.6).  An SM's CTAs fill its shared memory with their rings together (8 ranks, one token, H = 8192,
  // K = 1024: four to an SM 12.7 us, three 14.7).
  const int kc = (int)ceil_div(p.K, hq::kMmK);
  const long long tiles = ceil_div(p.H, hq::kFewFeatures) * p.P;
  int split = 1, split_log2 = 0;
  auto fits = [&](int s) {
    return kc / s >= (kTokens == 32 ? 2 : 4) && (s * tiles <= d.sms || (s * tiles <= 2 * d.sms && kc / s >= 8));
  };
  while (split < hq::kFewMaxSplit && fits(2 * split)) split *= 2, ++split_log2;
  const size_t red = split > 1 ? hq::few_red_bytes(kTokens) : 0;
  const int per_sm = (int)std::min<long long>(4, std::max<long long>(1, ceil_div(tiles * split, d.sms)));
  const int fit = (int)((kSmemPerSm / per_sm - 2560 - 4 * kTokens - red) / hq::few_stage_bytes(kTokens));
  const int stages = std::max(2, std::min({fit, hq::kFewMaxStages, (int)ceil_div(kc, split)}));
  const size_t smem = 1024 + (size_t)stages * hq::few_stage_bytes(kTokens) + red;
  const dim3 grid((unsigned)(ceil_div(p.H, hq::kFewFeatures) * split), (unsigned)p.P);
  return launch_dependent(kern, grid, hq::kFewThreads, smem, st, split, map_a, map_w, p, split_log2, stages, wait_limits());
}

template <int kOut, int kN>
hq_status launch_pair(const hq::MmArgs& p, DeviceInfo& d, cudaStream_t st) {
  CUtensorMap map_a, map_w, map_out;
  if (!encode_3d(&map_a, p.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.T, p.P, p.lda, hq::kMmHalf, 128) ||
      !encode_3d(&map_w, p.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.H, p.P, p.ldw, kN / 2, 128))
    return HQ_ERR_CUDA;
  memset(&map_out, 0, sizeof map_out);
  if (kOut == hq::kMmBf16 &&
      !encode_3d(&map_out, p.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.H, p.T, p.P, 2ull * p.ldo, 32, 64))
    return HQ_ERR_CUDA;
  if (kOut == hq::kMmF32 &&
      !encode_3d(&map_out, p.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.H, p.T, p.P, 4ull * p.ldo, 32, 64))
    return HQ_ERR_CUDA;
  // a token's words of codes start on 16 bytes (no other output has them)
  const bool wide = kOut != hq::kMmWire || ((p.H - p.k) % 32 == 0 && aligned(p.codes, 16));
  auto kern = wide ? hq::int8_matmul_pair_kernel<kOut, kN, true> : hq::int8_matmul_pair_kernel<kOut, kN, kOut != hq::kMmWire>;
  const size_t smem = sizeof(hq::MmSmem<kN>) + 1024;
  if (raise_smem(d.pair_smem_set[kOut][kN == 256][wide], kern, smem) != HQ_OK) return HQ_ERR_CUDA;
  const long long tiles = (long long)p.P * ceil_div(p.T, hq::kMmTile) * ceil_div(p.H, kN);
  const long long clusters = std::min<long long>(tiles, d.sms / 2);
  return launch_dependent(kern, dim3((unsigned)(2 * clusters)), hq::kMmThreads, smem, st, 2, map_a, map_w, map_out, p,
                          wait_limits());
}

template <int kOut>
hq_status launch_matmul(const hq::MmArgs& p, cudaStream_t st) {
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  // Up to 64 tokens the weights are the M operand: 8 ranks, H = 8192, K = 1024 take 13.7 us at 32 tokens
  // and 15.6 at 64 (the pair kernel: 16.4 and 16.9); 8192 x 8192 with one rank, 40 tokens 15.6 and 21.6.
  // Beyond, the pair kernel's tiles are the faster ones: 65 tokens 17.0 us (23.2 with the weights as M
  // and room for 128 tokens), 128 tokens 17.7 and 26.2; as a wire 21.4 and 41.1.
  if (p.T <= 16) return launch_few<kOut, 16>(p, *d, st);
  if (p.T <= 32) return launch_few<kOut, 32>(p, *d, st);
  if (p.T <= 64) return launch_few<kOut, 64>(p, *d, st);
  // Tiles of 128 features as long as there is one for every pair of SMs at most (one rank, H = 4096, K = 512,
  // 128 tokens: 4.4 us, 5.4 with 256 features; 200 tokens, 4096 x 4096: 12.2 and 14.1), else of 256 (two
  // ranks, 700 tokens, H = 4096, K = 512: 7.5 us, 8.2 with 128; 512 tokens, H = 8192, K = 4096: 15.5 and 21.4).
  if (p.P * ceil_div(p.T, hq::kMmTile) * ceil_div(p.H, 128) <= d->sms / 2) return launch_pair<kOut, 128>(p, *d, st);
  return launch_pair<kOut, 256>(p, *d, st);
}

template <typename Y, typename R>
hq_status launch_norm(const hq::NormArgs& a, DeviceInfo& d, cudaStream_t st) {
  const int nvec = a.H / 8;
  const dim3 rows((unsigned)a.T), fours((unsigned)ceil_div(a.T, 4));
  // Up to 1024 elements a row to a warp, with no more vectors a lane than it takes (65536 x 656 bf16: 62 us with
  // three, 82 with room for four); beyond, a CTA a row (32768 x 2048: 97 us, a warp with eight 121).
  if (nvec <= 32) return launch_dependent(hq::residual_norm_kernel<Y, R, 1, 128, true>, fours, 128, 0, st, 1, a);
  if (nvec <= 64) return launch_dependent(hq::residual_norm_kernel<Y, R, 2, 128, true>, fours, 128, 0, st, 1, a);
  if (nvec <= 96) return launch_dependent(hq::residual_norm_kernel<Y, R, 3, 128, true>, fours, 128, 0, st, 1, a);
  if (nvec <= 128) return launch_dependent(hq::residual_norm_kernel<Y, R, 4, 128, true>, fours, 128, 0, st, 1, a);
  auto threads = [&](int nv) { return (int)(32 * ceil_div(ceil_div(nvec, nv), 32)); };
  // Which kernel, by what was measured (bf16, gate, both weights): the row ring from 4096 < H <= 8192 and
  // eight rows an SM on (8192 x 8192: 99 us, a CTA a row 120; 1500 x 8192: 25.6 and 26.1; 777 x 8192: 16.9
  // and 16.1; 4096 x 4096: 33.4 and 32.0), without biases, which have no registers there (8192 x 8192 with a layer
  // norm's two biases, a CTA a row: 158 us); below two rows an SM one vector a thread (148 x 8192: 5.2 us,
  // two vectors 5.5; 300 x 8192: 11.9 and 9.1).
  if (nvec > hq::kRowsThreads && nvec <= hq::kRowsVec * hq::kRowsThreads && !a.post_b && !a.pre_b && a.T >= 8 * d.sms) {
    const int nt = threads(hq::kRowsVec);
    const bool full = a.H == 8 * hq::kRowsVec * nt;
    auto kern = full ? hq::residual_norm_rows_kernel<Y, R, true> : hq::residual_norm_rows_kernel<Y, R, false>;
    const size_t row = (size_t)a.H * (sizeof(Y) + sizeof(R));
    const int stages = (int)std::min<size_t>(hq::kRowsMaxStages, (kSmemPerSm - 2048) / row);
    if (raise_smem(d.norm_smem_set[sizeof(Y) == 4][sizeof(R) == 4][full], kern, kSmemPerSm - 2048) != HQ_OK)
      return HQ_ERR_CUDA;
    return launch_dependent(kern, dim3((unsigned)d.sms), nt, stages * row, st, 1, a, stages, wait_limits());
  }
  // Above 16384 elements a thread's 64 registers do not hold its four vectors of y, r and v: 160 to 408 bytes of
  // them go through local memory (4096 x 32768: 309 us, 3.5 TB/s; 4096 x 16384, with 512 threads: 144, 3.7).
  if (nvec > 2 * hq::kRowMaxThreads)
    return launch_dependent(hq::residual_norm_kernel<Y, R, 4, 1024, false>, rows, threads(4), 0, st, 1, a);
  if (nvec > hq::kRowMaxThreads)
    return launch_dependent(hq::residual_norm_kernel<Y, R, 4, 512, false>, rows, threads(4), 0, st, 1, a);
  if (a.T >= 2 * d.sms)
    return launch_dependent(hq::residual_norm_kernel<Y, R, 2, 512, false>, rows, threads(2), 0, st, 1, a);
  return launch_dependent(hq::residual_norm_kernel<Y, R, 1, 1024, false>, rows, threads(1), 0, st, 1, a);
}

// Scratch of hq_two_step_reduce_noalloc: a fixed array in every device's global memory, so that a
// caller that may not allocate device memory needs no workspace.  In host code the array's name
// only stands for it; its device address is fetched once per device (device_scratch) and passed to
// the kernels like any workspace pointer.
constexpr size_t kNoAllocScratchBytes = HQ_TWO_STEP_NOALLOC_MAX_BYTES;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

void* g_scratch_ptr[kMaxDevices] = {};
std::mutex g_scratch_mu;

// The current device's address of g_noalloc_scratch, looked up on the first call on that device.
hq_status device_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return HQ_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return HQ_ERR_CUDA;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return HQ_OK;
}

}  // namespace

extern "C" {

hq_status hq_two_step_reduce_noalloc(const uint16_t* x, int P, int T, int H, int k, const int32_t* keep_idx,
                                     const int32_t* rest_idx, const float* scale, const float* inv_scale,
                                     const uint8_t* zero, int k2, const int32_t* keep2, const int32_t* rest2,
                                     const float* scale2, const float* inv_scale2, const uint8_t* zero2, void* out,
                                     hq_out_dtype out_dtype, void* stream) {
  const size_t need = hq_two_step_workspace_bytes(P, T, H, k, k2);
  if (need == 0 || need > kNoAllocScratchBytes) return HQ_ERR_INVALID_ARG;  // rejected before any launch
  void* scratch = nullptr;
  if (device_scratch(&scratch) != HQ_OK) return HQ_ERR_CUDA;
  return two_step_entry(x, P, T, H, k, keep_idx, rest_idx, scale, inv_scale, zero, k2, keep2, rest2, scale2,
                        inv_scale2, zero2, scratch, kNoAllocScratchBytes, out, out_dtype, stream);
}

size_t hq_two_step_workspace_bytes(int P, int T, int H, int k, int k2) {
  if (check_shape(P, H, k) != HQ_OK || check_shape(P, H, k2) != HQ_OK || T < 0) return 0;
  return two_step_layout(P, T, H, k, k2).total;
}

hq_status hq_two_step_reduce(const uint16_t* x, int P, int T, int H, int k, const int32_t* keep_idx,
                             const int32_t* rest_idx, const float* scale, const float* inv_scale, const uint8_t* zero,
                             int k2, const int32_t* keep2, const int32_t* rest2, const float* scale2,
                             const float* inv_scale2, const uint8_t* zero2, void* workspace, size_t workspace_bytes,
                             void* out, hq_out_dtype out_dtype, void* stream) {
  return two_step_entry(x, P, T, H, k, keep_idx, rest_idx, scale, inv_scale, zero, k2, keep2, rest2, scale2,
                        inv_scale2, zero2, workspace, workspace_bytes, out, out_dtype, stream);
}

hq_status hq_calibrate(const uint16_t* x, int P, int T, int H, float beta, int first_batch,
                       float* ema_min, float* ema_max, void* stream) {
  return calibrate_entry(x, H, P, T, H, beta, first_batch, ema_min, ema_max, stream);
}

hq_status hq_calibrate_ld(const uint16_t* x, int ldx, int P, int T, int H, float beta, int first_batch,
                          float* ema_min, float* ema_max, void* stream) {
  return calibrate_entry(x, ldx, P, T, H, beta, first_batch, ema_min, ema_max, stream);
}

hq_status hq_select_topk(const float* ema_min, const float* ema_max, int P, int H, int k,
                         int32_t* keep_idx, int32_t* rest_idx, float* scale, float* inv_scale,
                         uint8_t* zero, void* stream) {
  if (check_shape(P, H, k) != HQ_OK) return HQ_ERR_INVALID_ARG;
  if (!ema_min || !ema_max || !scale || !inv_scale || !zero) return HQ_ERR_INVALID_ARG;
  if ((k > 0 && !keep_idx) || (k < H && !rest_idx)) return HQ_ERR_INVALID_ARG;
  if (!aligned(ema_min, 16) || !aligned(ema_max, 16) || !aligned(scale, 16) ||
      !aligned(inv_scale, 16) || !aligned(zero, 16) || !aligned(keep_idx, 4) || !aligned(rest_idx, 4))
    return HQ_ERR_MISALIGNED;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  const size_t smem = (size_t)H * sizeof(uint32_t);
  {
    std::lock_guard<std::mutex> lock(g_dev_mu);
    if (!d->select_smem_set) {
      if (cudaFuncSetAttribute(hq::select_topk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(hq::kMaxH * sizeof(uint32_t))) != cudaSuccess)
        return HQ_ERR_CUDA;
      d->select_smem_set = true;
    }
  }
  // parameters and keys over the whole GPU, then the selection in one CTA (same stream)
  const unsigned pgrid = (unsigned)ceil_div(H, hq::kSelParamFeatures);
  hq::select_params_kernel<<<pgrid, hq::kSelParamThreads, 0, (cudaStream_t)stream>>>(
      ema_min, ema_max, P, H, k, keep_idx, rest_idx, scale, inv_scale, zero);
  if (cudaGetLastError() != cudaSuccess) return HQ_ERR_CUDA;
  hq::select_topk_kernel<<<1, hq::kSelThreads, smem, (cudaStream_t)stream>>>(H, k, keep_idx, rest_idx);
  return launched();
}

hq_status hq_quantize_pack(const uint16_t* x, int P, int T, int H, int k, const int32_t* keep_idx,
                           const int32_t* rest_idx, const float* inv_scale, const uint8_t* zero,
                           uint32_t* codes, uint16_t* side, void* stream) {
  return quantize_entry(x, H, P, T, H, k, keep_idx, rest_idx, inv_scale, zero, codes, side, stream);
}

hq_status hq_quantize_pack_ld(const uint16_t* x, int ldx, int P, int T, int H, int k, const int32_t* keep_idx,
                              const int32_t* rest_idx, const float* inv_scale, const uint8_t* zero,
                              uint32_t* codes, uint16_t* side, void* stream) {
  return quantize_entry(x, ldx, P, T, H, k, keep_idx, rest_idx, inv_scale, zero, codes, side, stream);
}

hq_status hq_dequant_reduce(const uint32_t* codes, const uint16_t* side, int P, int T, int H, int k,
                            const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                            const uint8_t* zero, void* out, hq_out_dtype out_dtype, void* stream) {
  return dequant_entry<false>(codes, side, P, T, H, k, keep_idx, rest_idx, scale, zero, out, H, out_dtype, stream);
}

hq_status hq_dequant_reduce_ld(const uint32_t* codes, const uint16_t* side, int P, int T, int H, int k,
                               const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                               const uint8_t* zero, void* out, int ldo, hq_out_dtype out_dtype, void* stream) {
  return dequant_entry<false>(codes, side, P, T, H, k, keep_idx, rest_idx, scale, zero, out, ldo, out_dtype,
                              stream);
}

hq_status hq_dequant_reduce_ranks(const uint32_t* const* codes, const uint16_t* const* side, int P, int T, int H,
                                  int k, const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                                  const uint8_t* zero, void* out, hq_out_dtype out_dtype, void* stream) {
  return dequant_ranks_entry(codes, side, P, T, H, k, keep_idx, rest_idx, scale, zero, out, out_dtype, stream);
}

hq_status hq_dequant_reduce_bf16_shards(const uint32_t* codes, const uint16_t* side, int P, int T, int H, int k,
                                        const int32_t* keep_idx, const int32_t* rest_idx, const float* scale,
                                        const uint8_t* zero, void* out, hq_out_dtype out_dtype, void* stream) {
  return dequant_entry<true>(codes, side, P, T, H, k, keep_idx, rest_idx, scale, zero, out, H, out_dtype, stream);
}

hq_status hq_compress_reduce(const uint16_t* x, int P, int T, int H, int k, const int32_t* keep_idx,
                             const int32_t* rest_idx, const float* scale, const float* inv_scale,
                             const uint8_t* zero, void* out, hq_out_dtype out_dtype,
                             uint32_t* codes_or_null, uint16_t* side_or_null, void* stream) {
  return compress_entry(x, H, P, T, H, k, keep_idx, rest_idx, scale, inv_scale, zero, out, H, out_dtype,
                        codes_or_null, side_or_null, stream);
}

hq_status hq_compress_reduce_ld(const uint16_t* x, int ldx, int P, int T, int H, int k, const int32_t* keep_idx,
                                const int32_t* rest_idx, const float* scale, const float* inv_scale,
                                const uint8_t* zero, void* out, int ldo, hq_out_dtype out_dtype,
                                uint32_t* codes_or_null, uint16_t* side_or_null, void* stream) {
  return compress_entry(x, ldx, P, T, H, k, keep_idx, rest_idx, scale, inv_scale, zero, out, ldo, out_dtype,
                        codes_or_null, side_or_null, stream);
}

hq_status hq_quantize_tokens(const uint16_t* x, int ldx, int64_t rows, int K, int8_t* q, int ldq, float* scale,
                             void* stream) {
  return quantize_tokens_entry(x, ldx, rows, K, q, ldq, scale, stream);
}

hq_status hq_int8_matmul(const int8_t* a, int lda, const float* a_scale, const int8_t* w, int ldw,
                         const float* w_scale, const uint16_t* bias_or_null, int P, int T, int H, int K, void* out,
                         int ldo, hq_out_dtype out_dtype, void* stream) {
  const hq_status c = matmul_check(a, lda, a_scale, w, ldw, w_scale, P, T, H, HQ_INT8_MAX_H, K);
  if (c == HQ_ERR_INVALID_ARG || !ld_ok(ldo, H) || (T > 0 && !out)) return HQ_ERR_INVALID_ARG;
  if (out_dtype != HQ_OUT_BF16 && out_dtype != HQ_OUT_F32) return HQ_ERR_INVALID_ARG;
  if (c != HQ_OK || !aligned(bias_or_null, 16) || !aligned(out, 16)) return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  hq::MmArgs p{};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.w = w, p.ldw = ldw, p.w_scale = w_scale;
  p.P = P, p.T = T, p.H = H, p.K = K;
  p.bias = bias_or_null, p.out = out, p.ldo = ldo;
  if (out_dtype == HQ_OUT_BF16) return launch_matmul<hq::kMmBf16>(p, (cudaStream_t)stream);
  return launch_matmul<hq::kMmF32>(p, (cudaStream_t)stream);
}

hq_status hq_int8_matmul_pack(const int8_t* a, int lda, const float* a_scale, const int8_t* w, int ldw,
                              const float* w_scale, int P, int T, int H, int K, int k, const int32_t* keep_idx,
                              const int32_t* rest_idx, const float* inv_scale, const uint8_t* zero, uint32_t* codes,
                              uint16_t* side, void* stream) {
  const hq_status c = matmul_check(a, lda, a_scale, w, ldw, w_scale, P, T, H, hq::kMaxH, K);
  if (c == HQ_ERR_INVALID_ARG || check_shape(P, H, k) != HQ_OK) return HQ_ERR_INVALID_ARG;
  if (!inv_scale || !zero || (k > 0 && !keep_idx) || (k < H && !rest_idx)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && ((k > 0 && !side) || (k < H && !codes))) return HQ_ERR_INVALID_ARG;
  if (c != HQ_OK || !aligned(inv_scale, 16) || !aligned(zero, 16) || !aligned(keep_idx, 4) || !aligned(rest_idx, 4) ||
      !aligned(side, 16) || !aligned(codes, 4))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  hq::MmArgs p{};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.w = w, p.ldw = ldw, p.w_scale = w_scale;
  p.P = P, p.T = T, p.H = H, p.K = K;
  p.k = k, p.keep_idx = keep_idx, p.rest_idx = rest_idx, p.inv_scale = inv_scale, p.zero = zero, p.codes = codes, p.side = side;
  return launch_matmul<hq::kMmWire>(p, (cudaStream_t)stream);
}

hq_status hq_residual_norm(const void* y, hq_out_dtype y_dtype, const void* res, void* res_out,
                           hq_out_dtype res_dtype, int T, int H, hq_norm_kind post, const float* post_w,
                           const float* post_b, const uint16_t* gate, int gate_rows, float alpha, float beta,
                           hq_norm_kind pre, const float* pre_w, const float* pre_b, float eps, uint16_t* h, int8_t* q,
                           int ldq, float* q_scale, void* stream) {
  if (T < 0 || check_shape(1, H, 0) != HQ_OK) return HQ_ERR_INVALID_ARG;
  if ((y_dtype != HQ_OUT_BF16 && y_dtype != HQ_OUT_F32) || (res_dtype != HQ_OUT_BF16 && res_dtype != HQ_OUT_F32))
    return HQ_ERR_INVALID_ARG;
  if (post < HQ_NORM_NONE || post > HQ_NORM_LAYER || pre < HQ_NORM_NONE || pre > HQ_NORM_LAYER) return HQ_ERR_INVALID_ARG;
  if (!std::isfinite(alpha) || !std::isfinite(beta) || !(eps >= 0.0f) || !std::isfinite(eps)) return HQ_ERR_INVALID_ARG;
  if (gate && gate_rows < 1) return HQ_ERR_INVALID_ARG;
  if (!q != !q_scale || (q && (ldq < H || ldq % 16 != 0))) return HQ_ERR_INVALID_ARG;
  if (pre == HQ_NORM_NONE && (h || q)) return HQ_ERR_INVALID_ARG;
  if (T > 0 && (!y || !res || !res_out || (pre != HQ_NORM_NONE && !h && !q))) return HQ_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(res, 16) || !aligned(res_out, 16) || !aligned(post_w, 16) || !aligned(post_b, 16) ||
      !aligned(gate, 16) || !aligned(pre_w, 16) || !aligned(pre_b, 16) || !aligned(h, 16) || !aligned(q, 16) ||
      !aligned(q_scale, 4))
    return HQ_ERR_MISALIGNED;
  if (T == 0) return HQ_OK;
  hq::NormArgs a{y, res, res_out, T, H, (int)post, (int)pre, post_w, post_b, gate, gate ? gate_rows : 1, alpha, beta,
                 pre_w, pre_b, eps, h, q, ldq, q_scale};
  DeviceInfo* d = nullptr;
  if (device_info(&d) != HQ_OK) return HQ_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  if (y_dtype == HQ_OUT_BF16)
    return res_dtype == HQ_OUT_BF16 ? launch_norm<uint16_t, uint16_t>(a, *d, st)
                                    : launch_norm<uint16_t, float>(a, *d, st);
  return res_dtype == HQ_OUT_BF16 ? launch_norm<float, uint16_t>(a, *d, st) : launch_norm<float, float>(a, *d, st);
}

const char* hq_status_string(hq_status s) {
  switch (s) {
    case HQ_OK: return "HQ_OK";
    case HQ_ERR_INVALID_ARG: return "HQ_ERR_INVALID_ARG";
    case HQ_ERR_MISALIGNED: return "HQ_ERR_MISALIGNED";
    case HQ_ERR_CUDA: return "HQ_ERR_CUDA";
    case HQ_ERR_TIMEOUT: return "HQ_ERR_TIMEOUT";
    case HQ_ERR_BAD_INDEX: return "HQ_ERR_BAD_INDEX";
  }
  return "HQ_ERR_UNKNOWN";
}

hq_status hq_read_device_error(void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  std::lock_guard<std::mutex> lock(g_error_mu);
  take_error_kernel<<<1, 1, 0, st>>>();
  if (cudaGetLastError() != cudaSuccess) return HQ_ERR_CUDA;
  unsigned int v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_error_taken, sizeof v, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return HQ_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return HQ_ERR_CUDA;
  return (hq_status)v;
}

hq_status hq_selftest_bounded_wait(long long limit_cycles, void* stream) {
  if (limit_cycles < 0) return HQ_ERR_INVALID_ARG;
  selftest_wait_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(limit_cycles);
  return launched();
}

hq_status hq_selftest_set_pipeline_stall(long long consumer_limit_cycles, long long producer_delay_cycles) {
  if (consumer_limit_cycles < 0 || producer_delay_cycles < 0 || producer_delay_cycles > kMaxStallDelayCycles)
    return HQ_ERR_INVALID_ARG;
  if ((consumer_limit_cycles == 0) != (producer_delay_cycles == 0)) return HQ_ERR_INVALID_ARG;
  g_stall_consumer_limit.store(consumer_limit_cycles);
  g_stall_producer_delay.store(producer_delay_cycles);
  return HQ_OK;
}

int64_t hq_wire_bytes_per_row(int H, int k) {
  if (H < 0 || k < 0 || k > H) return -1;
  return (int64_t)(H - k) / 2 + 2 * (int64_t)k;
}

}  // extern "C"
