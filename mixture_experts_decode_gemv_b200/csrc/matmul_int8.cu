// moe_matmul_int8: rows of int8 codes times int8 matrices of the experts, scaled per row and per
// channel, with the gated activation of two products where a second matrix is given.
//
//   y[i, j] = x_scales[r(i)] * scales[e(i), j] * sum_k x[r(i), k] * w[e(i), j, k]
//
// The sums are int32 and exact (|x|, |w| <= 128 and k <= 131056 keep them below 2^31), so neither
// tiling nor order can change a bit of them; what follows is float32 and one rounding to the output
// type.
#include <mutex>

#include <cuda.h>

#include "common.cuh"
#include "host.h"
#include "rows.cuh"
#include "tc05.cuh"

namespace {

using namespace moe_rows;

struct MatmulArgs {
  long long x_rows, ld_x, rows, ld_out, w_stride, up_stride, ws_stride, ups_stride;
  int n, k, experts, top_k, act;
  bool out_f32;
  const int8_t* x;
  const float* x_scales;
  const int* offsets;
  const int* pairs;
  const float* pair_weights;
  const int8_t* w;
  const int8_t* up;
  const float* ws;
  const float* ups;
  void* out;
  int* status;
};

// ---- tiles ---------------------------------------------------------------------------------------
//
// The weights are the M operand (128 channels to a block) and the rows the N operand, so a short
// group of rows costs only as many columns as it has. With a second matrix the 128 rows of a block's
// M tile are 16 gate channels, the same 16 up channels, the next 16 gate channels, and so on: gate
// and up of a channel meet in one warp of the epilogue, 16 lanes apart.

constexpr int kStep = 128;                    // bytes of k per stage: one swizzle atom wide
constexpr long long kWaitLimit = 2000000000LL;  // about a second of SM clock cycles

// Rows [begin, end) of expert e, within the output whatever the offsets hold.
__device__ __forceinline__ void expert_range(const MatmulArgs& a, int e, long long& begin,
                                             long long& end) {
  if (!a.offsets) {
    begin = 0;
    end = a.rows;
    return;
  }
  begin = max(0, a.offsets[e]);
  end = min((long long)a.offsets[e + 1], a.rows);
  if (end < begin) end = begin;
}

// Row of x and factor of output row i; false when its pair lies outside x.
__device__ __forceinline__ bool source_row(const MatmulArgs& a, long long i, int& row, float& scale) {
  if (!a.pairs) {
    row = (int)i;
    scale = a.x_scales[i];
    return true;
  }
  const int p = a.pairs[i];
  row = p / a.top_k;
  if (p < 0 || row >= a.x_rows) return false;
  scale = a.x_scales[row];
  if (a.pair_weights) scale *= a.pair_weights[p];
  return true;
}

__device__ __forceinline__ void store_one(float* p, float y) { *p = y; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float y) { *p = __float2bfloat16_rn(y); }

// The gated activation with one fast exponential and one fast quotient: 2 + 1.2 |g| units of 2^-23
// from the exponent's argument, and 2 from the quotient.
__device__ __forceinline__ float gated(int act, float g, float u) {
  if (act == MOE_ACT_GEGLU) return moe::gelu_tanh_mul(g, u);
  return __fdividef(g * u, 1.0f + __expf(-g));
}

// ---- many rows: pairs of blocks ------------------------------------------------------------------

constexpr int kPairEpilogue = 256;  // threads that write out: two warps for each 32 channels
constexpr int kPairThreads = 64 + kPairEpilogue;   // warp 0 loads, warp 1 issues MMAs
constexpr int kPairStages = 6;
constexpr int kPairN = 256;         // rows of a tile at most
constexpr int kPairA = 128 * kStep, kPairB = (kPairN / 2) * kStep, kPairStage = kPairA + kPairB;

struct PairShared {
  uint64_t full[kPairStages], empty[kPairStages], done[2], free[2];
  uint32_t tmem;
  int abort;
  int tiles[MOE_ROUTE_MAX_EXPERTS + 1];   // row tiles before each expert
  int2 span[MOE_ROUTE_MAX_EXPERTS];       // its first row and its rows
  float2 cols[2][kPairN];                 // factor of a row, and whether it is written
};
constexpr size_t kPairSmem = 1024 + (size_t)kPairStages * kPairStage + sizeof(PairShared);

// Whether any thread of the epilogue says so (a barrier for them).
__device__ __forceinline__ bool any_writer(bool v) {
  int r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.s32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 1, %2, p;\n"
      "selp.s32 %0, 1, 0, q; }"
      : "=r"(r) : "r"((int)v), "n"(kPairEpilogue) : "memory");
  return r;
}

// Walks a cluster's tiles in order. The tiles of an expert go in bands of kBand row tiles: within a
// band the row tiles of one channel tile come one after another, so that the clusters at work share
// kBand row tiles and a few channel tiles, which L2 holds.
constexpr int kBand = 8;
struct TileWalk {
  int t, e = 0;
  __device__ __forceinline__ explicit TileWalk(int first) : t(first) {}
  // First row, rows and channel tile of tile t, and its expert in e; false behind the last.
  __device__ __forceinline__ bool get(const MatmulArgs& a, const PairShared& sh, int ch_tiles, int& i0,
                                      int& live, int& ch) {
    if (t >= sh.tiles[a.experts] * ch_tiles) return false;
    while (sh.tiles[e + 1] * ch_tiles <= t) ++e;
    const int n = sh.tiles[e + 1] - sh.tiles[e];
    int r = t - sh.tiles[e] * ch_tiles;
    const int band = r / (kBand * ch_tiles);
    r -= band * kBand * ch_tiles;
    const int wide = min(kBand, n - band * kBand);
    ch = r / wide;
    const int j = band * kBand + r - ch * wide;
    // the expert's rows in n nearly equal parts, whole multiples of 32
    const int2 span = sh.span[e];
    const int part = ((span.y - 1) / n + 32) & ~31;
    i0 = span.x + j * part;
    live = min(part, span.y - j * part);
    return true;
  }
};

// One warp's share of a finished tile: its 32 lanes' channels of every second chunk of 32 rows. `out`
// points at the thread's channel of the tile's first row, `d` at the warp's lanes in tensor memory.
template <bool ACT, typename T>
__device__ __forceinline__ void write_tile(const MatmulArgs& a, T* out, uint32_t d, const float2* cols, int live,
                                           int first_chunk, bool in, float wg, float wu) {
  const bool upper = threadIdx.x & 16;
  const long long ld = a.ld_out;
  for (int c0 = 32 * first_chunk; c0 < live; c0 += 64) {
    int v[32];
    __syncwarp();
    tmem_load32(d + c0, v);
    tmem_load_wait();
    T* p = out + c0 * ld;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float4 f = *(const float4*)(cols + c0 + j);
      if constexpr (ACT) {
        // the lower half of the warp holds gate and takes row j, the upper holds up and takes row j + 1
        const int got = __shfl_xor_sync(kFull, upper ? v[j] : v[j + 1], 16);
        const float s = upper ? f.z : f.x;
        const float g = (float)(upper ? got : v[j]) * s * wg;
        const float u = (float)(upper ? v[j + 1] : got) * s * wu;
        const float y = gated(a.act, g, u);
        if (in && (upper ? f.w : f.y) != 0.f) store_one(p + (upper ? ld : 0), y);
      } else {
        if (in && f.y != 0.f) store_one(p, (float)v[j] * f.x * wg);
        if (in && f.w != 0.f) store_one(p + ld, (float)v[j + 1] * f.z * wg);
      }
      p += 2 * ld;
    }
  }
}

// Two blocks share a tile of 256 channels (128 with gate and up) x up to 256 rows: each loads half of
// both operands and holds the accumulators of its channels (int32, 256 columns of tensor memory, two
// buffers, so that one tile is written out while the next is multiplied).
template <bool ACT>
__global__ void __launch_bounds__(kPairThreads, 1)
matmul_pair_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_up) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  PairShared& sh = *(PairShared*)(base + kPairStages * kPairStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  constexpr int kChPair = ACT ? 128 : 256, kChBlock = kChPair / 2;
  const int ch_tiles = (a.n + kChPair - 1) / kChPair;
  const int k_steps = (a.k + kStep - 1) / kStep;

  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      bar_init(smem_addr(&sh.full[s]), 1);
      bar_init(smem_addr(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&sh.done[b]), 1);
      bar_init(smem_addr(&sh.free[b]), 2 * kPairEpilogue / 32);   // the epilogue warps of both blocks
    }
    bar_init_fence();
    sh.abort = 0;
  }
  for (int e = tid; e < a.experts; e += kPairThreads) {
    long long begin, end;
    expert_range(a, e, begin, end);
    sh.tiles[e + 1] = (int)((end - begin + kPairN - 1) / kPairN);
    sh.span[e] = make_int2((int)begin, (int)(end - begin));
  }
  if (warp == 1) tmem_alloc<2>(smem_addr(&sh.tmem), 512);
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      int v = e0 + lane < a.experts ? sh.tiles[e0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
      }
      if (e0 + lane < a.experts) sh.tiles[e0 + lane + 1] = v + carry;
      carry += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0) sh.tiles[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;
  volatile int* abort = &sh.abort;
  bool ok = true;

  if (warp == 0) {
    // ---- loads: this block's 128 rows of weights and its half of the rows of x
    uint32_t s = 0, parity = 1;
    TileWalk walk(first);
    int i0, live, ch;
    for (; ok && walk.get(a, sh, ch_tiles, i0, live, ch); walk.t += stride) {
      const int half = (live + 31) / 32 * 16;
      const int r0 = i0 + (int)rank * half;
      int rows[4];
      if (a.pairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = r0 + lane * 4 + j;
          float unused;
          int row = 0;
          rows[j] = i < a.rows && source_row(a, i, row, unused) ? row : 0;
        }
      }
      const uint32_t bytes = 2 * (kPairA + (a.pairs ? half : 128) * kStep);
      const int ch0 = ch * kChPair + (int)rank * kChBlock;
      for (int kb = 0; kb < k_steps; ++kb) {
        ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, kWaitLimit);
        if (!ok) break;
        const uint32_t full = of_rank(smem_addr(&sh.full[s]), 0);
        const uint32_t sa = smem_addr(base + s * kPairStage), sb = sa + kPairA;
        const int x = kb * kStep;
        if (rank == 0 && lane == 0) bar_expect(smem_addr(&sh.full[s]), bytes);
        __syncwarp();
        if constexpr (ACT) {
          if (lane < 8)
            tma_load_3d<true>(sa + lane * 2048, (lane & 1) ? &map_up : &map_w, full, x, ch0 + (lane >> 1) * 16, walk.e);
        } else {
          if (lane == 0) tma_load_3d<true>(sa, &map_w, full, x, ch0, walk.e);
        }
        if (a.pairs) {
          if (lane * 4 < half) tma_gather4<true>(sb + lane * 512, &map_x, full, x, rows);
        } else {
          if (lane == 0) tma_load_2d<true>(sb, &map_x, full, x, r0);
        }
        if (++s == kPairStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // every stage has been read before the block may end
    for (int j = 0; ok && j < kPairStages; ++j) {
      ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, kWaitLimit);
      if (++s == kPairStages) {
        s = 0;
        parity ^= 1;
      }
    }
  } else if (warp == 1) {
    // ---- MMAs, issued by one lane of the first block. The loop stays uniform over the warp and the
    // four MMAs of a step unrolled: with a run-time count under a divergent branch the issue took
    // 190 cycles per MMA, more than the 128 that the MMA itself takes. Past k both operands are zero.
    if (rank == 0) {
      uint32_t s = 0, parity = 0, tile = 0;
      const uint64_t desc0 = operand_desc(smem_addr(base));
      TileWalk walk(first);
      int i0, live, ch;
      for (; ok && walk.get(a, sh, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
        const uint32_t b = tile & 1;
        ok = bar_wait(smem_addr(&sh.free[b]), ((tile >> 1) & 1) ^ 1, abort, kWaitLimit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t desc = i8_desc(256, (live + 31) / 32 * 32);
        const uint32_t d = tmem + b * kPairN;
        for (int kb = 0; kb < k_steps; ++kb) {
          ok = bar_wait(smem_addr(&sh.full[s]), parity, abort, kWaitLimit);
          if (!ok) break;
          tc_fence_after();
          if (elect()) {
            const uint64_t da = desc0 + s * (kPairStage >> 4), db = da + (kPairA >> 4);
            mma_i8<2>(d, da, db, desc, kb > 0);
            mma_i8<2>(d, da + 2, db + 2, desc, true);
            mma_i8<2>(d, da + 4, db + 4, desc, true);
            mma_i8<2>(d, da + 6, db + 6, desc, true);
            mma_commit<2>(smem_addr(&sh.empty[s]));
            if (kb + 1 == k_steps) mma_commit<2>(smem_addr(&sh.done[b]));
          }
          __syncwarp();
          if (++s == kPairStages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
    }
  } else {
    // ---- epilogue: this warp's 32 channels of every second 32 rows
    const int quarter = warp & 3, first_chunk = (warp - 2) >> 2;
    const int et = tid - 64;
    uint32_t tile = 0;
    TileWalk walk(first);
    int i0, live, ch;
    for (; walk.get(a, sh, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
      const uint32_t b = tile & 1;
      float2* cols = sh.cols[b];
      for (int c = et; c < (live + 31) / 32 * 32; c += kPairEpilogue) {
        int row;
        float scale = 0.f;
        const bool real = c < live && source_row(a, i0 + c, row, scale);
        cols[c] = make_float2(scale, real ? 1.f : 0.f);
      }
      const int channel = ACT ? ch * kChPair + (int)rank * kChBlock + quarter * 16 + (lane & 15)
                              : ch * kChPair + (int)rank * kChBlock + quarter * 32 + lane;
      const bool in = channel < a.n;
      const float wg = in ? *(const float*)((const char*)a.ws + (size_t)walk.e * a.ws_stride + (size_t)channel * 4) : 0.f;
      const float wu = ACT && in
          ? *(const float*)((const char*)a.ups + (size_t)walk.e * a.ups_stride + (size_t)channel * 4) : 0.f;
      // the warps leave together: one that gave up still comes to the next tile's barrier
      if (any_writer(!ok)) {
        ok = false;
        break;
      }
      ok = bar_wait(smem_addr(&sh.done[b]), (tile >> 1) & 1, abort, kWaitLimit);
      if (ok) {
        tc_fence_after();
        const uint32_t d = tmem + b * kPairN + ((uint32_t)(quarter * 32) << 16);
        const size_t at = (size_t)i0 * a.ld_out + channel;
        if (a.out_f32) write_tile<ACT>(a, (float*)a.out + at, d, cols, live, first_chunk, in, wg, wu);
        else write_tile<ACT>(a, (__nv_bfloat16*)a.out + at, d, cols, live, first_chunk, in, wg, wu);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_cluster(of_rank(smem_addr(&sh.free[b]), 0));
      }
    }
  }
  if (!ok) {   // a wait ran out: the others are told, and the host finds it in the workspace
    *abort = 1;
    *a.status = MOE_ERR_DEVICE_TIMEOUT;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_free<2>(tmem, 512);
}

// ---- host ----------------------------------------------------------------------------------------

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return fn;
}

// Rows of k bytes, `box` rows of 128 bytes to a load, swizzled by 128 bytes; bytes past k and rows past
// the last read as zero.
bool map_rows(CUtensorMap* m, const void* p, int k, long long rows, long long ld, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t boxes[2] = {kStep, (cuuint32_t)box}, ones[2] = {1, 1};
  return encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void*)p, dims, strides, boxes, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_experts(CUtensorMap* m, const void* p, int k, int n, int experts, long long stride, int box) {
  const cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)n, (cuuint64_t)experts};
  const cuuint64_t strides[2] = {(cuuint64_t)k, (cuuint64_t)(experts > 1 ? stride : (long long)n * k)};
  const cuuint32_t boxes[3] = {kStep, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
  return encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, (void*)p, dims, strides, boxes, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of two of this kernel that the device holds at once (cached per device).
template <bool ACT>
int pair_clusters(cudaError_t* err) {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= 64) return 0;
  if (!cache[dev]) {
    *err = cudaFuncSetAttribute(matmul_pair_kernel<ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (*err != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 74);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    *err = cudaOccupancyMaxActiveClusters(&n, matmul_pair_kernel<ACT>, &cfg);
    if (*err != cudaSuccess) return 0;
    cache[dev] = n > 0 ? n : 1;
  }
  return cache[dev];
}

template <bool ACT>
cudaError_t launch_pair(const MatmulArgs& a, const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& up,
                        cudaStream_t st) {
  cudaError_t e;
  const int clusters = pair_clusters<ACT>(&e);
  if (e != cudaSuccess) return e;
  const int ch = ACT ? 128 : 256;
  // every expert may end in a tile that is not full
  const long long tiles = ((a.rows + kPairN - 1) / kPairN + (a.offsets ? min((long long)a.experts, a.rows) : 0)) *
                          ((a.n + ch - 1) / ch);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;   // more output than any device holds
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(tiles < clusters ? tiles : clusters));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, matmul_pair_kernel<ACT>, a, x, w, up);
}

int check_cfg(const moe_matmul_cfg* c, int64_t rows) {
  if (!c) return MOE_ERR_NULL_POINTER;
  if (c->n < 1 || c->k < 16 || c->k > 131056) return MOE_ERR_BAD_SHAPE;
  if (c->k % 16) return MOE_ERR_BAD_FORMAT;
  if (c->num_experts < 1 || c->num_experts > MOE_ROUTE_MAX_EXPERTS) return MOE_ERR_BAD_SHAPE;
  if (c->top_k < 1 || c->top_k > MOE_ROUTE_MAX_TOP_K) return MOE_ERR_BAD_SHAPE;
  if (c->activation != MOE_ACT_SWIGLU && c->activation != MOE_ACT_GEGLU) return MOE_ERR_BAD_OPTION;
  if (!moe_host::float_format(c->out_dtype)) return MOE_ERR_BAD_FORMAT;
  if (rows < 0 || rows > 0x7fffffffLL) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

int check_weights(const moe_matrix* m, const moe_matmul_cfg& c) {
  using namespace moe_host;
  if (m->format != MOE_FMT_INT8) return MOE_ERR_BAD_FORMAT;
  if (!m->packed || !m->scales) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(m->packed, 16) || !aligned_to(m->scales, 4)) return MOE_ERR_MISALIGNED;
  if (c.num_experts > 1) {
    if (m->expert_stride % 16 || m->scale_stride % 4) return MOE_ERR_MISALIGNED;
    if (m->expert_stride < (int64_t)c.n * c.k || m->scale_stride < (int64_t)c.n * 4)
      return MOE_ERR_BAD_SHAPE;
  }
  return MOE_OK;
}

constexpr size_t kMatmulWorkspace = 256;

}  // namespace

extern "C" int moe_matmul_workspace_bytes(const moe_matmul_cfg* cfg, int64_t rows, size_t* out_bytes) {
  if (!out_bytes) return MOE_ERR_NULL_POINTER;
  const int rc = check_cfg(cfg, rows);
  if (rc) return rc;
  *out_bytes = kMatmulWorkspace;
  return MOE_OK;
}

extern "C" int moe_matmul_int8(const moe_matmul_cfg* cfg, int64_t x_rows, const int8_t* x, int64_t ld_x,
                               const float* x_scales, int64_t rows, const int32_t* expert_offsets,
                               const int32_t* sorted_pairs, const float* pair_weights,
                               const moe_matrix* w, const moe_matrix* up, void* out, int64_t ld_out,
                               void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe_host;
  int rc = check_cfg(cfg, rows);
  if (rc) return rc;
  const moe_matmul_cfg& c = *cfg;
  if (!w) return MOE_ERR_NULL_POINTER;
  if ((rc = check_weights(w, c))) return rc;
  if (up && (rc = check_weights(up, c))) return rc;
  if (!expert_offsets && c.num_experts != 1) return MOE_ERR_NULL_POINTER;
  if (pair_weights && !sorted_pairs) return MOE_ERR_BAD_OPTION;
  if (x_rows < 0 || x_rows > 0x7fffffffLL || (!sorted_pairs && x_rows < rows)) return MOE_ERR_BAD_SHAPE;
  if (ld_x < c.k || ld_out < c.n) return MOE_ERR_BAD_SHAPE;
  if (rows == 0 || x_rows == 0) return MOE_OK;
  if (!x || !x_scales || !out || !workspace) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(x, 16) || ld_x % 16 || !aligned_to(x_scales, 4) || !aligned_to(expert_offsets, 4) ||
      !aligned_to(sorted_pairs, 4) || !aligned_to(pair_weights, 4) ||
      !aligned_to(out, float_bytes(c.out_dtype)) || !aligned_to(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (workspace_bytes < kMatmulWorkspace) return MOE_ERR_WORKSPACE;
  if ((rc = supported_device())) return rc;
  Range range("moe_matmul_int8");
  MatmulArgs a;
  a.x_rows = x_rows; a.ld_x = ld_x; a.rows = rows; a.ld_out = ld_out;
  a.w_stride = c.num_experts > 1 ? w->expert_stride : 0;
  a.ws_stride = c.num_experts > 1 ? w->scale_stride : 0;
  a.up_stride = up && c.num_experts > 1 ? up->expert_stride : 0;
  a.ups_stride = up && c.num_experts > 1 ? up->scale_stride : 0;
  a.n = c.n; a.k = c.k; a.experts = c.num_experts; a.top_k = c.top_k; a.act = c.activation;
  a.out_f32 = c.out_dtype == MOE_FMT_F32;
  a.x = x; a.x_scales = x_scales; a.offsets = expert_offsets; a.pairs = sorted_pairs;
  a.pair_weights = pair_weights;
  a.w = (const int8_t*)w->packed; a.ws = (const float*)w->scales;
  a.up = up ? (const int8_t*)up->packed : nullptr;
  a.ups = up ? (const float*)up->scales : nullptr;
  a.out = out;
  a.status = (int*)workspace;
  if (!encode_tiled()) return fail(cudaErrorNotSupported);
  CUtensorMap mx, mw, mu;
  if (!map_rows(&mx, x, c.k, x_rows, ld_x, sorted_pairs ? 1 : 128) ||
      !map_experts(&mw, a.w, c.k, c.n, c.num_experts, a.w_stride, up ? 16 : 128) ||
      !map_experts(&mu, up ? a.up : a.w, c.k, c.n, c.num_experts, up ? a.up_stride : a.w_stride, up ? 16 : 128))
    return fail(cudaErrorInvalidValue);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = up ? launch_pair<true>(a, mx, mw, mu, st) : launch_pair<false>(a, mx, mw, mu, st);
  return e == cudaSuccess ? MOE_OK : fail(e);
}
