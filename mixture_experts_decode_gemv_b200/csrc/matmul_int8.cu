// moe_matmul_int8: rows of int8 codes times int8 matrices of the experts, scaled per row and per
// channel, with the gated activation of two products where a second matrix is given.
//
//   y[i, j] = x_scales[r(i)] * scales[e(i), j] * sum_k x[r(i), k] * w[e(i), j, k]
//
// The sums are int32 and exact (|x|, |w| <= 128 and k <= 131056 keep them below 2^31), so neither
// tiling nor order can change a bit of them; what follows is float32 and one rounding to the output
// type.
#include <atomic>

#include <cuda.h>

#include "common.cuh"
#include "host.h"
#include "rows.cuh"
#include "tc05.cuh"

namespace {

using namespace moe_rows;

struct MatmulArgs {
  long long x_rows, ld_x, rows, ld_out, w_stride, up_stride, ws_stride, ups_stride;
  int n, k, experts, top_k;
  bool out_f32;
  bool woven;      // one map reads the gate and up rows of a tile, as the tile wants them
  bool up_first;   // ... and finds up below gate in memory
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
  int extra;         // arrivals that no one makes (failure-detection tests)
  long long limit;   // cycles after which a wait gives up
};

// ---- tiles ---------------------------------------------------------------------------------------
//
// The weights are the M operand (128 channels to a block) and the rows the N operand, so a short
// group of rows costs only as many columns as it has. With a second matrix the 128 rows of a block's
// M tile are 16 gate channels, the same 16 up channels, the next 16 gate channels, and so on: gate
// and up of a channel meet in one warp of the epilogue, 16 lanes apart.

constexpr int kStep = 128;                    // bytes of k per stage: one swizzle atom wide
constexpr long long kSettle = 1000000;        // cycles in which copies and MMAs under way end

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

// Stores under a predicate: as branches they would serialise the columns (70 cycles a column).
__device__ __forceinline__ void store_if(bool on, float* p, float y) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p st.global.f32 [%0], %1; }" ::"l"(p), "f"(y), "r"((uint32_t)on));
}
__device__ __forceinline__ void store_if(bool on, __nv_bfloat16* p, float y) {
  const uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p st.global.b16 [%0], %1; }" ::"l"(p), "h"(h), "r"((uint32_t)on));
}

__device__ __forceinline__ void put(float* p, float y) { *p = y; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float y) { *p = __float2bfloat16_rn(y); }

// What a call does with its products. A template argument: a choice at run time in the middle of a chunk
// would keep the rows' exponentials from overlapping.
enum Act { kPlain, kSwiglu, kGeglu };

// The gated activation; SwiGLU with one fast exponential and one fast quotient: 2 + 1.2 |g| units of 2^-23
// from the exponent's argument, and 2 from the quotient.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
  if constexpr (ACT == kGeglu) return moe::gelu_tanh_mul(g, u);
  return __fdividef(g, 1.0f + __expf(-g)) * u;   // not g * u first: that may overflow where the gate is shut
}

// The row tiles of all experts, in expert order.
struct TileList {
  int tiles[MOE_ROUTE_MAX_EXPERTS + 1];   // row tiles before each expert
  int2 span[MOE_ROUTE_MAX_EXPERTS];       // its first row and its rows
};

// Fills the list (the whole block calls it; it ends with a barrier). ROWS: rows of a tile at most.
template <int ROWS>
__device__ __forceinline__ void list_tiles(const MatmulArgs& a, TileList& list) {
  const int lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    long long begin, end;
    expert_range(a, e, begin, end);
    list.tiles[e + 1] = (int)((end - begin + ROWS - 1) / ROWS);
    list.span[e] = make_int2((int)begin, (int)(end - begin));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      int v = e0 + lane < a.experts ? list.tiles[e0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
      }
      if (e0 + lane < a.experts) list.tiles[e0 + lane + 1] = v + carry;
      carry += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0) list.tiles[0] = 0;
  }
  __syncthreads();
}

// Walks a cluster's tiles in order. The tiles of an expert go in bands of kBand row tiles: within a
// band the row tiles of one channel tile come one after another, so that the clusters at work share
// kBand row tiles and a few channel tiles, which L2 holds.
constexpr int kBand = 8;
struct TileWalk {
  int t, e = 0;
  __device__ __forceinline__ explicit TileWalk(int first) : t(first) {}
  // First row, rows and channel tile of tile t, and its expert in e; false behind the last. The rows of
  // an expert are shared out in nearly equal parts, whole multiples of UNIT.
  template <int UNIT>
  __device__ __forceinline__ bool get(const MatmulArgs& a, const TileList& list, int ch_tiles, int& i0,
                                      int& live, int& ch) {
    if (t >= list.tiles[a.experts] * ch_tiles) return false;
    while (e + 1 < a.experts && list.tiles[e + 1] * ch_tiles <= t) ++e;
    const int n = list.tiles[e + 1] - list.tiles[e];
    int r = t - list.tiles[e] * ch_tiles;
    const int band = r / (kBand * ch_tiles);
    r -= band * kBand * ch_tiles;
    const int wide = min(kBand, n - band * kBand);
    ch = r / wide;
    const int j = band * kBand + r - ch * wide;
    const int2 span = list.span[e];
    const int part = ((span.y - 1) / n + UNIT) & ~(UNIT - 1);
    i0 = span.x + j * part;
    live = min(part, span.y - j * part);
    return true;
  }
};

// After a wait that ran out: time for this block's copies and MMAs under way to end, before its shared and
// tensor memory go to someone else.
__device__ __noinline__ void settle() {
  const long long t0 = clock64();
  while (clock64() - t0 < kSettle) {
  }
  __syncwarp();
}

// ---- many rows: pairs of blocks ------------------------------------------------------------------

// Warp 0 loads weights (and rows that lie together), warp 1 issues MMAs, warp 2 fetches the rows' factors,
// warp 3 tells the first block which gathered stages have landed, warps 4 to 7 gather scattered rows, warps
// 8 to 15 write out: two for each 32 channels (sixteen of them are left with 80 registers and spill: 226 us
// against 261 for 8192 rows x 8 of 128 experts, 2 x 768 channels, k = 2048).
constexpr int kGatherWarps = 4, kWriteWarps = 8, kFirstGather = 4, kFirstWriter = kFirstGather + kGatherWarps;
constexpr int kPairThreads = 32 * (kFirstWriter + kWriteWarps);
constexpr int kRowBox = 64;         // rows of x to a load
constexpr int kPairStages = 6;
constexpr int kPairN = 256;         // rows of a tile at most
constexpr int kPairA = 128 * kStep, kPairB = (kPairN / 2) * kStep, kPairStage = kPairA + kPairB;

struct PairShared {
  uint64_t full[kPairStages], empty[kPairStages], landed[kPairStages], done[2], free[2], cols_full[2], cols_free[2];
  uint32_t tmem;
  int abort;
  TileList list;
  alignas(16) float scale[2][kPairN];     // factors of the rows
  uint32_t valid[2][kPairN / 32];         // and which of them are written
};
constexpr size_t kPairSmem = 1024 + (size_t)kPairStages * kPairStage + sizeof(PairShared);

constexpr int kChunk = 16, kChunkStep = kChunk * kWriteWarps / 4;   // rows of a warp's chunk, and to its next

// What a writing thread knows of its tile: its channel, the factors of that channel, and whether its lane holds
// up (its partner gate, 16 lanes away).
struct Writer {
  int channel;
  float wg, wu;
  bool in, up;     // in: the matrix has this channel
};

// The values of a chunk: row j's value of the thread's channel (with gate and up: of rows j, j + 1 the one
// that its half of the warp takes). All factors are fetched before the first value is stored: they could
// not pass the stores.
template <int ACT, typename F>
__device__ __forceinline__ void chunk_values(const MatmulArgs& a, const int (&v)[kChunk], const float* scale,
                                             const Writer& t, F&& take) {
  float s[kChunk];
#pragma unroll
  for (int j = 0; j < kChunk; j += 4) {
    const float4 f = *(const float4*)(scale + j);
    s[j] = f.x;
    s[j + 1] = f.y;
    s[j + 2] = f.z;
    s[j + 3] = f.w;
  }
#pragma unroll
  for (int j = 0; j < kChunk; j += ACT ? 2 : 1) {
    if constexpr (ACT) {
      const int got = __shfl_xor_sync(kFull, t.up ? v[j] : v[j + 1], 16);
      const float f = t.up ? s[j + 1] : s[j];
      const float g = (float)(t.up ? got : v[j]) * f * t.wg;
      const float u = (float)(t.up ? v[j + 1] : got) * f * t.wu;
      take(j, gated<ACT>(g, u));
    } else {
      take(j, (float)v[j] * s[j] * t.wg);
    }
  }
}

// Writes 16 rows of the thread's channel: those whose bit is set in `rows`. `out` points at the channel in the
// chunk's first row. Whole chunks, which most are, go without a predicate to each store. (Laying the chunk out in
// shared memory for 16-byte stores took as long: 139 us against 138 for 65536 rows over 128 experts, 2048
// channels, k = 768; with a predicate everywhere 159.)
template <int ACT, typename T>
__device__ __forceinline__ void write_chunk(const MatmulArgs& a, T* out, const int (&v)[kChunk], const float* scale,
                                            uint32_t rows, const Writer& t) {
  const long long ld = a.ld_out;
  T* p = out + (ACT && t.up ? ld : 0);
  if (__all_sync(kFull, t.in) && (rows & 0xffffu) == 0xffffu) {
    chunk_values<ACT>(a, v, scale, t, [&](int j, float y) { put(p + j * ld, y); });
  } else {
    const uint32_t mine = ACT && t.up ? rows >> 1 : rows;
    chunk_values<ACT>(a, v, scale, t, [&](int j, float y) { store_if(t.in && (mine >> j & 1), p + j * ld, y); });
  }
}

// The warp's chunks of the tile; the next one is on its way from tensor memory while one is written.
template <int ACT, typename T>
__device__ __forceinline__ void write_tile(const MatmulArgs& a, T* out, uint32_t d, const float* scale,
                                           const uint32_t* valid, int live, int c0, const Writer& t) {
  int v[kChunk], w[kChunk];
  if (c0 >= live) return;
  tmem_load16(d + c0, v);
  for (; c0 < live; c0 += 2 * kChunkStep) {
    const int c1 = c0 + kChunkStep, c2 = c1 + kChunkStep;
    tmem_load_wait();
    if (c1 < live) tmem_load16(d + c1, w);
    write_chunk<ACT>(a, out + c0 * a.ld_out, v, scale + c0, valid[c0 / 32] >> (c0 & 16), t);
    __syncwarp();
    if (c1 < live) {
      tmem_load_wait();
      if (c2 < live) tmem_load16(d + c2, v);
      write_chunk<ACT>(a, out + c1 * a.ld_out, w, scale + c1, valid[c1 / 32] >> (c1 & 16), t);
      __syncwarp();
    }
  }
}

// Two blocks share a tile of 256 channels (128 with gate and up) x up to 256 rows: each loads half of
// both operands and holds the accumulators of its channels (int32, 256 columns of tensor memory, two
// buffers, so that one tile is written out while the next is multiplied). Per step of 128 bytes of k a block loads 32 KB
// for 512 cycles of MMA. 4099 rows, 2 x 8192 channels, k = 5120: 253 us, 2.72 POP/s, at the power cap (1320 MHz) with the
// tensor pipe busy 96 % of the cycles; over 128 experts, where tiles are short, it is busy 44 to 55 %.
template <int ACT>
__global__ void __launch_bounds__(kPairThreads, 1)
matmul_pair_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_up) {
  extern __shared__ uint8_t raw[];
  // an offset, not a rounded address: the compiler has to see that everything here is shared memory
  uint8_t* base = raw + (-smem_addr(raw) & 1023);
  PairShared& sh = *(PairShared*)(base + kPairStages * kPairStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  constexpr int kChPair = ACT ? 128 : 256, kChBlock = kChPair / 2;
  const int ch_tiles = (a.n - 1) / kChPair + 1;   // the last one's channels stay below 2^31
  const int k_steps = (a.k + kStep - 1) / kStep;

  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      // the weights' (and rows') bytes, and gathered rows of both blocks
      bar_init(smem_addr(&sh.full[s]), (a.pairs ? 1 + 2 : 1) + a.extra);
      bar_init(smem_addr(&sh.landed[s]), 32 * kGatherWarps);
      bar_init(smem_addr(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&sh.done[b]), 1);
      bar_init(smem_addr(&sh.free[b]), 2 * kWriteWarps);   // the writing warps of both blocks
      bar_init(smem_addr(&sh.cols_full[b]), 1);
      bar_init(smem_addr(&sh.cols_free[b]), kWriteWarps);
    }
    bar_init_fence();
    sh.abort = 0;
  }
  if (warp == 1) tmem_alloc<2>(smem_addr(&sh.tmem), 512);
  if (warp == 0 && elect()) {
    prefetch_map(&map_x);
    prefetch_map(&map_w);
    prefetch_map(&map_up);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  release_next();
  wait_previous();   // all of the above may overlap the kernel before
  list_tiles<kPairN>(a, sh.list);
  const uint32_t tmem = sh.tmem;
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;
  volatile int* abort = &sh.abort;
  bool ok = true;

  if (warp == 0) {
    // ---- loads: this block's 128 rows of weights and its half of the rows of x
    uint32_t s = 0, parity = 1;
    TileWalk walk(first);
    int i0, live, ch;
    for (; ok && walk.get<32>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride) {
      const int half = (live + 31) / 32 * 16;
      const int r0 = i0 + (int)rank * half;
      const int boxes = a.pairs ? 0 : (half + kRowBox - 1) / kRowBox;
      const uint32_t bytes = 2 * (kPairA + boxes * kRowBox * kStep);
      const int ch0 = ch * kChPair + (int)rank * kChBlock;
      for (int kb = 0; kb < k_steps; ++kb) {
        ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
        if (!ok) break;
        const uint32_t full = of_rank(smem_addr(&sh.full[s]), 0);
        const uint32_t sa = smem_addr(base + s * kPairStage), sb = sa + kPairA;
        const int x = kb * kStep;
        if (elect()) {
          if (rank == 0) bar_expect(smem_addr(&sh.full[s]), bytes);
          if constexpr (ACT) {
            if (a.woven) tma_load_5d<true>(sa, &map_w, full, x, 0, 0, ch0 / 16, walk.e);
            else
              for (int q = 0; q < 8; ++q)
                tma_load_3d<true>(sa + q * 2048, (q & 1) ? &map_up : &map_w, full, x, ch0 + (q >> 1) * 16, walk.e);
          } else {
            tma_load_3d<true>(sa, &map_w, full, x, ch0, walk.e);
          }
          for (int q = 0; q < boxes; ++q)
            tma_load_2d<true>(sb + q * kRowBox * kStep, &map_x, full, x, r0 + q * kRowBox);
        }
        __syncwarp();
        if (++s == kPairStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // every stage has been read before the block may end
    for (int j = 0; ok && j < kPairStages; ++j) {
      ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
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
      for (; ok && walk.get<32>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
        const uint32_t b = tile & 1;
        ok = bar_wait(smem_addr(&sh.free[b]), ((tile >> 1) & 1) ^ 1, abort, a.limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t desc = i8_desc(256, (live + 31) / 32 * 32);
        const uint32_t d = tmem + b * kPairN;
        for (int kb = 0; kb < k_steps; ++kb) {
          ok = bar_wait(smem_addr(&sh.full[s]), parity, abort, a.limit);
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
  } else if (warp == 2) {
    // ---- factors of the tile's rows
    uint32_t tile = 0;
    TileWalk walk(first);
    int i0, live, ch;
    for (; ok && walk.get<32>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
      const uint32_t b = tile & 1;
      float f[kPairN / 32];   // fetched before the wait for their place
      uint32_t valid[kPairN / 32];
#pragma unroll
      for (int j = 0; j < kPairN / 32; ++j) {
        const int c = lane + 32 * j;
        int row;
        f[j] = 0.f;
        valid[j] = __ballot_sync(kFull, c < live && source_row(a, i0 + c, row, f[j]));
      }
      ok = bar_wait(smem_addr(&sh.cols_free[b]), ((tile >> 1) & 1) ^ 1, abort, a.limit);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < kPairN / 32; ++j) {
        sh.scale[b][lane + 32 * j] = f[j];
        if (lane == j) sh.valid[b][j] = valid[j];
      }
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sh.cols_full[b]));
    }
  } else if (warp == 3) {
    // ---- a gathered stage has landed: the first block hears of it, after the proxy fence
    if (a.pairs) {
      uint32_t s = 0, parity = 0;
      TileWalk walk(first);
      int i0, live, ch;
      for (; ok && walk.get<32>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride)
        for (int kb = 0; kb < k_steps; ++kb) {
          ok = bar_wait(smem_addr(&sh.landed[s]), parity, abort, a.limit);
          if (!ok) break;
          fence_async_proxy();
          if (elect()) bar_arrive_cluster(of_rank(smem_addr(&sh.full[s]), 0));
          __syncwarp();
          if (++s == kPairStages) {
            s = 0;
            parity ^= 1;
          }
        }
    }
  } else if (warp < kFirstWriter) {
    // ---- scattered rows of x: eight threads to a row, 16 bytes each, into the swizzled tile. The next
    // tile's row numbers are fetched while this one's rows are.
    if (a.pairs) {
      const int gt = tid - 32 * kFirstGather, chunk = gt & 7;
      uint32_t s = 0, parity = 1;
      TileWalk walk(first);
      int i0, live, ch, half = 0, pair[8];
      auto fetch = [&]() {   // pairs of the walk's tile, -1 for rows that it does not have
        const bool more = walk.get<32>(a, sh.list, ch_tiles, i0, live, ch);
        half = more ? (live + 31) / 32 * 16 : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = (gt >> 3) + 16 * j, c = (int)rank * half + r;
          pair[j] = r < half && c < live ? a.pairs[i0 + c] : -1;
        }
      };
      fetch();
      while (ok && half > 0) {
        const int rows = half;
        const int8_t* src[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int row = pair[j] / a.top_k;
          src[j] = a.x + (size_t)(pair[j] >= 0 && row < a.x_rows ? row : 0) * a.ld_x + chunk * 16;
        }
        walk.t += stride;
        fetch();
        for (int kb = 0; kb < k_steps; ++kb) {
          ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
          if (!ok) break;
          const uint32_t sb = smem_addr(base + s * kPairStage) + kPairA;
          const bool in_k = kb * kStep + chunk * 16 < a.k;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = (gt >> 3) + 16 * j;
            if (16 * j < rows)
              copy16(sb + r * kStep + ((chunk ^ (r & 7)) << 4), in_k ? src[j] + kb * kStep : a.x, in_k);
          }
          copies_arrive(smem_addr(&sh.landed[s]));
          if (++s == kPairStages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      copies_wait_all();
    }
  } else {
    // ---- epilogue: this warp's 32 channels of every second 16 rows
    const int quarter = warp & 3, first_row = ((warp - kFirstWriter) >> 2) * kChunk;
    const bool up = ACT && ((lane & 16) != 0) != a.up_first;
    uint32_t tile = 0;
    TileWalk walk(first);
    int i0, live, ch;
    for (; ok && walk.get<32>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
      const uint32_t b = tile & 1;
      Writer t;
      t.channel = ch * kChPair + (int)rank * kChBlock + quarter * (ACT ? 16 : 32) + (ACT ? lane & 15 : lane);
      t.up = up;
      t.in = t.channel < a.n;
      t.wg = t.in ? *(const float*)((const char*)a.ws + (size_t)walk.e * a.ws_stride + (size_t)t.channel * 4) : 0.f;
      t.wu = ACT && t.in
          ? *(const float*)((const char*)a.ups + (size_t)walk.e * a.ups_stride + (size_t)t.channel * 4) : 0.f;
      ok = bar_wait(smem_addr(&sh.cols_full[b]), (tile >> 1) & 1, abort, a.limit) &&
           bar_wait(smem_addr(&sh.done[b]), (tile >> 1) & 1, abort, a.limit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * kPairN + ((uint32_t)(quarter * 32) << 16);
      const size_t at = (size_t)i0 * a.ld_out + t.channel;
      if (a.out_f32) write_tile<ACT>(a, (float*)a.out + at, d, sh.scale[b], sh.valid[b], live, first_row, t);
      else write_tile<ACT>(a, (__nv_bfloat16*)a.out + at, d, sh.scale[b], sh.valid[b], live, first_row, t);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(smem_addr(&sh.cols_free[b]));
        bar_arrive_cluster(of_rank(smem_addr(&sh.free[b]), 0));
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
  if (*abort) settle();
  cluster_sync();
  if (warp == 1) tmem_free<2>(tmem, 512);
}

// ---- few rows: single blocks, k split over a cluster ----------------------------------------------

// With a few rows per expert the product is one pass over the weights, so all that counts is that
// enough of them are under way on every multiprocessor: seven stages of 128 channels x 128 bytes (16 KB).
// Where the tiles are fewer than the blocks, the k steps of a tile are split over the blocks of a cluster,
// which add their int32 sums through each other's shared memory: exact in any order, no workspace, nothing
// to clear. (Two blocks of 16 or 32 rows and five or four stages on a multiprocessor took 46.5 and 49.0 us
// against 45.9 for one of 64 rows and seven, 16 rows x 8 of 128 experts, 2 x 768 channels, k = 2048; 61.4
// and 64.3 against 61.2 with 64 rows.)
// One row, 5120 channels, k = 8192: 11.3 us (42 MB; about 5 us are launch, first loads and exchange); 16 rows x 8 of 128
// experts, 2 x 768 channels, k = 2048: 41.5 us (256 MB, 6.1 TB/s).
constexpr int kFewThreads = 256;    // warp 0 weights, 1 MMAs, 2 and 3 rows of x, 4 to 7 write out
constexpr int kFewMaxCluster = 8;
constexpr int kFewStages = 7;
constexpr int kFewN = 64;           // rows of a tile at most
constexpr int kFewHalf = kFewN / 2;
constexpr int kFewRed = 2 * (kFewHalf + kFewMaxCluster - 1) * 128;   // a block's rows, rounded up, from every block
constexpr int kFewA = 128 * kStep, kFewB = kFewN * kStep, kFewStage = kFewA + kFewB;

struct FewShared {
  uint64_t full[kFewStages], empty[kFewStages], done[2], free[2], red_full, red_free;
  uint32_t tmem;
  int abort;
  TileList list;
  alignas(16) float scale[4][kFewN];                // factors of the rows, a copy for each writing warp
  int red[kFewRed];                                 // sums of this block's rows from every block
};
constexpr size_t kFewSmem = 1024 + (size_t)kFewStages * kFewStage + sizeof(FewShared);

__device__ __forceinline__ void store_remote(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int ACT>
__global__ void __launch_bounds__(kFewThreads, 1)
matmul_few_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_up) {
  extern __shared__ uint8_t raw[];
  // an offset, not a rounded address: the compiler has to see that everything here is shared memory
  uint8_t* base = raw + (-smem_addr(raw) & 1023);
  FewShared& sh = *(FewShared*)(base + kFewStages * kFewStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = (int)cluster_size(), rank = (int)cluster_rank();
  constexpr int kCh = ACT ? 64 : 128;
  const int ch_tiles = (a.n - 1) / kCh + 1;
  const int all_steps = (a.k + kStep - 1) / kStep;
  const int k_first = all_steps * rank / split, k_steps = all_steps * (rank + 1) / split - k_first;

  if (tid == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      bar_init(smem_addr(&sh.full[s]), 1 + 64 + a.extra);     // the weights' bytes, the threads that copy rows
      bar_init(smem_addr(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&sh.done[b]), 1);
      bar_init(smem_addr(&sh.free[b]), 4);
    }
    bar_init(smem_addr(&sh.red_full), 4 * split);
    bar_init(smem_addr(&sh.red_free), 4 * split);
    bar_init_fence();
    sh.abort = 0;
  }
  if (warp == 1) tmem_alloc<1>(smem_addr(&sh.tmem), 2 * kFewN);
  if (warp == 0 && elect()) {
    prefetch_map(&map_w);
    prefetch_map(&map_up);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  release_next();
  wait_previous();   // all of the above may overlap the kernel before
  list_tiles<kFewN>(a, sh.list);
  const uint32_t tmem = sh.tmem;
  const int first = blockIdx.x / split, stride = gridDim.x / split;
  volatile int* abort = &sh.abort;
  bool ok = true;
  TileWalk walk(first);
  int i0, live, ch;

  if (warp == 0) {
    uint32_t s = 0, parity = 1;
    for (; ok && walk.get<16>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride) {
      const int ch0 = ch * kCh;
      for (int kb = 0; kb < k_steps; ++kb) {
        ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
        if (!ok) break;
        const uint32_t full = smem_addr(&sh.full[s]), sa = smem_addr(base + s * kFewStage);
        const int x = (k_first + kb) * kStep;
        if (elect()) {
          bar_expect(full, kFewA);
          if constexpr (ACT) {
            if (a.woven) tma_load_5d<false>(sa, &map_w, full, x, 0, 0, ch0 / 16, walk.e);
            else
              for (int q = 0; q < 8; ++q)
                tma_load_3d<false>(sa + q * 2048, (q & 1) ? &map_up : &map_w, full, x, ch0 + (q >> 1) * 16, walk.e);
          } else {
            tma_load_3d<false>(sa, &map_w, full, x, ch0, walk.e);
          }
        }
        __syncwarp();
        if (++s == kFewStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // every stage has been read before the block may end
    for (int j = 0; ok && j < kFewStages; ++j) {
      ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
      if (++s == kFewStages) {
        s = 0;
        parity ^= 1;
      }
    }
  } else if (warp == 1) {
    uint32_t s = 0, parity = 0, tile = 0;
    const uint64_t desc0 = operand_desc(smem_addr(base));
    for (; ok && walk.get<16>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
      const uint32_t b = tile & 1;
      ok = bar_wait(smem_addr(&sh.free[b]), ((tile >> 1) & 1) ^ 1, abort, a.limit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t desc = i8_desc(128, (live + 15) & ~15);
      const uint32_t d = tmem + b * kFewN;
      for (int kb = 0; kb < k_steps; ++kb) {
        ok = bar_wait(smem_addr(&sh.full[s]), parity, abort, a.limit);
        if (!ok) break;
        fence_async_proxy();
        tc_fence_after();
        if (elect()) {
          const uint64_t da = desc0 + s * (kFewStage >> 4), db = da + (kFewA >> 4);
          mma_i8<1>(d, da, db, desc, kb > 0);
          mma_i8<1>(d, da + 2, db + 2, desc, true);
          mma_i8<1>(d, da + 4, db + 4, desc, true);
          mma_i8<1>(d, da + 6, db + 6, desc, true);
          mma_commit<1>(smem_addr(&sh.empty[s]));
          if (kb + 1 == k_steps) mma_commit<1>(smem_addr(&sh.done[b]));
        }
        __syncwarp();
        if (++s == kFewStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
  } else if (warp < 4) {
    // rows of x: eight threads to a row, 16 bytes each; rows that the tile does not have are left as
    // they are, and so are their columns of the sums, which nothing reads
    const int gt = tid - 64, chunk = gt & 7;
    uint32_t s = 0, parity = 1;
    for (; ok && walk.get<16>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride) {
      const int8_t* src[kFewN / 8];
#pragma unroll
      for (int j = 0; j < kFewN / 8; ++j) {
        const int r = (gt >> 3) + 8 * j;
        int row = 0;
        float unused;
        if (!(r < live && source_row(a, i0 + r, row, unused))) row = 0;
        src[j] = a.x + (size_t)row * a.ld_x + chunk * 16;
      }
      for (int kb = 0; kb < k_steps; ++kb) {
        ok = bar_wait(smem_addr(&sh.empty[s]), parity, abort, a.limit);
        if (!ok) break;
        const uint32_t sb = smem_addr(base + s * kFewStage) + kFewA;
        const int at = (k_first + kb) * kStep;
        const bool in_k = at + chunk * 16 < a.k;
#pragma unroll
        for (int j = 0; j < kFewN / 8; ++j) {
          const int r = (gt >> 3) + 8 * j;
          if (r < live) copy16(sb + r * kStep + ((chunk ^ (r & 7)) << 4), in_k ? src[j] + at : a.x, in_k);
        }
        copies_arrive(smem_addr(&sh.full[s]));
        if (++s == kFewStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    copies_wait_all();
  } else {
    // column c of the sums goes to block c % split, which adds it up and writes its row
    const int quarter = warp & 3, lane_ch = quarter * 32 + lane;
    const bool up = ACT && ((lane & 16) != 0) != a.up_first;
    // The exchange. With up to kFewHalf rows in every tile, the sums of odd and even tiles lie apart, and nothing else keeps a
    // tile's stores behind the reads of the tile that had its place: a block has seen the sums of the tile between
    // them arrive from every warp of the cluster, each of which had read the older one. More rows take the whole of
    // `red`, and say on red_free that they have read it, which costs 0.4 us a tile (one row, 20480 channels, k = 8192:
    // 28.7 us without, 31.8 with).
    bool wide = false;
    for (int e = lane; e < a.experts; e += 32) wide |= sh.list.span[e].y > kFewHalf;
    wide = __any_sync(kFull, wide);
    const int slots = ((wide ? kFewN : kFewHalf) + split - 1) / split, tiles = sh.list.tiles[a.experts] * ch_tiles;
    uint32_t tile = 0;
    for (; ok && walk.get<16>(a, sh.list, ch_tiles, i0, live, ch); walk.t += stride, ++tile) {
      const uint32_t b = tile & 1;
      Writer t;
      t.channel = ch * kCh + quarter * (ACT ? 16 : 32) + (ACT ? lane & 15 : lane);
      t.up = up;
      t.in = t.channel < a.n;
      t.wg = t.in ? *(const float*)((const char*)a.ws + (size_t)walk.e * a.ws_stride + (size_t)t.channel * 4) : 0.f;
      t.wu = ACT && t.in
          ? *(const float*)((const char*)a.ups + (size_t)walk.e * a.ups_stride + (size_t)t.channel * 4) : 0.f;
      // factors of the rows that this block writes: slot q is row rank + q * split
      float* scale = sh.scale[quarter];
      uint32_t valid[kFewN / 32];
#pragma unroll
      for (int j = 0; j < kFewN / 32; ++j) {
        const int q = lane + 32 * j, c = rank + q * split;
        int row;
        float f = 0.f;
        valid[j] = __ballot_sync(kFull, q < slots && c < live && source_row(a, i0 + c, row, f));
        scale[q] = f;
      }
      __syncwarp();
      ok = (split == 1 || !wide || bar_wait(smem_addr(&sh.red_free), (tile & 1) ^ 1, abort, a.limit)) &&
           bar_wait(smem_addr(&sh.done[b]), (tile >> 1) & 1, abort, a.limit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * kFewN + ((uint32_t)(quarter * 32) << 16);
      if (split == 1) {
        for (int c0 = 0; c0 < live; c0 += 16) {
          int v[16];
          tmem_load16(d + c0, v);
          tmem_load_wait();
          const size_t at = (size_t)(i0 + c0) * a.ld_out + t.channel;
          const uint32_t rows = (c0 < 32 ? valid[0] : valid[1]) >> (c0 & 16);
          if (a.out_f32) write_chunk<ACT>(a, (float*)a.out + at, v, scale + c0, rows, t);
          else write_chunk<ACT>(a, (__nv_bfloat16*)a.out + at, v, scale + c0, rows, t);
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.free[b]));
        continue;
      }
      const int place = (wide ? 0 : (int)(tile & 1) * (kFewRed / 2)) + lane_ch;
      const uint32_t mine = smem_addr(sh.red + place + rank * slots * 128);
      uint32_t to = 0, at_slot = mine;
      for (int c0 = 0; c0 < live; c0 += 16) {
        int v[16];
        tmem_load16(d + c0, v);
        tmem_load_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (c0 + j < live) store_remote(of_rank(at_slot, to), v[j]);
          if (++to == (uint32_t)split) {
            to = 0;
            at_slot += 128 * sizeof(int);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sh.free[b]));
      if (lane < split) bar_arrive_release(of_rank(smem_addr(&sh.red_full), lane));
      ok = bar_wait(smem_addr(&sh.red_full), tile & 1, abort, a.limit);
      if (!ok) break;
      // four rows at a time, so that their loads and exponentials overlap
      for (int q = 0, c = rank; c < live; q += 4, c += 4 * split) {
        int sum[4] = {0, 0, 0, 0};
        for (int src = 0; src < split; ++src)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (q + j < slots) sum[j] += sh.red[place + (src * slots + q + j) * 128];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float f = scale[min(q + j, kFewN - 1)];
          float y;
          if constexpr (ACT) {
            const int other = __shfl_xor_sync(kFull, sum[j], 16);
            y = gated<ACT>((float)(up ? other : sum[j]) * f * t.wg, (float)(up ? sum[j] : other) * f * t.wu);
          } else {
            y = (float)sum[j] * f * t.wg;
          }
          const int slot = q + j;
          const bool on = t.in && !up && slot < slots && ((slot < 32 ? valid[0] : valid[1]) >> (slot & 31) & 1);
          const size_t at = (size_t)(i0 + c + j * split) * a.ld_out + t.channel;
          if (a.out_f32) store_if(on, (float*)a.out + at, y);
          else store_if(on, (__nv_bfloat16*)a.out + at, y);
        }
      }
      if (wide && walk.t + stride < tiles) {   // these reads come before the other blocks' next stores
        __syncwarp();
        if (lane < split) bar_arrive_release(of_rank(smem_addr(&sh.red_free), lane));
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
  if (*abort) settle();
  cluster_sync();
  if (warp == 1) tmem_free<1>(tmem, 2 * kFewN);
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

// The rows of two matrices woven as a tile wants them: 16 of gate, 16 of up, the next 16 of gate, ...
// `lower` is the one at the lower address, `apart` the distance to the other.
bool map_woven(CUtensorMap* m, const void* lower, long long apart, int k, int n, int experts, long long stride,
               int blocks) {
  const cuuint64_t dims[5] = {(cuuint64_t)k, 16, 2, (cuuint64_t)n / 16, (cuuint64_t)experts};
  const cuuint64_t strides[4] = {(cuuint64_t)k, (cuuint64_t)apart, (cuuint64_t)k * 16,
                                 (cuuint64_t)(experts > 1 ? stride : (long long)n * k)};
  const cuuint32_t boxes[5] = {kStep, 16, 2, (cuuint32_t)blocks, 1}, ones[5] = {1, 1, 1, 1, 1};
  return encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, (void*)lower, dims, strides, boxes, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `size` blocks of the kernel that device `dev` holds at once (cached per kernel, device, size).
template <auto kernel>
cudaError_t resident_clusters(int dev, int threads, size_t smem, int size, int* out) {
  static std::atomic<int> cache[64][kFewMaxCluster + 1] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = cache[dev][size].load(std::memory_order_acquire);
  if (!n) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) n = 1;
    cache[dev][size].store(n, std::memory_order_release);
  }
  *out = n;
  return cudaSuccess;
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), long long clusters, int size, int threads, size_t smem,
                            cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)clusters * size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tiles of a call at most: an expert with r > 0 rows has at most 1 + (r - 1) / `rows` row tiles.
long long most_tiles(const MatmulArgs& a, int rows, int channels) {
  const long long experts = a.offsets ? (a.experts < a.rows ? a.experts : a.rows) : 1;
  return (experts + (a.rows - experts) / rows) * ((a.n - 1) / channels + 1);
}

// The tensor maps of a call; only those that its kernel reads are made.
struct Maps {
  CUtensorMap x, w, up;
};

template <int ACT>
cudaError_t launch_product(MatmulArgs& a, cudaStream_t st) {
  int dev = 0, pairs = 0, clusters = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = resident_clusters<matmul_pair_kernel<ACT>>(dev, kPairThreads, kPairSmem, 2, &pairs);
  if (e != cudaSuccess) return e;
  Maps m;
  // Gate and up of a tile in one load where the two matrices are laid out alike (one load of 128 rows
  // against eight of 16: 308 against 237 us for 4099 rows, 2 x 8192 channels, k = 5120).
  a.woven = a.up_first = false;
  if (ACT && a.n % 16 == 0 && a.up_stride == a.w_stride && a.up != a.w) {
    const long long apart = a.up > a.w ? a.up - a.w : a.w - a.up;
    a.up_first = a.up < a.w;
    a.woven = apart < (1LL << 40) &&
              map_woven(&m.w, a.up_first ? a.up : a.w, apart, a.k, a.n, a.experts, a.w_stride, 4);
    if (!a.woven) a.up_first = false;
  }
  if (!a.woven && !map_experts(&m.w, a.w, a.k, a.n, a.experts, a.w_stride, ACT ? 16 : 128)) return cudaErrorInvalidValue;
  if (ACT && !a.woven) {
    if (!map_experts(&m.up, a.up, a.k, a.n, a.experts, a.up_stride, 16)) return cudaErrorInvalidValue;
  } else {
    m.up = m.w;
  }

  // Which kernel, and how its k is split. Up to a tile's 64 rows an expert both are a pass over the weights, so
  // the shorter longest block decides: rounds of tiles x the steps of a tile (16 KB of weights a block in both)
  // and what the rest of a tile takes, in steps' time: 2 and one for each eight rows where the k steps of a tile
  // are added up, 6 in pairs. Measured, us, few rows / pairs: 128 experts, 2 x 768 channels, k = 2048, with 1, 4,
  // 8, 16, 32 rows an expert: 46 / 50, 61 / 65, 71 / 75, 77 / 77, 89 / 80. One matrix, 64 rows: 5120 channels,
  // k = 8192: 14.4 / 18.1; 2 x 8192 channels, k = 5120: 19.4 / 18.0. One row, k = 8192, 10240 and 20480 channels: 19.2
  // and 41.5 in single blocks, 17.3 and 28.7 with the splits that this gives.
  const int steps = (a.k + kStep - 1) / kStep;
  const long long per = a.rows / (a.offsets ? a.experts : 1);   // rows of an expert, if they were even
  const long long pair_tiles = most_tiles(a, kPairN, ACT ? 128 : 256), few_tiles = most_tiles(a, kFewN, ACT ? 64 : 128);
  if (pair_tiles > 0x7fffffffLL || few_tiles > 0x7fffffffLL) return cudaErrorInvalidValue;   // more output than any device holds
  if (per <= kFewN) {
    int best = 0, best_clusters = 1;
    long long best_cost = (pair_tiles + pairs - 1) / pairs * (steps + 6);
    for (int size = 1; size <= kFewMaxCluster && size <= steps; ++size) {
      e = resident_clusters<matmul_few_kernel<ACT>>(dev, kFewThreads, kFewSmem, size, &clusters);
      if (e != cudaSuccess) return e;
      const long long cost = (few_tiles + clusters - 1) / clusters * ((steps + size - 1) / size + 2 + per / 8);
      if (cost < best_cost) {
        best = size;
        best_clusters = clusters;
        best_cost = cost;
      }
    }
    if (best)
      return launch_clusters(matmul_few_kernel<ACT>, few_tiles < best_clusters ? few_tiles : best_clusters, best,
                             kFewThreads, kFewSmem, st, a, m.w, m.up);
  }
  if (a.pairs) m.x = m.w;   // gathered rows go without a map
  else if (!map_rows(&m.x, a.x, a.k, a.x_rows, a.ld_x, kRowBox)) return cudaErrorInvalidValue;
  return launch_clusters(matmul_pair_kernel<ACT>, pair_tiles < pairs ? pair_tiles : pairs, 2, kPairThreads, kPairSmem,
                         st, a, m.x, m.w, m.up);
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
  a.n = c.n; a.k = c.k; a.experts = c.num_experts; a.top_k = c.top_k;
  a.out_f32 = c.out_dtype == MOE_FMT_F32;
  a.x = x; a.x_scales = x_scales; a.offsets = expert_offsets; a.pairs = sorted_pairs;
  a.pair_weights = pair_weights;
  a.w = (const int8_t*)w->packed; a.ws = (const float*)w->scales;
  a.up = up ? (const int8_t*)up->packed : nullptr;
  a.ups = up ? (const float*)up->scales : nullptr;
  a.out = out;
  a.status = (int*)workspace;
  test_waits(&a.extra, &a.limit);
  if (!encode_tiled()) return fail(cudaErrorNotSupported);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = !up                               ? launch_product<kPlain>(a, st)
                        : c.activation == MOE_ACT_GEGLU ? launch_product<kGeglu>(a, st)
                                                        : launch_product<kSwiglu>(a, st);
  return e == cudaSuccess ? MOE_OK : fail(e);
}
