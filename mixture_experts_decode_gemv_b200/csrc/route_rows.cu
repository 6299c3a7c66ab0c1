// moe_route_rows: scores, group-limited top-k and weights of any number of rows, and the stable
// grouping of their (row, slot) pairs by expert.
//
// One warp routes a row. The experts of a group lie on consecutive lanes (32 / G lanes per group,
// each with up to NJ consecutive experts of it), so a group's score is a reduction over its own
// lanes, and the lane order is the expert order: the lowest lane among equal keys holds the lowest
// id. A selection round is one warp maximum over the lanes' best keys.
//
// Decisions are those of 64-bit arithmetic. Logits compare exactly as they are. A computed key
// (score + bias) or group score (a sum) carries rounding of a few 2^-24 of the magnitudes that it is
// made of; when two that decide something lie within 2^-20 of those magnitudes, the row is routed
// again with float64 scores (a few rows in a thousand).
//
// Grouping is a stable counting sort: blocks of rows count their pairs per expert into a table,
// and a second launch turns the table into positions (rows that fit one block do both in one
// launch).
#include <cfloat>
#include <cmath>

#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

constexpr int kRThreads = 512;
constexpr int kRWarps = kRThreads / 32;
constexpr int kMaxBlocks = 148;   // blocks of rows, and rows of the count table
constexpr int kMaxE = MOE_ROUTE_MAX_EXPERTS;
// Rows that one block routes and groups in one launch.
constexpr int kOneBlockRows = 64;

struct RouteArgs {
  long long rows, ld;
  long long rows_per_block;
  int E, k, routing, norm, raw, bias, G, keep, top2;
  int lanes, per;      // lanes of a group, experts of a lane
  int f32;
  float rsf;
  const void* logits;
  const float* bias_p;
  int* idx;
  float* weights;
  int* pairs;          // grouping (NULL: none)
  int* offsets;
  int* perm;
  int* table;          // [blocks][E] pairs per block and expert
};

// Order-preserving map of a float key to uint32; every key that can be selected maps above 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename R>
__device__ __forceinline__ R score_of(int routing, R l) {
  if (routing == MOE_ROUTE_SQRTSOFTPLUS) return sqrt(fmax(l, (R)0) + log1p(exp(-fabs(l))));
  return (R)1 / ((R)1 + exp(-l));
}

template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <typename R>
__device__ __forceinline__ R warp_max(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// What a routed row leaves in the warp: lane s < k holds slot s.
struct Slots {
  int id;           // -1: no expert was left
  float l;          // its logit
  float top, den;   // softmax: the row's largest logit, and the sum of exp(l - top)
};

// Routes one row with scores in R. Returns false when a decision hangs on less than R's rounding
// (R = float only).
template <int NJ, typename R>
__device__ __forceinline__ bool route_row(const RouteArgs& a, const float (&lg)[NJ],
                                          const float (&bs)[NJ], Slots& out) {
  constexpr bool kF32 = sizeof(R) == 4;
  constexpr R kNone = -INFINITY;
  const int lane = threadIdx.x & 31;
  const int g = lane / a.lanes, sub = lane - g * a.lanes;
  const int gs = a.E / a.G;
  const bool limited = a.keep < a.G;
  const bool soft = a.routing == MOE_ROUTE_SOFTMAX;
  const bool sums = limited && a.top2;               // group scores are sums of values
  const bool scored = a.bias || (sums && !a.raw);    // scores enter a decision
  bool sure = true;

  R top = 0, den = 1;
  if (soft) {
    float m = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < NJ; ++j) m = fmaxf(m, lg[j]);
    top = warp_max(m);
    if (scored || !a.norm) {
      den = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) den += exp((R)lg[j] - top);   // masked: exp(-inf) = 0
      den = warp_sum(den);
    }
  }
  // keys, in order; the values that group sums are made of
  R key[NJ], val[NJ];
  R mag = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool gone = !(lg[j] > -INFINITY);
    const R l = lg[j];
    R s = 0;
    if (scored && !gone) s = soft ? exp(l - top) / den : score_of<R>(a.routing, l);
    key[j] = gone ? kNone : a.bias ? s + (R)bs[j] : l;
    val[j] = gone ? kNone : (a.bias || a.raw) ? key[j] : s;
    if (!gone) mag = fmax(mag, fabs(s) + fabs((R)bs[j]) + (a.raw ? fabs(l) : (R)0));
  }
  R tol = 0;
  if (kF32 && (a.bias || sums)) tol = warp_max(mag) * (R)(soft ? 0x1p-18 : 0x1p-20);

  if (limited) {
    // score of this lane's group: the two largest of its values (or its largest key)
    R m1 = kNone, m2 = kNone;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const R v = a.top2 ? val[j] : key[j];
      m2 = fmax(m2, fmin(m1, v));
      m1 = fmax(m1, v);
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const R o1 = __shfl_down_sync(kFull, m1, o), o2 = __shfl_down_sync(kFull, m2, o);
      if (sub + o < a.lanes) {
        m2 = fmax(fmin(m1, o1), fmax(m2, o2));
        m1 = fmax(m1, o1);
      }
    }
    R of = a.top2 && m2 > kNone ? m1 + m2 : m1;
    of = __shfl_sync(kFull, of, min(g, a.G - 1) * a.lanes);
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
      const R other = __shfl_sync(kFull, of, o * a.lanes);
      rank += other > of || (other == of && o < g);
    }
    const bool kept = g < a.G && rank < a.keep && of > kNone;
    if (kF32 && (sums || a.bias)) {
      const R low = -warp_max(kept ? -of : kNone);
      const R high = warp_max(g < a.G && rank >= a.keep ? of : kNone);
      if (high > kNone && low - high <= 2 * tol) sure = false;
    }
    if (!kept) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) key[j] = kNone;
    }
  }

  // the lane's best key, lowest expert first
  const int base = g * gs + sub * a.per;
  R best = kNone;
  int at = 0;
  float bl = 0.f, bb = 0.f;
  auto pick = [&]() {
    best = kNone;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
        bl = lg[j];
        bb = bs[j];
      }
  };
  pick();
  out.id = -1;
  out.l = 0.f;
  out.top = (float)top;
  out.den = (float)den;
  R prev = 0;
  float prev_l = 0.f, prev_b = 0.f;
  const int rounds = a.k + (kF32 && a.bias ? 1 : 0);   // the first loser too: its gap counts
  for (int s = 0; s < rounds; ++s) {
    R win;
    if constexpr (kF32) {
      const uint32_t w = __reduce_max_sync(kFull, best > kNone ? ordered(best) : 0u);
      win = w ? unordered(w) : kNone;
    } else {
      win = warp_max(best);
    }
    if (!(win > kNone)) break;                         // no expert is left
    const int owner = __ffs(__ballot_sync(kFull, best == win)) - 1;
    const int id = __shfl_sync(kFull, base + at, owner);
    const float l = __shfl_sync(kFull, bl, owner);
    if (kF32 && a.bias) {
      const float b = __shfl_sync(kFull, bb, owner);
      // equal logits with equal biases tie in any arithmetic
      if (s > 0 && prev - win <= tol && (l != prev_l || b != prev_b)) sure = false;
      prev = win;
      prev_l = l;
      prev_b = b;
    }
    if (lane == s && s < a.k) {
      out.id = id;
      out.l = l;
    }
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (j == at) key[j] = kNone;
      pick();
    }
  }
  return sure;
}

// Logits and biases of this lane's experts; masked ones (and places without an expert) are -inf.
template <int NJ>
__device__ __forceinline__ void load_row(const RouteArgs& a, long long r, float (&lg)[NJ],
                                         float (&bs)[NJ]) {
  const int lane = threadIdx.x & 31;
  const int g = lane / a.lanes, sub = lane - g * a.lanes;
  const int gs = a.E / a.G;
  const size_t row = (size_t)r * (size_t)a.ld;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int in_group = sub * a.per + j;
    const bool real = g < a.G && j < a.per && in_group < gs;
    const int e = g * gs + in_group;
    float l = real ? load_one(a.logits, row + e, a.f32) : -INFINITY;
    const float b = real && a.bias ? a.bias_p[e] : 0.f;
    if (!(l > -INFINITY) || !(b > -INFINITY)) l = -INFINITY;   // NaN compares false
    lg[j] = fminf(l, FLT_MAX);
    bs[j] = b;
  }
}

// The same row with float64 scores, out of line: it is rare, and its registers stay out of the
// ordinary path.
template <int NJ>
__device__ __noinline__ void route_row_f64(const RouteArgs& a, long long r, Slots& out) {
  float lg[NJ], bs[NJ];
  load_row<NJ>(a, r, lg, bs);
  route_row<NJ, double>(a, lg, bs, out);
}

// Weight of this lane's slot. Renormalised scores are taken relative to a common factor, so that
// scores that underflow float32 (logits far below zero) keep their ratios.
__device__ __forceinline__ float weight_of(const RouteArgs& a, const Slots& s) {
  const bool live = s.id >= 0;
  const float most = warp_max(live ? s.l : -FLT_MAX);   // the largest selected logit
  float w;
  if (a.routing == MOE_ROUTE_SOFTMAX) {
    w = a.norm ? expf(s.l - most) : expf(s.l - s.top) / s.den;
  } else if (!a.norm) {
    w = score_of<float>(a.routing, s.l);
  } else if (a.routing == MOE_ROUTE_SIGMOID) {
    // e^l / (1 + e^l), over e^most when every logit is negative
    w = s.l <= 0.f ? expf(s.l - fminf(most, 0.f)) / (1.0f + expf(s.l))
                   : 1.0f / (1.0f + expf(-s.l));
  } else {
    // far below zero softplus(l) = e^l (its next term is under 2^-24 of it)
    w = most < -17.0f ? expf(0.5f * (s.l - most)) : score_of<float>(a.routing, s.l);
  }
  if (!live) w = 0.f;
  if (a.norm) {
    const float total = warp_sum(w);
    w = total > 0.f ? w / total : 0.f;
  }
  return w * a.rsf;
}

// Routes the block's rows; counts its pairs per expert in s_count when grouping.
template <int NJ>
__device__ __forceinline__ void route_block(const RouteArgs& a, long long first, long long last,
                                            int* s_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long r = first + warp; r < last; r += kRWarps) {
    float lg[NJ], bs[NJ];
    load_row<NJ>(a, r, lg, bs);
    Slots s;
    if (!route_row<NJ, float>(a, lg, bs, s)) route_row_f64<NJ>(a, r, s);
    const float w = weight_of(a, s);
    if (lane < a.k) {
      const size_t p = (size_t)r * a.k + lane;
      a.idx[p] = s.id;
      a.weights[p] = w;
      if (a.pairs && s.id >= 0) atomicAdd(s_count + s.id, 1);
    }
  }
}

struct GroupShared {
  int start[kMaxE];            // first position of this block's pairs of each expert
  int warp_count[kRWarps][kMaxE];
  int scan[kRWarps];
  int total;
};

// Positions of the block's pairs. `table` holds every block's counts.
__device__ __forceinline__ void group_block(const RouteArgs& a, long long first, long long last,
                                            int block, int blocks, const int* table,
                                            GroupShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = a.E;
  // expert tid: pairs of the blocks before this one, and of all blocks
  int before = 0, all = 0;
  if (tid < E) {
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) {
      const int c = table[(size_t)b * E + tid];
      all += c;
      before += b < block ? c : 0;
    }
  }
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh.scan[warp] = inc;
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < kRWarps; ++w) {
    if (w < warp) base += sh.scan[w];
    total += sh.scan[w];
  }
  const int begin = base + inc - all;
  if (tid < E) {
    sh.start[tid] = begin + before;
    if (block == 0) {
      a.offsets[tid] = begin;
      if (tid == E - 1) a.offsets[E] = begin + all;
    }
  }
  // each warp takes a contiguous run of the block's pairs: count, scan over the warps, place
  const long long p0 = first * a.k, p1 = last * a.k;
  const long long run = ((p1 - p0 + kRWarps - 1) / kRWarps + 31) / 32 * 32;
  const long long w0 = p0 + warp * run, w1 = min(p1, w0 + run);
  int* count = sh.warp_count[warp];
  for (int e = lane; e < E; e += 32) count[e] = 0;
  __syncwarp();
  for (long long p = w0 + lane; p - lane < w1; p += 32) {
    const int e = p < w1 ? a.idx[p] : -1;
    if (e >= 0) atomicAdd(count + e, 1);
  }
  __syncthreads();
  if (tid < E) {
    int at = sh.start[tid];
    for (int w = 0; w < kRWarps; ++w) {
      const int c = sh.warp_count[w][tid];
      sh.warp_count[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
  for (long long p = w0 + lane; p - lane < w1; p += 32) {
    const int e = p < w1 ? a.idx[p] : -1;
    const unsigned same = __match_any_sync(kFull, e);
    int pos = -1;
    if (e >= 0) {
      pos = count[e] + __popc(same & ((1u << lane) - 1u));
      a.pairs[pos] = (int)p;
    }
    __syncwarp();
    if (e >= 0 && lane == 31 - __clz(same)) count[e] += __popc(same);
    __syncwarp();
    if (p < w1) a.perm[p] = pos;
  }
  // entries behind the last pair that has an expert
  for (long long p = p0 + tid; p < p1; p += kRThreads)
    if (p >= total) a.pairs[p] = -1;
}

template <int NJ>
__global__ void __launch_bounds__(kRThreads) route_rows_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ int s_count[kMaxE];
  release_next();
  const long long first = blockIdx.x * a.rows_per_block;
  const long long last = min(a.rows, first + a.rows_per_block);
  if (a.pairs) {
    for (int e = threadIdx.x; e < a.E; e += kRThreads) s_count[e] = 0;
    __syncthreads();
  }
  route_block<NJ>(a, first, last, s_count);
  if (a.pairs) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRThreads)
      a.table[(size_t)blockIdx.x * a.E + e] = s_count[e];
  }
}

__global__ void __launch_bounds__(kRThreads) group_pairs_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ GroupShared sh;
  wait_previous();
  const long long first = blockIdx.x * a.rows_per_block;
  const long long last = min(a.rows, first + a.rows_per_block);
  group_block(a, first, last, blockIdx.x, gridDim.x, a.table, sh);
}

template <int NJ>
__global__ void __launch_bounds__(kRThreads) route_group_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ GroupShared sh;
  __shared__ int s_count[kMaxE];
  for (int e = threadIdx.x; e < a.E; e += kRThreads) s_count[e] = 0;
  __syncthreads();
  route_block<NJ>(a, 0, a.rows, s_count);
  __syncthreads();   // also orders the block's idx writes before its reads of them
  group_block(a, 0, a.rows, 0, 1, s_count, sh);
}

template <int NJ>
cudaError_t launch_route(const RouteArgs& a, int blocks, cudaStream_t st) {
  if (a.pairs && blocks == 1) {
    route_group_kernel<NJ><<<1, kRThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  route_rows_kernel<NJ><<<blocks, kRThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.pairs) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kRThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, group_pairs_kernel, a);
}

int check_cfg(const moe_route_cfg* c, int64_t rows) {
  if (!c) return MOE_ERR_NULL_POINTER;
  if (c->num_experts < 1 || c->num_experts > MOE_ROUTE_MAX_EXPERTS) return MOE_ERR_BAD_SHAPE;
  if (c->num_groups < 1 || c->num_groups > MOE_ROUTE_MAX_GROUPS || c->num_experts % c->num_groups)
    return MOE_ERR_BAD_SHAPE;
  if (c->topk_groups < 1 || c->topk_groups > c->num_groups) return MOE_ERR_BAD_SHAPE;
  const int size = c->num_experts / c->num_groups;
  if (c->top_k < 1 || c->top_k > MOE_ROUTE_MAX_TOP_K || c->top_k > c->topk_groups * size)
    return MOE_ERR_BAD_SHAPE;
  if (c->routing < MOE_ROUTE_SOFTMAX || c->routing > MOE_ROUTE_SQRTSOFTPLUS) return MOE_ERR_BAD_OPTION;
  auto is01 = [](int v) { return v == 0 || v == 1; };
  if (!is01(c->norm_topk_prob) || !is01(c->select_on_raw_logits) || !is01(c->has_expert_bias))
    return MOE_ERR_BAD_OPTION;
  if (c->routing == MOE_ROUTE_SOFTMAX && (c->select_on_raw_logits || c->has_expert_bias))
    return MOE_ERR_BAD_OPTION;
  if (c->select_on_raw_logits && c->has_expert_bias) return MOE_ERR_BAD_OPTION;
  if (c->group_score != MOE_GROUP_MAX && c->group_score != MOE_GROUP_TOP2) return MOE_ERR_BAD_OPTION;
  if (!std::isfinite(c->routed_scaling_factor)) return MOE_ERR_BAD_OPTION;
  if (!moe_host::float_format(c->logits_dtype)) return MOE_ERR_BAD_FORMAT;
  if (rows < 0 || rows > 0x7fffffffLL || rows * c->top_k > 0x7fffffffLL) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

long long blocks_of(int64_t rows) {
  if (rows <= kOneBlockRows) return 1;
  const long long b = (rows + kRWarps - 1) / kRWarps;
  return b < kMaxBlocks ? b : kMaxBlocks;
}

size_t workspace_of(const moe_route_cfg& c, int64_t rows) {
  const size_t table = (size_t)blocks_of(rows) * c.num_experts * sizeof(int);
  return (table + 255) / 256 * 256;
}

}  // namespace

extern "C" int moe_route_workspace_bytes(const moe_route_cfg* cfg, int64_t rows, size_t* out_bytes) {
  if (!out_bytes) return MOE_ERR_NULL_POINTER;
  const int rc = check_cfg(cfg, rows);
  if (rc) return rc;
  *out_bytes = workspace_of(*cfg, rows);
  return MOE_OK;
}

extern "C" int moe_route_rows(const moe_route_cfg* cfg, int64_t rows, const void* logits,
                              int64_t ld_logits, const float* expert_bias, int32_t* idx, float* weights,
                              int32_t* sorted_pairs, int32_t* expert_offsets, int32_t* token_to_perm,
                              void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe_host;
  int rc = check_cfg(cfg, rows);
  if (rc) return rc;
  const moe_route_cfg& c = *cfg;
  const bool group = sorted_pairs || expert_offsets || token_to_perm;
  if (ld_logits < c.num_experts) return MOE_ERR_BAD_SHAPE;
  if (c.has_expert_bias ? !expert_bias : expert_bias != nullptr)
    return c.has_expert_bias ? MOE_ERR_NULL_POINTER : MOE_ERR_BAD_OPTION;
  if (rows > 0 && (!logits || !idx || !weights)) return MOE_ERR_NULL_POINTER;
  if (group && (!expert_offsets || (rows > 0 && (!sorted_pairs || !token_to_perm))))
    return MOE_ERR_NULL_POINTER;
  if (!aligned_to(logits, float_bytes(c.logits_dtype)) || !aligned_to(expert_bias, 4) ||
      !aligned_to(idx, 4) || !aligned_to(weights, 4) || !aligned_to(sorted_pairs, 4) ||
      !aligned_to(expert_offsets, 4) || !aligned_to(token_to_perm, 4))
    return MOE_ERR_MISALIGNED;
  if (group && rows > 0) {
    if (!workspace) return MOE_ERR_NULL_POINTER;
    if (!aligned_to(workspace, 256)) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < workspace_of(c, rows)) return MOE_ERR_WORKSPACE;
  }
  if (rows == 0 && !group) return MOE_OK;
  if ((rc = supported_device())) return rc;
  Range range("moe_route_rows");
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {
    const cudaError_t e = cudaMemsetAsync(expert_offsets, 0, (size_t)(c.num_experts + 1) * 4, st);
    return e == cudaSuccess ? MOE_OK : fail(e);
  }
  const int blocks = (int)blocks_of(rows);
  RouteArgs a;
  a.rows = rows;
  a.ld = ld_logits;
  a.rows_per_block = (rows + blocks - 1) / blocks;
  a.E = c.num_experts; a.k = c.top_k; a.routing = c.routing; a.norm = c.norm_topk_prob;
  a.raw = c.select_on_raw_logits; a.bias = c.has_expert_bias; a.G = c.num_groups;
  a.keep = c.topk_groups; a.top2 = c.group_score == MOE_GROUP_TOP2;
  const int size = a.E / a.G;
  a.lanes = 32 / a.G;
  a.per = (size + a.lanes - 1) / a.lanes;
  a.f32 = c.logits_dtype == MOE_FMT_F32;
  a.rsf = c.routed_scaling_factor;
  a.logits = logits; a.bias_p = expert_bias; a.idx = idx; a.weights = weights;
  a.pairs = group ? sorted_pairs : nullptr;
  a.offsets = expert_offsets; a.perm = token_to_perm; a.table = (int*)workspace;
  const cudaError_t e = a.per <= 1   ? launch_route<1>(a, blocks, st)
                        : a.per <= 2 ? launch_route<2>(a, blocks, st)
                        : a.per <= 4 ? launch_route<4>(a, blocks, st)
                        : a.per <= 8 ? launch_route<8>(a, blocks, st)
                        : a.per <= 16 ? launch_route<16>(a, blocks, st)
                                      : launch_route<32>(a, blocks, st);
  return e == cudaSuccess ? MOE_OK : fail(e);
}
