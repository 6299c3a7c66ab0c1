// moe_route_rows: scores, group-limited top-k and weights of any number of rows, and the stable
// grouping of their (row, slot) pairs by expert.
//
// One warp routes a row. The experts of a group lie on consecutive lanes (32 / G lanes per group,
// each with up to NJ consecutive experts of it), so a group's score is a reduction over its own
// lanes, and the lane order is the expert order: the lowest lane among equal keys holds the lowest
// id. A selection round is one warp maximum over the lanes' best keys.
//
// Decisions are those of 64-bit arithmetic. Logits compare exactly as they are. A computed key
// (score + bias) or group score (a sum) carries rounding of a few 2^-24 of the largest score and of the
// magnitudes that it is made of; when two that decide something lie closer than such errors may add up to
// (2^-20 of the one, 3 * 2^-24 of the other), the row is settled in float64 (a few rows in a thousand).
//
// Bound by instructions (12.0 M of the warps, 66 % of the issue slots; 3 % of them are spills, as 1024 threads to a block
// leave 64 registers to a thread): 8191 rows of 256 experts, best 4 of 8 groups, top 8 with a bias, take 23 us, 6 of them the
// grouping; the logits alone would take 1.4 from HBM. A row that is settled in float64 costs its warp about 3 us.
//
// Grouping is a stable counting sort: blocks of rows count their pairs per expert into a table,
// and a second launch turns the table into positions (rows that fit one block do both in one
// launch).
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

constexpr int kRThreads = 1024;
constexpr int kRWarps = kRThreads / 32;
constexpr int kMaxBlocks = 148;   // blocks of rows, and rows of the count table
constexpr int kMaxE = MOE_ROUTE_MAX_EXPERTS;
// Rows that one block routes and groups in one launch, and rows of a block beyond that, up to kMaxBlocks blocks
// (256 experts in groups, top 8: 64 rows 20 us in one block, 14.3 in two, 10.7 in eight; 16 rows 10.2 either way).
constexpr int kOneBlockRows = 16, kBlockRows = 8;

struct RouteArgs {
  long long rows, ld;
  long long rows_per_block;
  int E, k, routing, norm, raw, bias, G, keep, top2;
  int lanes, per;      // lanes of a group, experts of a lane
  int f32;
  int vec;             // a lane's experts are whole aligned vectors of the row
  float rsf;
  const void* logits;
  const float* bias_p;
  int* idx;
  float* weights;
  int* pairs;          // grouping (NULL: none)
  int* offsets;
  int* perm;
  int* table;          // [blocks][pitch] pairs per block and expert
  int pitch;           // E, rounded up to a whole int4
};

// Order-preserving map of a float key to uint32; every key that can be selected maps above 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float score_of(int routing, float l) {
  if (routing == MOE_ROUTE_SQRTSOFTPLUS) {
    // far below zero softplus(l) = e^l (its next term is under 2^-24 of it), whose root float32 holds where it no longer
    // holds e^l
    const bool low = l < -17.0f;
    const float e = expf(low ? 0.5f * l : -fabsf(l));
    return low ? e : sqrtf(fmaxf(l, 0.f) + log1pf(e));
  }
  return 1.0f / (1.0f + expf(-l));
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
  float top, den;   // softmax: the row's largest logit, and the sum of exp(l - top)
};

// This lane's place: its group and its first expert in it.
struct Place {
  int g, sub, size, base;
  __device__ __forceinline__ explicit Place(const RouteArgs& a) {
    const int lane = threadIdx.x & 31;
    g = lane / a.lanes;
    sub = lane - g * a.lanes;
    size = a.E / a.G;
    base = g * size + sub * a.per;
  }
  __device__ __forceinline__ bool real(const RouteArgs& a, int j) const {
    return g < a.G && j < a.per && sub * a.per + j < size;
  }
};

__device__ __forceinline__ double score64(int routing, double l) {
  if (routing == MOE_ROUTE_SQRTSOFTPLUS) return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
  return 1.0 / (1.0 + exp(-l));
}

// Puts the experts that lanes 0 .. n-1 hold into the order of their float64 keys (score + bias): the rows
// where float32 has found the experts of the first n places, but not their order.
__device__ __noinline__ void settle_order(const RouteArgs& a, long long r, int n, Slots& s) {
  const int lane = threadIdx.x & 31;
  double key = -INFINITY;
  const int id = s.id;
  if (lane < n && id >= 0) {
    const float l = fminf(load_one(a.logits, (size_t)r * (size_t)a.ld + id, a.f32), FLT_MAX);
    key = score64(a.routing, (double)l) + (double)a.bias_p[id];
  }
  // places beyond n hold no expert and a key below every other: no bound but the largest k + 1, so that all
  // exchanges are under way together
  constexpr int kPlaces = MOE_ROUTE_MAX_TOP_K + 1;
  int rank = 0;
#pragma unroll
  for (int o = 0; o < kPlaces; ++o) {
    const double other = __shfl_sync(kFull, key, o);
    const int other_id = __shfl_sync(kFull, id, o);
    rank += other > key || (other == key && other_id < id);
  }
  if (lane >= n || id < 0) rank = 32;
  // lane `rank` takes this lane's expert
  int got = -1;
#pragma unroll
  for (int o = 0; o < kPlaces; ++o) {
    const int at = __shfl_sync(kFull, rank, o), from = __shfl_sync(kFull, id, o);
    if (lane == at) got = from;
  }
  s.id = got;
}

// The same decisions in float64: for the rows that float32 leaves open.
template <int NJ>
__device__ __noinline__ void route_row_f64(const RouteArgs& a, long long r, Slots& out) {
  constexpr double kNone = -INFINITY;
  const int lane = threadIdx.x & 31;
  const Place at_(a);
  const size_t row = (size_t)r * (size_t)a.ld;
  const bool limited = a.keep < a.G, soft = a.routing == MOE_ROUTE_SOFTMAX;
  double l[NJ], key[NJ], val[NJ];
  double top = -FLT_MAX, den = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool real = at_.real(a, j);
    const float v = real ? load_one(a.logits, row + at_.base + j, a.f32) : -INFINITY;
    const float b = real && a.bias ? a.bias_p[at_.base + j] : 0.f;
    l[j] = v > -INFINITY && b > -INFINITY ? (double)fminf(v, FLT_MAX) : kNone;
    val[j] = b;
    top = fmax(top, l[j]);
  }
  top = warp_max(top);
  if (soft) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) den += exp(l[j] - top);   // masked: exp(-inf) = 0
    den = warp_sum(den);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool gone = !(l[j] > kNone);
    double s = 0;
    if (!gone) {
      if (soft) s = exp(l[j] - top) / den;
      else s = score64(a.routing, l[j]);
    }
    key[j] = gone ? kNone : a.bias ? s + val[j] : l[j];
    val[j] = gone ? kNone : (a.bias || a.raw) ? key[j] : s;
  }
  if (limited) {
    double m1 = kNone, m2 = kNone;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const double v = a.top2 ? val[j] : key[j];
      m2 = fmax(m2, fmin(m1, v));
      m1 = fmax(m1, v);
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const double o1 = __shfl_down_sync(kFull, m1, o), o2 = __shfl_down_sync(kFull, m2, o);
      if (at_.sub + o < a.lanes) {
        m2 = fmax(fmin(m1, o1), fmax(m2, o2));
        m1 = fmax(m1, o1);
      }
    }
    double of = a.top2 && m2 > kNone ? m1 + m2 : m1;
    of = __shfl_sync(kFull, of, min(at_.g, a.G - 1) * a.lanes);
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
      const double other = __shfl_sync(kFull, of, o * a.lanes);
      rank += other > of || (other == of && o < at_.g);
    }
    if (!(at_.g < a.G && rank < a.keep)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) key[j] = kNone;
    }
  }
  out.id = -1;
  for (int s = 0; s < a.k; ++s) {
    double best = kNone;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const double win = warp_max(best);
    if (!(win > kNone)) break;
    const int owner = __ffs(__ballot_sync(kFull, best == win)) - 1;
    const int id = __shfl_sync(kFull, at_.base + at, owner);
    if (lane == s) out.id = id;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (lane == owner && j == at) key[j] = kNone;
  }
}

// Logits of this lane's experts; masked ones (and places without an expert) are -inf.
template <int NJ>
__device__ __forceinline__ void load_row(const RouteArgs& a, const Place& at, long long r,
                                         const float (&bs)[NJ], float (&lg)[NJ]) {
  const size_t row = (size_t)r * (size_t)a.ld;
  bool loaded = false;
  if constexpr (NJ >= 4 && NJ % 4 == 0) {
    if (a.vec) {
      loaded = true;
      if (at.g >= a.G) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) lg[j] = -INFINITY;
      } else if (a.f32) {
        const float4* p = (const float4*)((const float*)a.logits + row + at.base);
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
          const float4 v = p[j / 4];
          lg[j] = v.x;
          lg[j + 1] = v.y;
          lg[j + 2] = v.z;
          lg[j + 3] = v.w;
        }
      } else {
        const uint2* p = (const uint2*)((const __nv_bfloat16*)a.logits + row + at.base);
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
          const uint2 v = p[j / 4];
          lg[j] = bf16_lo(v.x);
          lg[j + 1] = bf16_hi(v.x);
          lg[j + 2] = bf16_lo(v.y);
          lg[j + 3] = bf16_hi(v.y);
        }
      }
    }
  }
  if (!loaded) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) lg[j] = at.real(a, j) ? load_one(a.logits, row + at.base + j, a.f32) : -INFINITY;
  }
  // NaN becomes -infinity (the larger of the two), +infinity the largest finite number, and -0 becomes 0, which
  // it ties with (keys are compared by their bits)
#pragma unroll
  for (int j = 0; j < NJ; ++j) lg[j] = fminf(fmaxf(lg[j], -INFINITY), FLT_MAX) + 0.0f;
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) lg[j] = bs[j] > -INFINITY ? lg[j] : -INFINITY;   // NaN compares false
  }
}

// Key and id in order: descending key, then ascending id. Selects, not branches.
template <int NJ>
__device__ __forceinline__ void order(uint32_t (&key)[NJ], int (&id)[NJ], int x, int y) {
  const uint32_t kx = key[x], ky = key[y];
  const int ix = id[x], iy = id[y];
  const bool swap = ky > kx || (ky == kx && iy < ix);
  key[x] = max(kx, ky);
  key[y] = min(kx, ky);
  id[x] = swap ? iy : ix;
  id[y] = swap ? ix : iy;
}

// Batcher's odd-even merge sort of the lane's experts.
template <int NJ>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[NJ], int (&id)[NJ]) {
#pragma unroll
  for (int p = 1; p < NJ; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < NJ; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < NJ && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order<NJ>(key, id, i + j, i + j + k);
}

enum Verdict { kSure, kOrderOpen, kOpen };

// Routes one row with float32 scores and tells which decisions hang on their rounding: none, the order of
// the experts found (k + 1 of them, one to a lane), or more. A score is off by at most 4 units of 2^-23 of the
// largest (fast exponential and reciprocal; 16 for softmax, whose scores carry the denominator's rounding too), and
// every sum by half a unit of its own: a large bias opens nothing but what it enters. What lies below the lower of two
// keys that are apart is apart from the higher one too: a key and its error grow together.
constexpr float kSumErr = 0x1.8p-23f;   // of the sums in two keys or in a group's score, relative to their magnitudes

// Whether 32 bits leave open that a key of x ranks before one of y.
__device__ __forceinline__ bool near(float x, float y, float score_err) {
  return x - y <= score_err + fmaxf(fabsf(x), fabsf(y)) * kSumErr;
}
__device__ __forceinline__ bool tie(const RouteArgs& a, size_t row, int x, int y) {
  return load_one(a.logits, row + x, a.f32) == load_one(a.logits, row + y, a.f32) && a.bias_p[x] == a.bias_p[y];
}
// Whether an expert of this lane is near `last`, the key of expert `id`, and does not tie with it.
__device__ __noinline__ bool rival(const RouteArgs& a, const Place& at, size_t row, int id, float last,
                                   float score_err) {
  bool found = false;
  for (int j = 0; j < a.per && at.real(a, j); ++j) {
    const int e = at.base + j;
    const float l = fminf(load_one(a.logits, row + e, a.f32), FLT_MAX), b = a.bias_p[e];
    if (l > -INFINITY && b > -INFINITY && near(last, score_of(a.routing, l) + b, score_err))
      found = found || !tie(a, row, e, id);
  }
  return found;
}

template <int NJ>
__device__ __forceinline__ Verdict route_row(const RouteArgs& a, const Place& at, long long r, const float (&lg)[NJ],
                                          const float (&bs)[NJ], Slots& out) {
  const int lane = threadIdx.x & 31;
  const bool limited = a.keep < a.G, soft = a.routing == MOE_ROUTE_SOFTMAX;
  const bool sums = limited && a.top2;               // group scores are sums of values
  const bool scored = a.bias || (sums && !a.raw);    // scores enter a decision
  bool sure = true, ordered_ok = true;

  out.top = 0.f;
  out.den = 1.f;
  float inv = 1.f;
  if (soft && (scored || !a.norm)) {
    float m = -FLT_MAX, den = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) m = fmaxf(m, lg[j]);
    m = unordered(__reduce_max_sync(kFull, ordered(m)));
#pragma unroll
    for (int j = 0; j < NJ; ++j) den += __expf(lg[j] - m);   // masked: exp(-inf) = 0
    out.top = m;
    out.den = warp_sum(den);
    inv = __fdividef(1.0f, out.den);
  }
  float sc[NJ];        // scores, where they decide something
  float mag = scored ? 1.f : 0.f;   // their largest magnitude
  if (scored) {
    if (soft) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) sc[j] = __expf(lg[j] - out.top) * inv;
    } else if (a.routing == MOE_ROUTE_SIGMOID) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) sc[j] = __fdividef(1.0f, 1.0f + __expf(-lg[j]));
    } else {
      mag = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        sc[j] = lg[j] > -INFINITY ? score_of(MOE_ROUTE_SQRTSOFTPLUS, lg[j]) : 0.f;
        mag = fmaxf(mag, sc[j]);
      }
      mag = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(mag)));
    }
  }
  // of two scores; below the normal numbers errors are no longer relative, and float64 decides
  const float score_err = fmaf(mag, soft ? 0x1p-18f : 0x1p-20f, FLT_MIN);
  float kf[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) kf[j] = a.bias && lg[j] > -INFINITY ? sc[j] + bs[j] : lg[j];

  bool kept = at.g < a.G;
  if (limited) {
    // score of this lane's group: the two largest of its values (or its largest key)
    float m1 = -INFINITY, m2 = -INFINITY;
    const bool plain = !a.bias && !a.raw && a.top2;   // values are the scores themselves
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float v = plain && lg[j] > -INFINITY ? sc[j] : kf[j];
      m2 = fmaxf(m2, fminf(m1, v));
      m1 = fmaxf(m1, v);
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const float o1 = __shfl_down_sync(kFull, m1, o), o2 = __shfl_down_sync(kFull, m2, o);
      if (at.sub + o < a.lanes) {
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
    }
    const int head = min(at.g, a.G - 1) * a.lanes;
    m1 = __shfl_sync(kFull, m1, head);
    m2 = __shfl_sync(kFull, m2, head);
    // a group takes part by its best value: the sum of two finite ones may pass the largest number
    const bool some = at.g < a.G && m1 > -INFINITY, two = a.top2 && m2 > -INFINITY;
    const float of = two ? m1 + m2 : m1;
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
      const float other = __shfl_sync(kFull, of, o * a.lanes);
      rank += other > of || (other == of && o < at.g);
    }
    kept = some && rank < a.keep;
    if (sums || a.bias) {
      // float32 does not rank infinite sums
      const bool infinite = !(fabsf(of) <= FLT_MAX);
      const float err = score_err + (fabsf(m1) + (two ? fabsf(m2) : 0.f)) * kSumErr;
      const uint32_t low = __reduce_min_sync(kFull, !kept ? ~0u : infinite ? 0u : ordered(of - err));
      const uint32_t high = __reduce_max_sync(kFull, !some || kept ? 0u : infinite ? ~0u : ordered(of + err));
      if (high >= low) sure = false;
    }
  }
  uint32_t key[NJ];
  int id[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    key[j] = kept && kf[j] > -INFINITY ? ordered(kf[j]) : 0u;
    id[j] = at.base + j;
  }
  sort_lane<NJ>(key, id);

  out.id = -1;
  uint32_t found = 0u;                               // key of this lane's slot
  const int rounds = a.k + (a.bias ? 1 : 0);         // with computed keys the first loser's gap counts too
#pragma unroll 1
  for (int s = 0; s < rounds; ++s) {
    const uint32_t win = __reduce_max_sync(kFull, key[0]);
    if (win == 0u) break;                            // no expert is left
    const int owner = __ffs(__ballot_sync(kFull, key[0] == win)) - 1;
    const int got = __shfl_sync(kFull, id[0], owner);
    if (lane == s) {
      out.id = got;
      found = win;
    }
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j + 1 < NJ; ++j) {
        key[j] = key[j + 1];
        id[j] = id[j + 1];
      }
      key[NJ - 1] = 0u;
    }
  }
  if (a.bias) {
    // gaps between neighbours in the order found
    const uint32_t above = __shfl_up_sync(kFull, found, 1);
    const int above_id = __shfl_up_sync(kFull, out.id, 1);
    const bool close = lane > 0 && found != 0u && near(unordered(above), unordered(found), score_err);
    if (__any_sync(kFull, close)) {
      // equal logits with equal biases tie in any arithmetic
      const size_t row = (size_t)r * (size_t)a.ld;
      if (__any_sync(kFull, close && !tie(a, row, out.id, above_id))) ordered_ok = false;
      // The k best are among the k + 1 found if the last of those is apart from the one before or from all others, or if
      // the order stands and the others near it tie with it. (Its own tie with the one before says nothing of the
      // others: they may share its key in 32 bits alone.)
      if (__shfl_sync(kFull, (int)close, a.k)) {
        const float last = unordered(__shfl_sync(kFull, found, a.k));
        const int last_id = __shfl_sync(kFull, out.id, a.k);
        if (__any_sync(kFull, key[0] != 0u && near(last, unordered(key[0]), score_err)) &&
            (!ordered_ok || __any_sync(kFull, kept && rival(a, at, row, last_id, last, score_err))))
          sure = false;
      }
    }
  }
  return !sure ? kOpen : ordered_ok ? kSure : kOrderOpen;
}

// Sum and maximum over the lanes that hold slots (the first 16).
__device__ __forceinline__ float slots_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Weight of this lane's slot, from its logit. Renormalised scores are taken relative to a common factor, so
// that scores that underflow float32 (logits far below zero) keep their ratios.
__device__ __forceinline__ float weight_of(const RouteArgs& a, const Slots& s, float l) {
  const bool live = s.id >= 0;
  const float most = unordered(__reduce_max_sync(kFull, ordered(live ? l : -FLT_MAX)));   // the largest selected
  float w;
  if (a.routing == MOE_ROUTE_SOFTMAX) {
    w = a.norm ? expf(l - most) : expf(l - s.top) / s.den;
  } else if (!a.norm) {
    w = score_of(a.routing, l);
  } else if (a.routing == MOE_ROUTE_SIGMOID) {
    // e^l / (1 + e^l), over e^most when every logit is negative
    w = l <= 0.f ? expf(l - fminf(most, 0.f)) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
  } else {
    // far below zero softplus(l) = e^l (its next term is under 2^-24 of it)
    w = most < -17.0f ? expf(0.5f * (l - most)) : score_of(a.routing, l);
  }
  if (!live) w = 0.f;
  if (a.norm) {
    const float total = slots_sum(w);
    w = total > 0.f ? w / total : 0.f;
  }
  return w * a.rsf;
}

// Routes the block's rows; counts its pairs per expert in s_count when grouping.
template <int NJ>
__device__ __forceinline__ void route_block(const RouteArgs& a, long long first, long long last,
                                            int* s_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place at(a);
  float bs[NJ];
  auto load_bias = [&] {
#pragma unroll
    for (int j = 0; j < NJ; ++j) bs[j] = a.bias && at.real(a, j) ? a.bias_p[at.base + j] : 0.f;
  };
  // sixteen and more would be spilled between the rows
  if (NJ < 16) load_bias();
  for (long long r = first + warp; r < last; r += kRWarps) {
    if (NJ >= 16) load_bias();
    float lg[NJ];
    load_row<NJ>(a, at, r, bs, lg);
    Slots s;
    const Verdict v = route_row<NJ>(a, at, r, lg, bs, s);
    if (v == kOrderOpen) settle_order(a, r, a.k + 1, s);
    else if (v == kOpen) route_row_f64<NJ>(a, r, s);
    if (lane >= a.k) s.id = -1;
    const float l = s.id >= 0 ? fminf(load_one(a.logits, (size_t)r * (size_t)a.ld + s.id, a.f32), FLT_MAX) : 0.f;
    const float w = weight_of(a, s, l);
    if (lane < a.k) {
      const size_t p = (size_t)r * a.k + lane;
      a.idx[p] = s.id;
      a.weights[p] = w;
      if (a.pairs && s.id >= 0) atomicAdd(s_count + s.id, 1);
    }
  }
}

struct GroupShared {
  int start[kMaxE];                  // first position of this block's pairs of each expert
  int scan[kRWarps];
  alignas(16) int warp_count[kRWarps * kMaxE];   // [warp][expert] (E experts to a row), and sums of the table
};

// Positions of the block's pairs. `table` holds every block's counts.
__device__ __forceinline__ void group_block(const RouteArgs& a, long long first, long long last,
                                            int block, int blocks, const int* table,
                                            GroupShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = a.E;
  // each warp has a contiguous run of the block's pairs; the first 32 are fetched now
  const long long p0 = first * a.k, p1 = last * a.k;
  const long long run = max(32LL, ((p1 - p0 + kRWarps - 1) / kRWarps + 31) / 32 * 32);
  const long long w0 = p0 + warp * run, w1 = min(p1, w0 + run);
  const int busy = (int)((p1 - p0 + run - 1) / run);   // warps that have pairs
  const int head = w0 + lane < w1 ? a.idx[w0 + lane] : -1;
  auto expert = [&](long long p) { return p == w0 + lane ? head : p < w1 ? a.idx[p] : -1; };
  // pairs of each expert in the blocks before this one, and in all; a thread takes four experts of
  // every parts-th block, with all of its loads on their way at once
  int before = 0, all = 0;
  {
    const int quads = a.pitch / 4, parts = min(kRThreads / quads, kRWarps / 2);
    const int part = tid / quads, q = tid - part * quads;
    int4* sums = (int4*)sh.warp_count;   // [parts][2][quads]
    if (part < parts) {
      int4 n = {0, 0, 0, 0}, m = {0, 0, 0, 0};
#pragma unroll 10
      for (int b = part; b < blocks; b += parts) {
        const int4 c = *(const int4*)(table + b * a.pitch + 4 * q);
        const bool low = b < block;
        n.x += c.x; n.y += c.y; n.z += c.z; n.w += c.w;
        m.x += low ? c.x : 0; m.y += low ? c.y : 0; m.z += low ? c.z : 0; m.w += low ? c.w : 0;
      }
      sums[(2 * part) * quads + q] = n;
      sums[(2 * part + 1) * quads + q] = m;
    }
    __syncthreads();
    if (tid < E)
#pragma unroll 16
      for (int r = 0; r < parts; ++r) {
        all += sh.warp_count[2 * r * a.pitch + tid];
        before += sh.warp_count[(2 * r + 1) * a.pitch + tid];
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
  static_assert(kRWarps == 32, "one lane to a warp's sum");
  const int sum = sh.scan[lane];
  const int base = __reduce_add_sync(kFull, lane < warp ? sum : 0), total = __reduce_add_sync(kFull, sum);
  const int begin = base + inc - all;
  if (tid < E) {
    sh.start[tid] = begin + before;
    if (block == 0) {
      a.offsets[tid] = begin;
      if (tid == E - 1) a.offsets[E] = begin + all;
    }
  }
  // count, scan over the warps, place
  int* count = sh.warp_count + warp * E;
  if (warp < busy) {
    for (int e = lane; e < E; e += 32) count[e] = 0;
    __syncwarp();
    for (long long p = w0 + lane; p - lane < w1; p += 32) {
      const int e = expert(p);
      if (e >= 0) atomicAdd(count + e, 1);
    }
  }
  __syncthreads();
  if (tid < E) {
    int at = sh.start[tid];
    for (int w = 0; w < busy; ++w) {
      const int c = sh.warp_count[w * E + tid];
      sh.warp_count[w * E + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  for (long long p = w0 + lane; p - lane < w1; p += 32) {
    const int e = expert(p);
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
  __shared__ __align__(16) int s_count[kMaxE];
  release_next();
  wait_previous();
  const long long first = min(a.rows, blockIdx.x * a.rows_per_block);   // the last blocks may have none
  const long long last = min(a.rows, first + a.rows_per_block);
  if (a.pairs) {
    for (int e = threadIdx.x; e < kMaxE; e += kRThreads) s_count[e] = 0;
    __syncthreads();
  }
  route_block<NJ>(a, first, last, s_count);
  if (a.pairs) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.pitch; e += kRThreads)
      a.table[(size_t)blockIdx.x * a.pitch + e] = s_count[e];
  }
}

__global__ void __launch_bounds__(kRThreads) group_pairs_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ int4 raw[];
  GroupShared& sh = *(GroupShared*)raw;
  wait_previous();
  const long long first = min(a.rows, blockIdx.x * a.rows_per_block);   // the last blocks may have none
  const long long last = min(a.rows, first + a.rows_per_block);
  group_block(a, first, last, blockIdx.x, gridDim.x, a.table, sh);
}

template <int NJ>
__global__ void __launch_bounds__(kRThreads) route_group_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ int4 raw[];
  GroupShared& sh = *(GroupShared*)raw;
  __shared__ __align__(16) int s_count[kMaxE];
  release_next();
  wait_previous();
  for (int e = threadIdx.x; e < kMaxE; e += kRThreads) s_count[e] = 0;
  __syncthreads();
  route_block<NJ>(a, 0, a.rows, s_count);
  __syncthreads();   // also orders the block's idx writes before its reads of them
  group_block(a, 0, a.rows, 0, 1, s_count, sh);
}

int pitch_of(int E) { return (E + 3) / 4 * 4; }

// Shared memory of the grouping: the warps' counts of E experts each.
size_t group_smem(int E) { return offsetof(GroupShared, warp_count) + sizeof(int) * (size_t)kRWarps * pitch_of(E); }

template <typename... P>
cudaError_t launch_after(void (*kernel)(P...), int blocks, size_t smem, cudaStream_t st, const RouteArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kRThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Opts a kernel into the grouping's shared memory, once per device.
template <auto kernel>
cudaError_t allow_group_smem() {
  static std::atomic<bool> done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GroupShared));
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int NJ>
cudaError_t launch_route(const RouteArgs& a, int blocks, cudaStream_t st) {
  cudaError_t e;
  if (a.pairs && blocks == 1) {
    if ((e = allow_group_smem<route_group_kernel<NJ>>()) != cudaSuccess) return e;
    return launch_after(route_group_kernel<NJ>, 1, group_smem(a.E), st, a);
  }
  if (a.pairs && (e = allow_group_smem<group_pairs_kernel>()) != cudaSuccess) return e;
  e = launch_after(route_rows_kernel<NJ>, blocks, 0, st, a);
  if (e != cudaSuccess || !a.pairs) return e;
  return launch_after(group_pairs_kernel, blocks, group_smem(a.E), st, a);
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
  const long long b = (rows + kBlockRows - 1) / kBlockRows;
  return b < kMaxBlocks ? b : kMaxBlocks;
}

size_t workspace_of(const moe_route_cfg& c, int64_t rows) {
  const size_t table = (size_t)blocks_of(rows) * pitch_of(c.num_experts) * sizeof(int);
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
  // whole vectors of four: every lane of a group is full, and rows start on a vector
  a.vec = a.per >= 4 && (a.per & (a.per - 1)) == 0 && size == a.per * a.lanes && ld_logits % 4 == 0 &&
          aligned_to(logits, 4 * float_bytes(c.logits_dtype));
  a.rsf = c.routed_scaling_factor;
  a.logits = logits; a.bias_p = expert_bias; a.idx = idx; a.weights = weights;
  a.pairs = group ? sorted_pairs : nullptr;
  a.offsets = expert_offsets; a.perm = token_to_perm; a.table = (int*)workspace;
  a.pitch = pitch_of(a.E);
  cudaError_t e;
  switch (a.per) {
    case 1: e = launch_route<1>(a, blocks, st); break;
    case 2: e = launch_route<2>(a, blocks, st); break;
    case 3: e = launch_route<3>(a, blocks, st); break;
    case 4: e = launch_route<4>(a, blocks, st); break;
    case 5: e = launch_route<5>(a, blocks, st); break;
    case 6: e = launch_route<6>(a, blocks, st); break;
    case 7: case 8: e = launch_route<8>(a, blocks, st); break;
    default: e = a.per <= 16 ? launch_route<16>(a, blocks, st) : launch_route<32>(a, blocks, st);
  }
  return e == cudaSuccess ? MOE_OK : fail(e);
}
