// moe_combine_rows: out[r] = sum_s weights[r, s] * y[token_to_perm[r * k + s]] + gate[r] * shared[r].
//
// Bound by memory: every row of y is read once and every row of out written once (8192 rows of 8 slots x 2048 bf16: 303 MB
// in 53 us from HBM, 45 where a loop leaves part of it in L2). A thread takes up to 16
// bytes of y in a row (one vector, or several narrower ones where the row's length or address allows no
// whole vector), has the loads of eight slots on their way together, and adds them in slot order in float32:
// a row's result does not depend on how the rows are shared out, and the one rounding is the store.
#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

struct CombineArgs {
  long long rows, ld_y, y_rows, ld_shared, ld_out;
  int n, top_k;
  int lanes;           // threads of a row
  const void* y;
  const int* perm;
  const float* weights;
  const void* shared;
  const float* gate;
  void* out;
};

constexpr int kCThreads = 128;
constexpr int kSlots = 8;    // slots whose loads go together

template <int BYTES>
struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

// Loads of what is read once; whole vectors stay out of L1 and are fetched into L2 in 256 bytes.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
template <typename T>
__device__ __forceinline__ T load_once(const T* p) { return __ldg(p); }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// VEC elements of Y to a load, U loads to a thread, `lanes` vectors apart.
template <typename Y, typename O, int VEC, int U>
__global__ void __launch_bounds__(kCThreads) combine_rows_kernel(const __grid_constant__ CombineArgs a) {
  using RawY = typename Raw<VEC * sizeof(Y)>::type;
  union Piece {
    RawY raw;
    Y v[VEC];
    __device__ Piece() {}
  };
  release_next();
  wait_previous();
  const long long id = (long long)blockIdx.x * kCThreads + threadIdx.x;
  // a 64-bit quotient only where there are that many threads
  const long long r = a.rows * a.lanes <= 0x7fffffffLL ? (int)id / a.lanes : id / a.lanes;
  if (r >= a.rows) return;
  const int first = (int)(id - r * a.lanes), vectors = a.n / VEC;
  const Y* y = (const Y*)a.y;
  float acc[U][VEC] = {};
  for (int s0 = 0; s0 < a.top_k; s0 += kSlots) {
    int at[kSlots];
    float w[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const bool real = s0 + s < a.top_k;
      at[s] = real ? a.perm[r * a.top_k + s0 + s] : -1;
      w[s] = real && a.weights ? a.weights[r * a.top_k + s0 + s] : 1.0f;
    }
    Piece p[kSlots][U];
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = first + u * a.lanes;
        if (at[s] >= 0 && at[s] < a.y_rows && c < vectors)
          p[s][u].raw = load_once((const RawY*)(y + (size_t)at[s] * a.ld_y + (size_t)c * VEC));
      }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (at[s] >= 0 && at[s] < a.y_rows)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[u][i] = fmaf(w[s], to_float(p[s][u].v[i]), acc[u][i]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = first + u * a.lanes;
    if (c >= vectors) continue;
    if (a.shared) {
      const float g = a.gate ? a.gate[r] : 1.0f;
      Piece p;
      p.raw = *(const RawY*)((const Y*)a.shared + (size_t)r * a.ld_shared + (size_t)c * VEC);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[u][i] = fmaf(g, to_float(p.v[i]), acc[u][i]);
    }
    alignas(16) O o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) from_float(o + i, acc[u][i]);
    O* out = (O*)a.out + (size_t)r * a.ld_out + (size_t)c * VEC;
    constexpr int kStore = VEC * sizeof(O) < 16 ? VEC * sizeof(O) : 16;
    using RawO = typename Raw<kStore>::type;
#pragma unroll
    for (int i = 0; i < (int)(VEC * sizeof(O)) / kStore; ++i) ((RawO*)out)[i] = ((const RawO*)o)[i];
  }
}

template <typename Y, typename O, int VEC>
cudaError_t launch_combine(CombineArgs a, cudaStream_t st) {
  constexpr int U = 16 / (int)(VEC * sizeof(Y));
  a.lanes = (a.n / VEC - 1) / U + 1;   // at most 2^31 / U, so that a thread's vectors stay below 2^31
  const long long blocks = (a.rows * a.lanes + kCThreads - 1) / kCThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;   // more output than any device holds
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kCThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_rows_kernel<Y, O, VEC, U>, a);
}

template <typename Y, typename O>
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st) {
  // the widest vectors that every row starts on and ends with
  auto fits = [&](int vec) {
    const size_t o = vec * sizeof(O) < 16 ? vec * sizeof(O) : 16;
    return a.n % vec == 0 && a.ld_y % vec == 0 && a.ld_out % vec == 0 && (!a.shared || a.ld_shared % vec == 0) &&
           moe_host::aligned_to(a.y, vec * sizeof(Y)) && moe_host::aligned_to(a.shared, vec * sizeof(Y)) &&
           moe_host::aligned_to(a.out, o);
  };
  if constexpr (sizeof(Y) == 2) {
    if (fits(8)) return launch_combine<Y, O, 8>(a, st);
  }
  if (fits(4)) return launch_combine<Y, O, 4>(a, st);
  if (fits(2)) return launch_combine<Y, O, 2>(a, st);
  return launch_combine<Y, O, 1>(a, st);
}

}  // namespace

extern "C" int moe_combine_rows(int64_t rows, int32_t n, int32_t top_k, int32_t y_dtype,
                                const void* y, int64_t ld_y, int64_t y_rows,
                                const int32_t* token_to_perm, const float* weights,
                                const void* shared, int64_t ld_shared, const float* shared_gate,
                                int32_t out_dtype, void* out, int64_t ld_out, void* stream) {
  using namespace moe_host;
  if (rows < 0 || rows > 0x7fffffffLL || n < 1 || top_k < 1 || top_k > MOE_ROUTE_MAX_TOP_K ||
      y_rows < 0 || rows * top_k > 0x7fffffffLL)
    return MOE_ERR_BAD_SHAPE;
  if (!float_format(y_dtype) || !float_format(out_dtype)) return MOE_ERR_BAD_FORMAT;
  if (ld_y < n || ld_out < n || (shared && ld_shared < n)) return MOE_ERR_BAD_SHAPE;
  if (shared_gate && !shared) return MOE_ERR_BAD_OPTION;
  if (rows == 0) return MOE_OK;
  if ((!y && y_rows > 0) || !token_to_perm || !out) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(y, float_bytes(y_dtype)) || !aligned_to(token_to_perm, 4) ||
      !aligned_to(weights, 4) || !aligned_to(shared, float_bytes(y_dtype)) ||
      !aligned_to(shared_gate, 4) || !aligned_to(out, float_bytes(out_dtype)))
    return MOE_ERR_MISALIGNED;
  int rc;
  if ((rc = supported_device())) return rc;
  Range range("moe_combine_rows");
  CombineArgs a;
  a.rows = rows; a.ld_y = ld_y; a.y_rows = y_rows; a.ld_shared = ld_shared; a.ld_out = ld_out;
  a.n = n; a.top_k = top_k;
  a.y = y; a.perm = token_to_perm; a.weights = weights; a.shared = shared; a.gate = shared_gate;
  a.out = out;
  cudaStream_t st = (cudaStream_t)stream;
  const bool y32 = y_dtype == MOE_FMT_F32, o32 = out_dtype == MOE_FMT_F32;
  const cudaError_t e = y32 ? (o32 ? launch_combine<float, float>(a, st) : launch_combine<float, __nv_bfloat16>(a, st))
                            : (o32 ? launch_combine<__nv_bfloat16, float>(a, st)
                                   : launch_combine<__nv_bfloat16, __nv_bfloat16>(a, st));
  return e == cudaSuccess ? MOE_OK : fail(e);
}
