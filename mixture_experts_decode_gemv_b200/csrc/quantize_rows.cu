// moe_quantize_rows_int8: symmetric 8-bit codes and one float32 scale per row.
//
//   scale = max(max|x| / 127, 2^-126),  q = x / scale rounded to the nearest integer, ties to even
//
// The rounding is that of the exact quotient, without a division per element: q0 = rint(x * (1 /
// scale)) is off by at most one, and the remainder r = x - q0 * scale, taken in one fma, is exact:
// x and q0 * scale are multiples of half an ulp of the scale, and where the choice is open (r near
// half a scale) r needs at most 24 bits. Comparing r with scale / 2 corrects q0.
//
// Bound by memory: each element is read once and one byte is written (8192 x 5120 bf16: 20.7 us, 6.1 TB/s). A row stays in the registers of
// the threads that read it (32, 128 or 512 of them, eight elements to a load) between the pass for its
// maximum and the pass that rounds. The ordinary element costs five instructions: the quotient rounded
// by adding 1.5 * 2^23 in the fma that forms it, the remainder, and its largest magnitude so far; only
// where that reaches half a scale are the group's eight elements looked at again.
#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

constexpr int kQThreads = 128;
constexpr int kQGroups = 8;    // groups of eight elements that a thread holds at most

__device__ __forceinline__ int quantise(float x, float scale, float inv, float half) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, scale, x);
  const bool odd = ((int)q) & 1;
  if (r > half || (r == half && odd)) q += 1.0f;
  if (r < -half || (r == -half && odd)) q -= 1.0f;
  return (int)fminf(127.0f, fmaxf(-127.0f, q));
}

// Scale of a row from the bits of its largest magnitude (infinity and NaN have the largest).
__device__ __forceinline__ float scale_of(uint32_t top) {
  return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
         : top == 0u        ? 1.0f
                            : fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), 0x1p-126f);
}

// A load of what is read once: kept out of L1, fetched into L2 in whole 256 bytes.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Eight elements as they lie in memory.
template <bool F32>
struct Eight {
  uint4 a, b;   // bf16: a alone
  __device__ __forceinline__ void load(const void* p) {
    a = load_once((const uint4*)p);
    if (F32) b = load_once((const uint4*)p + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (F32) {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  // The larger of `top` and the magnitudes, as float32 bits.
  __device__ __forceinline__ uint32_t most(uint32_t top) const {
    if constexpr (F32) {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7fffffffu);
      return top;
    } else {
      const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu),
                                  __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
      return max(top, max(m << 16, m & 0xffff0000u));
    }
  }
};

// Codes of eight elements. `far_limit` is half a scale, or infinity where the scale is a power of two: then
// the reciprocal, the quotients and their rounding are exact, ties (which such rows are full of) included.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float scale, float inv, float half, float far_limit) {
  constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even
  float t[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(v[i], inv, kRound);
    far = fmaxf(far, fabsf(fmaf(kRound - t[i], scale, v[i])));
  }
  if (far >= far_limit) {
    // one step towards the remainder where it is over half a scale, or is half and the code odd. (bf16 rows
    // come here for every element that is half of their largest.)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = fmaf(kRound - t[i], scale, v[i]);
      const bool odd = __float_as_uint(t[i]) & 1u;
      if (fabsf(r) > half || (fabsf(r) == half && odd)) t[i] += copysignf(1.0f, r);
    }
  }
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __float_as_uint(t[i]);
  auto pack = [](uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  };
  return make_uint2(pack(q[0], q[1], q[2], q[3]), pack(q[4], q[5], q[6], q[7]));
}

// TPR threads to a row, `groups` groups of eight elements to a row (at most TPR * NG).
template <bool F32, int TPR, int NG>
__global__ void __launch_bounds__(TPR < kQThreads ? kQThreads : TPR)
quantize_vectors_kernel(long long rows, int groups, const uint8_t* x, long long ld_bytes, int8_t* codes,
                        long long ld_codes, float* scales) {
  constexpr int kThreads = TPR < kQThreads ? kQThreads : TPR;
  __shared__ uint32_t s_max[kThreads / 32];
  const int t = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const bool live = row < rows;   // threads of a row agree; all of the block reach the barrier
  release_next();
  wait_previous();
  Eight<F32> e[NG];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const int g = t + j * TPR;
    if (live && g < groups) e[j].load(x + row * ld_bytes + (size_t)g * (F32 ? 32 : 16));
    else e[j].zero();
  }
#pragma unroll
  for (int j = 0; j < NG; ++j) top = e[j].most(top);
  top = __reduce_max_sync(kFull, top);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
    const int first = threadIdx.x / TPR * (TPR / 32);
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) top = max(top, s_max[first + w]);
  }
  if (!live) return;
  const float scale = scale_of(top);
  const bool bad = top >= 0x7f800000u;
  const float inv = __fdiv_rn(1.0f, scale), half = 0.5f * scale;
  const float far_limit = (__float_as_uint(scale) & 0x7fffffu) == 0u ? INFINITY : half;
  if (t == 0) scales[row] = scale;
  int8_t* out = codes + row * ld_codes;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const int g = t + j * TPR;
    if (g < groups) {
      float v[8];
      e[j].values(v);
      const uint2 q = codes_of(v, scale, inv, half, far_limit);
      *(uint2*)(out + (size_t)g * 8) = bad ? make_uint2(0, 0) : q;
    }
  }
}

// One block per row, two passes over it, any stride and alignment: for what the kernel above does not take
// (rows that do not start on whole vectors, or are longer than 32768 elements).
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(int k, bool f32, const void* x,
                                                                  long long ld_x, int8_t* codes,
                                                                  long long ld_codes, float* scales) {
  __shared__ uint32_t s_max[kQThreads / 32];
  release_next();
  wait_previous();
  const long long row = blockIdx.x;
  const size_t base = (size_t)row * (size_t)ld_x;
  const unsigned n = k;   // positions unsigned: the last step may pass 2^31 - 1
  // magnitudes as integers: the order of their bits is theirs, and infinity and NaN are largest
  uint32_t top = 0;
#pragma unroll 4
  for (unsigned j = threadIdx.x; j < n; j += kQThreads)
    top = max(top, __float_as_uint(load_one(x, base + j, f32)) & 0x7fffffffu);
  top = __reduce_max_sync(kFull, top);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
  __syncthreads();
  top = s_max[0];
  for (int w = 1; w < kQThreads / 32; ++w) top = max(top, s_max[w]);
  const bool bad = top >= 0x7f800000u;
  const float scale = scale_of(top);
  const float inv = __fdiv_rn(1.0f, scale), half = 0.5f * scale;
  int8_t* out = codes + (size_t)row * (size_t)ld_codes;
#pragma unroll 4
  for (unsigned j = threadIdx.x; j < n; j += kQThreads)
    out[j] = bad ? (int8_t)0 : (int8_t)quantise(load_one(x, base + j, f32), scale, inv, half);
  if (threadIdx.x == 0) scales[row] = scale;
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned blocks, int threads, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, (P)args...);
}

template <bool F32, int TPR, int NG>
cudaError_t launch_vectors(int64_t rows, int groups, const void* x, int64_t ld_x, int8_t* codes, int64_t ld_codes,
                           float* scales, cudaStream_t st) {
  constexpr int threads = TPR < kQThreads ? kQThreads : TPR, per = threads / TPR;
  return launch_after(quantize_vectors_kernel<F32, TPR, NG>, (unsigned)((rows + per - 1) / per), threads, st, rows,
                      groups, x, ld_x * (F32 ? 4 : 2), codes, ld_codes, scales);
}

template <bool F32, int TPR>
cudaError_t launch_vectors(int64_t rows, int groups, const void* x, int64_t ld_x, int8_t* codes, int64_t ld_codes,
                           float* scales, cudaStream_t st) {
  const int ng = (groups + TPR - 1) / TPR;   // by the caller's rule up to 4 for 32 threads, from 3 on for 512
  if constexpr (TPR < 512) {
    if (ng <= 2) return launch_vectors<F32, TPR, 2>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
  }
  if (ng <= 3) return launch_vectors<F32, TPR, 3>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
  if (TPR == 32 || ng <= 5) return launch_vectors<F32, TPR, 5>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
  if constexpr (TPR > 32) return launch_vectors<F32, TPR, kQGroups>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
}

// A warp to a row up to 1024 elements, where more threads would idle (65536 rows of 768: 31.7 us against 69
// with 128 threads to a row); 128 threads up to 8192 (64 rows of 2048: 1.4 us against 2.8 with a warp; 8192
// of 2048: 12.0 against 13.8, 10.2 now); 512 beyond.
template <bool F32>
cudaError_t launch_vectors(int64_t rows, int groups, const void* x, int64_t ld_x, int8_t* codes, int64_t ld_codes,
                           float* scales, cudaStream_t st) {
  if (groups <= 128) return launch_vectors<F32, 32>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
  if (groups <= 128 * kQGroups) return launch_vectors<F32, 128>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
  return launch_vectors<F32, 512>(rows, groups, x, ld_x, codes, ld_codes, scales, st);
}

}  // namespace

extern "C" int moe_quantize_rows_int8(int64_t rows, int32_t k, int32_t x_dtype, const void* x,
                                      int64_t ld_x, int8_t* codes, int64_t ld_codes, float* scales,
                                      void* stream) {
  using namespace moe_host;
  if (rows < 0 || rows > 0x7fffffffLL || k < 1) return MOE_ERR_BAD_SHAPE;
  if (!float_format(x_dtype)) return MOE_ERR_BAD_FORMAT;
  if (ld_x < k || ld_codes < k) return MOE_ERR_BAD_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(x, float_bytes(x_dtype)) || !aligned_to(scales, 4)) return MOE_ERR_MISALIGNED;
  int rc;
  if ((rc = supported_device())) return rc;
  Range range("moe_quantize_rows_int8");
  cudaStream_t st = (cudaStream_t)stream;
  const bool f32 = x_dtype == MOE_FMT_F32;
  const bool whole = k % 8 == 0 && k <= 512 * kQGroups * 8 && aligned_to(x, 16) && aligned_to(codes, 8) &&
                     ld_x * (int64_t)float_bytes(x_dtype) % 16 == 0 && ld_codes % 8 == 0;
  cudaError_t e;
  if (!whole) e = launch_after(quantize_rows_kernel, (unsigned)rows, kQThreads, st, k, f32, x, ld_x, codes, ld_codes, scales);
  else if (f32) e = launch_vectors<true>(rows, k / 8, x, ld_x, codes, ld_codes, scales, st);
  else e = launch_vectors<false>(rows, k / 8, x, ld_x, codes, ld_codes, scales, st);
  return e == cudaSuccess ? MOE_OK : fail(e);
}
