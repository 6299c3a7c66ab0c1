// moe_quantize_rows_int8: symmetric 8-bit codes and one float32 scale per row.
//
//   scale = max(max|x| / 127, 2^-126),  q = x / scale rounded to the nearest integer, ties to even
//
// The rounding is that of the exact quotient, without a division per element: q0 = rint(x * (1 /
// scale)) is off by at most one, and the remainder r = x - q0 * scale, taken in one fma, is exact:
// x and q0 * scale are multiples of half an ulp of the scale, and where the choice is open (r near
// half a scale) r needs at most 24 bits. Comparing r with scale / 2 corrects q0.
//
// Bound by memory: each element is read once and one byte is written.
#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

constexpr int kQThreads = 256;

__device__ __forceinline__ int quantise(float x, float scale, float inv, float half) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, scale, x);
  const bool odd = ((int)q) & 1;
  if (r > half || (r == half && odd)) q += 1.0f;
  if (r < -half || (r == -half && odd)) q -= 1.0f;
  return (int)fminf(127.0f, fmaxf(-127.0f, q));
}

// One block per row, two passes over it.
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(int k, bool f32, const void* x,
                                                                  long long ld_x, int8_t* codes,
                                                                  long long ld_codes, float* scales) {
  __shared__ uint32_t s_max[kQThreads / 32];
  const long long row = blockIdx.x;
  const size_t base = (size_t)row * (size_t)ld_x;
  // magnitudes as integers: the order of their bits is theirs, and infinity and NaN are largest
  uint32_t top = 0;
  for (int j = threadIdx.x; j < k; j += kQThreads)
    top = max(top, __float_as_uint(load_one(x, base + j, f32)) & 0x7fffffffu);
  top = __reduce_max_sync(kFull, top);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
  __syncthreads();
  top = s_max[0];
  for (int w = 1; w < kQThreads / 32; ++w) top = max(top, s_max[w]);
  const bool bad = top >= 0x7f800000u;
  const float scale = bad ? __uint_as_float(0x7fc00000u)
                      : top == 0 ? 1.0f : fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), 0x1p-126f);
  const float inv = __fdiv_rn(1.0f, scale), half = 0.5f * scale;
  int8_t* out = codes + (size_t)row * (size_t)ld_codes;
  for (int j = threadIdx.x; j < k; j += kQThreads)
    out[j] = bad ? (int8_t)0 : (int8_t)quantise(load_one(x, base + j, f32), scale, inv, half);
  if (threadIdx.x == 0) scales[row] = scale;
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
  quantize_rows_kernel<<<(unsigned)rows, kQThreads, 0, (cudaStream_t)stream>>>(
      k, x_dtype == MOE_FMT_F32, x, ld_x, codes, ld_codes, scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : fail(e);
}
