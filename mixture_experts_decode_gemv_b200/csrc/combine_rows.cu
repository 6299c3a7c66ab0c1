// moe_combine_rows: out[r] = sum_s weights[r, s] * y[token_to_perm[r * k + s]] + gate[r] * shared[r].
//
// Bound by memory: every row of y is read once and every row of out written once. A thread takes
// one column of a row and adds its slots in slot order in float32, so a row's result does not
// depend on how the rows are shared out; the one rounding is the store.
#include "host.h"
#include "rows.cuh"

namespace {

using namespace moe_rows;

struct CombineArgs {
  long long rows, ld_y, y_rows, ld_shared, ld_out;
  int n, top_k;
  bool y_f32, out_f32;
  const void* y;
  const int* perm;
  const float* weights;
  const void* shared;
  const float* gate;
  void* out;
};

constexpr int kCThreads = 128;

__global__ void __launch_bounds__(kCThreads) combine_rows_kernel(const __grid_constant__ CombineArgs a) {
  const int col = blockIdx.x * kCThreads + threadIdx.x;
  if (col >= a.n) return;
  for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
    float acc = 0.f;
    for (int s = 0; s < a.top_k; ++s) {
      const long long at = a.perm[r * a.top_k + s];
      if (at < 0 || at >= a.y_rows) continue;
      const float w = a.weights ? a.weights[r * a.top_k + s] : 1.0f;
      acc = fmaf(w, load_one(a.y, (size_t)at * a.ld_y + col, a.y_f32), acc);
    }
    if (a.shared) {
      const float g = a.gate ? a.gate[r] : 1.0f;
      acc = fmaf(g, load_one(a.shared, (size_t)r * a.ld_shared + col, a.y_f32), acc);
    }
    const size_t o = (size_t)r * a.ld_out + col;
    if (a.out_f32) ((float*)a.out)[o] = acc;
    else ((__nv_bfloat16*)a.out)[o] = __float2bfloat16_rn(acc);
  }
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
  a.y_f32 = y_dtype == MOE_FMT_F32; a.out_f32 = out_dtype == MOE_FMT_F32;
  a.y = y; a.perm = token_to_perm; a.weights = weights; a.shared = shared; a.gate = shared_gate;
  a.out = out;
  const dim3 grid((unsigned)((n + kCThreads - 1) / kCThreads), (unsigned)(rows < 65535 ? rows : 65535));
  combine_rows_kernel<<<grid, kCThreads, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : fail(e);
}
