// moe_matmul_int8: rows of int8 codes times int8 matrices of the experts, scaled per row and per
// channel, with the gated activation of two products where a second matrix is given.
//
//   y[i, j] = x_scales[r(i)] * scales[e(i), j] * sum_k x[r(i), k] * w[e(i), j, k]
//
// The sums are int32 and exact (|x|, |w| <= 128 and k <= 131056 keep them below 2^31), so neither
// tiling nor order can change a bit of them; what follows is float32 and one rounding to the output
// type.
#include "host.h"
#include "rows.cuh"

#include "common.cuh"

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
};

constexpr int kT = 64;        // rows and channels of a tile
constexpr int kKB = 64;       // bytes of k per step
constexpr int kMThreads = 256;

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
}

// Tiles of 64 rows x 64 channels with dp4a: the plain kernel that every other one is checked
// against.
template <bool ACT>
__global__ void __launch_bounds__(kMThreads) matmul_int8_kernel(const __grid_constant__ MatmulArgs a) {
  __shared__ int s_x[kT][kKB / 4 + 1], s_w[kT][kKB / 4 + 1], s_u[ACT ? kT : 1][kKB / 4 + 1];
  __shared__ long long s_row[kT];
  __shared__ float s_scale[kT];
  // block y -> (expert, tile of its rows)
  long long t = blockIdx.y, begin = 0, end = 0;
  int e = 0;
  for (; e < a.experts; ++e) {
    expert_range(a, e, begin, end);
    const long long tiles = end > begin ? (end - begin + kT - 1) / kT : 0;
    if (t < tiles) break;
    t -= tiles;
  }
  if (e == a.experts) return;
  const long long i0 = begin + t * kT;
  const int live = (int)min((long long)kT, end - i0);
  for (int j = threadIdx.x; j < kT; j += kMThreads) {
    long long row = -1;
    float sc = 0.f;
    if (j < live) {
      row = i0 + j;
      float pw = 1.f;
      if (a.pairs) {
        const int p = a.pairs[i0 + j];
        row = p >= 0 && p / a.top_k < a.x_rows ? p / a.top_k : -1;
        if (row >= 0 && a.pair_weights) pw = a.pair_weights[p];
      }
      if (row >= 0) sc = a.x_scales[row] * pw;
    }
    s_row[j] = row;
    s_scale[j] = sc;
  }
  __syncthreads();
  const int n0 = blockIdx.x * kT;
  const int8_t* w = a.w + (size_t)e * a.w_stride;
  const int8_t* up = ACT ? a.up + (size_t)e * a.up_stride : nullptr;
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  int acc[4][4] = {}, acu[4][4] = {};
  for (int k0 = 0; k0 < a.k; k0 += kKB) {
    for (int j = threadIdx.x; j < kT * (kKB / 4); j += kMThreads) {
      const int r = j / (kKB / 4), c = j % (kKB / 4);
      const bool in_k = k0 + 4 * c < a.k;
      s_x[r][c] = in_k && s_row[r] >= 0 ? *(const int*)(a.x + (size_t)s_row[r] * a.ld_x + k0 + 4 * c) : 0;
      const size_t at = (size_t)(n0 + r) * a.k + k0 + 4 * c;
      s_w[r][c] = in_k && n0 + r < a.n ? *(const int*)(w + at) : 0;
      if (ACT) s_u[r][c] = in_k && n0 + r < a.n ? *(const int*)(up + at) : 0;
    }
    __syncthreads();
#pragma unroll 4
    for (int c = 0; c < kKB / 4; ++c) {
      int xv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = s_x[tr * 4 + i][c];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int wv = s_w[tc + 16 * j][c], uv = ACT ? s_u[tc + 16 * j][c] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][j] = __dp4a(xv[i], wv, acc[i][j]);
          if (ACT) acu[i][j] = __dp4a(xv[i], uv, acu[i][j]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tr * 4 + i;
    if (s_row[r] < 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + tc + 16 * j;
      if (c >= a.n) continue;
      float y = (float)acc[i][j] * s_scale[r] *
                *(const float*)((const char*)a.ws + (size_t)e * a.ws_stride + (size_t)c * 4);
      if (ACT) {
        const float u = (float)acu[i][j] * s_scale[r] *
                        *(const float*)((const char*)a.ups + (size_t)e * a.ups_stride + (size_t)c * 4);
        y = moe::act_mul(a.act, y, u);
      }
      const size_t o = (size_t)(i0 + r) * a.ld_out + c;
      if (a.out_f32) ((float*)a.out)[o] = y;
      else ((__nv_bfloat16*)a.out)[o] = __float2bfloat16_rn(y);
    }
  }
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
  // every expert may end in a tile that is not full
  const int64_t tiles = (rows + kT - 1) / kT + (expert_offsets ? c.num_experts : 0);
  const dim3 grid((unsigned)((c.n + kT - 1) / kT), (unsigned)tiles);
  if (up) matmul_int8_kernel<true><<<grid, kMThreads, 0, (cudaStream_t)stream>>>(a);
  else matmul_int8_kernel<false><<<grid, kMThreads, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : fail(e);
}
