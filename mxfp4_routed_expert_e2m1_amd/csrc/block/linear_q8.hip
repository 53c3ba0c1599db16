// linear_q8.hip -- dense projection of int8 codes with a scale per row and per
// channel: y[t][n] = qs[t] ws[n] sum_k q[t][k] w[n][k] (+ bias[n]).
//
// The contraction runs on the int8 matrix core (32x32x32, int32 sums): lane l
// supplies channel row l % 32 of A and token row l % 32 of B, each with the
// 16 codes of K slot l / 32, and receives token column l % 32 of D, element i
// at channel row 8 (i / 4) + 4 (l / 32) + i % 4.  |sum| <= 2^14 d_in < 2^31.
#include "block.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct LinearArgs {
  const int8_t* w;
  int64_t ld_w;
  const float* ws;
  const float* bias;
  const int8_t* q;
  int64_t ld_q;
  const float* qs;
  int rows, n_out, d_in;
  void* y;
  int y_bf16;
  int64_t ld_y;
};

__device__ inline i32x16 mfma_i8(i32x4 a, i32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// 16 codes at row[k..k+15], those from d_in on 0; k % 16 == 0
__device__ inline i32x4 load_codes(const int8_t* row, int k, int d_in) {
  if (k + 16 <= d_in) return *(const i32x4*)(row + k);
  i32x4 v = {0, 0, 0, 0};
  for (int i = 0; k + i < d_in; ++i) v[i >> 2] |= (int)(uint8_t)row[k + i] << (8 * (i & 3));
  return v;
}

// the epilogue's arithmetic, shared by every kernel (each operation rounded by
// itself: no fused multiply-add with the bias)
__device__ inline float linear_value(int sum, float qs, float ws, const float* bias, int n) {
#pragma clang fp contract(off)
  float v = (float)sum * qs * ws;
  if (bias) v = v + bias[n];
  return v;
}
__device__ inline void linear_store(const LinearArgs& a, int t, int n, float v) {
  if (a.y_bf16) ((__bf16*)a.y)[(int64_t)t * a.ld_y + n] = (__bf16)v;
  else ((float*)a.y)[(int64_t)t * a.ld_y + n] = v;
}

// One wave per 32 x 32 outputs, operands from memory as they are.
__global__ __launch_bounds__(64) void linear_tile_kernel(LinearArgs a) {
  const int lane = lane_id(), r = lane & 31, slot = lane >> 5;
  const int n0 = blockIdx.x * 32, t0 = blockIdx.y * 32;
  const bool n_in = n0 + r < a.n_out, t_in = t0 + r < a.rows;
  const int8_t* w = a.w + (int64_t)min(n0 + r, a.n_out - 1) * a.ld_w;
  const int8_t* q = a.q + (int64_t)min(t0 + r, a.rows - 1) * a.ld_q;
  i32x16 c = {};
  for (int k = 0; k < a.d_in; k += 32) {
    i32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    if (n_in) x = load_codes(w, k + 16 * slot, a.d_in);
    if (t_in) y = load_codes(q, k + 16 * slot, a.d_in);
    c = mfma_i8(x, y, c);
  }
  const int t = t0 + r;
  if (t >= a.rows) return;
  const float qs = a.qs[t];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = n0 + 8 * (i / 4) + 4 * slot + i % 4;
    if (n < a.n_out) linear_store(a, t, n, linear_value(c[i], qs, a.ws[n], a.bias, n));
  }
}

static int linear_check(const moe_linear_t* L) {
  if (!L || !L->w || !L->w_scales) return MOE_ERR_INVALID_ARG;
  if (L->n_out < 1 || L->d_in < 1 || L->d_in > 65536) return MOE_ERR_SHAPE;
  if (L->ld_w < L->d_in) return MOE_ERR_STRIDE;
  if (!aligned(L->w, 16) || L->ld_w % 16 != 0 || !aligned(L->w_scales, 4) ||
      !aligned(L->bias, 4))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_q8_workspace_bytes(const moe_linear_t* L, int rows) {
  (void)L;
  (void)rows;
  return 0;
}

extern "C" int moe_linear_q8(const moe_linear_t* L, const int8_t* q, int64_t ld_q,
                             const float* qs, int rows, void* y, int y_type, int64_t ld_y,
                             void* ws, size_t ws_bytes, void* stream) {
  const int rc = linear_check(L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(y_type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!q || !qs || !y) return MOE_ERR_INVALID_ARG;
  if (ld_q < L->d_in || ld_y < L->n_out) return MOE_ERR_STRIDE;
  if (!aligned(q, 16) || ld_q % 16 != 0 || !aligned(qs, 4) || !aligned(y, type_size(y_type)))
    return MOE_ERR_ALIGNMENT;
  const size_t need = moe_linear_q8_workspace_bytes(L, rows);
  if (need > 0) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  }
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  hipStream_t s = (hipStream_t)stream;
  const LinearArgs a{L->w, L->ld_w, L->w_scales, L->bias, q, ld_q, qs, rows, L->n_out, L->d_in,
                     y, y_type == MOE_TYPE_BF16, ld_y};
  const dim3 grid((unsigned)((L->n_out + 31) / 32), (unsigned)((rows + 31) / 32));
  hipLaunchKernelGGL(linear_tile_kernel, grid, dim3(64), 0, s, a);
  return launch_status();
}
