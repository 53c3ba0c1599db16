// norm.hip -- the norms before and after a block, with the block's gate, the
// scaled residual and the next block's norm in the same pass, and the row
// quantiser.
//
//   before   h = x r w,  r = 1 / sqrt(sum x^2 / D + eps)
//   after    out = residual_scale * residual + gate * b,  b = y r w (or y),
//            then h = rms(out) * next_w of the stored out
//
// One workgroup holds one row in registers, 8 consecutive elements per thread
// and unit, so every input is read once and every output written once; a row
// statistic is a sum per thread, per wave, then over the waves through LDS.
#include "block.h"

#include <math.h>

namespace moe {

constexpr int kMaxNormCols = 16384;

struct NormOut {
  void* h;
  int h_type;
  int64_t ld_h;
  int quant;
  int8_t* q;
  int64_t ld_q;
  float* qs;
  int64_t ld_qs;
  const float* w;  // pre_w of the norm that makes h
  float eps;
};

struct NormArgs {
  const void* x;  // the rows to normalise: x before a block, y after one
  int64_t ld_x;
  int cols;
  // after a block
  int post_norm;
  float eps, res_scale;
  const float* w;
  const void* res;
  int64_t ld_res;
  const void* gate;
  int gate_type;
  int64_t gate_row, gate_col;
  void* out;
  int64_t ld_out;
  int has_next;
  NormOut o;
};

// Sum over the workgroup; `slots` is LDS of one float per wave, not shared
// with another reduction of the same row.
__device__ inline float wg_sum(float v, float* slots) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if (lane_id() == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += slots[i];
  return s;
}
__device__ inline float wg_max(float v, float* slots) {
  v = wave_max(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if (lane_id() == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = slots[0];
  for (int i = 1; i < waves; ++i) s = fmaxf(s, slots[i]);
  return s;
}

template <bool VEC, typename T>
__device__ inline Raw8<T> load_unit(const T* row, int e, int cols) {
  if constexpr (VEC) {
    return e < cols ? load8_vec(row + e) : Raw8<T>{};
  } else {
    return load8_part(row + e, min(8, cols - e));
  }
}

template <bool VEC, typename T>
__device__ inline void store_unit(T* row, int e, int cols, const float (&v)[8]) {
  if (e >= cols) return;
  if constexpr (VEC) {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (T)v[i];
    u32x4 r[sizeof(T) / 2];
    __builtin_memcpy(r, t, sizeof(t));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) ((u32x4*)(row + e))[i] = r[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < cols) row[e + i] = (T)v[i];
  }
}

// the value an element keeps once it is stored in T
template <typename T>
__device__ inline float stored(float v) {
  return (float)(T)v;
}

// One row's h = v * r * w from its values in registers, with its codes.
template <int U, bool VEC>
__device__ inline void finish_row(float (&v)[U][8], int row, int cols, float r, const NormOut& o,
                                  float* slots) {
  const int threads = blockDim.x;
  const bool h_bf16 = o.h != nullptr && o.h_type == MOE_TYPE_BF16;
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    if (o.w) {
      float w[8];
      to_f32(load_unit<VEC>(o.w, e, cols), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * r * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] *= r;
    }
    if (h_bf16) {
      store_unit<VEC>((__bf16*)o.h + (int64_t)row * o.ld_h, e, cols, v[u]);
      if (o.quant) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = stored<__bf16>(v[u][i]);
      }
    } else if (o.h) {
      store_unit<VEC>((float*)o.h + (int64_t)row * o.ld_h, e, cols, v[u]);
    }
    if (o.quant == MOE_QUANT_BLOCK) {
      // elements past the row are 0 (0 * r * 0); cols % 32 == 0 keeps the
      // four lanes of a block together
      uint32_t w0, w1;
      const float d = q8_quant8(v[u], w0, w1);
      if (e < cols) {
        *(u32x2*)(o.q + (int64_t)row * o.ld_q + e) = u32x2{w0, w1};
        if ((e & 31) == 0) o.qs[(int64_t)row * o.ld_qs + e / kBlock] = d;
      }
    } else if (o.quant == MOE_QUANT_ROW) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < cols) amax = fmaxf(amax, fabsf(v[u][i]));
    }
  }
  if (o.quant == MOE_QUANT_ROW) {
    amax = wg_max(amax, slots);
    const float d = amax / 127.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = 8 * (u * threads + (int)threadIdx.x);
      if (e >= cols) continue;
      int8_t* q = o.q + (int64_t)row * o.ld_q + e;
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i >> 2] |= ((uint32_t)(int32_t)q8_code(v[u][i], d) & 0xFFu) << (8 * (i & 3));
      if (e + 8 <= cols) {
        *(u32x2*)q = u32x2{w[0], w[1]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < cols) q[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
    }
    if (threadIdx.x == 0) o.qs[(int64_t)row * o.ld_qs] = d;
  }
}

template <typename XT, int U, bool VEC>
__global__ __launch_bounds__(512) void norm_pre_kernel(NormArgs a) {
  __shared__ float slots[2][16];
  const int row = blockIdx.x, cols = a.cols;
  const XT* x = (const XT*)a.x + (int64_t)row * a.ld_x;
  Raw8<XT> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    raw[u] = load_unit<VEC>(x, 8 * (u * (int)blockDim.x + (int)threadIdx.x), cols);
  float v[U][8], ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    to_f32(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
  }
  const float r = 1.0f / sqrtf(wg_sum(ss, slots[0]) / (float)cols + a.o.eps);
  finish_row<U, VEC>(v, row, cols, r, a.o, slots[1]);
}

template <typename XT, typename RT, int U, bool VEC>
__global__ __launch_bounds__(512) void norm_post_kernel(NormArgs a) {
  __shared__ float slots[3][16];
  const int row = blockIdx.x, cols = a.cols, threads = blockDim.x;
  const XT* x = (const XT*)a.x + (int64_t)row * a.ld_x;
  const RT* res = (const RT*)a.res + (int64_t)row * a.ld_res;
  Raw8<XT> raw[U];
  Raw8<RT> rres[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    raw[u] = load_unit<VEC>(x, e, cols);
    rres[u] = load_unit<VEC>(res, e, cols);
  }
  float v[U][8], ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    to_f32(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
  }
  float r = 1.f;
  if (a.post_norm) r = 1.0f / sqrtf(wg_sum(ss, slots[0]) / (float)cols + a.eps);
  float g1 = 1.f;  // a gate that is one number for the row
  if (a.gate && a.gate_col == 0)
    g1 = a.gate_type == MOE_TYPE_F32 ? ((const float*)a.gate)[(int64_t)row * a.gate_row]
                                     : (float)((const __bf16*)a.gate)[(int64_t)row * a.gate_row];
  ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    float s[8];
    to_f32(rres[u], s);
    if (a.post_norm) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] *= r;
      if (a.w) {
        float w[8];
        to_f32(load_unit<VEC>(a.w, e, cols), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= w[i];
      }
    }
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = g1;
    if (a.gate && a.gate_col) {
      if (a.gate_type == MOE_TYPE_F32)
        to_f32(load_unit<VEC>((const float*)a.gate + (int64_t)row * a.gate_row, e, cols), g);
      else
        to_f32(load_unit<VEC>((const __bf16*)a.gate + (int64_t)row * a.gate_row, e, cols), g);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = fmaf(a.res_scale, s[i], g[i] * v[u][i]);
    store_unit<VEC>((RT*)a.out + (int64_t)row * a.ld_out, e, cols, v[u]);
    if (a.has_next) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[u][i] = e + i < cols ? stored<RT>(v[u][i]) : 0.f;
        ss = fmaf(v[u][i], v[u][i], ss);
      }
    }
  }
  if (!a.has_next) return;
  r = 1.0f / sqrtf(wg_sum(ss, slots[1]) / (float)cols + a.o.eps);
  finish_row<U, VEC>(v, row, cols, r, a.o, slots[2]);
}

// Row quantiser: the row's largest magnitude, then its codes; the second
// read comes from the caches.
template <typename XT>
__global__ __launch_bounds__(512) void quant_row_kernel(const XT* x0, int64_t ld_x, int cols, int8_t* q0, int64_t ld_q,
                                 float* scales, int vec) {
  __shared__ float slots[16];
  const int row = blockIdx.x;
  const XT* x = x0 + (int64_t)row * ld_x;
  int8_t* q = q0 + (int64_t)row * ld_q;
  float amax = 0.f, v[8];
  for (int e = 8 * (int)threadIdx.x; e < cols; e += 8 * (int)blockDim.x) {
    to_f32(vec ? load_unit<true>(x, e, cols) : load_unit<false>(x, e, cols), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  }
  const float d = wg_max(amax, slots) / 127.0f;
  for (int e = 8 * (int)threadIdx.x; e < cols; e += 8 * (int)blockDim.x) {
    to_f32(vec ? load_unit<true>(x, e, cols) : load_unit<false>(x, e, cols), v);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= ((uint32_t)(int32_t)q8_code(v[i], d) & 0xFFu) << (8 * (i & 3));
    if (e + 8 <= cols) {
      *(u32x2*)(q + e) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < cols) q[e + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
  if (threadIdx.x == 0) scales[row] = d;
}

// ------------------------------------------------------------- host side
int norm_args_check(const moe_norm_t* N) {
  if (!N) return MOE_ERR_INVALID_ARG;
  if (N->d_model < 1 || N->d_model > kMaxNormCols) return MOE_ERR_SHAPE;
  if (!(N->eps > 0.f) || !isfinite(N->eps) || !isfinite(N->residual_scale) ||
      (N->post_norm != 0 && N->post_norm != 1))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(N->pre_w, 4) || !aligned(N->post_w, 4)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

static int norm_out_check(int cols, const NormOut& o) {
  if (o.quant != MOE_QUANT_NONE && o.quant != MOE_QUANT_BLOCK && o.quant != MOE_QUANT_ROW)
    return MOE_ERR_INVALID_ARG;
  if (!o.h && o.quant == MOE_QUANT_NONE) return MOE_ERR_INVALID_ARG;
  if (o.h) {
    if (!type_ok(o.h_type)) return MOE_ERR_INVALID_ARG;
    if (o.ld_h < cols) return MOE_ERR_STRIDE;
    if (!aligned(o.h, type_size(o.h_type))) return MOE_ERR_ALIGNMENT;
  }
  if (o.quant != MOE_QUANT_NONE) {
    if (!o.q || !o.qs) return MOE_ERR_INVALID_ARG;
    if (o.quant == MOE_QUANT_BLOCK && cols % kBlock != 0) return MOE_ERR_SHAPE;
    if (o.ld_q < cols) return MOE_ERR_STRIDE;
    if (o.ld_qs < (o.quant == MOE_QUANT_BLOCK ? cols / kBlock : 1)) return MOE_ERR_STRIDE;
    if (!aligned(o.q, 8) || o.ld_q % 8 != 0 || !aligned(o.qs, 4)) return MOE_ERR_ALIGNMENT;
  }
  return MOE_OK;
}

// rows in 16-byte pieces of 8 (bf16) or 4 (f32) elements
static bool vec_rows(const void* p, int type, int64_t ld) {
  return aligned(p, 16) && ld % (type == MOE_TYPE_F32 ? 4 : 8) == 0;
}
static bool vec_out(const NormOut& o) {
  return (!o.h || vec_rows(o.h, o.h_type, o.ld_h)) && aligned(o.w, 16);
}

// Threads of a row and units of 8 elements per thread, by the row's length
// alone (so a row's bits do not depend on the call).
struct RowShape {
  int threads, units;
};
static RowShape row_shape(int cols) {
  const int n = (cols + 7) / 8;
  const int units = n <= 512 ? 1 : n <= 1024 ? 2 : 4;
  return {((n + units - 1) / units + 63) / 64 * 64, units};
}

template <typename XT>
static void launch_pre(const NormArgs& a, int rows, bool vec, hipStream_t s) {
  const RowShape r = row_shape(a.cols);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(rows), dim3(r.threads), 0, s, a);
  };
  if (vec) {
    if (r.units == 1) go(norm_pre_kernel<XT, 1, true>);
    else if (r.units == 2) go(norm_pre_kernel<XT, 2, true>);
    else go(norm_pre_kernel<XT, 4, true>);
  } else {
    if (r.units == 1) go(norm_pre_kernel<XT, 1, false>);
    else if (r.units == 2) go(norm_pre_kernel<XT, 2, false>);
    else go(norm_pre_kernel<XT, 4, false>);
  }
}

template <typename XT, typename RT>
static void launch_post(const NormArgs& a, int rows, bool vec, hipStream_t s) {
  const RowShape r = row_shape(a.cols);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(rows), dim3(r.threads), 0, s, a);
  };
  if (vec) {
    if (r.units == 1) go(norm_post_kernel<XT, RT, 1, true>);
    else if (r.units == 2) go(norm_post_kernel<XT, RT, 2, true>);
    else go(norm_post_kernel<XT, RT, 4, true>);
  } else {
    if (r.units == 1) go(norm_post_kernel<XT, RT, 1, false>);
    else if (r.units == 2) go(norm_post_kernel<XT, RT, 2, false>);
    else go(norm_post_kernel<XT, RT, 4, false>);
  }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_norm_pre(const moe_norm_t* N, const void* x, int x_type, int64_t ld_x,
                            int rows, void* h, int h_type, int64_t ld_h, int quant, int8_t* q,
                            int64_t ld_q, float* qs, int64_t ld_qs, void* stream) {
  int rc = norm_args_check(N);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(x_type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x) return MOE_ERR_INVALID_ARG;
  const int cols = N->d_model;
  if (ld_x < cols) return MOE_ERR_STRIDE;
  if (!aligned(x, type_size(x_type))) return MOE_ERR_ALIGNMENT;
  const NormOut o{h, h_type, ld_h, quant, q, ld_q, qs, ld_qs, N->pre_w, N->eps};
  rc = norm_out_check(cols, o);
  if (rc != MOE_OK) return rc;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  NormArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.cols = cols;
  a.o = o;
  const bool vec = cols % 8 == 0 && vec_rows(x, x_type, ld_x) && vec_out(o);
  hipStream_t s = (hipStream_t)stream;
  if (x_type == MOE_TYPE_F32) launch_pre<float>(a, rows, vec, s);
  else launch_pre<__bf16>(a, rows, vec, s);
  return launch_status();
}

extern "C" int moe_norm_post(const moe_norm_t* N, const void* y, int y_type, int64_t ld_y,
                             const void* res, int res_type, int64_t ld_res, const void* gate,
                             int gate_type, int64_t gate_row, int64_t gate_col, int rows,
                             void* out, int64_t ld_out, const moe_norm_t* next, void* h,
                             int h_type, int64_t ld_h, int quant, int8_t* q, int64_t ld_q,
                             float* qs, int64_t ld_qs, void* stream) {
  int rc = norm_args_check(N);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(y_type) || !type_ok(res_type)) return MOE_ERR_INVALID_ARG;
  if (next) {
    rc = norm_args_check(next);
    if (rc != MOE_OK) return rc;
    if (next->d_model != N->d_model) return MOE_ERR_SHAPE;
  }
  if (gate && (!type_ok(gate_type) || gate_row < 0 || gate_col < 0 || gate_col > 1))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!y || !res || !out) return MOE_ERR_INVALID_ARG;
  const int cols = N->d_model;
  if (ld_y < cols || ld_res < cols || ld_out < cols) return MOE_ERR_STRIDE;
  if (!aligned(y, type_size(y_type)) || !aligned(res, type_size(res_type)) ||
      !aligned(out, type_size(res_type)) || (gate && !aligned(gate, type_size(gate_type))))
    return MOE_ERR_ALIGNMENT;
  NormOut o{};
  if (next) {
    o = NormOut{h, h_type, ld_h, quant, q, ld_q, qs, ld_qs, next->pre_w, next->eps};
    rc = norm_out_check(cols, o);
    if (rc != MOE_OK) return rc;
  }
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  NormArgs a{y, ld_y, cols, N->post_norm, N->eps, N->residual_scale, N->post_w, res, ld_res,
             gate, gate_type, gate_row, gate_col, out, ld_out, next != nullptr, o};
  const bool vec = cols % 8 == 0 && vec_rows(y, y_type, ld_y) &&
                   vec_rows(res, res_type, ld_res) && vec_rows(out, res_type, ld_out) &&
                   (!gate || gate_col == 0 || vec_rows(gate, gate_type, gate_row)) &&
                   aligned(N->post_w, 16) && (!next || vec_out(o));
  hipStream_t s = (hipStream_t)stream;
  const bool yf = y_type == MOE_TYPE_F32, rf = res_type == MOE_TYPE_F32;
  if (yf && rf) launch_post<float, float>(a, rows, vec, s);
  else if (yf) launch_post<float, __bf16>(a, rows, vec, s);
  else if (rf) launch_post<__bf16, float>(a, rows, vec, s);
  else launch_post<__bf16, __bf16>(a, rows, vec, s);
  return launch_status();
}

extern "C" int moe_quant_row_q8(const void* x, int x_type, int64_t ld_x, int rows, int cols,
                                int8_t* q, int64_t ld_q, float* scales, void* stream) {
  if (rows < 0 || !type_ok(x_type)) return MOE_ERR_INVALID_ARG;
  if (cols < 1) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales) return MOE_ERR_INVALID_ARG;
  if (ld_x < cols || ld_q < cols) return MOE_ERR_STRIDE;
  if (!aligned(x, type_size(x_type)) || !aligned(q, 8) || ld_q % 8 != 0 || !aligned(scales, 4))
    return MOE_ERR_ALIGNMENT;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  const int threads = min(512, ((cols + 7) / 8 + 63) / 64 * 64);
  const int vec = cols % 8 == 0 && vec_rows(x, x_type, ld_x);
  hipStream_t s = (hipStream_t)stream;
  if (x_type == MOE_TYPE_F32)
    hipLaunchKernelGGL(quant_row_kernel<float>, dim3(rows), dim3(threads), 0, s, (const float*)x,
                       ld_x, cols, q, ld_q, scales, vec);
  else
    hipLaunchKernelGGL(quant_row_kernel<__bf16>, dim3(rows), dim3(threads), 0, s,
                       (const __bf16*)x, ld_x, cols, q, ld_q, scales, vec);
  return launch_status();
}
