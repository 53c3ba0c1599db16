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
// Few rows are bound by a launch and one memory round trip (one row of 4096 f32
// before a block: 2.0 us of GPU time; 16 f32 rows after a block, a gate per
// channel, with the next norm: 3.9 us), many by memory (4096 rows of 4096, y f32,
// residual and next norm bf16, a gate per token: 34 us, 4.9 TB/s, a large copy's
// rate; 26.6 us where the rows are in the last-level cache).  Codes cost a
// reduction more and their bytes: with the next norm, all f32, 16 rows take 4.1
// us without codes, 4.9 with a scale per row, 4.6 with one per 32 elements; 4096
// rows from memory 52.8, 59.0 and 59.2 us (268, 285 and 287 MB).
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
  int row0;       // of the launch
  const void* x;  // the rows to normalise: x before a block, y after one
  int64_t ld_x;
  int cols;
  double inv_cols;
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

// Sum over the workgroup of up to 16 waves, in every lane; `slots` is LDS of one
// value per wave, not shared with another reduction of the same row.  A
// thread's and a 16-lane row's part are added in fp32, whose errors average
// out over the row's many parts; the last additions, whose errors would stay,
// in fp64.
__device__ inline double wg_sum(float v, double* slots) {
  v += dpp_mov<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp_mov<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp_mov<0x141>(v);  // row_half_mirror
  v += dpp_mov<0x140>(v);  // row_mirror
  auto lane_value = [&](int l) {
    return (double)__builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
  };
  double s = (lane_value(0) + lane_value(16)) + (lane_value(32) + lane_value(48));
  const int waves = blockDim.x >> 6, lane = lane_id();
  if (waves == 1) return s;
  if (lane == 0) slots[threadIdx.x >> 6] = s;
  __syncthreads();
  s = (lane & 15) < waves ? slots[lane & 15] : 0.;
  s += dpp_f64<0xB1>(s);
  s += dpp_f64<0x4E>(s);
  s += dpp_f64<0x141>(s);
  return s + dpp_f64<0x140>(s);
}
// Largest magnitude of the workgroup, likewise, from the bits of |v|: their
// order is that of the numbers, with a NaN above them all, so a row that holds
// one has a NaN scale (a floating-point maximum would drop it).
__device__ inline uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
template <int CTRL>
__device__ inline uint32_t max_moved(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false));
}
__device__ inline float wg_max(uint32_t v, uint32_t* slots) {
  v = wave_max_u32(v);
  const int waves = blockDim.x >> 6, lane = lane_id();
  if (waves > 1) {
    if (lane == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lane & 15) < waves ? slots[lane & 15] : 0u;
    v = max_moved<0x140>(max_moved<0x141>(max_moved<0x4E>(max_moved<0xB1>(v))));
  }
  return __uint_as_float(v);
}

// WHOLE: the row is a whole number of units.  (e and cols are up to 2^31 - 1 in
// the row quantiser, so e + 8 is not formed.)
template <bool WHOLE, typename T>
__device__ inline Raw8<T> load_unit(const T* row, int e, int cols) {
  if (cols - e >= 8) return load8(row + e);
  if (!WHOLE && e < cols) return load8_part(row + e, cols - e);
  return Raw8<T>{};
}

template <bool WHOLE, typename T>
__device__ inline void store_unit(T* row, int e, int cols, const float (&v)[8]) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (T)v[i];
  if (e + 8 <= cols) {
    __builtin_memcpy(row + e, t, sizeof(t));
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < cols) row[e + i] = t[i];
  }
}

// a x + b y, each operation rounded by itself
__device__ inline float scaled_sum(float a, float x, float b, float y) {
#pragma clang fp contract(off)
  return a * x + b * y;
}

// 1 / rms of a row from the sum of its squares (the hardware's root, one step
// of the last place)
__device__ inline float inverse_rms(double ss, double inv_cols, float eps) {
  return rsqrtf((float)(ss * inv_cols) + eps);
}

// the value an element keeps once it is stored in T
template <typename T>
__device__ inline float stored(float v) {
  return (float)(T)v;
}

// The codes of 8 values for a row's scale d, little-endian: rint(v / d) within
// +-127, 0 for d = 0.  The quotient by way of the reciprocal is off by less
// than 127 * 3 * 2^-24 < 2^-15, so it rounds to the same code unless it lies
// within 2^-12 of a midpoint; a wave that holds such a value (or a scale whose
// reciprocal is not safe) divides.  4096 rows of 4096 bf16 in the last-level
// cache: 14.8 -> 12.9 us.
__device__ inline u32x2 row_codes(const float (&v)[8], float d) {
  const float inv = 1.0f / d;
  const bool safe = d > 0x1p-100f && d < 0x1p100f;
  float q[8];
  bool near = !safe;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[i] * inv;
    q[i] = rintf(t);
    near |= fabsf(t - q[i]) > 0.5f - 0x1p-12f;
  }
  if (__any(near)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = q8_code(v[i], d);
  }
  u32x2 w = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= ((uint32_t)(int32_t)q[i] & 0xFFu) << (8 * (i & 3));
  return w;
}

// One row's h = v * r * w from its values in registers, with its codes.
template <int U, bool WHOLE>
__device__ inline void finish_row(float (&v)[U][8], const Raw8<float> (&rw)[U], int row, int cols,
                                  float r, const NormOut& o, uint32_t* slots) {
  const int threads = blockDim.x;
  const bool h_bf16 = o.h != nullptr && o.h_type == MOE_TYPE_BF16;
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    float w[8];
    to_f32(rw[u], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = o.w ? v[u][i] * r * w[i] : v[u][i] * r;
    if (h_bf16) {
      store_unit<WHOLE>((__bf16*)o.h + (int64_t)row * o.ld_h, e, cols, v[u]);
      if (o.quant) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = stored<__bf16>(v[u][i]);
      }
    } else if (o.h) {
      store_unit<WHOLE>((float*)o.h + (int64_t)row * o.ld_h, e, cols, v[u]);
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
        if (e + i < cols) amax = max(amax, magnitude(v[u][i]));
    }
  }
  if (o.quant == MOE_QUANT_ROW) {
    const float d = wg_max(amax, slots) / 127.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = 8 * (u * threads + (int)threadIdx.x);
      if (e >= cols) continue;
      int8_t* q = o.q + (int64_t)row * o.ld_q + e;
      const u32x2 w = row_codes(v[u], d);
      if (e + 8 <= cols) {
        *(u32x2*)q = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < cols) q[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
    }
    if (threadIdx.x == 0) o.qs[(int64_t)row * o.ld_qs] = d;
  }
}

// Every load of a row goes out before the first reduction: a row's time is one
// memory round trip and two reductions, not one round trip per operand.
template <typename XT, int U, bool WHOLE>
__global__ __launch_bounds__(1024) void norm_pre_kernel(NormArgs a) {
  __shared__ double sums[16];
  __shared__ uint32_t slots[16];
  const int row = a.row0 + (int)blockIdx.x, cols = a.cols;
  const XT* x = (const XT*)a.x + (int64_t)row * a.ld_x;
  Raw8<XT> raw[U];
  Raw8<float> rw[U] = {};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * (int)blockDim.x + (int)threadIdx.x);
    raw[u] = load_unit<WHOLE>(x, e, cols);
    if (a.o.w) rw[u] = load_unit<WHOLE>(a.o.w, e, cols);
  }
  float v[U][8], ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    to_f32(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
  }
  const float r = inverse_rms(wg_sum(ss, sums), a.inv_cols, a.o.eps);
  finish_row<U, WHOLE>(v, rw, row, cols, r, a.o, slots);
}

template <typename XT, typename RT, int U, bool WHOLE>
__global__ __launch_bounds__(1024) void norm_post_kernel(NormArgs a) {
  __shared__ double sums[2][16];
  __shared__ uint32_t slots[16];
  const int row = a.row0 + (int)blockIdx.x, cols = a.cols, threads = blockDim.x;
  const XT* x = (const XT*)a.x + (int64_t)row * a.ld_x;
  const RT* res = (const RT*)a.res + (int64_t)row * a.ld_res;
  const bool wide = a.gate && a.gate_col;  // a gate for each element
  const bool gate_f32 = a.gate_type == MOE_TYPE_F32;
  const int64_t g0 = (int64_t)row * a.gate_row;
  Raw8<XT> raw[U];
  Raw8<RT> rres[U];
  Raw8<float> rw[U] = {}, rg[U] = {}, rn[U] = {};
  Raw8<__bf16> rh[U] = {};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    raw[u] = load_unit<WHOLE>(x, e, cols);
    rres[u] = load_unit<WHOLE>(res, e, cols);
    if (a.post_norm && a.w) rw[u] = load_unit<WHOLE>(a.w, e, cols);
    if (wide) {
      if (gate_f32) rg[u] = load_unit<WHOLE>((const float*)a.gate + g0, e, cols);
      else rh[u] = load_unit<WHOLE>((const __bf16*)a.gate + g0, e, cols);
    }
    if (a.has_next && a.o.w) rn[u] = load_unit<WHOLE>(a.o.w, e, cols);
  }
  float g1 = 1.f;  // a gate that is one number for the row
  if (a.gate && !wide)
    g1 = gate_f32 ? ((const float*)a.gate)[g0] : (float)((const __bf16*)a.gate)[g0];
  float v[U][8], ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    to_f32(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
  }
  float r = 1.f;
  if (a.post_norm) r = inverse_rms(wg_sum(ss, sums[0]), a.inv_cols, a.eps);
  ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    float s[8], w[8], g[8], gh[8];
    to_f32(rres[u], s);
    to_f32(rw[u], w);
    to_f32(rg[u], g);
    to_f32(rh[u], gh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.post_norm) v[u][i] = a.w ? v[u][i] * r * w[i] : v[u][i] * r;
      const float gi = !wide ? g1 : gate_f32 ? g[i] : gh[i];
      v[u][i] = scaled_sum(a.res_scale, s[i], gi, v[u][i]);
    }
    store_unit<WHOLE>((RT*)a.out + (int64_t)row * a.ld_out, e, cols, v[u]);
    if (a.has_next) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[u][i] = e + i < cols ? stored<RT>(v[u][i]) : 0.f;
        ss = fmaf(v[u][i], v[u][i], ss);
      }
    }
  }
  if (!a.has_next) return;
  r = inverse_rms(wg_sum(ss, sums[1]), a.inv_cols, a.o.eps);
  finish_row<U, WHOLE>(v, rn, row, cols, r, a.o, slots);
}

// Row quantiser: a row of up to 8 kThreads U elements is held in registers;
// what is longer is read again, from the caches.
constexpr int kQuantThreads = 512, kQuantUnits = 4;

template <typename XT, bool WHOLE>
__global__ __launch_bounds__(kQuantThreads) void quant_row_kernel(const XT* x0, int64_t ld_x,
                                                                  int cols, int8_t* q0,
                                                                  int64_t ld_q, float* scales) {
  __shared__ uint32_t slots[16];
  const int row = blockIdx.x, threads = blockDim.x, stride = 8 * threads;
  const XT* x = x0 + (int64_t)row * ld_x;
  int8_t* q = q0 + (int64_t)row * ld_q;
  Raw8<XT> raw[kQuantUnits];
  uint32_t amax = 0;
  float v[8];
#pragma unroll
  for (int u = 0; u < kQuantUnits; ++u)
    raw[u] = load_unit<WHOLE>(x, 8 * (u * threads + (int)threadIdx.x), cols);
#pragma unroll
  for (int u = 0; u < kQuantUnits; ++u) {
    to_f32(raw[u], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(v[i]));
  }
  // (unsigned: the step past the end of the longest row is past 2^31 - 1)
  for (uint32_t e = kQuantUnits * stride + 8 * threadIdx.x; e < (uint32_t)cols; e += stride) {
    to_f32(load_unit<WHOLE>(x, (int)e, cols), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(v[i]));
  }
  const float d = wg_max(amax, slots) / 127.0f;
  auto write = [&](int e) {
    const u32x2 w = row_codes(v, d);
    if (cols - e >= 8) {
      *(u32x2*)(q + e) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cols - e) q[e + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  };
#pragma unroll
  for (int u = 0; u < kQuantUnits; ++u) {
    const int e = 8 * (u * threads + (int)threadIdx.x);
    if (e >= cols) break;
    to_f32(raw[u], v);
    write(e);
  }
  for (uint32_t e = kQuantUnits * stride + 8 * threadIdx.x; e < (uint32_t)cols; e += stride) {
    to_f32(load_unit<WHOLE>(x, (int)e, cols), v);
    write((int)e);
  }
  if (threadIdx.x == 0) scales[row] = d;
}

// ------------------------------------------------------------- host side
static int norm_args_check(const moe_norm_t* N) {
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

// A launch takes fewer than 2^32 threads: more rows go in several.
constexpr int kLaunchRows = 1 << 21;

// Threads of a row and units of 8 elements per thread, by the row's length
// alone (so a row's bits do not depend on the call).
struct RowShape {
  int threads, units;
};
static RowShape row_shape(int cols) {
  const int n = (cols + 7) / 8, units = n <= 1024 ? 1 : 2;
  return {((n + units - 1) / units + 63) / 64 * 64, units};
}

template <typename XT>
static void launch_pre(NormArgs a, int rows, hipStream_t s) {
  const RowShape r = row_shape(a.cols);
  auto go = [&](auto kernel) {
    for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
      a.row0 = (int)r0;
      hipLaunchKernelGGL(kernel, dim3(min(kLaunchRows, rows - a.row0)), dim3(r.threads), 0, s, a);
    }
  };
  if (a.cols % 8 == 0) {
    if (r.units == 1) go(norm_pre_kernel<XT, 1, true>);
    else go(norm_pre_kernel<XT, 2, true>);
  } else {
    if (r.units == 1) go(norm_pre_kernel<XT, 1, false>);
    else go(norm_pre_kernel<XT, 2, false>);
  }
}

template <typename XT, typename RT>
static void launch_post(NormArgs a, int rows, hipStream_t s) {
  const RowShape r = row_shape(a.cols);
  auto go = [&](auto kernel) {
    for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
      a.row0 = (int)r0;
      hipLaunchKernelGGL(kernel, dim3(min(kLaunchRows, rows - a.row0)), dim3(r.threads), 0, s, a);
    }
  };
  if (a.cols % 8 == 0) {
    if (r.units == 1) go(norm_post_kernel<XT, RT, 1, true>);
    else go(norm_post_kernel<XT, RT, 2, true>);
  } else {
    if (r.units == 1) go(norm_post_kernel<XT, RT, 1, false>);
    else go(norm_post_kernel<XT, RT, 2, false>);
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
  a.inv_cols = 1.0 / cols;
  a.o = o;
  hipStream_t s = (hipStream_t)stream;
  if (x_type == MOE_TYPE_F32) launch_pre<float>(a, rows, s);
  else launch_pre<__bf16>(a, rows, s);
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
  NormArgs a{0, y, ld_y, cols, 1.0 / cols, N->post_norm, N->eps, N->residual_scale, N->post_w,
             res, ld_res, gate, gate_type, gate_row, gate_col, out, ld_out, next != nullptr, o};
  hipStream_t s = (hipStream_t)stream;
  const bool yf = y_type == MOE_TYPE_F32, rf = res_type == MOE_TYPE_F32;
  if (yf && rf) launch_post<float, float>(a, rows, s);
  else if (yf) launch_post<float, __bf16>(a, rows, s);
  else if (rf) launch_post<__bf16, float>(a, rows, s);
  else launch_post<__bf16, __bf16>(a, rows, s);
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
  const int n = (int)(((int64_t)cols + 7) / 8);
  // (two units per thread keep more loads on their way: 4096 rows of 4096 bf16
  // in the last-level cache 15.7 -> 12.9 us; from memory it is 15.1)
  const int threads = min(kQuantThreads, ((n + 1) / 2 + 63) / 64 * 64);
  hipStream_t s = (hipStream_t)stream;
  auto go = [&](auto kernel, auto* p) {
    for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows)
      hipLaunchKernelGGL(kernel, dim3((unsigned)min((int64_t)kLaunchRows, rows - r0)),
                         dim3(threads), 0, s, p + r0 * ld_x, ld_x, cols, q + r0 * ld_q, ld_q,
                         scales + r0);
  };
  if (x_type == MOE_TYPE_F32) {
    if (cols % 8 == 0) go(quant_row_kernel<float, true>, (const float*)x);
    else go(quant_row_kernel<float, false>, (const float*)x);
  } else {
    if (cols % 8 == 0) go(quant_row_kernel<__bf16, true>, (const __bf16*)x);
    else go(quant_row_kernel<__bf16, false>, (const __bf16*)x);
  }
  return launch_status();
}
