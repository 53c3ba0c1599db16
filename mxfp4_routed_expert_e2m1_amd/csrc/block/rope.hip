// rope.hip -- rotary positions with one or several axes.
//
// Angles.  A position times a frequency in fp32 is wrong by whole radians at far positions (2^20
// positions leave 2^-4).  Here a frequency is turns per position in 64-bit fixed point, so the
// product of two whole numbers modulo 2^64 is the angle's fraction of a turn, exact but for the
// frequency's own rounding; its two top bits (rounded) are the quadrant, the rest an angle within
// +-pi/4, where Taylor's series to x^9 (sine) and x^10 (cosine) are off by 2e-9 and 1e-10.
//
// Bound by memory: each element is read and written once, 16 bytes a lane (4096 rows of 40 heads of
// 128, bf16: 17.0 us, 4.9 TB/s; through the L2s 20.8); a row or some hundreds by the chain position ->
// sine -> row (4.0 and 6.5 us).  A thread holds the
// sines and cosines of 8 pairs and takes several heads with them where there are rows enough to
// fill the chip without splitting heads.
#include "block.h"
#include "kv_cache.h"

namespace moe {

__device__ inline void sincos_turns(uint64_t phase, float& s, float& c) {
  const uint64_t q = phase + ((uint64_t)1 << 61);  // quadrant in the top two bits
  const int32_t r = (int32_t)((int64_t)(phase - (q & ((uint64_t)3 << 62))) >> 30);
  const float x = (float)r * 3.657295198e-10f;  // 2 pi 2^-34
  const float z = x * x;
  float ps = 2.7557319e-6f;  // 1/9!, -1/7!, 1/5!, -1/3!
  ps = fmaf(ps, z, -1.9841270e-4f);
  ps = fmaf(ps, z, 8.3333333e-3f);
  ps = fmaf(ps, z, -1.6666667e-1f);
  const float sn = fmaf(x * z, ps, x);
  float pc = -2.7557319e-7f;  // -1/10!, 1/8!, -1/6!, 1/4!, -1/2!
  pc = fmaf(pc, z, 2.4801587e-5f);
  pc = fmaf(pc, z, -1.3888889e-3f);
  pc = fmaf(pc, z, 4.1666667e-2f);
  pc = fmaf(pc, z, -0.5f);
  const float cs = fmaf(z, pc, 1.f);
  const uint32_t k = (uint32_t)(q >> 62);
  s = (k & 1) ? cs : sn;
  c = (k & 1) ? sn : cs;
  if (k & 2) s = -s;
  if (k == 1 || k == 2) c = -c;
}

template <typename T>
__device__ inline void load_some(const T* p, int n, float (&v)[8]) {
  if (n == 8) {
    const Raw8<T> r = load8(p);
    to_f32<T>(r, v);
  } else {
    const Raw8<T> r = load8_part(p, n);
    to_f32<T>(r, v);
  }
}
template <typename T, bool PAST>
__device__ inline void store_some(T* p, int n, const float (&v)[8]) {
  if (n == 8) {
    store8<T, PAST>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (T)v[i];
  }
}

// A thread's chunk: 8 pairs (the last chunk of a head fewer), or, from `pair_chunks` on, 8
// channels to copy.  Chunks of a (row, group of `hpt` heads) lie side by side, in a power of two of
// threads.
template <typename T, bool INTERLEAVED, bool PAST>
__global__ __launch_bounds__(256) void rope_kernel(
    const T* __restrict__ x, int64_t ld_x, int64_t hs_x, int rows, int n_heads, int dim, int half,
    int pair_chunks, int chunks, int chunk_log, int hpt, int groups, const int32_t* __restrict__ pos,
    int64_t ld_pos, const uint64_t* __restrict__ steps, const uint8_t* __restrict__ axes,
    int n_axes, float scale, T* __restrict__ out, int64_t ld_out, int64_t hs_out) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rg = t >> chunk_log;
  const int c = (int)(t - (rg << chunk_log));
  const int64_t row = groups == 1 ? rg : (int64_t)((uint32_t)rg / (uint32_t)groups);
  if (row >= rows || c >= chunks) return;
  const int h0 = (int)(rg - row * groups) * hpt;
  const int h1 = h0 + hpt < n_heads ? h0 + hpt : n_heads;
  x += row * ld_x;
  out += row * ld_out;
  if (c >= pair_chunks) {
    const int at = 2 * half + 8 * (c - pair_chunks);
    const int n = dim - at < 8 ? dim - at : 8;
    for (int h = h0; h < h1; ++h) {
      float v[8];
      load_some<T>(x + h * hs_x + at, n, v);
      store_some<T, PAST>(out + h * hs_out + at, n, v);
    }
    return;
  }
  const int i0 = 8 * c, n = half - i0 < 8 ? half - i0 : 8;
  // everything that the angles are made of in one round of loads: positions of up to 4 axes, of
  // which each pair takes its own
  uint64_t step[8];
  uint8_t axis[8] = {};
  if (n == 8) {
    __builtin_memcpy(step, steps + i0, sizeof(step));
    if (axes) __builtin_memcpy(axis, axes + i0, sizeof(axis));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      step[i] = i < n ? steps[i0 + i] : 0;
      axis[i] = axes && i < n ? axes[i0 + i] : 0;
    }
  }
  int32_t at[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) at[k] = pos[(k < n_axes ? k : 0) * ld_pos + row];
  float sn[8], cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = axis[i];
    int64_t p = k == 1 ? at[1] : k == 2 ? at[2] : k == 3 ? at[3] : at[0];
    if (k > 3 && k < n_axes) p = pos[k * ld_pos + row];
    sincos_turns((uint64_t)p * step[i], sn[i], cs[i]);
    sn[i] *= scale;
    cs[i] *= scale;
  }
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    const T* xp = x + h * hs_x;
    T* op = out + h * hs_out;
    float a[8], b[8], u[8], w[8];
    if constexpr (INTERLEAVED) {
      // (2i, 2i+1): 16 channels in a row
      const int n0 = 2 * n < 8 ? 2 * n : 8, n1 = 2 * n - n0;
      float e[8], f[8] = {};
      load_some<T>(xp + 2 * i0, n0, e);
      if (n1) load_some<T>(xp + 2 * i0 + 8, n1, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = e[2 * i];
        b[i] = e[2 * i + 1];
        a[4 + i] = f[2 * i];
        b[4 + i] = f[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = a[i] * cs[i] - b[i] * sn[i];
        w[i] = b[i] * cs[i] + a[i] * sn[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[2 * i] = u[i];
        e[2 * i + 1] = w[i];
        f[2 * i] = u[4 + i];
        f[2 * i + 1] = w[4 + i];
      }
      store_some<T, PAST>(op + 2 * i0, n0, e);
      if (n1) store_some<T, PAST>(op + 2 * i0 + 8, n1, f);
    } else {
      load_some<T>(xp + i0, n, a);
      load_some<T>(xp + half + i0, n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = a[i] * cs[i] - b[i] * sn[i];
        w[i] = b[i] * cs[i] + a[i] * sn[i];
      }
      store_some<T, PAST>(op + i0, n, u);
      store_some<T, PAST>(op + half + i0, n, w);
    }
  }
}

// How a call's threads lie.
struct RopePlan {
  int pair_chunks, chunks, chunk_log, hpt, groups;
  int64_t threads;
};
static RopePlan rope_plan(const moe_rope_t* R, int rows, int n_heads, int dim, bool in_place) {
  RopePlan p;
  p.pair_chunks = (R->rot_dim / 2 + 7) / 8;
  p.chunks = p.pair_chunks + (in_place ? 0 : (dim - R->rot_dim + 7) / 8);
  // a head per thread until there are two workgroups for each CU, then up to 8 (4096 rows of 40 heads
  // of 128, bf16: 17.0 us; 4 heads 18.1, 2 heads 28.5)
  const int64_t hpt = (int64_t)rows * n_heads * p.chunks / (256 * 512);
  p.hpt = hpt < 1 ? 1 : hpt > 8 ? 8 : (int)hpt;
  p.groups = (n_heads + p.hpt - 1) / p.hpt;
  p.chunk_log = 0;
  while ((1 << p.chunk_log) < p.chunks) ++p.chunk_log;
  p.threads = ((int64_t)rows * p.groups) << p.chunk_log;
  return p;
}

template <typename T>
static void rope_launch(const moe_rope_t* R, const RopePlan& p, const void* x, int64_t ld_x,
                        int64_t hs_x, int rows, int n_heads, int dim, const int32_t* pos,
                        int64_t ld_pos, void* out, int64_t ld_out, int64_t hs_out,
                        hipStream_t stream) {
  const dim3 grid((unsigned)((p.threads + 255) / 256));
  // (results of a call that fills the chip leave past the L2s)
  const bool past = p.hpt > 1;
  auto k = R->interleaved ? (past ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                          : (past ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
  hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, (const T*)x, ld_x, hs_x, rows, n_heads, dim,
                     R->rot_dim / 2, p.pair_chunks, p.chunks, p.chunk_log, p.hpt, p.groups, pos,
                     ld_pos, R->steps, R->axes, R->n_axes, R->scale, (T*)out, ld_out, hs_out);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_rope(const moe_rope_t* R, const void* x, int x_type, int64_t ld_x, int64_t hs_x,
                        int rows, int n_heads, int head_dim, const int32_t* pos, int64_t ld_pos,
                        void* out, int64_t ld_out, int64_t hs_out, void* stream) {
  if (!R || rows < 0 || n_heads < 0) return MOE_ERR_INVALID_ARG;
  if (R->rot_dim < 2 || R->rot_dim % 2 || head_dim < R->rot_dim || head_dim > 1024 ||
      R->n_axes < 1 || R->n_axes > 8)
    return MOE_ERR_SHAPE;
  if ((R->interleaved != 0 && R->interleaved != 1) || !__builtin_isfinite(R->scale) ||
      !type_ok(x_type))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0 || n_heads == 0) return MOE_OK;
  if (!R->steps || !x || !pos || !out) return MOE_ERR_INVALID_ARG;
  if (!head_strides_ok(ld_x, hs_x, rows, n_heads, head_dim) ||
      !head_strides_ok(ld_out, hs_out, rows, n_heads, head_dim) ||
      (R->n_axes > 1 && ld_pos < rows))
    return MOE_ERR_STRIDE;
  if (x == out && ((rows > 1 && ld_x != ld_out) || (n_heads > 1 && hs_x != hs_out)))
    return MOE_ERR_INVALID_ARG;
  const size_t size = type_size(x_type);
  if (!aligned(x, size) || !aligned(out, size) || !aligned(pos, 4) || !aligned(R->steps, 8))
    return MOE_ERR_ALIGNMENT;
  // (rows' groups of heads and the threads of a launch)
  if ((int64_t)rows * n_heads >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
  const RopePlan p = rope_plan(R, rows, n_heads, head_dim, x == out);
  if (p.threads > 0xFFFFFF00) return MOE_ERR_SHAPE;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (x_type == MOE_TYPE_F32)
    rope_launch<float>(R, p, x, ld_x, hs_x, rows, n_heads, head_dim, pos, ld_pos, out, ld_out, hs_out,
                       (hipStream_t)stream);
  else
    rope_launch<__bf16>(R, p, x, ld_x, hs_x, rows, n_heads, head_dim, pos, ld_pos, out, ld_out,
                        hs_out, (hipStream_t)stream);
  return launch_status();
}
