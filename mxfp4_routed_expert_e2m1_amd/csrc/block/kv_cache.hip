// kv_cache.hip -- keys and values into the pages of the 4-bit cache, and back.
//
// A thread takes 8 channels of a token's head (16 or 32 bytes of a row, 4 bytes of codes), four
// threads a block of 32: its largest magnitude is a maximum over the quad in registers.  The
// scale is a power of two, so dividing by it is exact and the only rounding is the converter's,
// to the nearest E2M1 value with ties to the even code.  Both kernels are bound by the rows in
// memory, 32 times the scales and 4 to 8 times the codes; V's order (kv_cache.h) puts a token's
// codes at 4-byte pieces, which meet in L2 with those of the 3 tokens beside it.
#include "kv_cache.h"

namespace moe {

// Where 8 channels (octet o) of a token lie in a piece: K in one run, V in pieces of NB bytes.
template <int D>
__device__ inline int v_codes_at(int t, int o) {
  constexpr int NB = D / 32;
  const int m = 8 * o / (2 * NB);  // run of D/16 channels
  const int within = (8 * o - 2 * NB * m) / 2;
  return ((t >> 2) * 16 + m) * 4 * NB + (t & 3) * NB + within;
}

template <int D>
__device__ inline void store_v(uint8_t* codes, int t, int o, uint32_t w) {
  if constexpr (D == 64) {  // two runs of 4 channels
    *(uint16_t*)(codes + v_codes_at<D>(t, o)) = (uint16_t)w;
    *(uint16_t*)(codes + v_codes_at<D>(t, o) + 8) = (uint16_t)(w >> 16);
  } else {
    *(uint32_t*)(codes + v_codes_at<D>(t, o)) = w;
  }
}
template <int D>
__device__ inline uint32_t load_v(const uint8_t* codes, int t, int o) {
  if constexpr (D == 64) {
    const uint32_t lo = *(const uint16_t*)(codes + v_codes_at<D>(t, o));
    return lo | (uint32_t) * (const uint16_t*)(codes + v_codes_at<D>(t, o) + 8) << 16;
  } else {
    return *(const uint32_t*)(codes + v_codes_at<D>(t, o));
  }
}

struct KvPlace {
  int64_t row;
  int head, octet, v;  // v: 0 keys, 1 values
};
// Threads run over the octets of a head, then heads, then keys and values, then rows.
template <int D>
__device__ inline KvPlace kv_place(int64_t t, int n_heads) {
  KvPlace p;
  p.octet = (int)(t % (D / 8));
  t /= D / 8;
  p.head = (int)(t % n_heads);
  t /= n_heads;
  p.v = (int)(t & 1);
  p.row = t >> 1;
  return p;
}

template <typename T, int D>
__global__ __launch_bounds__(256) void kv_write_kernel(uint8_t* __restrict__ data, int page_log,
                                                       int n_pages, int n_heads,
                                                       const T* __restrict__ k, int64_t ld_k,
                                                       int64_t hs_k, const T* __restrict__ v,
                                                       int64_t ld_v, int64_t hs_v, int64_t threads,
                                                       const int32_t* __restrict__ slots) {
  constexpr int NB = D / 32;
  // (whole quads of lanes are past the end or not: D/8 is a multiple of 4)
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= threads) return;
  const KvPlace p = kv_place<D>(t, n_heads);
  const int slot = slots[p.row];
  const T* src = p.v ? v + p.row * ld_v + p.head * hs_v : k + p.row * ld_k + p.head * hs_k;
  const Raw8<T> raw = load8(src + 8 * p.octet);
  const int pg = slot >> page_log;
  if (slot < 0 || pg >= n_pages) return;
  float x[8];
  to_f32<T>(raw, x);
  // the largest magnitude as bits (which order as magnitudes do, infinities and NaN on top)
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    most = b > most ? b : most;
  }
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0xB1, 0xF, 0xF, false);
  most = o > most ? o : most;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0x4E, 0xF, 0xF, false);
  most = o > most ? o : most;
  int u = (int)((most + 0x200000u) >> 23) - 2;
  u = u < 2 ? 2 : u > (int)kMaxScaleByte ? (int)kMaxScaleByte : u;
  const float scale = __uint_as_float((uint32_t)u << 23);
  uint32_t w = 0;
  if (most >= 0x7F800000u) {
    u = 255;
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  }
  const KvUnit<D> unit{1 << page_log};
  uint8_t* at = data + ((int64_t)pg * n_heads + p.head) * unit.bytes();
  const int tok = slot & ((1 << page_log) - 1), block = p.octet >> 2;
  if (p.v) {
    store_v<D>(at + unit.v_codes(), tok, p.octet, w);
    if ((p.octet & 3) == 0) at[unit.v_scales() + ((tok >> 2) * NB + block) * 4 + (tok & 3)] = (uint8_t)u;
  } else {
    *(uint32_t*)(at + tok * (D / 2) + 4 * p.octet) = w;
    if ((p.octet & 3) == 0) at[unit.k_scales() + tok * NB + block] = (uint8_t)u;
  }
}

template <typename T, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(const uint8_t* __restrict__ data,
                                                      int page_log, int n_pages, int n_heads,
                                                      T* __restrict__ k, int64_t ld_k, int64_t hs_k,
                                                      T* __restrict__ v, int64_t ld_v, int64_t hs_v,
                                                      int64_t threads,
                                                      const int32_t* __restrict__ slots) {
  constexpr int NB = D / 32;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= threads) return;
  const KvPlace p = kv_place<D>(t, n_heads);
  const int slot = slots[p.row];
  const int pg = slot >> page_log;
  uint32_t w = 0, u = 127;
  if (slot >= 0 && pg < n_pages) {
    const KvUnit<D> unit{1 << page_log};
    const uint8_t* at = data + ((int64_t)pg * n_heads + p.head) * unit.bytes();
    const int tok = slot & ((1 << page_log) - 1), block = p.octet >> 2;
    if (p.v) {
      w = load_v<D>(at + unit.v_codes(), tok, p.octet);
      u = at[unit.v_scales() + ((tok >> 2) * NB + block) * 4 + (tok & 3)];
    } else {
      w = *(const uint32_t*)(at + tok * (D / 2) + 4 * p.octet);
      u = at[unit.k_scales() + tok * NB + block];
    }
  }
  const bool nan = u > kMaxScaleByte;
  const float scale = __uint_as_float((nan ? 127u : u) << 23);
  float x[8];
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  x[0] = x0[0], x[1] = x0[1], x[2] = x1[0], x[3] = x1[1];
  x[4] = x2[0], x[5] = x2[1], x[6] = x3[0], x[7] = x3[1];
  T y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (T)(nan ? __builtin_nanf("") : x[i]);
  T* dst = p.v ? v + p.row * ld_v + p.head * hs_v : k + p.row * ld_k + p.head * hs_k;
  __builtin_memcpy(dst + 8 * p.octet, y, sizeof(y));
}

static int log2_of(int page) { return __builtin_ctz((unsigned)page); }

// Rows and strides of a call (MOE_OK with rows == 0 before pointers are looked at).
static int kv_rows_check(const moe_kv_cache_t* C, const void* k, int64_t ld_k, int64_t hs_k,
                         const void* v, int64_t ld_v, int64_t hs_v, int type, int rows,
                         const int32_t* slots) {
  if (!k || !v || !slots) return MOE_ERR_INVALID_ARG;
  if (!head_strides_ok(ld_k, hs_k, rows, C->n_heads, C->head_dim) ||
      !head_strides_ok(ld_v, hs_v, rows, C->n_heads, C->head_dim))
    return MOE_ERR_STRIDE;
  const size_t size = type_size(type);
  if (!aligned(k, size) || !aligned(v, size) || !aligned(slots, 4)) return MOE_ERR_ALIGNMENT;
  // (workgroups of a launch)
  if ((int64_t)rows * C->n_heads > ((int64_t)1 << 40) / C->head_dim) return MOE_ERR_SHAPE;
  return MOE_OK;
}

template <typename T>
static void kv_write_launch(const moe_kv_cache_t* C, const void* k, int64_t ld_k, int64_t hs_k,
                            const void* v, int64_t ld_v, int64_t hs_v, int rows,
                            const int32_t* slots, hipStream_t stream) {
  const int64_t threads = (int64_t)rows * 2 * C->n_heads * (C->head_dim / 8);
  auto kernel = C->head_dim == 64    ? kv_write_kernel<T, 64>
                : C->head_dim == 128 ? kv_write_kernel<T, 128>
                                     : kv_write_kernel<T, 256>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream,
                     (uint8_t*)C->data, log2_of(C->page), C->n_pages, C->n_heads, (const T*)k,
                     ld_k, hs_k, (const T*)v, ld_v, hs_v, threads, slots);
}

template <typename T>
static void kv_read_launch(const moe_kv_cache_t* C, const int32_t* slots, int rows, void* k,
                           int64_t ld_k, int64_t hs_k, void* v, int64_t ld_v, int64_t hs_v,
                           hipStream_t stream) {
  const int64_t threads = (int64_t)rows * 2 * C->n_heads * (C->head_dim / 8);
  auto kernel = C->head_dim == 64    ? kv_read_kernel<T, 64>
                : C->head_dim == 128 ? kv_read_kernel<T, 128>
                                     : kv_read_kernel<T, 256>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream,
                     (const uint8_t*)C->data, log2_of(C->page), C->n_pages, C->n_heads, (T*)k,
                     ld_k, hs_k, (T*)v, ld_v, hs_v, threads, slots);
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_cache_bytes(const moe_kv_cache_t* C) {
  if (!C || !kv_sizes_ok(C)) return 0;
  return (size_t)C->n_pages * C->n_heads * C->page * (C->head_dim + C->head_dim / 16);
}

extern "C" int moe_kv_write(const moe_kv_cache_t* C, const void* k, int64_t ld_k, int64_t hs_k,
                            const void* v, int64_t ld_v, int64_t hs_v, int type, int rows,
                            const int32_t* slots, void* stream) {
  const int rc = kv_cache_check(C);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int rr = kv_rows_check(C, k, ld_k, hs_k, v, ld_v, hs_v, type, rows, slots);
  if (rr != MOE_OK) return rr;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (type == MOE_TYPE_F32)
    kv_write_launch<float>(C, k, ld_k, hs_k, v, ld_v, hs_v, rows, slots, (hipStream_t)stream);
  else
    kv_write_launch<__bf16>(C, k, ld_k, hs_k, v, ld_v, hs_v, rows, slots, (hipStream_t)stream);
  return launch_status();
}

extern "C" int moe_kv_read(const moe_kv_cache_t* C, const int32_t* slots, int rows, void* k,
                           int64_t ld_k, int64_t hs_k, void* v, int64_t ld_v, int64_t hs_v,
                           int type, void* stream) {
  const int rc = kv_cache_check(C);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int rr = kv_rows_check(C, k, ld_k, hs_k, v, ld_v, hs_v, type, rows, slots);
  if (rr != MOE_OK) return rr;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (type == MOE_TYPE_F32)
    kv_read_launch<float>(C, slots, rows, k, ld_k, hs_k, v, ld_v, hs_v, (hipStream_t)stream);
  else
    kv_read_launch<__bf16>(C, slots, rows, k, ld_k, hs_k, v, ld_v, hs_v, (hipStream_t)stream);
  return launch_status();
}
