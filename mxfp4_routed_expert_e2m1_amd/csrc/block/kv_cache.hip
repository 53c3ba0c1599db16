// kv_cache.hip -- keys and values into the pages of the 4-bit cache, and back.
//
// A thread takes 8 channels of a token's head (16 or 32 bytes of a row, 4 bytes of codes), four
// threads a block of 32, whose largest magnitude is a maximum over the quad in registers.  The
// scale is a power of two, so dividing by it is exact and the only rounding is the converter's,
// to the nearest E2M1 value with ties to the even code.  Both kernels are bound by the rows in
// memory (8 heads of 128, bf16: 4096 rows written 7.1 us, read 6.2; 65536 read 55 us, 6.1 TB/s, past
// the L2s; 16 rows 2.8), 32 times the scales and 4 to 8 times the codes; V's order (kv_cache.h)
// puts a token's codes at 4-byte pieces, which meet in L2 with those of the 3 tokens beside it.
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

// A workgroup's rows and channels: a row has 2 * n_heads * D/8 octets, keys before values; as many
// threads, to the next power of two (at most the workgroup's 256, which then take several octets
// each), do ROWS rows of it, all of whose loads are on their way before the first is used.
struct KvGrid {
  int row_log;  // threads of a row
  int octets;   // of a row
};

template <typename T, int D, int ROWS>
__global__ __launch_bounds__(256) void kv_write_kernel(uint8_t* __restrict__ data, int page_log,
                                                       int n_pages, int n_heads,
                                                       const T* __restrict__ k, int64_t ld_k,
                                                       int64_t hs_k, const T* __restrict__ v,
                                                       int64_t ld_v, int64_t hs_v, int rows,
                                                       const int32_t* __restrict__ slots,
                                                       KvGrid grid) {
  constexpr int NB = D / 32;
  const KvUnit<D> unit{1 << page_log};
  const int row0 = (blockIdx.x * (256 >> grid.row_log) + (threadIdx.x >> grid.row_log)) * ROWS;
  // (whole quads of lanes are past the end or not: D/8 is a multiple of 4)
  for (int u = threadIdx.x & ((1 << grid.row_log) - 1); u < grid.octets; u += 256) {
    const bool is_v = 2 * u >= grid.octets;
    const int w = is_v ? u - grid.octets / 2 : u;
    const int head = w / (D / 8), octet = w % (D / 8);
    const T* src = (is_v ? v + head * hs_v : k + head * hs_k) + 8 * octet;
    const int64_t ld = is_v ? ld_v : ld_k;
    int slot[ROWS];
    Raw8<T> raw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int row = row0 + r < rows ? row0 + r : rows - 1;
      slot[r] = row0 + r < rows ? slots[row] : -1;
      raw[r] = load8(src + row * ld);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float x[8];
      to_f32<T>(raw[r], x);
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
      int ub = (int)((most + 0x200000u) >> 23) - 2;
      ub = ub < 2 ? 2 : ub > (int)kMaxScaleByte ? (int)kMaxScaleByte : ub;
      const float scale = __uint_as_float((uint32_t)ub << 23);
      uint32_t c = 0;
      if (most >= 0x7F800000u) {
        ub = 255;
      } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], scale, 3);
      }
      const int pg = slot[r] >> page_log;
      if (slot[r] < 0 || pg >= n_pages) continue;
      uint8_t* at = data + ((int64_t)pg * n_heads + head) * unit.bytes();
      const int tok = slot[r] & ((1 << page_log) - 1), block = octet >> 2;
      if (is_v) {
        store_v<D>(at + unit.v_codes(), tok, octet, c);
        if ((octet & 3) == 0)
          at[unit.v_scales() + ((tok >> 2) * NB + block) * 4 + (tok & 3)] = (uint8_t)ub;
      } else {
        *(uint32_t*)(at + tok * (D / 2) + 4 * octet) = c;
        if ((octet & 3) == 0) at[unit.k_scales() + tok * NB + block] = (uint8_t)ub;
      }
    }
  }
}

template <typename T, int D, int ROWS>
__global__ __launch_bounds__(256) void kv_read_kernel(const uint8_t* __restrict__ data,
                                                      int page_log, int n_pages, int n_heads,
                                                      T* __restrict__ k, int64_t ld_k, int64_t hs_k,
                                                      T* __restrict__ v, int64_t ld_v, int64_t hs_v,
                                                      int rows, const int32_t* __restrict__ slots,
                                                      KvGrid grid) {
  constexpr int NB = D / 32;
  const KvUnit<D> unit{1 << page_log};
  const int row0 = (blockIdx.x * (256 >> grid.row_log) + (threadIdx.x >> grid.row_log)) * ROWS;
  for (int u = threadIdx.x & ((1 << grid.row_log) - 1); u < grid.octets; u += 256) {
    const bool is_v = 2 * u >= grid.octets;
    const int w = is_v ? u - grid.octets / 2 : u;
    const int head = w / (D / 8), octet = w % (D / 8);
    uint32_t code[ROWS], scale[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int slot = row0 + r < rows ? slots[row0 + r] : -1;
      const int pg = slot >> page_log;
      code[r] = 0;
      scale[r] = 127;
      if (slot >= 0 && pg < n_pages) {
        const uint8_t* at = data + ((int64_t)pg * n_heads + head) * unit.bytes();
        const int tok = slot & ((1 << page_log) - 1), block = octet >> 2;
        if (is_v) {
          code[r] = load_v<D>(at + unit.v_codes(), tok, octet);
          scale[r] = at[unit.v_scales() + ((tok >> 2) * NB + block) * 4 + (tok & 3)];
        } else {
          code[r] = *(const uint32_t*)(at + tok * (D / 2) + 4 * octet);
          scale[r] = at[unit.k_scales() + tok * NB + block];
        }
      }
    }
    T* dst = (is_v ? v + head * hs_v : k + head * hs_k) + 8 * octet;
    const int64_t ld = is_v ? ld_v : ld_k;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (row0 + r >= rows) break;
      // (a byte of 255, and nothing else that a write leaves, makes the converter's scale NaN)
      const float s = __uint_as_float((scale[r] > kMaxScaleByte ? 255u : scale[r]) << 23);
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[r], s, 0);
      const f32x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[r], s, 1);
      const f32x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[r], s, 2);
      const f32x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[r], s, 3);
      const float x[8] = {x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
      store8<T, (ROWS > 1)>(dst + (row0 + r) * ld, x);
    }
  }
}

// Four rows a thread once that leaves two workgroups for each CU; what such a call reads leaves past
// the L2s (65536 rows of 8 heads of 128 to bf16: 56 us, through them 89, a row a thread 107; 4096
// rows: 4.1, 5.1, 6.0).
constexpr int kManyRows = 4;
static bool many_rows(const KvGrid& g, int rows) {
  return (int64_t)(rows / kManyRows) >= (int64_t)512 * (256 >> g.row_log);
}
static KvGrid kv_grid(const moe_kv_cache_t* C) {
  KvGrid g;
  g.octets = 2 * C->n_heads * (C->head_dim / 8);
  g.row_log = 0;
  while ((1 << g.row_log) < g.octets && g.row_log < 8) ++g.row_log;
  return g;
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
  // (a launch has fewer than 2^32 threads; they take 4 rows of 8 channels of k or v, and at most as
  // many again are idle)
  if ((int64_t)rows * C->n_heads * C->head_dim >= ((int64_t)1 << 35)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

template <typename T, int D>
static void kv_write_launch(const moe_kv_cache_t* C, const void* k, int64_t ld_k, int64_t hs_k,
                            const void* v, int64_t ld_v, int64_t hs_v, int rows,
                            const int32_t* slots, hipStream_t stream) {
  const KvGrid g = kv_grid(C);
  const bool many = many_rows(g, rows);
  const int per = (256 >> g.row_log) * (many ? kManyRows : 1);
  auto kernel = many ? kv_write_kernel<T, D, kManyRows> : kv_write_kernel<T, D, 1>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + (int64_t)per - 1) / per)), dim3(256), 0, stream,
                     (uint8_t*)C->data, log2_of(C->page), C->n_pages, C->n_heads, (const T*)k, ld_k,
                     hs_k, (const T*)v, ld_v, hs_v, rows, slots, g);
}

template <typename T, int D>
static void kv_read_launch(const moe_kv_cache_t* C, const int32_t* slots, int rows, void* k,
                           int64_t ld_k, int64_t hs_k, void* v, int64_t ld_v, int64_t hs_v,
                           hipStream_t stream) {
  const KvGrid g = kv_grid(C);
  const bool many = many_rows(g, rows);
  const int per = (256 >> g.row_log) * (many ? kManyRows : 1);
  auto kernel = many ? kv_read_kernel<T, D, kManyRows> : kv_read_kernel<T, D, 1>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + (int64_t)per - 1) / per)), dim3(256), 0, stream,
                     (const uint8_t*)C->data, log2_of(C->page), C->n_pages, C->n_heads, (T*)k, ld_k,
                     hs_k, (T*)v, ld_v, hs_v, rows, slots, g);
}

template <typename T>
static void kv_write_dim(const moe_kv_cache_t* C, const void* k, int64_t ld_k, int64_t hs_k,
                         const void* v, int64_t ld_v, int64_t hs_v, int rows, const int32_t* slots,
                         hipStream_t stream) {
  auto go = C->head_dim == 64    ? kv_write_launch<T, 64>
            : C->head_dim == 128 ? kv_write_launch<T, 128>
                                 : kv_write_launch<T, 256>;
  go(C, k, ld_k, hs_k, v, ld_v, hs_v, rows, slots, stream);
}

template <typename T>
static void kv_read_dim(const moe_kv_cache_t* C, const int32_t* slots, int rows, void* k,
                        int64_t ld_k, int64_t hs_k, void* v, int64_t ld_v, int64_t hs_v,
                        hipStream_t stream) {
  auto go = C->head_dim == 64    ? kv_read_launch<T, 64>
            : C->head_dim == 128 ? kv_read_launch<T, 128>
                                 : kv_read_launch<T, 256>;
  go(C, slots, rows, k, ld_k, hs_k, v, ld_v, hs_v, stream);
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
  if (rows > 0x7FFFFFFF - 2048) return MOE_ERR_SHAPE;  // (row numbers of a launch)
  const int rr = kv_rows_check(C, k, ld_k, hs_k, v, ld_v, hs_v, type, rows, slots);
  if (rr != MOE_OK) return rr;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (type == MOE_TYPE_F32)
    kv_write_dim<float>(C, k, ld_k, hs_k, v, ld_v, hs_v, rows, slots, (hipStream_t)stream);
  else
    kv_write_dim<__bf16>(C, k, ld_k, hs_k, v, ld_v, hs_v, rows, slots, (hipStream_t)stream);
  return launch_status();
}

extern "C" int moe_kv_read(const moe_kv_cache_t* C, const int32_t* slots, int rows, void* k,
                           int64_t ld_k, int64_t hs_k, void* v, int64_t ld_v, int64_t hs_v,
                           int type, void* stream) {
  const int rc = kv_cache_check(C);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (rows > 0x7FFFFFFF - 2048) return MOE_ERR_SHAPE;  // (row numbers of a launch)
  const int rr = kv_rows_check(C, k, ld_k, hs_k, v, ld_v, hs_v, type, rows, slots);
  if (rr != MOE_OK) return rr;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (type == MOE_TYPE_F32)
    kv_read_dim<float>(C, slots, rows, k, ld_k, hs_k, v, ld_v, hs_v, (hipStream_t)stream);
  else
    kv_read_dim<__bf16>(C, slots, rows, k, ld_k, hs_k, v, ld_v, hs_v, (hipStream_t)stream);
  return launch_status();
}
