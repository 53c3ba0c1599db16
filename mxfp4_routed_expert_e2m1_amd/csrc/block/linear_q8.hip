// linear_q8.hip -- dense projection of int8 codes with a scale per row and per
// channel: y[t][n] = qs[t] ws[n] sum_k q[t][k] w[n][k] (+ bias[n]).
//
// The contraction runs on the int8 matrix core (32x32x32, int32 sums): lane l
// supplies channel row l % 32 of A and token row l % 32 of B, each with the
// 16 codes of K slot l / 32, and receives token column l % 32 of D, element i
// at channel row 8 (i / 4) + 4 (l / 32) + i % 4.  |sum| <= 2^14 d_in < 2^31.
// The sums are exact, so tiles and splits of K change no bit.
//
// Two kernels: tiles through LDS (any rows), and a weight stream for up to 16
// rows; plan() below says which, from the sizes alone.
#include "block.h"

#include <type_traits>

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
  // split K: int32 sums of split i at parts + i * rows * parts_ld
  int32_t* parts;
  int64_t parts_ld;
};

__device__ inline i32x16 mfma_i8(i32x4 a, i32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// the 16 codes of columns k.. with those from d_in on made 0
__device__ inline i32x4 mask_codes(i32x4 v, int k, int d_in) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = d_in - (k + 4 * i);  // codes of this dword inside the row
    v[i] &= n >= 4 ? -1 : n <= 0 ? 0 : (int)((1u << (8 * n)) - 1);
  }
  return v;
}
// the epilogue's arithmetic, shared by every kernel (each operation rounded by
// itself: no fused multiply-add with the bias); without a bias, bias is -0,
// which changes no value
__device__ inline float linear_value(int sum, float qs, float ws, float bias) {
#pragma clang fp contract(off)
  return (float)sum * qs * ws + bias;
}
__device__ inline void linear_store(const LinearArgs& a, int t, int n, float v) {
  if (a.y_bf16) ((__bf16*)a.y)[(int64_t)t * a.ld_y + n] = (__bf16)v;
  else ((float*)a.y)[(int64_t)t * a.ld_y + n] = v;
}

// ------------------------------------------------------ tiles through LDS
// A workgroup of 4 waves, 2 x 2, computes 64 TT tokens x 64 TN channels, each
// wave 32 TT x 32 TN of them.  K goes in steps of STEP codes, copied from
// memory to LDS directly into a ring of four stages, three steps ahead, so that
// a step has to wait neither for memory nor for the copy unit (which takes 64
// bytes a cycle: the copies are spread evenly over the products).  The two
// larger tiles take steps of 64 codes (the ring of the largest fills the LDS),
// the others 128, for half the barriers (512 rows of 4096 x 4096: 16.5 -> 13.8
// us).  A row's P = STEP / 16 pieces sit in LDS at
// piece ^ (row / (16 / P) % P), so the 16 rows that a read takes at once lie in
// different banks; the copy takes the pieces from memory in that order, since
// it can only write LDS in lane order.
//
// Within a step, the matrix core works on the operands of one K slice of 32
// while the next slice's are read from LDS.
constexpr int kStages = 4;

template <int STEP>
__device__ inline int swizzle(int row) {
  return row / (256 / STEP) % (STEP / 16);
}

// Workgroup id -> tile.  Consecutive ids go to the 8 XCDs in turn; each XCD
// takes a contiguous run of an order that walks 8 token tiles, then the next
// channel tile, so the tiles that share an L2 at one time share their rows.
struct TilePlace {
  int t, n;
};
__device__ inline TilePlace place_tile(int id, int total, int tiles_t) {
  const int xcd = id & 7, per = total >> 3, extra = total & 7;
  const int i = xcd * per + min(xcd, extra) + (id >> 3);
  const int tiles_n = total / tiles_t;
  const int band = i / (8 * tiles_n), left = i - band * 8 * tiles_n;
  const int width = min(8, tiles_t - band * 8);
  return {band * 8 + left % width, left / width};
}

// The 16-byte piece that holds a row's last code is read whole, what lies past
// the code masked.
__device__ inline int piece_end(int d_in) { return (d_in + 15) & ~15; }

template <int ROWS, int STEP>
struct TileSource {
  static constexpr int kPieces = STEP / 16, kCopyRows = 64 / kPieces;
  static constexpr int kCopies = ROWS / (4 * kCopyRows);  // per wave
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off[kCopies];  // per lane: byte of this lane's piece in the tile's copy j

  // rows r0.. of a matrix of n rows of d_in codes, ld apart; rows past the
  // last repeat it (their products are not stored)
  __device__ inline void set(const int8_t* p, int64_t ld, int r0, int n, int d_in) {
    const int have = min(ROWS, n - r0);
    rsrc = buf_rsrc(p + uniform((int64_t)r0 * ld), (uint32_t)((have - 1) * ld + piece_end(d_in)));
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int row = (j * 4 + wave) * kCopyRows + lane / kPieces;
      off[j] = (uint32_t)min(row, have - 1) * (uint32_t)ld +
               16 * (lane % kPieces ^ swizzle<STEP>(row));
    }
  }
  // copy j of the step at column k (k a whole step inside every row)
  __device__ inline void copy(int j, int8_t* stage, int k) const { put(j, stage, off[j], k); }
  // the same where the step may reach past the rows: what is past the last
  // row's end reads as 0
  __device__ inline void copy_tail(int j, int8_t* stage, int k) const {
    put(j, stage, off[j] + k, 0);
  }

 private:
  __device__ inline void put(int j, int8_t* stage, uint32_t lane_off, int off0) const {
#ifdef __HIP_DEVICE_COMPILE__  // (the host pass does not know the 16-byte form)
    const int wave = uniform((int)threadIdx.x >> 6);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(stage + (j * 4 + wave) * 1024), 16,
                                             lane_off, off0, 0, 0);
#endif
  }
};

// Barrier after which every wave's copies but its newest N are in LDS and
// every wave's LDS reads are done.
template <int N>
__device__ inline void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4 << 14));  // vmcnt N, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A wave's 32 tokens x 32 TN channels of results, from the matrix core's lanes
// through LDS to rows: 4 channels at a time in, 16 bytes per lane out (at any
// address: the rows of y need their elements' alignment alone), and what is
// left of a row at the last channel one element at a time.
struct RowsOut {
  void* y;
  int64_t ld;
  int rows, cols;
};
typedef u32x4 any_u32x4 __attribute__((aligned(2)));

// STREAM: the two larger tiles, whose calls are the larger ones, write their
// results past the L2s, which leaves the operands there.  Without and with it, us:
//   rows x channels x codes   the call     with a norm of its results after it
//   2048 x 4096 x 4096        48.9, 47.4   69.3, 70.1
//   4096 x 4096 x 4096        73.0, 70.0   113.2, 110.6
//   4096 x 14336 x 4096       253, 240     419, 417
template <int TN, bool STREAM, typename T>
__device__ inline void store_rows(const RowsOut& o, i32x16 (&c)[TN], int t0, int n0, float qs,
                                  const float* ws, const float* bias, T* buf) {
  constexpr int kCols = 32 * TN, kLd = kCols + 16 / (int)sizeof(T), kPer = 16 / (int)sizeof(T);
  const int lane = lane_id(), half = lane >> 5;
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int n = 32 * i + 8 * g + 4 * half;
      T v[4];
      if constexpr (std::is_same_v<T, int32_t>) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c[i][4 * g + e];
      } else {
        const f32x4 w = *(const f32x4*)(ws + n), b = *(const f32x4*)(bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (T)linear_value(c[i][4 * g + e], qs, w[e], b[e]);
      }
      __builtin_memcpy(__builtin_assume_aligned(buf + (lane & 31) * kLd + n, 4 * sizeof(T)), v,
                       sizeof(v));
    }
  __builtin_amdgcn_wave_barrier();
  const int rows = min(32, o.rows - t0), cols = min(kCols, o.cols - n0);
  T* y = (T*)o.y + uniform((int64_t)t0 * o.ld + n0);
  constexpr int kLanes = kCols / kPer, kPasses = kLanes / 2;  // lanes per row
  auto store16 = [](T* p, u32x4 x) {
    if constexpr (STREAM) __builtin_nontemporal_store(x, (any_u32x4*)p);
    else *(any_u32x4*)p = x;
  };
  const int col = (lane % kLanes) * kPer, r0 = lane / kLanes;
  u32x4 v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    v[i] = *(const u32x4*)(buf + (r0 + i * (64 / kLanes)) * kLd + col);
  if (col + kPer <= cols) {
    T* p = y + (int64_t)r0 * o.ld + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (r0 + i * (64 / kLanes) < rows)
        store16(p + (int64_t)(i * (64 / kLanes)) * o.ld, v[i]);
  }
  if (cols % kPer && lane < rows) {
    for (int n = cols / kPer * kPer; n < cols; ++n)
      y[(int64_t)lane * o.ld + n] = buf[lane * kLd + n];
  }
  __builtin_amdgcn_wave_barrier();
}

template <int TT, int TN, int STEP>
__global__ __launch_bounds__(256) void linear_gemm_kernel(LinearArgs a, int tiles_t, int splits) {
  constexpr int BT = 64 * TT, BN = 64 * TN, kStage = (BT + BN) * STEP;
  // (an array per stage: the compiler then knows that a read waits for the
  // copies into its own stage alone)
  __shared__ __align__(1024) int8_t lds0[kStage], lds1[kStage], lds2[kStage], lds3[kStage];
  int8_t* const ring[kStages] = {lds0, lds1, lds2, lds3};
  __shared__ float row_scale[BT];
  __shared__ __align__(16) float channel_scale[BN], channel_bias[BN];
  static_assert(BT <= 256 && BN <= 256, "a thread per row and per channel");
  static_assert(kStage >= 32 * (32 * TN + 4) * 4, "a wave's results fit its share");
  const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
  const int wt = wave >> 1, wn = wave & 1;
  const int split = blockIdx.x % splits;
  const TilePlace at = place_tile(blockIdx.x / splits, gridDim.x / splits, tiles_t);
  const int t0 = at.t * BT, n0 = at.n * BN;
  TileSource<BT, STEP> xs;
  TileSource<BN, STEP> ws;
  xs.set(a.q, a.ld_q, t0, a.rows, a.d_in);
  ws.set(a.w, a.ld_w, n0, a.n_out, a.d_in);
  constexpr int kCopiesX = decltype(xs)::kCopies, kCopies = kCopiesX + decltype(ws)::kCopies;
  constexpr int kSlices = STEP / 32, kReads = TT + TN, kProducts = TT * TN;
  auto copy = [&](int j, int8_t* to, int k) {
    if (j < kCopiesX) xs.copy(j, to, k);
    else ws.copy(j - kCopiesX, to + BT * STEP, k);
  };
  // the epilogue's factors, loaded ahead of the copies
  const int lt = threadIdx.x % BT, ln = threadIdx.x % BN;
  const float my_row = a.qs[min(t0 + lt, a.rows - 1)];
  const float my_channel = a.ws[min(n0 + ln, a.n_out - 1)];
  const float my_bias = a.bias ? a.bias[min(n0 + ln, a.n_out - 1)] : -0.f;
  // past the last step it is copied again, unread, so that every step has as
  // many copies in flight
  const int steps_all = a.d_in / STEP, first = (int64_t)steps_all * split / splits;
  const int steps = (int64_t)steps_all * (split + 1) / splits - first;
  const int base = first * STEP, last = base + (steps - 1) * STEP;
  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy(j, ring[i], min(base + i * STEP, last));
  }
  // this lane's byte in a tile of 32 rows, by K slice (2 pieces: lane / 32)
  uint32_t rd[kSlices];
#pragma unroll
  for (int s = 0; s < kSlices; ++s)
    rd[s] = (lane & 31) * STEP + 16 * ((2 * s + (lane >> 5)) ^ swizzle<STEP>(lane & 31));
  i32x16 c[TN][TT];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) c[i][j] = i32x16{};
  i32x4 fw[2][TN], fx[2][TT];
#pragma unroll
  for (int i = 0; i < TN; ++i) fw[1][i] = i32x4{};
#pragma unroll
  for (int j = 0; j < TT; ++j) fx[1][j] = i32x4{};
  auto read = [&](const int8_t* stage, int s, int set) {
    const int8_t* x = stage + wt * 32 * TT * STEP + rd[s];
    const int8_t* w = stage + (BT + wn * 32 * TN) * STEP + rd[s];
#pragma unroll
    for (int i = 0; i < TN; ++i) fw[set][i] = *(const i32x4*)(w + i * 32 * STEP);
#pragma unroll
    for (int j = 0; j < TT; ++j) fx[set][j] = *(const i32x4*)(x + j * 32 * STEP);
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) c[i][j] = mfma_i8(fw[set][i], fx[set][j], c[i][j]);
  };

  auto step = [&](int k, const int8_t* stage, int8_t* to) {
    stage_barrier<(kStages - 2) * kCopies>();
    const int kn = min(base + (k + kStages - 1) * STEP, last);
    // the products of the slice before come first; a slice's reads and its share
    // of the step's copies are spread over them
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      const int c0 = s * kCopies / kSlices, c1 = (s + 1) * kCopies / kSlices;
      read(stage, s, s & 1);
#pragma unroll
      for (int j = c0; j < c1; ++j) copy(j, to, kn);
      multiply((s & 1) ^ 1);
      const int gaps = kReads + (c1 - c0);
#pragma unroll
      for (int i = 0; i < gaps; ++i) {
        if (i < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        else __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);             // copy
        if (i < kProducts) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < kProducts - gaps; ++i)
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  };
  int k = 0;
  for (; k + kStages <= steps; k += kStages) {
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      step(k + i, ring[i], ring[(i + kStages - 1) % kStages]);
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (k + i >= steps) break;
    step(k + i, ring[i], ring[(i + kStages - 1) % kStages]);
  }
  if (a.d_in % STEP && split == splits - 1) {
    // the partial step, into stage 0; masking one operand is enough
    stage_barrier<0>();
    const int k0 = steps_all * STEP;
#pragma unroll
    for (int j = 0; j < kCopiesX; ++j) xs.copy_tail(j, lds0, k0);
#pragma unroll
    for (int j = 0; j < kCopies - kCopiesX; ++j) ws.copy_tail(j, lds0 + BT * STEP, k0);
    stage_barrier<0>();
    multiply(1);
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      read(lds0, s, s & 1);
#pragma unroll
      for (int i = 0; i < TN; ++i)
        fw[s & 1][i] = mask_codes(fw[s & 1][i], k0 + 32 * s + 16 * (lane >> 5), a.d_in);
      if (s < kSlices - 1) multiply(s & 1);
    }
  }
  multiply(1);

  row_scale[lt] = my_row;  // (threads past BT or BN write what others write)
  channel_scale[ln] = my_channel;
  channel_bias[ln] = my_bias;
  // every wave is done with the stages (and the copies that nobody reads are in)
  stage_barrier<0>();
  int8_t* mine = wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = t0 + (wt * TT + j) * 32, n = n0 + wn * 32 * TN;
    if (t >= a.rows || n >= a.n_out) break;
    i32x16 cj[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) cj[i] = c[i][j];
    const float qs = row_scale[t - t0 + (lane & 31)];
    const float *cs = channel_scale + (n - n0), *cb = channel_bias + (n - n0);
    const RowsOut o{a.y, a.ld_y, a.rows, a.n_out};
    if (a.parts) {
      const RowsOut po{a.parts + split * (a.rows * a.parts_ld), a.parts_ld, a.rows,
                       (int)a.parts_ld};
      store_rows<TN, false>(po, cj, t, n, qs, cs, cb, (int32_t*)mine);
    } else if (a.y_bf16) {
      store_rows<TN, TT * TN >= 8>(o, cj, t, n, qs, cs, cb, (__bf16*)mine);
    } else {
      store_rows<TN, TT * TN >= 8>(o, cj, t, n, qs, cs, cb, (float*)mine);
    }
  }
}

// The splits' sums joined, 4 channels per thread.
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a, int splits) {
  const int n = 4 * (blockIdx.x * 256 + threadIdx.x), t = blockIdx.y;
  if (n >= a.n_out) return;
  const int32_t* p = a.parts + t * a.parts_ld + n;
  i32x4 v = *(const i32x4*)p;
  for (int i = 1; i < splits; ++i) v += *(const i32x4*)(p + i * (a.rows * a.parts_ld));
  const float qs = a.qs[t];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.n_out)
      linear_store(a, t, n + i, linear_value(v[i], qs, a.ws[n + i], a.bias ? a.bias[n + i] : -0.f));
}

// ------------------------------------------------- few tokens: weight stream
// Up to 16 tokens the weights are the traffic.  A workgroup of 4 waves takes
// 16 channels and all tokens; its waves split K and work alone, each with a
// ring of four stages of its own in LDS: 128 codes of every row, copied from
// memory three stages ahead, so a wave keeps 6 KiB of weights on their way and
// never waits for another (two workgroups share a CU; stages of 256 codes, one
// workgroup per CU, took 17.8 us instead of 12.9 for a row of 14336 x 4096).
// The products are 16x16x64: lane l supplies row l % 16 with the 16 codes of K
// slot l / 16 and receives token column l % 16, element i at channel row
// 4 (l / 16) + i.  Piece p of a row sits in LDS at p ^ (row / 2 & 7), so the 16
// rows of a read lie in different banks.  The waves' sums, exact in int32, meet
// in LDS at the end.  16 rows of 4096 x 14336 take 14.1 us with the weights from
// memory, 4.2 TB/s (one row 12.6); 11.4 us where they rotate over three sets, which
// the last-level cache can hold.
constexpr int kStreamWaves = 4, kStreamK = 128;

__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(LinearArgs a) {
  constexpr int kHalf = 16 * kStreamK, kStage = 2 * kHalf;  // a wave's: channels, tokens
  constexpr int kCopyRows = 8, kCopies = 16 / kCopyRows;    // rows of a copy, copies of 16 rows
  __shared__ __align__(1024) int8_t lds0[kStreamWaves * kStage], lds1[kStreamWaves * kStage],
      lds2[kStreamWaves * kStage], lds3[kStreamWaves * kStage];
  __shared__ i32x4 sums[kStreamWaves][64];
  int8_t* const ring[kStages] = {lds0, lds1, lds2, lds3};
  const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, r = lane & 15, slot = lane >> 4;
  const int have_n = min(16, a.n_out - n0);
  [[maybe_unused]] const auto ws = buf_rsrc(a.w + uniform((int64_t)n0 * a.ld_w),
                                            (uint32_t)((have_n - 1) * a.ld_w + piece_end(a.d_in)));
  [[maybe_unused]] const auto qs =
      buf_rsrc(a.q, (uint32_t)((a.rows - 1) * a.ld_q + piece_end(a.d_in)));
  // this wave's steps [s0, s1)
  const int steps = (a.d_in + kStreamK - 1) / kStreamK;
  const int s0 = wave * steps / kStreamWaves, s1 = (wave + 1) * steps / kStreamWaves;
  // per lane: byte of its piece in copy j; rows past the last repeat it (their
  // sums are not stored)
  uint32_t off_w[kCopies], off_q[kCopies];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int row = kCopyRows * j + (lane >> 3), piece = 16 * ((lane & 7) ^ ((row >> 1) & 7));
    off_w[j] = (uint32_t)min(row, have_n - 1) * (uint32_t)a.ld_w + piece;
    off_q[j] = (uint32_t)min(row, a.rows - 1) * (uint32_t)a.ld_q + piece;
  }
  // a step's copies; what is past the last row's end reads as 0
  auto copy = [&](int8_t* to, int s) {
#ifdef __HIP_DEVICE_COMPILE__  // (the host pass does not know the 16-byte form)
    const uint32_t k = (uint32_t)s * kStreamK;
    int8_t* mine = to + wave * kStage;
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ws, (lds_ptr)(mine + j * 1024), 16, off_w[j] + k, 0,
                                               0, 0);
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(qs, (lds_ptr)(mine + kHalf + j * 1024), 16,
                                               off_q[j] + k, 0, 0, 0);
#endif
  };
  i32x4 c = {0, 0, 0, 0};
  auto multiply = [&](const int8_t* stage, int s, bool masked) {
    const int8_t* mine = stage + wave * kStage + r * kStreamK;
#pragma unroll
    for (int h = 0; h < kStreamK / 64; ++h) {
      const int at = 16 * ((4 * h + slot) ^ ((r >> 1) & 7));
      i32x4 w = *(const i32x4*)(mine + at);
      const i32x4 x = *(const i32x4*)(mine + kHalf + at);
      if (masked) w = mask_codes(w, s * kStreamK + 64 * h + 16 * slot, a.d_in);
      c = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
    }
  };
  // copies step s + 3 into the stage that step s - 1 was read from, once those
  // reads are done, then waits for step s (past the wave's last step it is
  // copied again, unread)
  auto advance = [&](int s, int8_t* to) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0
    asm volatile("" ::: "memory");
    copy(to, min(s + kStages - 1, s1 - 1));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kStages - 1) * 2 * kCopies | 0xF70);  // vmcnt
    asm volatile("" ::: "memory");
  };
  if (s0 < s1) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(ring[i], min(s0 + i, s1 - 1));
    const int full = min(s1, a.d_in / kStreamK);
    int s = s0;
    for (; s + kStages <= full; s += kStages) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        advance(s + i, ring[(i + kStages - 1) % kStages]);
        multiply(ring[i], s + i, false);
      }
    }
    // the remaining steps, the partial one among them
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (s + i >= s1) break;
      advance(s + i, ring[(i + kStages - 1) % kStages]);
      multiply(ring[i], s + i, true);
    }
  }
  sums[wave][lane] = c;
  __syncthreads();
  if (wave > 0 || r >= a.rows) return;
  i32x4 v = sums[0][lane];
#pragma unroll
  for (int i = 1; i < kStreamWaves; ++i) v += sums[i][lane];
  const int n = n0 + 4 * slot;
  const float scale = a.qs[r];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.n_out)
      linear_store(a, r, n + i,
                   linear_value(v[i], scale, a.ws[n + i], a.bias ? a.bias[n + i] : -0.f));
}

// ------------------------------------------------------------- host side
constexpr int64_t kMaxLd = 1 << 22;  // 256 rows of any operand within 32-bit offsets
constexpr int kMaxRows = 0x7FFFFFFF - 255;  // the rows of the last tile have numbers too

static int linear_check(const moe_linear_t* L) {
  if (!L || !L->w || !L->w_scales) return MOE_ERR_INVALID_ARG;
  if (L->n_out < 1 || L->d_in < 1 || L->d_in > 65536) return MOE_ERR_SHAPE;
  if (L->ld_w < L->d_in || L->ld_w > kMaxLd) return MOE_ERR_STRIDE;
  if (!aligned(L->w, 16) || L->ld_w % 16 != 0 || !aligned(L->w_scales, 4) ||
      !aligned(L->bias, 4))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// The tile sizes, tokens x channels in units of 64, with what a K step of 64
// costs a tile alone and on a full chip, and a tile's start and end (us,
// measured; the smaller tiles share a CU, so theirs are per tile in turn).
struct Tile8 {
  int tt, tn;
  float alone_us, full_us, ends_us;
};
constexpr Tile8 kTiles[] = {{4, 4, 0.53f, 0.88f, 4.f},
                            {4, 2, 0.36f, 0.52f, 3.f},
                            {2, 2, 0.18f, 0.30f, 2.f},
                            {1, 2, 0.12f, 0.15f, 1.5f},
                            {1, 1, 0.08f, 0.085f, 1.2f}};
constexpr int kChipCus = 256;

// One launch: a tile size (-1: the weight stream), K splits, and the channels
// it takes from the first that is left.
struct LinearPart {
  int tile, splits, channels;
};
struct LinearPlan {
  LinearPart part[2];
  int n_parts;
};

static int ceil_div(int64_t a, int b) { return (int)((a + b - 1) / b); }

// Estimated time of `tiles` tiles of `steps` K steps each: full rounds over the
// chip, then the tiles that are left.  (It orders the tile sizes; it knows nothing
// of memory, so for few rows, where the weights' bytes take longer, it is less
// than what the call takes.)
static double rounds_us(const Tile8& t, int64_t tiles, double steps) {
  const double left = (double)(tiles % kChipCus) / kChipCus;
  const double full = (double)(tiles / kChipCus) * (steps * t.full_us + t.ends_us);
  return left == 0 ? full
                   : full + steps * (t.alone_us + left * (t.full_us - t.alone_us)) + t.ends_us;
}

// The tile and the number of K splits with the least estimated time for
// `channels` channels: rounds of tiles over the chip, plus, for splits, the
// launch that joins them and its traffic (48 rows of 4096 x 14336: 21.5 us in
// one, 14.9 in four; 512 rows of 4096 x 4096: 13.8 in one, 24.6 in two).
static LinearPart best_part(int rows, int channels, int d_in, int most_splits, double* us) {
  LinearPart best{0, 1, channels};
  *us = 1e30;
  const double steps = ceil_div(d_in, 64);
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile8& t = kTiles[i];
    const int64_t tiles = (int64_t)ceil_div(rows, 64 * t.tt) * ceil_div(channels, 64 * t.tn);
    for (int s = 1; s <= most_splits; s *= 2) {
      if (s > 1 && (steps / s < 8 || tiles * s > kChipCus)) break;
      double x = rounds_us(t, tiles * s, steps / s);
      if (s > 1) x += 4. + (double)s * rows * channels * 8 / 5e6;
      if (x < *us) {
        *us = x;
        best = {i, s, channels};
      }
    }
  }
  return best;
}

// Up to 16 rows the weight stream, unless there are channels enough for small
// tiles to fill the chip.  Stream and tiles, weights from memory, us:
//   channels x codes   1 row        16 rows
//   4096 x 4096        6.4, 11.2    6.9, 11.5
//   8192 x 4096        9.4, 13.5    9.9, 12.8
//   10240 x 4096       12.4, 14.0   13.4, 12.9
//   12288 x 4096       14.1, 14.5   14.7, 13.8
//   14336 x 4096       15.4, 15.2   16.9, 14.7
// The row's length moves the point where they meet, which the rule leaves out: at
// 1024 codes it is near 8192 channels (10240: 8.0, 5.8), at 14336 codes one row is
// faster in the stream at 12288 channels too (31.2, 35.8; 16 rows 37.1, 37.0).
// Otherwise the best tile; or, where its
// last round would leave much of the chip idle, whole rounds of it and a second
// launch with the best tile for the channels left.
constexpr int kStreamRows = 16;
static bool streams(int rows, int n_out) {
  return rows <= kStreamRows && ceil_div(n_out, 64) < 3 * kChipCus / 4;
}
static LinearPlan plan(int rows, int n_out, int d_in) {
  if (streams(rows, n_out)) return {{{-1, 1, n_out}, {}}, 1};
  double us;
  LinearPlan best{{best_part(rows, n_out, d_in, 8, &us), {}}, 1};
  for (int i = 0; i < 2; ++i) {  // (smaller tiles have short last rounds)
    const Tile8& t = kTiles[i];
    const int tiles_t = ceil_div(rows, 64 * t.tt);
    const int64_t tiles = (int64_t)tiles_t * ceil_div(n_out, 64 * t.tn);
    const int rounds = (int)(tiles / kChipCus);
    const int64_t main = (int64_t)rounds * kChipCus / tiles_t * 64 * t.tn;
    if (rounds == 0 || main == 0 || main >= n_out) continue;
    double rest_us;
    const LinearPart rest = best_part(rows, (int)(n_out - main), d_in, 1, &rest_us);
    const double x = 2. + rest_us + rounds_us(t, (int64_t)rounds * kChipCus, ceil_div(d_in, 64));
    if (x < us) {
      us = x;
      best = {{{i, 1, (int)main}, rest}, 2};
    }
  }
  return best;
}

static int64_t part_tiles(const LinearPart& p, int rows) {
  const Tile8& t = kTiles[p.tile];
  return (int64_t)ceil_div(rows, 64 * t.tt) * ceil_div(p.channels, 64 * t.tn);
}

static int64_t parts_ld(int n_out) { return (n_out + 3) / 4 * 4; }

// Workspace of a plan (a second launch has no splits).
static size_t plan_bytes(const LinearPlan& p, int rows) {
  const LinearPart& f = p.part[0];
  return f.splits > 1 ? (size_t)f.splits * rows * parts_ld(f.channels) * sizeof(int32_t) : 0;
}

// The most workspace that a call of up to `rows` rows needs.  Within 64 rows
// whose tiles are the same in number, only the cost of joining the splits grows
// with the rows, so the first of them has the most splits; past the rows whose
// largest tiles fill half the chip there are none.
static size_t most_bytes(int rows, int n_out, int d_in) {
  const Tile8& t = kTiles[0];
  const int64_t end = (int64_t)64 * t.tt * (kChipCus / 2 / ceil_div(n_out, 64 * t.tn));
  size_t most = 0;
  for (int r = 0; r < rows && r < end; r += 64) {
    const int first = r == 0 && streams(1, n_out) ? kStreamRows + 1 : r + 1;
    if (first > rows) break;
    most = max(most, plan_bytes(plan(first, n_out, d_in), min(rows, r + 64)));
  }
  return most;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_q8_workspace_bytes(const moe_linear_t* L, int rows) {
  if (linear_check(L) != MOE_OK || rows < 1) return 0;
  return most_bytes(rows, L->n_out, L->d_in);
}

extern "C" int moe_linear_q8(const moe_linear_t* L, const int8_t* q, int64_t ld_q,
                             const float* qs, int rows, void* y, int y_type, int64_t ld_y,
                             void* ws, size_t ws_bytes, void* stream) {
  const int rc = linear_check(L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(y_type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (rows > kMaxRows) return MOE_ERR_SHAPE;
  if (!q || !qs || !y) return MOE_ERR_INVALID_ARG;
  if (ld_q < L->d_in || ld_y < L->n_out || ld_q > kMaxLd || ld_y > kMaxLd) return MOE_ERR_STRIDE;
  if (!aligned(q, 16) || ld_q % 16 != 0 || !aligned(qs, 4) || !aligned(y, type_size(y_type)))
    return MOE_ERR_ALIGNMENT;
  const LinearPlan p = plan(rows, L->n_out, L->d_in);
  for (int i = 0; i < p.n_parts; ++i)  // (a launch takes fewer than 2^32 threads)
    if (p.part[i].tile >= 0 && part_tiles(p.part[i], rows) >= 1 << 24) return MOE_ERR_SHAPE;
  const size_t need = plan_bytes(p, rows);
  if (need > 0) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  }
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  hipStream_t s = (hipStream_t)stream;
  const int bf16 = y_type == MOE_TYPE_BF16;
  int first = 0;  // channel
  for (int i = 0; i < p.n_parts; ++i) {
    const LinearPart& part = p.part[i];
    const LinearArgs a{L->w + first * L->ld_w, L->ld_w, L->w_scales + first,
                       L->bias ? L->bias + first : nullptr, q, ld_q, qs, rows, part.channels,
                       L->d_in, (char*)y + first * type_size(y_type), bf16, ld_y,
                       part.splits > 1 ? (int32_t*)ws : nullptr, parts_ld(part.channels)};
    first += part.channels;
    if (part.tile < 0) {
      hipLaunchKernelGGL(linear_stream_kernel, dim3(ceil_div(part.channels, 16)),
                         dim3(64 * kStreamWaves), 0, s, a);
      continue;
    }
    const int tiles_t = ceil_div(rows, 64 * kTiles[part.tile].tt);
    const int tiles = (int)part_tiles(part, rows);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * part.splits)), dim3(256), 0, s, a,
                         tiles_t, part.splits);
    };
    switch (part.tile) {
      case 0: go(linear_gemm_kernel<4, 4, 64>); break;
      case 1: go(linear_gemm_kernel<4, 2, 64>); break;
      case 2: go(linear_gemm_kernel<2, 2, 128>); break;
      case 3: go(linear_gemm_kernel<1, 2, 128>); break;
      default: go(linear_gemm_kernel<1, 1, 128>); break;
    }
    if (part.splits > 1)
      hipLaunchKernelGGL(linear_join_kernel, dim3(ceil_div(part.channels, 1024), rows), dim3(256),
                         0, s, a, part.splits);
  }
  return launch_status();
}
