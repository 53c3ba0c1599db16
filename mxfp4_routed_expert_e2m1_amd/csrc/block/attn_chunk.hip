// attn_chunk.hip -- attention of many rows of a sequence over the 4-bit cache, bf16.
//
// A workgroup has 32 rows a wave, in 32 x 32 tiles of the matrix core; the tokens pass 16 a wave
// at a time, in two buffers with one barrier.  The pass is attn.hip's, in other operands:
//   scores: the keys' codes and scale bytes go to the scaled instruction as they lie in the cache,
//     without conversion (32 x 32 x 64: a lane's 32 channels are one block).  The other operand is
//     q in two E4M3 planes with a scale for 32 channels: q rounded to 4 significant bits, and the
//     rest, which is exact in 4 more, so the planes hold all 8 bits of a bf16 number (and drop what
//     lies 2^-22 below the block's largest).  The planes cost what one bf16 product would.  Codes and
//     scale bytes are copied to LDS in the order of the operands' lanes, while the stage before is
//     worked on.
//   out: a thread turns 4 tokens' codes of D/16 channels into bf16 once for the workgroup, through
//     LDS, in the order in which the lanes read them as operands.  The reads take half of LDS's
//     rate, where the keys the same way would fill it.
// A row's base of the exponential is raised when its maximum has grown by 2^8 (or is the first):
// weights of up to 2^8 are as exact as those up to 1, and the accumulators are rarely rescaled.  Bound by
// the matrix core at the clock that the power limit leaves: 4096 new rows over 8192 tokens, 32 query
// heads on 8 of 128, take 351 us, 1170 TF/s, what a large library product reaches.  Chunks with heads of
// 64 are bound by their exponentials, short prompts by the chain before the first product.  (To do
// without the maximum as long as the weights' sum stays small was slower, 477 us: the sum has to be
// known before the products.)  The sum that divides is that of the rounded weights.
#include "attn.h"

namespace moe {

__device__ __forceinline__ float max2(float v) {  // over lanes l and l ^ 32
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum2(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// S += K Q^T for 32 tokens, 32 rows, 64 channels; byte J of `scales` is the lane's block's.
template <int J>
__device__ __forceinline__ f32x16 scores_32(v8i32 k, v8i32 q, f32x16 s, uint32_t scales, int e) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q, s, 4, 0, J, (int)scales, 0, e);
}

// HALVES: two waves for the same 32 rows, each with 64 of a stage's 128 tokens, joined in LDS at the
// end: for tiles that leave CUs idle, where a stage's time is its chain of steps and not its work.
template <int D, int WAVES, bool HALVES>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void attn_chunk_kernel(const AttnArgs a) {
  constexpr int ROW_WAVES = HALVES ? WAVES / 2 : WAVES;
  constexpr int NB = D / 32, NI = NB / 2, NC = D / 16, RB = 32 / NC;
  constexpr int STAGE = 16 * WAVES;  // tokens between barriers: a quad of them for each 16 threads
  constexpr int BUF = STAGE * D * 2;
  constexpr int KSCALES = STAGE * NB < 256 ? 256 : STAGE * NB;
  typedef uint32_t VRaw __attribute__((ext_vector_type(NB)));
  constexpr int LD = 33;  // floats of a row in the rows' way out
  constexpr int OUT = WAVES * 32 * LD * 4;
  __shared__ __attribute__((aligned(16))) uint8_t vbuf[2 * BUF > OUT ? 2 * BUF : OUT];
  // (an array for each of the two stages, so that reads of one wait for no copies into the other)
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf0[STAGE * D / 2], kbuf1[STAGE * D / 2];
  __shared__ __attribute__((aligned(1024))) uint8_t kscale0[KSCALES], kscale1[KSCALES];
  __shared__ uint32_t over[2][WAVES];

  const int wave = uniform((int)(threadIdx.x >> 6)), lane = lane_id();
  const int rw = HALVES ? wave % ROW_WAVES : wave;  // rows 32 rw ..
  const int q32 = lane & 31, h = lane >> 5;
  const int item = block_item(), kvh = blockIdx.x;

  int cut;
  Found f;
  __shared__ FoundShared found;
  if (!find_item(a, item, f, cut, wave, found)) return;
  const Seq& sq = f.seq;
  const int local = item - f.first_item;
  // the last rows first: they see the most tokens
  const int up = f.pieces == 1 ? local : local / f.pieces, piece = local - up * f.pieces;
  const int tile = sq.tiles(a) - 1 - up;
  const int rows_here = sq.m * a.group;
  const int tile0 = tile << a.tile_log, row0 = tile0 + 32 * rw;
  const RowSplit rs(a, tile0);

  // this lane's row, and what it sees
  const int r = row0 + q32;
  const bool real = r < rows_here;
  int tok, head;
  rs.at(a, 32 * rw + q32, tok, head);
  if (!real) tok = head = 0;
  head += kvh * a.group;
  Sight see = sight_of(a, sq, tok);
  if (!real) see = {0, 0};
  const float slope = a.slopes && real ? a.slopes[head] * kLog2e : 0.f;
  const int place = sq.n - sq.m + tok;

  // q on its way: an 8-bit operand's lane has channels 16 h .. of both of its blocks, 32 (2i) + and
  // 32 (2i + 1) +
  Raw8<__bf16> qraw[NB][2];
  {
    const __bf16* qp = (const __bf16*)a.q + (int64_t)(sq.row0 + tok) * a.ld_q + head * a.hs_q + 16 * h;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qraw[b][k] = Raw8<__bf16>{};
        if (real) qraw[b][k] = load8(qp + 32 * b + 8 * k);
      }
  }

  // the tokens of the workgroup's rows, of this wave's, and those that all of the wave's rows see
  const auto row_sight = [&](int i) {
    int t, hd;
    rs.at(a, i, t, hd);
    return sight_of(a, sq, uniform(t < sq.m - 1 ? t : sq.m - 1));
  };
  const int64_t p0 = sq.first(a) + (int64_t)piece * cut;
  const int wg_lo0 = row_sight(0).lo, wg_hi0 = row_sight(32 * ROW_WAVES - 1).hi;
  const int wg_lo = p0 > wg_lo0 ? (int)p0 : wg_lo0 & ~(kStep - 1);
  const int wg_hi = p0 + cut < wg_hi0 ? (int)(p0 + cut) : wg_hi0;
  const bool any = row0 < rows_here;
  const Sight s0 = row_sight(32 * rw), s1 = row_sight(32 * rw + 31);
  const int lo = s0.lo, hi = any ? s1.hi : 0;
  const int all_lo = s1.lo, all_hi = s0.hi;

  const KvUnit<D> unit{1 << a.page_log};
  const int32_t* pages = a.table + f.at * a.ld_table;
  const int in_page = (1 << a.page_log) - 1;
  const uint32_t page_bytes = (uint32_t)unit.bytes() * a.kv_heads;  // (of all heads: < 2^27)
  const uint8_t* pieces0 = a.data + (uint32_t)unit.bytes() * (uint32_t)kvh;
  // a token's piece of the cache; a page that is none: the first, and `bad`
  const auto piece_of = [&](int page, bool& bad) {
    bad = page < 0 || page >= a.n_pages;
    return pieces0 + (uint64_t)(bad ? 0u : (uint32_t)page) * page_bytes;
  };
  const int last = wg_hi - 1;

  // ---- global memory: values to registers, keys and their scale bytes to LDS.  A thread's token of
  // each kind; its page is looked up a stage ahead.
  const int v_run = threadIdx.x & 15, v_tok = 4 * (threadIdx.x >> 4);
  constexpr int FRAGS = STAGE / 32 * NI, PER = (FRAGS + WAVES - 1) / WAVES;  // of keys: [32 tokens][NI]
  constexpr int SDWORDS = STAGE * NB / 4, SCOPIES = (SDWORDS + 63) / 64;
  const int s_dword = (64 * wave + lane) % SDWORDS, s_tok = 4 * s_dword / NB & ~(NB == 2 ? 1 : 0);
  const auto clamped = [&](int t) { return t < last ? t : last; };
  const auto page_at = [&](int t) { return pages[clamped(t) >> a.page_log]; };
  int v_page, s_page, k_page[PER];
  const auto load_pages = [&](int t0) {
    v_page = page_at(t0 + v_tok);
    s_page = page_at(t0 + s_tok);
#pragma unroll
    for (int p = 0; p < PER; ++p) k_page[p] = page_at(t0 + (wave + p * WAVES) / NI * 32 + q32);
  };
  VRaw vr;
  uint32_t vs;
  bool v_bad;
  const auto load = [&](int t0, uint8_t* kb, uint8_t* sb) __attribute__((always_inline)) {
    bool bad;
    {
      const uint8_t* at = piece_of(v_page, v_bad);
      const int quad = (clamped(t0 + v_tok) & in_page) >> 2;
      __builtin_memcpy(&vr, at + unit.v_codes() + (quad * 16 + v_run) * 4 * NB, 4 * NB);
      __builtin_memcpy(&vs, at + unit.v_scales() + (quad * NB + v_run * NB / 16) * 4, 4);
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int f = wave + p * WAVES;
      if (FRAGS % WAVES == 0 || f < FRAGS) {
        const uint8_t* at = piece_of(k_page[p], bad);
        const int in = clamped(t0 + f / NI * 32 + q32) & in_page;
        load_to_lds(at + in * (D / 2) + 32 * (f % NI) + 16 * h, kb + f * 1024, 16);
      }
    }
    if (wave < SCOPIES) {
      const uint8_t* at = piece_of(s_page, bad);
      const int in = clamped(t0 + s_tok) & in_page & ~(NB == 2 ? 1 : 0);
      load_to_lds(at + unit.k_scales() + in * NB + (NB == 8 ? 4 * (s_dword & 1) : 0), sb + 256 * wave, 4);
    }
    load_pages(t0 + STAGE);
  };
  // Unit of 16 bytes: 8 tokens of a channel, [block][16 tokens][half of the lanes][32 channels].
  // Channel j of run o of its block is at place RB j + o, xor a number of the block and half, so
  // that a wave's 8-byte stores of one j spread over the banks.
  const auto v_store = [&](int buf) __attribute__((always_inline)) {
    const int quad = threadIdx.x >> 4, blk = v_run * NB / 16, o = v_run % RB;
    const int s = quad >> 2, hh = quad & 1, half = (quad >> 1) & 1;
    const uint32_t ov = over_bytes(vs);
    uint32_t sc = vs;
    if (ov) {  // NaN (or, behind the last token, anything): 0 here
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (((sc >> (8 * b)) & 0xFF) > kMaxScaleByte) sc &= ~(0xFFu << (8 * b));
    }
    uint8_t* dst = vbuf + buf * BUF + ((blk * (STAGE / 16) + s) * 2 + hh) * 512 + half * 8;
    const int swz = RB * ((2 * blk + hh) & (NC - 1));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int byte = e * NB + b;
        const uint32_t w = vr[byte / 4];
        const float k = scale_byte(sc, e);
        bf16x2 y;
        switch (byte & 3) {
          case 0: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k, 0); break;
          case 1: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k, 1); break;
          case 2: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k, 2); break;
          default: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k, 3); break;
        }
        x[e] = __builtin_bit_cast(uint32_t, y);
      }
      *(u32x2*)(dst + (((RB * 2 * b + o) ^ swz) * 16)) =
          u32x2{__builtin_amdgcn_perm(x[1], x[0], 0x05040100), __builtin_amdgcn_perm(x[3], x[2], 0x05040100)};
      *(u32x2*)(dst + (((RB * (2 * b + 1) + o) ^ swz) * 16)) =
          u32x2{__builtin_amdgcn_perm(x[1], x[0], 0x07060302), __builtin_amdgcn_perm(x[3], x[2], 0x07060302)};
    }
    const bool f2 = __ballot(ov != 0 || v_bad) != 0;
    if (lane == 0) over[buf][wave] = f2;
  };

  v8i32 qh[NI], ql[NI];
  int e0[NI], e1[NI];
  float m = -__builtin_inff(), l = 0.f;
  uint32_t nan_blocks = 0;  // blocks of channels in which this row has seen a NaN
  f32x16 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f32x16{};

  const bool plain = a.softcap == 0.f && !a.slopes && a.scale > 0.f;
  const float qk_scale = a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
  const float cap_k = cap_factor(a.softcap);
  const float unit_scale = plain ? qk_scale : 1.f;

  const auto arrived = [] {  // every load and copy that this wave has started
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
    asm volatile("" ::: "memory");
  };

  // A wave in its products goes before the one that shares its SIMD, so that one's products fall into
  // the other's exponentials (heads of 128: 367 -> 355 us for 4096 rows over 8192 tokens; heads of 64
  // have fewer products than exponentials and get slower, 126 -> 132).
  const auto ahead = [](bool yes) __attribute__((always_inline)) {
    if constexpr (D == 128) {
      if (yes) __builtin_amdgcn_s_setprio(2);
      else __builtin_amdgcn_s_setprio(0);
    }
  };

  // One stage: the next one's loads, this one's tokens in 64s, then the next one's values to LDS.
  const auto pass = [&](int t0, int buf, const uint8_t* kb, const uint8_t* sb, uint8_t* next_kb,
                        uint8_t* next_sb) __attribute__((always_inline)) {
    const bool more = t0 + STAGE < wg_hi;
    if (more) load(t0 + STAGE, next_kb, next_sb);
    uint32_t nan_here = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) nan_here |= over[buf][w];
    nan_here = uniform((int)nan_here);
#pragma unroll
    for (int part = 0; part < (HALVES ? 1 : STAGE / 64); ++part) {
      const int half = HALVES ? wave / ROW_WAVES : part;
      const int t = t0 + 64 * half;
      if (t >= hi || t + 64 <= lo || t >= wg_hi) continue;
      // ---- scores: all operands on their way before the first product
      f32x16 s[2];
      u32x4 kr[2][NI];
      uint32_t sw[2][2];  // the token's scale bytes, its lane's blocks 2 i + h from byte 0
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok32 = 2 * half + u;
        sw[u][1] = 0;
        if constexpr (NB == 2) {
          sw[u][0] = *(const uint16_t*)(sb + (32 * tok32 + q32) * 2) >> (8 * h);
        } else if constexpr (NB == 4) {
          sw[u][0] = *(const uint32_t*)(sb + (32 * tok32 + q32) * 4) >> (8 * h);
        } else {
          const u32x2 w = *(const u32x2*)(sb + (32 * tok32 + q32) * 8);
          sw[u][0] = w[0] >> (8 * h);
          sw[u][1] = w[1] >> (8 * h);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) kr[u][i] = *(const u32x4*)(kb + (tok32 * NI + i) * 1024 + lane * 16);
        s[u] = f32x16{};
      }
      __builtin_amdgcn_sched_barrier(0);
      ahead(true);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        v8i32 k[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          k[u] = v8i32{(int)kr[u][i][0], (int)kr[u][i][1], (int)kr[u][i][2], (int)kr[u][i][3], 0, 0, 0, 0};
        if (i & 1) {
          s[0] = scores_32<2>(k[0], qh[i], s[0], sw[0][i / 2], e0[i]);
          s[1] = scores_32<2>(k[1], qh[i], s[1], sw[1][i / 2], e0[i]);
          s[0] = scores_32<2>(k[0], ql[i], s[0], sw[0][i / 2], e1[i]);
          s[1] = scores_32<2>(k[1], ql[i], s[1], sw[1][i / 2], e1[i]);
        } else {
          s[0] = scores_32<0>(k[0], qh[i], s[0], sw[0][i / 2], e0[i]);
          s[1] = scores_32<0>(k[1], qh[i], s[1], sw[1][i / 2], e0[i]);
          s[0] = scores_32<0>(k[0], ql[i], s[0], sw[0][i / 2], e1[i]);
          s[1] = scores_32<0>(k[1], ql[i], s[1], sw[1][i / 2], e1[i]);
        }
      }
      // Values that are NaN (0 in LDS): noted for the rows that see them, a token a lane.  Pages that
      // are none: their scores are NaN.
      if (nan_here) {
        bool bad;
        const int j = clamped(t + lane);
        const uint8_t* at = piece_of(page_at(j), bad);
        const int in = j & in_page;
        const uint64_t none = __ballot(bad);
        const int lo_bit = see.lo > t ? see.lo - t : 0, hi_bit = see.hi - t;
        uint64_t sees_here = hi_bit >= 64 ? ~(uint64_t)0 : hi_bit > 0 ? ((uint64_t)1 << hi_bit) - 1 : 0;
        sees_here = lo_bit < 64 ? sees_here >> lo_bit << lo_bit : 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t u = at[unit.v_scales() + ((in >> 2) * NB + b) * 4 + (in & 3)];
          if (__ballot(u > kMaxScaleByte) & sees_here) nan_blocks |= 1u << b;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t here = (uint32_t)(none >> (32 * u)) >> (4 * h);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (here >> (8 * (e >> 2) + (e & 3)) & 1) s[u][e] = __builtin_nanf("");
        }
      }
      if (!plain) {
        const auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[u][e] = f(s[u][e] * qk_scale);
        };
        if (a.softcap > kNearCap)
          each([&](float x) { return capped_wide(x, a.softcap, cap_k) * kLog2e; });
        else if (a.softcap > 0.f)
          each([&](float x) { return capped<false>(x, a.softcap, cap_k) * kLog2e; });
        else
          each([](float x) { return x; });
        if (a.slopes) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = t + 32 * u + 8 * (e >> 2) + 4 * h + (e & 3);
              s[u][e] -= slope * (float)abs(place - j);
            }
        }
      }
      if (t < all_lo || t + 64 > all_hi) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = t + 32 * u + 8 * (e >> 2) + 4 * h + (e & 3);
            s[u][e] = j >= see.lo && j < see.hi ? s[u][e] : -__builtin_inff();
          }
      }
      // (the first values are on their way while the weights are made, the next ones while they are used)
      bf16x8 v[2][NB];
      const auto v_read = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int swz = RB * ((2 * b + h) & (NC - 1));
          v[c & 1][b] = *(const bf16x8*)(vbuf + buf * BUF + ((b * (STAGE / 16) + 4 * half + c) * 2 + h) * 512 +
                                         (q32 ^ swz) * 16);
        }
      };
      // ---- softmax
      float top = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[u][e]);
      top = max2(top) * unit_scale;
      if (__ballot(top > m + 8.f)) {
        const float next = fmaxf(m, top);
        const float base = next == -__builtin_inff() ? 0.f : next;
        const float old = exp2_fast(m - base);
        l *= old;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[b][e] *= old;
        m = next;
      }
      const float base = m == -__builtin_inff() ? 0.f : m;
      ahead(false);
      v_read(0);
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 p[4];
      float sum[4] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const bf16x2 w = {(__bf16)exp2_fast(fmaf(s[u][e], unit_scale, -base)),
                            (__bf16)exp2_fast(fmaf(s[u][e + 1], unit_scale, -base))};
          p[2 * u + (e >> 3)][e & 7] = w[0];
          p[2 * u + (e >> 3)][(e & 7) + 1] = w[1];
          const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
          sum[e >> 1 & 3] = __builtin_amdgcn_fdot2_f32_bf16(w, one, sum[e >> 1 & 3], false);
        }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // ---- out
      ahead(true);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < 3) v_read(c + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[c & 1][b], p[c], acc[b], 0, 0, 0);
      }
    }
    ahead(false);
    if (more) {
      arrived();
      v_store(buf ^ 1);
    }
    lds_barrier();
  };
  if (wg_lo < wg_hi) {
    load_pages(wg_lo);
    load(wg_lo, kbuf0, kscale0);
  }
  // (while the first tokens are on their way)
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    int e[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v[8];
        to_f32<__bf16>(qraw[2 * i + b][k], v);
#pragma unroll
        for (int n = 0; n < 8; ++n) x[8 * k + n] = v[n];
      }
      const uint32_t own = most_bits(x);
      const auto other = __builtin_amdgcn_permlane32_swap(own, own, false, false);
      const uint32_t most = other[0] > other[1] ? other[0] : other[1];
      e[b] = plane_exponent(most);
      if (b == 0) e4m3_planes<0>(x, e[b], qh[i], ql[i]);
      else e4m3_planes<4>(x, e[b], qh[i], ql[i]);
      if (most >= 0x7F800000u) e[b] = 255;  // infinite or NaN: so are all of its products
    }
    e0[i] = h ? e[1] : e[0];
    e1[i] = e0[i] == 255 ? 255 : e0[i] - 5;
  }
  if (wg_lo < wg_hi) {
    arrived();
    v_store(0);
    lds_barrier();
  }
  for (int t0 = wg_lo; t0 < wg_hi; t0 += 2 * STAGE) {
    pass(t0, 0, kbuf0, kscale0, kbuf1, kscale1);
    if (t0 + STAGE < wg_hi) pass(t0 + STAGE, 1, kbuf1, kscale1, kbuf0, kscale0);
  }
  l = sum2(l);
  if constexpr (HALVES) {
    // (every wave is past its last read of the stages)
    static_assert(WAVES == 8 && 4 * 64 * NB * 64 <= 2 * BUF);
    __shared__ float others[3][ROW_WAVES][64];
    float* const theirs = (float*)vbuf + rw * (NB * 16 * 64) + lane;
    if (wave >= ROW_WAVES) {
      others[0][rw][lane] = m;
      others[1][rw][lane] = l;
      others[2][rw][lane] = __uint_as_float(nan_blocks);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) theirs[(16 * b + e) * 64] = acc[b][e];
    }
    lds_barrier();
    if (wave < ROW_WAVES) {
      const float m2 = others[0][rw][lane], l2 = others[1][rw][lane];
      nan_blocks |= __float_as_uint(others[2][rw][lane]);
      const float up = fmaxf(m, m2), base = up == -__builtin_inff() ? 0.f : up;
      // (a wave without weights has nothing to add)
      const float k1 = l == 0.f ? 0.f : exp2_fast(m - base), k2 = l2 == 0.f ? 0.f : exp2_fast(m2 - base);
      l = l * k1 + l2 * k2;
      m = up;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[b][e] = acc[b][e] * k1 + theirs[(16 * b + e) * 64] * k2;
    }
    lds_barrier();  // (the rows' way out goes through the same memory)
    if (wave >= ROW_WAVES) return;
  }
  if (__ballot(nan_blocks != 0)) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[b][e] = nan_blocks >> b & 1 ? __builtin_nanf("") : acc[b][e];
  }

  if (a.target && piece == 0 && kvh == 0 && h == 0 && real && head == 0) put_record(a, f, tok, see);

  // ---- rows out: through LDS, a block of channels at a time, so that they leave in order
  const bool sees = see.lo < see.hi;
  const bool part = f.pieces > 1;
  const float inv = part ? 1.f : sees ? 1.f / l : 0.f;
  const int64_t slot0 = (((int64_t)item * a.kv_heads + kvh) << a.tile_log) + 32 * rw;
  if (part && real && h == 0) {
    a.part[a.ml_at + 2 * (slot0 + q32)] = m;
    a.part[a.ml_at + 2 * (slot0 + q32) + 1] = l;
  }
  float* mine = (float*)vbuf + rw * 32 * LD;
  const int orow = lane >> 1, oc = (lane & 1) * 16;
  const int orr = row0 + orow;
  int otok, ohead;
  rs.at(a, 32 * rw + orow, otok, ohead);
  __bf16* dst = (__bf16*)a.out + (int64_t)(sq.row0 + otok) * a.ld_out +
                (int64_t)(kvh * a.group + ohead) * a.hs_out + oc;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int place_in = 8 * (e >> 2) + 4 * h + (e & 3);  // RB j + o
      const int ch = (place_in % RB) * NC + place_in / RB;
      mine[q32 * LD + ch] = part ? acc[b][e] : sees ? acc[b][e] * inv : 0.f;
    }
    __builtin_amdgcn_wave_barrier();
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = mine[orow * LD + oc + i];
    __builtin_amdgcn_wave_barrier();
    if (orr < rows_here) {
      if (part) {
        __builtin_memcpy(a.part + (slot0 + orow) * D + 32 * b + oc, o, sizeof(o));
      } else {
        __bf16 res[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) res[i] = (__bf16)o[i];
        __builtin_memcpy(dst + 32 * b, res, sizeof(res));
      }
    }
  }
}

template <int D, int WAVES, bool HALVES>
static void launch_one(const AttnArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((attn_chunk_kernel<D, WAVES, HALVES>), item_grid(a.items, a.kv_heads),
                     dim3(64 * WAVES), 0, stream, a);
}
template <int D>
static void launch_dim(const AttnArgs& a, int tile_rows, bool halves, hipStream_t stream) {
  if (halves) launch_one<D, 8, true>(a, stream);
  else if (tile_rows == 256) launch_one<D, 8, false>(a, stream);
  else launch_one<D, 4, false>(a, stream);
}

void attn_chunk_launch(const AttnArgs& a, int head_dim, int tile_rows, bool halves, hipStream_t stream) {
  switch (head_dim) {
    case 64: launch_dim<64>(a, tile_rows, halves, stream); break;
    case 128: launch_dim<128>(a, tile_rows, halves, stream); break;
    default: launch_one<256, 4, false>(a, stream); break;
  }
}

}  // namespace moe
