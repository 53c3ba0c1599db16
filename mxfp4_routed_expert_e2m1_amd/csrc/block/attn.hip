// attn.hip -- attention of a ragged batch's rows over a 4-bit cache.
//
// One pass over the tokens with the running maximum and sum of a softmax, 32 tokens a step:
//   S^T = K Q^T          (matrix core, tokens x rows)
//   m' = max(m, max S),  P = 2^(S - m'),  l = l 2^(m - m') + sum P
//   O^T = O^T 2^(m - m') + V^T P^T
// with S in units of log2.  A tile's rows are (token, query head of the key head's group) pairs,
// row r = token r / G, head r % G, so one pass over a key head's tokens serves its whole group.
// Here are tiles of 16 or 32 rows a wave: few new rows a sequence, and every f32 call.  Tiles of 128 and
// 256 rows are in attn_chunk.hip.
//
// Operands.  bf16 calls: keys' E2M1 codes and their scale bytes go into the scaled 8-bit matrix
// instruction as they are in the cache, against q in two E4M3 planes.  f32 calls, and V in all: E2M1
// values times a power of two are exact in bf16, and the converter makes two in one instruction.  Lane
// l of a wave holds row l % 16 of an operand and a part of the contraction, group l / 16; which part
// is free, as long as both operands agree:
//   scores: group g has block g of 32 channels (of 4 at a time), which lie side by side in the cache;
//   out:    group g has the tokens 4g .. 4g+3 and 16 + 4g .. + 3 of 32, since that is what it
//           holds of S^T as the matrix core leaves it: P goes from one product into the next in
//           the registers where it was made.  V's order in the cache makes these 4 tokens of
//           D/16 channels one load.
// Rounding.  K and V are exact.  q in bf16 calls: all 8 bits, less what is below 2^-22 of the largest of
// its block of 32 channels.  P is rounded to bf16 (by 2^-8 of a weight at most; the second product at this
// rate has no more bits), and l is the sum of the rounded weights, by the matrix core: they are exact
// weights of an average, so equal values are its result however they round (the sum of unrounded ones
// left a row 2^-8 short where all rounded down, in the same time).  f32 calls split q and P into three
// bf16 parts each, which hold all 24 bits.
//
// Work.  A call's tiles (sequence, rows) times key heads fill the chip or not; where they do not, a
// sequence's tokens are cut into pieces of equal length, as many over all sequences as fill it,
// and a second launch joins them.  Lengths are on the GPU alone, so a workgroup finds its tile and the
// cut from them when it starts.
//
// What bounds it: the cache's bytes, read once for each tile, for few rows of long contexts; the
// latency of the chain lengths -> page -> tokens -> softmax -> join for short ones; f32 calls the six
// products for the scores and the weights.  32 query heads on 8 of 128 channels, one new row a request:
//   64 requests of 2048 to 4096 tokens  55 us (3.9 TB/s)   16 of 2048 to 8192  29 us with its join of 5
//   one of 1003 tokens  9.3 us                             one of 65536  25 us
// and 5 new rows of 3 requests of up to 100001 tokens, 24 heads on 8: bf16 77 us (4.0 TB/s), f32 97 us.
#include "attn.h"

namespace moe {

// ------------------------------------------------------------------- the pass
// SHARED: the waves of a workgroup have one tile of 16 NQ rows and take its tokens in turn, 32 each,
// joined in LDS at the end; otherwise each wave has a tile of its own among the workgroup's.
// Each wave copies the tokens of its next two steps straight into LDS (one step for D 256, by the
// room) while it has the current ones.  16 requests of 2048 to 8192 tokens took 53 us with codes loaded
// into registers just before their use, 31 with copies into LDS.
template <typename T, int D, int NQ, int WAVES, bool SHARED>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? resident(sizeof(T) == 4, D, NQ) : 1)
void attn_rows_kernel(const AttnArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NB = D / 32, NC = D / 16, NI = (D + 127) / 128, PARTS = F32 ? 3 : 1;
  constexpr int STEP = 32, STRIDE = SHARED ? STEP * WAVES : STEP;
  // a wave's step in LDS: keys' codes, values' codes, scale bytes
  constexpr int STAGE = 32 * D + 256 * NI, RING = D == 256 ? 2 : 3;
  typedef uint32_t VRaw __attribute__((ext_vector_type(NB)));
  // (an array for each stage, so that reads of one wait for no copies into the others)
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[WAVES * STAGE], ring1[WAVES * STAGE],
      ring2[RING > 2 ? WAVES * STAGE : 16];
  uint8_t* const ring[3] = {ring0, ring1, ring2};
  const int wave = uniform((int)(threadIdx.x >> 6)), lane = lane_id();
  const int r16 = lane & 15, g = lane >> 4;
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
  const int trow0 = (tile << a.tile_log) + (SHARED ? 0 : wave * 16 * NQ);
  const RowSplit rs(a, trow0);
  const int rows_here = sq.m * a.group;  // (row, head) pairs of the sequence and key head

  // this lane's rows: trow0 + 16 nq + r16
  int tok[NQ], head[NQ];
  bool real[NQ];
  Sight see[NQ];
  float slope[NQ];
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) {
    real[nq] = trow0 + 16 * nq + r16 < rows_here;
    rs.at(a, 16 * nq + r16, tok[nq], head[nq]);
    if (!real[nq]) tok[nq] = head[nq] = 0;
    head[nq] += kvh * a.group;
    see[nq] = sight_of(a, sq, tok[nq]);
    if (!real[nq]) see[nq] = {0, 0};
    slope[nq] = a.slopes && real[nq] ? a.slopes[head[nq]] * kLog2e : 0.f;
  }
  // q on its way: f32 calls 8 channels of each of a lane's blocks 4 i + g; bf16 calls D/64 channels of
  // the rows that a wave prepares for the workgroup
  constexpr int QROWS = 16 * NQ / WAVES, QCH = D / 64;
  Raw8<float> qraw[NQ][NI][4];
  __bf16 qmine[QROWS][QCH];
  if constexpr (F32) {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const T* qp = (const T*)a.q + (int64_t)(sq.row0 + tok[nq]) * a.ld_q + head[nq] * a.hs_q;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int c = 32 * (4 * i + g) + 8 * n;
          qraw[nq][i][n] = Raw8<float>{};
          if (real[nq] && c < D) qraw[nq][i][n] = load8((const float*)qp + c);
        }
    }
  } else {
#pragma unroll
    for (int n = 0; n < QROWS; ++n) {
      const int row = wave * QROWS + n;
      int qt, qhd;
      rs.at(a, row, qt, qhd);
#pragma unroll
      for (int c = 0; c < QCH; ++c) qmine[n][c] = (__bf16)0.f;
      if (trow0 + row < rows_here)
        __builtin_memcpy(qmine[n],
                         (const __bf16*)a.q + (int64_t)(sq.row0 + qt) * a.ld_q +
                             (int64_t)(kvh * a.group + qhd) * a.hs_q + QCH * lane,
                         sizeof(qmine[n]));
    }
  }

  // the tile's tokens: what its first row (window) and its last (causal) see, and all of them
  const bool any = trow0 < rows_here;
  int tok1, head1;
  rs.at(a, 16 * NQ - 1, tok1, head1);
  tok1 = tok1 < sq.m - 1 ? tok1 : sq.m - 1;
  const Sight s0 = sight_of(a, sq, any ? rs.tok0 : 0), s1 = sight_of(a, sq, uniform(tok1));
  const int64_t p0 = sq.first(a) + (int64_t)piece * cut;
  const int lo = p0 > s0.lo ? (int)p0 : s0.lo & ~(kStep - 1);
  const int hi = !any ? 0 : p0 + cut < s1.hi ? (int)(p0 + cut) : s1.hi;
  const int all_lo = s1.lo, all_hi = s0.hi;

  float m[NQ], l[NQ];
  f32x4 acc[NQ][NC], lsum[NQ];  // (lsum: bf16 calls' l, in every register and group alike)
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) {
    lsum[nq] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[nq] = -__builtin_inff();
    l[nq] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[nq][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const KvUnit<D> unit{1 << a.page_log};
  const uint32_t page_bytes = (uint32_t)unit.bytes() * a.kv_heads;  // (of all heads: < 2^27)
  const uint8_t* pieces0 = a.data + (uint32_t)unit.bytes() * (uint32_t)kvh;
  // (scalar loads: as vector loads their arrival would be that of every copy before them)
  const auto* pages = (const __attribute__((address_space(4))) int32_t*)(a.table + f.at * a.ld_table);
  const bool plain = a.softcap == 0.f && !a.slopes && a.scale > 0.f;
  const float qk_scale = a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
  const float cap_k = cap_factor(a.softcap);
  const float unit_scale = plain ? qk_scale : 1.f;

  // ---- tokens: a wave's steps of 32, copied straight into its part of LDS, RING - 1 steps ahead.  16
  // tokens lie in one page; those past the last are taken as the last 16 and masked.
  const int t_first = lo + (SHARED ? wave * STEP : 0);
  const int n_steps = t_first < hi ? (hi - t_first + STRIDE - 1) / STRIDE : 0;
  const int last16 = (hi - 1) & ~15;
  const auto sub_of = [&](int step, int u) {
    const int t = t_first + step * STRIDE + 16 * u;
    return t < last16 ? t : last16;
  };
  int pg[2];          // pages of the step to copy next
  uint32_t bad = 0;   // two bits a step, the latest lowest: whether its pages are none
  const auto load_pages = [&](int step) {
#pragma unroll
    for (int u = 0; u < 2; ++u) pg[u] = pages[uniform(sub_of(step, u) >> a.page_log)];
  };
  const auto copy = [&](uint8_t* to, int step) {
    const uint8_t* at[2];
    int in[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool none = pg[u] < 0 || pg[u] >= a.n_pages;
      bad = bad << 1 | none;
      at[u] = pieces0 + (uint64_t)(none ? 0u : (uint32_t)pg[u]) * page_bytes;
      in[u] = sub_of(step, u) & ((1 << a.page_log) - 1);
    }
    load_pages(step + 1);
    uint8_t* mine = to + wave * STAGE;
    const int u5 = lane >> 5, l5 = lane & 31;
    if constexpr (D == 64) {  // both halves of the step in one copy
      const uint8_t* p = (u5 ? at[1] : at[0]) + (u5 ? in[1] : in[0]) * (D / 2);
      load_to_lds(p + (l5 & 15) * (D / 2) + (l5 >> 4) * 16, mine, 16);
      load_to_lds(p + unit.v_codes() + l5 * 16, mine + 16 * D, 16);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          load_to_lds(at[u] + in[u] * (D / 2) + r16 * (D / 2) + 64 * i + 16 * g,
                      mine + (u * NI + i) * 1024, 16);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          load_to_lds(at[u] + unit.v_codes() + in[u] * (D / 2) + 1024 * i + 16 * lane,
                      mine + 16 * D + (u * NI + i) * 1024, 16);
    }
    // scale bytes: [keys, values][half of the step][4 NB dwords]
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int d = (64 * i + lane) % (16 * NB), u = d / (4 * NB) & 1;
      load_to_lds((u ? at[1] : at[0]) + (d < 8 * NB ? unit.k_scales() : unit.v_scales()) +
                      (u ? in[1] : in[0]) * NB + 4 * (d % (4 * NB)),
                  mine + 32 * D + 256 * i, 4);
    }
  };
  constexpr int COPIES = D == 64 ? 3 : 5 * NI;
  // Tiles of many rows copy their last tokens again for the steps past the end, so that nothing
  // depends on how many are left: 1024 new rows of a request of 2048 tokens, 32 query heads on 8 of
  // 128, f32: 103 -> 98 us.  For a single row the copies themselves count: 1003 tokens in bf16 take
  // 9.3 us without them, 10.0 with them.
  constexpr bool PAST_END = !SHARED;
  if (n_steps) {
    load_pages(0);
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) {
      if (PAST_END || i == 0 || i < n_steps) copy(ring[i], i);
      else bad <<= 2;
    }
  }

  // q as the matrix core takes it: bf16 calls in two E4M3 planes (128 channels an instruction), f32
  // calls in three bf16 parts (32 channels an instruction)
  v8i32 qh[NQ][NI], ql[NQ][NI];
  int e0[NQ][NI], e1[NQ][NI];
  bf16x8 q[NQ][NI][4][PARTS];
  if constexpr (F32) {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float v[8], x[2][4];
          to_f32<float>(qraw[nq][i][n], v);
#pragma unroll
          for (int e = 0; e < 8; ++e)  // (a row with an infinity has no finite score)
            x[e / 4][e % 4] = fabsf(v[e]) < __builtin_inff() ? v[e] : __builtin_nanf("");
          split8<PARTS>(x, q[nq][i][n]);
        }
  } else {
    // Each wave's rows into the last stage's memory, which has no copies yet: planes [row][D], scale
    // bytes [row][NB].  An 8-bit operand's lane has channels 16 g .. and 64 + 16 g .. of 128, and the
    // scale of block 4 i + g.
    uint8_t* const qs = ring[RING - 1];
    constexpr int ROWS = 16 * NQ;
    static_assert(ROWS * (2 * D + NB) <= WAVES * STAGE);
#pragma unroll
    for (int n = 0; n < QROWS; ++n) {
      const int row = wave * QROWS + n;
      uint32_t most = 0;
      float x[QCH];
#pragma unroll
      for (int c = 0; c < QCH; ++c) {
        x[c] = (float)qmine[n][c];
        const uint32_t b = __float_as_uint(x[c]) & 0x7FFFFFFFu;
        most = b > most ? b : most;
      }
      most = block_max<32 / QCH>(most);
      const int e = plane_exponent(most);
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);
      uint8_t hi8[QCH], lo8[QCH];
#pragma unroll
      for (int c = 0; c < QCH; ++c) {
        const float r = x[c] * down;
        const int hi = __builtin_amdgcn_cvt_pk_fp8_f32(r, r, 0, false);
        const float rest = (r - __builtin_amdgcn_cvt_f32_fp8(hi, 0)) * 32.f;
        hi8[c] = (uint8_t)hi;
        lo8[c] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(rest, rest, 0, false);
      }
      __builtin_memcpy(qs + row * D + QCH * lane, hi8, QCH);
      __builtin_memcpy(qs + (ROWS + row) * D + QCH * lane, lo8, QCH);
      if (lane % (32 / QCH) == 0)  // (infinite or NaN: so are all of its products)
        qs[2 * ROWS * D + row * NB + lane / (32 / QCH)] = (uint8_t)(most >= 0x7F800000u ? 255 : e);
    }
    lds_barrier();
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = 16 * nq + r16;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int c = 128 * i + 64 * b + 16 * g;
          u32x4 hi = {}, lo = {};
          if (c < D) {
            hi = *(const u32x4*)(qs + row * D + c);
            lo = *(const u32x4*)(qs + (ROWS + row) * D + c);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            qh[nq][i][4 * b + k] = (int)hi[k];
            ql[nq][i][4 * b + k] = (int)lo[k];
          }
        }
        const int block = 4 * i + g;
        e0[nq][i] = block < NB ? qs[2 * ROWS * D + row * NB + block] : 127;
        e1[nq][i] = e0[nq][i] == 255 ? 255 : e0[nq][i] - 5;
      }
    lds_barrier();  // (copies into that stage start behind this)
  }

  // One step: the copies of step + RING - 1, if there is one, into the stage that was read last, once
  // those reads are done, then this step's tokens.
  const auto pass = [&](int step, const uint8_t* stage, uint8_t* to) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0
    asm volatile("" ::: "memory");
    if (PAST_END || step + RING - 1 < n_steps) {
      copy(to, step + RING - 1);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((RING - 1) * COPIES | 0xF70);  // vmcnt
    } else {
      bad <<= 2;
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
    }
    asm volatile("" ::: "memory");
    const int t = t_first + step * STRIDE;
    const uint8_t* mine = stage + wave * STAGE;
    u32x4 kr[2][NI];
    VRaw vr[2];
    uint32_t ks[2][NI], vs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        kr[u][i] = *(const u32x4*)(mine + (D == 64 ? u * 512 + ((g & 1) * 16 + r16) * 16
                                                   : (u * NI + i) * 1024 + lane * 16));
        const uint32_t b = mine[32 * D + u * 16 * NB + r16 * NB + (D == 64 ? g & 1 : g) + 4 * i];
        ks[u][i] = bad >> (2 * RING - 1 - u) & 1 ? 255u : b;
      }
      vr[u] = *(const VRaw*)(mine + 16 * D + u * 8 * D + lane * 4 * NB);
      vs[u] = *(const uint32_t*)(mine + 32 * D + 32 * NB + u * 16 * NB + (g * NB + r16 * NB / 16) * 4);
    }
    // ---- scores
    float s[NQ][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 c[NQ];
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) c[nq] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4 kk = kr[u][i];
        const uint32_t sb = ks[u][i];
        if constexpr (F32) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const bf16x8 k = fp4x8_to_bf16x8(kk[n], __uint_as_float(sb << 23));  // (255: NaN)
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int p = 0; p < PARTS; ++p)
                c[nq] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[nq][i][n][p], c[nq], 0, 0, 0);
          }
        } else {
          const v8i32 k = {(int)kk[0], (int)kk[1], (int)kk[2], (int)kk[3], 0, 0, 0, 0};
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            c[nq] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                k, qh[nq][i], c[nq], 4, 0, 0, (int)sb, 0, e0[nq][i]);
            c[nq] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                k, ql[nq][i], c[nq], 4, 0, 0, (int)sb, 0, e1[nq][i]);
          }
        }
      }
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nq][u][e] = c[nq][e];
    }
    if (!plain) {
      const auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nq][u][e] = f(s[nq][u][e] * qk_scale);
      };
      if (a.softcap > kNearCap)
        each([&](float x) { return capped_wide(x, a.softcap, cap_k) * kLog2e; });
      else if (a.softcap > 0.f)
        each([&](float x) { return capped<F32>(x, a.softcap, cap_k) * kLog2e; });
      else
        each([](float x) { return x; });
      if (a.slopes) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = t + 16 * u + 4 * g + e;
              s[nq][u][e] -= slope[nq] * (float)abs(sq.n - sq.m + tok[nq] - j);
            }
      }
    }
    if (t < all_lo || t + STEP > all_hi) {
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = t + 16 * u + 4 * g + e;
            s[nq][u][e] = j >= see[nq].lo && j < see[nq].hi ? s[nq][u][e] : -__builtin_inff();
          }
    }

    // ---- values that are NaN (or, behind the last token, anything): 0 in the product, and NaN
    // in the channels of the rows that see them
    if (__ballot((over_bytes(vs[0]) | over_bytes(vs[1])) != 0)) {
      bf16x8 nan;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        nan[e] = (__bf16)(((vs[e / 4] >> (8 * (e & 3))) & 0xFF) > kMaxScaleByte ? 1.f : 0.f);
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        bf16x8 seen;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = t + 16 * (e / 4) + 4 * g + (e & 3);
          seen[e] = (__bf16)(j >= see[nq].lo && j < see[nq].hi ? 1.f : 0.f);
        }
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nan, seen, c, 0, 0, 0);
        // (c: of the runs of channels 4g + e, which a block's scale covers whole)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c[e] > 0.f) {
#pragma unroll
            for (int j = 0; j < NC; ++j) acc[nq][j][e] = __builtin_nanf("");
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (((vs[u] >> (8 * b)) & 0xFF) > kMaxScaleByte) vs[u] &= ~(0xFFu << (8 * b));
    }

    // ---- softmax.  A row's base is raised when its maximum has grown by 2^8 (or is the first):
    // weights of up to 2^8 are as exact as those up to 1.
    bf16x8 p[NQ][PARTS];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float top = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[nq][u][e]);
      top = max16(top) * unit_scale;
      if (__ballot(top > m[nq] + 8.f)) {
        const float up = fmaxf(m[nq], top);
        const float old = exp2_fast(m[nq] - (up == -__builtin_inff() ? 0.f : up));
        l[nq] *= old;
        lsum[nq] *= old;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nq][j][e] *= old;
        m[nq] = up;
      }
      const float base = m[nq] == -__builtin_inff() ? 0.f : m[nq];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = exp2_fast(fmaf(s[nq][u][e], unit_scale, -base));
          if constexpr (F32) l[nq] += w;
          s[nq][u][e] = w;
        }
      split8<PARTS>(s[nq], p[nq]);
    }

    // ---- out
    float sc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sc[e] = scale_byte(vs[e / 4], e & 3);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // channels 2b and 2b + 1 of the lane's run, 8 tokens
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int byte = (e & 3) * NB + b;  // of the 4 NB loaded
        const uint32_t w = vr[e / 4][byte / 4];
        bf16x2 y;
        switch (byte & 3) {
          case 0: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc[e], 0); break;
          case 1: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc[e], 1); break;
          case 2: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc[e], 2); break;
          default: y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc[e], 3); break;
        }
        x[e] = __builtin_bit_cast(uint32_t, y);
      }
      u32x4 even, odd;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        even[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x05040100);
        odd[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x07060302);
      }
      const bf16x8 v0 = __builtin_bit_cast(bf16x8, even), v1 = __builtin_bit_cast(bf16x8, odd);
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          acc[nq][2 * b] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[nq][k], acc[nq][2 * b], 0, 0, 0);
          acc[nq][2 * b + 1] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[nq][k], acc[nq][2 * b + 1], 0, 0, 0);
        }
    }
    if constexpr (!F32) {
      bf16x8 one;
#pragma unroll
      for (int e = 0; e < 8; ++e) one[e] = (__bf16)1.f;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
        lsum[nq] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, p[nq][0], lsum[nq], 0, 0, 0);
    }
  };
  for (int step = 0; step < n_steps; step += RING) {
#pragma unroll
    for (int i = 0; i < RING; ++i) {
      if (step + i >= n_steps) break;
      pass(step + i, ring[i], ring[(i + RING - 1) % RING]);
    }
  }
  if constexpr (PAST_END) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
    asm volatile("" ::: "memory");
  }
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) l[nq] = F32 ? sum16(l[nq]) : lsum[nq][0];

  if (a.target && piece == 0 && kvh == 0 && g == 0 && (!SHARED || wave == 0)) {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
      if (real[nq] && head[nq] == 0) put_record(a, f, tok[nq], see[nq]);
  }

  // ---- the waves' parts into one
  const int64_t slot0 =
      (((int64_t)item * a.kv_heads + kvh) << a.tile_log) + (SHARED ? 0 : wave * 16 * NQ);
  if constexpr (SHARED) {
    // Through the first two stages' memory, half of a run's channels in each; rows that are none stay
    // out of it.  The waves bring their parts to the largest base first.
    constexpr int HC = NC / 2, LD = D / 2 + 4, LANES = 4 * WAVES, PER = D / 2 / LANES;
    static_assert(16 * LD * 4 <= STAGE && PER >= 1 && HC % PER == 0);
    __shared__ float bases[NQ][WAVES][16], sums[NQ][WAVES][16];
    const int row = threadIdx.x / LANES, ch = (threadIdx.x % LANES) * PER;  // of D/2
    if (g == 0) {
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) bases[nq][wave][r16] = m[nq];
    }
    lds_barrier();
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, bases[nq][w][r16]);
      // (a wave without weights has nothing to add, and its base is no number to take an exponential
      // with)
      const float k = l[nq] == 0.f ? 0.f : exp2_fast(m[nq] - (top == -__builtin_inff() ? 0.f : top));
      if (g == 0) sums[nq][wave][r16] = l[nq] * k;
      if (nq) lds_barrier();
      if (real[nq]) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float* to = (float*)((half ? ring1 : ring0) + wave * STAGE) + r16 * LD;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < HC; j += 2)
              *(f32x2*)(to + HC * (4 * g + e) + j) =
                  f32x2{acc[nq][half * HC + j][e] * k, acc[nq][half * HC + j + 1][e] * k};
        }
      }
      lds_barrier();
      const int r = trow0 + 16 * nq + row;
      if (r >= rows_here) continue;
      int token, hd;
      rs.at(a, 16 * nq + row, token, hd);
      hd += kvh * a.group;
      float sum = 0.f, o[2][PER] = {};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        sum += sums[nq][w][row];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float* from = (const float*)((half ? ring1 : ring0) + w * STAGE) + row * LD + ch;
#pragma unroll
          for (int j = 0; j < PER; ++j) o[half][j] += from[j];
        }
      }
      const Sight sg = sight_of(a, sq, token);
      const bool sees = sg.lo < sg.hi;
      const float inv = 1.f / sum;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int c = ch / HC * NC + half * HC + ch % HC;  // channel of the first
        if (f.pieces > 1) {
          const int64_t slot = slot0 + 16 * nq + row;
          __builtin_memcpy(a.part + slot * D + c, o[half], sizeof(o[half]));
          if (ch == 0 && half == 0) {
            float up = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) up = fmaxf(up, bases[nq][w][row]);
            a.part[a.ml_at + 2 * slot] = up;
            a.part[a.ml_at + 2 * slot + 1] = sum;
          }
        } else {
          T res[PER];
#pragma unroll
          for (int j = 0; j < PER; ++j) res[j] = (T)(sees ? o[half][j] * inv : 0.f);
          T* dst = (T*)a.out + (int64_t)(sq.row0 + token) * a.ld_out + hd * a.hs_out + c;
          __builtin_memcpy(dst, res, sizeof(res));
        }
      }
    }
  } else {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      if (!real[nq]) continue;
      const bool sees = see[nq].lo < see[nq].hi;
      const int64_t slot = slot0 + 16 * nq + r16;
      const float inv = 1.f / l[nq];
      T* dst = (T*)a.out + (int64_t)(sq.row0 + tok[nq]) * a.ld_out + head[nq] * a.hs_out;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ch = NC * (4 * g + e);
        float o[NC];
        T res[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) o[j] = acc[nq][j][e];
        if (f.pieces > 1) {
          __builtin_memcpy(a.part + slot * D + ch, o, sizeof(o));
        } else {
#pragma unroll
          for (int j = 0; j < NC; ++j) res[j] = (T)(sees ? o[j] * inv : 0.f);
          __builtin_memcpy(dst + ch, res, sizeof(res));
        }
      }
      if (f.pieces > 1 && g == 0) {
        a.part[a.ml_at + 2 * slot] = m[nq];
        a.part[a.ml_at + 2 * slot + 1] = l[nq];
      }
    }
  }
}

// Pieces into rows: WAVES waves for each (row, head).  A lane has a piece's base and sum, then D/64
// channels of pieces w, w + WAVES, ..  A launch of its own, 5 us, most of them its start and its chain
// record -> bases -> parts: the pieces' bytes are few.
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 64, BATCH = 8;
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  const int row = blockIdx.x, head = WAVES == 1 ? blockIdx.y * 4 + wave : blockIdx.y;
  const int w0 = WAVES == 1 ? 0 : wave;
  if (head >= a.n_heads) return;
  if (a.q_offsets && (row < a.q_offsets[0] || row >= a.q_offsets[a.n_seqs])) return;
  const RowRecord rec = ((const RowRecord*)(a.part + a.rec_at))[row];
  const bool sees = rec.pieces > 0;
  const int pieces = sees ? rec.pieces : -rec.pieces;
  if (pieces == 1) return;
  const int kvh = head / a.group;
  const int r = (row - rec.row0) * a.group + head - kvh * a.group, tile = r >> a.tile_log;
  const int64_t item0 = rec.first_item + (int64_t)(rec.tiles - 1 - tile) * pieces;
  if (pieces < 1 || item0 < 0 || item0 + pieces > a.items) return;  // (offsets that overlap)
  const int64_t slot0 = ((item0 * a.kv_heads + kvh) << a.tile_log) + (r - (tile << a.tile_log));
  const int64_t step = (int64_t)a.kv_heads << a.tile_log;
  const float* ml = a.part + a.ml_at;
  float top = -__builtin_inff(), sum = 0.f, o[PER] = {};
  for (int p0 = 0; p0 < pieces; p0 += 64) {
    const int n = pieces - p0 < 64 ? pieces - p0 : 64;
    float mine = -__builtin_inff(), lp = 0.f;
    if (lane < n) {
      mine = ml[2 * (slot0 + (p0 + lane) * step)];
      lp = ml[2 * (slot0 + (p0 + lane) * step) + 1];
    }
    const float* src = a.part + (slot0 + p0 * step) * D + lane * PER;
    float up = -__builtin_inff(), k = 0.f;
    uint64_t skips = 0;
    for (int p = w0; p < n; p += BATCH * WAVES) {
      float v[BATCH][PER];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int at_p = p + i * WAVES < n ? p + i * WAVES : n - 1;
        __builtin_memcpy(v[i], src + at_p * step * D, sizeof(v[i]));
      }
      if (p == w0) {  // (while the first ones are on their way)
        up = fmaxf(top, wave_max(mine));
        const float base = up == -__builtin_inff() ? 0.f : up, old = exp2_fast(top - base);
        // (a piece without weights has nothing to add, and may hold no numbers)
        k = lp == 0.f ? 0.f : exp2_fast(mine - base);
        skips = __ballot(lp == 0.f);
        sum = sum * old + wave_sum(lp == 0.f ? 0.f : lp * k);
#pragma unroll
        for (int j = 0; j < PER; ++j) o[j] *= old;
        top = up;
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int at_p = p + i * WAVES;
        if (at_p >= n || ((skips >> at_p) & 1)) continue;
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(k), at_p));
#pragma unroll
        for (int j = 0; j < PER; ++j) o[j] += v[i][j] * w;
      }
    }
    if (w0 >= n) {  // (no piece for this wave among these: their base and sum all the same)
      up = fmaxf(top, wave_max(mine));
      const float base = up == -__builtin_inff() ? 0.f : up, old = exp2_fast(top - base);
      sum = sum * old + wave_sum(lp == 0.f ? 0.f : lp * exp2_fast(mine - base));
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] *= old;
      top = up;
    }
  }
  if constexpr (WAVES > 1) {
    __shared__ float others[WAVES - 1][64 * PER];
    if (wave) {
#pragma unroll
      for (int j = 0; j < PER; ++j) others[wave - 1][lane * PER + j] = o[j];
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 0; w < WAVES - 1; ++w)
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] += others[w][lane * PER + j];
  }
  const float inv = 1.f / sum;
  T res[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) res[j] = (T)(sees ? o[j] * inv : 0.f);
  __builtin_memcpy((T*)a.out + (int64_t)row * a.ld_out + head * a.hs_out + lane * PER, res, sizeof(res));
}

// ------------------------------------------------------------------ the host side
static bool attn_sizes_ok(const moe_attn_t* A, const moe_kv_cache_t* C) {
  return A->n_heads >= 1 && A->n_heads <= 16384 && A->n_heads % C->n_heads == 0;
}

template <typename T, int D>
static void attn_launch(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.chunk) {
    attn_chunk_launch(a, D, p.tile_rows, p.halves, stream);
  } else {
    const dim3 grid = item_grid(p.items, a.kv_heads);
    // (a tile of 32 rows and 256 channels has no room for 8 waves)
    constexpr int WIDE = 8, WIDE2 = D == 256 ? 4 : 8;
    if constexpr (sizeof(T) == 4) {
      auto k = !p.shared  ? attn_rows_kernel<T, D, 1, 4, false>
               : p.wide   ? attn_rows_kernel<T, D, 1, WIDE, true>
                          : attn_rows_kernel<T, D, 1, 4, true>;
      hipLaunchKernelGGL(k, grid, dim3(p.shared && p.wide ? 64 * WIDE : 256), 0, stream, a);
    } else {
      auto k = p.nq == 1 ? (p.wide ? attn_rows_kernel<T, D, 1, WIDE, true>
                                   : attn_rows_kernel<T, D, 1, 4, true>)
                         : (p.wide ? attn_rows_kernel<T, D, 2, WIDE2, true>
                                   : attn_rows_kernel<T, D, 2, 4, true>);
      hipLaunchKernelGGL(k, grid, dim3(64 * (!p.wide ? 4 : p.nq == 1 ? WIDE : WIDE2)), 0, stream, a);
    }
  }
  if (p.target) {
    // a workgroup for each row's head while they are few
    const bool many = (int64_t)a.rows * a.n_heads > 2048;
    const dim3 grid((unsigned)a.rows, (unsigned)(many ? (a.n_heads + 3) / 4 : a.n_heads));
    auto join = many ? attn_join_kernel<T, D, 1> : attn_join_kernel<T, D, 4>;
    hipLaunchKernelGGL(join, grid, dim3(256), 0, stream, a);
  }
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_attn_cache_workspace_bytes(const moe_attn_t* A, const moe_kv_cache_t* C,
                                                 int rows, int n_seqs) {
  if (!A || !C || !kv_sizes_ok(C) || !attn_sizes_ok(A, C) || rows <= 0 || n_seqs <= 0) return 0;
  int cus = device_cu_count();
  if (cus <= 0) cus = 256;
  return (size_t)attn_workspace(A, C, rows, n_seqs, cus);
}

extern "C" int moe_attn_cache(const moe_attn_t* A, const moe_kv_cache_t* C, const void* q,
                              int type, int64_t ld_q, int64_t hs_q, int rows,
                              const int32_t* q_offsets, int n_seqs, const int32_t* kv_lens,
                              const int32_t* table, int64_t ld_table, int max_pages,
                              const int32_t* prefix, void* out, int64_t ld_out, int64_t hs_out,
                              void* ws, size_t ws_bytes, void* stream) {
  if (!A) return MOE_ERR_INVALID_ARG;
  const int rc = kv_cache_check(C);
  if (rc != MOE_OK) return rc;
  if (!attn_sizes_ok(A, C)) return MOE_ERR_SHAPE;
  if (A->window < 0 || !__builtin_isfinite(A->scale) || !__builtin_isfinite(A->softcap) ||
      A->softcap < 0.f || rows < 0 || n_seqs < 0 || max_pages < 0 || !type_ok(type))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0 || n_seqs == 0) return MOE_OK;
  if (!q || !out || q == out || !kv_lens || (!table && max_pages)) return MOE_ERR_INVALID_ARG;
  if (!q_offsets && rows != n_seqs) return MOE_ERR_INVALID_ARG;
  if ((int64_t)max_pages * C->page >= ((int64_t)1 << 30) ||
      (int64_t)rows * (A->n_heads / C->n_heads) >= ((int64_t)1 << 28) || n_seqs > (1 << 24))
    return MOE_ERR_SHAPE;
  if (!head_strides_ok(ld_q, hs_q, rows, A->n_heads, C->head_dim) ||
      !head_strides_ok(ld_out, hs_out, rows, A->n_heads, C->head_dim) ||
      (n_seqs > 1 && ld_table < max_pages))
    return MOE_ERR_STRIDE;
  const size_t size = type_size(type);
  if (!aligned(q, size) || !aligned(out, size) || !aligned(kv_lens, 4) || !aligned(table, 4) ||
      (q_offsets && !aligned(q_offsets, 4)) || (prefix && !aligned(prefix, 4)) ||
      (A->slopes && !aligned(A->slopes, 4)))
    return MOE_ERR_ALIGNMENT;
  int cus = device_cu_count();
  if (cus <= 0) cus = 256;
  const AttnPlan p = attn_plan(A, C, type == MOE_TYPE_F32, rows, n_seqs,
                               (int64_t)max_pages * C->page, cus);
  const int64_t need = p.target ? 4 * part_floats(C, p.items, p.tile_rows, rows) : 0;
  if (need && !ws) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < (size_t)need) return MOE_ERR_WORKSPACE;
  if (need && !aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  AttnArgs a;
  a.q = q;
  a.out = out;
  a.data = (const uint8_t*)C->data;
  a.q_offsets = q_offsets;
  a.kv_lens = kv_lens;
  a.table = table;
  a.prefix = prefix;
  a.slopes = A->slopes;
  a.part = (float*)ws;
  a.ld_q = ld_q;
  a.hs_q = hs_q;
  a.ld_out = ld_out;
  a.hs_out = hs_out;
  a.ld_table = n_seqs > 1 ? ld_table : 0;
  a.ml_at = p.items * C->n_heads * p.tile_rows * C->head_dim;
  a.rec_at = a.ml_at + 2 * p.items * C->n_heads * p.tile_rows;
  a.rows = rows;
  a.n_seqs = n_seqs;
  a.n_heads = A->n_heads;
  a.kv_heads = C->n_heads;
  a.group = A->n_heads / C->n_heads;
  a.page_log = __builtin_ctz((unsigned)C->page);
  a.n_pages = C->n_pages;
  a.max_pages = max_pages;
  a.window = A->window;
  a.target = p.target;
  a.items = p.items;
  a.tile_log = __builtin_ctz((unsigned)p.tile_rows);
  a.group_inv = (uint32_t)((((uint64_t)1 << 32) / (uint32_t)a.group) + 1);
  a.quantum = p.quantum;
  a.scale = A->scale;
  a.softcap = A->softcap;
  const hipStream_t st = (hipStream_t)stream;
  const bool f32 = type == MOE_TYPE_F32;
  switch (C->head_dim) {
    case 64: f32 ? attn_launch<float, 64>(a, p, st) : attn_launch<__bf16, 64>(a, p, st); break;
    case 128: f32 ? attn_launch<float, 128>(a, p, st) : attn_launch<__bf16, 128>(a, p, st); break;
    default: f32 ? attn_launch<float, 256>(a, p, st) : attn_launch<__bf16, 256>(a, p, st); break;
  }
  return launch_status();
}
