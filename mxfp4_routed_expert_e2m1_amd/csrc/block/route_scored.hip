// route_scored.hip -- routing by a scoring rule: softmax or sigmoid scores, a
// balance bias for the choice alone, expert groups, top-k, weights, and the
// stable grouping by expert.
//
// One wave per row.  A lane holds PER_LANE consecutive experts as
// order-preserving integer keys (0: out of reach or already picked), so a round
// is each lane's first largest key, the wave's maximum, and the first lane that
// holds it: the lowest expert among equals.  A row's time is this chain of
// dependent steps, 0.2 us a round.
//
// Grouping.  An expert takes a row at most once, so the rows that chose it are
// a bit set: an assignment's place among its expert's is the number of
// earlier rows in the set.  The sets are built with LDS ORs, whose order does
// not matter, and the result is the unique stable one.  Decode-sized calls do
// all of it in one workgroup.  Larger ones take two launches: the first
// counts each expert in every run of rows, the second turns the counts of the
// earlier runs into first positions and places its own rows, 64 at a time.
// Up to about a thousand rows it is bound by latency, of launches and of the
// picks' chain (0.18 us a pick), not by its bytes: one row of 256 experts, top 6,
// takes 4.6 us, 777 rows of 160, top 6, 5.3 + 5.7 us.  At 4096 rows of 256, top 8
// (7.6 + 5.8 us), four waves share each SIMD in the first launch and the picks'
// instructions count too.
#include "block.h"

#include <math.h>

namespace moe {

constexpr int kRuleMaxExperts = 512;
constexpr int kRuleMaxGroups = 64;
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kSmallRows = 2 * kRouteWaves;  // rows that one workgroup routes and groups alone

struct RuleArgs {
  const void* logits;
  int l_type;
  int64_t ld_l;
  int rows, n_experts, top_k, n_groups, top_groups, group_size, score, group_score, renorm;
  uint32_t group_inv;  // ceil(2^20 / group_size): e / group_size = e * group_inv >> 20
  int lanes_log2;      // lanes that share a group's reduction
  float scale;
  const float* bias;
  int32_t* ids;
  float* w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* sorted;
};

// exp_rows (the same operations on the same values, so the same bits) without
// a branch: a lane's several scores are computed side by side.
__device__ inline float exp_flat(float x) {
  const float c = fminf(fmaxf(x, -104.0f), 89.0f);
  const float k = rintf(c * 0x1.715476p+0f);
  float r = fmaf(-k, 0x1.62e4p-1f, c);
  r = fmaf(-k, 0x1.7f7d1cp-20f, r);
  float p = 0x1.a01a02p-13f;
  p = fmaf(p, r, 0x1.6c16c2p-10f);
  p = fmaf(p, r, 0x1.111112p-7f);
  p = fmaf(p, r, 0x1.555556p-5f);
  p = fmaf(p, r, 0x1.555556p-3f);
  p = fmaf(p, r, 0x1p-1f);
  p = fmaf(p, r, 1.0f);
  p = fmaf(p, r, 1.0f);
  const float e = ldexpf(p, (int)k);
  return x > 89.0f ? __builtin_inff() : x >= -104.0f ? e : 0.0f;
}

template <int CTRL>
__device__ inline uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}

// Maximum over the wave, wave-uniform.  (Lanes that a step does not reach take
// part with 0, the least key, so that each step is one instruction.)
template <int CTRL, int ROWS>
__device__ inline uint32_t max_step(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true));
}
__device__ inline uint32_t wave_max_key(uint32_t v) {
  v = max_step<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
  v = max_step<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
  v = max_step<0x141, 0xF>(v);  // row_half_mirror
  v = max_step<0x140, 0xF>(v);  // row_mirror
  v = max_step<0x142, 0xA>(v);  // row_bcast:15 into rows 1, 3
  v = max_step<0x143, 0xC>(v);  // row_bcast:31 into rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A lane's experts e0.. of a row of E, as floats, in one load where all are in
// the row; 0 past it.
template <int N, typename T>
__device__ inline void load_lane(const T* row, int e0, int E, float (&v)[N]) {
  T t[N];
  if (e0 + N <= E) {
    __builtin_memcpy(t, row + e0, sizeof(t));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = e0 + j < E ? row[e0 + j] : (T)0.f;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = (float)t[j];
}

// The picks of one row: lane s < top_k gets pick s (-1: none left) and its
// weight.  `lds` holds 64 * PER_LANE words of this wave.
template <int PER_LANE>
__device__ inline void choose_row(const RuleArgs& p, int row, uint32_t* lds, int* my_id,
                                  float* my_w) {
  const int lane = lane_id(), E = p.n_experts, e0 = PER_LANE * lane;
  float l[PER_LANE], s[PER_LANE], b[PER_LANE];
  if (p.l_type == MOE_TYPE_F32)
    load_lane<PER_LANE>((const float*)p.logits + (int64_t)row * p.ld_l, e0, E, l);
  else
    load_lane<PER_LANE>((const __bf16*)p.logits + (int64_t)row * p.ld_l, e0, E, l);
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) b[j] = 0.f;
  if (p.bias) load_lane<PER_LANE>(p.bias, e0, E, b);
  bool in[PER_LANE];
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j)
    in[j] = e0 + j < E && l[j] > -__builtin_inff();  // not NaN either
  if (p.score == MOE_SCORE_SOFTMAX) {
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j)
      if (in[j]) m = fmaxf(m, l[j]);
    m = wave_max(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      // (an infinite maximum: its holders share, the others get 0)
      const float e = exp_flat(l[j] - m);
      s[j] = !in[j] ? 0.f : l[j] == m ? 1.f : e;
      sum += s[j];
    }
    sum = wave_sum(sum);  // (0 where no expert is in reach: the quotients are not used)
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const float q = s[j] / sum;
      s[j] = in[j] ? q : 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const float q = 1.0f / (1.0f + exp_flat(-l[j]));
      s[j] = in[j] ? q : 0.f;
    }
  }
  uint32_t k[PER_LANE];
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) k[j] = in[j] ? logit_key(s[j] + b[j]) : 0u;

  if (p.n_groups > 1 && p.top_groups < p.n_groups) {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) lds[e0 + j] = k[j];
    __builtin_amdgcn_wave_barrier();
    // group g's lanes are g << lanes_log2 on; each reads every 2^lanes_log2-th
    // member, four at a time, then the lanes' two largest are merged
    const int P = 1 << p.lanes_log2, g = lane >> p.lanes_log2;
    uint32_t k1 = 0, k2 = 0;
    for (int i0 = lane & (P - 1); i0 < p.group_size; i0 += 4 * P) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * P;
        v[u] = g < p.n_groups && i < p.group_size ? lds[g * p.group_size + i] : 0u;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        k2 = max(k2, min(k1, v[u]));
        k1 = max(k1, v[u]);
      }
    }
    auto merge = [&](uint32_t o1, uint32_t o2) {
      k2 = max(min(k1, o1), max(k2, o2));
      k1 = max(k1, o1);
    };
    // (lanes that have merged hold the same pair, so a mirror is a swap)
    if (P >= 2) merge(dpp_u32<0xB1>(k1), dpp_u32<0xB1>(k2));    // quad_perm [1,0,3,2]
    if (P >= 4) merge(dpp_u32<0x4E>(k1), dpp_u32<0x4E>(k2));    // quad_perm [2,3,0,1]
    if (P >= 8) merge(dpp_u32<0x141>(k1), dpp_u32<0x141>(k2));  // row_half_mirror
    if (P >= 16) merge(dpp_u32<0x140>(k1), dpp_u32<0x140>(k2));  // row_mirror
    if (P >= 32) merge(__shfl_xor(k1, 16, 64), __shfl_xor(k2, 16, 64));
    uint32_t gk = k1;
    if (p.group_score == MOE_GROUP_TOP2 && k2 != 0)
      gk = logit_key(logit_of_key(k1) + logit_of_key(k2));
    // a group stays if fewer than top_groups groups come before it
    int before = 0;
    for (int h = 0; h < p.n_groups; ++h) {
      const uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)gk, h << p.lanes_log2);
      before += (v > gk || (v == gk && h < g)) ? 1 : 0;
    }
    const uint64_t stays = __ballot(g < p.n_groups && gk != 0 && before < p.top_groups);
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const uint32_t mine = ((uint32_t)(e0 + j) * p.group_inv) >> 20;
      if (mine >= (uint32_t)p.n_groups || !((stays >> (mine << p.lanes_log2)) & 1)) k[j] = 0u;
    }
  }

  // the scores wait in LDS for the picks
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) lds[e0 + j] = __builtin_bit_cast(uint32_t, s[j]);
  int id = -1;
  for (int r = 0; r < p.top_k; ++r) {
    uint32_t most = k[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < PER_LANE; ++j) {
      at = k[j] > most ? j : at;
      most = max(most, k[j]);
    }
    const uint32_t best = wave_max_key(most);
    if (best == 0u) break;  // none left: the remaining slots keep -1
    const int first = __ffsll((unsigned long long)__ballot(most == best)) - 1;
    const int pick = PER_LANE * first + __builtin_amdgcn_readlane(at, first);
    const int gone = lane == first ? at : -1;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) k[j] = gone == j ? 0u : k[j];
    id = lane == r ? pick : id;
  }
  __builtin_amdgcn_wave_barrier();
  float w = id >= 0 ? __builtin_bit_cast(float, lds[id]) : 0.f;
  __builtin_amdgcn_wave_barrier();
  if (p.renorm) {
    float sum = 0.f;
    for (int r = 0; r < p.top_k; ++r)
      sum += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), r));
    if (sum > 0.f) w = w / sum;
  }
  *my_id = id;
  *my_w = w * p.scale;
}

// Exclusive scan over the experts of `c` (thread e < n_experts holds expert
// e's count) in a workgroup of kRouteThreads; returns this thread's, and the
// total.  `slots` is LDS of one int per wave.
__device__ inline int expert_scan(int c, int* slots, int* total) {
  const int incl = wave_incl_scan(c), wave = threadIdx.x >> 6;
  if (lane_id() == 63) slots[wave] = incl;
  __syncthreads();
  int base = 0, all = 0;
  for (int i = 0; i < kRouteWaves; ++i) {
    const int t = slots[i];
    base += i < wave ? t : 0;
    all += t;
  }
  *total = all;
  return base + incl - c;
}

// Few rows (decode): choice and grouping in one workgroup, two rows per wave at
// most.
template <int PER_LANE>
__global__ __launch_bounds__(kRouteThreads) void route_small_kernel(RuleArgs p) {
  __shared__ uint32_t keys[kRouteWaves][64 * PER_LANE];
  __shared__ int ids[kSmallRows * MOE_MAX_TOP_K];
  __shared__ uint32_t rows_of[kRuleMaxExperts];
  __shared__ int first[kRuleMaxExperts];
  __shared__ int slots[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.rows * p.top_k;
  if (tid < p.n_experts) rows_of[tid] = 0;
  for (int row = wave; row < p.rows; row += kRouteWaves) {
    int id;
    float w;
    choose_row<PER_LANE>(p, row, keys[wave], &id, &w);
    if (lane < p.top_k) {
      const int a = row * p.top_k + lane;
      p.ids[a] = id;
      p.w[a] = w;
      ids[a] = id;
    }
  }
  __syncthreads();
  const int e = tid < n ? ids[tid] : -1, row = tid / p.top_k;
  if (e >= 0) atomicOr(&rows_of[e], 1u << row);
  __syncthreads();
  const int c = tid < p.n_experts ? __popc(rows_of[tid]) : 0;
  int total;
  const int at = expert_scan(c, slots, &total);
  if (tid < p.n_experts) {
    p.counts[tid] = c;
    p.offsets[tid] = at;
    first[tid] = at;
  }
  if (tid == 0) p.offsets[p.n_experts] = total;
  __syncthreads();
  if (e >= 0) p.sorted[first[e] + __popc(rows_of[e] & ((1u << row) - 1))] = tid;
  if (tid >= total && tid < n) p.sorted[tid] = -1;
}

// More rows, launch 1: run b (rows b*run_rows on) writes its rows' picks and
// how many of them chose each expert, hist[b][e].
template <int PER_LANE, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void route_choose_kernel(RuleArgs p, int run_rows,
                                                                  uint16_t* hist, int hist_ld) {
  __shared__ uint32_t keys[WAVES][64 * PER_LANE];
  __shared__ int count[kRuleMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < hist_ld; e += 64 * WAVES) count[e] = 0;
  __syncthreads();
  const int r1 = min(p.rows, ((int)blockIdx.x + 1) * run_rows);
  for (int row = blockIdx.x * run_rows + wave; row < r1; row += WAVES) {
    int id;
    float w;
    choose_row<PER_LANE>(p, row, keys[wave], &id, &w);
    if (lane < p.top_k) {
      p.ids[(int64_t)row * p.top_k + lane] = id;
      p.w[(int64_t)row * p.top_k + lane] = w;
      if (id >= 0) atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < hist_ld; e += 64 * WAVES)
    hist[(int64_t)blockIdx.x * hist_ld + e] = (uint16_t)count[e];
}

// Launch 2: workgroup g places the rows of runs [g * group_runs, ..).
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(
    RuleArgs p, int run_rows, int n_runs, int group_runs, const uint16_t* __restrict__ hist,
    int hist_ld) {
  __shared__ int total_of[kRuleMaxExperts], next[kRuleMaxExperts];
  __shared__ unsigned long long rows_of[kRuleMaxExperts];
  __shared__ int slots[kRouteWaves];
  const int tid = threadIdx.x;
  const int run0 = blockIdx.x * group_runs;
  const int r0 = run0 * run_rows, r1 = min(p.rows, (run0 + group_runs) * run_rows);
  // (the first 64 rows' ids: on their way while the counts are read)
  const bool early = tid < 64 * p.top_k && r0 + tid / p.top_k < r1;
  int e = early ? p.ids[(int64_t)r0 * p.top_k + tid] : -1;
  for (int x = tid; x < kRuleMaxExperts; x += kRouteThreads) {
    total_of[x] = next[x] = 0;
    rows_of[x] = 0;
  }
  __syncthreads();
  // counts over all runs and over the runs before this workgroup's: eight
  // experts per thread, every strips-th run, eight runs' loads at a time
  const int cols = hist_ld / 8, strips = kRouteThreads / cols;
  const int col = tid % cols, strip = tid / cols;
  if (strip < strips) {
    int t[8] = {}, b[8] = {};
    for (int r8 = strip; r8 < n_runs; r8 += 8 * strips) {
      u32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = ((const u32x4*)hist)[(int64_t)min(r8 + u * strips, n_runs - 1) * cols + col];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = r8 + u * strips;
        const uint32_t in = r < n_runs ? ~0u : 0u, earlier = r < run0 ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = (v[u][i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
          t[i] += (int)(x & in);
          b[i] += (int)(x & earlier);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      atomicAdd(&total_of[8 * col + i], t[i]);
      if (b[i] != 0) atomicAdd(&next[8 * col + i], b[i]);
    }
  }
  __syncthreads();
  const int c = tid < p.n_experts ? total_of[tid] : 0;
  int total;
  const int at = expert_scan(c, slots, &total);
  if (tid < p.n_experts) {
    next[tid] += at;
    if (blockIdx.x == 0) {
      p.counts[tid] = c;
      p.offsets[tid] = at;
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.n_experts] = total;
  __syncthreads();
  for (int rb = r0; rb < r1; rb += 64) {
    // one thread per assignment of 64 rows: at most 64 * MOE_MAX_TOP_K
    const int row = rb + tid / p.top_k;
    const bool mine = tid < 64 * p.top_k && row < r1;
    const int64_t a = (int64_t)rb * p.top_k + tid;
    if (rb > r0) e = mine ? p.ids[a] : -1;
    if (e >= 0) atomicOr(&rows_of[e], 1ull << (row - rb));
    __syncthreads();
    if (e >= 0)
      p.sorted[next[e] + __popcll(rows_of[e] & ((1ull << (row - rb)) - 1))] = (int)a;
    if (mine && a >= total) p.sorted[a] = -1;
    if (rb + 64 >= r1) break;
    __syncthreads();
    if (tid < p.n_experts) {
      next[tid] += __popcll(rows_of[tid]);
      rows_of[tid] = 0;
    }
    __syncthreads();
  }
}

__global__ void route_none_kernel(int n_experts, int32_t* counts, int32_t* offsets) {
  for (int e = threadIdx.x; e <= n_experts; e += blockDim.x) {
    if (e < n_experts) counts[e] = 0;
    offsets[e] = 0;
  }
}

// ------------------------------------------------------------- host side
static int rule_check(const moe_router_rule_t* R) {
  if (!R) return MOE_ERR_INVALID_ARG;
  if (R->n_experts < 1 || R->n_experts > kRuleMaxExperts) return MOE_ERR_SHAPE;
  if (R->n_groups < 1 || R->n_groups > kRuleMaxGroups || R->n_experts % R->n_groups != 0 ||
      R->top_groups < 1 || R->top_groups > R->n_groups)
    return MOE_ERR_SHAPE;
  if (R->top_k < 1 || R->top_k > MOE_MAX_TOP_K ||
      R->top_k > R->top_groups * (R->n_experts / R->n_groups))
    return MOE_ERR_SHAPE;
  if ((R->score != MOE_SCORE_SOFTMAX && R->score != MOE_SCORE_SIGMOID) ||
      (R->group_score != MOE_GROUP_MAX && R->group_score != MOE_GROUP_TOP2) ||
      (R->renorm != 0 && R->renorm != 1) || !isfinite(R->scale))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(R->bias, 4)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Runs of launch 1: 4 rows each, a wave per row and SIMD, up to 1024 rows (a
// wave's work is long, so waves are better apart: 777 rows 7.7 -> 5.2 us), 16
// rows beyond, and longer past 8192 rows, so that there are never more than
// 512 (a run's count of an expert, at most 2^24 / 512 rows, fits 16 bits).
// Launch 2 takes 64 rows or more, four or sixteen runs, per workgroup.
struct RouteShape {
  int waves, run_rows, n_runs, group_runs, hist_ld;
};
static RouteShape route_shape(int n_experts, int rows) {
  RouteShape s;
  s.waves = rows <= 1024 ? 4 : kRouteWaves;
  const int m = (rows + 512 * s.waves - 1) / (512 * s.waves);
  s.run_rows = s.waves * m;
  s.n_runs = (rows + s.run_rows - 1) / s.run_rows;
  s.group_runs = 64 / s.waves;
  s.hist_ld = (n_experts + 7) / 8 * 8;
  return s;
}

// Workspace of a call: its runs' counts (all that is not decode has one, also
// where one workgroup does without).
static size_t route_bytes(int n_experts, int64_t runs) {
  return (size_t)runs * ((n_experts + 7) / 8 * 8) * sizeof(uint16_t);
}
static size_t route_need(int n_experts, int rows) {
  return rows <= MOE_MAX_DECODE_ROWS ? 0 : route_bytes(n_experts, route_shape(n_experts, rows).n_runs);
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_scored_workspace_bytes(const moe_router_rule_t* R, int rows) {
  if (rule_check(R) != MOE_OK || rows <= MOE_MAX_DECODE_ROWS) return 0;
  // the most runs that as many rows or fewer come in: 4 rows each up to 1024
  // rows, then 16 each up to 8192 (512 runs), then fewer
  const int64_t runs = rows <= 1024 ? (rows + 3) / 4 : max(256, min(512, (rows - 1) / 16 + 1));
  return route_bytes(R->n_experts, runs);
}

extern "C" int moe_route_scored(const moe_router_rule_t* R, const void* logits, int l_type,
                                int64_t ld_l, int rows, int32_t* ids, float* w, int32_t* counts,
                                int32_t* offsets, int32_t* sorted, void* ws, size_t ws_bytes,
                                void* stream) {
  const int rc = rule_check(R);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !type_ok(l_type) || !counts || !offsets) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!logits || !ids || !w || !sorted)) return MOE_ERR_INVALID_ARG;
  if ((int64_t)rows * R->top_k > (1 << 24)) return MOE_ERR_SHAPE;
  if (rows > 0 && ld_l < R->n_experts) return MOE_ERR_STRIDE;
  if (!aligned(counts, 4) || !aligned(offsets, 4) ||
      (rows > 0 && (!aligned(logits, type_size(l_type)) || !aligned(ids, 4) || !aligned(w, 4) ||
                    !aligned(sorted, 4))))
    return MOE_ERR_ALIGNMENT;
  const size_t need = route_need(R->n_experts, rows);
  if (need > 0) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  }
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  hipStream_t s = (hipStream_t)stream;
  if (rows == 0) {
    hipLaunchKernelGGL(route_none_kernel, dim3(1), dim3(256), 0, s, R->n_experts, counts,
                       offsets);
    return launch_status();
  }
  RuleArgs p{};
  p.logits = logits;
  p.l_type = l_type;
  p.ld_l = ld_l;
  p.rows = rows;
  p.n_experts = R->n_experts;
  p.top_k = R->top_k;
  p.n_groups = R->n_groups;
  p.top_groups = R->top_groups;
  p.group_size = R->n_experts / R->n_groups;
  p.score = R->score;
  p.group_score = R->group_score;
  p.renorm = R->renorm;
  p.group_inv = (uint32_t)(((1 << 20) + p.group_size - 1) / p.group_size);
  p.lanes_log2 = 0;
  while ((R->n_groups << (p.lanes_log2 + 1)) <= 64) ++p.lanes_log2;
  p.scale = R->scale;
  p.bias = R->bias;
  p.ids = ids;
  p.w = w;
  p.counts = counts;
  p.offsets = offsets;
  p.sorted = sorted;
  const int per_lane = (R->n_experts + 63) / 64;
  // one launch for a row per wave, or for two where a row is short (18 rows of
  // 8 experts take 13.5 us in two launches; 28 rows of 272 take 16.3 in one and
  // 12.1 in two)
  if (rows <= kRouteWaves || (rows <= kSmallRows && per_lane <= 2)) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(1), dim3(kRouteThreads), 0, s, p);
    };
    if (per_lane <= 2) go(route_small_kernel<2>);
    else if (per_lane <= 4) go(route_small_kernel<4>);
    else go(route_small_kernel<8>);
    return launch_status();
  }
  const RouteShape sh = route_shape(R->n_experts, rows);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(sh.n_runs), dim3(64 * sh.waves), 0, s, p, sh.run_rows,
                       (uint16_t*)ws, sh.hist_ld);
  };
  if (sh.waves == 4) {
    if (per_lane <= 2) go(route_choose_kernel<2, 4>);
    else if (per_lane <= 4) go(route_choose_kernel<4, 4>);
    else go(route_choose_kernel<8, 4>);
  } else {
    if (per_lane <= 2) go(route_choose_kernel<2, kRouteWaves>);
    else if (per_lane <= 4) go(route_choose_kernel<4, kRouteWaves>);
    else go(route_choose_kernel<8, kRouteWaves>);
  }
  hipLaunchKernelGGL(route_place_kernel, dim3((sh.n_runs + sh.group_runs - 1) / sh.group_runs),
                     dim3(kRouteThreads), 0, s, p, sh.run_rows, sh.n_runs, sh.group_runs,
                     (const uint16_t*)ws, sh.hist_ld);
  return launch_status();
}
