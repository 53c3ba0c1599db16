// attn_cut_check.cpp -- the cut of the attention's work, from the header that the kernels take it from,
// over lengths of up to 2^30 tokens: a call's pieces have workgroups, and its parts have workspace.
// Host code alone.  Prints what failed, and "ok N cut calls of M".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../mxfp4_routed_expert_e2m1_amd/csrc/block/attn_plan.h"

using namespace moe;

static uint64_t seed = 1;
static uint64_t draw(uint64_t below) {
  seed = seed * 6364136223846793005ull + 1442695040888963407ull;
  return (uint64_t)(((unsigned __int128)(seed ^ seed >> 33) * below) >> 64);
}
static int64_t spread(int64_t most) {  // 1..most, over its logarithm
  const int bits = 64 - __builtin_clzll((uint64_t)most);
  const int64_t top = (int64_t)1 << (1 + draw(bits)), v = 1 + (int64_t)draw(top);
  return v < most ? v : most;
}

struct Call {
  bool f32;
  moe_attn_t A;
  moe_kv_cache_t C;
  std::vector<int> rows, lens;  // of the sequences
  int64_t tokens;               // that the table has room for
};

// 1: cut, 0: not, -1: wrong
static int check(const Call& c) {
  int64_t rows = 0;
  for (int m : c.rows) rows += m;
  const int64_t n_seqs = (int64_t)c.rows.size();
  const int cus = 256;
  const AttnPlan p = attn_plan(&c.A, &c.C, c.f32, rows, n_seqs, c.tokens, cus);
  if (p.target == 0) return 0;
  const int64_t group = c.A.n_heads / c.C.n_heads;
  int64_t work = 0, all = 0;
  std::vector<int> tiles, span;
  for (size_t s = 0; s < c.rows.size(); ++s) {
    const int64_t first = c.A.window > 0 ? (int64_t)c.lens[s] - c.rows[s] - c.A.window + 1 : 0;
    tiles.push_back((int)((c.rows[s] * group + p.tile_rows - 1) / p.tile_rows));
    span.push_back(c.lens[s] - (first > 0 ? (int)first & ~(kStep - 1) : 0));
    work += steps_of(tiles[s], span[s]);
    all += tiles[s];
  }
  const auto count = [&](int cut) {
    int64_t n = 0;
    for (size_t s = 0; s < tiles.size(); ++s) n += (int64_t)tiles[s] * pieces_of(span[s], cut);
    return n;
  };
  const int cut = choose_cut(work, all, p.target, p.quantum, n_seqs <= 64, count);
  bool ok = cut >= p.quantum && cut % p.quantum == 0 && cut <= 0x40000000 && count(cut) <= p.items;
  for (size_t s = 0; s < tiles.size(); ++s)
    ok = ok && (int64_t)pieces_of(span[s], cut) * cut >= span[s];
  const int64_t need = 4 * part_floats(&c.C, p.items, p.tile_rows, rows);
  ok = ok && need <= attn_workspace(&c.A, &c.C, rows, n_seqs, cus);
  if (!ok)
    printf("%s, %d heads on %d of %d, %lld rows in %lld sequences, %lld tokens: cut %d, %lld pieces for %lld "
           "items\n", c.f32 ? "f32" : "bf16", c.A.n_heads, c.C.n_heads, c.C.head_dim, (long long)rows,
           (long long)n_seqs, (long long)c.tokens, cut, (long long)count(cut), (long long)p.items);
  return ok ? 1 : -1;
}

int main(int argc, char** argv) {
  const int n = argc > 1 ? atoi(argv[1]) : 1000;
  int cut = 0, wrong = 0;
  const auto take = [&](const Call& c) {
    const int r = check(c);
    cut += r != 0;
    wrong += r < 0;
  };
  // work past 2^25 and past 2^31 steps, of one text and of many
  take({true, {16, 0, 1.f, 0.f, nullptr}, {1, 64, 256, 1 << 20, nullptr}, {2800}, {12582912}, 12582912});
  take({true, {8, 0, 1.f, 0.f, nullptr}, {1, 64, 256, 1 << 20, nullptr}, std::vector<int>(13, 299),
        std::vector<int>(13, 14900000), 14900224});
  take({true, {16, 0, 1.f, 0.f, nullptr}, {1, 128, 256, 1 << 20, nullptr}, {1800}, {1 << 24}, 1 << 24});
  take({false, {1, 0, 1.f, 0.f, nullptr}, {1, 64, 256, 1 << 20, nullptr}, std::vector<int>(700, 1),
        std::vector<int>(700, (1 << 30) - 256), (1 << 30) - 256});
  for (int i = 0; i < n; ++i) {
    Call c;
    c.f32 = draw(2);
    c.C = {1 << draw(4), 64 << draw(3), 16 << draw(5), 1 << 20, nullptr};
    c.A = {c.C.n_heads * (int)spread(64), draw(4) ? 0 : (int)spread(1 << 30), 1.f, 0.f, nullptr};
    const int64_t most = ((int64_t)1 << 30) - c.C.page;
    c.tokens = spread(most) / c.C.page * c.C.page + c.C.page;
    const int n_seqs = (int)spread(draw(2) ? 4 : 900);
    const int64_t each = spread(4096);
    for (int s = 0; s < n_seqs; ++s) {
      c.rows.push_back((int)(draw(3) ? spread(each) - 1 : each));
      c.lens.push_back((int)(draw(3) ? draw(c.tokens + 1) : draw(8) ? c.tokens : spread(c.tokens)));
    }
    int64_t rows = 0;
    for (int m : c.rows) rows += m;
    if (rows) take(c);
  }
  if (wrong) printf("%d wrong\n", wrong);
  else printf("ok %d cut calls of %d\n", cut, n + 4);
  return wrong != 0;
}
