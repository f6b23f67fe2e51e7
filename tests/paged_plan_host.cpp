// Host check of the work split of the paged attention kernels (paged_plan.cuh):
// the runs of all CTAs, walked the way the kernels walk them, visit every (KV
// head, sequence, tile, key tile) unit once and in order, whatever the lengths
// say, and nothing that a CTA would address lies outside the buffers.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using std::max;
using std::min;
static unsigned g_status;
static unsigned atomicCAS(unsigned* p, unsigned, unsigned v) { return *p = v; }
static unsigned __float_as_uint(float) { return 0; }  // named by the header, not called here
static void __nanosleep(unsigned) {}
#include "../long_context_tsa_b200/csrc/paged_plan.cuh"

using namespace tsa;

#define CHECK(x) \
  if (!(x)) { std::printf("case %d: %s\n", trial, #x); return 1; }

int main(int argc, char** argv) {
  std::mt19937 rng(argc > 1 ? std::atoi(argv[1]) : 1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int trial = 0; trial < 1000; ++trial) {
    Paged p = {};
    p.status = &g_status;
    g_status = 0;
    p.S = trial % 7 == 0 ? 1 : pick(1, 40);
    p.Hkv = 1 << pick(0, 3);
    p.g_log2 = pick(0, 4);
    p.G = 1 << p.g_log2;
    p.page_log2 = pick(4, 8);
    p.max_pages = pick(1, 40);
    const int cap = p.max_pages << p.page_log2;
    std::vector<int> len(p.S), start(p.S + 1);
    start[0] = pick(0, 3);
    for (int s = 0; s < p.S; ++s) {
      len[s] = pick(0, 3) ? pick(1, cap) : pick(1, min(cap, 300));
      start[s + 1] = start[s] + pick(0, pick(0, 1) ? min(len[s], 3) : len[s]);
    }
    p.T = start[p.S] + pick(0, 2);
    if (p.T == 0) p.T = 1;
    bool bad = false;
    if (trial % 3 == 0) {  // lengths and starts that are wrong
      bad = true;
      for (int k = 0; k < 3; ++k) {
        const int wild[] = {-5, 0, 1, cap + 1, 0x7fffffff, (int)0x80000000, pick(-cap, 2 * cap)};
        if (rng() & 1) len[rng() % p.S] = wild[rng() % 7];
        else start[rng() % (p.S + 1)] = wild[rng() % 7];
      }
    }
    p.seq_len = len.data();
    p.token_start = start.data();
    Plan pl;
    pl.which = pick(0, 2);
    pl.kt_log2 = pick(6, 7);
    pl.tt_log2 = pick(0, 8 - p.g_log2);

    struct Unit { int g, s, j, kt; };
    std::vector<Unit> all;
    std::vector<long long> seq(p.S);
    long long total = 0;
    for (int s = 0; s < p.S; ++s) {
      const Span sp = load_span(p, s);
      long long u = 0;
      if (pl.takes(p, sp.n))
        for (int j = 0; j < pl.tiles(sp.n); ++j) u += pl.units(sp, j);
      if (u) CHECK(u == pl.seq_units(sp));
      seq[s] = u;
      total += u;
    }
    if (!bad) CHECK(g_status == 0);
    for (int g = 0; g < p.Hkv; ++g)
      for (int s = 0; s < p.S; ++s) {
        const Span sp = load_span(p, s);
        if (!pl.takes(p, sp.n)) continue;
        for (int j = 0; j < pl.tiles(sp.n); ++j)
          for (int k = 0; k < pl.units(sp, j); ++k) all.push_back({g, s, j, k});
      }
    const int ctas = pick(0, 1) ? 148 : 296;
    const long long units = total * p.Hkv, run = (units + ctas - 1) / ctas;
    CHECK(units == (long long)all.size());
    size_t at = 0;
    for (int b = 0; b < ctas; ++b) {
      const long long u0 = run * b, u1 = min(u0 + run, units);
      long long left = max(0LL, u1 - u0);
      if (!left) continue;
      Cursor c;
      c.g = (int)(u0 / total);
      long long r = u0 - c.g * total;
      for (c.s = 0; r >= seq[c.s]; ++c.s) r -= seq[c.s];
      plan_seek(p, pl, &c, r);
      while (left > 0) {
        const int n = pl.units(c.span, c.j), keys = pl.keys(c.span, c.j);
        const int kt1 = (int)min((long long)n, c.kt + left);
        CHECK(kt1 > c.kt);
        CHECK(keys >= 0 && keys <= cap);  // every key below `keys` has an entry in the table's row
        const int first = c.j << pl.tt_log2, n_tok = min(1 << pl.tt_log2, c.span.n - first);
        CHECK(n_tok > 0 && c.span.tok0 + first >= 0 && (long long)c.span.tok0 + first + n_tok <= p.T);
        for (int k = c.kt; k < kt1; ++k, ++at) {
          CHECK(at < all.size());
          CHECK(all[at].g == c.g && all[at].s == c.s && all[at].j == c.j && all[at].kt == k);
        }
        if (kt1 < n) {  // the CTAs that continue the tile
          const int end = b + (int)((n - kt1 + run - 1) / run);
          CHECK(end < ctas);
        }
        left -= kt1 - c.kt;
        if (left > 0) plan_next(p, pl, &c);
      }
    }
    CHECK(at == all.size());
    for (int e : {-1, p.n_pages, 0x7fffffff}) CHECK(checked_page(p, e) == 0);
  }
  std::printf("ok\n");
  return 0;
}
