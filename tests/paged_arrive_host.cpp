// Host check of the counts by which the paged attention kernels find the last part of a cut tile
// (paged_arrive.cuh): over random lists of tiles, cut into runs as the kernels cut them, and random
// orders of arrival, every cut tile has exactly one last part, which is the last to arrive; the counts
// are 0 afterwards; and only header words from 2 on are touched.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

static unsigned atomicXor(unsigned* p, unsigned v) { const unsigned o = *p; *p ^= v; return o; }
static unsigned atomicAdd(unsigned* p, unsigned v) { const unsigned o = *p; *p += v; return o; }
static unsigned atomicSub(unsigned* p, unsigned v) { const unsigned o = *p; *p -= v; return o; }
#include "../long_context_tsa_b200/csrc/paged_arrive.cuh"

using namespace tsa;

#define CHECK(x) \
  if (!(x)) { std::printf("case %d: %s\n", trial, #x); return 1; }

int main(int argc, char** argv) {
  std::mt19937 rng(argc > 1 ? std::atoi(argv[1]) : 1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  uint32_t header[kHeaderWords + 2] = {};
  uint32_t* words = header + 1;  // a word on either side that must stay 0
  for (int trial = 0; trial < 3000; ++trial) {
    const int ctas = pick(0, 1) ? kPagedCtas : 2 * kPagedCtas;
    std::vector<int> units;  // of each tile
    const int tiles = trial % 5 == 0 ? 1 : pick(1, 400), most = 1 << pick(0, 10);
    long long all = 0;
    for (int i = 0; i < tiles; ++i) {
      units.push_back(pick(1, most));
      all += units.back();
    }
    const long long run = (all + ctas - 1) / ctas;
    struct Part { Owners own; int tile; };
    std::vector<Part> parts;
    std::vector<int> want(tiles, 0), last(tiles, 0);
    long long at = 0;
    for (int i = 0; i < tiles; ++i) {
      const long long first = at / run, end = (at + units[i] - 1) / run;
      if (end > first)
        for (long long c = first; c <= end; ++c) {  // the part of CTA c: its place in the list, and in the tile
          const long long upos = std::max(at, c * run);
          const Owners own = tile_owners(upos, (int)(upos - at), units[i], run);
          CHECK(own.first == first && own.n == end - first + 1 && end < ctas);
          parts.push_back({own, i});
          ++want[i];
        }
      at += units[i];
    }
    std::shuffle(parts.begin(), parts.end(), rng);
    for (const Part& p : parts) {
      --want[p.tile];
      const bool is_last = part_arrives(words, p.own);
      CHECK(is_last == (want[p.tile] == 0));
      last[p.tile] += is_last;
      CHECK(header[0] == 0 && words[0] == 0 && words[1] == 0 && header[kHeaderWords + 1] == 0);
    }
    for (const Part& p : parts) CHECK(last[p.tile] == 1);
    for (uint32_t w : header) CHECK(w == 0);
  }
  std::printf("ok\n");
  return 0;
}
