// Counting the parts of a cut tile, so that the last CTA to leave one knows it.
//
// The counts are in the workspace's header, which all calls of the library leave
// alone and which is 0 between calls: one workspace may serve any of them in turn.
// Its 64 words hold the counts of 2 * 148 CTAs because few tiles can be cut at once:
// a CTA begins at most one tile that others continue, and one with three or more
// parts covers the CTA after its first.  So CTAs 2i and 2i + 1 between them need one
// field that counts to n, and one bit for a tile of two parts that 2i begins (the
// second part finds it set and clears it).
#pragma once

#include "paged.h"

namespace tsa {

// The CTAs with a part of the tile that the cursor is at: `upos` is the cursor's place in the list of units.
struct Owners {
  int first, n;
};
__device__ __forceinline__ Owners tile_owners(long long upos, int kt, int units, long long run) {
  Owners o;
  o.first = (int)((upos - kt) / run);
  o.n = (int)((upos - kt + units - 1) / run) - o.first + 1;
  return o;
}

struct ArrivalSlot {
  int word, shift;
  bool toggle;
};
constexpr int kBitWords = (kPagedCtas + 31) / 32, kFieldBits = 10;
constexpr int kBitWord0 = 2, kFieldWord0 = kBitWord0 + kBitWords;
static_assert(kFieldWord0 + (kPagedCtas + 2) / 3 <= kHeaderWords, "counts in the header");
static_assert(2 * kPagedCtas < 1 << kFieldBits, "a count of all CTAs");
__device__ __forceinline__ ArrivalSlot arrival_slot(const Owners& own) {
  const int pair = own.first >> 1;
  if (own.n == 2 && (own.first & 1) == 0) return {kBitWord0 + pair / 32, pair % 32, true};
  return {kFieldWord0 + pair / 3, pair % 3 * kFieldBits, false};
}

// Notes that a part is there; true for the last one, which leaves the field at 0.
__device__ __forceinline__ bool part_arrives(uint32_t* header, const Owners& own) {
  const ArrivalSlot at = arrival_slot(own);
  if (at.toggle) return (atomicXor(header + at.word, 1u << at.shift) >> at.shift & 1u) != 0;
  const uint32_t there = atomicAdd(header + at.word, 1u << at.shift) >> at.shift & ((1u << kFieldBits) - 1);
  if (there != (uint32_t)own.n - 1) return false;
  atomicSub(header + at.word, (uint32_t)own.n << at.shift);
  return true;
}

}  // namespace tsa
