// Work split of the paged attention kernels.
//
// An item is one tile of new tokens (TT = tile rows / G tokens) of one sequence
// for one KV head; its work is the number of key tiles (units of KT keys) that
// its last token sees.  The items, in the order KV head, sequence, tile, form
// one list of units that is cut into equal runs, one for each CTA: lengths may
// be as uneven as they like and every CTA still gets the same number of key
// tiles, read from the device's own seq_len and token_start (a captured call
// follows them).  A tile that a run's end cuts leaves unnormalised partial
// results, joined in the order of the CTAs (by a second kernel for paged_chunk,
// by the last CTA to finish the tile for the others), so the result does not
// depend on timing.
#pragma once

#include "device_common.cuh"
#include "paged.h"

namespace tsa {

struct Span {
  int tok0;  // packed row of the first new token
  int n;     // new tokens
  int base;  // position of the first new token
  int len;   // cached tokens, the new ones among them, clamped to what the table's row can hold
};

// Sequence s.  Entries outside the packed rows or the table are device bounds
// errors; they are clamped so that nothing outside the buffers is addressed.
__device__ __forceinline__ Span load_span(const Paged& p, int s) {
  const int a = p.token_start[s], b = p.token_start[s + 1];
  const int len = p.seq_len[s];
  Span r;
  r.tok0 = a;
  r.n = b - a;
  r.len = len;
  if (a < 0 || b < a || b > p.T) {
    record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
    r.tok0 = r.n = 0;
  }
  const long long cap = (long long)p.max_pages << p.page_log2;
  if (len < r.n || len > cap) {
    record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
    r.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
  }
  r.base = (len < 0 ? 0 : len) - r.n;
  return r;
}

// Page holding position `pos`; a bad entry is a device bounds error and reads page 0.
__device__ __forceinline__ int checked_page(const Paged& p, int entry) {
  if ((unsigned)entry >= (unsigned)p.n_pages) {
    record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
    return 0;
  }
  return entry;
}

// The work list for tiles of 2^tt_log2 tokens and units of 2^kt_log2 keys.
struct Plan {
  int tt_log2, kt_log2;
  int which;  // 0 every sequence, 1 those with at most kSplitRows rows, 2 the others

  __device__ __forceinline__ bool takes(const Paged& p, int n) const {
    if (n <= 0) return false;
    if (which == 0) return true;
    return (((long long)n << p.g_log2) <= kSplitRows) == (which == 1);
  }
  __device__ __forceinline__ int tiles(int n) const {
    return (int)(((long long)n + (1 << tt_log2) - 1) >> tt_log2);
  }
  // Keys that the last token of tile j sees (0 for a tile before the sequence's start).
  __device__ __forceinline__ int keys(const Span& s, int j) const {
    const long long end = (long long)s.base + min((long long)s.n, (long long)(j + 1) << tt_log2);
    return (int)max(0LL, min(end, (long long)s.len));
  }
  __device__ __forceinline__ int units(const Span& s, int j) const {
    const int u = (int)(((long long)keys(s, j) + (1 << kt_log2) - 1) >> kt_log2);
    return u > 0 ? u : 1;  // a tile that sees nothing still writes its zeros
  }
  // Sum of units() over the tiles of a sequence.
  __device__ __forceinline__ long long seq_units(const Span& s) const {
    const int J = tiles(s.n);
    const long long kt = 1LL << kt_log2;
    if (s.base < 0 || (long long)s.base + s.n > s.len) {  // clamped sequence: tile by tile
      long long u = 0;
      for (int j = 0; j < J; ++j) u += units(s, j);
      return u;
    }
    const long long last = ((long long)s.base + s.n + kt - 1) >> kt_log2;  // n >= 1: at least one
    const long long m = J - 1;  // full tiles: sum over x = 1..m of floor((base + kt - 1 + x 2^tt) / kt)
    const long long a = (long long)s.base + kt - 1;
    long long sum;
    if (tt_log2 >= kt_log2) {
      sum = m * (a >> kt_log2) + ((m * (m + 1) / 2) << (tt_log2 - kt_log2));
    } else {  // floor((c + x) / r) with c = floor(a / 2^tt), r = kt / 2^tt
      const int rl = kt_log2 - tt_log2;
      const long long c = a >> tt_log2;
      sum = floor_sum(c + m, rl) - floor_sum(c, rl);
    }
    return sum + last;
  }
  // Sum over z = 0..y of floor(z / 2^rl).
  __device__ __forceinline__ static long long floor_sum(long long y, int rl) {
    const long long q = (y + 1) >> rl, rem = (y + 1) & ((1LL << rl) - 1);
    return ((q * (q - 1) / 2) << rl) + rem * q;
  }
};

// A position in the work list.
struct Cursor {
  int g, s, j, kt;  // kt: first key tile of the item still to do
  Span span;
};

// Sets the cursor to unit `off` of sequence cur->s for KV head cur->g.
__device__ __forceinline__ void plan_seek(const Paged& p, const Plan& pl, Cursor* cur, long long off) {
  cur->span = load_span(p, cur->s);
  int lo = 0, hi = pl.tiles(cur->span.n) - 1;
  if (cur->span.base < 0 || (long long)cur->span.base + cur->span.n > cur->span.len) {
    while (lo < hi) {
      const int u = pl.units(cur->span, lo);
      if (off < u) break;
      off -= u;
      ++lo;
    }
  } else {
    Span part = cur->span;
    auto before_tile = [&](int j) -> long long {  // units of tiles 0..j-1 (all full)
      if (j == 0) return 0;
      part.n = j << pl.tt_log2;
      part.len = part.base + part.n;
      return pl.seq_units(part);
    };
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before_tile(mid) <= off) lo = mid;
      else hi = mid - 1;
    }
    off -= before_tile(lo);
  }
  cur->j = lo;
  cur->kt = (int)min(off, (long long)pl.units(cur->span, lo) - 1);  // off is below units() unless the lengths change meanwhile
}

// The next item after the cursor's.  Only called while units are left, so it exists.
__device__ __forceinline__ void plan_next(const Paged& p, const Plan& pl, Cursor* cur) {
  cur->kt = 0;
  if (++cur->j < pl.tiles(cur->span.n)) return;
  cur->j = 0;
  for (int tries = 0; tries <= p.S; ++tries) {
    if (++cur->s == p.S) {
      cur->s = 0;
      ++cur->g;
    }
    cur->span = load_span(p, cur->s);
    if (pl.takes(p, cur->span.n)) return;
  }
}

#ifdef __CUDACC__  // the rest of the header also serves the host checks

// Programmatic launches: the joining kernel may be set up from here on, and waits for this one's end.
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct PlanSmem {
  long long warp_sum[32];
  int s;
  long long off;  // units of sequence s before the target
  int g;
};

// Block-wide (THREADS a multiple of 32): the CTA's first item, its number of units
// and the length of every CTA's run.
// Ends with a __syncthreads.
template <int THREADS>
__device__ __forceinline__ void plan_start(const Paged& p, const Plan& pl, PlanSmem* sm, Cursor* cur, long long* left,
                                           long long* run_out) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (p.S + THREADS - 1) / THREADS;
  const int s0 = min(p.S, t * per), s1 = min(p.S, s0 + per);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Span sp = load_span(p, s);
    if (pl.takes(p, sp.n)) mine += pl.seq_units(sp);
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sm->warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long x = sm->warp_sum[w];
    before += w < warp ? x : 0;
    total += x;
  }
  const long long all = total * p.Hkv;
  const long long run = (all + gridDim.x - 1) / gridDim.x;  // units for each CTA
  *run_out = run;
  const long long u0 = run * blockIdx.x;
  const long long u1 = u0 + run < all ? u0 + run : all;
  *left = u1 > u0 ? u1 - u0 : 0;
  if (*left > 0) {
    const int g = (int)(u0 / total);
    const long long r = u0 - g * total;
    long long at = before + incl - mine;
    if (r >= at && r < at + mine) {  // the one thread whose sequences hold unit u0
      for (int s = s0; s < s1; ++s) {
        const Span sp = load_span(p, s);
        const long long u = pl.takes(p, sp.n) ? pl.seq_units(sp) : 0;
        if (r < at + u) {
          sm->s = s;
          sm->off = r - at;
          sm->g = g;
          break;
        }
        at += u;
      }
    }
  }
  __syncthreads();
  if (*left > 0) {
    cur->g = sm->g;
    cur->s = sm->s;
    plan_seek(p, pl, cur, sm->off);
  }
}

// The last CTA with a part of the item whose first unit lies in this CTA's run:
// `ahead` units of the item come after the run's end.
__device__ __forceinline__ int plan_last_cta(const Paged& p, long long ahead, long long run) {
  return (int)blockIdx.x + (int)((ahead + run - 1) / run);
}

#endif

}  // namespace tsa
