// Joining the partial tiles of a kernel in the kernel itself: the CTA that finishes
// last with a tile adds all its parts, in the order of the CTAs, so the result does
// not depend on which one that is.  (A kernel of its own for this costs a small call
// some 5 us: a launch, and waiting for the last CTA of all.)
//
// Part i has the reference m_i, the sum l_i and the unnormalised o_i; with m = max m_i
// the result is sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
#pragma once

#include <math.h>

#include "paged.h"
#include "paged_codes.cuh"
#include "paged_plan.cuh"

namespace tsa {

template <int ROWS>
struct JoinSmem {
  float top[ROWS], inverse[ROWS];
  int last;
};

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

// Called by all THREADS threads after the CTA's part of the tile has been written; sync() is their barrier.
// Rows are token * G + query head.
template <typename T, int D, int ROWS, int THREADS, typename Sync>
__device__ __forceinline__ void join_parts(const Paged& p, const Rows& out, const Parts& parts, JoinSmem<ROWS>* sm, const Owners& own, int g,
                                           int tok0, int n_rows, int tid, Sync&& sync) {
  sync();  // everyone's stores are before thread 0's fence
  if (tid == 0) {
    __threadfence();
    sm->last = atomicAdd(parts.arrived + own.first, 1u) == (uint32_t)own.n - 1;
    if (sm->last) parts.arrived[own.first] = 0u;  // for the next call
    __threadfence();
  }
  sync();
  if (!sm->last) return;
  auto slot = [&](int k) { return (size_t)(own.first + k) * 2 + (k == 0 ? 1 : 0); };
  {
    constexpr int L = THREADS / ROWS < 16 ? THREADS / ROWS : 16;  // lanes of a row
    const int row = tid / L, lane = tid % L;
    if (row < ROWS) {  // whole warps
      float top = -INFINITY, sum = 0.f;
      for (int k = lane; k < own.n; k += L) top = fmaxf(top, __ldcg(parts.ml + slot(k) * 2 * ROWS + row));
#pragma unroll
      for (int d = 1; d < L; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      for (int k = lane; k < own.n; k += L) {
        const float m = __ldcg(parts.ml + slot(k) * 2 * ROWS + row);
        sum += (m == top ? 1.f : exp2f(m - top)) * __ldcg(parts.ml + (slot(k) * 2 + 1) * ROWS + row);
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) {
        sm->top[row] = top;
        sm->inverse[row] = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no key: zeros
      }
    }
  }
  sync();
  for (int i = tid; i < n_rows * (D / 4); i += THREADS) {
    const int row = i / (D / 4), c = i % (D / 4) * 4;
    const float top = sm->top[row], inv = sm->inverse[row];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < own.n; ++k) {
      const float m = __ldcg(parts.ml + slot(k) * 2 * ROWS + row);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(parts.o + (slot(k) * ROWS + row) * D + c));
      const float f = m == top ? 1.f : exp2f(m - top);
      a.x += f * o.x;
      a.y += f * o.y;
      a.z += f * o.z;
      a.w += f * o.w;
    }
    T* dst = static_cast<T*>(out.data) + (int64_t)(tok0 + (row >> p.g_log2)) * out.ts + (int64_t)(g * p.G + (row & (p.G - 1))) * out.hs + c;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
}

}  // namespace tsa
