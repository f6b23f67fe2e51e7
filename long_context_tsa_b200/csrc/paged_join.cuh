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
#include "paged_arrive.cuh"
#include "paged_codes.cuh"
#include "paged_plan.cuh"

namespace tsa {

constexpr int kJoinWeights = 8;  // parts whose weights are kept in shared memory

template <int ROWS>
struct JoinSmem {
  float top[ROWS], inverse[ROWS], weight[kJoinWeights][ROWS];
  int last;
};

// Called by all THREADS threads after the CTA's part of the tile has been written; sync() is their barrier.
// Rows are token * G + query head.
template <typename T, int D, int ROWS, int THREADS, typename Sync>
__device__ __forceinline__ void join_parts(const Paged& p, const Rows& out, const Parts& parts, JoinSmem<ROWS>* sm, const Owners& own, int g,
                                           int tok0, int n_rows, int tid, Sync&& sync) {
  sync();  // everyone's stores are before thread 0's fence
  if (tid == 0) {
    __threadfence();
    sm->last = part_arrives(parts.header, own);
    __threadfence();
  }
  sync();
  if (!sm->last) return;
  auto slot = [&](int k) { return (size_t)(own.first + k) * 2 + (k == 0 ? 1 : 0); };
  // Items are float4s of the tile; a thread has NB at a time.  The first parts of its first items are
  // under way while the weights are found.
  constexpr int NI = ROWS * (D / 4) / THREADS, NB = NI < 4 ? NI : 4, DEPTH = 2;
  auto part = [&](int k, int j) {
    const int i = j * THREADS + tid;
    return __ldcg(reinterpret_cast<const float4*>(parts.o + (slot(k) * ROWS + i / (D / 4)) * D + i % (D / 4) * 4));
  };
  float4 x[DEPTH][NB];
  auto load = [&](int k0, int j0) {
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (k0 + k < own.n) x[k][j] = part(k0 + k, j0 + j);
  };
  load(0, 0);
  {
    constexpr int L = THREADS / ROWS < 16 ? THREADS / ROWS : 16;  // lanes of a row
    const int row = tid / L, lane = tid % L;
    if (row < ROWS) {  // whole warps
      auto m_of = [&](int k) { return __ldcg(parts.ml + slot(k) * 2 * ROWS + row); };
      auto l_of = [&](int k) { return __ldcg(parts.ml + (slot(k) * 2 + 1) * ROWS + row); };
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane + j * L < own.n) {
          m[j] = m_of(lane + j * L);
          l[j] = l_of(lane + j * L);
        }
      float top = fmaxf(m[0], m[1]), sum = 0.f;
      for (int k = lane + 2 * L; k < own.n; k += L) top = fmaxf(top, m_of(k));
#pragma unroll
      for (int d = 1; d < L; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      auto weight = [&](int k, float mk, float lk) {
        const float f = mk == top ? 1.f : exp2f(mk - top);
        if (k < kJoinWeights) sm->weight[k][row] = f;
        sum += f * lk;
      };
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane + j * L < own.n) weight(lane + j * L, m[j], l[j]);
      for (int k = lane + 2 * L; k < own.n; k += L) weight(k, m_of(k), l_of(k));
#pragma unroll
      for (int d = 1; d < L; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) {
        sm->top[row] = top;
        sm->inverse[row] = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no key: zeros
      }
    }
  }
  sync();
#pragma unroll 1
  for (int j0 = 0; j0 < NI; j0 += NB) {
    float4 a[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, const float4 (&o)[NB]) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int row = ((j0 + j) * THREADS + tid) / (D / 4);
        float f;
        if (k < kJoinWeights) {
          f = sm->weight[k][row];
        } else {
          const float m = __ldcg(parts.ml + slot(k) * 2 * ROWS + row);
          f = m == sm->top[row] ? 1.f : exp2f(m - sm->top[row]);
        }
        a[j].x += f * o[j].x;
        a[j].y += f * o[j].y;
        a[j].z += f * o[j].z;
        a[j].w += f * o[j].w;
      }
    };
#pragma unroll 1
    for (int k0 = 0; k0 < own.n; k0 += DEPTH) {
      if (j0 > 0 || k0 > 0) load(k0, j0);
#pragma unroll
      for (int k = 0; k < DEPTH; ++k)
        if (k0 + k < own.n) add(k0 + k, x[k]);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int i = (j0 + j) * THREADS + tid, row = i / (D / 4), c = i % (D / 4) * 4;
      if (row >= n_rows) continue;
      const float inv = sm->inverse[row];
      T* dst = static_cast<T*>(out.data) + (int64_t)(tok0 + (row >> p.g_log2)) * out.ts + (int64_t)(g * p.G + (row & (p.G - 1))) * out.hs + c;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(a[j].x * inv, a[j].y * inv, a[j].z * inv, a[j].w * inv);
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(a[j].x * inv, a[j].y * inv), pack_bf16x2(a[j].z * inv, a[j].w * inv));
    }
  }
}

}  // namespace tsa
