// Attention of f32 new tokens over the paged cache on CUDA cores: exact fp32 products.
//
// A tile is ROWS rows of one KV head, row = token * G + query head, against key
// tiles of 64 cached positions; CTAs take equal runs of (tile, key tile) pairs
// (paged_plan.cuh).  Thread (ty, tx) of 16 x 16 holds rows ty + 16 i and, of the
// logits, keys tx + 16 j: whole float4s along d for both operands, so the K tile
// is stored as it is read.  Online softmax in base 2; a row's 16 threads keep
// parts of its sum until the tile ends.
//
// Rows behind the sequence's end are never read (zeros stand in the tiles).  In
// tiles at the causal border the second product skips the keys that a row does
// not see, so that a hidden value row may hold infinities or NaN.
#include <math.h>

#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"
#include "paged_join.cuh"

namespace tsa {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;

template <int D, int ROWS>
struct Cfg {
  static constexpr int KS = D + 4;      // stride of Q and K rows: 16 rows' float4s fall into different banks
  static constexpr int PS = kKeys + 4;  // stride of probability rows
  static constexpr int OFF_K = ROWS * KS;
  static constexpr int OFF_V = OFF_K + (kKeys * KS > ROWS * PS ? kKeys * KS : ROWS * PS);  // P takes K's place
  static constexpr int OFF_ROWS = OFF_V + kKeys * D;
  static constexpr int OFF_PLAN = OFF_ROWS + 2 * kKeys;
  static constexpr int OFF_LAST = OFF_PLAN + ((int)sizeof(PlanSmem) + 3) / 4;
  static constexpr int SMEM = OFF_LAST * 4 + (int)sizeof(JoinSmem<ROWS>);
  static constexpr int CTAS = kPagedCtas * 2;  // two to an SM
};

struct SimtParams {
  Paged p;
  Rows q, out;
  Parts parts;
  Plan plan;
  float scale_log2;
};

// Sixteen bytes of a cached row (plain) or eight codes of it, as floats.
template <int CODE>
struct Piece {
  static constexpr int N = CODE != kPlain ? 8 : 4;
  float f[N];
  __device__ __forceinline__ void load(const void* pool, size_t elem, float scale) {
    if constexpr (CODE != kPlain) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + elem));
      const uint32_t h[4] = {codes_next<CODE, 0>(x.x), codes_next<CODE, 2>(x.x), codes_next<CODE, 0>(x.y), codes_next<CODE, 2>(x.y)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16_lo(h[e]) * scale;
        f[2 * e + 1] = bf16_hi(h[e]) * scale;
      }
    } else {
      const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(pool) + elem));
      f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    }
  }
};

template <int CODE, int D, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) paged_simt(const __grid_constant__ SimtParams P) {
  using C = Cfg<D, ROWS>;
  constexpr int R = ROWS / 16;  // rows of a thread
  constexpr int K4 = kKeys / 16;
  constexpr int DJ = D / 64;    // float4 columns of a thread
  constexpr bool kAhead = ROWS == 16;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = sm + C::OFF_K;
  float* Ps = Ks;
  float* Vs = sm + C::OFF_V;
  int* rows_of = reinterpret_cast<int*>(sm + C::OFF_ROWS);  // [2][64]: row of the pools, -1 behind the end
  PlanSmem* psm = reinterpret_cast<PlanSmem*>(sm + C::OFF_PLAN);
  const Paged& p = P.p;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;

  Cursor cur;
  long long left, run;
  plan_start<kThreads>(p, P.plan, psm, &cur, &left, &run);
  const long long all_left = left;
  const int tt = 1 << P.plan.tt_log2;

  while (left > 0) {
    const int keys = P.plan.keys(cur.span, cur.j), units = P.plan.units(cur.span, cur.j);
    const int kt1 = (int)min((long long)units, cur.kt + left);
    const int first_tok = cur.j * tt, n_tok = min(tt, cur.span.n - first_tok);
    const int pos0 = cur.span.base + first_tok;
    const int n_rows = n_tok << p.g_log2;

    auto find_rows = [&](int kt) {
      if (tid < kKeys) {
        const int key = kt * kKeys + tid;
        int r = -1;
        if (key < keys) {
          const int page = checked_page(p, __ldg(p.table + (size_t)cur.s * p.max_pages + (key >> p.page_log2)));
          r = ((page * p.Hkv + cur.g) << p.page_log2) + (key & ((1 << p.page_log2) - 1));
        }
        rows_of[(kt & 1) * kKeys + tid] = r;
      }
    };
    __syncthreads();  // the previous tile's buffers are free
    find_rows(cur.kt);
    if (kAhead && cur.kt + 1 < kt1) find_rows(cur.kt + 1);
#pragma unroll 4
    for (int j = 0; j < ROWS * (D / 4) / kThreads; ++j) {
      const int i = j * kThreads + tid, r = i / (D / 4), c = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n_rows)
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(P.q.data) + (int64_t)(cur.span.tok0 + first_tok + (r >> p.g_log2)) * P.q.ts +
                                             (int64_t)(cur.g * p.G + (r & (p.G - 1))) * P.q.hs + c);
      *reinterpret_cast<float4*>(Qs + r * C::KS + c) = x;
    }

    int rpos[R];
    float m[R], l[R];
    float4 o[R][DJ];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      rpos[i] = pos0 + min((ty + 16 * i) >> p.g_log2, n_tok - 1);
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < DJ; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    using Pc = Piece<CODE>;
    constexpr int PPR = D / Pc::N, N = kKeys * PPR / kThreads;  // pieces of a row, and of a thread
    constexpr int B = kAhead || N < 4 ? N : 4;                 // in flight, of K and V each
    Pc k[B], v[B];
    auto load = [&](int kt, int i0) {
      const int* rows = rows_of + (kt & 1) * kKeys;
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int i = (i0 + j) * kThreads + tid, c = i % PPR * Pc::N, r = rows[i / PPR];
        k[j] = v[j] = Pc{};
        if (r >= 0) {
          k[j].load(p.k_pages, (size_t)r * D + c, CODE == kPlain ? 1.f : __ldg(p.k_scales + r));
          v[j].load(p.v_pages, (size_t)r * D + c, CODE == kPlain ? 1.f : __ldg(p.v_scales + r));
        }
      }
    };
    auto store = [&](int i0) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int i = (i0 + j) * kThreads + tid, n = i / PPR, c = i % PPR * Pc::N;
#pragma unroll
        for (int e = 0; e < Pc::N; e += 4) {
          *reinterpret_cast<float4*>(Ks + n * C::KS + c + e) = make_float4(k[j].f[e], k[j].f[e + 1], k[j].f[e + 2], k[j].f[e + 3]);
          *reinterpret_cast<float4*>(Vs + n * D + c + e) = make_float4(v[j].f[e], v[j].f[e + 1], v[j].f[e + 2], v[j].f[e + 3]);
        }
      }
    };
    if (kAhead) {
      __syncthreads();
      load(cur.kt, 0);
    }
    for (int kt = cur.kt; kt < kt1; ++kt) {
      const int key0 = kt * kKeys;
      __syncthreads();  // rows found; K and V of the previous tile are done with
      if constexpr (kAhead) {  // few rows: bound by the loads, so the next tile's are under way during this one's products
        store(0);
        if (kt + 1 < kt1) load(kt + 1, 0);
        if (kt + 2 < kt1) find_rows(kt + 2);
      } else {
#pragma unroll 1
        for (int i0 = 0; i0 < N; i0 += B) {
          load(kt, i0);
          store(i0);
        }
        if (kt + 1 < kt1) find_rows(kt + 1);
      }
      __syncthreads();

      float s[R][K4];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < K4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 k[K4];
#pragma unroll
        for (int j = 0; j < K4; ++j) k[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * C::KS + d);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * C::KS + d);
#pragma unroll
          for (int j = 0; j < K4; ++j)
            s[i][j] = fmaf(q.w, k[j].w, fmaf(q.z, k[j].z, fmaf(q.y, k[j].y, fmaf(q.x, k[j].x, s[i][j]))));
        }
      }
      __syncthreads();  // K is done with: P takes its place
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int last = min(rpos[i] + 1, keys) - key0;  // keys of the tile that the row sees
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < K4; ++j) {
          s[i][j] = tx + 16 * j < last ? s[i][j] * P.scale_log2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (top > m[i]) {
          const float alpha = exp2f(m[i] - top);  // 0 for the first keys
          m[i] = top;
          l[i] *= alpha;
#pragma unroll
          for (int j = 0; j < DJ; ++j) {
            o[i][j].x *= alpha;
            o[i][j].y *= alpha;
            o[i][j].z *= alpha;
            o[i][j].w *= alpha;
          }
        }
        const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int j = 0; j < K4; ++j) {
          const float x = exp2f(s[i][j] - ref);
          l[i] += x;
          Ps[(ty + 16 * i) * C::PS + tx + 16 * j] = x;
        }
      }
      __syncthreads();
      const bool border = key0 + kKeys - 1 > pos0;
#pragma unroll 2
      for (int c = 0; c < kKeys; c += 4) {
        float4 pr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) pr[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * C::PS + c);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float4 v[DJ];
#pragma unroll
          for (int j = 0; j < DJ; ++j) v[j] = *reinterpret_cast<const float4*>(Vs + (c + u) * D + tx * 4 + 64 * j);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float x = u == 0 ? pr[i].x : u == 1 ? pr[i].y : u == 2 ? pr[i].z : pr[i].w;
            if (border && key0 + c + u > rpos[i]) continue;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
              o[i][j].x = fmaf(x, v[j].x, o[i][j].x);
              o[i][j].y = fmaf(x, v[j].y, o[i][j].y);
              o[i][j].z = fmaf(x, v[j].z, o[i][j].z);
              o[i][j].w = fmaf(x, v[j].w, o[i][j].w);
            }
          }
        }
      }
    }

    const bool whole = cur.kt == 0 && kt1 == units;
    const size_t part = (size_t)blockIdx.x * 2 + (cur.kt == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float sum = l[i];
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int row = ty + 16 * i;
      if (row >= n_rows) continue;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no key: zeros
        float* dst = static_cast<float*>(P.out.data) + (int64_t)(cur.span.tok0 + first_tok + (row >> p.g_log2)) * P.out.ts +
                 (int64_t)(cur.g * p.G + (row & (p.G - 1))) * P.out.hs;
#pragma unroll
        for (int j = 0; j < DJ; ++j) {
          const float4 a = o[i][j];
          *reinterpret_cast<float4*>(dst + tx * 4 + 64 * j) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        }
      } else {
#pragma unroll
        for (int j = 0; j < DJ; ++j)
          *reinterpret_cast<float4*>(P.parts.o + (part * ROWS + row) * D + tx * 4 + 64 * j) = o[i][j];
        if (tx == 0) {
          P.parts.ml[part * 2 * ROWS + row] = m[i];
          P.parts.ml[(part * 2 + 1) * ROWS + row] = sum;
        }
      }
    }
    if (!whole)
      join_parts<float, D, ROWS, kThreads>(p, P.out, P.parts, reinterpret_cast<JoinSmem<ROWS>*>(sm + C::OFF_LAST),
                                           tile_owners(run * blockIdx.x + (all_left - left), cur.kt, units, run), cur.g,
                                           cur.span.tok0 + first_tok, n_rows, tid, [] { __syncthreads(); });
    left -= kt1 - cur.kt;
    if (left > 0) plan_next(p, P.plan, &cur);
  }
}

// Few rows take the small tile: fewer of its rows are empty.
int rows_log2(const Paged& p) { return (long long)p.max_new * p.G <= 16 ? 4 : 6; }

template <int CODE, int D, int ROWS>
cudaError_t launch(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, cudaStream_t st) {
  using C = Cfg<D, ROWS>;
  SimtParams P;
  P.p = p;
  P.q = q;
  P.out = out;
  P.parts = make_parts(base, ROWS, C::CTAS, D);
  P.parts.header = header;
  P.plan.tt_log2 = (ROWS == 16 ? 4 : 6) - p.g_log2;
  P.plan.kt_log2 = 6;
  P.plan.which = 0;
  P.scale_log2 = p.scale * 1.4426950408889634f;
  cudaError_t e = cudaFuncSetAttribute(paged_simt<CODE, D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  paged_simt<CODE, D, ROWS><<<C::CTAS, kThreads, C::SMEM, st>>>(P);
  count_launches(1);
  return cudaGetLastError();
}

template <int CODE, int D>
cudaError_t by_rows(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, cudaStream_t st) {
  return rows_log2(p) == 4 ? launch<CODE, D, 16>(p, q, out, base, header, st) : launch<CODE, D, 64>(p, q, out, base, header, st);
}

template <int D>
cudaError_t by_code(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, cudaStream_t st) {
  if (p.cache_dtype == TSA_I8) return by_rows<kI8, D>(p, q, out, base, header, st);
  if (p.cache_dtype == TSA_E4M3) return by_rows<kE4M3, D>(p, q, out, base, header, st);
  return by_rows<kPlain, D>(p, q, out, base, header, st);
}

}  // namespace

size_t paged_simt_bytes(const Paged& p) { return parts_bytes(1 << rows_log2(p), 2 * kPagedCtas, p.D); }

cudaError_t launch_paged_simt(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, cudaStream_t st) {
  return p.D == 64 ? by_code<64>(p, q, out, base, header, st) : by_code<128>(p, q, out, base, header, st);
}

}  // namespace tsa
