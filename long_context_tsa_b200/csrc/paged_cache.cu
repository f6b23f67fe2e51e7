// Writing new tokens' keys and values into the paged cache, with 8-bit codes
// where the cache has them, and reading them back.
//
// A row is one token's K or V of one KV head.  With a = max |x| and M = 127
// (int8) or 448 (e4m3):  scale = a / M in fp32,  code = x M / a rounded to the
// nearest code, ties to even, from the exact quotient;  a row of zeros has scale
// 0, a row with a NaN or an infinity codes 0 and scale NaN (it reads back as
// NaN).  Reading gives code * scale in fp32, rounded to the output's type.
//
// Both kernels move bytes and nothing bounds them but HBM.  A block takes up to
// 8 consecutive tokens; its first warp finds their places (in the write kernel
// while the first loads are under way), then all threads walk over the (head,
// token) rows, tokens first.
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"

namespace tsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of a block

// The row of the pools (head 0) for each of the block's tokens t0 .. t0 + n - 1, or -1.
// One warp; n <= 32.
__device__ __forceinline__ void find_rows(const Paged& p, int t0, int n, int* rows) {
  const int lane = threadIdx.x & 31;
  // s = number of sequences that end at or before t0: 32 probes, then 32 more in between.
  int lo = 0;
  for (int m = p.S; m > 0;) {
    const int step = (m + 31) / 32;
    const int s = lo + (lane + 1) * step;  // sequences lo .. s-1 end at or before t0?
    const bool done = s <= lo + m && p.token_start[s] <= t0;
    const int c = __popc(__ballot_sync(0xffffffffu, done));
    lo += c * step;
    if (step == 1) break;
    m = min(step, p.S - lo);
  }
  const int t = t0 + lane;
  int row = -1;
  if (lane < n) {
    while (lo < p.S && p.token_start[lo + 1] <= t) ++lo;
    if (lo < p.S) {  // else behind the last sequence: left as it is
      const int a = p.token_start[lo], b = p.token_start[lo + 1];
      const long long pos = (long long)p.seq_len[lo] - b + t;  // len - n + (t - a)
      if (a < 0 || t < a || t >= b || b > p.T || pos < 0 || (pos >> p.page_log2) >= p.max_pages) {
        if (t >= a || a < 0 || b > p.T) record_status(p.status, TSA_ERR_DEVICE_BOUNDS);  // t < a: a gap between sequences
      } else {
        const int page = p.table[(size_t)lo * p.max_pages + (pos >> p.page_log2)];
        if ((unsigned)page >= (unsigned)p.n_pages) record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
        else row = ((page * p.Hkv) << p.page_log2) + (int)(pos & ((1 << p.page_log2) - 1));
      }
    }
    rows[lane] = row;
  }
}

// The first block looks over all starts: a descending pair may lie where no token's search comes past.
__device__ __forceinline__ void check_starts(const Paged& p) {
  if (blockIdx.x != 0) return;
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    const int a = p.token_start[s], b = p.token_start[s + 1];
    if (a < 0 || b < a || b > p.T) record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
  }
}

// Codes of the eight (bf16) or four (f32) elements f of a lane, four to a word, for a row with
// largest magnitude a.
template <int CODE, int E>
__device__ __forceinline__ void pack_codes(const float (&q)[E], uint32_t (&code)[E / 4]) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    if constexpr (CODE == kI8) {  // adding 1.5 2^23 rounds to the nearest integer, ties to even; its low byte is the code
      uint32_t m[4];
#pragma unroll
      for (int o = 0; o < 4; o += 2) {
        float f, g;
        tc::f2_unpack(tc::f2_add(tc::f2_pack(q[e + o], q[e + o + 1]), tc::f2_pack(12582912.f, 12582912.f)), f, g);
        m[o] = __float_as_uint(f);
        m[o + 1] = __float_as_uint(g);
      }
      code[e / 4] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
    } else {
      uint32_t h[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) h[o] = __nv_cvt_float2_to_fp8x2(make_float2(q[e + 2 * o], q[e + 2 * o + 1]), __NV_SATFINITE, __NV_E4M3);
      code[e / 4] = h[0] | (h[1] << 16);
    }
  }
}

// a / M, correctly rounded: the product with the correctly rounded 1 / M and one correction by its
// remainder (Markstein, as for the codes).  a and a / M normal numbers.
template <int CODE>
__device__ __forceinline__ float scale_of(float a) {
  constexpr float M = code_max<CODE>(), r = 1.f / M;
  const float q = a * r;
  return fmaf(-fmaf(q, M, -a), r, q);
}

// A thread has the same piece of a K row and of the V row beside it: one place and one pair of
// offsets for both, and two loads in flight.  Full occupancy hides more than longer flights do.
//
// IN: float or bf16; CODE: kPlain keeps IN.
template <typename IN, int CODE, int D>
__global__ void __launch_bounds__(kThreads, 8) cache_write(const Paged p, const Rows k, const Rows v, int tb_log2) {
  constexpr int E = 16 / (int)sizeof(IN);  // elements of a lane
  constexpr int LPR = D / E;               // lanes of a row
  __shared__ int rows[kMaxTokens];
  const int t0 = blockIdx.x << tb_log2, n = min(1 << tb_log2, p.T - t0);
  const int all = (p.Hkv << tb_log2) * LPR;  // pieces of the block
  const int c = threadIdx.x % LPR;
  check_starts(p);
  for (int base = 0; base < all; base += kThreads) {
    const int r = (base + (int)threadIdx.x) / LPR, tok = r & ((1 << tb_log2) - 1), h = r >> tb_log2;
    const bool live = h < p.Hkv && tok < n;
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (live) {
      const IN* kr = static_cast<const IN*>(k.data) + (int64_t)(t0 + tok) * k.ts + (int64_t)h * k.hs + c * E;
      const IN* vr = static_cast<const IN*>(v.data) + (int64_t)(t0 + tok) * v.ts + (int64_t)h * v.hs + c * E;
      x[0] = __ldcs(reinterpret_cast<const uint4*>(kr));
      x[1] = __ldcs(reinterpret_cast<const uint4*>(vr));
    }
    if (base == 0) {
      if (threadIdx.x < 32) find_rows(p, t0, n, rows);
      __syncthreads();
    }
    const int at = live ? rows[tok] : -1;
    const size_t row = (size_t)at + ((size_t)h << p.page_log2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      void* pages = i ? p.v_pages : p.k_pages;
      if constexpr (CODE == kPlain) {
        if (at >= 0) *reinterpret_cast<uint4*>(static_cast<IN*>(pages) + row * D + c * E) = x[i];
      } else {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float f[E];
        uint32_t top = 0;  // magnitudes order like their bits; a NaN's are above infinity's
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (E == 8) {
            f[2 * e] = bf16_lo(u[e]);
            f[2 * e + 1] = bf16_hi(u[e]);
            top = __vmaxu2(top, u[e] & 0x7fff7fffu);
          } else {
            f[e] = __uint_as_float(u[e]);
            top = max(top, u[e] & 0x7fffffffu);
          }
        }
        if constexpr (E == 8) top = max(top << 16, top & 0xffff0000u);
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float a = __uint_as_float(top);
        float q[E], scale;
        if (E == 8 && __all_sync(0xffffffffu, a > 8.6736174e-19f && a < 1.2676506e30f)) {  // 2^-60, 2^100
          const float rinv = rcp_approx(a);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            q[e] = f[e];
            q[e + 1] = f[e + 1];
            code_quotients<CODE>(q[e], q[e + 1], a, rinv);
          }
          scale = scale_of<CODE>(a);
        } else {
          const bool finite = top < 0x7f800000u;
          // A power of two brings the row to where products and remainders neither over- nor underflow.
          const float two = a > 1.2676506e30f ? 5.4210109e-20f : a < 8.6736174e-19f ? 1.8446744e19f : 1.f;  // 2^-64, 2^64
          const float as = finite ? a * two : 0.f;
          const float rinv = as > 0.f ? 1.f / as : 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float t = code_quotient<CODE, sizeof(IN) == 4>(finite ? fabsf(f[e]) * two : 0.f, as, rinv);
            q[e] = finite ? copysignf(t, f[e]) : 0.f;
          }
          scale = finite ? a / code_max<CODE>() : __uint_as_float(0x7fffffffu);
        }
        uint32_t code[E / 4];
        pack_codes<CODE, E>(q, code);
        if (at >= 0) {
          uint8_t* dst = static_cast<uint8_t*>(pages) + row * D + c * E;
          if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
          else *reinterpret_cast<uint32_t*>(dst) = code[0];
          if (c == 0) (i ? p.v_scales : p.k_scales)[row] = scale;
        }
      }
    }
  }
}

// OUT: float or bf16; CODE: kPlain copies.
template <typename OUT, int CODE, int D>
__global__ void __launch_bounds__(kThreads, 8) cache_read(const Paged p, const Rows k, const Rows v, int tb_log2) {
  constexpr int E = CODE == kPlain ? 16 / (int)sizeof(OUT) : 8;  // elements of a lane
  constexpr int LPR = D / E;
  using Raw = typename std::conditional<CODE == kPlain, uint4, uint2>::type;
  __shared__ int rows[kMaxTokens];
  const int t0 = blockIdx.x << tb_log2, n = min(1 << tb_log2, p.T - t0);
  const int all = (p.Hkv << tb_log2) * LPR;
  const int c = threadIdx.x % LPR;
  check_starts(p);
  if (threadIdx.x < 32) find_rows(p, t0, n, rows);
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < all; base += kThreads) {
    const int r = (base + (int)threadIdx.x) / LPR, tok = r & ((1 << tb_log2) - 1), h = r >> tb_log2;
    if (h >= p.Hkv || tok >= n) continue;
    const int at = rows[tok];
    if (at < 0) continue;
    const size_t row = (size_t)at + ((size_t)h << p.page_log2), from = row * (D * (CODE == kPlain ? sizeof(OUT) : 1)) + c * sizeof(Raw);
    Raw x[2];
    float scale[2];
    x[0] = __ldg(reinterpret_cast<const Raw*>(static_cast<const char*>(p.k_pages) + from));
    x[1] = __ldg(reinterpret_cast<const Raw*>(static_cast<const char*>(p.v_pages) + from));
    if (CODE != kPlain) {
      scale[0] = __ldg(p.k_scales + row);
      scale[1] = __ldg(p.v_scales + row);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Rows& dst = i ? v : k;
      OUT* to = static_cast<OUT*>(dst.data) + (int64_t)(t0 + tok) * dst.ts + (int64_t)h * dst.hs + c * E;
      if constexpr (CODE == kPlain) {
        __stcs(reinterpret_cast<uint4*>(to), x[i]);
      } else {
        const uint32_t y[2] = {x[i].x, x[i].y};
        float f[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t lo = codes_next<CODE, 0>(y[e]), hi = codes_next<CODE, 2>(y[e]);
          f[4 * e] = bf16_lo(lo) * scale[i];
          f[4 * e + 1] = bf16_hi(lo) * scale[i];
          f[4 * e + 2] = bf16_lo(hi) * scale[i];
          f[4 * e + 3] = bf16_hi(hi) * scale[i];
        }
        if constexpr (sizeof(OUT) == 2) {
          __stcs(reinterpret_cast<uint4*>(to), make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
        } else {
          __stcs(reinterpret_cast<float4*>(to), make_float4(f[0], f[1], f[2], f[3]));
          __stcs(reinterpret_cast<float4*>(to) + 1, make_float4(f[4], f[5], f[6], f[7]));
        }
      }
    }
  }
}

template <typename X, int CODE, int D>
cudaError_t launch(bool write, const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  // Tokens of a block, as long as that leaves four blocks for every SM.  bf16: 8 (131072 x 8 rows to
  // int8 and back in 286 us; 4: 297, 16: 294).  f32: 4 (98000 x 8 rows from int8 in 137 us; 2: 164, 8: 147).
  int tb_log2 = sizeof(X) == 2 ? 3 : 2;
  while (tb_log2 > 0 && (p.T >> tb_log2) < 4 * kPagedCtas) --tb_log2;
  const unsigned blocks = (unsigned)(((long long)p.T + (1 << tb_log2) - 1) >> tb_log2);
  if (write) cache_write<X, CODE, D><<<blocks, kThreads, 0, st>>>(p, k, v, tb_log2);
  else cache_read<X, CODE, D><<<blocks, kThreads, 0, st>>>(p, k, v, tb_log2);
  count_launches(1);
  return cudaGetLastError();
}

template <typename X, int D>
cudaError_t by_code(bool write, const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  if (p.cache_dtype == TSA_I8) return launch<X, kI8, D>(write, p, k, v, st);
  if (p.cache_dtype == TSA_E4M3) return launch<X, kE4M3, D>(write, p, k, v, st);
  return launch<X, kPlain, D>(write, p, k, v, st);
}

cudaError_t by_shape(bool write, const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  if (p.dtype == TSA_BF16) return p.D == 64 ? by_code<__nv_bfloat16, 64>(write, p, k, v, st) : by_code<__nv_bfloat16, 128>(write, p, k, v, st);
  return p.D == 64 ? by_code<float, 64>(write, p, k, v, st) : by_code<float, 128>(write, p, k, v, st);
}

}  // namespace

cudaError_t launch_cache_write(const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  return by_shape(true, p, k, v, st);
}
cudaError_t launch_cache_read(const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  return by_shape(false, p, k, v, st);
}

}  // namespace tsa
