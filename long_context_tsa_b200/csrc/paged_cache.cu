// Writing new tokens' keys and values into the paged cache, with 8-bit codes
// where the cache has them, and reading them back.
//
// A row is one token's K or V of one KV head.  With a = max |x| and M = 127
// (int8) or 448 (e4m3):  scale = a / M in fp32,  code = x M / a rounded to the
// nearest code, ties to even, from the exact quotient;  a row of zeros has scale
// 0, a row with a NaN or an infinity codes 0 and scale NaN (it reads back as
// NaN).  Reading gives code * scale in fp32, rounded to the output's type.
//
// Both kernels move bytes and nothing bounds them but HBM.  A warp takes a
// token and eight 16-byte-a-lane rows of it (four loads a lane in flight); the
// page is looked up once for those rows, in the write kernel while the loads
// are under way.
#include "device_common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"

namespace tsa {
namespace {

constexpr int kThreads = 256;
constexpr int kIters = 4;  // rows in flight for each lane

// The place of packed token t: 0 not of any sequence, 1 found, with page and slot.
struct Place {
  int page, slot;
  bool ok;
};

// All lanes of a warp call this with the same t.
__device__ __forceinline__ Place find_place(const Paged& p, int t, int lane) {
  // s = number of sequences that end at or before t: 32 probes, then 32 more in between.
  int lo = 0;
  for (int n = p.S; n > 0;) {
    const int step = (n + 31) / 32;
    const int s = lo + (lane + 1) * step;  // sequences lo .. s-1 end at or before t?
    const bool done = s <= lo + n && p.token_start[s] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, done));
    lo += c * step;
    if (step == 1) break;
    n = min(step, p.S - lo);
  }
  Place r;
  r.page = r.slot = 0;
  r.ok = false;
  if (lo >= p.S) return r;  // behind the last sequence: left as it is
  const int a = p.token_start[lo], b = p.token_start[lo + 1];
  const long long pos = (long long)p.seq_len[lo] - b + t;  // len - n + (t - a)
  if (a < 0 || t < a || t >= b || b > p.T || pos < 0 || (pos >> p.page_log2) >= p.max_pages) {
    if (t >= a || a < 0 || b > p.T) record_status(p.status, TSA_ERR_DEVICE_BOUNDS);  // t < a: a gap between sequences
    return r;
  }
  const int entry = p.table[(size_t)lo * p.max_pages + (pos >> p.page_log2)];
  if ((unsigned)entry >= (unsigned)p.n_pages) {
    record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
    return r;
  }
  r.page = entry;
  r.slot = (int)(pos & ((1 << p.page_log2) - 1));
  r.ok = true;
  return r;
}

// The first block looks over all starts: a descending pair may lie where no token's search comes past.
__device__ __forceinline__ void check_starts(const Paged& p) {
  if (blockIdx.x != 0) return;
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    const int a = p.token_start[s], b = p.token_start[s + 1];
    if (a < 0 || b < a || b > p.T) record_status(p.status, TSA_ERR_DEVICE_BOUNDS);
  }
}

// IN: float or bf16; CODE: kPlain keeps IN.
template <typename IN, int CODE, int D>
__global__ void __launch_bounds__(kThreads) cache_write(const Paged p, const Rows k, const Rows v, int chunks) {
  constexpr int E = 16 / (int)sizeof(IN);  // elements of a lane
  constexpr int LPR = D / E;               // lanes of a row
  constexpr int RPW = 32 / LPR;            // rows of a warp's load
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / chunks), chunk = (int)(w - (long long)t * chunks);
  check_starts(p);
  if (t >= p.T) return;
  const int c = lane % LPR, r0 = chunk * (kIters * RPW) + lane / LPR;
  uint4 x[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = r0 + i * RPW;  // 0 .. 2 Hkv - 1: K heads, then V heads
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < 2 * p.Hkv) {
      const bool is_v = r >= p.Hkv;
      const Rows& src = is_v ? v : k;
      const IN* row = static_cast<const IN*>(src.data) + (int64_t)t * src.ts + (int64_t)(is_v ? r - p.Hkv : r) * src.hs;
      x[i] = __ldcs(reinterpret_cast<const uint4*>(row + c * E));
    }
  }
  const Place at = find_place(p, t, lane);
  if (!at.ok) return;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = r0 + i * RPW;
    const bool is_v = r >= p.Hkv;
    const bool live = r < 2 * p.Hkv;
    const size_t row = ((((size_t)at.page * p.Hkv) + (is_v ? r - p.Hkv : r)) << p.page_log2) + at.slot;
    if constexpr (CODE == kPlain) {
      if (live) *reinterpret_cast<uint4*>(static_cast<IN*>(is_v ? p.v_pages : p.k_pages) + row * D + c * E) = x[i];
    } else {
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float f[E];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (E == 8) {
          f[2 * e] = bf16_lo(u[e]);
          f[2 * e + 1] = bf16_hi(u[e]);
        } else {
          f[e] = __uint_as_float(u[e]);
        }
      }
      uint32_t top = 0;  // magnitudes order like their bits; a NaN's are above infinity's
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float a = __uint_as_float(top);
      const bool finite = top < 0x7f800000u;
      // A power of two brings the row to where products and remainders neither over- nor underflow.
      const float two = a > 1.2676506e30f ? 5.4210109e-20f : a < 8.6736174e-19f ? 1.8446744e19f : 1.f;  // 2^100: 2^-64; 2^-60: 2^64
      const float as = finite ? a * two : 0.f;
      const float rinv = as > 0.f ? 1.f / as : 0.f;
      uint32_t b[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xs = finite ? fabsf(f[e]) * two : 0.f;
        const float q = code_quotient<CODE, sizeof(IN) == 4>(xs, as, rinv);
        b[e] = finite ? __float_as_uint(copysignf(q, f[e])) : 0u;
      }
      uint32_t code[E / 4];
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        if constexpr (CODE == kI8) {  // adding 1.5 2^23 rounds to the nearest integer, ties to even; its low byte is the code
          uint32_t m[4];
#pragma unroll
          for (int o = 0; o < 4; ++o) m[o] = __float_as_uint(__uint_as_float(b[e + o]) + 12582912.f);
          code[e / 4] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
        } else {
          uint32_t h[2];
#pragma unroll
          for (int o = 0; o < 2; ++o)
            h[o] = __nv_cvt_float2_to_fp8x2(
                make_float2(__uint_as_float(b[e + 2 * o]), __uint_as_float(b[e + 2 * o + 1])), __NV_SATFINITE, __NV_E4M3);
          code[e / 4] = h[0] | (h[1] << 16);
        }
      }
      if (live) {
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * D + c * E;
        if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
        else *reinterpret_cast<uint32_t*>(dst) = code[0];
        if (c == 0) (is_v ? p.v_scales : p.k_scales)[row] = finite ? a / code_max<CODE>() : __uint_as_float(0x7fffffffu);
      }
    }
  }
}

// OUT: float or bf16; CODE: kPlain copies.
template <typename OUT, int CODE, int D>
__global__ void __launch_bounds__(kThreads) cache_read(const Paged p, const Rows k, const Rows v, int chunks) {
  constexpr int E = CODE == kPlain ? 16 / (int)sizeof(OUT) : 8;  // elements of a lane
  constexpr int LPR = D / E;
  constexpr int RPW = 32 / LPR;
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / chunks), chunk = (int)(w - (long long)t * chunks);
  check_starts(p);
  if (t >= p.T) return;
  const int c = lane % LPR, r0 = chunk * (kIters * RPW) + lane / LPR;
  const Place at = find_place(p, t, lane);
  if (!at.ok) return;
  uint4 x[kIters];
  float scale[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = r0 + i * RPW;
    const bool is_v = r >= p.Hkv;
    const size_t row = ((((size_t)at.page * p.Hkv) + (is_v ? r - p.Hkv : r)) << p.page_log2) + at.slot;
    x[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 0.f;
    if (r < 2 * p.Hkv) {
      if constexpr (CODE == kPlain) {
        x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const OUT*>(is_v ? p.v_pages : p.k_pages) + row * D + c * E));
      } else {
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * D + c * E));
        x[i].x = y.x;
        x[i].y = y.y;
        scale[i] = __ldg((is_v ? p.v_scales : p.k_scales) + row);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = r0 + i * RPW;
    if (r >= 2 * p.Hkv) continue;
    const bool is_v = r >= p.Hkv;
    const Rows& dst = is_v ? v : k;
    OUT* row = static_cast<OUT*>(dst.data) + (int64_t)t * dst.ts + (int64_t)(is_v ? r - p.Hkv : r) * dst.hs + c * E;
    if constexpr (CODE == kPlain) {
      __stcs(reinterpret_cast<uint4*>(row), x[i]);
    } else {
      const uint32_t h[4] = {codes_next<CODE, 0>(x[i].x), codes_next<CODE, 2>(x[i].x), codes_next<CODE, 0>(x[i].y),
                             codes_next<CODE, 2>(x[i].y)};
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16_lo(h[e]) * scale[i];
        f[2 * e + 1] = bf16_hi(h[e]) * scale[i];
      }
      if constexpr (sizeof(OUT) == 2) {
        __stcs(reinterpret_cast<uint4*>(row), make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                         pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
      } else {
        __stcs(reinterpret_cast<float4*>(row), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(row) + 1, make_float4(f[4], f[5], f[6], f[7]));
      }
    }
  }
}

template <typename X, int CODE, int D>
cudaError_t launch(bool write, const Paged& p, const Rows& k, const Rows& v, cudaStream_t st) {
  const int e = write || CODE == kPlain ? 16 / (int)sizeof(X) : 8;
  const int rows = kIters * (32 / (D / e));
  const int chunks = (2 * p.Hkv + rows - 1) / rows;
  const long long blocks = ((long long)p.T * chunks * 32 + kThreads - 1) / kThreads;
  if (write) cache_write<X, CODE, D><<<(unsigned)blocks, kThreads, 0, st>>>(p, k, v, chunks);
  else cache_read<X, CODE, D><<<(unsigned)blocks, kThreads, 0, st>>>(p, k, v, chunks);
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
