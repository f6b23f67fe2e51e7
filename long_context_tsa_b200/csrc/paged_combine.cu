// Joins the partial tiles of paged_chunk.
//
// Part i of a tile has the reference m_i, the sum l_i and the unnormalised o_i;
// with m = max m_i the result is sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,
// added in the order of the CTAs that left the parts.  Up to 40 MB that the kernel
// before has just written: read from L2, some 10 us.  (paged_small and paged_simt join
// their few rows themselves; here 8 warps of a CTA would do 128 KB a part.)
#include <math.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"
#include "paged_plan.cuh"

namespace tsa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 8;  // rows of a block
constexpr int kMaxParts = kPagedCtas;

template <int D>
__global__ void __launch_bounds__(kThreads) paged_combine(const Paged p, const Rows out, const Parts parts) {
  __shared__ float weight[kMaxParts][kRows];  // of each part: 2^(m_i - m)
  __shared__ float total[kMaxParts][kRows];
  __shared__ float inverse[kRows];
  grid_dependency_wait();  // launched while the kernel before still runs
  const PartMeta meta = parts.meta[blockIdx.x];
  if (meta.c_end < 0) return;
  const int first = blockIdx.x, n = min(meta.c_end, parts.ctas - 1) - first + 1;
  const int rp_log2 = 7 - p.g_log2;
  auto slot = [&](int k) { return (size_t)(first + k) * 2 + (k == 0 ? 1 : 0); };
  // Neighbouring threads take neighbouring float4s of the parts' layout.  The first parts' values are
  // under way while the weights are found: with few parts the kernel is two round trips to L2.
  constexpr int kItems = kRows * (D / 4) / kThreads, kFirst = 4;
  auto row_of = [&](int j) { return (j * kThreads + (int)threadIdx.x) % kRows; };
  auto col_of = [&](int j) { return (j * kThreads + (int)threadIdx.x) / kRows; };
  auto source = [&](int j) { return parts.o + (blockIdx.y * kRows + row_of(j)) * 4 + col_of(j) * 4 * parts.rows; };
  float4 x[kItems][kFirst];
#pragma unroll
  for (int j = 0; j < kItems; ++j)
#pragma unroll
    for (int k = 0; k < kFirst; ++k)
      if (k < n) x[j][k] = *reinterpret_cast<const float4*>(source(j) + slot(k) * parts.rows * D);
  {  // sixteen lanes for each row
    const int lr = threadIdx.x / 16, lane = threadIdx.x % 16, row = blockIdx.y * kRows + lr;
    float top = -INFINITY;
    for (int k = lane; k < n; k += 16) {
      const float m = parts.ml[slot(k) * 2 * parts.rows + row];
      total[k][lr] = parts.ml[(slot(k) * 2 + 1) * parts.rows + row];
      weight[k][lr] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.f;
    for (int k = lane; k < n; k += 16) {
      const float m = weight[k][lr], f = m == top ? 1.f : exp2f(m - top);
      weight[k][lr] = f;
      sum += f * total[k][lr];
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) inverse[lr] = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no key: zeros
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int lr = row_of(j), c4 = col_of(j), row = blockIdx.y * kRows + lr;
    const int tok = ((row >> 7) << rp_log2) + (row & ((1 << rp_log2) - 1)), head = (row & 127) >> rp_log2;
    if (tok >= meta.n_tok) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, const float4& o) {
      const float f = weight[k][lr];
      a.x += f * o.x;
      a.y += f * o.y;
      a.z += f * o.z;
      a.w += f * o.w;
    };
#pragma unroll
    for (int k = 0; k < kFirst; ++k)
      if (k < n) add(k, x[j][k]);
    const float* src = source(j);
#pragma unroll 8
    for (int k = kFirst; k < n; ++k) add(k, *reinterpret_cast<const float4*>(src + slot(k) * parts.rows * D));
    const float inv = inverse[lr];
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.data) + (int64_t)(meta.tok0 + tok) * out.ts + (int64_t)(meta.g * p.G + head) * out.hs + c4 * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
}

}  // namespace

cudaError_t launch_paged_combine(const Paged& p, const Rows& out, const Parts& parts, cudaStream_t st) {
  // A programmatic launch: the blocks are in place when the kernel that leaves the parts ends.
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts.ctas, (parts.rows + kRows - 1) / kRows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = p.D == 64 ? cudaLaunchKernelEx(&cfg, paged_combine<64>, p, out, parts)
                                  : cudaLaunchKernelEx(&cfg, paged_combine<128>, p, out, parts);
  count_launches(1);
  return e;
}

}  // namespace tsa
