// Attention of a chunk of new tokens over the paged cache on the tcgen05 tensor
// cores (bf16 queries, fp32 accumulators in TMEM).
//
// A tile has 256 rows: two M tiles of 128, row r of tile t being query head
// r / RP of the KV head's G and new token t RP + r % RP, RP = 128 / G, so that
// every K/V tile in shared memory serves all G heads.  Keys come in tiles of 128
// cached positions.  CTAs are persistent, one per SM, each with an equal run of
// (tile, key tile) pairs (paged_plan.cuh); a tile cut by a run's end leaves fp32
// partial results for the combining kernel.
//
// Warp roles (512 threads):
//   warps 0-3, 4-7  softmax and epilogue of M tile 0 / 1 (thread = TMEM lane = row)
//   warps 8-11      preparation: Q tiles (16-byte copies into the swizzled layout);
//                   8-bit codes -> bf16 K/V tiles; bf16 V tiles at the causal border
//   warps 12, 14    MMA issuers (a whole warp each, one elected lane) of M tile 0 / 1: S_t = Q_t K^T, O_t += P_t V
//   warp 13         loads: one TMA box or bulk copy for each page of a tile, issued
//                   by as many lanes
// A step is half a key tile, 64 keys.  TMEM: for each M tile two buffers of 64 columns
// for S, [0,128) and [128,256); O0 [256,256+D) O1 [256+D,256+2D); P (bf16) overwrites
// the first 32 columns of its S.
//
// The two buffers of S let the softmax work on half u + 1 while the tensor core
// does PV of half u and QK of half u + 2.  An issuing warp executes as a whole with
// one elected lane, so that the products' operands stay in uniform registers: in a
// branch of one lane each product cost some 80 clocks to issue, as long as it takes
// to execute (8192 tokens: 659 us that way, 572 this way).  What bounds the kernel
// now is the softmax of each M tile: about 1500 clocks for a half, of which the
// exponential unit needs 512 (and as many for the other M tile).
//
// 8-bit caches: the codes are exact in bf16; the preparing warps convert them and
// put the scales of the key tile where the softmax warps find them: the scale of a
// key multiplies its logits, the scale of a value its probability, in fp32.  (Rows
// rounded to bf16 with their scale in them: twice the error.)
//
// Measured: a prompt of 8192 tokens in bf16, 32/8 heads: 561 us, 980 TFLOP/s, in
// short runs and 610 to 620 in long ones (the power limit lowers the clock); 1023
// tokens over 131071 in int8: 2.6 ms, 830 TFLOP/s.
//
// Hidden keys have P = 0.  A hidden value row that is not finite would still give
// 0 * inf, and memory behind the sequence's end may hold anything (codes are always
// finite, bf16 rows are not), so for bf16 key tiles at the causal border the
// preparing warps clear what lies behind the last key, and take non-finite elements
// out of the V tile, noting the first row that sees each (three kinds for each
// column); the epilogue adds them back to the rows that do.
//
// Every mbarrier wait is bounded; on timeout the CTA records TSA_ERR_TIMEOUT,
// drains its own copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"
#include "paged_plan.cuh"
#include "paged_ptx.cuh"
#include "tma_maps.h"

namespace tsa {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kChunkRows = 256;  // rows of a tile
constexpr int kPrepWarp0 = 8;
constexpr int kPrepWarps = 4;
constexpr int kMmaWarp0 = 12;  // M tile 0; M tile 1: warp 14, on another scheduler
constexpr int kLoadWarp = 13;
constexpr int kMmaWarp1 = 14;
constexpr uint32_t kDrainPolls = 1u << 26;
constexpr float kMoveReference = 8.0f;  // log2 units
constexpr uint32_t kNever = 1023;       // "no row": tiles have at most 256 tokens and border keys 383 behind the first
constexpr uint32_t kNoneOdd = kNever | (kNever << 10) | (kNever << 20);

template <int D, int CODE>
struct Cfg {
  static constexpr bool QUANT = CODE != kPlain;
  static constexpr int TILE = 128 * D * 2;                      // a bf16 K, V or Q tile
  static constexpr int NS = QUANT ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);  // K/V ring
  static constexpr int NR = QUANT ? 3 : 0;                      // ring of raw code tiles
  static constexpr int RAW = 128 * D + 1024;                    // codes, then (K tiles) the scales of 128 keys and values
  // Scales of a key tile stay until both M tiles' softmax has used them.  The tile that is converted
  // when V of key tile j has been released is at most NS - 1 tiles further on.
  static constexpr int SD = QUANT ? NS / 2 + 1 : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_RAW = OFF_KV + NS * TILE;
  static constexpr int OFF_SCALE = OFF_RAW + NR * RAW;          // [SD][2][128] floats
  static constexpr int OFF_ODD = OFF_SCALE + SD * 1024;         // [3][D] packed first rows of non-finite values
  static constexpr int OFF_BAR = OFF_ODD + (QUANT ? 0 : 3 * D * 4);
  // q[2], qfree[2], full[NS], empty[NS], s[4], p[4], o[2], teardown, border[NS] or raw_full[NR], raw_empty[NR]
  static constexpr int NBAR = 4 + 2 * NS + 10 + 1 + (QUANT ? 2 * NR : NS);
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;           // tmem slot, abort flag, odd[3], done[8]
  static constexpr int OFF_PLAN = (OFF_MISC + 64 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_PLAN + (int)sizeof(PlanSmem);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static constexpr int CPR = D / 8;      // 16-byte chunks of a bf16 row
  static constexpr int RPI = 32 / CPR;   // rows of a warp-wide copy
  static constexpr uint32_t O_COL0 = 256u;
};

struct ChunkParams {
  Paged p;
  Rows q, out;
  Parts parts;
  Plan plan;
  int rp_log2;  // tokens of an M tile
  float scale_log2;
  uint64_t wait_limit;
};

// Orders uses of r after an earlier wait for TMEM loads.
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

__device__ __forceinline__ void mul2(uint32_t& a, uint32_t& b, uint32_t x, uint32_t y) {
  float f, g;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(a), __uint_as_float(b)), f2_pack(__uint_as_float(x), __uint_as_float(y))), f, g);
  a = __float_as_uint(f);
  b = __float_as_uint(g);
}

// Register split: the softmax warps hold a row of S.  The block is launched with 512 x 128
// registers; 256 x 184 + 256 x 72 is exactly that, and both sides run this before anything else.
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;
static_assert(256 * (kSoftmaxRegs + kOtherRegs) <= kThreads * 128, "registers of the block");

__device__ __forceinline__ bool any_odd(uint32_t w) { return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0; }

// Notes that rows from `off` tokens behind the tile's first on see a non-finite
// value of bf16 bits h in this column.  Three fields: +inf, -inf, NaN.
__device__ __noinline__ void note_odd(uint32_t* word, uint32_t h, uint32_t off) {
  const int f = (h & 0x7f) ? 20 : (h & 0x8000) ? 10 : 0;
  uint32_t old = *reinterpret_cast<volatile uint32_t*>(word);
  while (((old >> f) & 1023u) > off) {
    const uint32_t put = (old & ~(1023u << f)) | (off << f);
    const uint32_t seen = atomicCAS(word, old, put);
    if (seen == old) break;
    old = seen;
  }
}

// One tile of rows, or the part of it that this CTA does: every role walks the same list.
struct Seg {
  Cursor c;
  int kt1, units, keys;
  int tok0, n_tok, pos0;  // packed row, tokens and first position of the tile
  int nt;                 // M tiles with rows
  int nh;                 // steps: halves of key tiles with keys (at least one)
};

__device__ __forceinline__ Seg make_seg(const ChunkParams& P, const Cursor& c, long long left) {
  Seg s;
  s.c = c;
  s.units = P.plan.units(c.span, c.j);
  s.keys = P.plan.keys(c.span, c.j);
  s.kt1 = (int)min((long long)s.units, c.kt + left);
  const int first = c.j << P.plan.tt_log2;
  s.tok0 = c.span.tok0 + first;
  s.n_tok = min(1 << P.plan.tt_log2, c.span.n - first);
  s.pos0 = c.span.base + first;
  s.nt = s.n_tok > (1 << P.rp_log2) ? 2 : 1;
  s.nh = max(1, min(2 * (s.kt1 - c.kt), (int)(((long long)s.keys + 63) >> 6) - 2 * c.kt));
  return s;
}

template <int D, int CODE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk(const __grid_constant__ ChunkParams P, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, CODE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const Paged& p = P.p;
  const uint32_t sQ = base + C::OFF_Q, sKV = base + C::OFF_KV, sRaw = base + C::OFF_RAW;
  const uint32_t bar0 = base + C::OFF_BAR;
  auto bar_q = [&](int t) { return bar0 + 8u * t; };
  auto bar_qfree = [&](int t) { return bar0 + 8u * (2 + t); };
  auto bar_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto bar_empty = [&](int s) { return bar0 + 8u * (4 + C::NS + s); };
  auto bar_s = [&](int t, int b) { return bar0 + 8u * (4 + 2 * C::NS + 2 * t + b); };
  auto bar_p = [&](int t, int b) { return bar0 + 8u * (8 + 2 * C::NS + 2 * t + b); };
  auto bar_o = [&](int t) { return bar0 + 8u * (12 + 2 * C::NS + t); };
  const uint32_t bar_td = bar0 + 8u * (14 + 2 * C::NS);
  // What the preparing warps wait for: V tiles at the border (by ring stage), or raw tiles.
  auto bar_border = [&](int s) { return bar0 + 8u * (15 + 2 * C::NS + s); };
  auto bar_rfull = [&](int s) { return bar0 + 8u * (15 + 2 * C::NS + s); };
  auto bar_rempty = [&](int s) { return bar0 + 8u * (15 + 2 * C::NS + C::NR + s); };
  uint32_t* odd_cols = reinterpret_cast<uint32_t*>(smem + C::OFF_ODD);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* odd_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);  // [3]
  volatile int* done = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 20);     // [8]: segments that each softmax warp has left
  PlanSmem* psm = reinterpret_cast<PlanSmem*>(smem + C::OFF_PLAN);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_q(t), 32 * kPrepWarps);
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_s(t, b), 1);
        mbar_init(bar_p(t, b), 4);  // the softmax warps of an M tile
      }
      mbar_init(bar_o(t), 1);
      mbar_init(bar_qfree(t), 1);
    }
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar_full(s), kPrepWarps);  // one arrival of each preparing warp, or as many of the loading one
      mbar_init(bar_empty(s), 2);
      if (!C::QUANT) mbar_init(bar_border(s), 1);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(bar_rfull(s), 1);
      mbar_init(bar_rempty(s), kPrepWarps);
    }
    mbar_init(bar_td, 2);
    *abort_flag = 0;
    odd_flag[0] = odd_flag[1] = odd_flag[2] = 0;
    for (int w = 0; w < 8; ++w) done[w] = 0;
    fence_mbar_init();
    P.parts.meta[blockIdx.x].c_end = -1;
  }
  if (!C::QUANT)
    for (int i = threadIdx.x; i < 3 * D; i += kThreads) odd_cols[i] = kNoneOdd;
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  Cursor cur;
  long long left, run;
  grid_dependency_launch();
  plan_start<kThreads>(p, P.plan, psm, &cur, &left, &run);  // ends with __syncthreads
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    record_status(p.status, TSA_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  // Walks the CTA's segments: f(segment, its index) returns false to stop.
  auto walk = [&](auto&& f) {
    for (int i = 0; left > 0; ++i) {
      const Seg s = make_seg(P, cur, left);
      if (!f(s, i)) break;
      left -= s.kt1 - cur.kt;
      if (left > 0) plan_next(p, P.plan, &cur);
    }
  };

  if (warp >= 8) {
    regs_dec<kOtherRegs>();
  if (warp >= kPrepWarp0 && warp < kPrepWarp0 + kPrepWarps) {
    // ------------------------------------------------------------ preparation
    const int pw = warp - kPrepWarp0;
    uint32_t kv = 0;   // K/V tiles so far: ring stage kv % NS
    uint32_t q1_used = 0;  // Q tiles of M tile 1 so far (M tile 0 has one in every segment)
    [[maybe_unused]] uint32_t seen = 0;  // phase of each stage's border barrier
    walk([&](const Seg& s, int i) -> bool {
      uint32_t* odd = odd_cols + (i % 3) * D;
      // Clear the next segment's notes once every softmax warp has left the segment that used them
      // last.  The other preparing warps write there only after all have arrived on bar_q below.
      if constexpr (!C::QUANT) {
        bool free = i < 2 || lane >= 8 || done[lane] >= i - 1;
        for (uint64_t k = 0; k < P.wait_limit && !free && *abort_flag == 0; ++k) {
          __nanosleep(32);
          free = done[lane] >= i - 1;
        }
        if (!__all_sync(0xffffffffu, free)) {
          if (lane == 0) fail();
          return false;
        }
        __threadfence_block();
        uint32_t* next = odd_cols + ((i + 1) % 3) * D;
        for (int c = pw * 32 + lane; c < D; c += 32 * kPrepWarps) next[c] = kNoneOdd;
        if (pw == 0 && lane == 0) odd_flag[(i + 1) % 3] = 0;
        __threadfence_block();
      }
      const int my_c = lane % C::CPR, my_r = lane / C::CPR;
      for (int t = 0; t < s.nt; ++t) {
        if (t == 0 ? i > 0 : q1_used > 0) {  // the tensor core has read the Q tile that was here
          const uint32_t ph = (t == 0 ? (uint32_t)i : q1_used) - 1;
          if (!__all_sync(0xffffffffu, mbar_wait(bar_qfree(t), ph & 1, P.wait_limit, abort_flag))) {
            if (lane == 0) fail();
            return false;
          }
        }
        q1_used += t;
#pragma unroll 4
        for (int n = 0; n < 32 / C::RPI; ++n) {
          const int row = 32 * pw + n * C::RPI + my_r;
          const int hh = row >> P.rp_log2;
          const int tok = min((t << P.rp_log2) + (row & ((1 << P.rp_log2) - 1)), s.n_tok - 1);
          const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(P.q.data) + (int64_t)(s.tok0 + tok) * P.q.ts +
                                   (int64_t)(s.c.g * p.G + hh) * P.q.hs + my_c * 8;
          cp_async16(sQ + t * C::TILE + (uint32_t)(my_c >> 3) * 16384u + row * 128 +
                         ((((uint32_t)my_c & 7u) ^ ((uint32_t)row & 7u)) << 4), g);
        }
        cp_async_mbar_arrive(bar_q(t));
      }
      for (int kt = s.c.kt; kt < s.kt1; ++kt) {
        const int key0 = kt * 128;
        const bool border = key0 + 127 > s.pos0;
        if constexpr (!C::QUANT) {
          if (border) {  // V tile kv + 1
            const uint32_t st = (kv + 1) % C::NS;
            if (!__all_sync(0xffffffffu, mbar_wait(bar_border(st), (seen >> st) & 1, P.wait_limit, abort_flag))) {
              if (lane == 0) fail();
              return false;
            }
            seen ^= 1u << st;
            const uint32_t sv = sKV + st * C::TILE;
#pragma unroll 4
            for (int n = 0; n < 32 / C::RPI; ++n) {
              const int row = 32 * pw + n * C::RPI + my_r;
              const uint32_t addr = sv + (uint32_t)(my_c >> 3) * 16384u + row * 128 + ((((uint32_t)my_c & 7u) ^ ((uint32_t)row & 7u)) << 4);
              if (key0 + row >= s.keys) {
                st_shared_v4(addr, 0u, 0u, 0u, 0u);
              } else if (key0 + row > s.pos0) {
                const uint4 x = lds128(addr);
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                if (any_odd(w[0]) || any_odd(w[1]) || any_odd(w[2]) || any_odd(w[3])) {
                  for (int e = 0; e < 8; ++e) {
                    const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                    if ((h & 0x7f80u) == 0x7f80u) {
                      note_odd(odd + my_c * 8 + e, h, (uint32_t)(key0 + row - s.pos0));
                      w[e >> 1] &= 0xffff0000u >> (16 * (e & 1));
                    }
                  }
                  odd_flag[i % 3] = 1;
                  st_shared_v4(addr, w[0], w[1], w[2], w[3]);
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full(st));
          }
          kv += 2;
        } else {
#pragma unroll 1
          for (int is_v = 0; is_v < 2; ++is_v, ++kv) {
            const uint32_t rs = kv % C::NR, st = kv % C::NS;
            bool got = mbar_wait(bar_rfull(rs), (kv / C::NR) & 1, P.wait_limit, abort_flag);
            if (got && kv >= C::NS) got = mbar_wait(bar_empty(st), ((kv / C::NS) - 1) & 1, P.wait_limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
              if (lane == 0) fail();
              return false;
            }
            if (!is_v) {  // a thread for each key: its scales
              const int key = 32 * pw + lane;
              const float* sc = reinterpret_cast<const float*>(smem + C::OFF_RAW + rs * C::RAW + 128 * D);
              float* to = reinterpret_cast<float*>(smem + C::OFF_SCALE + (kv >> 1) % C::SD * 1024);
              to[key] = sc[key] * P.scale_log2;
              to[128 + key] = sc[128 + key];
            }
            const uint32_t src = sRaw + rs * C::RAW + (32 * pw + my_r) * D + my_c * 8;
            const uint32_t dst = sKV + st * C::TILE + (uint32_t)(my_c >> 3) * 16384u;
            constexpr int B = 8;  // pieces in flight
#pragma unroll 1
            for (int n0 = 0; n0 < 32 / C::RPI; n0 += B) {
              uint2 x[B];
#pragma unroll
              for (int n = 0; n < B; ++n) x[n] = lds64(src + (n0 + n) * C::RPI * D);
#pragma unroll
              for (int n = 0; n < B; ++n) {
                const uint32_t row = 32 * pw + (n0 + n) * C::RPI + my_r;
                st_shared_v4(dst + row * 128 + ((((uint32_t)my_c ^ row) & 7u) << 4), codes_next<CODE, 0>(x[n].x),
                             codes_next<CODE, 2>(x[n].x), codes_next<CODE, 0>(x[n].y), codes_next<CODE, 2>(x[n].y));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar_rempty(rs));
              mbar_arrive(bar_full(st));
            }
          }
        }
      }
      return true;
    });
    cp_async_wait_all();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    const int box_log2 = min(p.page_log2, 7);  // keys of one copy
    const int box = 1 << box_log2;
    uint32_t n = 0;  // tiles so far
    uint32_t at_border = 0, borders = 0;  // by stage: the last tile is one of the border; phase of its border barrier
    constexpr uint32_t RING = C::QUANT ? C::NR : C::NS;
    auto empty = [&](uint32_t s) { return C::QUANT ? bar_rempty(s) : bar_empty(s); };
    walk([&](const Seg& s, int) -> bool {
      // Lane b copies page piece b of a tile; its page is read one tile ahead.
      auto lookup = [&](int kt) -> int {
        const int key = kt * 128 + (lane << box_log2);
        return lane < (128 >> box_log2) && key < s.keys ? __ldg(p.table + (size_t)s.c.s * p.max_pages + (key >> p.page_log2)) : 0;
      };
      int entry = lookup(s.c.kt);
      for (int kt = s.c.kt; kt < s.kt1; ++kt) {
        const int key = kt * 128 + (lane << box_log2);
        const bool mine = lane < (128 >> box_log2) && key < s.keys;
        const int page = mine ? checked_page(p, entry) : 0;
        const int next = kt + 1 < s.kt1 ? lookup(kt + 1) : 0;
        const size_t row = (((size_t)page * p.Hkv + s.c.g) << p.page_log2) + (key & ((1 << p.page_log2) - 1));
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll 1
        for (int is_v = 0; is_v < 2; ++is_v, ++n) {
          const uint32_t st = n % RING;
          if (n >= RING && !__all_sync(0xffffffffu, mbar_wait(empty(st), ((n / RING) - 1) & 1, P.wait_limit, abort_flag))) {
            if (lane == 0) fail();
            return false;
          }
          const bool border = !C::QUANT && is_v && kt * 128 + 127 > s.pos0;  // goes through the preparing warps
          const uint32_t b = C::QUANT ? bar_rfull(st) : border ? bar_border(st) : bar_full(st);
          if (!C::QUANT) at_border = (at_border & ~(1u << st)) | ((uint32_t)border << st);
          if (border) borders ^= 1u << st;
          if (lane == 0) {
            mbar_arrive_expect_tx(b, boxes * box * (C::QUANT ? (is_v ? D : D + 8) : D * 2));
            if (!C::QUANT && !border)
              for (int w = 1; w < kPrepWarps; ++w) mbar_arrive(b);
          }
          __syncwarp();
          if (mine) {
            if constexpr (C::QUANT) {
              const uint32_t dst = sRaw + st * C::RAW;
              const uint8_t* codes = static_cast<const uint8_t*>(is_v ? p.v_pages : p.k_pages);
              bulk_load(dst + (lane << box_log2) * D, codes + row * D, box * D, b);
              if (!is_v) {
                bulk_load(dst + 128 * D + (lane << box_log2) * 4, p.k_scales + row, box * 4, b);
                bulk_load(dst + 128 * D + 512 + (lane << box_log2) * 4, p.v_scales + row, box * 4, b);
              }
            } else {
              const uint32_t dst = sKV + st * C::TILE + (lane << box_log2) * 128;
#pragma unroll
              for (int h = 0; h < D / 64; ++h) tma_load_2d(dst + h * 16384, is_v ? &vmap : &kmap, b, h * 64, (int)row);
            }
          }
          __syncwarp();
        }
        entry = next;
      }
      return true;
    });
    // The last copies must land before the CTA exits, and after an abort nobody else may be waiting for them.
    for (uint32_t k = n > RING ? n - RING : 0; k < n; ++k) {
      const uint32_t st = k % RING;
      if (C::QUANT) mbar_wait(bar_rfull(st), (k / RING) & 1, kDrainPolls, nullptr);
      else if ((at_border >> st) & 1) mbar_wait(bar_border(st), ((borders >> st) & 1) ^ 1, kDrainPolls, nullptr);
      else mbar_wait(bar_full(st), (k / RING) & 1, kDrainPolls, nullptr);
    }
  } else if (warp == kMmaWarp0 || warp == kMmaWarp1) {
    // ------------------------------------------------------------ MMA issuers, one for each M tile
    // Step u: PV of half u, then QK of half u + 2 into the place that P_u leaves.  The softmax works on
    // half u + 1 meanwhile, so neither a barrier's latency nor the other M tile's products hold it up.
    {
      const uint32_t on = elect_one();
      const int t = warp == kMmaWarp1;
      constexpr uint32_t IDESC_QK = idesc_bf16(128, 64, 0, 0);
      constexpr uint32_t IDESC_PV = idesc_bf16(128, D, 0, 1);
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      const uint32_t tS = tmem + t * 128u, tO = tmem + C::O_COL0 + t * D;
      const uint32_t q_lo = sdesc_lo(sQ + t * C::TILE, 16), k_lo = sdesc_lo(sKV, 16), v_lo = sdesc_lo(sKV, 16384);
      bool ok = true;
      // Ring stage and phase of the next K and V tile.  A segment's tiles alternate from K on.
      uint32_t kst = 0, kph = 0, vst = 1, vph = 0;
      uint32_t pph = 0, nq = 0;  // phases of bar_p by buffer; Q tiles so far
      auto advance = [&](uint32_t& st, uint32_t& ph) {
        st += 2;
        if (st >= (uint32_t)C::NS) {
          st -= C::NS;
          ph ^= 1;
        }
      };
      auto wait_full = [&](uint32_t st, uint32_t ph) { return __all_sync(0xffffffffu, mbar_wait(bar_full(st), ph, P.wait_limit, abort_flag)); };
      auto qk = [&](int u) {  // half u into its buffer
        const uint32_t b = k_lo + kst * (C::TILE >> 4) + (u & 1) * 512, d = tS + (u & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
          if (kk == 0) mma_bf16_ss_lo<false>(on, d, q_lo + off, b + off, HI, IDESC_QK);
          else mma_bf16_ss_lo<true>(on, d, q_lo + off, b + off, HI, IDESC_QK);
        }
        tc_commit_on(on, bar_s(t, u & 1));
      };
      walk([&](const Seg& s, int) -> bool {
        const int nh = s.nh;
        // The K tile is done with after its second half, or the last half of all.
        auto k_done = [&](int u) {
          if (u & 1 || u == nh - 1) {
            tc_commit_on(on, bar_empty(kst));
            advance(kst, kph);
          }
          if (u == nh - 1) tc_commit_on(on, bar_qfree(t));
        };
        if (t >= s.nt) {  // no rows here: release the tiles as they come
          for (int kt = s.c.kt; kt < s.kt1; ++kt) {
            if (!(ok = wait_full(kst, kph))) return false;
            if (on) mbar_arrive(bar_empty(kst));
            advance(kst, kph);
            if (!(ok = wait_full(vst, vph))) return false;
            if (on) mbar_arrive(bar_empty(vst));
            advance(vst, vph);
          }
          return true;
        }
        if (!(ok = wait_full(kst, kph))) return false;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar_q(t), nq++ & 1, P.wait_limit, abort_flag)))) return false;
        fence_proxy_async_smem();  // rows landed by cp.async are read by the tensor core
        tc_fence_after();
        for (int u = 0; u < 2 && u < nh; ++u) {
          qk(u);
          k_done(u);
        }
        for (int u = 0; u < nh; ++u) {
          bool k_ready = true;  // asked before the wait for P, so that the answer is there after it
          if ((u & 1) == 0) {
            if (!(ok = wait_full(vst, vph))) return false;
            k_ready = u + 2 >= nh || __all_sync(0xffffffffu, mbar_test(bar_full(kst), kph));
          }
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar_p(t, u & 1), (pph >> (u & 1)) & 1, P.wait_limit, abort_flag)))) return false;
          pph ^= 1u << (u & 1);
          tc_fence_after();
          const uint32_t a = tS + (u & 1) * 64, b = v_lo + vst * (C::TILE >> 4) + (u & 1) * 512;
          if (u == 0) mma_bf16_ts_lo<false>(on, tO, a, b, HI, IDESC_PV);
          else mma_bf16_ts_lo<true>(on, tO, a, b, HI, IDESC_PV);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) mma_bf16_ts_lo<true>(on, tO, a + kk * 8, b + kk * 128, HI, IDESC_PV);
          if (u + 2 < nh) {
            if (!k_ready) {
              if (!(ok = wait_full(kst, kph))) return false;
              tc_fence_after();
            }
            qk(u + 2);
          } else {
            tc_commit_on(on, bar_o(t));  // the last two steps
          }
          if (u & 1 || u == nh - 1) {
            tc_commit_on(on, bar_empty(vst));
            advance(vst, vph);
          }
          if (u + 2 < nh) k_done(u + 2);
        }
        return true;
      });
      if (!ok && lane == 0) fail();
      __syncwarp();
      tc_commit_on(on, bar_td);  // every MMA has finished before TMEM is released
      mbar_wait(bar_td, 0, kDrainPolls, nullptr);
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    regs_inc<kSoftmaxRegs>();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS0 = tmem + lane_off + (uint32_t)t * 128u;
    const uint32_t tO = tmem + lane_off + C::O_COL0 + t * D;
    const int hh = r >> P.rp_log2, tok = (t << P.rp_log2) + (r & ((1 << P.rp_log2) - 1));
    uint32_t sph = 0, no = 0;  // phases of bar_s by buffer; waits on bar_o
    [[maybe_unused]] uint32_t unit = 0;  // key tiles so far
    bool ok = true;
    auto wait_o = [&]() {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_o(t), no++ & 1, P.wait_limit, abort_flag));
      return ok;
    };
    walk([&](const Seg& s, int i) -> bool {
      auto leave = [&]() {
        __threadfence_block();
        __syncwarp();
        if (lane == 0) done[warp] = i + 1;
      };
      if (t >= s.nt) {
        leave();
        unit += s.kt1 - s.c.kt;
        return true;
      }
      const int pos = s.pos0 + min(tok, s.n_tok - 1);
      const int last = min(pos + 1, s.keys);  // keys this row sees
      float m_use = -INFINITY, l = 0.f;
      bool s_ready = false;
      for (int u = 0; u < s.nh; ++u) {
        const int buf = u & 1;
        if (!s_ready) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar_s(t, buf), (sph >> buf) & 1, P.wait_limit, abort_flag));
          if (!ok) return false;
        }
        sph ^= 1u << buf;
        tc_fence_after();
        const uint32_t tS = tS0 + buf * 64;
        const int nvis = last - (2 * s.c.kt + u) * 64;
        const bool masked = (2 * s.c.kt + u) * 64 + 63 > s.pos0;  // some row of the tile does not see all of it
        float alpha = 1.f;
        bool rescaled = false;
        uint64_t acc2 = 0ull;
        // 8 bits: the scales of this half (K's already in log2 units)
        [[maybe_unused]] const uint32_t ksc =
            base + C::OFF_SCALE + (C::QUANT ? (unit + (u >> 1)) % (C::SD + !C::QUANT) : 0) * 1024 + buf * 256, vsc = ksc + 512;
        auto tile = [&](auto masked_c) {
          constexpr bool kMasked = decltype(masked_c)::value;
          auto xval = [&](const uint32_t* v, int q4, int e) -> float {
            const float x = __uint_as_float(v[e]);
            return (!kMasked || q4 * 32 + e < nvis) ? x : -INFINITY;
          };
          uint32_t v[2][32];
          tmem_ld32_async(tS, v[0]);
          tmem_ld32_async(tS + 32, v[1]);
          tmem_wait_ld32(v[0]);
          tie32(v[1]);
          if constexpr (C::QUANT) {  // logits in place
#pragma unroll
            for (int q4 = 0; q4 < 2; ++q4)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const uint4 f = lds128(ksc + (q4 * 32 + e) * 4);
                const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int c = 0; c < 4; c += 2) mul2(v[q4][e + c], v[q4][e + c + 1], w[c], w[c + 1]);
              }
          }
          float mxs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q4 = 0; q4 < 2; ++q4)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int c = 0; c < 4; ++c) mxs[c] = fmax3(mxs[c], xval(v[q4], q4, e + 2 * c), xval(v[q4], q4, e + 2 * c + 1));
          const float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3]));
          const float mt = C::QUANT ? mx : mx * P.scale_log2;
          const bool need = mt > m_use + kMoveReference;
          alpha = need ? ex2_approx(m_use - mt) : 1.f;
          m_use = need ? mt : m_use;
          rescaled = u > 0 && __any_sync(0xffffffffu, need);
          const uint64_t scale2 = f2_pack(P.scale_log2, P.scale_log2);
          const float mref = m_use == -INFINITY ? 0.f : m_use;
          const uint64_t negm2 = f2_pack(-mref, -mref);
          uint64_t accq[2] = {0ull, 0ull};
#pragma unroll
          for (int q4 = 0; q4 < 2; ++q4) {
            uint32_t pk[16];
            [[maybe_unused]] uint4 vs;
#pragma unroll
            for (int e2 = 0; e2 < 16; ++e2) {
              float t0, t1;
              const uint64_t x2 = f2_pack(xval(v[q4], q4, 2 * e2), xval(v[q4], q4, 2 * e2 + 1));
              f2_unpack(C::QUANT ? f2_add(x2, negm2) : f2_fma(x2, scale2, negm2), t0, t1);
              float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              accq[e2 & 1] = f2_add(accq[e2 & 1], f2_pack(p0, p1));
              if constexpr (C::QUANT) {
                if ((e2 & 1) == 0) vs = lds128(vsc + (q4 * 32 + 2 * e2) * 4);
                const uint32_t s0 = (e2 & 1) ? vs.z : vs.x, s1 = (e2 & 1) ? vs.w : vs.y;
                f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(__uint_as_float(s0), __uint_as_float(s1))), p0, p1);
                if (kMasked) {  // the scale of a key that is not seen may be anything
                  if (q4 * 32 + 2 * e2 >= nvis) p0 = 0.f;
                  if (q4 * 32 + 2 * e2 + 1 >= nvis) p1 = 0.f;
                }
              }
              pk[e2] = pack_bf16x2(p0, p1);
            }
            tmem_st16(tS + q4 * 16, pk);
          }
          acc2 = f2_add(accq[0], accq[1]);
        };
        if (masked) tile(std::true_type{});
        else tile(std::false_type{});
        float s0, s1;
        f2_unpack(acc2, s0, s1);
        l = l * alpha + (s0 + s1);
        if (rescaled) {
          // The previous PV must have finished: the commit of the next S covers it, or the last but one of all.
          if (u + 1 < s.nh) ok = __all_sync(0xffffffffu, mbar_wait(bar_s(t, buf ^ 1), (sph >> (buf ^ 1)) & 1, P.wait_limit, abort_flag));
          else wait_o();
          if (!ok) return false;
          tc_fence_after();
#pragma unroll
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t v[32];
            tmem_ld32(tO + q4 * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st32(tO + q4 * 32, v);
          }
        }
        // The next half's logits are mostly there by now: asking here hides the answer's latency.
        const bool s_next = u + 1 < s.nh && mbar_test(bar_s(t, buf ^ 1), (sph >> (buf ^ 1)) & 1);
        tmem_st_wait();
        tc_fence_before();
        s_ready = __all_sync(0xffffffffu, s_next);
        // Every phase of bar_o is waited for before the next can complete: the last but one's needs this P.
        if (u == s.nh - 1 && u > 0 && !rescaled && !wait_o()) return false;
        if (lane == 0) mbar_arrive(bar_p(t, buf));
      }
      if (!wait_o()) return false;
      tc_fence_after();
      unit += s.kt1 - s.c.kt;
      const bool valid = tok < s.n_tok;
      const bool whole = s.c.kt == 0 && s.kt1 == s.units;
      const bool odd = !C::QUANT && s.kt1 * 128 > s.pos0 && odd_flag[i % 3] != 0;
      const uint32_t* oc = odd_cols + (i % 3) * D;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that saw no key: zeros
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(P.out.data) + (int64_t)(s.tok0 + min(tok, s.n_tok - 1)) * P.out.ts +
                            (int64_t)(s.c.g * p.G + hh) * P.out.hs;
      const size_t part = (size_t)blockIdx.x * 2 + (s.c.kt == 0 ? 1 : 0);
      const int prow = t * 128 + r;
      float* po = P.parts.o + part * kChunkRows * D + prow * 4;  // lanes are rows: their float4s side by side
#pragma unroll 1
      for (int q4 = 0; q4 < D / 32; ++q4) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tO + q4 * 32, v);  // warp-collective: every lane loads, valid rows store
        if (odd) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t w = oc[q4 * 32 + e];
            const uint32_t off = (uint32_t)tok;
            float x = __uint_as_float(v[e]);
            if (off >= (w & 1023u)) x += INFINITY;
            if (off >= ((w >> 10) & 1023u)) x -= INFINITY;
            if (off >= ((w >> 20) & 1023u)) x += __uint_as_float(0x7fffffffu);
            v[e] = __float_as_uint(x);
          }
        }
        if (!valid) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(orow + q4 * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = __uint_as_float(v[8 * e + u]) * inv;
            dst[e] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(po + (q4 * 8 + e) * (4 * kChunkRows)) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      if (!whole && valid) {
        P.parts.ml[(part * 2) * kChunkRows + prow] = m_use;
        P.parts.ml[(part * 2 + 1) * kChunkRows + prow] = l;
      }
      if (s.c.kt == 0 && s.kt1 < s.units && threadIdx.x == 0) {
        PartMeta mt;
        mt.c_end = plan_last_cta(p, s.units - s.kt1, run);
        mt.g = s.c.g;
        mt.tok0 = s.tok0;
        mt.n_tok = s.n_tok;
        P.parts.meta[blockIdx.x] = mt;
      }
      leave();
      return true;
    });
    if (!ok) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int CODE>
cudaError_t launch(const Paged& p, const Rows& q, const Rows& out, void* base, int which, cudaStream_t st) {
  using C = Cfg<D, CODE>;
  ChunkParams P;
  P.p = p;
  P.q = q;
  P.out = out;
  P.parts = make_parts(base, kChunkRows, kPagedCtas, D);
  P.plan.which = which;
  P.plan.kt_log2 = 7;
  P.plan.tt_log2 = 8 - p.g_log2;
  P.rp_log2 = 7 - p.g_log2;
  P.scale_log2 = p.scale * 1.4426950408889634f;
  P.wait_limit = wait_limit();
  CUtensorMap km = {}, vm = {};
  if (!C::QUANT) {
    const uint64_t rows = ((uint64_t)p.n_pages * p.Hkv) << p.page_log2;
    const int box = 1 << (p.page_log2 < 7 ? p.page_log2 : 7);
    if (!make_tile_map(&km, p.k_pages, rows, D, box) || !make_tile_map(&vm, p.v_pages, rows, D, box)) return cudaErrorInvalidValue;
  }
  // The register split counts on 128 registers a thread at launch: with fewer it would wait for ever.
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, paged_chunk<D, CODE>);
  if (e != cudaSuccess) return e;
  if (at.numRegs <= 120) return cudaErrorInvalidKernelImage;
  e = cudaFuncSetAttribute(paged_chunk<D, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  paged_chunk<D, CODE><<<kPagedCtas, kThreads, C::SMEM, st>>>(P, km, vm);
  count_launches(1);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_paged_combine(p, out, P.parts, st);
}

template <int D>
cudaError_t by_code(const Paged& p, const Rows& q, const Rows& out, void* base, int which, cudaStream_t st) {
  if (p.cache_dtype == TSA_I8) return launch<D, kI8>(p, q, out, base, which, st);
  if (p.cache_dtype == TSA_E4M3) return launch<D, kE4M3>(p, q, out, base, which, st);
  return launch<D, kPlain>(p, q, out, base, which, st);
}

}  // namespace

size_t paged_chunk_bytes(const Paged& p) { return parts_bytes(kChunkRows, kPagedCtas, p.D); }

cudaError_t launch_paged_chunk(const Paged& p, const Rows& q, const Rows& out, void* base, int which, cudaStream_t st) {
  return p.D == 64 ? by_code<64>(p, q, out, base, which, st) : by_code<128>(p, q, out, base, which, st);
}

}  // namespace tsa
