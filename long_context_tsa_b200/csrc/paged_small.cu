// Attention of a few new tokens over the paged cache (bf16 queries): single
// tokens of a decoding step, and short runs of up to 32 rows, a row being a new
// token and one of the G query heads of the KV head.
//
// Bound by reading the cache: per cached token and KV head 4 D bytes (bf16) or
// 2 D + 8 (8-bit) against 4 G D flops a new token.  So the tile is one of 16 or
// 32 rows in registers (mma.sync m16n8k16: with so few rows the tensor rate is no
// concern, and accumulators in registers need no round trip through TMEM), and
// everything else serves to keep loads in flight:
//
// - A CTA, one on each SM, has an equal run of the key tiles (paged_plan.cuh).
//   Stages of 128 keys go through a ring of TMA boxes, one box a page; each of
//   the 8 working warps takes 16 keys of a stage and has its own running
//   reference and sum and its own accumulators, joined when a tile of rows ends.
//   The ring runs on across the ends of tiles.
// - Four warps load.  Issuing a copy costs a warp some 80 clocks, so the working
//   warps must not do it (four 131072-token int8 contexts: 363 us with a loading
//   lane in each working warp, 287 with loading warps), and a copy covers as much
//   of a page as a stage holds.
// - 8-bit codes become bf16 (K) and f16 (V) without rounding: both kinds are exact
//   in both.  The scale of a key multiplies its logits, the scale of a value its
//   probability, in fp32; that product becomes f16 (bf16 there: error against 64
//   bits 0.0024 for 0.0017, half of it from the output's own rounding).  f16 has too
//   few exponents for that, so o has a reference of its own, which follows the row's
//   largest product as m follows its largest logit: products are at most 2^15 in the
//   unit of o, the largest so far at least 2^7, so that those down to 2^-21 of it keep
//   f16's 11 bits and smaller ones are off by at most 2^-32 of it.  (A unit set by the
//   scales alone loses all others to one large scale of no probability.)
// - Codes are read as whole 16-byte pieces of a row: the order of the contraction
//   index d, of the 16 keys and of the output columns is free as long as both
//   operands agree, and is chosen so that a thread's pieces are contiguous, a
//   quarter warp's fall into different banks, and K's codes need no byte moves.
//   The conversions (3 or 4 integer operations for 2 codes) are what bounds the
//   8-bit kernels: the ALU pipe is 58 % busy with one row tile, 44 % with two, where
//   two warps a scheduler do not cover each other's waits.
// - A step of one row tile takes a block of two stages at once for 8-bit caches,
//   which gives the scheduler two independent halves (int8: 241 us against 257 when
//   it was tried); with two row tiles the registers do not suffice for that (then
//   237 us against 217 for 16 x 8 tokens in e4m3).
// - The reference m of the softmax (and o's) moves only when a logit passes it by 2^8
//   (P <= 2^8, bf16's relative precision is the same there), found with one vote
//   a block; the sum over a row's four threads waits until the tile ends.
//
// bf16 caches: P is rounded to bf16 for the second product (at most 2^-8 relative,
// the precision of the output).  Sums, references and accumulators are fp32.
//
// A masked key has P = 0 exactly, also where its scale is not finite, and its scale
// does not move o's reference.  A value row that is not finite and hidden from some
// row of the tile would still give 0 * inf: where the causal border crosses the 16
// keys, non-finite values of an unscaled cache are added to the rows that see them
// and cleared in the tile.
//
// Measured: 61 sequences of up to 8192 tokens, bf16, one token each: 142 us, 5.6
// TB/s (86 % of a copy's rate); four of 131072 in int8: 260 us, 4.3 TB/s; 16 of up
// to 32768 in e4m3, up to 8 tokens each: 248 us, 2.4 TB/s.
#include <cuda.h>
#include <math.h>

#include "internal.h"
#include "paged.h"
#include "paged_codes.cuh"
#include "paged_join.cuh"
#include "paged_ptx.cuh"
#include "tma_maps.h"

namespace tsa {
namespace {

using namespace tc;

constexpr int kWarps = 8;        // working warps
constexpr int kLoaders = 4;      // loading warps
constexpr int kWork = 32 * kWarps;
constexpr int kThreads = kWork + 32 * kLoaders;
// Register split: 384 threads x 168 at launch; 256 x 224 + 128 x 56 is exactly that.
constexpr int kWorkRegs = 224, kLoadRegs = 56;
static_assert(kWork * kWorkRegs + 128 * kLoadRegs <= kThreads * 168, "registers of the block");
constexpr int kKeys = 16;               // keys of a block: a warp's part of a stage
constexpr int kStageKeys = kKeys * kWarps;
constexpr float kMoveReference = 8.f;   // log2 units
// The reference of o (8-bit caches), in log2 units.  A product at the reference is 2^kUnit; m is at most
// kMostAbove above the reference, so that the factor between the two fits fp32; o is multiplied by no less
// than 2^-126: what that brings down is lost in any case, but an infinity stays one.
constexpr float kUnit = 7.f, kMostAbove = 119.f, kLeastFactor = 1.17549435e-38f;
static_assert(kUnit + kMoveReference < 15.99f && kUnit + kMostAbove <= 126.f, "products as f16, factors as fp32");
constexpr uint32_t kDrainPolls = 1u << 20;

template <int D, int CODE, int MT>
struct Cfg {
  static constexpr int ESZ = CODE == kPlain ? 2 : 1;
  static constexpr int NB = CODE == kPlain || MT == 2 ? 1 : 2;      // stages of a step: a block of each for every warp
  static constexpr int KT_LOG2 = NB == 1 ? 7 : 8;  // keys of a step: the unit of the work split
  static constexpr bool QSM = MT == 2;                   // Q fragments in shared memory
  static constexpr int KV_BYTES = kStageKeys * D * ESZ;  // K or V of a stage
  static constexpr int SC_BYTES = CODE == kPlain ? 0 : 2 * kStageKeys * 4;
  static constexpr int STAGE = 2 * KV_BYTES + SC_BYTES;
  static constexpr int RING = (CODE == kPlain && MT == 1 ? 192 : 170) * 1024;  // what the rest leaves
  static constexpr int NS = RING / STAGE > 8 ? 8 : RING / STAGE;
  static constexpr int ROWS = 16 * MT;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_JOIN = NS * STAGE;            // 4 partial tiles of 16 rows
  static constexpr int OFF_Q = OFF_JOIN + 4 * 16 * D * 4;  // [MT][D / 16][32 lanes] 16 bytes
  static constexpr int OFF_ML = OFF_Q + (QSM ? MT * (D / 16) * 512 : 0);  // [8 warps][ROWS][m, l]
  static constexpr int OFF_BAR = OFF_ML + kWarps * ROWS * 8;
  static constexpr int OFF_PLAN = OFF_BAR + 2 * NS * 8 + 16;  // full and empty barriers, abort flag
  static constexpr int OFF_LAST = OFF_PLAN + (int)sizeof(PlanSmem);
  static constexpr int SMEM = OFF_LAST + (int)sizeof(JoinSmem<ROWS>);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static constexpr int NKS = D / 16;  // k steps of QK
  static constexpr int NNT = D / 8;   // column tiles of O
};

struct SmallParams {
  Paged p;
  Rows q, out;
  Parts parts;
  Plan plan;
  float scale_log2;
  uint64_t wait_limit;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// The order of keys, contraction index and output columns inside a block of 16 keys.
template <int D, int CODE>
struct Order {
  // Key of index n (0..7) of a column tile of S, and of index k = 2j, 2j+1 of P.
  __device__ static __forceinline__ int key(int n) {
    return CODE != kPlain && D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
  }
  // Piece of an 8-bit V row that thread row c (0..7) reads.
  __device__ static __forceinline__ int piece(int c) { return D == 128 ? (c >> 1) | ((c & 1) << 2) : c; }
  // First column d of output index n (0..7): column tile nt is at first + nt (8-bit) or 8 nt + n.
  __device__ static __forceinline__ int col(int n, int nt) {
    return CODE == kPlain ? 8 * nt + n : piece(n) * (D / 8) + nt;
  }
};

template <int D, int CODE, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_small(const __grid_constant__ SmallParams P, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, CODE, MT>;
  using O = Order<D, CODE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const Paged& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 2, qj = lane & 3;  // fragment row and column group
  PlanSmem* psm = reinterpret_cast<PlanSmem*>(smem + C::OFF_PLAN);
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  float* join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
  auto bar_full = [&](uint32_t st) { return sbase + C::OFF_BAR + 8 * st; };
  auto bar_empty = [&](uint32_t st) { return sbase + C::OFF_BAR + 8 * (C::NS + st); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 2 * C::NS * 8);
  [[maybe_unused]] const uint32_t sq = sbase + C::OFF_Q;

  if (threadIdx.x == 0) {
    for (int st = 0; st < C::NS; ++st) {
      mbar_init(bar_full(st), kLoaders);
      mbar_init(bar_empty(st), kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  Cursor cur;
  long long left, run;
  plan_start<kThreads>(p, P.plan, psm, &cur, &left, &run);
  if (left == 0) return;
  const long long all_left = left;

  if (warp >= kWarps) {
    // ------------------------------------------------------------ loads
    // A copy for each page of a stage (128 keys at most), and each costs its warp some 80 clocks: K and
    // V, and the stage's halves, are different warps'.  Lane i has copy i of its warp; the page of a
    // copy is looked up a stage ahead.
    regs_dec<kLoadRegs>();
    const int box_log2 = min(p.page_log2, 7), box = 1 << box_log2;
    const int copies = kStageKeys >> box_log2, part = (copies + 1) >> 1;
    const bool is_v = (warp & 1) != 0;
    const int at = ((warp >> 1) & 1) * part + lane;  // this lane's copy
    const bool has_copy = lane < part && at < copies;
    uint32_t n = 0, st = 0, ph = 1;  // stages so far; next stage; parity that its release has
    bool good = true;
    while (left > 0) {
      const int keys = P.plan.keys(cur.span, cur.j), units = P.plan.units(cur.span, cur.j);
      const int kt1 = (int)min((long long)units, cur.kt + left);
      const int end = (int)min((long long)keys, (long long)kt1 << C::KT_LOG2);
      auto lookup = [&](int key) -> int {
        return has_copy && key < end ? __ldg(p.table + (size_t)cur.s * p.max_pages + (key >> p.page_log2)) : 0;
      };
      int key = (cur.kt << C::KT_LOG2) + (at << box_log2);
      int entry = lookup(key);
      for (int key0 = cur.kt << C::KT_LOG2; key0 < end && good; key0 += kStageKeys, key += kStageKeys) {
        const int next = lookup(key + kStageKeys);
        const bool mine = has_copy && key < end;
        const size_t row = (((size_t)(mine ? checked_page(p, entry) : 0) * p.Hkv + cur.g) << p.page_log2) + (key & ((1 << p.page_log2) - 1));
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
        if (n >= C::NS) good = __all_sync(0xffffffffu, mbar_wait(bar_empty(st), ph, P.wait_limit, abort_flag));
        if (!good) break;
        const uint32_t full = bar_full(st);
        if (lane == 0) mbar_arrive_expect_tx(full, boxes * box * (D * C::ESZ + (CODE == kPlain ? 0 : 4)));
        __syncwarp();
        if (mine) {
          const uint32_t dst = sbase + C::OFF_RING + st * C::STAGE + (is_v ? C::KV_BYTES : 0);
          if constexpr (CODE == kPlain) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_2d(dst + h * (kStageKeys * 128) + ((at << box_log2) * 128), is_v ? &vmap : &kmap, full, h * 64, (int)row);
          } else {  // rows of 128 bytes: one key (D = 128) or two (D = 64)
            tma_load_2d(dst + (at << box_log2) * D, is_v ? &vmap : &kmap, full, 0, (int)(D == 128 ? row : row >> 1));
            bulk_load(sbase + C::OFF_RING + st * C::STAGE + 2 * C::KV_BYTES + (is_v ? kStageKeys * 4 : 0) + (at << box_log2) * 4,
                      (is_v ? p.v_scales : p.k_scales) + row, box * 4, full);
          }
        }
        __syncwarp();
        ++n;
        if (++st == C::NS) {
          st = 0;
          ph ^= 1;
        }
        entry = next;
      }
      if (!good) break;
      left -= kt1 - cur.kt;
      if (left > 0) plan_next(p, P.plan, &cur);
    }
    if (!good) {
      record_status(p.status, TSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // The last copies must land before the CTA exits, and after an abort nobody else waits for them.
    for (uint32_t k = n > C::NS ? n - C::NS : 0; k < n; ++k) mbar_wait(bar_full(k % C::NS), (k / C::NS) & 1, kDrainPolls, nullptr);
    return;
  }
  regs_inc<kWorkRegs>();

  uint32_t stage = 0, phase = 0;
  bool ok = true;
  const int tt = 1 << P.plan.tt_log2;
  auto work_sync = [&]() { named_sync(1u, kWork); };

  while (left > 0) {
    // ------------------------------------------------ one tile of rows, or a part of it
    const int keys = P.plan.keys(cur.span, cur.j), units = P.plan.units(cur.span, cur.j);
    const int kt1 = (int)min((long long)units, cur.kt + left);
    const int first_tok = cur.j * tt;
    const int n_tok = min(tt, cur.span.n - first_tok);
    const int pos0 = cur.span.base + first_tok;  // position of the tile's first token
    const int n_rows = n_tok << p.g_log2;

    // Queries as A fragments: thread (rg, qj) holds rows rg, rg + 8 at the d of its k indices.
    auto q_row = [&](int r) {
      r = min(r, n_rows - 1);
      return static_cast<const __nv_bfloat16*>(P.q.data) + (int64_t)(cur.span.tok0 + first_tok + (r >> p.g_log2)) * P.q.ts +
             (int64_t)(cur.g * p.G + (r & (p.G - 1))) * P.q.hs;
    };
    auto q_frag = [&](int mt, int ks, uint32_t (&f)[4]) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const __nv_bfloat16* qr = q_row(mt * 16 + rg + 8 * hf);
        if constexpr (CODE == kPlain) {
          f[hf] = __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * qj));
          f[hf + 2] = __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * qj));
        } else {  // the four codes of a word: bytes 0, 2 are one pair of the contraction, bytes 1, 3 the other
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(qr + 64 * (ks >> 2) + 16 * qj + 4 * (ks & 3)));
          f[hf] = __byte_perm(v.x, v.y, 0x5410);
          f[hf + 2] = __byte_perm(v.x, v.y, 0x7632);
        }
      }
    };
    uint32_t qa[C::QSM ? 1 : MT][C::QSM ? 1 : C::NKS][4];
    if constexpr (C::QSM) {
#pragma unroll 1
      for (int i = warp; i < MT * C::NKS; i += kWarps) {
        uint32_t f[4];
        q_frag(i / C::NKS, i % C::NKS, f);
        st_shared_v4(sq + i * 512 + lane * 16, f[0], f[1], f[2], f[3]);
      }
      work_sync();  // the previous tile's readers have passed the barriers of its join
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ks = 0; ks < C::NKS; ++ks) q_frag(mt, ks, qa[mt][ks]);
    }
    auto frag = [&](int mt, int ks, uint32_t (&f)[4]) {
      if constexpr (C::QSM) {
        const uint4 x = lds128(sq + (mt * C::NKS + ks) * 512 + lane * 16);
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = qa[mt][ks][e];
      }
    };
    int rpos[MT][2];  // position of the thread's rows: they see keys up to it
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) rpos[mt][hf] = pos0 + min((mt * 16 + rg + 8 * hf) >> p.g_log2, n_tok - 1);

    float m[MT][2], l[MT][2], o[MT][C::NNT][4];
    [[maybe_unused]] float ro[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
      ro[mt][0] = ro[mt][1] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < C::NNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }

#pragma unroll 1
    for (int kt = cur.kt; kt < kt1; ++kt) {
      if (kt << C::KT_LOG2 >= keys) break;  // a tile that sees nothing
      const int key0 = (kt << C::KT_LOG2) + warp * kKeys;
      const bool two = C::NB == 2 && (kt << C::KT_LOG2) + kStageKeys < keys;  // a second stage (else its place holds any codes)
      const uint32_t stage1 = stage + 1 == C::NS ? 0 : stage + 1, phase1 = stage1 == 0 ? phase ^ 1 : phase;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, P.wait_limit, abort_flag));
      if (ok && two) ok = __all_sync(0xffffffffu, mbar_wait(bar_full(stage1), phase1, P.wait_limit, abort_flag));
      if (!ok) {
        *abort_flag = 1;
        break;
      }
      if (key0 < keys) {
        const uint32_t st0 = sbase + C::OFF_RING + stage * C::STAGE, st1 = sbase + C::OFF_RING + stage1 * C::STAGE;
        const uint32_t sk = st0 + warp * (C::KV_BYTES / (D * C::ESZ / 128 > 1 ? 2 : 1) / kWarps), sv = sk + C::KV_BYTES;
        [[maybe_unused]] const uint32_t kb[2] = {sk, st1 + (sk - st0)};
        [[maybe_unused]] const uint32_t sb[2] = {st0 + 2 * C::KV_BYTES + warp * kKeys * 4, st1 + 2 * C::KV_BYTES + warp * kKeys * 4};
        // Rows hide keys behind their own position; keys from `keys` on are not of this sequence.
        const bool border = key0 + (C::NB - 1) * kStageKeys + kKeys - 1 > pos0;

        if (CODE == kPlain && border) {
          // Values that some row must not see: clear what lies behind the tile's last key, and
          // take non-finite values out of the product (they reach the rows that see them here).
          bool odd = false;
#pragma unroll
          for (int i = 0; i < kKeys * D * 2 / 512; ++i) {
            const int at = i * 32 + lane;            // 16-byte piece: row, piece
            const int row = at / (D / 8), pc = at % (D / 8);
            const uint32_t addr = sv + (pc >> 3) * (kStageKeys * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4);
            if (key0 + row >= keys) {
              st_shared_v4(addr, 0u, 0u, 0u, 0u);
            } else if (key0 + row > pos0) {
              const uint4 x = lds128(addr);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) odd |= ((((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0);
            }
          }
          __syncwarp();
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int row = 0; row < kKeys; ++row) {
              if (key0 + row <= pos0 || key0 + row >= keys) continue;
#pragma unroll
              for (int nt = 0; nt < C::NNT; ++nt) {  // the two columns 8 nt + 2 qj of this thread's accumulators
                const uint32_t addr = sv + (nt >> 3) * (kStageKeys * 128) + row * 128 + (((nt & 7) ^ (row & 7)) << 4) + 4 * qj;
                const uint32_t w = __float_as_uint(lds32(addr));
                const float x0 = bf16_lo(w), x1 = bf16_hi(w);
                const bool b0 = !(fabsf(x0) < INFINITY), b1 = !(fabsf(x1) < INFINITY);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) {
                    if (b0 && key0 + row <= rpos[mt][hf]) o[mt][nt][2 * hf] += x0;
                    if (b1 && key0 + row <= rpos[mt][hf]) o[mt][nt][2 * hf + 1] += x1;
                  }
                __syncwarp();
                if (rg == 0 && (b0 || b1))
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"((b0 ? 0u : w & 0xffffu) | (b1 ? 0u : w & 0xffff0000u)) : "memory");
              }
            }
          }
          fence_proxy_async_smem();  // the ring's next TMA box overwrites these stores
          __syncwarp();
        }

        // ---- S = Q K^T: two column tiles of 8 keys in each block
        constexpr int NT = 2 * C::NB;
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.f;
        if constexpr (CODE == kPlain) {
          const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < C::NKS; ++ks) {
            const int pc = 2 * ks + half;
            uint32_t b[4];
            ldsm4(b, sk + (pc >> 3) * (kStageKeys * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a[4];
              frag(mt, ks, a);
              mma16816(s[mt][0], a, b[0], b[1]);
              mma16816(s[mt][1], a, b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            uint32_t w[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int key = 8 * (n & 1) + O::key(rg);
              uint32_t addr = kb[n >> 1];
              if (D == 128) addr += key * 128 + (((4 * h + qj) ^ (key & 7)) << 4);
              else addr += (key >> 1) * 128 + ((((key & 1) * 4 + qj) ^ ((key >> 1) & 7)) << 4);
              const uint4 v = lds128(addr);
              w[n][0] = v.x, w[n][1] = v.y, w[n][2] = v.z, w[n][3] = v.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t a[MT][4];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) frag(mt, 4 * h + x, a[mt]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint32_t b0 = codes_even<CODE>(w[n][x]), b1 = codes_odd<CODE>(w[n][x]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16816(s[mt][n], a[mt], b0, b1);
              }
            }
          }
        }

        // ---- softmax: columns 2 qj, 2 qj + 1 of each column tile
        [[maybe_unused]] float vs[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int in_block = 8 * (n & 1) + O::key(2 * qj + e), key = (n >> 1) * kStageKeys + in_block;
            float f = P.scale_log2;
            if constexpr (CODE != kPlain) {
              f *= lds32(sb[n >> 1] + 4 * in_block);
              vs[n][e] = lds32(sb[n >> 1] + kStageKeys * 4 + 4 * in_block);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              s[mt][n][e] *= f;
              s[mt][n][e + 2] *= f;
              if (border) {
                if (key0 + key > rpos[mt][0] || key0 + key >= keys) s[mt][n][e] = -INFINITY;
                if (key0 + key > rpos[mt][1] || key0 + key >= keys) s[mt][n][e + 2] = -INFINITY;
              }
            }
          }
        bool move = false;
        float mx[MT][2];
        [[maybe_unused]] float tx[MT][2];  // largest logit plus log2 of the value's scale; -inf or NaN where the key is not seen
        if constexpr (CODE != kPlain) {
          float lv[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) lv[n][e] = lg2_approx(fabsf(vs[n][e]));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              tx[mt][hf] = -INFINITY;
#pragma unroll
              for (int n = 0; n < NT; ++n) tx[mt][hf] = fmax3(tx[mt][hf], s[mt][n][2 * hf] + lv[n][0], s[mt][n][2 * hf + 1] + lv[n][1]);
              move |= tx[mt][hf] > ro[mt][hf] + kMoveReference;
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            mx[mt][hf] = fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]);
#pragma unroll
            for (int n = 1; n < NT; ++n) mx[mt][hf] = fmax3(mx[mt][hf], s[mt][n][2 * hf], s[mt][n][2 * hf + 1]);
            move |= mx[mt][hf] > m[mt][hf] + kMoveReference;
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              auto of_row = [](float x) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              };
              const float x = of_row(mx[mt][hf]);
              float alpha = 1.f;
              if (x > m[mt][hf] + kMoveReference) {
                // Before the first key o holds zeros, or infinities that the border's values have just added.
                alpha = m[mt][hf] == -INFINITY ? 1.f : ex2_approx(m[mt][hf] - x);
                m[mt][hf] = x;
                l[mt][hf] *= alpha;
              }
              if constexpr (CODE != kPlain) {
                const float y = of_row(tx[mt][hf]);
                float r = y > ro[mt][hf] + kMoveReference && y < INFINITY ? y : ro[mt][hf];
                r = fmaxf(r, m[mt][hf] - kMostAbove);
                alpha = r > ro[mt][hf] ? fmaxf(ex2_approx(ro[mt][hf] - r), kLeastFactor) : 1.f;
                ro[mt][hf] = r;
              }
#pragma unroll
              for (int nt = 0; nt < C::NNT; ++nt) {
                o[mt][nt][2 * hf] *= alpha;
                o[mt][nt][2 * hf + 1] *= alpha;
              }
            }
        }
        uint32_t pa[C::NB][MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float ref = m[mt][hf] == -INFINITY ? 0.f : m[mt][hf];  // no key seen yet: 2^-inf = 0
            [[maybe_unused]] float unit = 0.f;
            if constexpr (CODE != kPlain) unit = ex2_approx(fminf(ref - ro[mt][hf], kMostAbove) + kUnit);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float p0 = ex2_approx(s[mt][n][2 * hf] - ref), p1 = ex2_approx(s[mt][n][2 * hf + 1] - ref);
              l[mt][hf] += p0 + p1;
              if constexpr (CODE != kPlain) {
                p0 = p0 * vs[n][0] * unit;
                p1 = p1 * vs[n][1] * unit;
                if (border) {  // the scale of a key that is not seen may be anything
                  if (s[mt][n][2 * hf] == -INFINITY) p0 = 0.f;
                  if (s[mt][n][2 * hf + 1] == -INFINITY) p1 = 0.f;
                }
              }
              pa[n >> 1][mt][2 * (n & 1) + hf] = CODE == kPlain ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
            }
          }

        // ---- O += P V
        if constexpr (CODE == kPlain) {
          const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int pc = 2 * i + (lane >> 4);
            uint32_t b[4];
            ldsm4_t(b, sv + (pc >> 3) * (kStageKeys * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816(o[mt][2 * i], pa[0][mt], b[0], b[1]);
              mma16816(o[mt][2 * i + 1], pa[0][mt], b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < C::NB; ++k) {
            const uint32_t svk = kb[k] + C::KV_BYTES;
            uint32_t w[4][D / 32];  // the thread's four keys, D / 8 columns each
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = 8 * (x >> 1) + O::key(2 * qj + (x & 1));
              if constexpr (D == 128) {
                const uint4 v = lds128(svk + key * 128 + ((O::piece(rg) ^ (key & 7)) << 4));
                w[x][0] = v.x, w[x][1] = v.y, w[x][2] = v.z, w[x][3] = v.w;
              } else {
                const uint2 v = lds64(svk + (key >> 1) * 128 + ((((key & 1) * 4 + (rg >> 1)) ^ ((key >> 1) & 7)) << 4) + (rg & 1) * 8);
                w[x][0] = v.x, w[x][1] = v.y;
              }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
#pragma unroll
              for (int x = 0; x < 4; ++x) w[x][i] = codes_unsigned<CODE>(w[x][i]);
              const uint32_t b[4][2] = {
                  {codes_across_f16<CODE, 0>(w[0][i], w[1][i]), codes_across_f16<CODE, 0>(w[2][i], w[3][i])},
                  {codes_across_f16<CODE, 1>(w[0][i], w[1][i]), codes_across_f16<CODE, 1>(w[2][i], w[3][i])},
                  {codes_across_f16<CODE, 2>(w[0][i], w[1][i]), codes_across_f16<CODE, 2>(w[2][i], w[3][i])},
                  {codes_across_f16<CODE, 3>(w[0][i], w[1][i]), codes_across_f16<CODE, 3>(w[2][i], w[3][i])}};
#pragma unroll
              for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16816_f16(o[mt][4 * i + x], pa[k][mt], b[x][0], b[x][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stages before they are filled again
#pragma unroll
      for (int k = 0; k < C::NB; ++k) {
        if (k == 1 && !two) break;
        if (lane == 0) mbar_arrive(bar_empty(stage));
        if (++stage == C::NS) {
          stage = 0;
          phase ^= 1;
        }
      }
    }

    // ------------------------------------------------ join the warps' parts
    const int did = kt1 - cur.kt;
    const bool whole = cur.kt == 0 && kt1 == units;
    const int slot = cur.kt == 0 ? 1 : 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 1);
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 2);
        if (qj == 0) ml[warp * C::ROWS + mt * 16 + rg + 8 * hf] = make_float2(m[mt][hf], l[mt][hf]);
      }
    work_sync();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float f[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::ROWS + mt * 16 + rg + 8 * hf].x);
        f[hf] = m[mt][hf] == top ? 1.f : ex2_approx(m[mt][hf] - top);
        // 8 bits: o's unit against the rows' top, as its square root: the factor itself may pass fp32's range where the product does not.
        if (CODE != kPlain) f[hf] = ro[mt][hf] == -INFINITY ? 0.f : ex2_approx(0.5f * (ro[mt][hf] - kUnit + code_f16_unit<CODE>() - top));
      }
      auto scaled = [&](int nt, int e) { return CODE == kPlain ? o[mt][nt][e] * f[e >> 1] : o[mt][nt][e] * f[e >> 1] * f[e >> 1]; };
      float* mine = join + (warp & 3) * 16 * D;
      auto at = [&](int hf, int nt, int e) -> float& {  // column groups of 8 swapped by row against bank conflicts
        const int r = rg + 8 * hf, d = O::col(2 * qj + e, nt);
        return mine[r * D + (d ^ ((r & 3) << 3))];
      };
      if (warp >= 4) {
#pragma unroll
        for (int nt = 0; nt < C::NNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) at(e >> 1, nt, e & 1) = scaled(nt, e);
      }
      work_sync();
      if (warp < 4) {
#pragma unroll
        for (int nt = 0; nt < C::NNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) at(e >> 1, nt, e & 1) += scaled(nt, e);
      }
      work_sync();
      for (int i = threadIdx.x; i < 16 * D / 4; i += kWork) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const int row = mt * 16 + r;
        if (row >= n_rows) continue;
        const int dd = d ^ ((r & 3) << 3);
        float4 a = *reinterpret_cast<const float4*>(join + r * D + dd);
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          const float4 b = *reinterpret_cast<const float4*>(join + w * 16 * D + r * D + dd);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::ROWS + row].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 x = ml[w * C::ROWS + row];
          sum += (x.x == top ? 1.f : ex2_approx(x.x - top)) * x.y;
        }
        if (whole) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no key: zeros
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(P.out.data) +
                               (int64_t)(cur.span.tok0 + first_tok + (row >> p.g_log2)) * P.out.ts +
                               (int64_t)(cur.g * p.G + (row & (p.G - 1))) * P.out.hs + d;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        } else {
          const size_t part = (size_t)blockIdx.x * 2 + slot;
          *reinterpret_cast<float4*>(P.parts.o + (part * C::ROWS + row) * D + d) = a;
          if (d == 0) {
            P.parts.ml[(part * 2) * C::ROWS + row] = top;
            P.parts.ml[(part * 2 + 1) * C::ROWS + row] = sum;
          }
        }
      }
      work_sync();
    }
    if (!whole)
      join_parts<__nv_bfloat16, D, C::ROWS, kWork>(p, P.out, P.parts, reinterpret_cast<JoinSmem<C::ROWS>*>(smem + C::OFF_LAST),
                                                   tile_owners(run * blockIdx.x + (all_left - left), cur.kt, units, run), cur.g,
                                                   cur.span.tok0 + first_tok, n_rows, (int)threadIdx.x, work_sync);
    left -= did;
    if (left > 0) plan_next(p, P.plan, &cur);
  }

  if (!ok && lane == 0) record_status(p.status, TSA_ERR_TIMEOUT);
}

template <int D, int CODE, int MT>
cudaError_t launch(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, int which, cudaStream_t st) {
  using C = Cfg<D, CODE, MT>;
  SmallParams P;
  P.p = p;
  P.q = q;
  P.out = out;
  P.parts = make_parts(base, C::ROWS, kPagedCtas, D);
  P.parts.header = header;
  P.plan.which = which;
  P.plan.kt_log2 = C::KT_LOG2;
  P.plan.tt_log2 = (MT == 2 ? 5 : 4) - p.g_log2;
  P.scale_log2 = p.scale * 1.4426950408889634f;
  P.wait_limit = wait_limit();
  const uint64_t rows = ((uint64_t)p.n_pages * p.Hkv) << p.page_log2;
  CUtensorMap km, vm;
  const int box = 1 << (p.page_log2 < 7 ? p.page_log2 : 7);
  const bool made = CODE == kPlain ? make_tile_map(&km, p.k_pages, rows, D, box) && make_tile_map(&vm, p.v_pages, rows, D, box)
                                   : make_code_map(&km, p.k_pages, rows * D / 128, box * D / 128) &&
                                         make_code_map(&vm, p.v_pages, rows * D / 128, box * D / 128);
  if (!made) return cudaErrorInvalidValue;
  // The register split counts on 168 registers a thread at launch: with fewer it would wait for ever.
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, paged_small<D, CODE, MT>);
  if (e != cudaSuccess) return e;
  if (at.numRegs <= 160) return cudaErrorInvalidKernelImage;
  e = cudaFuncSetAttribute(paged_small<D, CODE, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  paged_small<D, CODE, MT><<<kPagedCtas, kThreads, C::SMEM, st>>>(P, km, vm);
  count_launches(1);
  return cudaGetLastError();
}

// Up to 16 rows (a row tile of one mma) the second row tile would be empty.
bool one_tile(const Paged& p) { return (long long)p.max_new * p.G <= 16; }

template <int D, int CODE>
cudaError_t by_rows(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, int which, cudaStream_t st) {
  return one_tile(p) ? launch<D, CODE, 1>(p, q, out, base, header, which, st) : launch<D, CODE, 2>(p, q, out, base, header, which, st);
}

template <int D>
cudaError_t by_code(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, int which, cudaStream_t st) {
  if (p.cache_dtype == TSA_I8) return by_rows<D, kI8>(p, q, out, base, header, which, st);
  if (p.cache_dtype == TSA_E4M3) return by_rows<D, kE4M3>(p, q, out, base, header, which, st);
  return by_rows<D, kPlain>(p, q, out, base, header, which, st);
}

}  // namespace

size_t paged_small_bytes(const Paged& p) { return parts_bytes(one_tile(p) ? 16 : 32, kPagedCtas, p.D); }

cudaError_t launch_paged_small(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, int which, cudaStream_t st) {
  return p.D == 64 ? by_code<64>(p, q, out, base, header, which, st) : by_code<128>(p, q, out, base, header, which, st);
}

}  // namespace tsa
