// Declarations of the paged-cache operators shared by their translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tsa.h"

namespace tsa {

constexpr int kPagedMaxSeqs = 1024;  // the work split scans the sequences in one block
constexpr int kPagedCtas = 148;      // SMs: the attention kernels run one or two CTAs on each
constexpr int kSplitRows = 32;       // rows (new tokens x query heads of a group) up to which a sequence counts as short

// Checked arguments of a paged call, in device terms.  Offsets into the pools
// and the packed tensors are 64-bit: a pool of one layer passes 2^32 bytes.
struct Paged {
  int T, S, Hq, Hkv, G, g_log2, D, dtype, cache_dtype;
  int page_log2, n_pages, max_pages, max_new;
  float scale;  // resolved (> 0)
  void *k_pages, *v_pages;
  float *k_scales, *v_scales;
  const int32_t *table, *seq_len, *token_start;
  uint32_t* status;
};

// Packed rows [token][head][D]: element offset token * ts + head * hs.
struct Rows {
  void* data;
  int64_t ts, hs;
};

// Where a CTA leaves a tile that another CTA continues.  Slot 0 of a CTA holds
// a tile that an earlier CTA began, slot 1 one that it began itself.
struct PartMeta {
  int32_t c_end;  // last CTA with a part of the tile begun by this CTA, or -1
  int32_t g;      // KV head
  int32_t tok0;   // packed row of the tile's first token
  int32_t n_tok;  // tokens of the tile
};
struct Parts {
  float* o;          // [ctas][2][rows][D], unnormalised
  float* ml;         // [ctas][2][2][rows]: reference (log2 units), sum
  PartMeta* meta;    // [ctas], for paged_combine
  uint32_t* header;  // the workspace's first kHeaderWords words: join_parts counts there
  int rows;          // rows of a tile
  int ctas;
};

// The header that every workspace of the library begins with: no call keeps scratch there, and it is zero
// between calls but for the status.  Word 0: status.  Word 1: never set (tsa_debug_wait_never_set).
constexpr int kHeaderWords = 64;

inline size_t parts_bytes(int rows, int ctas, int D) {
  return (size_t)ctas * 2 * rows * (D + 2) * sizeof(float) + (size_t)ctas * sizeof(PartMeta);
}
// Parts at `base` (16-byte aligned).
inline Parts make_parts(void* base, int rows, int ctas, int D) {
  Parts p;
  p.o = static_cast<float*>(base);
  p.ml = p.o + (size_t)ctas * 2 * rows * D;
  p.meta = reinterpret_cast<PartMeta*>(p.ml + (size_t)ctas * 4 * rows);
  p.rows = rows;
  p.ctas = ctas;
  p.header = nullptr;
  return p;
}

cudaError_t launch_cache_write(const Paged& p, const Rows& k, const Rows& v, cudaStream_t st);
cudaError_t launch_cache_read(const Paged& p, const Rows& k, const Rows& v, cudaStream_t st);
// Attention: each launcher takes `base` of at least paged_*_bytes() (16-byte aligned) for its
// partial tiles.  paged_simt and paged_small join them themselves (header: the workspace's, where they
// count the parts); paged_chunk leaves them to paged_combine, in an order of its own: row =
// M tile * 128 + query head * (128 / G) + token, columns in groups of four [D / 4][rows][4].
// which: 0 every sequence, 1 those with at most kSplitRows rows, 2 the others.
size_t paged_simt_bytes(const Paged& p);
cudaError_t launch_paged_simt(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, cudaStream_t st);
size_t paged_small_bytes(const Paged& p);
cudaError_t launch_paged_small(const Paged& p, const Rows& q, const Rows& out, void* base, uint32_t* header, int which, cudaStream_t st);
size_t paged_chunk_bytes(const Paged& p);
cudaError_t launch_paged_chunk(const Paged& p, const Rows& q, const Rows& out, void* base, int which, cudaStream_t st);
cudaError_t launch_paged_combine(const Paged& p, const Rows& out, const Parts& parts, cudaStream_t st);

}  // namespace tsa
