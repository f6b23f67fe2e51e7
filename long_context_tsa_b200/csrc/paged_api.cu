// C entry points of the paged cache declared in include/tsa.h: argument checks,
// workspace layout and the choice of kernels.
#include <math.h>

#include "internal.h"
#include "paged.h"

namespace tsa {
namespace {

constexpr size_t kHeaderBytes = kHeaderWords * sizeof(uint32_t);  // tsa_workspace_init zeroes it

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

tsa_status check_paged_desc(const tsa_paged_desc* desc, Paged* p) {
  if (desc == nullptr) return TSA_ERR_INVALID_ARG;
  if (desc->n_tokens < 1 || desc->n_seqs < 1 || desc->Hq < 1 || desc->Hkv < 1 || desc->D < 1 || desc->page_size < 1 ||
      desc->n_pages < 1 || desc->max_pages < 1 || desc->max_new < 1)
    return TSA_ERR_INVALID_ARG;
  if (desc->dtype != TSA_F32 && desc->dtype != TSA_BF16) return TSA_ERR_INVALID_ARG;
  if (desc->cache_dtype != desc->dtype && desc->cache_dtype != TSA_I8 && desc->cache_dtype != TSA_E4M3)
    return TSA_ERR_INVALID_ARG;
  if (desc->Hq % desc->Hkv != 0) return TSA_ERR_INVALID_ARG;
  if (!(desc->scale >= 0.f) && !(desc->scale < 0.f)) return TSA_ERR_INVALID_ARG;  // NaN
  if (desc->D != 64 && desc->D != 128) return TSA_ERR_UNSUPPORTED;
  const int G = desc->Hq / desc->Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16) return TSA_ERR_UNSUPPORTED;
  if (desc->page_size < 16 || desc->page_size > 1024 || (desc->page_size & (desc->page_size - 1)) != 0)
    return TSA_ERR_UNSUPPORTED;
  if (desc->n_seqs > kPagedMaxSeqs || desc->Hkv > kMaxGroups) return TSA_ERR_UNSUPPORTED;
  constexpr long long lim = 1LL << 31;
  if ((long long)desc->n_tokens * desc->Hq >= lim || (long long)desc->max_pages * desc->page_size >= lim / 2)
    return TSA_ERR_UNSUPPORTED;  // positions of a whole tile behind the last one still fit 31 bits
  if ((long long)desc->n_pages * desc->Hkv >= lim || (long long)desc->n_pages * desc->Hkv * desc->page_size >= lim)
    return TSA_ERR_UNSUPPORTED;
  p->T = desc->n_tokens;
  p->S = desc->n_seqs;
  p->Hq = desc->Hq;
  p->Hkv = desc->Hkv;
  p->G = G;
  p->g_log2 = log2_exact(G);
  p->D = desc->D;
  p->dtype = desc->dtype;
  p->cache_dtype = desc->cache_dtype;
  p->page_log2 = log2_exact(desc->page_size);
  p->n_pages = desc->n_pages;
  p->max_pages = desc->max_pages;
  p->max_new = desc->max_new;
  p->scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)desc->D);
  return TSA_OK;
}

tsa_status check_cache(const tsa_paged_cache* c, Paged* p) {
  if (c == nullptr || !aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return TSA_ERR_INVALID_ARG;
  if (!aligned(c->page_table, 4) || !aligned(c->seq_len, 4) || !aligned(c->token_start, 4)) return TSA_ERR_INVALID_ARG;
  if (p->cache_dtype != p->dtype) {
    if (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16)) return TSA_ERR_INVALID_ARG;
  } else if (c->k_scales != nullptr || c->v_scales != nullptr) {
    return TSA_ERR_INVALID_ARG;
  }
  p->k_pages = c->k_pages;
  p->v_pages = c->v_pages;
  p->k_scales = c->k_scales;
  p->v_scales = c->v_scales;
  p->table = c->page_table;
  p->seq_len = c->seq_len;
  p->token_start = c->token_start;
  return TSA_OK;
}

// Strides of a dimension of one element do not matter.
tsa_status check_rows(const tsa_rows* r, const Paged& p, int heads, bool written, Rows* out) {
  if (r == nullptr || !aligned(r->data, 16)) return TSA_ERR_INVALID_ARG;
  const int64_t unit = p.dtype == TSA_BF16 ? 8 : 4;
  const int64_t ts = p.T == 1 ? 0 : r->token_stride, hs = heads == 1 ? 0 : r->head_stride;
  if (ts < 0 || hs < 0 || ts % unit != 0 || hs % unit != 0) return TSA_ERR_INVALID_ARG;
  constexpr int64_t lim = int64_t(1) << 40;  // bounds the offsets
  if (ts > lim / p.T || hs > lim / heads) return TSA_ERR_INVALID_ARG;
  if (written) {
    if ((p.T > 1 && ts < p.D) || (heads > 1 && hs < p.D)) return TSA_ERR_INVALID_ARG;
    if (p.T > 1 && heads > 1 && (ts < hs ? hs < (p.T - 1) * ts + p.D : ts < (heads - 1) * hs + p.D))
      return TSA_ERR_INVALID_ARG;
  }
  out->data = r->data;
  out->ts = ts;
  out->hs = hs;
  return TSA_OK;
}

tsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TSA_OK : TSA_ERR_CUDA; }

// f32 runs on CUDA cores.  bf16: short sequences go to the kernel for few rows,
// longer ones to the kernel for chunks; a batch that may hold both kinds takes
// both, each doing its own (a token over a long cache takes the chunk kernel
// nearly twice as long).
bool all_short(const Paged& p) { return (long long)p.max_new * p.G <= kSplitRows; }

size_t workspace_bytes(const Paged& p) {
  if (p.dtype != TSA_BF16) return kHeaderBytes + paged_simt_bytes(p);
  if (all_short(p)) return kHeaderBytes + paged_small_bytes(p);
  return kHeaderBytes + paged_chunk_bytes(p);  // larger than paged_small's
}

cudaError_t launch_attend(const Paged& p, const Rows& q, const Rows& out, char* ws, cudaStream_t st) {
  uint32_t* header = reinterpret_cast<uint32_t*>(ws);
  char* base = ws + kHeaderBytes;
  if (p.dtype != TSA_BF16) return launch_paged_simt(p, q, out, base, header, st);
  if (all_short(p)) return launch_paged_small(p, q, out, base, header, 0, st);
  if (p.S == 1) return launch_paged_chunk(p, q, out, base, 0, st);
  const cudaError_t e = launch_paged_small(p, q, out, base, header, 1, st);  // one after the other: the parts share a place
  return e != cudaSuccess ? e : launch_paged_chunk(p, q, out, base, 2, st);
}

// The checks that the three calls share; a and b: the packed tensors.
tsa_status check_call(const tsa_paged_desc* desc, const tsa_paged_cache* cache, const tsa_rows* a, const tsa_rows* b,
                      bool attend, bool write_a, bool write_b, void* ws, size_t ws_bytes, Paged* p, Rows* ra, Rows* rb) {
  tsa_status s = check_paged_desc(desc, p);
  if (s != TSA_OK) return s;
  if ((s = check_cache(cache, p)) != TSA_OK) return s;
  const int heads = attend ? p->Hq : p->Hkv;
  if ((s = check_rows(a, *p, heads, write_a, ra)) != TSA_OK) return s;
  if ((s = check_rows(b, *p, heads, write_b, rb)) != TSA_OK) return s;
  if (!aligned(ws, 16)) return TSA_ERR_INVALID_ARG;
  if (ws_bytes < workspace_bytes(*p)) return TSA_ERR_WORKSPACE;
  p->status = static_cast<uint32_t*>(ws);
  return TSA_OK;
}

}  // namespace
}  // namespace tsa

using namespace tsa;

extern "C" {

size_t tsa_paged_workspace_size(const tsa_paged_desc* desc) {
  Paged p;
  return check_paged_desc(desc, &p) == TSA_OK ? workspace_bytes(p) : 0;
}

tsa_status tsa_cache_write(const tsa_paged_desc* desc, const tsa_paged_cache* cache, const tsa_rows* k,
                           const tsa_rows* v, void* ws, size_t ws_bytes, void* stream) {
  Paged p;
  Rows rk, rv;
  const tsa_status s = check_call(desc, cache, k, v, false, false, false, ws, ws_bytes, &p, &rk, &rv);
  if (s != TSA_OK) return s;
  return cuda_status(launch_cache_write(p, rk, rv, static_cast<cudaStream_t>(stream)));
}

tsa_status tsa_cache_read(const tsa_paged_desc* desc, const tsa_paged_cache* cache, const tsa_rows* k,
                          const tsa_rows* v, void* ws, size_t ws_bytes, void* stream) {
  Paged p;
  Rows rk, rv;
  const tsa_status s = check_call(desc, cache, k, v, false, true, true, ws, ws_bytes, &p, &rk, &rv);
  if (s != TSA_OK) return s;
  return cuda_status(launch_cache_read(p, rk, rv, static_cast<cudaStream_t>(stream)));
}

tsa_status tsa_attend_paged(const tsa_paged_desc* desc, const tsa_paged_cache* cache, const tsa_rows* q,
                            const tsa_rows* out, void* ws, size_t ws_bytes, void* stream) {
  Paged p;
  Rows rq, ro;
  const tsa_status s = check_call(desc, cache, q, out, true, false, true, ws, ws_bytes, &p, &rq, &ro);
  if (s != TSA_OK) return s;
  return cuda_status(launch_attend(p, rq, ro, static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
