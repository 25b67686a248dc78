// The KV cache that grows token by token (declarations shared by the C ABI,
// kv_append.cu, cache_attn.cu and decode.cu).
#pragma once

#include <stdint.h>

#include "hope.cuh"
#include "kernels.h"

namespace hils {

// Mirror of hils_kv_cache with the element type resolved.  Pages hold one
// chunk of kC tokens of every KV head.  q8 = false: pages of the parameter
// dtype [num_pages][Hkv][C][d].  q8 = true: e4m3 codes in pages of the same
// shape, one power-of-two scale per (page, KV head), and full-precision tails
// [B][2][Hkv][C][d] of each sequence's last two chunks (chunk c in half c & 1).
struct CacheKV {
  bool q8;
  int max_pages;  // page-table columns
  int lmk_rows;   // landmark rows per (sequence, KV head)
  long long num_pages;
  void *k_pages, *v_pages;
  const int32_t *table;
  void *lmk;
  float *k_scale, *v_scale;
  void *k_tail, *v_tail;
};

// Rows [B][H][T][d] with strides in elements, d contiguous.
struct RowsIn {
  const void *p;
  long long sb, sh, st;
};

struct AppendSpec {
  int B, Hq, Hkv, L, d, T;
  const int32_t *pos, *n_new;  // n_new == nullptr: T tokens of every sequence
  int32_t *seq_lens;           // may be nullptr
};

// New keys and values into the cache (kv_append.cu).
cudaError_t kv_append(const AppendSpec &as, bool bf16, const CacheKV &c, const RowsIn &k,
                      const RowsIn &v, const RowsIn &q, void *q_out, const HopeParams &hp,
                      uint32_t *err, cudaStream_t st, int *launches);

// A union entry of a completed chunk resolved (cache_select or decode_union
// writes it), two uint4: the block of the chunk, or kEntNoPage; the mask of the
// heads that attend it; the two scales (fp32 bits); and, a byte per head, the
// place of the chunk in the head's selection.  The own chunk, the union's last, has
// none: its attention needs no selection (u_count counts it all the same).
constexpr int kEntNoPage = -1;  // the page lies outside the pool

constexpr int kCacheWarps = 4;       // warps of a tensor-core attention CTA
constexpr int kCacheMaxPer = 128;    // most union entries per warp, where parts are fixed
constexpr int kCacheMaxEntries = 16; // most union entries per fp32 attention CTA

// Landmark scores of every completed chunk, bf16 (cache_select.cu): scores
// [B*Hq][ds.n_c], row h's first (len-1)/C entries written.
cudaError_t cache_scores(const DecodeSpec &ds, const void *q, const void *lmk, float *scores,
                         uint32_t *err, cudaStream_t st);
// Top-k, log-sum-exp and the union of every KV head in one launch, for
// ds.n_c <= kSelectMax.  Where cache_select_scores() holds the launch computes
// the scores too; otherwise they are there already (written by the launch
// before this one when ds.n_c > 0).  With ent (bf16) the union is written as
// resolved entries and next is set to 0, otherwise (fp32) as u_c, u_mask, u_logit.
constexpr int kSelectMax = 8192;
constexpr int kSelectMaxG = 8;
bool cache_select_scores(const DecodeSpec &ds, bool bf16);
cudaError_t cache_select(const DecodeSpec &ds, const CacheKV &cache, bool bf16, const void *q,
                         float *scores, int32_t *sel, float *w, float *lse_lmk, int32_t *u_c,
                         uint32_t *u_mask, float *u_logit, int32_t *u_count, uint4 *ent,
                         int *next, uint32_t *err, cudaStream_t st);

// Chunk attention and combine of the decode step (cache_attn.cu), bf16: the
// list of all union entries -> out, lse.  next: a counter that the selection
// has set to 0; part: [B*Hq][topk][d] floats, one record per selected chunk of a
// head; own_part: [B*Hq][2 + d], written before the step's other kernels are
// done.
cudaError_t cache_attn(const DecodeSpec &ds, const CacheKV &c, const void *q, const uint4 *ent,
                       const int32_t *u_count, int *next, const float *chunk_w, float *part,
                       float *own_part, void *out, float *lse, uint32_t *err, cudaStream_t st);
// fp32, 8-bit cache: the union entries of every (b, kv-head) -> partial records as
// decode.cu's own chunk attention writes them.
cudaError_t cache_attn_f32(const DecodeSpec &ds, const CacheKV &c, const void *q,
                           const int32_t *u_c, const uint32_t *u_mask, const float *u_logit,
                           const int32_t *u_count, float *part, uint32_t *err, cudaStream_t st);

// The decode step over the cache, with a length per sequence (decode.cu).
DecodeSpec cache_decode_spec(int B, int Hq, int Hkv, int N, int d, int topk, float scale, bool q8,
                             bool bf16);
cudaError_t decode_fwd_cache(const DecodeSpec &ds, bool bf16, const void *q, const CacheKV &c,
                             int32_t *sel, float *w, float *lse_lmk, void *out, float *lse,
                             void *ws, uint32_t *err, cudaStream_t st, int *launches);

}  // namespace hils
