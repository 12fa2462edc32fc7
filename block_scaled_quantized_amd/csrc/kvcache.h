// kvcache.h -- what the rotary, cache and attention sources share: 16-byte vectors, the argument
// checks of the cache descriptors, and exact division by a launch constant.
#pragma once
#include "codec_math.h"

namespace mx {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxHeadDim = 256, kMaxHeads = 65536;

// n / d for 0 <= n < 2^31 and a fixed 1 <= d < 2^31, as (n * m) >> s: with s = 31 + ceil(log2 d) and
// m = floor(2^s / d) + 1 < 2^32, m d exceeds 2^s by at most d <= 2^(s-31), so the error term
// n (m d - 2^s) / (d 2^s) stays below 1/d and the floor is exact.
struct FastDiv {
  uint32_t m, d;
  int s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    int log = 0;
    while (((uint64_t)1 << log) < div) log++;
    s = 31 + log;
    m = (uint32_t)((((uint64_t)1 << s) / div) + 1);
  }
  MX_DEV uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> s); }
};

// Status of a [tokens][heads][dim] tensor: rows 16-byte aligned.
inline int check_heads(const mx_heads* t, int elem_bytes) {
  if (!t || !t->data) return MX_ERR_NULL;
  const int64_t unit = 16 / elem_bytes;
  if (t->heads < 1 || t->heads > kMaxHeads || t->token_stride % unit || t->head_stride % unit) return MX_ERR_SHAPE;
  return aligned16(t->data) ? MX_OK : MX_ERR_ALIGN;
}

inline bool dim_ok(int dim) { return dim >= 8 && dim <= kMaxHeadDim && dim % 8 == 0; }

// Status of a cache's format and geometry (its pointers apart).
inline int check_geometry(const mxkv_cache* c) {
  if (c->fmt != MX_F16 && c->fmt != MX_BF16 && c->fmt != MX_E4M3) return MX_ERR_FORMAT;
  if (c->order != MXKV_HEADS_FIRST && c->order != MXKV_SLOTS_FIRST) return MX_ERR_FORMAT;
  const int unit = c->fmt == MX_E4M3 ? 32 : 8;
  if (!dim_ok(c->dim) || c->dim % unit || c->heads < 1 || c->heads > 1024 || c->pages < 1 || c->page_size < 1 ||
      c->page_size > MX_MAX_DIM || (int64_t)c->pages * c->page_size >= (int64_t)1 << 31)
    return MX_ERR_SHAPE;
  if (c->page_stride % unit || c->page_stride < (int64_t)c->heads * c->page_size * c->dim) return MX_ERR_SHAPE;
  return MX_OK;
}

inline int check_cache(const mxkv_cache* c) {
  if (!c) return MX_ERR_NULL;
  if (int s = check_geometry(c)) return s;
  const bool mx8 = c->fmt == MX_E4M3;
  if (!c->k || !c->v || (mx8 && (!c->ks || !c->vs))) return MX_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || (mx8 && (!aligned16(c->ks) || !aligned16(c->vs)))) return MX_ERR_ALIGN;
  return MX_OK;
}

inline int check_table(const mxkv_table* t) {
  if (!t) return MX_ERR_NULL;
  if (t->seqs < 0 || t->seqs > MX_MAX_DIM || t->cols < 1 || t->cols > (1 << 30)) return MX_ERR_SHAPE;
  return t->pages || t->seqs == 0 ? MX_OK : MX_ERR_NULL;
}

inline int64_t slot_stride(const mxkv_cache* c) {
  return c->order == MXKV_HEADS_FIRST ? c->dim : (int64_t)c->heads * c->dim;
}
inline int64_t kv_head_stride(const mxkv_cache* c) {
  return c->order == MXKV_HEADS_FIRST ? (int64_t)c->page_size * c->dim : c->dim;
}

}  // namespace mx
