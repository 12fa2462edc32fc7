// page_pool.cpp -- host bookkeeping of a paged key-value cache: page tables, shared pages and the
// page moves that the device has to make. No GPU work.
#include <algorithm>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "common.h"

struct mxkv_pool_state {
  int pages, page_size, seqs, cols;
  int used = 0;
  std::vector<int32_t> table, lengths, holders;  // holders: sequences that hold a page
  // Free pages, the lowest first. Every free page is in it once: a page enters when its last holder
  // lets go of it and leaves when it is taken.
  std::priority_queue<int32_t, std::vector<int32_t>, std::greater<int32_t>> free;

  int32_t* row(int s) { return table.data() + (size_t)s * cols; }
  int pages_of(int tokens) const { return (int)(((int64_t)tokens + page_size - 1) / page_size); }  // the sum can pass 2^31
  int held(int s) const { return pages_of(lengths[s]); }
  int32_t take() {
    const int32_t p = free.top();
    free.pop();
    holders[p] = 1;
    used++;
    return p;
  }
  void drop(int32_t p) {
    if (--holders[p]) return;
    free.push(p);
    used--;
  }
};

namespace {

// Runs f and turns what it throws into a status: no exception leaves a C entry point.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return MX_ERR_NOMEM;
  } catch (...) {
    return MX_ERR_NOMEM;
  }
}

bool has(const mxkv_pool_state* p, int seq) { return seq >= 0 && seq < p->seqs; }

}  // namespace

extern "C" {

int mxkv_pool_create(mxkv_pool* out, int pages, int page_size, int seqs, int cols) {
  if (!out) return MX_ERR_NULL;
  *out = nullptr;
  for (int v : {pages, page_size, seqs, cols})
    if (v < 1 || v > MX_MAX_DIM) return MX_ERR_SHAPE;
  const int64_t most = (int64_t)1 << 31;
  if ((int64_t)seqs * cols >= most || (int64_t)pages * page_size >= most || (int64_t)cols * page_size >= most) return MX_ERR_SHAPE;
  return guarded([&] {
    mxkv_pool_state* p = new mxkv_pool_state;
    try {
      p->pages = pages, p->page_size = page_size, p->seqs = seqs, p->cols = cols;
      p->table.assign((size_t)seqs * cols, -1);
      p->lengths.assign(seqs, 0);
      p->holders.assign(pages, 0);
      std::vector<int32_t> all;
      all.reserve(pages);  // and so never grows again: drop() cannot throw
      for (int i = 0; i < pages; i++) all.push_back(i);
      p->free = decltype(p->free)(std::greater<int32_t>(), std::move(all));
    } catch (...) {
      delete p;
      throw;
    }
    *out = p;
    return (int)MX_OK;
  });
}

int mxkv_pool_destroy(mxkv_pool p) {
  delete p;
  return MX_OK;
}

int mxkv_pool_resize(mxkv_pool p, int seq, int tokens, int32_t pair[2], int* n_pairs) {
  if (!p || !pair || !n_pairs) return MX_ERR_NULL;
  if (!has(p, seq) || tokens < 0 || tokens > (int64_t)p->cols * p->page_size) return MX_ERR_SHAPE;
  const int had = p->held(seq), need = p->pages_of(tokens);
  int32_t* row = p->row(seq);
  const bool grows = tokens > p->lengths[seq];
  const bool own = grows && p->lengths[seq] % p->page_size != 0 && p->holders[row[had - 1]] > 1;
  const int more = (need > had ? need - had : 0) + (own ? 1 : 0);
  if (more > p->pages - p->used) return MX_ERR_NOMEM;
  *n_pairs = 0;
  if (own) {
    const int32_t to = p->take();
    pair[0] = row[had - 1], pair[1] = to;
    *n_pairs = 1;
    p->drop(row[had - 1]);
    row[had - 1] = to;
  }
  for (int c = had; c < need; c++) row[c] = p->take();
  for (int c = need; c < had; c++) {
    p->drop(row[c]);
    row[c] = -1;
  }
  p->lengths[seq] = tokens;
  return MX_OK;
}

int mxkv_pool_fork(mxkv_pool p, int src, int dst) {
  if (!p) return MX_ERR_NULL;
  if (!has(p, src) || !has(p, dst) || src == dst || p->lengths[dst]) return MX_ERR_SHAPE;
  const int n = p->held(src);
  std::copy(p->row(src), p->row(src) + n, p->row(dst));
  for (int c = 0; c < n; c++) p->holders[p->row(dst)[c]]++;
  p->lengths[dst] = p->lengths[src];
  return MX_OK;
}

int mxkv_pool_reorder(mxkv_pool p, const int32_t* from) {
  if (!p || !from) return MX_ERR_NULL;
  for (int s = 0; s < p->seqs; s++)
    if (!has(p, from[s])) return MX_ERR_SHAPE;
  return guarded([&] {
    const std::vector<int32_t> table = p->table, lengths = p->lengths;  // may throw: nothing has changed yet
    const auto held = [&](int s) { return p->pages_of(lengths[s]); };
    for (int s = 0; s < p->seqs; s++)  // the new holders first, so that no page that stays is given up
      for (int c = 0; c < held(from[s]); c++) p->holders[table[(size_t)from[s] * p->cols + c]]++;
    for (int s = 0; s < p->seqs; s++) {
      for (int c = 0; c < held(s); c++) p->drop(table[(size_t)s * p->cols + c]);
      std::copy(table.begin() + (size_t)from[s] * p->cols, table.begin() + (size_t)(from[s] + 1) * p->cols, p->row(s));
      p->lengths[s] = lengths[from[s]];
    }
    return (int)MX_OK;
  });
}

int mxkv_pool_compact(mxkv_pool p, int32_t* pairs, int max_pairs, int* n_pairs) {
  if (!p || !n_pairs || (max_pairs > 0 && !pairs)) return MX_ERR_NULL;
  if (max_pairs < 0) return MX_ERR_SHAPE;
  return guarded([&] {
    std::vector<int32_t> now(p->pages, -1);  // where a moved page lies now; may throw
    std::vector<int32_t> left;               // free pages after the moves
    left.reserve(p->pages);
    int n = 0, lo = 0, hi = p->pages - 1;
    for (;;) {
      while (lo < hi && p->holders[lo]) lo++;
      while (hi > lo && !p->holders[hi]) hi--;
      if (lo >= hi || n == max_pairs) break;
      pairs[2 * n] = hi, pairs[2 * n + 1] = lo;
      n++;
      now[hi] = lo;
      std::swap(p->holders[lo], p->holders[hi]);
    }
    for (int i = 0; i < p->pages; i++)
      if (!p->holders[i]) left.push_back(i);
    if (n) {
      for (int s = 0; s < p->seqs; s++)
        for (int c = 0; c < p->held(s); c++)
          if (now[p->row(s)[c]] >= 0) p->row(s)[c] = now[p->row(s)[c]];
      p->free = decltype(p->free)(std::greater<int32_t>(), std::move(left));
    }
    *n_pairs = n;
    return (int)MX_OK;
  });
}

const int32_t* mxkv_pool_table(mxkv_pool p) { return p ? p->table.data() : nullptr; }
const int32_t* mxkv_pool_lengths(mxkv_pool p) { return p ? p->lengths.data() : nullptr; }
int mxkv_pool_used(mxkv_pool p) { return p ? p->used : 0; }

}  // extern "C"
