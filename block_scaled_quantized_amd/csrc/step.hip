// step.hip -- a serving step's bookkeeping on the device: from the tokens that each row has and will have, the pages that it takes
// or gives back, its table, and the step's tokens with their rows, positions and slots.
//
// Integers throughout. Rows' pages and tokens are counted, summed over the rows before each (one workgroup, a row per thread), and
// the pages and tokens then numbered through: thread i finds the row of page or token i by bisection of the sums. The free pages are
// a stack; what a call gives back goes onto it in the order that undoes taking the same pages. Bound by the chain of dependent
// memory latencies (rows, stack, table, slots), so one launch does all where the tokens are few: 256 rows, one token each, 4.6 us, of which a kernel
// of one store takes 3.6. With more tokens than one workgroup writes in the time of a launch, a second kernel writes them.
#include <algorithm>

#include "kvcache.h"

using namespace mx;

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kFew = 8192;         // tokens that the one workgroup writes itself
constexpr int kTokenThreads = 256;

struct Args {
  int32_t* table;
  const int32_t *lengths, *wants, *kept;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t *lengths_out, *n_free_out, *offsets, *seq, *positions, *slots, *status;
  int seqs, cols, page_size, pages, max_tokens, most;  // most: cols * page_size
  FastDiv page_div;
};

struct Row {
  int has, tokens, takes, clears, gives, old_pages, new_pages, keep;
  bool bad;
};

// A count is cut to one above what any limit allows, so that sums of 1024 stay in 32 bits.
MX_DEV int cut(int n) { return min(n, MX_MAX_DIM + 1); }

MX_DEV Row row_of(const Args& a, int b) {
  Row r = {};
  if (b >= a.seqs) return r;
  const int want = a.wants[b];
  r.has = max(0, min(a.lengths[b], a.most));
  r.bad = want > a.most;
  const int to = want < 0 ? r.has : min(want, a.most);
  const auto pages = [&](int n) { return n == 0 ? 0 : (int)a.page_div.div((uint32_t)(n - 1)) + 1; };
  r.old_pages = pages(r.has), r.new_pages = pages(to);
  r.keep = a.kept ? max(0, a.kept[b]) : 0;
  r.tokens = cut(max(0, to - r.has));
  r.takes = cut(max(0, r.new_pages - r.old_pages));
  r.clears = cut(max(0, r.old_pages - r.new_pages));
  r.gives = cut(max(0, r.old_pages - max(r.new_pages, r.keep)));
  return r;
}

MX_DEV uint32_t wave_scan(uint32_t x) {  // sum over the lanes up to this one
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // lane 15 of a row to the next row
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return x;
}

enum { kTokens, kTakes, kClears, kGives, kBad, kKinds };
struct Sums {
  int n[kKinds];
};

// Sums over the workgroup's rows before this thread's, and all of them. Two barriers.
MX_DEV void scan(const Row& r, Sums& before, Sums& all, int (*lds)[kKinds]) {
  const int v[kBad] = {r.tokens, r.takes, r.clears, r.gives}, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int own[kBad];
#pragma unroll
  for (int i = 0; i < kBad; i++) {
    own[i] = (int)wave_scan((uint32_t)v[i]);
    if (lane == 63) lds[wave][i] = own[i];
  }
  const bool bad = __any(r.bad);
  if (lane == 0) lds[wave][kBad] = bad;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKinds; i++) {  // lane w has wave w's sum
    const int sum = (int)wave_scan(lane < kWaves ? (uint32_t)lds[lane][i] : 0u), w = __builtin_amdgcn_readfirstlane(wave);
    all.n[i] = __builtin_amdgcn_readlane(sum, kWaves - 1);
    if (i < kBad) before.n[i] = (w ? __builtin_amdgcn_readlane(sum, w - 1) : 0) + own[i] - v[i];
  }
  __syncthreads();
}

// The last i with sums[i] <= x, of n + 1 rising sums that begin with one <= x.
MX_DEV int row_at(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

MX_DEV void put_token(const Args& a, int t, int row, int pos) {
  a.seq[t] = row, a.positions[t] = pos;
  if (!a.slots) return;
  int slot = -1;
  if (row >= 0) {
    const int col = (int)a.page_div.div((uint32_t)pos), page = a.table[(int64_t)row * a.cols + col];
    if (page >= 0 && page < a.pages) slot = page * a.page_size + pos - col * a.page_size;
  }
  a.slots[t] = slot;
}

__global__ __launch_bounds__(kThreads) void step_kernel(Args a, int fill) {
  __shared__ int waves[kWaves][kKinds];
  __shared__ int sums[kThreads + 1], first[kThreads], other[kThreads];
  const int t = threadIdx.x;
  const bool one = a.seqs <= kThreads;  // all rows at once: each is read once
  const int n_free = max(0, min(a.n_free[0], a.pages));

  Row row = row_of(a, t);
  Sums before, all;
  scan(row, before, all, waves);
  for (int b0 = kThreads; b0 < a.seqs; b0 += kThreads) {
    Sums x, more;
    scan(row_of(a, b0 + t), x, more, waves);
#pragma unroll
    for (int i = 0; i < kKinds; i++) all.n[i] = cut(cut(all.n[i]) + more.n[i]);
  }
  const int top = n_free + all.n[kGives];  // of the stack, when everything is given back
  const int status = (all.n[kBad] ? MXKV_STEP_LONG : 0) | (all.n[kTokens] > a.max_tokens ? MXKV_STEP_TOKENS : 0) |
                     (all.n[kTakes] > top ? MXKV_STEP_PAGES : 0) | (top > a.pages ? MXKV_STEP_STACK : 0);
  if (t == 0) a.status[0] = status;
  if (status) {  // nothing changes, and the step has no tokens
    for (int b = t; b < a.seqs; b += kThreads) a.lengths_out[b] = a.lengths[b];
    for (int b = t; b <= a.seqs; b += kThreads) a.offsets[b] = 0;
    if (t == 0) a.n_free_out[0] = n_free;
    if (fill)
      for (int i = t; i < a.max_tokens; i += kThreads) put_token(a, i, -1, -1);
    return;
  }

  // give back: page i of all that are goes to place top - 1 - i
  if (all.n[kClears]) {
    int given = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
      Sums here = all;
      if (!one) {
        row = row_of(a, b0 + t);
        scan(row, before, here, waves);
      }
      sums[t] = before.n[kClears], first[t] = row.new_pages, other[t] = given + before.n[kGives] - max(0, row.keep - row.new_pages);
      if (t == 0) sums[kThreads] = here.n[kClears];
      __syncthreads();
      for (int i = t; i < here.n[kClears]; i += kThreads) {
        const int r = row_at(sums, kThreads, i), step = i - sums[r], col = first[r] + step;
        int32_t* cell = a.table + (int64_t)(b0 + r) * a.cols + col;
        const int kept = a.kept ? a.kept[b0 + r] : 0;
        // other: the number of the row's first cleared page among all given back, were none of the row's kept
        if (col >= kept) a.free_pages[top - 1 - (other[r] + step)] = *cell;
        *cell = -1;
      }
      given += here.n[kGives];
      __syncthreads();
    }
    __threadfence_block();
    __syncthreads();
  }

  // take: page i comes from place top - 1 - i
  int taken = 0, tokens = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    Sums here = all;
    if (!one) {
      row = row_of(a, b0 + t);
      scan(row, before, here, waves);
    }
    const int b = b0 + t;
    sums[t] = before.n[kTakes], first[t] = row.old_pages;
    if (t == 0) sums[kThreads] = here.n[kTakes];
    if (b < a.seqs) {
      a.offsets[b] = tokens + before.n[kTokens];
      const int want = a.wants[b];
      a.lengths_out[b] = want < 0 ? row.has : want;
    }
    __syncthreads();
    for (int i = t; i < here.n[kTakes]; i += kThreads) {
      const int r = row_at(sums, kThreads, i), col = first[r] + i - sums[r];
      a.table[(int64_t)(b0 + r) * a.cols + col] = a.free_pages[top - 1 - (taken + i)];
    }
    taken += here.n[kTakes], tokens += here.n[kTokens];
    __syncthreads();
  }
  if (t == 0) a.offsets[a.seqs] = tokens, a.n_free_out[0] = top - taken;
  if (!fill) return;

  if (one) {  // the rows' first tokens and positions stay in LDS
    sums[t] = before.n[kTokens], first[t] = row.has;
    if (t == 0) sums[kThreads] = tokens;
  }
  __threadfence_block();
  __syncthreads();
  for (int i = t; i < a.max_tokens; i += kThreads) {
    if (i >= tokens) {
      put_token(a, i, -1, -1);
    } else if (one) {
      const int r = row_at(sums, kThreads, i);
      put_token(a, i, r, first[r] + i - sums[r]);
    } else {
      const int r = row_at(a.offsets, a.seqs, i), from = a.offsets[r];
      put_token(a, i, r, a.lengths_out[r] - (a.offsets[r + 1] - from) + i - from);
    }
  }
}

// The tokens of a step that has many of them.
__global__ __launch_bounds__(kTokenThreads) void tokens_kernel(Args a) {
  const int i = blockIdx.x * kTokenThreads + threadIdx.x;
  if (i >= a.max_tokens) return;
  if (i >= a.offsets[a.seqs]) {
    put_token(a, i, -1, -1);
    return;
  }
  const int r = row_at(a.offsets, a.seqs, i), from = a.offsets[r];
  put_token(a, i, r, a.lengths_out[r] - (a.offsets[r + 1] - from) + i - from);
}

}  // namespace

extern "C" int mxkv_step_run(const mxkv_step* s, void* stream) {
  if (!s) return MX_ERR_NULL;
  if (s->seqs < 0 || s->seqs > MX_MAX_DIM || s->cols < 1 || s->page_size < 1 || s->page_size > MX_MAX_DIM || s->pages < 1 || s->pages > MX_MAX_DIM ||
      s->max_tokens < 0 || s->max_tokens > MX_MAX_DIM || (int64_t)s->cols * s->page_size >= (int64_t)1 << 31 || (int64_t)s->pages * s->page_size >= (int64_t)1 << 31)
    return MX_ERR_SHAPE;
  if (s->seqs == 0) return MX_OK;
  if (!s->table || !s->lengths || !s->wants || !s->free_pages || !s->n_free || !s->lengths_out || !s->n_free_out || !s->offsets || !s->status) return MX_ERR_NULL;
  if (s->max_tokens > 0 && (!s->seq || !s->positions)) return MX_ERR_NULL;
  Args a = {};
  a.table = s->table, a.lengths = s->lengths, a.wants = s->wants, a.kept = s->kept, a.free_pages = s->free_pages, a.n_free = s->n_free;
  a.lengths_out = s->lengths_out, a.n_free_out = s->n_free_out, a.offsets = s->offsets, a.seq = s->seq, a.positions = s->positions;
  a.slots = s->slots, a.status = s->status;
  a.seqs = s->seqs, a.cols = s->cols, a.page_size = s->page_size, a.pages = s->pages, a.max_tokens = s->max_tokens;
  a.most = s->cols * s->page_size;
  a.page_div = FastDiv((uint32_t)s->page_size);
  if (int e = check_arch()) return e;
  const hipStream_t st = as_stream(stream);
  const bool fill = s->max_tokens <= kFew;
  hipLaunchKernelGGL(step_kernel, dim3(1), dim3(kThreads), 0, st, a, fill ? 1 : 0);
  if (int e = launch_status()) return e;
  if (!fill) {
    hipLaunchKernelGGL(tokens_kernel, dim3((unsigned)ceil_div(s->max_tokens, kTokenThreads)), dim3(kTokenThreads), 0, st, a);
    if (int e = launch_status()) return e;
  }
  return sync_check(MX_OK, st);
}
