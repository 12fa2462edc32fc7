// pages.hip -- copies of whole pages of a paged key-value cache, over all layers in one launch.
//
// A page's elements lie together in either order, so a copy is a gather of contiguous pieces: the pairs'
// bytes of a plane are numbered through, each thread takes one 16-byte word and finds its pair by a
// division by the page's words, exact in one product (a division of 64-bit numbers per workgroup before: 4 pages over 8
// layers 4.4 -> 3.7 us in a graph of calls; 4.6 us a call where the host queues each). Bound by memory: each byte is read and written
// once (700 pairs of 64 slots x 8 x 128 E4M3 over four layers, 755 MB moved: 134 us, 5.6 TB/s, where torch's copy of as
// much reaches 5.3; with two words per thread 145, with four 153 before stores were non-temporal). The stores leave the caches to what
// is read; non-temporal loads gained a little more on large copies but lost a third on pages that the caches still held.
#include "kvcache.h"

using namespace mx;

namespace {

constexpr int kThreads = 256;  // words of a workgroup
constexpr int kLayers = 32;  // layers of one launch (their addresses are kernel arguments)

struct Planes {
  uint8_t* p[kLayers][4];  // k, v, ks, vs
};

// One kind of plane: `words` words of a page that is copied, one page every `stride` words.
struct Shape {
  int64_t stride;
  int words, blocks;  // blocks: workgroups over all pairs
  FastDiv div;
};

template <typename W>
MX_DEV void copy_words(W* base, const Shape& s, const int32_t* __restrict__ pairs, int n_pairs, int pages, int block) {
  const uint32_t i = (uint32_t)block * kThreads + threadIdx.x;  // below 2^31
  const int pair = (int)s.div.div(i);
  if (pair >= n_pairs) return;
  const int src = pairs[2 * pair], dst = pairs[2 * pair + 1];
  if (src < 0 || src >= pages || dst < 0 || dst >= pages || src == dst) return;
  const int64_t at = i - (uint32_t)pair * (uint32_t)s.words;
  __builtin_nontemporal_store(base[src * s.stride + at], base + dst * s.stride + at);
}

__global__ __launch_bounds__(kThreads) void copy_kernel(Planes planes, Shape data, Shape scale, int scale_bytes,
                                                        const int32_t* __restrict__ pairs, int n_pairs, int pages) {
  // x: workgroups of the data plane, then of the scale plane; y: layer; z: keys or values
  const int layer = blockIdx.y, kv = blockIdx.z;
  int block = blockIdx.x;
  if (block < data.blocks) {
    copy_words((u32x4*)planes.p[layer][kv], data, pairs, n_pairs, pages, block);
    return;
  }
  block -= data.blocks;
  uint8_t* s = planes.p[layer][2 + kv];
  if (scale_bytes == 16) copy_words((u32x4*)s, scale, pairs, n_pairs, pages, block);
  else if (scale_bytes == 4) copy_words((uint32_t*)s, scale, pairs, n_pairs, pages, block);
  else copy_words(s, scale, pairs, n_pairs, pages, block);
}

// False where a page has 2^30 words or more (a launch numbers the words of its pairs in 31 bits).
bool shape_of(int64_t page_bytes, int64_t stride_bytes, int word, Shape& s) {
  if (page_bytes / word >= (int64_t)1 << 30) return false;
  s.words = (int)(page_bytes / word);
  s.stride = stride_bytes / word;
  s.div = FastDiv((uint32_t)s.words);
  return true;
}

int blocks_of(const Shape& s, int n_pairs) { return (int)ceil_div((int64_t)s.words * n_pairs, (int64_t)kThreads); }

}  // namespace

extern "C" int mxkv_copy_run(const mxkv_cache* layers, int n_layers, const int32_t* pairs, int n_pairs, void* stream) {
  if (n_layers < 0 || n_layers > MX_MAX_DIM || n_pairs < 0 || n_pairs > MX_MAX_DIM) return MX_ERR_SHAPE;
  if (n_layers > 0 && !layers) return MX_ERR_NULL;
  for (int i = 0; i < n_layers; i++) {
    const mxkv_cache &c = layers[i], &z = layers[0];
    if (int s = check_cache(&c)) return s;
    if (c.fmt != z.fmt || c.order != z.order || c.pages != z.pages || c.page_size != z.page_size || c.heads != z.heads ||
        c.dim != z.dim || c.page_stride != z.page_stride)
      return MX_ERR_SHAPE;
  }
  if (n_layers == 0 || n_pairs == 0) return MX_OK;
  if (!pairs) return MX_ERR_NULL;
  const mxkv_cache& c = layers[0];
  const bool mx8 = c.fmt == MX_E4M3;
  const int bytes = mx8 ? 1 : 2;
  const int64_t elems = (int64_t)c.heads * c.page_size * c.dim;
  Shape data = {}, scale = {};
  if (!shape_of(elems * bytes, c.page_stride * bytes, 16, data)) return MX_ERR_SHAPE;
  int word = 16;  // a page's scales need not be whole 16-byte words
  if (mx8) {
    while (word > 1 && ((elems / 32) % word || (c.page_stride / 32) % word)) word /= 4;
    if (!shape_of(elems / 32, c.page_stride / 32, word, scale)) return MX_ERR_SHAPE;  // (fewer words than the data has)
  }
  const int most = (int)(((int64_t)1 << 31) - kThreads) / data.words;  // pairs of one launch
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  for (int first = 0; first < n_layers; first += kLayers) {
    const int n = n_layers - first < kLayers ? n_layers - first : kLayers;
    Planes p = {};
    for (int i = 0; i < n; i++) {
      const mxkv_cache& l = layers[first + i];
      p.p[i][0] = (uint8_t*)l.k, p.p[i][1] = (uint8_t*)l.v, p.p[i][2] = (uint8_t*)l.ks, p.p[i][3] = (uint8_t*)l.vs;
    }
    for (int at = 0; at < n_pairs;) {
      const int count = n_pairs - at < most ? n_pairs - at : most;
      data.blocks = blocks_of(data, count), scale.blocks = blocks_of(scale, count);
      hipLaunchKernelGGL(copy_kernel, dim3((unsigned)(data.blocks + scale.blocks), (unsigned)n, 2), dim3(kThreads), 0, st, p, data, scale,
                         word, pairs + 2 * (int64_t)at, count, c.pages);
      if (int s = launch_status()) return s;
      at += count;
    }
  }
  return sync_check(MX_OK, st);
}
