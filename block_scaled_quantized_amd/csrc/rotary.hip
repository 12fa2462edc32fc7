// rotary.hip -- rotary positions and the append to a paged key-value cache.
//
// Rotation: pair (a, b) of token t turns by w = pos[t] f[i]: (a cos w - b sin w, b cos w + a sin w).
// Both kernels move each element once and are bound by memory (by latency for few tokens), so the
// work per element is kept small: a workgroup takes a few tokens and a run of their heads, computes
// the tokens' cosines and sines once into LDS, one (token, pair) per thread, while its first rows
// are on their way, and every head reads them from there. The angle is reduced in 64 bits:
// pos * f / 2 pi loses about 2^-52 of its value (2^20 positions: 2^-32 turns), where 32 bits would
// lose the phase of far positions altogether. The reduced angle is rounded to fp32 for the sine and cosine (2 ulp),
// and its rest, up to 2^-25 half turns, turns them on: alone the rounding would be off by 9e-8, far more than
// 2 ulp of a small one.
//
// Rows move in 16-byte units whatever rot_dim is. Halves of whole units are loaded as pairs of units,
// neighbouring pairs lie in one; halves that begin within a unit (rot_dim / 2 not a multiple of it) are
// staged in LDS, where each element finds its partner. Measured, us of a call among others on changing inputs, 4096 tokens x
// 32 heads x 128 bf16, 67 MB: 10.9 with rot_dim = 128 in halves, 11.3 in pairs, 13.9 with rot_dim = 126 in halves (one pair at
// a time it took twice that). Append of 8191 tokens, 32 query and 8 cache heads of 128 bf16, 201 MB: 35 us, 5.7 TB/s; into an
// E4M3 cache 4096 tokens take 18 us. Pairs of times below compare two choices side by side in graphs of calls, about 1 us more each.
#include <cmath>
#include <type_traits>

#include "kvcache.h"
#include "quant_rules.h"

using namespace mx;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTrig = 512;        // (token, pair) angles of a workgroup
constexpr int kStageBytes = 16384;   // rows that a workgroup stages in LDS
// How a head's pairs lie: halves of whole 16-byte units; neighbours; halves that begin within a unit.
enum Layout { kHalves, kNeighbours, kOddHalves };

template <typename T>
struct Unit {  // 16 bytes of elements
  static constexpr int N = 16 / sizeof(T);
  T e[N];
};

// What is written is not read by this launch: stored non-temporally, it leaves the caches to the rows that are
// read (4096 x 32 x 128 bf16: 14.4 -> 12.4 us). Reads gain by it (STREAM) where a call's rows exceed what the
// caches can hold from the kernel that made them, and lose below (201 MB: 43 -> 38 us; 26 MB: 6.9 -> 8.5); the
// reads from memory also want four rows of a thread on their way where two do for the caches (38 against
// 41 us; 12.4 against 11.9).
constexpr int64_t kStreamBytes = 128 << 20;
constexpr int batch_of(bool stream) { return stream ? 4 : 2; }  // rows that a thread loads before it uses the first
template <bool STREAM, typename T>
MX_DEV Unit<T> load_unit(const T* p) {
  const u32x4* q = reinterpret_cast<const u32x4*>(p);
  if constexpr (STREAM) return __builtin_bit_cast(Unit<T>, __builtin_nontemporal_load(q));
  else return __builtin_bit_cast(Unit<T>, *q);
}
template <typename T>
MX_DEV void store_unit(T* p, const Unit<T>& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
}

// n / d for 0 <= n < 2^20 by one product: n + 1/2 is at least 1 / (2 d) of d away from a multiple, more than the
// reciprocal's and the product's roundings (2^-22 of the quotient) move it. The compiler's own division of whole
// numbers takes some twenty instructions (4096 tokens x 8 heads of 128 bf16 into an E4M3 cache: 10.0 -> 9.3 us;
// 2047 x 20 x 80 fp32 turned: 7.0 -> 6.4 us).
struct SmallDiv {
  int d;
  float inv;
  MX_DEV explicit SmallDiv(int div) : d(div), inv(__builtin_amdgcn_rcpf((float)div)) {}
  MX_DEV int div(int n) const { return (int)(((float)n + 0.5f) * inv); }
  MX_DEV int mod(int n) const { return n - div(n) * d; }
};

MX_DEV float to_f32(_Float16 x) { return (float)x; }
MX_DEV float to_f32(__bf16 x) { return (float)x; }
MX_DEV float to_f32(float x) { return x; }

// A pair (a, b) turned, w = (cos, sin). One product is rounded, the other is not, and the sum is rounded to fp32
// before it is to T: the same steps in every kernel, so that the append writes the bits that mxrope_run
// does. (For binary16 a barrier keeps the compiler from its mixed fma, which rounds once.)
template <typename T>
MX_DEV T round_to(float x) {
  if constexpr (std::is_same<T, _Float16>::value) asm("" : "+v"(x));
  return (T)x;
}
template <typename T>
MX_DEV T turn_a(float a, float b, float2 w) { return round_to<T>(__builtin_fmaf(a, w.x, -(b * w.y))); }
template <typename T>
MX_DEV T turn_b(float a, float b, float2 w) { return round_to<T>(__builtin_fmaf(b, w.x, a * w.y)); }

struct Rotation {
  const double* freq;
  int half;
  float factor, sign;
};

// cos and sin of `tokens` x half angles from pos[t0] into trig[token * half + pair].
MX_DEV void fill_trig(const Rotation& r, const int32_t* __restrict__ pos, int t0, int tokens, float2* trig) {
  const SmallDiv by_half(r.half);
  for (int i = threadIdx.x; i < tokens * r.half; i += kThreads) {
    const int t = by_half.div(i);
    double w = (double)pos[t0 + t] * r.freq[i - t * r.half] * 0.15915494309189533577;  // in turns
    w -= __builtin_rint(w);
    w += w;  // in half turns
    const float near = (float)w, rest = (float)(w - near) * 3.14159265358979323846f;
    float s, c;
    sincospif(near, &s, &c);
    const float cos_w = __builtin_fmaf(-rest, s, c), sin_w = __builtin_fmaf(rest, c, s);
    trig[i] = make_float2(cos_w * r.factor, sin_w * r.factor * r.sign);
  }
}

// How a head's 16-byte units are dealt to threads: `pairs` items that rotate (kHalves: a unit of each half
// together), then those that are copied.
struct Split {
  int pairs, items;
};

// A workgroup's rows: tokens t0 .. t0 + tokens - 1 times heads h0 .. h0 + heads - 1 of x.
template <typename T>
struct Rows {
  const T* x;
  int64_t xt, xh;
  int t0, tokens, h0, heads;
  MX_DEV const T* at(int t, int h) const { return x + (int64_t)(t0 + t) * xt + (int64_t)(h0 + h) * xh; }
};

// Units to store(token, head, element, unit). copy_tail: whether copied units need a store. Not for kOddHalves.
template <typename T, Layout L, bool STREAM, typename Store>
MX_DEV void rotate_rows(const Rotation& rot, const int32_t* __restrict__ pos, const Rows<T>& z, Split sp, bool copy_tail,
                        float2* trig, Store store) {
  constexpr int kBatch = batch_of(STREAM);
  constexpr int U = Unit<T>::N;
  const SmallDiv by_items(sp.items), by_heads(z.heads);
  const int per = by_items.div(kThreads);  // rows of one pass
  const int item = by_items.mod(threadIdx.x), r0 = by_items.div(threadIdx.x);
  const bool turns = item < sp.pairs, mine = r0 < per && (turns || copy_tail);
  const int rows = z.tokens * z.heads, half = rot.half;
  const int a = L == kNeighbours || turns ? U * item : 2 * half + U * (item - sp.pairs);  // first element
  bool ready = false;
  for (int base = r0; base - r0 < rows; base += per * kBatch) {  // the same number of turns for every thread
    Unit<T> lo[kBatch], hi[kBatch];
    int tok[kBatch], head[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      const int row = base + u * per;
      tok[u] = by_heads.div(row);
      head[u] = row - tok[u] * z.heads;
      if (mine && row < rows) {
        const T* p = z.at(tok[u], head[u]) + a;
        lo[u] = load_unit<STREAM>(p);
        if (L == kHalves && turns) hi[u] = load_unit<STREAM>(p + half);
      }
    }
    if (!ready) {
      fill_trig(rot, pos, z.t0, z.tokens, trig);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      if (!mine || base + u * per >= rows) continue;
      if (turns) {
        const float2* cs = trig + tok[u] * half + (L == kNeighbours ? item * (U / 2) : item * U);
        if constexpr (L == kNeighbours) {
#pragma unroll
          for (int i = 0; i < U / 2; i++) {
            const float p = to_f32(lo[u].e[2 * i]), q = to_f32(lo[u].e[2 * i + 1]);
            const float2 w = cs[i];  // (past the last pair: of the next token, or the padding, and unused)
            const bool turned = item * (U / 2) + i < half;
            lo[u].e[2 * i] = turned ? turn_a<T>(p, q, w) : lo[u].e[2 * i];
            lo[u].e[2 * i + 1] = turned ? turn_b<T>(p, q, w) : lo[u].e[2 * i + 1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < U; i++) {
            const float p = to_f32(lo[u].e[i]), q = to_f32(hi[u].e[i]);
            const float2 w = cs[i];
            lo[u].e[i] = turn_a<T>(p, q, w);
            hi[u].e[i] = turn_b<T>(p, q, w);
          }
        }
      }
      store(tok[u], head[u], a, lo[u]);
      if (L == kHalves && turns) store(tok[u], head[u], a + half, hi[u]);
    }
  }
}

// The rows as they are to LDS [row][dim] in units, and the angles; the caller synchronises.
template <typename T, bool STREAM>
MX_DEV void stage_rows(const Rotation& rot, const int32_t* __restrict__ pos, const Rows<T>& z, int dim, float2* trig, T* stage) {
  constexpr int kBatch = batch_of(STREAM), U = Unit<T>::N;
  const SmallDiv by_units(dim / U), by_heads(z.heads);
  const int per = by_units.div(kThreads), unit = by_units.mod(threadIdx.x), r0 = by_units.div(threadIdx.x);
  const int rows = z.tokens * z.heads;
  for (int base = r0; base < rows && r0 < per; base += per * kBatch) {
    Unit<T> v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      const int row = base + u * per, t = by_heads.div(row);
      if (row < rows) v[u] = load_unit<STREAM>(z.at(t, row - t * z.heads) + U * unit);
    }
#pragma unroll
    for (int u = 0; u < kBatch; u++)
      if (base + u * per < rows) *reinterpret_cast<Unit<T>*>(stage + (base + u * per) * dim + U * unit) = v[u];
  }
  fill_trig(rot, pos, z.t0, z.tokens, trig);
}

// The unit from element e0 of a staged row, turned (kOddHalves): each element's partner is read by itself, as its unit
// begins elsewhere.
template <typename T>
MX_DEV Unit<T> turned_unit(const T* row, int e0, int half, const float2* cs) {
  Unit<T> v = *reinterpret_cast<const Unit<T>*>(row + e0);
  if (e0 >= 2 * half) return v;
#pragma unroll
  for (int i = 0; i < Unit<T>::N; i++) {
    const int e = e0 + i;
    const bool second = e >= half;
    const int at = second ? e - half : e + half;  // within the row, whatever e
    const float2 w = cs[min(second ? e - half : e, half - 1)];
    // turn_b's step, or turn_a's: -(b sin) is b (-sin)
    const T turned = round_to<T>(__builtin_fmaf(to_f32(v.e[i]), w.x, to_f32(row[at]) * (second ? w.y : -w.y)));
    v.e[i] = e < 2 * half ? turned : v.e[i];
  }
  return v;
}

struct RopeArgs {
  Rotation rot;
  const int32_t* pos;
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh;
  int tokens, heads, tile_t, tile_h, groups;  // groups: runs of tile_h heads
  FastDiv groups_div;
  Split split;
  bool stream;
};

template <typename T, Layout L, bool STREAM>
MX_DEV void rope_block(const RopeArgs& a, int block, float2* trig, T* stage) {
  constexpr int U = Unit<T>::N;
  const int tile = (int)a.groups_div.div(block), g = block - tile * a.groups, t0 = tile * a.tile_t, h0 = g * a.tile_h;
  const Rows<T> z = {(const T*)a.x, a.xt, a.xh, t0, min(a.tile_t, a.tokens - t0), h0, min(a.tile_h, a.heads - h0)};
  const auto out = [&](int t, int h) -> T* { return (T*)a.out + (int64_t)(t0 + t) * a.ot + (int64_t)(h0 + h) * a.oh; };
  if constexpr (L != kOddHalves) {
    rotate_rows<T, L, STREAM>(a.rot, a.pos, z, a.split, a.x != a.out, trig,
                              [&](int t, int h, int e, const Unit<T>& v) { store_unit(out(t, h) + e, v); });
  } else {
    const SmallDiv by_units(a.split.items), by_heads(z.heads);
    const int dim = U * a.split.items, per = by_units.div(kThreads), unit = by_units.mod(threadIdx.x), r0 = by_units.div(threadIdx.x);
    stage_rows<T, STREAM>(a.rot, a.pos, z, dim, trig, stage);
    __syncthreads();
    if (r0 >= per || (unit >= a.split.pairs && a.x == a.out)) return;
    for (int row = r0; row < z.tokens * z.heads; row += per) {
      const int t = by_heads.div(row);
      store_unit(out(t, row - t * z.heads) + U * unit, turned_unit(stage + row * dim, U * unit, a.rot.half, trig + t * a.rot.half));
    }
  }
}

template <typename T, Layout L, bool STREAM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  __shared__ float2 trig[kMaxTrig + 8];
  __shared__ __attribute__((aligned(16))) T stage[L == kOddHalves ? kStageBytes / sizeof(T) : 1];
  rope_block<T, L, STREAM>(a, blockIdx.x, trig, stage);
}

// ---- append ---------------------------------------------------------------------------------

struct AppendArgs {
  RopeArgs q;       // the queries' blocks come first ...
  RopeArgs k;       // ... then the keys' ... (out unused)
  const void* v;    // ... then the values'
  int64_t vt, vh;
  int q_blocks, k_blocks;
  bool turn;  // keys are rotated
  const int32_t *seq, *table;
  int seqs, cols, pages, page_size, dim;
  int64_t page_stride, head_stride, slot_stride;
  uint8_t *kc, *vc, *ks, *vs;
  FastDiv page_div;
};

// Element offset of each token's slot (head 0) in the cache, -1 where it has none.
MX_DEV void fill_slots(const AppendArgs& a, int t0, int tokens, int64_t* slot) {
  for (int t = threadIdx.x; t < tokens; t += kThreads) {
    const int p = a.k.pos[t0 + t], s = a.seq ? a.seq[t0 + t] : t0 + t;
    int64_t at = -1;
    if (p >= 0 && s >= 0 && s < a.seqs) {
      const int c = (int)a.page_div.div((uint32_t)p);
      if (c < a.cols) {
        const int page = a.table[(int64_t)s * a.cols + c];
        if (page >= 0 && page < a.pages) at = page * a.page_stride + (p - c * a.page_size) * a.slot_stride;
      }
    }
    slot[t] = at;
  }
}

// Eight elements of a row to their place `at` in a plane (-1: nowhere).
template <typename T>
MX_DEV void write_unit(const Unit<T>& v, bool mx8, uint8_t* codes, uint8_t* scales, int64_t at) {
  if (!mx8) {
    if (at >= 0) store_unit(reinterpret_cast<T*>(codes + 2 * at), v);
    return;
  }
  // Four neighbouring lanes hold a block of 32: they agree on its scale, and each writes its 8 codes.
  float x[8];
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    x[i] = to_f32(v.e[i]);
    amax = max(amax, fbits(x[i]) & 0x7FFFFFFFu);  // NaN and Inf have the largest patterns
  }
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
  const bool nonfinite = amax >= 0x7F800000u;
  int t;
  const uint32_t E = mx_block_scale(amax, nonfinite, MX_E4M3, &t);
  // gfx950's scaled conversion rounds as the rule does and writes NaN where it should saturate: those
  // bytes become +-448 (the GPU pack's conversion).
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float scale = bitsf(E << 23);
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    s16x2 r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32((s16x2){0, 0}, x[4 * i], x[4 * i + 1], scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, x[4 * i + 2], x[4 * i + 3], scale, true);
    uint32_t c = __builtin_bit_cast(uint32_t, r);
    c ^= (((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
    w[i] = nonfinite ? 0u : c;
  }
  if (at < 0) return;
  __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(codes + at));
  if (at % 32 == 0) scales[at / 32] = (uint8_t)E;
}

template <typename T, Layout L, bool STREAM>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, bool mx8) {
  __shared__ float2 trig[kMaxTrig + 8];
  __shared__ __attribute__((aligned(16))) T stage[kStageBytes / sizeof(T)];
  __shared__ int64_t slot[kMaxTrig];
  int block = blockIdx.x;
  if (block < a.q_blocks) {
    rope_block<T, L, STREAM>(a.q, block, trig, stage);
    return;
  }
  block -= a.q_blocks;
  const bool key = block < a.k_blocks;
  if (!key) block -= a.k_blocks;
  const int tile = (int)a.k.groups_div.div(block), g = block - tile * a.k.groups, t0 = tile * a.k.tile_t, h0 = g * a.k.tile_h;
  const int tokens = min(a.k.tile_t, a.k.tokens - t0), heads = min(a.k.tile_h, a.k.heads - h0);
  fill_slots(a, t0, tokens, slot);
  if (key && a.turn) {
    const Rows<T> z = {(const T*)a.k.x, a.k.xt, a.k.xh, t0, tokens, h0, heads};
    if constexpr (L == kOddHalves)
      stage_rows<T, STREAM>(a.k.rot, a.k.pos, z, a.dim, trig, stage);
    else
      rotate_rows<T, L, STREAM>(a.k.rot, a.k.pos, z, a.k.split, true, trig, [&](int t, int h, int e, const Unit<T>& v) {
        *reinterpret_cast<Unit<T>*>(stage + (t * heads + h) * a.dim + e) = v;
      });
  }
  __syncthreads();
  // Rows go out in units of 8 elements; dim / 8 divides nothing in general, so threads past the last
  // whole row of a pass idle (they still take part in the lane exchange).
  const SmallDiv by_units(a.dim / 8), by_heads(heads);
  const int per = by_units.div(kThreads), unit = by_units.mod(threadIdx.x), r0 = by_units.div(threadIdx.x);
  const T* x = key ? (const T*)a.k.x : (const T*)a.v;
  const int64_t xt = key ? a.k.xt : a.vt, xh = key ? a.k.xh : a.vh;
  uint8_t *codes = key ? a.kc : a.vc, *scales = key ? a.ks : a.vs;
  for (int base = 0; base < tokens * heads; base += per) {
    const int row = base + r0;
    const bool mine = r0 < per && row < tokens * heads;
    const int t = mine ? by_heads.div(row) : 0, h = mine ? row - t * heads : 0;
    Unit<T> v = {};
    if (mine && L == kOddHalves && key && a.turn)
      v = turned_unit(stage + row * a.dim, 8 * unit, a.k.rot.half, trig + t * a.k.rot.half);
    else if (mine)
      v = key && a.turn ? *reinterpret_cast<const Unit<T>*>(stage + row * a.dim + 8 * unit)
                        : load_unit<false>(x + (int64_t)(t0 + t) * xt + (int64_t)(h0 + h) * xh + 8 * unit);
    const int64_t s = mine ? slot[t] : -1;
    write_unit<T>(v, mx8, codes, scales, s < 0 ? -1 : s + (h0 + h) * a.head_stride + 8 * unit);
  }
}

// ---- host -----------------------------------------------------------------------------------

Layout layout_of(int layout, int rot_dim, int unit) {
  return layout == MXROPE_PAIRS ? kNeighbours : rot_dim / 2 % unit == 0 ? kHalves : kOddHalves;
}

Split split_of(Layout layout, int rot_dim, int dim, int unit) {
  if (layout == kHalves) return {rot_dim / 2 / unit, rot_dim / 2 / unit + (dim - rot_dim) / unit};
  return {ceil_div(rot_dim, unit), dim / unit};
}

// Tokens and heads of a workgroup. max_rows bounds tile_t * tile_h.
void tile(RopeArgs& a, int max_rows) {
  const int per = kThreads / a.split.items;  // rows of a pass
  const int half = a.rot.half > 0 ? a.rot.half : 1;
  a.tile_h = a.heads < max_rows ? a.heads : max_rows;
  const int cap = max_rows < per * batch_of(a.stream) ? max_rows : per * batch_of(a.stream);  // one batch of loads per thread
  a.tile_t = 1;
  while (2 * a.tile_t * a.tile_h <= cap && 2 * a.tile_t * half <= kMaxTrig && (a.tokens + a.tile_t - 1) / a.tile_t > 1024)
    a.tile_t *= 2;
  // few tokens: spread a token's heads over workgroups instead
  while (a.tile_t == 1 && a.tile_h > per && (int64_t)a.tokens * ceil_div(a.heads, a.tile_h) < 512) a.tile_h = ceil_div(a.tile_h, 2);
  a.groups = ceil_div(a.heads, a.tile_h);
  a.groups_div = FastDiv((uint32_t)a.groups);
}

int64_t blocks_of(const RopeArgs& a) { return (int64_t)ceil_div(a.tokens, a.tile_t) * a.groups; }

int check_rope(const mxrope* r, int dim) {
  if (!r || !r->freq) return MX_ERR_NULL;
  if (r->layout != MXROPE_HALF && r->layout != MXROPE_PAIRS) return MX_ERR_FORMAT;
  if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > dim) return MX_ERR_SHAPE;
  return (reinterpret_cast<uintptr_t>(r->freq) & 7u) ? MX_ERR_ALIGN : MX_OK;
}

RopeArgs rope_args(const mxrope* r, int tokens, int dim, const mx_heads* x, const mx_heads* out, const int32_t* pos, int inverse,
                   int unit, Layout layout) {
  RopeArgs a = {};
  a.rot = {r ? r->freq : nullptr, r ? r->rot_dim / 2 : 0, r ? r->factor : 1.0f, inverse ? -1.0f : 1.0f};
  a.pos = pos;
  a.x = x->data, a.xt = x->token_stride, a.xh = x->head_stride;
  if (out) a.out = out->data, a.ot = out->token_stride, a.oh = out->head_stride;
  a.tokens = tokens, a.heads = x->heads;
  a.split = split_of(layout, r ? r->rot_dim : 0, dim, unit);
  return a;
}

template <typename T, Layout L>
void rope_launch(const RopeArgs& a, dim3 grid, hipStream_t st) {
  if (a.stream) hipLaunchKernelGGL((rope_kernel<T, L, true>), grid, dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((rope_kernel<T, L, false>), grid, dim3(kThreads), 0, st, a);
}
template <typename T>
void rope_launch(const RopeArgs& a, Layout layout, dim3 grid, hipStream_t st) {
  if (layout == kHalves) rope_launch<T, kHalves>(a, grid, st);
  else if (layout == kNeighbours) rope_launch<T, kNeighbours>(a, grid, st);
  else rope_launch<T, kOddHalves>(a, grid, st);
}

template <typename T, Layout L>
void append_launch(const AppendArgs& a, bool mx8, dim3 grid, hipStream_t st) {
  if (a.k.stream) hipLaunchKernelGGL((append_kernel<T, L, true>), grid, dim3(kThreads), 0, st, a, mx8);
  else hipLaunchKernelGGL((append_kernel<T, L, false>), grid, dim3(kThreads), 0, st, a, mx8);
}
template <typename T>
void append_launch(const AppendArgs& a, Layout layout, bool mx8, dim3 grid, hipStream_t st) {
  if (layout == kHalves) append_launch<T, kHalves>(a, mx8, grid, st);
  else if (layout == kNeighbours) append_launch<T, kNeighbours>(a, mx8, grid, st);
  else append_launch<T, kOddHalves>(a, mx8, grid, st);
}

}  // namespace

extern "C" int mxrope_freqs_host(int rot_dim, double base, int rule, const double* params, double* freq, float* factor) {
  if (!freq || !factor) return MX_ERR_NULL;
  if (rule < MXROPE_PLAIN || rule > MXROPE_YARN) return MX_ERR_FORMAT;
  if (rule != MXROPE_PLAIN && !params) return MX_ERR_NULL;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > kMaxHeadDim || !(base > 0) || !std::isfinite(base)) return MX_ERR_SHAPE;
  const int count = rule == MXROPE_PLAIN ? 0 : rule <= MXROPE_NTK ? 1 : 4;
  for (int i = 0; i < count; i++)
    if (!std::isfinite(params[i]) || (i < 2 && !(params[i] > 0))) return MX_ERR_SHAPE;
  if (rule == MXROPE_BANDS && !(params[3] > params[2])) return MX_ERR_SHAPE;
  if (rule == MXROPE_YARN && !(base > 1 && params[2] > 0 && params[3] > 0)) return MX_ERR_SHAPE;
  if (rule == MXROPE_NTK && rot_dim > 2) base *= std::pow(params[0], rot_dim / (rot_dim - 2.0));
  const double turn = 2 * 3.14159265358979323846;
  double lo = 0, hi = 0;
  if (rule == MXROPE_YARN) {
    const auto at = [&](double turns) { return rot_dim * std::log(params[1] / (turns * turn)) / (2 * std::log(base)); };
    lo = std::fmax(std::floor(at(params[2])), 0.0);
    hi = std::fmin(std::ceil(at(params[3])), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; i++) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double k;  // share of the frequency that is kept
    switch (rule) {
      case MXROPE_LINEAR: k = 0; break;
      case MXROPE_BANDS: k = std::fmin(std::fmax((params[1] * f / turn - params[2]) / (params[3] - params[2]), 0.0), 1.0); break;
      case MXROPE_YARN: k = 1 - std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0); break;
      default: k = 1;
    }
    freq[i] = k == 1 ? f : (1 - k) * f / params[0] + k * f;
  }
  *factor = rule == MXROPE_YARN && params[0] > 1 ? (float)(0.1 * std::log(params[0]) + 1.0) : 1.0f;
  return MX_OK;
}

extern "C" int mxrope_run(int f, const mxrope* rope, int tokens, int dim, const mx_heads* x, const mx_heads* out,
                          const int32_t* positions, int inverse, void* stream) {
  if (f != MX_F16 && f != MX_BF16 && f != MX_F32) return MX_ERR_FORMAT;
  if (!rope || !x || !out) return MX_ERR_NULL;
  if (tokens < 0 || tokens > MX_MAX_DIM || !dim_ok(dim)) return MX_ERR_SHAPE;
  if (int s = check_rope(rope, dim)) return s;
  const int bytes = f == MX_F32 ? 4 : 2;
  if (tokens == 0) return MX_OK;
  if (!positions) return MX_ERR_NULL;
  if (int s = check_heads(x, bytes)) return s;
  if (int s = check_heads(out, bytes)) return s;
  if (x->heads != out->heads) return MX_ERR_SHAPE;
  if (x->data == out->data && (x->token_stride != out->token_stride || x->head_stride != out->head_stride)) return MX_ERR_SHAPE;
  const Layout layout = layout_of(rope->layout, rope->rot_dim, 16 / bytes);
  RopeArgs a = rope_args(rope, tokens, dim, x, out, positions, inverse, 16 / bytes, layout);
  a.stream = 2ll * tokens * x->heads * dim * bytes >= kStreamBytes;
  tile(a, layout == kOddHalves ? kStageBytes / (dim * bytes) : 1 << 20);
  // at most tokens + 1024, but a workgroup per kStageBytes of staged rows
  if (blocks_of(a) >= 1 << 24) return MX_ERR_SHAPE;
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  const dim3 grid((unsigned)blocks_of(a));
  if (f == MX_F16) rope_launch<_Float16>(a, layout, grid, st);
  else if (f == MX_BF16) rope_launch<__bf16>(a, layout, grid, st);
  else rope_launch<float>(a, layout, grid, st);
  return sync_check(launch_status(), st);
}

extern "C" int mxkv_append_run(const mxkv_cache* cache, int f, int tokens, const mx_heads* k, const mx_heads* v,
                               const int32_t* positions, const int32_t* seq, const mxkv_table* table, const mxrope* rope,
                               const mx_heads* q, const mx_heads* q_out, void* stream) {
  if (!cache || !k || !v || !table) return MX_ERR_NULL;
  if (f != MX_F16 && f != MX_BF16) return MX_ERR_FORMAT;
  if (int s = check_cache(cache)) return s;
  const bool mx8 = cache->fmt == MX_E4M3;
  if (!mx8 && cache->fmt != f) return MX_ERR_FORMAT;
  if (tokens < 0 || tokens > MX_MAX_DIM) return MX_ERR_SHAPE;
  if (int s = check_table(table)) return s;
  if ((q == nullptr) != (q_out == nullptr) || (q && !rope)) return MX_ERR_NULL;
  if (rope)
    if (int s = check_rope(rope, cache->dim)) return s;
  if (tokens == 0) return MX_OK;
  if (!positions) return MX_ERR_NULL;
  if (int s = check_heads(k, 2)) return s;
  if (int s = check_heads(v, 2)) return s;
  if (k->heads != cache->heads || v->heads != cache->heads) return MX_ERR_SHAPE;
  if (q) {
    if (int s = check_heads(q, 2)) return s;
    if (int s = check_heads(q_out, 2)) return s;
    if (q->heads != q_out->heads) return MX_ERR_SHAPE;
    if (q->data == q_out->data && (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
      return MX_ERR_SHAPE;
  }
  const Layout layout = rope ? layout_of(rope->layout, rope->rot_dim, 8) : kHalves;
  AppendArgs a = {};
  a.k = rope_args(rope, tokens, cache->dim, k, nullptr, positions, 0, 8, layout);
  a.k.stream = 4ll * tokens * (cache->heads * 2 + (q ? q->heads : 0)) * cache->dim >= kStreamBytes;
  const int staged = kStageBytes / (2 * cache->dim);  // rows
  tile(a.k, staged);
  int64_t q_blocks = 0;
  if (q) {
    a.q = rope_args(rope, tokens, cache->dim, q, q_out, positions, 0, 8, layout);
    a.q.stream = a.k.stream;
    tile(a.q, layout == kOddHalves ? staged : 1 << 20);
    q_blocks = blocks_of(a.q);
  }
  const int64_t k_blocks = blocks_of(a.k);
  if (q_blocks + 2 * k_blocks >= 1 << 24) return MX_ERR_SHAPE;
  a.v = v->data, a.vt = v->token_stride, a.vh = v->head_stride;
  a.q_blocks = (int)q_blocks, a.k_blocks = (int)k_blocks;
  a.turn = rope != nullptr;
  a.seq = seq, a.table = table->pages, a.seqs = table->seqs, a.cols = table->cols;
  a.pages = cache->pages, a.page_size = cache->page_size, a.dim = cache->dim;
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.kc = (uint8_t*)cache->k, a.vc = (uint8_t*)cache->v, a.ks = (uint8_t*)cache->ks, a.vs = (uint8_t*)cache->vs;
  a.page_div = FastDiv((uint32_t)cache->page_size);
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  const dim3 grid((unsigned)(q_blocks + 2 * k_blocks));
  if (f == MX_F16) append_launch<_Float16>(a, layout, mx8, grid, st);
  else append_launch<__bf16>(a, layout, mx8, grid, st);
  return sync_check(launch_status(), st);
}
