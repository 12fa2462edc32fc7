// attention.hip -- attention of one new token per sequence over a paged key-value cache.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = e^(s_j - m), s_j = scale q.k_j, in one pass over the cache: a
// wave keeps the running maximum m, sum and output of its keys and rescales them where m grows. The
// cache is read once and bounds the time (each key-value pair of bytes meets the few query heads that
// share it), so everything else serves its loads: 16 query heads of one cache head are the columns of a
// 16x16x32 matrix instruction (columns without a head idle: the matrix cores have more than ten times
// the rate that the memory asks of them), K and V go from global memory to registers with no LDS
// between, and the lengths are split over workgroups.
//
// A wave takes tiles of 32 keys, as two halves of 16. Scores are formed transposed, S^T = K Q^T (rows:
// keys, columns: heads): lane (c = lane % 16, g = lane / 16) loads 16 bytes of key row c. It then
// holds S^T of head c and keys 4 g .. 4 g + 3 of each half, which is an operand of out^T = V^T P^T as it
// stands if the sum over the tile's keys runs in the order (g, half, key): the same lane's V rows are
// those eight keys, 8 (D = 64: 4) neighbouring elements of each, and an 8 x 8 transpose within the lane (32
// byte permutes) gives V^T operands whose row c of instruction i is element 8 c + i. No lane ever needs
// another's keys, and every load instruction covers whole rows.
//
// E4M3 elements become 16-bit ones on the way by gfx950's scaled conversion, which takes the block's
// power of two: a lane's 8 K elements and its V elements of one key lie in one block of 32.
#include "kvcache.h"

using namespace mx;

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 32;                // keys of a wave's tile
constexpr int kGrain = kTile * kWaves;   // keys that the workgroup's waves take in turn
constexpr int kSpan = 2048;              // keys whose pages are looked up at a time
constexpr int kMaxChunks = 256;          // workgroups over one sequence's length
constexpr int kPad = 4;                  // floats that keep the heads' rows of the merge on different banks
// Probabilities are rounded to f's format for the matrix cores. p = 2^(x - m) is at most 1; binary16
// would lose those under 2^-24, which can matter in number in a long row, so they are scaled by 2^15
// (which cancels in the division by their sum).
constexpr float kShift = 15.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct Args {
  const uint8_t *k, *v, *ks, *vs;
  const void* q;
  void* out;
  float* lse;
  const int32_t *table, *lengths, *starts;
  uint32_t* counters;
  float* partial;
  int64_t qt, qh, ot, oh, page_stride, head_stride, slot_stride;
  int heads, group, tiles, dim, cols, pages, page_size, max_len, window, chunk, chunks;
  float scale, softcap;
  FastDiv page_div;
};

template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  typedef f16x8 x8;
  typedef f16x2 x2;
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static MX_DEV uint32_t from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HI));
  }
};
template <>
struct Vec<__bf16> {
  typedef bf16x8 x8;
  typedef bf16x2 x2;
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static MX_DEV uint32_t from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
  }
};

// Eight E4M3 codes times 2^(e - 127) as eight 16-bit values; a NaN scale (255) makes NaN of each.
template <typename T>
MX_DEV u32x4 widen(u32x2 c, uint32_t e) {
  const float s = bitsf(e << 23);
  u32x4 r = {Vec<T>::template from_e4m3<false>(c[0], s), Vec<T>::template from_e4m3<true>(c[0], s),
             Vec<T>::template from_e4m3<false>(c[1], s), Vec<T>::template from_e4m3<true>(c[1], s)};
  if (e == 255u) r = (u32x4){~0u, ~0u, ~0u, ~0u};
  return r;
}

MX_DEV float wave_max(float x) {  // over the four lanes that hold one head
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
MX_DEV float wave_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
MX_DEV float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

template <typename T>
MX_DEV void store4(T* p, f32x4 v) {
  typedef T x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<x4*>(p) = (x4){(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
}

// Partials cross XCDs: written through and read past the caches that are not coherent (sc0 sc1).
MX_DEV void put4(rsrc_t r, uint32_t off, f32x4 v) {
  const float a = v[0], b = v[1], c = v[2], d = v[3];
  __builtin_amdgcn_raw_buffer_store_b128((u32x4){fbits(a), fbits(b), fbits(c), fbits(d)}, r, off, 0, 17);
}
MX_DEV f32x4 get4(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 17));
}

// D: 64, 128 or 256, the head size rounded up. T: type of q, out and the arithmetic. MX8: E4M3 cache.
template <int D, typename T, bool MX8>
__global__ __launch_bounds__(kThreads) void decode_kernel(Args a) {
  typedef typename Vec<T>::x8 x8;
  constexpr int kSteps = D / 32;          // matrix instructions of one score tile
  constexpr int kRuns = D == 256 ? 2 : 1; // runs of kRow elements of V per lane and key
  constexpr int kRow = D == 64 ? 4 : 8;
  constexpr int kOut = D / 16;            // accumulators
  extern __shared__ float lds[];          // merge: [2][head][D + kPad]; join: sums, then [head][chunk] weights
  __shared__ int32_t page_of[kSpan + 1];
  __shared__ float wave_m[kWaves][16], wave_l[kWaves][16];
  __shared__ int is_last;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int unit = blockIdx.x, chunk = blockIdx.y;  // unit: (sequence, cache head, tile of 16 query heads)
  const int ht = unit % a.tiles, hk = (unit / a.tiles) % a.heads, b = unit / (a.tiles * a.heads);
  const int first_head = hk * a.group + 16 * ht, n_heads = min(16, a.group - 16 * ht);

  int hi = min(min(a.lengths[b], a.max_len), (int)min((int64_t)a.cols * a.page_size, (int64_t)INT32_MAX));
  int lo = a.starts ? max(a.starts[b], 0) : 0;
  if (a.window > 0) lo = max(lo, hi - a.window);
  // chunks count from the first attended tile; a row without keys still has chunk 0, which writes it
  const int base = lo & ~(kTile - 1);
  const int active = hi > lo ? (hi - base + a.chunk - 1) / a.chunk : 1;
  if (chunk >= active) return;
  const int from = hi > lo ? base + chunk * a.chunk : 0;
  const int to = hi > lo ? (min(hi, from + a.chunk)) : 0;

  // Query fragments: column c, the elements that this lane's K loads hold.
  x8 qf[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; s++) {
    const int d = MX8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (c < n_heads && d < a.dim)
      w = *reinterpret_cast<const u32x4*>((const T*)a.q + (int64_t)b * a.qt + (int64_t)(first_head + c) * a.qh + d);
    qf[s] = __builtin_bit_cast(x8, w);
  }

  const int64_t head_at = (int64_t)hk * a.head_stride;
  f32x4 acc[kOut];
#pragma unroll
  for (int i = 0; i < kOut; i++) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  for (int span = from; span < to; span += kSpan) {
    const int span_to = min(to, span + kSpan);
    const int page0 = (int)a.page_div.div((uint32_t)span);
    const int n_pages = (int)a.page_div.div((uint32_t)(span_to - 1)) - page0 + 1;
    if (span != from) __syncthreads();
    for (int i = threadIdx.x; i < n_pages; i += kThreads) {
      const int p = a.table[(int64_t)b * a.cols + page0 + i];
      page_of[i] = p >= 0 && p < a.pages ? p : -1;
    }
    __syncthreads();

    for (int t0 = span + wave * kTile; t0 < span_to; t0 += kGrain) {
      // Element offset of a key's row, and whether the key is attended. Others read the cache's first
      // row: memory that is there, and values that are dropped.
      const auto row_of = [&](int key, bool& ok) -> int64_t {
        ok = key >= lo && key < span_to;
        const int at = ok ? key : span;
        const int pi = (int)a.page_div.div((uint32_t)at);
        const int p = page_of[pi - page0];
        ok = ok && p >= 0;
        return ok ? p * a.page_stride + (at - pi * a.page_size) * a.slot_stride + head_at : head_at;
      };
      bool seen_v[8], seen;
      int64_t row_k[2], row_v[8];
#pragma unroll
      for (int h = 0; h < 2; h++) row_k[h] = row_of(t0 + 16 * h + c, seen);
#pragma unroll
      for (int j = 0; j < 8; j++) row_v[j] = row_of(t0 + 16 * (j / 4) + 4 * g + j % 4, seen_v[j]);

      // Loads: all of K, then all of V.
      u32x4 kw[2][MX8 ? D / 64 : kSteps];
      uint32_t ke[2][MX8 ? D / 64 : 1];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if constexpr (MX8) {
#pragma unroll
          for (int s = 0; s < D / 64; s++) {
            const int d = 64 * s + 16 * g;
            const int64_t e = row_k[h] + (d < a.dim ? d : 0);
            kw[h][s] = *reinterpret_cast<const u32x4*>(a.k + e);
            ke[h][s] = a.ks[e >> 5];
          }
        } else {
#pragma unroll
          for (int s = 0; s < kSteps; s++) {
            const int d = 32 * s + 8 * g;
            kw[h][s] = *reinterpret_cast<const u32x4*>(a.k + 2 * (row_k[h] + (d < a.dim ? d : 0)));
          }
        }
      }
      // V: kRow elements from kRow * c (+ 128 per run) of each of the eight keys; past dim: element 0, whose
      // output rows are not written
      u32x4 vw[8][kRuns];
      u32x2 vc[8][kRuns];
      uint32_t ve[8][kRuns];
#pragma unroll
      for (int j = 0; j < 8; j++) {
#pragma unroll
        for (int r = 0; r < kRuns; r++) {
          const int d = 128 * r + kRow * c;
          const int64_t e = row_v[j] + (d < a.dim ? d : 0);
          if constexpr (MX8) {
            if constexpr (kRow == 8) vc[j][r] = *reinterpret_cast<const u32x2*>(a.v + e);
            else vc[j][r] = (u32x2){*reinterpret_cast<const uint32_t*>(a.v + e), 0u};
            ve[j][r] = a.vs[e >> 5];
          } else if constexpr (kRow == 8) {
            vw[j][r] = *reinterpret_cast<const u32x4*>(a.v + 2 * e);
          } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(a.v + 2 * e);
            vw[j][r] = (u32x4){w[0], w[1], 0u, 0u};
          }
        }
      }

      // S^T: keys 4 g + i of half h, head c.
      float x[8];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < kSteps; st++) {
          u32x4 w;
          int d;
          if constexpr (MX8) {
            d = 64 * (st / 2) + 16 * g;
            const u32x4 p = kw[h][st / 2];
            w = widen<T>(st % 2 ? (u32x2){p[2], p[3]} : (u32x2){p[0], p[1]}, ke[h][st / 2]);
          } else {
            d = 32 * st + 8 * g;
            w = kw[h][st];
          }
          if (d >= a.dim) w = (u32x4){0u, 0u, 0u, 0u};
          s = Vec<T>::mfma(__builtin_bit_cast(x8, w), qf[st], s);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) x[4 * h + i] = s[i];
      }
      if (a.softcap > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = a.softcap * kLog2e * tanhf(x[j] * a.scale / a.softcap);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] *= a.scale * kLog2e;
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        x[j] = seen_v[j] ? x[j] : -INFINITY;
        top = fmaxf(top, x[j]);
      }
      top = fmaxf(wave_max(top), m);
      if (__any(top > m)) {
        const float f = __builtin_amdgcn_exp2f(m - finite_or_zero(top));
        l *= f;
#pragma unroll
        for (int i = 0; i < kOut; i++) acc[i] *= f;
        m = top;
      }
      const float ref = finite_or_zero(m) - kShift;
      x8 p;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float e = __builtin_amdgcn_exp2f(x[j] - ref);
        l += e;
        p[j] = (T)e;
      }

      // out^T += V^T P^T
#pragma unroll
      for (int r = 0; r < kRuns; r++) {
        u32x4 w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          if constexpr (MX8) w[j] = widen<T>(vc[j][r], ve[j][r]);
          else w[j] = vw[j][r];
          if (!seen_v[j]) w[j] = (u32x4){0u, 0u, 0u, 0u};  // p = 0 there, and 0 * NaN is NaN
        }
#pragma unroll
        for (int i = 0; i < kRow; i++) {
          const uint32_t sel = i % 2 ? 0x07060302u : 0x05040100u;
          u32x4 f;
#pragma unroll
          for (int j = 0; j < 4; j++) f[j] = __builtin_amdgcn_perm(w[2 * j + 1][i / 2], w[2 * j][i / 2], sel);
          acc[kRow * r + i] = Vec<T>::mfma(__builtin_bit_cast(x8, f), p, acc[kRow * r + i]);
        }
      }
    }
  }

  // Merge the four waves, referred to their common maximum: two put their rows into LDS, the other two add
  // theirs, and the readers below add the remaining two.
  l = wave_sum(l);
  if (g == 0) wave_m[wave][c] = m, wave_l[wave][c] = l;
  __syncthreads();
  constexpr int kLd = D + kPad;
  {
    float top = wave_m[0][c];
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = fmaxf(top, wave_m[w][c]);
    const float f = __builtin_amdgcn_exp2f(m - finite_or_zero(top));
    float* o = lds + ((wave & 1) * n_heads + c) * kLd;
#pragma unroll
    for (int round = 1; round >= 0; round--) {
      if (wave / 2 == round && c < n_heads) {
#pragma unroll
        for (int i = 0; i < kOut; i += 4)
#pragma unroll
          for (int v = 0; v < 4; v++) {
            // neighbouring accumulators hold neighbouring elements
            f32x4* p = reinterpret_cast<f32x4*>(o + 128 * (i / 8) + kRow * (4 * g + v) + i % kRow);
            f32x4 w = {acc[i][v] * f, acc[i + 1][v] * f, acc[i + 2][v] * f, acc[i + 3][v] * f};
            if (round == 0) w += *p;
            *p = w;
          }
      }
      __syncthreads();
    }
  }

  const int quads = a.dim / 4;
  const auto finish = [&](int h, int d, f32x4 o, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    store4<T>((T*)a.out + (int64_t)b * a.ot + (int64_t)(first_head + h) * a.oh + d, o * inv);
  };
  const auto put_lse = [&](int h, float top, float sum) {
    if (a.lse) a.lse[(int64_t)b * a.heads * a.group + first_head + h] = sum == 0.f ? -INFINITY : kLn2 * (top - kShift + __log2f(sum));
  };
  // a head's maximum and sum over the waves
  const auto merged = [&](int h, float& sum) -> float {
    float top = wave_m[0][h];
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = fmaxf(top, wave_m[w][h]);
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) sum += wave_l[w][h] * __builtin_amdgcn_exp2f(wave_m[w][h] - finite_or_zero(top));
    return top;
  };
  const uint32_t o_bytes = (uint32_t)(16 * a.dim * 4), rows_bytes = (uint32_t)a.chunks * o_bytes;
  rsrc_t pr;
  if (active > 1) {  // partials of this unit: [chunk][16][dim] outputs, then [chunk][16] {maximum, sum}
    const int64_t unit_floats = (int64_t)a.chunks * 16 * (a.dim + 2);
    pr = __builtin_amdgcn_make_buffer_rsrc(a.partial + unit * unit_floats, (short)0, (int)(unit_floats * 4), 0x00020000);
  }
  for (int i = threadIdx.x; i < n_heads * quads; i += kThreads) {
    const int h = i / quads, d = 4 * (i - h * quads);
    const f32x4 o = *reinterpret_cast<const f32x4*>(lds + h * kLd + d) +
                    *reinterpret_cast<const f32x4*>(lds + (n_heads + h) * kLd + d);
    float sum;
    const float top = merged(h, sum);
    if (active == 1) {
      finish(h, d, o, sum);
      if (d == 0) put_lse(h, top, sum);
    } else {
      put4(pr, chunk * o_bytes + (uint32_t)(h * a.dim + d) * 4u, o);
      if (d == 0) {
        __builtin_amdgcn_raw_buffer_store_b64((u32x2){fbits(top), fbits(sum)}, pr, rows_bytes + (uint32_t)(chunk * 16 + h) * 8u, 0, 17);
      }
    }
  }
  if (active == 1) return;

  // Join: the unit's last workgroup to arrive adds the chunks' partials in chunk order. Every wave waits for
  // its stores to be acknowledged before the barrier and the counter's increment, so the last one
  // (which takes the counter back to 0) sees them all.
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicInc(&a.counters[unit], (unsigned)(active - 1)) == (unsigned)(active - 1);
  __syncthreads();
  if (!is_last) return;
  // Weights 2^(m_chunk - m) of every head and chunk, and the sums, a wave to four heads.
  float* share = lds;                    // sums of a head's chunk groups, below
  float* weight = lds + 4 * kThreads;    // [head][chunk]
  for (int h = wave; h < n_heads; h += kWaves) {
    float cm[kMaxChunks / 64], cl[kMaxChunks / 64], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 64; i++) {
      const int ch = lane + 64 * i;
      cm[i] = -INFINITY, cl[i] = 0.f;
      if (ch < active) {
        const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(pr, rows_bytes + (uint32_t)(ch * 16 + h) * 8u, 0, 17));
        const uint32_t w0 = w[0], w1 = w[1];
        cm[i] = bitsf(w0), cl[i] = bitsf(w1);
      }
      top = fmaxf(top, cm[i]);
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 64; i++) {
      const float w = __builtin_amdgcn_exp2f(cm[i] - finite_or_zero(top));
      if (lane + 64 * i < active) weight[h * a.chunks + lane + 64 * i] = w;
      sum += w * cl[i];
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) {
      wave_l[0][h] = sum;
      put_lse(h, top, sum);
    }
  }
  __syncthreads();
  // Where a unit has fewer output quads than threads, groups of threads take every n-th chunk.
  const int items = n_heads * quads, split = items < kThreads ? kThreads / items : 1;
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int part = split > 1 ? (int)threadIdx.x / items : 0, i = split > 1 ? (int)threadIdx.x - part * items : i0 + (int)threadIdx.x;
    const bool mine = part < split && i < items;
    const int h = mine ? i / quads : 0, d = mine ? 4 * (i - h * quads) : 0;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if (mine) {
      const uint32_t at = (uint32_t)(h * a.dim + d) * 4u;
      for (int ch = part; ch < active; ch += 8 * split) {
        f32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; u++)
          if (ch + u * split < active) v[u] = get4(pr, (ch + u * split) * o_bytes + at);
#pragma unroll
        for (int u = 0; u < 8; u++)
          if (ch + u * split < active) o += v[u] * weight[h * a.chunks + ch + u * split];
      }
    }
    if (split > 1) {
      if (mine) *reinterpret_cast<f32x4*>(share + 4 * threadIdx.x) = o;
      __syncthreads();
      if (mine && part == 0)
        for (int p = 1; p < split; p++) o += *reinterpret_cast<const f32x4*>(share + 4 * (p * items + i));
    }
    if (mine && part == 0) finish(h, d, o, wave_l[0][h]);
  }
}

// ---- host -----------------------------------------------------------------------------------

// LDS bytes: the merge's rows, or the join's weights and sums.
size_t lds_bytes(int D, int n_heads, int chunks) {
  const size_t merge = (size_t)2 * n_heads * (D + kPad) * 4, weights = (size_t)(n_heads * chunks + 4 * kThreads) * 4;
  return chunks > 1 && weights > merge ? weights : merge;
}

struct Plan {
  int64_t units;
  int chunk, chunks, tiles;
  size_t counter_bytes, bytes;
};

// How the lengths are split: enough workgroups for every CU to hold kPerCu of them, chunks of at
// least kLeast keys (below that the partials' traffic and the join cost what the split gains).
constexpr int kCUs = 256, kPerCu = 8, kLeast = 256;

Plan plan_for(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  Plan p = {};
  const int group = q_heads / c->heads;
  p.tiles = ceil_div(group, 16);
  p.units = (int64_t)seqs * c->heads * p.tiles;
  // positions that a sequence's chunks cover: a window's first tile may start before its first key
  const int64_t span = window > 0 && (int64_t)window + kTile < max_len ? (int64_t)window + kTile : max_len;
  int64_t chunks = ceil_div((int64_t)kCUs * kPerCu, p.units);
  chunks = chunks < kMaxChunks ? chunks : kMaxChunks;
  int64_t chunk = ceil_div(span, chunks);
  chunk = chunk < kLeast ? kLeast : chunk;
  chunk = ceil_div(chunk, (int64_t)kGrain) * kGrain;
  p.chunk = (int)chunk;
  p.chunks = (int)ceil_div(span, chunk);
  p.counter_bytes = ceil_div((size_t)p.units * 4, (size_t)256) * 256;
  // sized by a bound that grows with the span, so that a workspace for max_len serves every window
  const int64_t least = ceil_div((int64_t)kLeast, (int64_t)kGrain) * kGrain;
  const int64_t bound = chunks < ceil_div(span, least) ? chunks : ceil_div(span, least);
  p.bytes = bound > 1 ? p.counter_bytes + (size_t)(p.units * bound) * 16 * (c->dim + 2) * 4 : 0;
  return p;
}

bool sizes_ok(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  return seqs >= 0 && seqs <= MX_MAX_DIM && q_heads >= 1 && q_heads <= MX_MAX_DIM && q_heads % c->heads == 0 && max_len >= 1 &&
         max_len < 1 << 30 && window >= 0 && (int64_t)seqs * q_heads < (int64_t)1 << 24;
}

template <int D, typename T>
void launch(const Args& a, bool mx8, dim3 grid, size_t lds, hipStream_t st) {
  if (mx8) hipLaunchKernelGGL((decode_kernel<D, T, true>), grid, dim3(kThreads), lds, st, a);
  else hipLaunchKernelGGL((decode_kernel<D, T, false>), grid, dim3(kThreads), lds, st, a);
}

template <typename T>
void launch_dim(const Args& a, bool mx8, dim3 grid, hipStream_t st) {
  const int n = a.group < 16 ? a.group : 16;
  if (a.dim <= 64) launch<64, T>(a, mx8, grid, lds_bytes(64, n, a.chunks), st);
  else if (a.dim <= 128) launch<128, T>(a, mx8, grid, lds_bytes(128, n, a.chunks), st);
  else launch<256, T>(a, mx8, grid, lds_bytes(256, n, a.chunks), st);
}

}  // namespace

extern "C" size_t mxattn_decode_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window) {
  if (!cache || check_geometry(cache) || !sizes_ok(cache, seqs, q_heads, max_len, window) || seqs == 0) return 0;
  return plan_for(cache, seqs, q_heads, max_len, window).bytes;
}

extern "C" int mxattn_decode_run(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse,
                                 const mxkv_table* table, const int32_t* lengths, const int32_t* starts, int max_len,
                                 const mxattn_opts* opts, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !q || !out || !table || !opts) return MX_ERR_NULL;
  if (f != MX_F16 && f != MX_BF16) return MX_ERR_FORMAT;
  if (int s = check_cache(cache)) return s;
  const bool mx8 = cache->fmt == MX_E4M3;
  if (!mx8 && cache->fmt != f) return MX_ERR_FORMAT;
  if (int s = check_table(table)) return s;
  if (!sizes_ok(cache, table->seqs, q->heads, max_len, opts->window) || q->heads != out->heads) return MX_ERR_SHAPE;
  if (!__builtin_isfinite(opts->scale) || !__builtin_isfinite(opts->softcap) || opts->softcap < 0.f) return MX_ERR_SHAPE;
  if (table->seqs == 0) return MX_OK;
  if (!lengths) return MX_ERR_NULL;
  if (int s = check_heads(q, 2)) return s;
  if (int s = check_heads(out, 2)) return s;
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  Plan p = plan_for(cache, table->seqs, q->heads, max_len, opts->window);
  if (!workspace || workspace_bytes < p.bytes) {  // one workgroup per unit takes the whole length
    p.chunk = 1 << 30;
    p.chunks = 1;
  }
  Args a = {};
  a.k = (const uint8_t*)cache->k, a.v = (const uint8_t*)cache->v;
  a.ks = (const uint8_t*)cache->ks, a.vs = (const uint8_t*)cache->vs;
  a.q = q->data, a.qt = q->token_stride, a.qh = q->head_stride;
  a.out = out->data, a.ot = out->token_stride, a.oh = out->head_stride;
  a.lse = lse;
  a.table = table->pages, a.cols = table->cols, a.lengths = lengths, a.starts = starts;
  if (p.chunks > 1) {
    a.counters = (uint32_t*)workspace;
    a.partial = (float*)((uint8_t*)workspace + p.counter_bytes);
  }
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.heads = cache->heads, a.group = q->heads / cache->heads, a.tiles = p.tiles, a.dim = cache->dim;
  a.pages = cache->pages, a.page_size = cache->page_size, a.max_len = max_len, a.window = opts->window;
  a.chunk = p.chunk, a.chunks = p.chunks;
  a.scale = opts->scale, a.softcap = opts->softcap;
  a.page_div = FastDiv((uint32_t)cache->page_size);
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  const dim3 grid((unsigned)p.units, (unsigned)p.chunks);
  if (f == MX_F16) launch_dim<_Float16>(a, mx8, grid, st);
  else launch_dim<__bf16>(a, mx8, grid, st);
  return sync_check(launch_status(), st);
}
