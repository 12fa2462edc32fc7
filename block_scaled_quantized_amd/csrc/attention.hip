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
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 32;                // keys of a wave's tile
constexpr int kGrain = kTile * kWaves;   // keys that the workgroup's waves take in turn: the unit of work
constexpr int kLeast = 2;                // grains: no unit is cut within this of its ends
constexpr int kFan = 128, kGroup = 64;   // partials that one workgroup joins; groups of more
constexpr int kDeep = 16;                // partials that a joining thread has on their way
constexpr int kPad = 4;                  // floats that keep the heads' rows of the merge on different banks
constexpr int kFar = 1 << 30;            // a byte offset past every buffer: loads give 0
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
  int seqs, heads, group, tiles, dim, cols, pages, page_size, max_len, window, wgs;
  bool split;
  float scale, softcap;
  FastDiv page_div;
};

template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  typedef f16x8 x8;
  // Probabilities are rounded to T for the matrix cores. p = 2^(x - m) is at most 1; binary16 would lose
  // those under 2^-24, which can matter in number in a long row, so they are scaled by 2^15 (which
  // cancels in the division by their sum). bfloat16 has the range.
  static constexpr float kShift = 15.0f;
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static MX_DEV uint32_t from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HI));
  }
};
template <>
struct Vec<__bf16> {
  typedef bf16x8 x8;
  static constexpr float kShift = 0.0f;
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static MX_DEV uint32_t from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
  }
};

// Eight E4M3 codes times 2^(e - 127) as eight 16-bit values: the conversion reads the scale's exponent bits
// as an E8M0 number, 0 as 2^-127 and 255 as NaN.
template <typename T>
MX_DEV u32x4 widen(u32x2 c, uint32_t e) {
  const float s = bitsf(e << 23);
  return (u32x4){Vec<T>::template from_e4m3<false>(c[0], s), Vec<T>::template from_e4m3<true>(c[0], s),
                 Vec<T>::template from_e4m3<false>(c[1], s), Vec<T>::template from_e4m3<true>(c[1], s)};
}

// Over the four lanes that hold one head (lane % 16): exchanges of rows of 16 and of halves of the wave.
MX_DEV float wave_max(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(fbits(x), fbits(x), false, false);
  x = fmaxf(bitsf(r[0]), bitsf(r[1]));
  r = __builtin_amdgcn_permlane32_swap(fbits(x), fbits(x), false, false);
  return fmaxf(bitsf(r[0]), bitsf(r[1]));
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

// One sequence's attended positions lo .. hi - 1, counted in grains from the tile that holds lo. A row
// without positions still has a grain, whose workgroup writes it.
struct Row {
  int lo, hi, base, grains;
};

MX_DEV Row row_of(const Args& a, int b) {
  Row r;
  r.hi = max(0, min(min(a.lengths[b], a.max_len), (int)min((int64_t)a.cols * a.page_size, (int64_t)INT32_MAX)));
  r.lo = a.starts ? max(a.starts[b], 0) : 0;
  if (a.window > 0) r.lo = max(r.lo, r.hi - a.window);
  if (r.lo >= r.hi) r.lo = r.hi = 0;
  r.base = r.lo & ~(kTile - 1);
  r.grains = max(1, ceil_div(r.hi - r.base, kGrain));
  return r;
}

MX_DEV int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
MX_DEV int64_t uniform64(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}
MX_DEV uint64_t quotient(uint64_t n, uint64_t d) { return (n | d) >> 32 ? n / d : (uint32_t)n / (uint32_t)d; }

// A place in the list of all units' grains: sequence, unit within it, grain; `at` numbers the sequence's
// first grain.
struct Place {
  int b, unit, grain;
  int64_t at;
};

// This workgroup's share of the grains, from..to, of equal size but for the cuts' distance from the
// units' ends. Every workgroup sums up the lengths by itself: a handful of loads that all of them find in
// the caches, where a launch that planned would cost its own latency.
MX_DEV int64_t share_of(const Args& a, Place& from, Place& to) {
  __shared__ uint32_t wave_total[kWaves];
  __shared__ Place place[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, units = a.heads * a.tiles;
  const auto scan = [&](uint32_t n, uint32_t& total) -> uint32_t {  // sum of the lower threads' n
    uint32_t s = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_up(s, d);
      s += lane >= d ? o : 0u;
    }
    __syncthreads();
    if (lane == 63) wave_total[wave] = s;
    __syncthreads();
    uint32_t before = 0u;
    total = 0u;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const uint32_t t = wave_total[w];
      before += w < wave ? t : 0u;
      total += t;
    }
    return before + s - n;
  };
  const auto grains_of = [&](int b) -> uint32_t { return b < a.seqs ? (uint32_t)row_of(a, b).grains : 0u; };
  int64_t all = 0;
  uint32_t total, n = grains_of(threadIdx.x), before = scan(n, total);
  all = total;
  for (int b = kThreads; b < a.seqs; b += kThreads) {
    scan(grains_of(b + threadIdx.x), total);
    all += total;
  }
  const int64_t per = max((int64_t)kLeast, (int64_t)quotient((uint64_t)(all * units + a.wgs - 1), (uint64_t)a.wgs));
  const int64_t cut[2] = {blockIdx.x * per, (blockIdx.x + 1) * per};
  if (threadIdx.x < 2) place[threadIdx.x] = Place{a.seqs, 0, 0, all * units};
  int64_t sum = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    if (a.seqs > kThreads) {
      n = grains_of(b);
      before = scan(n, total);
    } else {
      __syncthreads();
    }
    const int64_t at = (sum + before) * units;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if (n == 0u || cut[i] < at || cut[i] >= at + (int64_t)n * units) continue;
      Place p = {b, (int)quotient((uint64_t)(cut[i] - at), n), 0, at};
      p.grain = (int)(cut[i] - at - (int64_t)p.unit * n);
      if (p.grain < kLeast) p.grain = 0;
      else if ((int)n - p.grain < kLeast) p.grain = 0, p.unit++;
      if (p.unit == units) p = Place{b + 1, 0, 0, at + (int64_t)n * units};
      place[i] = p;
    }
    sum += total;
  }
  __syncthreads();
  from = place[0], to = place[1];
  from = Place{uniform(from.b), uniform(from.unit), uniform(from.grain), uniform64(from.at)};
  to = Place{uniform(to.b), uniform(to.unit), uniform(to.grain), uniform64(to.at)};
  return uniform64(per);
}

// D: 64, 128 or 256, the head size rounded up. T: type of q, out and the arithmetic. MX8: E4M3 cache.
// PAGED16: page_size % 16 == 0, so that the 16 keys of half a tile lie in one page: their place is a
// buffer descriptor in scalar registers, whose size also turns keys past the end, missing pages and
// elements past dim into zeros. Other page sizes look every key's page up in the lanes.
template <int D, typename T, bool MX8, bool PAGED16>
__global__ __launch_bounds__(kThreads) void decode_kernel(Args a) {
  typedef typename Vec<T>::x8 x8;
  constexpr float kShift = Vec<T>::kShift;
  constexpr int kSteps = D / 32;          // matrix instructions of one score tile
  constexpr int kLoads = MX8 ? D / 64 : kSteps;  // 16-byte loads of a key's row
  constexpr int kRuns = D == 256 ? 2 : 1; // runs of kRow elements of V per lane and key
  constexpr int kRow = D == 64 ? 4 : 8;
  constexpr int kOut = D / 16;            // accumulators
  constexpr int kSize = MX8 ? 1 : 2;      // bytes of an element
  constexpr int kBlock = 32;              // tiles of a wave whose pages it looks up at a time
  extern __shared__ float lds[];          // merge: [kWaves / 2][head][D + kPad]; join: sums, then [head][kFan] weights
  __shared__ float wave_m[kWaves][16], wave_l[kWaves][16];
  __shared__ int is_last;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  const int units = a.heads * a.tiles, quads = a.dim / 4;
  Place at, end;
  int64_t per = 1;
  if (a.split) {
    per = share_of(a, at, end);
  } else {
    at = Place{(int)blockIdx.x / units, (int)blockIdx.x % units, 0, 0};
    end = at.unit + 1 < units ? Place{at.b, at.unit + 1, 0, 0} : Place{at.b + 1, 0, 0, 0};
  }

  // Byte offsets of this lane's loads within 16 keys' rows.
  const int slot_bytes = (int)a.slot_stride * kSize, slot_scales = (int)a.slot_stride / 32;
  int k_at[kLoads], v_at[4][kRuns];
#pragma unroll
  for (int s = 0; s < kLoads; s++) {
    const int d = MX8 ? 64 * s + 16 * g : 32 * s + 8 * g;
    k_at[s] = d < a.dim ? c * slot_bytes + d * kSize : kFar;
  }
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int r = 0; r < kRuns; r++) {
      const int d = 128 * r + kRow * c;
      v_at[j][r] = d < a.dim ? (4 * g + j) * slot_bytes + d * kSize : kFar;
    }

  while (at.b < end.b || (at.b == end.b && (at.unit < end.unit || (at.unit == end.unit && at.grain < end.grain)))) {
    const int b = at.b;
    Row row = row_of(a, b);
    row = Row{uniform(row.lo), uniform(row.hi), uniform(row.base), uniform(row.grains)};
    const int ht = at.unit % a.tiles, hk = at.unit / a.tiles;
    const int first_head = hk * a.group + 16 * ht, n_heads = min(16, a.group - 16 * ht);
    const int stop = b == end.b && at.unit == end.unit ? end.grain : row.grains;
    const int from = row.base + at.grain * kGrain, to = min(row.hi, row.base + stop * kGrain), lo = row.lo;
    const int64_t head_at = (int64_t)hk * a.head_stride;
    const int32_t* table = a.table + (int64_t)b * a.cols;

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

    f32x4 acc[kOut];
#pragma unroll
    for (int i = 0; i < kOut; i++) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    u32x4 kw[2][kLoads], vw[8][kRuns];
    u32x2 vc[8][kRuns];
    uint32_t ke[2][kLoads], ve[8][kRuns];
    for (int first = from + wave * kTile; first < to; first += kBlock * kGrain) {
      const int upto = min(to, first + kBlock * kGrain);  // the next tiles of this block end here
      const int n_tiles = ceil_div(upto - first, kGrain);

      // PAGED16: lane i holds the element offset of half i % 2 of tile i / 2 (negative: no page).
      int off_lo = 0, off_hi = -1;
      // else: lane i holds the i-th page from the tile's first one, here and in the next tile
      int page = -1, page_next = -1;
      const auto lookup = [&](int index) -> int {
        const int p = table[index];
        return p >= 0 && p < a.pages ? p : -1;
      };
      const auto fetch_pages = [&](int t) -> int {  // of the tile at key t
        const int i = (int)a.page_div.div((uint32_t)min(t, to - 1)) + lane, last = (int)a.page_div.div((uint32_t)(to - 1));
        return i <= last && lane <= kTile ? lookup(i) : -1;
      };
      if constexpr (PAGED16) {
        const int key = first + (lane >> 1) * kGrain + (lane & 1) * 16;
        if (key < upto) {
          const int i = (int)a.page_div.div((uint32_t)key), p = lookup(i);
          const int64_t off = p * a.page_stride + (key - i * a.page_size) * a.slot_stride + head_at;
          off_lo = (int)off, off_hi = p < 0 ? -1 : (int)(off >> 32);
        }
      } else {
        page = fetch_pages(first);
      }

      int rows[2] = {0, 0};           // PAGED16: keys of each half of the tile whose K is loaded
      int64_t off[2] = {0, 0};
      uint32_t seen = 0u, seen_now;   // bit 4 h + i: key 16 h + 4 g + i of the tile is attended (not PAGED16)
      const auto place_tile = [&](int it) {
        if constexpr (PAGED16) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const int hi = __builtin_amdgcn_readlane(off_hi, 2 * it + h), lw = __builtin_amdgcn_readlane(off_lo, 2 * it + h);
            off[h] = (int64_t)((uint64_t)(uint32_t)max(hi, 0) << 32 | (uint32_t)lw);
            rows[h] = hi < 0 ? 0 : min(16, max(0, upto - (first + it * kGrain + 16 * h)));
          }
        }
      };
      // Element offset of a key's row, and whether it is attended; others read the cache's first row, memory
      // that is there and values that are dropped.
      const auto row_at = [&](int t, int key, bool& ok) -> int64_t {
        ok = key >= lo && key < upto;
        const int at = ok ? key : t, i = (int)a.page_div.div((uint32_t)at);
        const int p = __shfl(page, i - (int)a.page_div.div((uint32_t)t));
        ok = ok && p >= 0;
        return ok ? p * a.page_stride + (at - i * a.page_size) * a.slot_stride + head_at : head_at;
      };
      const auto load_k = [&](int it) {
        if constexpr (PAGED16) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)(a.k + off[h] * kSize), (short)0, rows[h] * slot_bytes, 0x00020000);
#pragma unroll
            for (int s = 0; s < kLoads; s++) kw[h][s] = __builtin_amdgcn_raw_buffer_load_b128(r, k_at[s], 0, 0);
            if constexpr (MX8) {
              const rsrc_t e = __builtin_amdgcn_make_buffer_rsrc((void*)(a.ks + (off[h] >> 5)), (short)0, rows[h] * slot_scales, 0x00020000);
#pragma unroll
              for (int s = 0; s < kLoads; s++) ke[h][s] = __builtin_amdgcn_raw_buffer_load_b8(e, k_at[s] >> 5, 0, 0);
            }
          }
        } else {
          const int t = min(first + it * kGrain, to - 1);
#pragma unroll
          for (int h = 0; h < 2; h++) {
            bool ok;
            const int64_t o = row_at(t, first + it * kGrain + 16 * h + c, ok);
#pragma unroll
            for (int s = 0; s < kLoads; s++) {
              const int d = MX8 ? 64 * s + 16 * g : 32 * s + 8 * g;
              const int64_t e = o + (d < a.dim ? d : 0);
              kw[h][s] = *reinterpret_cast<const u32x4*>(a.k + e * kSize);
              if constexpr (MX8) ke[h][s] = a.ks[e >> 5];
            }
          }
        }
      };
      // V: kRow elements from kRow * c (+ 128 per run) of each of the eight keys; past dim: zeros or element
      // 0, whose output rows are not written
      const auto load_v = [&](int it) {
        const int t = min(first + it * kGrain, to - 1);
        seen = 0u;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          rsrc_t rv, re;
          if constexpr (PAGED16) {
            rv = __builtin_amdgcn_make_buffer_rsrc((void*)(a.v + off[h] * kSize), (short)0, rows[h] * slot_bytes, 0x00020000);
            if constexpr (MX8) re = __builtin_amdgcn_make_buffer_rsrc((void*)(a.vs + (off[h] >> 5)), (short)0, rows[h] * slot_scales, 0x00020000);
          }
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int j = 4 * h + i;
            bool ok = false;
            int64_t o = 0;
            if constexpr (!PAGED16) {
              o = row_at(t, first + it * kGrain + 16 * h + 4 * g + i, ok);
              seen |= ok ? 1u << j : 0u;
            }
#pragma unroll
            for (int r = 0; r < kRuns; r++) {
              const int d = 128 * r + kRow * c;
              const int64_t e = o + (d < a.dim ? d : 0);
              if constexpr (PAGED16 && MX8) {
                if constexpr (kRow == 8) vc[j][r] = __builtin_amdgcn_raw_buffer_load_b64(rv, v_at[i][r], 0, 0);
                else vc[j][r] = (u32x2){__builtin_amdgcn_raw_buffer_load_b32(rv, v_at[i][r], 0, 0), 0u};
                ve[j][r] = __builtin_amdgcn_raw_buffer_load_b8(re, v_at[i][r] >> 5, 0, 0);
              } else if constexpr (PAGED16) {
                if constexpr (kRow == 8) {
                  vw[j][r] = __builtin_amdgcn_raw_buffer_load_b128(rv, v_at[i][r], 0, 0);
                } else {
                  const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rv, v_at[i][r], 0, 0);
                  vw[j][r] = (u32x4){w[0], w[1], 0u, 0u};
                }
              } else if constexpr (MX8) {
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
        }
      };

      place_tile(0);
      load_k(0);
      load_v(0);
      for (int it = 0; it < n_tiles; it++) {
        const int t = first + it * kGrain;
        bool all_seen, head_masked = false;  // every key is attended; keys before lo have to be cleared in V
        if constexpr (PAGED16) {
          all_seen = rows[0] == 16 && rows[1] == 16 && t >= lo;
          head_masked = t < lo;
          seen_now = 0xFFu;
          if (!all_seen) {
            seen_now = 0u;
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const int i = 4 * g + j % 4;
              seen_now |= i < rows[j / 4] && t + 16 * (j / 4) + i >= lo ? 1u << j : 0u;
            }
          }
        } else {
          seen_now = seen;
          all_seen = __all(seen == 0xFFu);
          head_masked = !all_seen;
          page_next = fetch_pages(first + (it + 1) * kGrain);
        }

        // S^T: keys 4 g + i of half h, head c.
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = 0; st < kSteps; st++) {
            u32x4 w;
            if constexpr (MX8) {
              const u32x4 p = kw[h][st / 2];
              w = widen<T>(st % 2 ? (u32x2){p[2], p[3]} : (u32x2){p[0], p[1]}, ke[h][st / 2]);
            } else {
              w = kw[h][st];
            }
            if constexpr (!PAGED16) {
              if ((MX8 ? 64 * (st / 2) + 16 * g : 32 * st + 8 * g) >= a.dim) w = (u32x4){0u, 0u, 0u, 0u};
            }
            s = Vec<T>::mfma(__builtin_bit_cast(x8, w), qf[st], s);
          }
#pragma unroll
          for (int i = 0; i < 4; i++) x[4 * h + i] = s[i];
        }
        page = page_next;
        place_tile(it + 1);
        load_k(it + 1);
        if (a.softcap > 0.f) {
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] = a.softcap * kLog2e * tanhf(x[j] * a.scale / a.softcap);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] *= a.scale * kLog2e;
        }
        if (!all_seen) {
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] = seen_now >> j & 1u ? x[j] : -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 8; j++) top = fmaxf(top, x[j]);
        if (__any(top > m)) {  // seldom after the first tiles
          top = fmaxf(wave_max(top), m);
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
          }
          if (head_masked) {  // p = 0 there, and 0 * NaN is NaN
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (!(seen_now >> j & 1u)) w[j] = (u32x4){0u, 0u, 0u, 0u};
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
        load_v(it + 1);
      }
    }

    // Merge the waves, referred to their common maximum: half of them put their rows into LDS, the others add
    // theirs, and the readers below add the remaining ones.
    l = wave_sum(l);
    if (g == 0) wave_m[wave][c] = m, wave_l[wave][c] = l;
    __syncthreads();
    constexpr int kLd = D + kPad, kHalf = kWaves / 2;
    {
      float top = wave_m[0][c];
#pragma unroll
      for (int w = 1; w < kWaves; w++) top = fmaxf(top, wave_m[w][c]);
      const float f = __builtin_amdgcn_exp2f(m - finite_or_zero(top));
      float* o = lds + ((wave % kHalf) * n_heads + c) * kLd;
#pragma unroll
      for (int round = 1; round >= 0; round--) {
        if (wave / kHalf == round && c < n_heads) {
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
    const bool whole = at.grain == 0 && stop == row.grains;
    // Partials, one for a share that begins within a unit and one for a unit that ends past the share:
    // [16][dim] outputs, then [16] {maximum, sum}.
    const uint32_t rows_at = (uint32_t)(16 * a.dim * 4), slot_size = rows_at + 16 * 8;
    rsrc_t pr;
    if (!whole) pr = __builtin_amdgcn_make_buffer_rsrc(a.partial, (short)0, (int)(2 * a.wgs * slot_size), 0x00020000);
    const uint32_t mine_at = (2 * blockIdx.x + (at.grain == 0 ? 1u : 0u)) * slot_size;
    for (int i = threadIdx.x; i < n_heads * quads; i += kThreads) {
      const int h = i / quads, d = 4 * (i - h * quads);
      f32x4 o = *reinterpret_cast<const f32x4*>(lds + h * kLd + d);
#pragma unroll
      for (int w = 1; w < kHalf; w++) o += *reinterpret_cast<const f32x4*>(lds + (w * n_heads + h) * kLd + d);
      float sum;
      const float top = merged(h, sum);
      if (whole) {
        finish(h, d, o, sum);
        if (d == 0) put_lse(h, top, sum);
      } else {
        put4(pr, mine_at + (uint32_t)(h * a.dim + d) * 4u, o);
        if (d == 0) __builtin_amdgcn_raw_buffer_store_b64((u32x2){fbits(top), fbits(sum)}, pr, mine_at + rows_at + h * 8, 0, 17);
      }
    }

    // Join: the workgroup that arrives last adds the unit's partials in their order, of more than kFan in two steps:
    // groups of kGroup, then the groups. Every wave waits for its stores to be acknowledged before the
    // barrier and the counter's increment, so the last one (which takes the counter back to 0) sees all.
    // A partial's counter is its group's first one's.
    if (!whole) {
      const int64_t u0 = at.at + (int64_t)at.unit * row.grains;
      const int first = (int)quotient((uint64_t)(u0 + kLeast + per - 1), (uint64_t)per) - 1;  // the unit's first workgroup
      const int members = (int)quotient((uint64_t)(u0 + row.grains - kLeast), (uint64_t)per) - first + 1;
      const auto slot_of = [&](int i) -> int { return 2 * (first + i) + (i == 0 ? 1 : 0); };
      const int groups = members <= kFan ? 1 : ceil_div(members, kGroup), group = groups == 1 ? 0 : ((int)blockIdx.x - first) / kGroup;
      for (int level = 0; level < 2; level++) {
        // the partials start, start + step, ... of this step, and whether their sum is the result
        const int start = level == 0 ? group * kGroup : 0, step = level == 0 ? 1 : kGroup;
        const int n = level == 1 ? groups : groups == 1 ? members : min(kGroup, members - start);
        const bool result = level == 1 || groups == 1;
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
        if (threadIdx.x == 0)
          is_last = atomicInc(a.counters + (level == 1 ? 2 * a.wgs + first : slot_of(start)), (unsigned)(n - 1)) == (unsigned)(n - 1);
        __syncthreads();
        if (!is_last) break;
        // Weights 2^(m_i - m) of every head and partial, and the sums, a wave to a head at a time.
        float* share = lds;                    // sums of a head's runs of partials, below
        float* weight = lds + 4 * kThreads;    // [head][kFan]
        for (int h = wave; h < n_heads; h += kWaves) {
          float cm[kFan / 64], cl[kFan / 64], top = -INFINITY;
#pragma unroll
          for (int i = 0; i < kFan / 64; i++) {
            const int ch = lane + 64 * i;
            cm[i] = -INFINITY, cl[i] = 0.f;
            if (ch < n) {
              const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                  pr, slot_of(start + ch * step) * slot_size + rows_at + h * 8, 0, 17));
              const uint32_t w0 = w[0], w1 = w[1];
              cm[i] = bitsf(w0), cl[i] = bitsf(w1);
            }
            top = fmaxf(top, cm[i]);
          }
#pragma unroll
          for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < kFan / 64; i++) {
            const float w = __builtin_amdgcn_exp2f(cm[i] - finite_or_zero(top));
            weight[h * kFan + lane + 64 * i] = lane + 64 * i < n ? w : 0.f;
            sum += w * cl[i];
          }
#pragma unroll
          for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
          if (lane == 0) {
            wave_l[0][h] = sum, wave_m[0][h] = top;
            if (result) put_lse(h, top, sum);
          }
        }
        __syncthreads();
        // Where a unit has fewer output quads than threads, groups of threads take every n-th partial.
        const int items = n_heads * quads, split = items < kThreads ? kThreads / items : 1;
        for (int i0 = 0; i0 < items; i0 += kThreads) {
          const int part = split > 1 ? (int)threadIdx.x / items : 0, i = split > 1 ? (int)threadIdx.x - part * items : i0 + (int)threadIdx.x;
          const bool mine = part < split && i < items;
          const int h = mine ? i / quads : 0, d = mine ? 4 * (i - h * quads) : 0;
          f32x4 o = {0.f, 0.f, 0.f, 0.f};
          if (mine) {
            const uint32_t from_row = (uint32_t)(h * a.dim + d) * 4u;
            for (int ch = part; ch < n; ch += kDeep * split) {
              f32x4 v[kDeep];
#pragma unroll
              for (int u = 0; u < kDeep; u++)
                v[u] = get4(pr, ch + u * split < n ? slot_of(start + (ch + u * split) * step) * slot_size + from_row : (uint32_t)kFar * 2u);
#pragma unroll
              for (int u = 0; u < kDeep; u++) o += v[u] * weight[h * kFan + min(ch + u * split, kFan - 1)];
            }
          }
          if (split > 1) {
            if (mine) *reinterpret_cast<f32x4*>(share + 4 * threadIdx.x) = o;
            __syncthreads();
            if (mine && part == 0)
              for (int p = 1; p < split; p++) o += *reinterpret_cast<const f32x4*>(share + 4 * (p * items + i));
          }
          if (mine && part == 0) {
            if (result) finish(h, d, o, wave_l[0][h]);
            else put4(pr, slot_of(start) * slot_size + (uint32_t)(h * a.dim + d) * 4u, o);
          }
        }
        if (result) break;
        if (threadIdx.x < n_heads)
          __builtin_amdgcn_raw_buffer_store_b64((u32x2){fbits(wave_m[0][threadIdx.x]), fbits(wave_l[0][threadIdx.x])}, pr,
                                                slot_of(start) * slot_size + rows_at + threadIdx.x * 8, 0, 17);
      }
    }
    __syncthreads();  // the next unit's merge uses the same memory

    at.grain = 0;
    if (stop < row.grains) break;
    if (++at.unit == units) at = Place{b + 1, 0, 0, at.at + (int64_t)row.grains * units};
  }
}

// ---- host -----------------------------------------------------------------------------------

// LDS bytes: the merge's rows, or the join's weights and sums.
size_t lds_bytes(int D, int n_heads, bool split) {
  const size_t merge = (size_t)(kWaves / 2) * n_heads * (D + kPad) * 4, weights = (size_t)(n_heads * kFan + 4 * kThreads) * 4;
  return split && weights > merge ? weights : merge;
}

struct Plan {
  int64_t units;
  int tiles, wgs;  // wgs: workgroups that share the grains; 0: no unit is worth splitting
  size_t counter_bytes, bytes;
};

// The lengths are known on the device only. The grid is one round of workgroups, as many as the CUs hold at
// a time, or fewer where max_len bounds the grains.
constexpr int kCUs = 256;
int per_cu(int dim) { return dim <= 64 ? 4 : dim <= 128 ? 2 : 1; }

Plan plan_for(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  Plan p = {};
  p.tiles = ceil_div(q_heads / c->heads, 16);
  p.units = (int64_t)seqs * c->heads * p.tiles;
  // positions from a sequence's first tile: a window may start within it
  const int64_t span = window > 0 && (int64_t)window + kTile < max_len ? (int64_t)window + kTile : max_len;
  const int64_t grains = ceil_div(span, (int64_t)kGrain), wgs = ceil_div(p.units * grains, (int64_t)kLeast);
  if (grains < 2 * kLeast) return p;
  p.wgs = (int)(wgs < kCUs * per_cu(c->dim) ? wgs : kCUs * per_cu(c->dim));
  const size_t counters = (size_t)(p.units > 3 * p.wgs ? p.units : 3 * p.wgs);
  p.counter_bytes = ceil_div(counters * 4, (size_t)256) * 256;
  p.bytes = p.counter_bytes + (size_t)(2 * p.wgs) * 16 * (c->dim + 2) * 4;
  return p;
}

bool sizes_ok(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  return seqs >= 0 && seqs <= MX_MAX_DIM && q_heads >= 1 && q_heads <= MX_MAX_DIM && q_heads % c->heads == 0 && max_len >= 1 &&
         max_len < 1 << 30 && window >= 0 && (int64_t)seqs * q_heads < (int64_t)1 << 24;
}

template <int D, typename T, bool MX8>
void launch(const Args& a, dim3 grid, hipStream_t st) {
  const size_t lds = lds_bytes(D, a.group < 16 ? a.group : 16, a.split);
  if (a.page_size % 16 == 0) hipLaunchKernelGGL((decode_kernel<D, T, MX8, true>), grid, dim3(kThreads), lds, st, a);
  else hipLaunchKernelGGL((decode_kernel<D, T, MX8, false>), grid, dim3(kThreads), lds, st, a);
}

template <typename T, bool MX8>
void launch_dim(const Args& a, dim3 grid, hipStream_t st) {
  if (a.dim <= 64) launch<64, T, MX8>(a, grid, st);
  else if (a.dim <= 128) launch<128, T, MX8>(a, grid, st);
  else launch<256, T, MX8>(a, grid, st);
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
  const Plan p = plan_for(cache, table->seqs, q->heads, max_len, opts->window);
  Args a = {};
  a.k = (const uint8_t*)cache->k, a.v = (const uint8_t*)cache->v;
  a.ks = (const uint8_t*)cache->ks, a.vs = (const uint8_t*)cache->vs;
  a.q = q->data, a.qt = q->token_stride, a.qh = q->head_stride;
  a.out = out->data, a.ot = out->token_stride, a.oh = out->head_stride;
  a.lse = lse;
  a.table = table->pages, a.cols = table->cols, a.lengths = lengths, a.starts = starts;
  a.split = p.wgs > 0 && workspace && workspace_bytes >= p.bytes;  // else a workgroup takes a whole unit
  a.wgs = p.wgs;
  if (a.split) {
    a.counters = (uint32_t*)workspace;
    a.partial = (float*)((uint8_t*)workspace + p.counter_bytes);
  }
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.seqs = table->seqs, a.heads = cache->heads, a.group = q->heads / cache->heads, a.tiles = p.tiles, a.dim = cache->dim;
  a.pages = cache->pages, a.page_size = cache->page_size, a.max_len = max_len, a.window = opts->window;
  a.scale = opts->scale, a.softcap = opts->softcap;
  a.page_div = FastDiv((uint32_t)cache->page_size);
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  const dim3 grid((unsigned)(a.split ? p.wgs : p.units));
  if (f == MX_F16 && mx8) launch_dim<_Float16, true>(a, grid, st);
  else if (f == MX_F16) launch_dim<_Float16, false>(a, grid, st);
  else if (mx8) launch_dim<__bf16, true>(a, grid, st);
  else launch_dim<__bf16, false>(a, grid, st);
  return sync_check(launch_status(), st);
}
