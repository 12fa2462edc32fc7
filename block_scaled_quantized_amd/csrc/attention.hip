// attention.hip -- attention of one new token per sequence over a paged key-value cache.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = e^(s_j - m), s_j = scale q.k_j, in one pass over the cache: a
// wave keeps the running maximum m, sum and output of its keys and rescales them where m grows. The
// cache is read once and bounds the time (each key-value pair of bytes meets the few query heads that
// share it), so everything else serves its loads: 16 query heads of one cache head are the columns of a
// 16x16x32 matrix instruction (columns without a head idle: the matrix cores have at least eight times
// the rate that the memory asks of them), K and V go from global memory to registers with no LDS
// between, up to two tiles ahead, and the keys of long rows are shared evenly among one round of workgroups.
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
//
// Measured, us of a call among others on changing inputs (reads of a large array by a row maximum: 6.4 TB/s): 64 x 16384
// keys x 8 x 128 E4M3, 2.2 GB, 345 us, 6.4 TB/s; 131072 keys x 8 x 128 fp16, 537 MB, 86 us, 6.2 TB/s; the same bytes
// over 16 x 8192 keys x 4 x 256, 93 us. Where a call's work is a few grains per workgroup, its time is the chain of dependent memory
// latencies (lengths and pages, keys, and for cut units partials, counter, partials) and the instructions that come from
// memory: 5.1 us for rows of a few keys, 8.7 to 10.6 us for 8 x 500 keys of 128 (a kernel of one store: 3.6 us).
// Pairs of times below compare two choices side by side in graphs of calls, as they were when the choice was made: a call
// takes up to 2 us more there, and boxes differ by a tenth.
#include <algorithm>

#include "attention.h"

using namespace mx;

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 32;                // keys of a wave's tile
constexpr int kGrain = kTile * kWaves;   // keys that the workgroup's waves take in turn: the unit of work
// Partials that one workgroup joins, and the groups of more. Small numbers make short code and spread long joins (8
// rows of up to 47091 keys of one head: 25.8 us with 128 and 64, 20.1 with 32 and 16; 12 x 5 rows: 13.6 and 12.9).
constexpr int kFan = 32, kGroup = 16;
constexpr int kDeep = 8;                 // partials that a joining thread has on their way
constexpr int kPad = 4;                  // floats that keep the heads' rows of the merge on different banks
// Keys and values are read once: marked non-temporal, they leave the L2 to the program, whose prologue and
// joins otherwise wait for their instructions (131072 x 8 x 128 fp16: 114 -> 103 us).
constexpr int kStream = 2;
constexpr int kFar = 1 << 30;            // a byte offset past every buffer: loads give 0

struct Args {
  const uint8_t *k, *v, *ks, *vs;
  const void* q;
  void* out;
  float* lse;
  const int32_t *table, *lengths, *starts;
  uint32_t* counters;
  float* partial;
  int64_t qt, qh, ot, oh, page_stride, head_stride, slot_stride;
  int seqs, heads, group, tiles, dim, cols, pages, page_size, max_len, max_keys, window, wgs;
  float scale, softcap;
  FastDiv page_div, units_div, tiles_div, wgs_div, quads_div;  // units: of one sequence
  Prefix prefix;  // shared positions' results, which a row's own are added to
};

// Over the four lanes that hold one head (lane % 16): exchanges of rows of 16 and of halves of the wave.
MX_DEV float wave_max(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(fbits(x), fbits(x), false, false);
  x = fmaxf(bitsf(r[0]), bitsf(r[1]));
  r = __builtin_amdgcn_permlane32_swap(fbits(x), fbits(x), false, false);
  return fmaxf(bitsf(r[0]), bitsf(r[1]));
}
MX_DEV float wave_sum(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(fbits(x), fbits(x), false, false);
  x = bitsf(r[0]) + bitsf(r[1]);
  r = __builtin_amdgcn_permlane32_swap(fbits(x), fbits(x), false, false);
  return bitsf(r[0]) + bitsf(r[1]);
}

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

// The kernel's arguments where the launch left them. A phase that reads them through a fresh() pointer has
// them loaded anew (a hit of the scalar cache) instead of held in scalar registers since the kernel's start,
// which are too few for that.
typedef const __attribute__((address_space(4))) Args Kernarg;
MX_DEV Kernarg* fresh(Kernarg* p) {
  asm("" : "+s"(p));
  return p;
}
MX_DEV FastDiv copy_of(const __attribute__((address_space(4))) FastDiv& d) {
  FastDiv f;
  f.m = d.m, f.d = d.d, f.s = d.s;
  return f;
}

// One sequence's attended positions lo .. hi - 1, counted in grains from the tile that holds lo. A row
// without positions still has a grain, whose workgroup writes it.
struct Row {
  int lo, hi, base, grains;
};

MX_DEV Row row_of(Kernarg& a, int length, int start) {
  Row r;
  r.hi = max(0, min(min(length, a.max_len), a.max_keys));
  r.lo = max(start, 0);
  if (a.window > 0) r.lo = max(r.lo, r.hi - a.window);
  if (r.lo >= r.hi) r.lo = r.hi = 0;
  r.base = r.lo & ~(kTile - 1);
  r.grains = max(1, (r.hi - r.base + kGrain - 1) / kGrain);
  return r;
}

MX_DEV int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Sum over the lanes up to this one: within rows of 16, then over the rows.
MX_DEV uint32_t wave_scan(uint32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // lane 15 of a row to the next row
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return x;
}

// A place in the list of all units' grains: sequence, unit within it, grain; `at` is the sequence's place in the list.
struct Place {
  int b, unit, grain;
  uint32_t at;
};

// No unit is cut within this many grains of its ends, for shares of `per` grains: a cut costs two partials
// and their join, about as much as four grains, so larger shares leave small units whole (8 x 8 units of 6 to
// 368 grains, per = 4: 22.5 us with 2, 25.4 with 1; 12 x 5 units of 11 grains, per = 2: 14.5 us with 1, 15.8
// with 2). Units of fewer than kCut are not cut (8 units of four grains: 9.4 us, in four workgroups each 11.9;
// of five: 13.3 whole, 11.1 cut).
constexpr int kCut = 5;
MX_DEV int least_of(uint32_t per, int grains) { return grains < kCut ? grains : (int)min(max(per / 2u, 1u), 4u); }

// The list of `all` places is cut into equal shares: cut i is at ceil(i all / wgs) (rounded up, so that units of one
// length are cut as if their beginnings did not count). Shares of one to four places are rounded up to whole ones
// where that makes them a quarter longer at most, as fewer cuts then count for more (64 x 8 ragged rows of up to 1000
// keys E4M3: 20.7 us, 23.2 cut evenly; 16 x 8 of up to 2000: 18.7 and 19.8; where it makes them longer, the
// even cuts win: 12 x 5 rows of up to 4000, 2.1 places: 17.9 us, 21.3 rounded up; and so they do above four: 16 x 4 of
// 2000, 4.25 places: 19.2 and 22.1). Where a share has more than a grain, `entry` = 1: each unit's grains follow one
// place for its beginning and end, which cost about as much (128 ragged rows of up to 1000 keys: 20.5 -> 14.9 us;
// 32 x 8 of up to 8192: 60.4 -> 54.4; 12 x 5 rows in 512 shares: 13.7 us with it, 13.0 without).
struct Cuts {
  uint32_t all, per, rest, entry;  // rest: places that even shares of `per` leave
  uint32_t num, den;               // cuts per place
};
MX_DEV uint32_t cut_at(const Cuts& c, Kernarg& a, uint32_t i) {
  return min(c.all, i * c.per + copy_of(a.wgs_div).div(i * c.rest + (uint32_t)a.wgs - 1u));
}
// The last cut at or before place x, x num / den, by a product's guess, which is off by one at most.
MX_DEV int cut_before(const Cuts& c, uint32_t x) {
  const int q = uniform((int)((float)x * (float)c.num * __builtin_amdgcn_rcpf((float)c.den)));
  const int64_t left = (int64_t)x * c.num - (int64_t)q * c.den;
  return q + (left >= c.den ? 1 : 0) - (left < 0 ? 1 : 0);
}

// This workgroup's share of the grains, from..to, equal but for the cuts' distance from the units' ends. Every
// wave sums up the lengths by itself, a sequence to a lane: a handful of loads that all find in the caches,
// where a launch that planned would cost its own latency, and no barrier. (Short code counts here: a
// workgroup runs it once, and its instructions come from memory.)
MX_DEV Cuts share_of(Kernarg& a, int units, Place& from, Place& to) {
  const int lane = threadIdx.x & 63;
  Cuts cuts = {};
  uint32_t size, before, total;
  const int32_t *lengths = a.lengths, *starts = a.starts ? a.starts : lengths;
  const auto look = [&](int b0) {
    const int b = min(b0 + lane, a.seqs - 1), length = lengths[b], start = starts[b];
    size = (uint32_t)row_of(a, length, a.starts ? start : 0).grains + cuts.entry;
    if (b0 + lane >= a.seqs) size = 0u;
    before = wave_scan(size);
    total = (uint32_t)__builtin_amdgcn_readlane((int)before, 63);
    before -= size;
  };
  look(0);
  uint32_t all = total;
  for (int b0 = 64; b0 < a.seqs; b0 += 64) {
    look(b0);
    all += total;
  }
  all *= (uint32_t)units;
  if (all > (uint32_t)a.wgs) {
    cuts.entry = 1u, all += (uint32_t)(a.seqs * units);  // below 2^31
    if (a.seqs <= 64) size += lane < a.seqs ? 1u : 0u, before += (uint32_t)min(lane, a.seqs), total += (uint32_t)a.seqs;
  }
  cuts.all = all, cuts.per = copy_of(a.wgs_div).div(all);
  cuts.rest = all - cuts.per * (uint32_t)a.wgs, cuts.num = (uint32_t)a.wgs, cuts.den = all;
  if (cuts.per == 0u || (cuts.per < 4u && 4u * ((uint32_t)a.wgs - cuts.rest) <= all)) {
    cuts.per += cuts.rest ? 1u : 0u;
    cuts.rest = 0u, cuts.num = 1u, cuts.den = cuts.per;
  }
  uint32_t sum = 0u;
  from = to = Place{a.seqs, 0, 0, all};
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    if (a.seqs > 64) look(b0);
#pragma unroll 1
    for (int side = 0; side < 2; side++) {
      const uint32_t cut = cut_at(cuts, a, blockIdx.x + side);
      const uint32_t q = copy_of(a.units_div).div(cut) - sum;  // grains of a unit's column before the cut's
      if (cut >= all || q >= total) continue;  // (a cut before this block wraps around)
      const int at_lane = 63 - __builtin_clzll(__ballot(before <= q));  // the last one that starts at or before q
      const uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)size, at_lane);
      Place p = {b0 + at_lane, 0, 0, (sum + (uint32_t)__builtin_amdgcn_readlane((int)before, at_lane)) * units};
      p.unit = uniform((int)((cut - p.at) / n));
      const int grains = (int)(n - cuts.entry), least = least_of(cuts.per, grains);
      p.grain = (int)(cut - p.at - p.unit * n - cuts.entry);
      if (p.grain < least) p.grain = 0;
      else if (grains - p.grain < least) p.grain = 0, p.unit++;
      if (p.unit == units) p = Place{p.b + 1, 0, 0, p.at + n * units};
      if (side) to = p;
      else from = p;
    }
    sum += total;
  }
  return cuts;
}

// Tiles of a wave on their way: two, or one of D = 256, whose registers would not hold a second; and one where
// workgroups take whole units, a few tiles of a wave, whose time is the code's length (8 x 500 keys: 9.4 us, 10.0
// with two).
constexpr int tiles_ahead(int D, bool split, int ht = 1) { return D == 256 || ht > 1 || !split ? 1 : 2; }
// The queries' 32 registers would be spilled of D = 256 or two head tiles: a lane keeps them in LDS, where the merge's
// rows come later.
constexpr bool query_in_lds(int D, int ht) { return D == 256 || ht > 1; }
// Shares of D = 256 16-bit rows take more than 256 registers (16 x 8192 x 4 fp16: 88 us, spilled into 256 of them
// 101; E4M3 fits: 64 us against 69), which whole units, small and many, do better without (200 x 4 rows of 30 keys:
// 15 us against 25). Shares of D = 64 fit three waves (78 x 16 short rows E4M3: 17 us, 20 with two, 24 spilled into four), but for 7 to 9
// registers of rows that go on from shared positions.
constexpr int waves_per_simd(int D, bool mx8, bool split, int ht) { return !split || ht > 1 ? 2 : D == 64 ? 3 : D == 256 && !mx8 ? 1 : 2; }

// D: 64, 128 or 256, the head size rounded up. T: type of q, out and the arithmetic. MX8: E4M3 cache.
// PAGED16: page_size % 16 == 0, so that the 16 keys of half a tile lie in one page: their place is a
// buffer descriptor in scalar registers, whose size also turns keys past the end, missing pages and
// elements past dim into zeros. For other page sizes a lane works out one key's place and the others
// read it from LDS.
// SPLIT: workgroups take shares of the grains and join what they cut; else one takes a whole unit, and the code
// of shares and joins, whose instructions would be waited for, is left out (4 x 12 rows of 30 keys: 5.6 us, 6.4
// with it; eight waves for a unit were slower than four: 8 x 500 keys 11.1 us against 10.0).
// SHARED: rows begin with positions whose results another kernel has left. (A switch at run time cost calls without them: shares of D = 64
// kept 7 to 9 registers in scratch memory, and 64 ragged rows of up to 2000 keys of 8 x 64 fp16 took 38.9 us for 36.0, 32 of up to 8000 of 2 x 64 E4M3
// for 20 heads each 27.6 for 24.1.)
template <int D, typename T, bool MX8, bool PAGED16, bool SPLIT, int HT, bool SHARED>
__global__ __launch_bounds__(kThreads, waves_per_simd(D, MX8, SPLIT, HT)) void decode_kernel(Args) {
  typedef typename Vec<T>::x8 x8;
  constexpr float kShift = Vec<T>::kShift;
  constexpr int kSteps = D / 32;          // matrix instructions of one score tile
  constexpr int kLoads = MX8 ? D / 64 : kSteps;  // 16-byte loads of a key's row
  constexpr int kRuns = D == 256 ? 2 : 1; // runs of kRow elements of V per lane and key
  constexpr int kRow = D == 64 ? 4 : 8;
  constexpr int kOut = D / 16;            // accumulators
  constexpr int kSize = MX8 ? 1 : 2;      // bytes of an element
  constexpr int kAhead = tiles_ahead(D, SPLIT, HT);
  constexpr int kHeads = 16 * HT;         // query heads of a unit
  constexpr int kBlock = 32;              // tiles of a wave whose pages it looks up at a time
  extern __shared__ float lds[];          // queries: [wave][step][lane]; merge: [kWaves / 2][head][D + kPad]; join: sums, then [head][kFan] weights
  __shared__ float wave_m[kWaves][kHeads], wave_l[kWaves][kHeads], head_m[kHeads], head_l[kHeads];
  __shared__ int is_last;
  constexpr bool kQueryInLds = query_in_lds(D, HT);
  u32x4* const query = reinterpret_cast<u32x4*>(lds) + (threadIdx.x >> 6) * HT * kSteps * 64 + (threadIdx.x & 63);
  __shared__ int64_t place_of[PAGED16 ? 1 : kWaves][2][kTile];  // of the keys of a wave's two tiles

  Kernarg* const args = (Kernarg*)__builtin_amdgcn_kernarg_segment_ptr();
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  const int units = args->heads * args->tiles;
  Place at, end = {};
  Cuts cuts = {};
  if constexpr (SPLIT) {
    cuts = share_of(*args, units, at, end);
  } else {
    const int b = (int)copy_of(args->units_div).div(blockIdx.x);
    at = Place{b, (int)blockIdx.x - b * units, 0, 0};
  }

  for (;;) {
    if constexpr (SPLIT) {
      if (!(at.b < end.b || (at.b == end.b && (at.unit < end.unit || (at.unit == end.unit && at.grain < end.grain))))) break;
    }
    Kernarg& a = *fresh(args);
    const int b = at.b, dim = a.dim;
    const int hk = (int)copy_of(a.tiles_div).div((uint32_t)at.unit), ht = at.unit - hk * a.tiles;
    const int first_head = hk * a.group + kHeads * ht, n_heads = min(kHeads, a.group - kHeads * ht);
    const int64_t head_at = (int64_t)hk * a.head_stride, page_stride = a.page_stride, slot_stride = a.slot_stride;
    const int32_t* table = a.table + (int64_t)b * a.cols;
    const FastDiv page_div = copy_of(a.page_div);
    const int page_size = a.page_size, pages = a.pages, cols = a.cols;
    const float score_scale = a.scale, softcap = a.softcap;

    // The unit's first loads wait together: its row's length, the pages that the wave's first keys have if the row
    // starts at 0 (a page's number is read before it is known that its keys count), and the queries.
    const bool from_zero = !a.starts && a.window == 0;
    const int ahead = at.grain * kGrain + wave * kTile;  // the wave's first key, if the row starts at 0
    const auto page_at = [&](int key) -> int { return table[min((int)page_div.div((uint32_t)key), cols - 1)]; };
    const auto page_or_none = [&](int p) -> int { return p >= 0 && p < pages ? p : -1; };
    int page_ahead = -1;
    const int length = a.lengths[b], start = (a.starts ? a.starts : a.lengths)[b];
    if (from_zero) page_ahead = page_at(ahead + (PAGED16 ? (lane >> 1) * kGrain + (lane & 1) * 16 : lane & (kTile - 1)));

    // Query fragments: columns c of each head tile, the elements that this lane's K loads hold; zeros past the
    // heads and past dim.
    x8 qf[kQueryInLds ? 1 : kSteps];
#pragma unroll
    for (int t = 0; t < HT; t++) {
      const int head = 16 * t + c;
      const T* q = (const T*)a.q + (int64_t)b * a.qt + (int64_t)(first_head + (head < n_heads ? head : 0)) * a.qh;
      u32x4 w[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
        const int d = MX8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
        w[s] = *reinterpret_cast<const u32x4*>(q + (d < dim ? d : 0));
      }
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
        const int d = MX8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
        if (head >= n_heads || d >= dim) w[s] = (u32x4){0u, 0u, 0u, 0u};
        if constexpr (kQueryInLds) query[64 * (t * kSteps + s)] = w[s];
        else qf[s] = __builtin_bit_cast(x8, w[s]);
      }
    }
    Row row = row_of(a, length, a.starts ? start : 0);
    row = Row{uniform(row.lo), uniform(row.hi), from_zero ? 0 : uniform(row.base), uniform(row.grains)};
    const int stop = SPLIT && b == end.b && at.unit == end.unit ? end.grain : row.grains;
    const int from = row.base + at.grain * kGrain, to = min(row.hi, row.base + stop * kGrain), lo = row.lo;

    // Byte offsets of this lane's loads within 16 keys' rows.
    const int slot_bytes = (int)slot_stride * kSize, slot_scales = (int)slot_stride / 32;
    int k_at[kLoads], v_at[4][kRuns];
#pragma unroll
    for (int s = 0; s < kLoads; s++) {
      const int d = MX8 ? 64 * s + 16 * g : 32 * s + 8 * g;
      k_at[s] = d < dim ? c * slot_bytes + d * kSize : kFar;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int r = 0; r < kRuns; r++) {
        const int d = 128 * r + kRow * c;
        v_at[j][r] = d < dim ? (4 * g + j) * slot_bytes + d * kSize : kFar;
      }
    const uint8_t *kp = a.k, *vp = a.v, *ksp = a.ks, *vsp = a.vs;

    f32x4 acc[HT][kOut];
    float m[HT], l[HT];
#pragma unroll
    for (int t = 0; t < HT; t++) {
#pragma unroll
      for (int i = 0; i < kOut; i++) acc[t][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
      m[t] = -INFINITY, l[t] = 0.f;
    }

    // A tile's K is loaded again as soon as its scores are formed, its V as soon as it is added up.
    struct Tile {
      u32x4 k[2][kLoads], v[8][kRuns];
      uint32_t ke[2][kLoads], ve[8][kRuns];
      int64_t off[2];        // PAGED16: element offset of each half's page slot, and its keys
      int rows[2];
      uint32_t mask;         // not PAGED16: bit i: key i is attended
    } tile[kAhead];
    for (int first = from + wave * kTile; first < to; first += kBlock * kGrain) {
      const int upto = min(to, first + kBlock * kGrain);  // the tiles of this block end here
      const int n_tiles = (upto - first + kGrain - 1) / kGrain;

      // PAGED16: lane i holds the element offset of half i % 2 of tile i / 2 (negative: no page).
      int off_lo = 0, off_hi = -1;
      // else: lane i % 32 holds the page of key i of the next tile to be placed
      int page = -1;
      const auto fetch_page = [&](int it) -> int {
        return page_or_none(page_at(min(first + it * kGrain + (lane & (kTile - 1)), to)));
      };
      if constexpr (PAGED16) {
        const int key = first + (lane >> 1) * kGrain + (lane & 1) * 16, i = (int)page_div.div((uint32_t)key);
        int p = page_ahead;
        if (!from_zero || first != ahead) p = page_at(key);
        p = page_or_none(p);
        const int64_t off = p * page_stride + (key - i * page_size) * slot_stride + head_at;
        off_lo = (int)off, off_hi = p < 0 ? -1 : (int)(off >> 32);
      } else {
        page = from_zero && first == ahead ? page_or_none(page_ahead) : fetch_page(0);
      }

      const auto place_tile = [&](Tile& z, int it) {
        if constexpr (PAGED16) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const int hi = __builtin_amdgcn_readlane(off_hi, 2 * it + h), lw = __builtin_amdgcn_readlane(off_lo, 2 * it + h);
            z.off[h] = (int64_t)((uint64_t)(uint32_t)max(hi, 0) << 32 | (uint32_t)lw);
            z.rows[h] = hi < 0 ? 0 : uniform(min(16, max(0, upto - (first + it * kGrain + 16 * h))));  // a clamp is a vector instruction
          }
        } else {
          // keys that do not count have the cache's first row: memory that is there, and values that are dropped
          const int key = first + it * kGrain + (lane & (kTile - 1));
          const bool ok = key >= lo && key < upto && page >= 0;
          const int64_t off = page * page_stride + (key - (int)page_div.div((uint32_t)key) * page_size) * slot_stride;
          if (lane < kTile) place_of[wave][it & 1][lane] = head_at + (ok ? off : 0);
          z.mask = (uint32_t)__ballot(ok);
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          page = fetch_page(it + 1);
        }
      };
      const auto load_k = [&](Tile& z, int it) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          if constexpr (PAGED16) {
            const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)(kp + z.off[h] * kSize), (short)0, z.rows[h] * slot_bytes, 0x00020000);
#pragma unroll
            for (int s = 0; s < kLoads; s++) z.k[h][s] = __builtin_amdgcn_raw_buffer_load_b128(r, k_at[s], 0, kStream);
            if constexpr (MX8) {
              const rsrc_t e = __builtin_amdgcn_make_buffer_rsrc((void*)(ksp + (z.off[h] >> 5)), (short)0, z.rows[h] * slot_scales, 0x00020000);
#pragma unroll
              for (int s = 0; s < kLoads; s++) z.ke[h][s] = __builtin_amdgcn_raw_buffer_load_b8(e, k_at[s] >> 5, 0, 0);
            }
          } else {
            const int64_t o = place_of[wave][it & 1][16 * h + c];
#pragma unroll
            for (int s = 0; s < kLoads; s++) {
              const int d = MX8 ? 64 * s + 16 * g : 32 * s + 8 * g;
              const int64_t e = o + (d < dim ? d : 0);
              z.k[h][s] = *reinterpret_cast<const u32x4*>(kp + e * kSize);
              if constexpr (MX8) z.ke[h][s] = ksp[e >> 5];
            }
          }
        }
      };
      // V: kRow elements from kRow * c (+ 128 per run) of each of the eight keys; past dim: zeros or element
      // 0, whose output rows are not written
      const auto load_v = [&](Tile& z, int it) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          rsrc_t rv, re;
          if constexpr (PAGED16) {
            rv = __builtin_amdgcn_make_buffer_rsrc((void*)(vp + z.off[h] * kSize), (short)0, z.rows[h] * slot_bytes, 0x00020000);
            if constexpr (MX8) re = __builtin_amdgcn_make_buffer_rsrc((void*)(vsp + (z.off[h] >> 5)), (short)0, z.rows[h] * slot_scales, 0x00020000);
          }
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int j = 4 * h + i;
            int64_t o = 0;
            if constexpr (!PAGED16) o = place_of[wave][it & 1][16 * h + 4 * g + i];
#pragma unroll
            for (int r = 0; r < kRuns; r++) {
              const int d = 128 * r + kRow * c;
              const int64_t e = o + (d < dim ? d : 0);
              u32x4& w = z.v[j][r];
              if constexpr (kSize * kRow == 16) {
                if constexpr (PAGED16) w = __builtin_amdgcn_raw_buffer_load_b128(rv, v_at[i][r], 0, kStream);
                else w = *reinterpret_cast<const u32x4*>(vp + e * kSize);
              } else if constexpr (kSize * kRow == 8) {
                u32x2 x;
                if constexpr (PAGED16) x = __builtin_amdgcn_raw_buffer_load_b64(rv, v_at[i][r], 0, kStream);
                else x = *reinterpret_cast<const u32x2*>(vp + e * kSize);
                w = (u32x4){x[0], x[1], 0u, 0u};
              } else {
                uint32_t x;
                if constexpr (PAGED16) x = __builtin_amdgcn_raw_buffer_load_b32(rv, v_at[i][r], 0, kStream);
                else x = *reinterpret_cast<const uint32_t*>(vp + e);
                w = (u32x4){x, 0u, 0u, 0u};
              }
              if constexpr (MX8) {
                if constexpr (PAGED16) z.ve[j][r] = __builtin_amdgcn_raw_buffer_load_b8(re, v_at[i][r] >> 5, 0, 0);
                else z.ve[j][r] = vsp[e >> 5];
              }
            }
          }
        }
      };

      const auto attend = [&](Tile& z, int it) {
        const int t = first + it * kGrain;
        // whether every key is attended, which of this lane's are (bit j: key 16 (j / 4) + 4 g + j % 4), and
        // whether V holds others
        bool all_seen, clear_v;
        uint32_t seen = 0xFFu;
        if constexpr (PAGED16) {
          all_seen = z.rows[0] == 16 && z.rows[1] == 16 && t >= lo;
          clear_v = t < lo;
          if (!all_seen) {
            seen = 0u;
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const int i = 4 * g + j % 4;
              seen |= i < z.rows[j / 4] && t + 16 * (j / 4) + i >= lo ? 1u << j : 0u;
            }
          }
        } else {
          all_seen = z.mask == ~0u;
          clear_v = !all_seen;
          seen = (z.mask >> (4 * g) & 15u) | (z.mask >> (4 * g + 16) & 15u) << 4;
        }

        // S^T: keys 4 g + i of half h, head c of each head tile.
        f32x4 s[HT][2];
#pragma unroll
        for (int u = 0; u < HT; u++) s[u][0] = s[u][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < kSteps; st++) {
          x8 q[HT];
#pragma unroll
          for (int u = 0; u < HT; u++) {
            if constexpr (kQueryInLds) q[u] = __builtin_bit_cast(x8, query[64 * (u * kSteps + st)]);
            else q[u] = qf[st];
          }
#pragma unroll
          for (int h = 0; h < 2; h++) {
            u32x4 w;
            if constexpr (MX8) {
              const u32x4 p = z.k[h][st / 2];
              w = widen<T>(st % 2 ? (u32x2){p[2], p[3]} : (u32x2){p[0], p[1]}, z.ke[h][st / 2]);
            } else {
              w = z.k[h][st];
            }
            if constexpr (!PAGED16) {
              if ((MX8 ? 64 * (st / 2) + 16 * g : 32 * st + 8 * g) >= dim) w = (u32x4){0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int u = 0; u < HT; u++) s[u][h] = Vec<T>::mfma(__builtin_bit_cast(x8, w), q[u], s[u][h]);
          }
        }
        place_tile(z, it + kAhead);
        load_k(z, it + kAhead);
        x8 p[HT], rest[HT];
#pragma unroll
        for (int u = 0; u < HT; u++) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] = s[u][j / 4][j % 4];
          if (softcap > 0.f) {
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = kLog2e * soft_cap(x[j] * score_scale, softcap);
          } else {
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] *= score_scale * kLog2e;
          }
          if (!all_seen) {
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = seen >> j & 1u ? x[j] : -INFINITY;
          }
          float top = x[0];
#pragma unroll
          for (int j = 1; j < 8; j++) top = fmaxf(top, x[j]);
          if (__any(top > m[u])) {  // seldom after the first tiles
            top = fmaxf(wave_max(top), m[u]);
            const float f = __builtin_amdgcn_exp2f(m[u] - finite_or_zero(top));
            l[u] *= f;
#pragma unroll
            for (int i = 0; i < kOut; i++) acc[u][i] *= f;
            m[u] = top;
          }
          const float ref = finite_or_zero(m[u]) - kShift;
#pragma unroll
          for (int j = 0; j < 8; j++) {
            x[j] = __builtin_amdgcn_exp2f(x[j] - ref);
            l[u] += x[j];
          }
          p[u] = __builtin_bit_cast(x8, (u32x4){Vec<T>::cut(x[0], x[1]), Vec<T>::cut(x[2], x[3]), Vec<T>::cut(x[4], x[5]), Vec<T>::cut(x[6], x[7])});
#pragma unroll
          for (int j = 0; j < 8; j++) rest[u][j] = (T)fmaxf(x[j] - (float)p[u][j], Vec<T>::kLeast);
        }

        // out^T += V^T P^T
#pragma unroll
        for (int r = 0; r < kRuns; r++) {
          if constexpr (kRuns > 1) __builtin_amdgcn_sched_barrier(0);  // one run's values at a time: else they spill
          u32x4 w[8];
#pragma unroll
          for (int j = 0; j < 8; j++) {
            if constexpr (MX8) w[j] = widen<T>((u32x2){z.v[j][r][0], z.v[j][r][1]}, z.ve[j][r]);
            else w[j] = z.v[j][r];
          }
          if (clear_v) {  // p = 0 there, and 0 * NaN is NaN
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (!(seen >> j & 1u)) w[j] = (u32x4){0u, 0u, 0u, 0u};
          }
#pragma unroll
          for (int i = 0; i < kRow; i++) {
            const uint32_t sel = i % 2 ? 0x07060302u : 0x05040100u;
            u32x4 f;
#pragma unroll
            for (int j = 0; j < 4; j++) f[j] = __builtin_amdgcn_perm(w[2 * j + 1][i / 2], w[2 * j][i / 2], sel);
#pragma unroll
            for (int u = 0; u < HT; u++) {
              f32x4& o = acc[u][kRow * r + i];
              o = Vec<T>::mfma(__builtin_bit_cast(x8, f), rest[u], o);
              o = Vec<T>::mfma(__builtin_bit_cast(x8, f), p[u], o);
            }
          }
        }
        load_v(z, it + kAhead);
      };

#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        place_tile(tile[i], i);
        load_k(tile[i], i);
        load_v(tile[i], i);
      }
      if constexpr (kAhead == 1) {
        for (int it = 0; it < n_tiles; it++) attend(tile[0], it);
      } else {
        for (int it = 0;; it += 2) {
          attend(tile[0], it);
          if (it + 1 >= n_tiles) break;
          attend(tile[1], it + 1);
          if (it + 2 >= n_tiles) break;
        }
      }
    }

    // On its way during the merge: where the results of the positions that the row shares are.
    i32x4 shared_at = {0, 0, 0, 0};
    if constexpr (SHARED) shared_at = fresh(args)->prefix.rows[b];

    // Merge the waves, referred to their common maximum: half of them put their rows into LDS, the others add
    // theirs, and the readers below add the remaining ones.
#pragma unroll
    for (int u = 0; u < HT; u++) {
      l[u] = wave_sum(l[u]);
      if (g == 0) wave_m[wave][16 * u + c] = m[u], wave_l[wave][16 * u + c] = l[u];
    }
    __syncthreads();
    constexpr int kLd = D + kPad, kHalf = kWaves / 2;
    {
      float f[HT];
#pragma unroll
      for (int u = 0; u < HT; u++) {
        const int head = 16 * u + c;
        float top = wave_m[0][head], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, wave_m[w][head]);
#pragma unroll
        for (int w = 0; w < kWaves; w++) sum += wave_l[w][head] * __builtin_amdgcn_exp2f(wave_m[w][head] - finite_or_zero(top));
        if (wave == 0) head_m[head] = top, head_l[head] = sum;
        f[u] = __builtin_amdgcn_exp2f(m[u] - finite_or_zero(top));
      }
#pragma unroll
      for (int round = 1; round >= 0; round--) {
#pragma unroll
        for (int u = 0; u < HT; u++) {
          if (wave / kHalf != round || 16 * u + c >= n_heads) continue;
          float* o = lds + ((wave % kHalf) * n_heads + 16 * u + c) * kLd;
#pragma unroll
          for (int i = 0; i < kOut; i += 4)
#pragma unroll
            for (int v = 0; v < 4; v++) {
              // neighbouring accumulators hold neighbouring elements
              f32x4* p = reinterpret_cast<f32x4*>(o + 128 * (i / 8) + kRow * (4 * g + v) + i % kRow);
              f32x4 w = {acc[u][i][v] * f[u], acc[u][i + 1][v] * f[u], acc[u][i + 2][v] * f[u], acc[u][i + 3][v] * f[u]};
              if (round == 0) w += *p;
              *p = w;
            }
        }
        __syncthreads();
      }
    }

    Kernarg& z = *fresh(args);
    const int quads = dim / 4;
    const FastDiv quads_div = copy_of(z.quads_div);
    const auto finish = [&](int h, int d, f32x4 o, float sum) {
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      store4<T>((T*)z.out + (int64_t)b * z.ot + (int64_t)(first_head + h) * z.oh + d, o * inv);
    };
    const auto put_lse = [&](int h, float top, float sum) {
      if (z.lse) z.lse[(int64_t)b * z.heads * z.group + first_head + h] = sum == 0.f ? -INFINITY : kLn2 * (top - kShift + __log2f(sum));
    };
    // The head's results of the positions that its row shares, kDeep splits of them at a time.
    const auto add_shared = [&](int h, int d, f32x4& o, float& top, float& sum) {
      if (!SHARED || !shared_at[3]) return;
      const int head = shared_at[2] + kHeads * ht + h;
      const int2 unit = z.prefix.units[shared_at[0] + hk * shared_at[1] + head / kPrefixUnit];
      const int splits = unit.y;
      const int64_t slot = prefix_slot_floats(dim), size = kPrefixSlots * slot;
      const float* p = z.prefix.partial + unit.x * size + head % kPrefixUnit / kPrefixRows * slot;
      const int outs = (d * (kPrefixRows / 4) + head % kPrefixRows) * 4, stats = kPrefixRows * dim + 2 * (head % kPrefixRows);
#pragma unroll 1
      for (int i = 0; i < splits; i += kDeep, p += kDeep * size) {
        float2 w[kDeep];
        f32x4 v[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; u++) {
          const int64_t at = i + u < splits ? u * size : 0;
          w[u] = *reinterpret_cast<const float2*>(p + at + stats), v[u] = *reinterpret_cast<const f32x4*>(p + at + outs);
        }
        float most = fmaxf(top, w[0].x);
#pragma unroll
        for (int u = 1; u < kDeep; u++) most = fmaxf(most, w[u].x);
        const float ref = finite_or_zero(most), f = __builtin_amdgcn_exp2f(top - ref);
        o *= f, sum *= f, top = most;
#pragma unroll
        for (int u = 0; u < kDeep; u++) {
          const float x = __builtin_amdgcn_exp2f(w[u].x - ref);  // NaN where the maximum is infinite
          // (a part that counts nothing is left out, unless it is NaN)
          if (i + u < splits && (x != 0.f || w[u].y != w[u].y)) o += v[u] * x, sum += w[u].y * x;
        }
      }
    };
    const bool whole = !SPLIT || (at.grain == 0 && stop == row.grains);
    // Partials, one for a share that begins within a unit and one for a unit that ends past the share:
    // [kHeads][dim] outputs, then [kHeads] {maximum, sum}.
    const uint32_t rows_at = (uint32_t)(kHeads * dim * 4), slot_size = rows_at + kHeads * 8;
    rsrc_t pr;
    if (!whole) pr = __builtin_amdgcn_make_buffer_rsrc(z.partial, (short)0, (int)(2 * z.wgs * slot_size), 0x00020000);
    const int items = n_heads * quads;
    const uint32_t mine_at = (2 * blockIdx.x + (at.grain == 0 ? 1u : 0u)) * slot_size;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int h = (int)quads_div.div((uint32_t)i), d = 4 * (i - h * quads);
      f32x4 o = *reinterpret_cast<const f32x4*>(lds + h * kLd + d);
#pragma unroll
      for (int w = 1; w < kHalf; w++) o += *reinterpret_cast<const f32x4*>(lds + (w * n_heads + h) * kLd + d);
      float sum = head_l[h], top = head_m[h];
      if (whole) {
        add_shared(h, d, o, top, sum);
        finish(h, d, o, sum);
        if (d == 0) put_lse(h, top, sum);
      } else {
        put4(pr, mine_at + 16u * i, o);
        if (d == 0) __builtin_amdgcn_raw_buffer_store_b64((u32x2){fbits(top), fbits(sum)}, pr, mine_at + rows_at + h * 8, 0, 17);
      }
    }

    // Join: the workgroup that arrives last adds the unit's partials in their order, of more than kFan in two steps:
    // groups of kGroup, then the groups. Every wave waits for its stores to be acknowledged before the
    // barrier and the counter's increment, so the last one (which takes the counter back to 0) sees all.
    // A partial's counter is its group's first one's. The code is kept short: its instructions come from
    // memory, as each workgroup runs it once.
    if constexpr (!SPLIT) break;
    if (!whole) {
      const uint32_t u0 = at.at + (uint32_t)at.unit * (row.grains + cuts.entry) + cuts.entry, least = least_of(cuts.per, row.grains);
      const int first = cut_before(cuts, u0 + least - 1u);  // the unit's first workgroup
      const int members = cut_before(cuts, u0 + row.grains - least) - first + 1;
      const int groups = members <= kFan ? 1 : ceil_div(members, kGroup), group = groups == 1 ? 0 : ((int)blockIdx.x - first) / kGroup;
      float* share = lds;                  // sums of a head's runs of partials, below
      float* weight = lds + 4 * kThreads;  // [head][kFan]
#pragma unroll 1
      for (int level = 0; level < 2; level++) {
        // the n partials start, start + step, ... of this step, and whether their sum is the result
        const int start = level == 0 ? group * kGroup : 0, step = level == 0 ? 1 : kGroup;
        const int n = level == 1 ? groups : groups == 1 ? members : min(kGroup, members - start);
        const bool result = level == 1 || groups == 1;
        const uint32_t head_slot = 2u * (first + start) + (start == 0 ? 1u : 0u);  // others: every second one after it
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
        if (threadIdx.x == 0)
          is_last = atomicInc(z.counters + (level == 1 ? 2 * z.wgs + first : head_slot), (unsigned)(n - 1)) == (unsigned)(n - 1);
        __syncthreads();
        if (!uniform(is_last)) break;
        const uint32_t at0 = 2u * (first + start) * slot_size, stride = 2u * step * slot_size, extra = start == 0 ? slot_size : 0u;
        // a descriptor that ends with the n-th partial: loads past it give 0
        const rsrc_t jr = __builtin_amdgcn_make_buffer_rsrc(z.partial, (short)0, (int)(at0 + (n - 1) * stride + (n == 1 ? extra : 0u) + slot_size), 0x00020000);
        // The first outputs are on their way while the weights are worked out. Where a unit has fewer output
        // quads than threads, groups of threads take every n-th partial.
        const int split = items < kThreads ? kThreads / items : 1;
        const int part = split > 1 ? (int)threadIdx.x / items : 0;
        f32x4 v[kDeep];
        const auto request = [&](int i, int ch) {  // partials ch, ch + split, ... of output quad i
          uint32_t off = part < split && i < items ? at0 + ch * stride + 16u * i : 2u * kFar;
          v[0] = get4(jr, off + (ch == 0 ? extra : 0u));
#pragma unroll
          for (int u = 1; u < kDeep; u++) {
            off += split * stride;
            v[u] = get4(jr, part < split && i < items ? off : 2u * kFar);
          }
        };
        request((int)threadIdx.x - part * items, part);
        // Weights 2^(m_i - m) of the lane's heads and every 4 kWaves-th partial, and the sums
        constexpr int kParts = kFan / (4 * kWaves);
        float cm[HT][kParts], cl[HT][kParts], top[HT];
#pragma unroll
        for (int u = 0; u < HT; u++) {
          const int head = 16 * u + c;
#pragma unroll
          for (int i = 0; i < kParts; i++) {
            const int ch = 4 * wave + g + 4 * kWaves * i;
            const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(jr, at0 + ch * stride + (ch == 0 ? extra : 0u) + rows_at + 8 * head, 0, 17));
            const uint32_t w0 = w[0], w1 = w[1];
            cm[u][i] = ch < n && head < n_heads ? bitsf(w0) : -INFINITY, cl[u][i] = ch < n && head < n_heads ? bitsf(w1) : 0.f;
          }
          top[u] = cm[u][0];
#pragma unroll
          for (int i = 1; i < kParts; i++) top[u] = fmaxf(top[u], cm[u][i]);
          top[u] = wave_max(top[u]);
          wave_m[wave][head] = top[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < HT; u++) {
          const int head = 16 * u + c;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; w++) top[u] = fmaxf(top[u], wave_m[w][head]);
#pragma unroll
          for (int i = 0; i < kParts; i++) {
            const float w = __builtin_amdgcn_exp2f(cm[u][i] - finite_or_zero(top[u]));
            if (head < n_heads) weight[head * kFan + 4 * wave + g + 4 * kWaves * i] = w;
            sum += w * cl[u][i];
          }
          sum = wave_sum(sum);
          wave_l[wave][head] = sum;
        }
        __syncthreads();
        const auto joined = [&](int h, float& sum) -> float {  // a head's maximum and sum over the partials
          float top = wave_m[0][h];
          sum = wave_l[0][h];
#pragma unroll
          for (int w = 1; w < kWaves; w++) top = fmaxf(top, wave_m[w][h]), sum += wave_l[w][h];
          return top;
        };
#pragma unroll 1
        for (int i0 = 0; i0 < items; i0 += kThreads) {
          const int i = i0 + (int)threadIdx.x - part * items;
          const bool mine = part < split && i < items;
          const int h = mine ? (int)quads_div.div((uint32_t)i) : 0, d = mine ? 4 * (i - h * quads) : 0;
          f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int ch = part; ch < n; ch += kDeep * split) {
            if (i0 > 0 || ch != part) request(i, ch);
#pragma unroll
            for (int u = 0; u < kDeep; u++) o += v[u] * weight[h * kFan + min(ch + u * split, kFan - 1)];
          }
          if (split > 1) {
            if (mine) *reinterpret_cast<f32x4*>(share + 4 * threadIdx.x) = o;
            __syncthreads();
            if (mine && part == 0)
              for (int p = 1; p < split; p++) o += *reinterpret_cast<const f32x4*>(share + 4 * (p * items + i));
          }
          if (mine && part == 0) {
            float sum;
            float top = joined(h, sum);
            if (result) {
              add_shared(h, d, o, top, sum);
              finish(h, d, o, sum);
              if (d == 0) put_lse(h, top, sum);
            } else {
              put4(pr, head_slot * slot_size + 16u * i, o);
              if (d == 0) __builtin_amdgcn_raw_buffer_store_b64((u32x2){fbits(top), fbits(sum)}, pr, head_slot * slot_size + rows_at + h * 8, 0, 17);
            }
          }
        }
        if (result) break;
      }
    }
    __syncthreads();  // the next unit's merge uses the same memory

    at.grain = 0;
    if (stop < row.grains) break;
    if (++at.unit == units) at = Place{b + 1, 0, 0, at.at + (row.grains + cuts.entry) * units};
  }
}

// ---- host -----------------------------------------------------------------------------------

// LDS bytes: the merge's rows, the queries, or the join's weights and sums.
size_t lds_bytes(int D, int ht, int n_heads, bool split) {
  const size_t merge = (size_t)(kWaves / 2) * n_heads * (D + kPad) * 4, weights = (size_t)(n_heads * kFan + 4 * kThreads) * 4;
  const size_t query = query_in_lds(D, ht) ? (size_t)kWaves * D * 32 * ht : 0;
  return std::max(std::max(merge, query), split ? weights : 0);
}

int padded(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

struct Plan {
  int64_t units;
  int ht, tiles;  // head tiles of 16 of a unit, and units of a cache head
  int wgs;        // workgroups that share the grains; 0: no unit is worth splitting
  size_t bytes;
};

constexpr int kCUs = 256;
static_assert(2 * kCUs <= kFan * kGroup, "a row's groups are joined in one step");
// The lengths are known on the device only. The grid is one round of workgroups: one to a CU, whose waves
// have 128 KB on their way, or two where two tiles per wave are less than that (131072 x 8 x 128 fp16:
// 92 us with one, 97 with two, which double the partials; 64 x 16384 x 8 x 128 E4M3: 366 and 346); fewer where
// max_len bounds the grains.
int workgroups(int D, int fmt, int ht) {
  return kCUs * (tiles_ahead(D, true, ht) * kGrain * 2 * D * (fmt == MX_E4M3 ? 1 : 2) < 131072 ? 2 : 1);
}

// Three counters per workgroup, at one place for every call: a workspace that served another shape has its
// partials past them.
constexpr size_t kCounterBytes = 3 * 2 * kCUs * 4;
static_assert(kCounterBytes == kDecodeCounterBytes, "counters");

Plan plan_for(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  Plan p = {};
  const int D = padded(c->dim), group = q_heads / c->heads;
  // positions from a sequence's first tile: a window may start within it
  const int64_t span = window > 0 && (int64_t)window + kTile < max_len ? (int64_t)window + kTile : max_len;
  const int64_t grains = ceil_div(span, (int64_t)kGrain);
  // Two head tiles, so that the keys of more than 16 query heads are read once, where that is what the time goes
  // to: at 16 grains and more of a workgroup (20 heads of 128 bf16, rows of 8192 keys: 94 -> 57 us at 32 grains; of
  // 32768: 31.0 and 32.5 at 8; of 4096: 20.5 and 28 at 4). Heads above 128 have one tile: a second would take the E4M3 shares' second wave per SIMD
  // and a merge in two rounds, and is not built.
  const int64_t units = (int64_t)seqs * c->heads * ceil_div(group, 16);
  p.ht = D < 256 && group > 16 && units * grains >= 16 * workgroups(D, c->fmt, 1) ? 2 : 1;
  p.tiles = ceil_div(group, 16 * p.ht);
  p.units = (int64_t)seqs * c->heads * p.tiles;
  const int64_t wgs = p.units * grains;
  if (grains < kCut || p.units * (grains + 1) >= (int64_t)1 << 30) return p;  // (the device counts in 32 bits)
  const int most = workgroups(D, c->fmt, p.ht);
  p.wgs = (int)(wgs < most ? wgs : most);
  p.bytes = kCounterBytes + (size_t)(2 * p.wgs) * 16 * p.ht * (c->dim + 2) * 4;
  return p;
}

bool sizes_ok(const mxkv_cache* c, int seqs, int q_heads, int max_len, int window) {
  return seqs >= 0 && seqs <= MX_MAX_DIM && q_heads >= 1 && q_heads <= MX_MAX_DIM && q_heads % c->heads == 0 && max_len >= 1 &&
         max_len < 1 << 30 && window >= 0 && (int64_t)seqs * q_heads < (int64_t)1 << 24;
}

template <int D, typename T, bool MX8, bool SPLIT, int HT, bool SHARED>
void launch(const Args& a, unsigned wgs, hipStream_t st) {
  const size_t lds = lds_bytes(D, HT, a.group < 16 * HT ? a.group : 16 * HT, SPLIT);
  if (a.page_size % 16 == 0) hipLaunchKernelGGL((decode_kernel<D, T, MX8, true, SPLIT, HT, SHARED>), dim3(wgs), dim3(kThreads), lds, st, a);
  else hipLaunchKernelGGL((decode_kernel<D, T, MX8, false, SPLIT, HT, SHARED>), dim3(wgs), dim3(kThreads), lds, st, a);
}

template <int D, typename T, bool MX8, int HT, bool SHARED>
void launch_split(const Args& a, const Plan& p, bool split, hipStream_t st) {
  if (split) launch<D, T, MX8, true, HT, SHARED>(a, (unsigned)p.wgs, st);
  else launch<D, T, MX8, false, HT, SHARED>(a, (unsigned)p.units, st);
}

template <typename T, bool MX8, bool SHARED>
void launch_dim(const Args& a, const Plan& p, bool split, hipStream_t st) {
  const int D = padded(a.dim);
  if (D == 64 && p.ht == 1) launch_split<64, T, MX8, 1, SHARED>(a, p, split, st);
  else if (D == 64) launch_split<64, T, MX8, 2, SHARED>(a, p, split, st);
  else if (D == 128 && p.ht == 1) launch_split<128, T, MX8, 1, SHARED>(a, p, split, st);
  else if (D == 128) launch_split<128, T, MX8, 2, SHARED>(a, p, split, st);
  else launch_split<256, T, MX8, 1, SHARED>(a, p, split, st);
}

template <typename T, bool MX8>
void launch_shared(const Args& a, const Plan& p, bool split, hipStream_t st) {
  if (a.prefix.partial) launch_dim<T, MX8, true>(a, p, split, st);
  else launch_dim<T, MX8, false>(a, p, split, st);
}

}  // namespace

namespace mx {

bool decode_sizes_ok(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window) { return sizes_ok(cache, seqs, q_heads, max_len, window); }

size_t decode_workspace(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window) {
  if (!cache || check_geometry(cache) || !sizes_ok(cache, seqs, q_heads, max_len, window) || seqs == 0) return 0;
  return plan_for(cache, seqs, q_heads, max_len, window).bytes;
}

int check_attention(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, const mxkv_table* table, const int32_t* lengths, int max_len,
                    const mxattn_opts* opts) {
  if (!cache || !q || !out || !table || !opts) return MX_ERR_NULL;
  if (f != MX_F16 && f != MX_BF16) return MX_ERR_FORMAT;
  if (int s = check_cache(cache)) return s;
  if (cache->fmt != MX_E4M3 && cache->fmt != f) return MX_ERR_FORMAT;
  if (int s = check_table(table)) return s;
  if (!sizes_ok(cache, table->seqs, q->heads, max_len, opts->window) || q->heads != out->heads) return MX_ERR_SHAPE;
  if (!__builtin_isfinite(opts->scale) || !__builtin_isfinite(opts->softcap) || opts->softcap < 0.f) return MX_ERR_SHAPE;
  if (table->seqs == 0) return MX_OK;
  if (!lengths) return MX_ERR_NULL;
  if (int s = check_heads(q, 2)) return s;
  return check_heads(out, 2);
}

int decode_launch(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse, const mxkv_table* table, const int32_t* lengths,
                  const int32_t* starts, int max_len, const mxattn_opts* opts, const Prefix& prefix, void* workspace, size_t workspace_bytes, hipStream_t st) {
  const bool mx8 = cache->fmt == MX_E4M3;
  const Plan p = plan_for(cache, table->seqs, q->heads, max_len, opts->window);
  Args a = {};
  a.prefix = prefix;
  a.k = (const uint8_t*)cache->k, a.v = (const uint8_t*)cache->v;
  a.ks = (const uint8_t*)cache->ks, a.vs = (const uint8_t*)cache->vs;
  a.q = q->data, a.qt = q->token_stride, a.qh = q->head_stride;
  a.out = out->data, a.ot = out->token_stride, a.oh = out->head_stride;
  a.lse = lse;
  a.table = table->pages, a.cols = table->cols, a.lengths = lengths, a.starts = starts;
  const bool split = p.wgs > 0 && workspace && workspace_bytes >= p.bytes;  // else a workgroup takes a whole unit
  a.wgs = p.wgs;
  if (split) {
    a.counters = (uint32_t*)workspace;
    a.partial = (float*)((uint8_t*)workspace + kCounterBytes);
  }
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.seqs = table->seqs, a.heads = cache->heads, a.group = q->heads / cache->heads, a.tiles = p.tiles, a.dim = cache->dim;
  a.pages = cache->pages, a.page_size = cache->page_size, a.max_len = max_len, a.max_keys = (int)std::min<int64_t>((int64_t)table->cols * cache->page_size, INT32_MAX);
  a.window = opts->window;
  a.scale = opts->scale, a.softcap = opts->softcap;
  a.page_div = FastDiv((uint32_t)cache->page_size);
  a.units_div = FastDiv((uint32_t)(cache->heads * p.tiles));
  a.tiles_div = FastDiv((uint32_t)p.tiles);
  a.wgs_div = FastDiv((uint32_t)(split ? p.wgs : 1));
  a.quads_div = FastDiv((uint32_t)cache->dim / 4);
  if (f == MX_F16 && mx8) launch_shared<_Float16, true>(a, p, split, st);
  else if (f == MX_F16) launch_shared<_Float16, false>(a, p, split, st);
  else if (mx8) launch_shared<__bf16, true>(a, p, split, st);
  else launch_shared<__bf16, false>(a, p, split, st);
  return launch_status();
}

}  // namespace mx

extern "C" size_t mxattn_decode_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window) {
  return decode_workspace(cache, seqs, q_heads, max_len, window);
}

extern "C" int mxattn_decode_run(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse,
                                 const mxkv_table* table, const int32_t* lengths, const int32_t* starts, int max_len,
                                 const mxattn_opts* opts, void* workspace, size_t workspace_bytes, void* stream) {
  if (int s = check_attention(cache, f, q, out, table, lengths, max_len, opts)) return s;
  if (table->seqs == 0) return MX_OK;
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  return sync_check(decode_launch(cache, f, q, out, lse, table, lengths, starts, max_len, opts, Prefix{}, workspace, workspace_bytes, st), st);
}
