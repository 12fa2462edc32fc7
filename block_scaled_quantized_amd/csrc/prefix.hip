// prefix.hip -- attention of one new token per sequence where groups of sequences share their first positions: the shared keys
// and values meet all of the group's queries at once, as matrix products, and are read once for them.
//
// Two launches. This kernel takes the shared positions: the queries of a group's rows and of the heads that read one cache head are the
// columns of 32 x 32 x 16 instructions, 32 to a wave. A workgroup stages tiles of 64 keys and values in LDS for its waves, which form scores
// transposed, S^T = K Q^T, whose registers are at once the second operand of out^T = V^T P^T if the sum over keys runs in the order in
// which a lane holds them; V^T comes from LDS by transposing reads. Long beginnings are split among workgroups. Each leaves its rows' running maximum,
// sum and output, which the decode kernel, the second launch, adds to those of the row's own positions.
//
// The shared positions of a group end where the shortest of its rows does, and with a whole tile: what is left is the rows' own, so
// no key here is masked for some rows and not for others.
//
// What bounds it: one round of workgroups, each of which works out the shares and fetches its first keys (some 15000 clocks) before turns of 128
// keys, 6100 to 6700 clocks for 128 rows, in which the matrix cores have 35% and the vector units most of the rest. 64 rows of 64 heads behind 8192
// positions of 8 x 128 bf16: 38 us here, 36 in the decode kernel (512 positions of each row and the joining of 17 MB of partial results), where
// the decode kernel alone takes 335. 96 rows in five groups behind up to 12000 positions, E4M3: 85 to 101 us and 52, alone 232.
#include <algorithm>

#include "attention.h"

using namespace mx;

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kRowWaves = kPrefixSlots, kRows = kPrefixUnit;  // query rows of a workgroup, 32 to a wave
constexpr int kGrain = 64;                                    // what is shared ends at a multiple of these
constexpr int kLeastShared = kGrain;
constexpr int kMaxGroups = 1024;
constexpr int kLeastTiles = 2;                                // of a workgroup

struct Args {
  const uint8_t *k, *v, *ks, *vs;
  const void* q;
  const int32_t *table, *lengths, *first, *shared;
  i32x4* rows;       // written for the decode kernel, as are units and starts
  int2* units;
  int32_t* starts;
  float* partial;
  int64_t qt, qh, page_stride, head_stride, slot_stride;
  int seqs, groups, heads, share, dim, cols, pages, max_len, max_keys, max_shared, wgs, page_size;
  float scale, softcap;
  FastDiv page_div, share_div;
};

MX_DEV int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// What every workgroup works out for itself from the lengths, in LDS. The work is a list of units (a group's cache head and 128 rows) of
// tiles of keys, one after the other; the workgroups take equal shares of it, so a share may end one unit and begin others. Share w's
// part of unit u is split w + u: that rises along the list, and a unit's splits are next to each other.
struct Plan {
  int* first;    // [groups + 1] sequences
  int* work;     // [groups + 1] tiles before the group's
  int* units;    // units before the group's
  int* end;      // shared positions
  int* lead;     // first sequence with positions, whose table row names the shared pages
};
constexpr int plan_ints(int groups) { return 5 * (groups + 1); }
MX_DEV Plan plan_in(int* lds, int groups) {
  const int n = groups + 1;
  return Plan{lds, lds + n, lds + 2 * n, lds + 3 * n, lds + 4 * n};
}
struct Shares {
  int all, per, rest;  // tiles; of a share; shares that have one more
  MX_DEV int cut(int w) const { return w * per + min(w, rest); }
  MX_DEV int share_of(int x) const { return x < rest * (per + 1) ? x / (per + 1) : rest + (x - rest * (per + 1)) / per; }
};

MX_DEV int length_of(const Args& a, int n) { return max(0, min(min(n, a.max_len), a.max_keys)); }

// The last i with sums[i] <= x, of n + 1 rising sums; 0 where the first is above.
MX_DEV int last_at(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// The group of sequence b, -1 if none.
MX_DEV int group_of(const Plan& p, int groups, int b) {
  const int g = last_at(p.first, groups, b);
  return p.first[g] <= b && b < p.first[g + 1] ? g : -1;
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

struct Shape {
  int rows, tiles, keys;  // of one group: query rows of a cache head, their units, tiles of keys
};
MX_DEV Shape shape_of(const Args& a, const Plan& p, int g, int tile) {
  Shape s;
  s.keys = ceil_div(p.end[g], tile), s.rows = max(0, p.first[g + 1] - p.first[g]) * a.share;
  s.tiles = s.keys ? ceil_div(s.rows, kRows) : 0;
  return s;
}

template <int THREADS>
MX_DEV Shares plan(const Args& a, const Plan& p, int tile) {
  constexpr int kOfThread = kMaxGroups / THREADS, kWaves = THREADS / 64;
  __shared__ unsigned long long all_work;
  __shared__ int falls;                // whether the firsts do, which makes them no groups
  __shared__ int wave_work[kWaves], wave_units[kWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // the first loads wait together
  const int own = a.lengths[min(t, a.seqs - 1)];
  for (int g = t; g <= a.groups; g += THREADS) {
    const int f = a.first[g], n = a.shared[min(g, a.groups - 1)];
    p.first[g] = max(0, min(f, a.seqs));
    p.end[g] = max(0, min(n, a.max_shared)), p.lead[g] = a.seqs, p.work[g] = 0;
  }
  if (t == 0) all_work = 0, falls = 0;
  __syncthreads();
  for (int g = t; g < a.groups; g += THREADS)
    if (p.first[g + 1] < p.first[g]) falls = 1;
  // rows without positions do not count (work: the others, for now); a beginning that no two rows share is not worth its own pass
  for (int b = t; b < a.seqs; b += THREADS) {
    const int n = length_of(a, b == t ? own : a.lengths[b]), g = group_of(p, a.groups, b);
    if (g >= 0 && n > 0) atomicMin(&p.end[g], n), atomicMin(&p.lead[g], b), atomicAdd(&p.work[g], 1);
  }
  __syncthreads();
  int work[kOfThread], units[kOfThread], my_work = 0, my_units = 0;
  unsigned long long mine = 0;
  for (int i = 0; i < kOfThread; i++) {
    const int g = t * kOfThread + i;
    work[i] = my_work, units[i] = my_units;
    if (g >= a.groups) continue;
    p.end[g] = p.work[g] < 2 || falls || p.end[g] < kLeastShared ? 0 : p.end[g] & ~(kGrain - 1);
    const Shape s = shape_of(a, p, g, tile);
    mine += (unsigned long long)a.heads * s.tiles * s.keys;
    my_work += a.heads * s.tiles * s.keys, my_units += a.heads * s.tiles;
  }
  if (mine) atomicAdd(&all_work, mine);
  const int upto_work = (int)wave_scan((uint32_t)my_work), upto_units = (int)wave_scan((uint32_t)my_units);
  if (lane == 63) wave_work[wave] = upto_work, wave_units[wave] = upto_units;
  __syncthreads();
  int before_work = upto_work - my_work, before_units = upto_units - my_units;
  for (int w = 0; w < wave; w++) before_work += wave_work[w], before_units += wave_units[w];
  for (int i = 0; i < kOfThread; i++) {
    const int g = t * kOfThread + i;
    if (g < a.groups) p.work[g] = before_work + work[i], p.units[g] = before_units + units[i];
  }
  // (work that does not fit an int, which would run for hours, is left to the rows themselves)
  Shares s;
  s.all = all_work < 1ull << 31 ? (int)all_work : 0;
  if (t == 0) p.work[a.groups] = s.all;
  const int shares = max(1, min(a.wgs, s.all / kLeastTiles));
  s.per = s.all / shares, s.rest = s.all - s.per * shares;
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1) {  // for the decode kernel
    for (int b = t; b < a.seqs; b += THREADS) {
      const int g = group_of(p, a.groups, b), n = length_of(a, b == t ? own : a.lengths[b]);
      const bool in = g >= 0 && p.end[max(g, 0)] > 0 && n > 0 && s.all > 0;
      a.starts[b] = in ? p.end[g] : 0;
      a.rows[b] = in ? (i32x4){p.units[g], shape_of(a, p, g, tile).tiles, (b - p.first[g]) * a.share, 1} : (i32x4){0, 0, 0, 0};
    }
  }
  return s;
}

// Two waves to a SIMD: two waves have the same rows and each half of a tile's keys, and take turns at the matrix cores and the vector
// units (below). Heads above 128 have twice the accumulators and queries, and one wave to a SIMD.
constexpr int halves_of(int D) { return D == 256 ? 1 : 2; }
constexpr int threads_of(int D) { return 64 * kRowWaves * halves_of(D); }
constexpr int keys_of(int D) { return 64 * halves_of(D); }            // of a tile
constexpr int lds_of(int D) { return 4 * keys_of(D) * 2 * D; }        // two tiles of keys, two of values

__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// Waits until at most N of the wave's accesses to memory, the last ones, are outstanding.
template <int N>
MX_DEV void wait_memory() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0F70 | (N >> 4) << 14);
}
// One wave's copy of 16 bytes per lane from memory to LDS, `to` and on. (In assembly, as the compiler would wait for every copy on its way before
// a read of LDS that it can see; the kernel waits by counts. The instruction has no result, and M0 needs a state between.)
MX_DEV void copy16(uint32_t to, const void* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0", "memory");
}
MX_DEV void barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// D: 64, 128 or 256, the head size rounded up. T: type of q and the arithmetic. MX8: E4M3 cache. CAP: scores are capped.
template <int D, typename T, bool MX8, bool CAP>
__global__ __launch_bounds__(threads_of(D), halves_of(D)) void prefix_kernel(Args a) {
  typedef typename Vec<T>::x8 x8;
  // A probability is at most 2^kSlack. binary16's, scaled by 2^15, stay in its range below 2: scaled by 2^9, for the same 2^6, the least second part would be
  // 2^-33 of the largest, which runs of thousands of keys that count nothing beside one would show (3 times the decode call's bound; 96 rows in five
  // groups E4M3: 130 us, and 132 as it is, with more turns that rescale).
  constexpr float kShift = Vec<T>::kShift, kSlack = kShift > 0.f ? 0.99f : 6.f;
  constexpr int kThreads = threads_of(D), kHalves = halves_of(D), kWaves = kThreads / 64, kKeys = keys_of(D);
  constexpr int kSteps = D / 16, kOut = D / 32;
  constexpr int kPitch = 2 * D, kPlane = kKeys * kPitch;                     // bytes of a key's row in LDS, and of a tile
  constexpr int kBlock = kThreads / kKeys;                                   // tiles whose keys' places are worked out at a time
  constexpr int kRowLanes = kPitch / 16, kCopies = kPlane / 1024 / kWaves;   // lanes of a row, copies of a wave and tile
  constexpr int kPieces = D / 16, kLoads = MX8 ? (kKeys * kPieces + kThreads - 1) / kThreads : 1;  // E4M3: 16-byte pieces of a row, of a thread
  constexpr bool kAll = kKeys * kPieces >= kThreads;                         // whether every thread has them
  extern __shared__ __attribute__((aligned(16))) char lds[];                 // two tiles of keys, two of values, the plan
  __shared__ int64_t place[2][kThreads];                                     // element offsets of the keys of two blocks of tiles, -1: none
  __shared__ unsigned long long there[2][kWaves];                            // which keys there are
  __shared__ float2 stats[kRowWaves][32];

  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), c = lane & 31, h = lane >> 5;
  const int row_wave = wave % kRowWaves, half = wave / kRowWaves;
  const int dim = a.dim;
  const Plan groups = plan_in(reinterpret_cast<int*>(lds + lds_of(D)), a.groups);
  const Shares shares = plan<kThreads>(a, groups, kKeys);
  // each XCD takes a run of the shares: those that read the same keys are next to each other
  const int share = gridDim.x % 8 == 0 ? (blockIdx.x & 7) * (gridDim.x / 8) + (blockIdx.x >> 3) : blockIdx.x;
  const int upto = uniform(min(shares.all, shares.cut(share + 1)));

  for (int x = uniform(shares.cut(share)); x < upto;) {
    const int g = uniform(last_at(groups.work, a.groups, x));
    const Shape shape = shape_of(a, groups, g, kKeys);
    const int rows = uniform(shape.rows), keys = uniform(shape.keys), tiles = uniform(shape.tiles), first = uniform(groups.first[g]);
    const int in = x - uniform(groups.work[g]), unit_in = in / keys, hk = unit_in / tiles, row_tile = unit_in - hk * tiles;
    const int unit = uniform(groups.units[g]) + unit_in, begin = in - unit_in * keys, end = min(keys, begin + upto - x);
    const int last_key = uniform(groups.end[g]);
    if (begin == 0 && t == 0) a.units[unit] = int2{share + unit, shares.share_of(x + keys - 1) - share + 1};
    x += end - begin;
    const int64_t slot = ((int64_t)(share + unit) * kRowWaves + row_wave) * prefix_slot_floats(dim);
    const int64_t head_at = (int64_t)hk * a.head_stride;
    const int32_t* table = a.table + (int64_t)uniform(groups.lead[g]) * a.cols;
    const int row0 = row_tile * kRows + 32 * row_wave;

    // The keys of tiles begin + kBlock b and on, one to a thread: its page, then its place.
    const auto key_of = [&](int b) { return (begin + kBlock * b) * kKeys + t; };
    const auto page_of = [&](int b) -> int { return table[min((int)a.page_div.div((uint32_t)key_of(b)), a.cols - 1)]; };
    const auto put_place = [&](int b, int page) {
      const int key = key_of(b);
      const bool ok = page >= 0 && page < a.pages && key < last_key;
      place[b & 1][t] = ok ? head_at + page * a.page_stride + (key - (int)a.page_div.div((uint32_t)key) * a.page_size) * a.slot_stride : -1;
      const unsigned long long mask = __ballot(ok);
      if (lane == 0) there[b & 1][wave] = mask;
    };
    const int page0 = page_of(0);

    // queries: column c of the instructions, elements 16 s + 8 h ..; rows past the group's repeat its first
    x8 q[kSteps];
    {
      const int r = row0 + c < rows ? row0 + c : 0, member = (int)a.share_div.div((uint32_t)r);
      const T* p = (const T*)a.q + (int64_t)(first + member) * a.qt + (int64_t)(hk * a.share + r - member * a.share) * a.qh;
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
        const int d = 16 * s + 8 * h;
        u32x4 w = *reinterpret_cast<const u32x4*>(p + (d < dim ? d : 0));
        if (d >= dim) w = (u32x4){0u, 0u, 0u, 0u};
        if (a.scale < 0.f) w ^= 0x80008000u;  // a negative scale turns the queries, so that scores rise with their products
        q[s] = __builtin_bit_cast(x8, w);
      }
    }

    f32x16 acc[kOut];
#pragma unroll
    for (int i = 0; i < kOut; i++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][e] = 0.f;
    float m = -INFINITY, l = 0.f;

    // (Offsets are worked out anew for each tile: kept in registers over the loop, they would be most of them.)
    const auto anew = [](int x) {
      asm volatile("" : "+v"(x));
      return x;
    };
    const auto keys_at = [&](int tile) { return (tile & 1) * kPlane; };
    const auto values_at = [&](int tile) { return (2 + (tile & 1)) * kPlane; };
    const auto place_of = [&](int tile, int key) { return place[(tile - begin) / kBlock & 1][(tile - begin) % kBlock * kKeys + key]; };
    const auto there_of = [&](int tile, int part) { return there[(tile - begin) / kBlock & 1][(tile - begin) % kBlock * kHalves + part]; };
    // Chunk g (16 bytes) of key r stands at g ^ (r's low bits): a read of K takes one chunk of 16 rows, one of V 64 bytes of four.
    const auto swap = [](int r) { return (D == 64 ? (r >> 1 & 1) << 2 | (r >> 2 & 3) : (r & 3) << 2 | (r >> 2 & 3)) * 16; };

    // 16-bit caches: copies from memory to LDS. Copy j of a wave fills 1 KB, lane i its 16 bytes at 16 i: the row's chunk that stands there.
    // A key that is not there, and elements past dim, are zeros (0 * NaN is NaN).
    const uint64_t zeros = (uint64_t)kZeros;
    uint64_t from[kCopies];  // of the copies of a tile's keys; its values are at the same offsets
    const auto prepare = [&](int tile) {
      const int i = anew(threadIdx.x) & 63;
#pragma unroll
      for (int j = 0; j < kCopies; j++) {
        const int key = (wave * kCopies + j) * (64 / kRowLanes) + i / kRowLanes, d = ((i % kRowLanes * 16) ^ swap(key)) / 2;
        const int64_t at = place_of(tile, key);
        from[j] = ((at >= 0) & (d < dim)) ? (uint64_t)(a.k + 2 * (at + d)) : zeros;
      }
    };
    const auto copy = [&](int to, int64_t plane, int first = 0, int last = 64) {
#pragma unroll
      for (int j = 0; j < kCopies; j++) {
        if (j < first || j >= last) continue;
        const uint64_t p = from[j] == zeros ? zeros : from[j] + plane;
        copy16((uint32_t)(uintptr_t)(lds_ptr_t)(lds + to) + (wave * kCopies + j) * 1024, (const void*)p);
      }
    };
    const auto copy_keys = [&](int tile) { copy(keys_at(tile), 0); };
    const auto copy_values = [&](int tile) { copy(values_at(tile), a.v - a.k); };
    // E4M3 caches: piece i of a thread, row (t + kThreads i) / kPieces, goes through registers, where it becomes 16-bit values.
    struct {
      u32x4 k[kLoads], v[kLoads];
      uint32_t ke[kLoads], ve[kLoads];
    } next;
    const auto load = [&](int k_tile, int v_tile) {
      const int t = anew(threadIdx.x), d = (t % kPieces) * 16;
      if (!kAll && t >= kKeys * kPieces) return;
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const int key = t / kPieces + i * (kThreads / kPieces);
        const auto offset = [&](int tile) {
          const int64_t p = place_of(tile, key);
          return p >= 0 && d < dim ? p + d : 0;  // others: the cache's first row, memory that is there
        };
        if (k_tile < end) {
          const int64_t from = offset(k_tile);
          next.k[i] = *reinterpret_cast<const u32x4*>(a.k + from), next.ke[i] = a.ks[from >> 5];
        }
        if (v_tile < end) {
          const int64_t from = offset(v_tile);
          next.v[i] = *reinterpret_cast<const u32x4*>(a.v + from), next.ve[i] = a.vs[from >> 5];
        }
      }
    };
    const auto stage = [&](int k_tile, int v_tile) {
      const int t = anew(threadIdx.x), g = (t % kPieces) * 32;
      if (!kAll && t >= kKeys * kPieces) return;
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const int key = t / kPieces + i * (kThreads / kPieces);
        const auto put = [&](int tile, int to, u32x4 w, uint32_t e) {
          if (tile >= end) return;
          const bool ok = g < 2 * dim && (there_of(tile, key / 64) >> (key % 64) & 1);
          const u32x4 none = {0u, 0u, 0u, 0u}, x = widen<T>((u32x2){w[0], w[1]}, e), y = widen<T>((u32x2){w[2], w[3]}, e);
          *reinterpret_cast<u32x4*>(lds + to + key * kPitch + (g ^ swap(key))) = ok ? x : none;
          *reinterpret_cast<u32x4*>(lds + to + key * kPitch + ((g + 16) ^ swap(key))) = ok ? y : none;
        };
        put(k_tile, keys_at(k_tile), next.k[i], next.ke[i]);
        put(v_tile, values_at(v_tile), next.v[i], next.ve[i]);
      }
    };
    // A lane's place in K: row c, chunk h of a step's two. In V by transposing reads: lane i of 16 names key i / 4 (and 4 h) and four of
    // its group's 16 columns, and gets column i of the four keys.
    const int v_key = 4 * h + (lane & 15) / 4, key0 = 64 * half;
    const int k_at = (key0 + c) * kPitch + ((16 * h) ^ swap(c));
    const int v_at = (key0 + v_key) * kPitch + ((32 * ((lane >> 4) & 1) + 8 * (lane & 3)) ^ swap(v_key));  // 8 keys on: 32 bytes swapped
    const float f = (CAP ? 1.f : fabsf(a.scale)) * kLog2e;  // a score's, in steps of its exponent

    // S^T of a tile, 32 keys at a time: element e of a lane is key 8 (e / 4) + 4 h + e % 4 of them, row c.
    f32x16 s[2];
    const auto score = [&](int tile) {
      const int from = anew(k_at) + keys_at(tile);
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 16; e++) s[u][e] = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; st++) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const x8 w = *reinterpret_cast<const x8*>(lds + (from ^ (32 * st)) + 32 * kPitch * u);
          s[u] = Vec<T>::mfma(w, q[st], s[u]);
        }
      }
    };
    // The scores become probabilities, as operands of 16 keys each: a lane's eight are 4 h + {0 .. 3, 8 .. 11}. The reference m of their exponents is
    // a maximum that follows the rows' own by kSlack at most: with 32 rows one would grow at nearly every tile.
    x8 p[4], rest[4];
    const auto soften = [&](int tile, auto step) {
      const unsigned long long mask = there_of(tile, half);
      if constexpr (CAP) {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int e = 0; e < 16; e++) s[u][e] = soft_cap(s[u][e] * fabsf(a.scale), a.softcap);
      }
      float by = f;
      if (mask != ~0ull) {  // scaled first: a scale of 0 times a masked score would be NaN
        by = 1.f;
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const uint32_t mine = (uint32_t)(mask >> 32 * u) >> 4 * h;
#pragma unroll
          for (int e = 0; e < 16; e++) s[u][e] = mine >> (8 * (e / 4) + e % 4) & 1u ? s[u][e] * f : -INFINITY;
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 16; e++) top = fmaxf(top, s[u][e]);
      top *= by;
      if (__any(top > m + kSlack)) {
        const auto r = __builtin_amdgcn_permlane32_swap(fbits(top), fbits(top), false, false);
        top = fmaxf(fmaxf(bitsf(r[0]), bitsf(r[1])), m);
        const float w = __builtin_amdgcn_exp2f(m - finite_or_zero(top));
        l *= w, m = top;
#pragma unroll
        for (int i = 0; i < kOut; i++) acc[i] *= w;
      }
      const float ref = kShift - finite_or_zero(m);
#pragma unroll
      for (int st = 0; st < 4; st++) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          x[e] = __builtin_amdgcn_exp2f(fmaf(s[st / 2][8 * (st % 2) + e], by, ref));
          l += x[e];
        }
        Vec<T>::split(x, p[st], rest[st]);
        step(st);
      }
#pragma unroll
      for (int st = 0; st < 4; st++) asm volatile("" : "+v"(p[st]), "+v"(rest[st]));  // here, and not where they are used
      asm volatile("" : "+v"(l));
    };
    // out^T += V^T P^T
    const auto add_values = [&](int tile, auto step) {
      const int from = anew(v_at) + values_at(tile);
#pragma unroll
      for (int st = 0; st < 4; st++) {
        constexpr int kSome = kOut < 4 ? kOut : 4;  // accumulators whose values are read together
#pragma unroll
        for (int i0 = 0; i0 < kOut; i0 += kSome) {
          union {
            s16x4 half[2];
            x8 whole;
          } w[kSome];
#pragma unroll
          for (int i = 0; i < kSome; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
              w[i].half[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds + (from ^ (64 * (i0 + i) + 32 * j)) + (16 * st + 8 * j) * kPitch));
#pragma unroll
          for (int i = 0; i < kSome; i++) acc[i0 + i] = Vec<T>::mfma(w[i].whole, rest[st], acc[i0 + i]);
#pragma unroll
          for (int i = 0; i < kSome; i++) acc[i0 + i] = Vec<T>::mfma(w[i].whole, p[st], acc[i0 + i]);
        }
        step(st);
        if (st == 1) __builtin_amdgcn_sched_barrier(0);
      }
    };
    const auto nothing = [](int) {};

    // Where a SIMD has two waves, each has a phase of the vector units, the softmax, and one of the matrix cores, a tile's values and the next
    // one's scores, and the two waves take turns at them: the halves have loops of their own with the same barriers, a phase apart. Keys and
    // values are used for two phases and are on their way for two. (Waves without rows go along; the other SIMDs do not notice.)
    int page = 0;
    // The places of the next block of tiles. Its first one's keys are fetched two tiles ahead, so they are written three ahead, with barriers between.
    static_assert(kBlock == 4, "look_up");
    const auto look_up = [&](int tile) {
      if ((tile - begin) % kBlock == 0) page = page_of((tile - begin) / kBlock + 1);
      if ((tile - begin) % kBlock == 1) put_place((tile - begin) / kBlock + 1, page);
    };

    __syncthreads();  // the unit before is done with what is shared here
    put_place(0, page0);
    __syncthreads();
    if constexpr (kHalves == 1) {
      if constexpr (MX8) {
        load(begin, begin);
        stage(begin, begin);
      } else {
        prepare(begin);
        copy_keys(begin), copy_values(begin);
        wait_memory<0>();
      }
      barrier();
      for (int tile = begin; tile < end; tile++) {
        look_up(tile);
        if constexpr (MX8) {
          load(tile + 1, tile + 1);
        } else if (tile + 1 < end) {
          prepare(tile + 1);
          copy_keys(tile + 1), copy_values(tile + 1);
        }
        score(tile);
        soften(tile, nothing);
        add_values(tile, nothing);
        if constexpr (MX8) stage(tile + 1, tile + 1);
        else wait_memory<0>();
        barrier();
      }
    } else {
      if constexpr (MX8) {
        load(begin, begin);
        stage(begin, begin);
        load(begin + 1, end);
        stage(begin + 1, end);
      } else {
        prepare(begin);
        copy_keys(begin), copy_values(begin);
        if (begin + 1 < end) {
          prepare(begin + 1);
          copy_keys(begin + 1);
        }
        wait_memory<0>();
      }
      barrier();
      const auto first_phase = [&](int tile) {
        look_up(tile);
        if constexpr (MX8) load(tile + 2, tile + 1);
      };
      const auto between = [&](int tile) {
        if constexpr (!MX8) wait_memory<0>();  // the next tile's keys and this one's values, on their way since the last phase
        barrier();
        if constexpr (MX8) stage(tile + 2, tile + 1);
      };
      // The second phase's copies, a few between other work: a CU takes 64 bytes a clock, and all at once they would hold the waves up. The
      // next tile's values have the places that its keys had a turn ago.
      const auto copies = [&](int tile) {
        return [&, tile](int step) {
          if constexpr (MX8) return;
          constexpr int kHalf = kCopies / 2;
          if (step < 2 && tile + 1 < end) copy(values_at(tile + 1), a.v - a.k, step * kHalf, (step + 1) * kHalf);
          if (step >= 2 && tile + 2 < end) {
            if (step == 2) prepare(tile + 2);
            copy(keys_at(tile + 2), 0, (step - 2) * kHalf, (step - 1) * kHalf);
          }
        };
      };
      if (half == 0) {
        score(begin);
        for (int tile = begin; tile < end; tile++) {
          first_phase(tile);
          soften(tile, nothing);
          between(tile);
          add_values(tile, copies(tile));
          score(tile + 1);  // (of the last one: not used)
          barrier();
        }
      } else {
        first_phase(begin);
        score(begin);
        between(begin);
        soften(begin, copies(begin));
        barrier();
        for (int tile = begin + 1; tile < end; tile++) {
          first_phase(tile);
          add_values(tile - 1, nothing);
          score(tile);
          between(tile);
          soften(tile, copies(tile));
          barrier();
        }
        add_values(end - 1, nothing);
      }
      __syncthreads();
    }

    // The two halves of the keys join in LDS, where tiles are no longer needed, and the rows' results go out.
    {
      const auto r = __builtin_amdgcn_permlane32_swap(fbits(l), fbits(l), false, false);
      l = bitsf(r[0]) + bitsf(r[1]);
      const int lane = anew(threadIdx.x) & 63, c = lane & 31, h = lane >> 5, width = anew(dim);
      f32x4* const shared_acc = reinterpret_cast<f32x4*>(lds) + row_wave * 8 * D + h * 32 + c;  // [D / 4][32]
      if constexpr (kHalves == 2) {
        if (half == 1) {
          if (h == 0) stats[row_wave][c] = float2{m, l};
#pragma unroll
          for (int i = 0; i < kOut; i++)
#pragma unroll
            for (int g = 0; g < 4; g++) shared_acc[(8 * i + 2 * g) * 32] = (f32x4){acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
        }
        __syncthreads();
      }
      if (half == 0 && row0 + c < rows) {
        float own = 1.f, other = 0.f;
        if constexpr (kHalves == 2) {
          const float2 o = stats[row_wave][c];
          const float top = fmaxf(m, o.x), ref = finite_or_zero(top);
          own = __builtin_amdgcn_exp2f(m - ref), other = __builtin_amdgcn_exp2f(o.x - ref);
          m = top, l = l * own + o.y * other;
        }
        float* const out = a.partial + slot;
        f32x4* const quads = reinterpret_cast<f32x4*>(out) + h * kPrefixRows + c;
#pragma unroll
        for (int i = 0; i < kOut; i++)
#pragma unroll
          for (int g = 0; g < 4; g++) {
            f32x4 v = {acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
            if constexpr (kHalves == 2) v = v * own + shared_acc[(8 * i + 2 * g) * 32] * other;
            if (32 * i + 8 * g + 4 * h < width) quads[(8 * i + 2 * g) * kPrefixRows] = v;
          }
        if (h == 0) *reinterpret_cast<float2*>(out + kPrefixRows * width + 2 * c) = float2{m, l};
      }
    }
  }
}

// ---- host -----------------------------------------------------------------------------------

constexpr int kCUs = 256;
int padded(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
constexpr int kWgs = kCUs;  // one to a CU

// A workspace: the decode kernel's (its counters first, whatever the shape), the rows' places and starts, the units, the splits.
struct Space {
  size_t rows_at, starts_at, units_at, splits_at, bytes;
};

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

bool sizes_ok(int groups, int max_shared) { return groups >= 0 && groups <= kMaxGroups && max_shared >= 0; }

// Whether there may be enough to share: a pass of its own and the joining of its results take some 12 us, in which the decode kernel reads 64 MB
// (4 rows behind 992 positions of 8 x 128 fp16, 12 MB that need not be read again: 11.5 us without, 20 with). A turn of 128 keys takes as long for few
// rows as for 128, which is not weighed: 16 groups of 4 rows behind 4096 positions of 8 x 128 take 90 us and 154 without (E4M3: 82 and 82), of 2 rows 80
// and 75 (E4M3: 82 and 49).
bool worth(const mxkv_cache* c, int seqs, int groups, int max_len, int max_shared) {
  const int shared = std::min(max_len, max_shared), again = std::max(0, seqs - groups);
  return groups > 0 && shared >= kLeastShared && (double)again * shared * c->heads * c->dim * (c->fmt == MX_E4M3 ? 2 : 4) >= (double)(64 << 20);
}

Space space_for(const mxkv_cache* c, int seqs, int q_heads, int groups, int max_len) {
  // units are at most those of full rows and one more of each group and head; split w + u has w below the shares and u below the units
  const size_t share = q_heads / c->heads, units = (size_t)c->heads * ((size_t)seqs * share / kRows + groups);
  Space s;
  s.rows_at = std::max(kDecodeCounterBytes, up16(decode_workspace(c, seqs, q_heads, max_len, 0)));
  s.starts_at = s.rows_at + 16 * (size_t)seqs;
  s.units_at = up16(s.starts_at + 4 * (size_t)seqs);
  s.splits_at = up16(s.units_at + 8 * units);
  s.bytes = s.splits_at + (kWgs + units) * kPrefixSlots * (size_t)prefix_slot_floats(c->dim) * 4;
  return s;
}

template <int D, typename T, bool MX8>
void launch(const Args& a, hipStream_t st) {
  const size_t lds = lds_of(D) + 4 * plan_ints(a.groups);
  if (a.softcap > 0.f) hipLaunchKernelGGL((prefix_kernel<D, T, MX8, true>), dim3((unsigned)a.wgs), dim3(threads_of(D)), lds, st, a);
  else hipLaunchKernelGGL((prefix_kernel<D, T, MX8, false>), dim3((unsigned)a.wgs), dim3(threads_of(D)), lds, st, a);
}

template <typename T, bool MX8>
void launch_dim(const Args& a, hipStream_t st) {
  const int D = padded(a.dim);
  if (D == 64) launch<64, T, MX8>(a, st);
  else if (D == 128) launch<128, T, MX8>(a, st);
  else launch<256, T, MX8>(a, st);
}

}  // namespace

extern "C" size_t mxattn_prefix_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int groups, int max_len, int max_shared) {
  if (!cache || check_geometry(cache) || !sizes_ok(groups, max_shared) || !decode_sizes_ok(cache, seqs, q_heads, max_len, 0) || seqs == 0) return 0;
  if (!worth(cache, seqs, groups, max_len, max_shared)) return decode_workspace(cache, seqs, q_heads, max_len, 0);
  return space_for(cache, seqs, q_heads, groups, max_len).bytes;
}

extern "C" int mxattn_prefix_run(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse, const mxkv_table* table,
                                 const int32_t* lengths, const mxattn_groups* groups, int max_len, const mxattn_opts* opts, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (int s = check_attention(cache, f, q, out, table, lengths, max_len, opts)) return s;
  if (!groups) return MX_ERR_NULL;
  if (opts->window != 0 || !sizes_ok(groups->count, groups->max_shared)) return MX_ERR_SHAPE;
  if (groups->count > 0 && (!groups->first || !groups->shared)) return MX_ERR_NULL;
  if (table->seqs == 0) return MX_OK;
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  const int seqs = table->seqs;
  const bool sharing = workspace && worth(cache, seqs, groups->count, max_len, groups->max_shared);
  const Space space = sharing ? space_for(cache, seqs, q->heads, groups->count, max_len) : Space{};
  if (!sharing || workspace_bytes < space.bytes)
    return sync_check(decode_launch(cache, f, q, out, lse, table, lengths, nullptr, max_len, opts, Prefix{}, workspace, workspace_bytes, st), st);
  uint8_t* at = (uint8_t*)workspace;
  Args a = {};
  a.k = (const uint8_t*)cache->k, a.v = (const uint8_t*)cache->v, a.ks = (const uint8_t*)cache->ks, a.vs = (const uint8_t*)cache->vs;
  a.q = q->data, a.qt = q->token_stride, a.qh = q->head_stride;
  a.table = table->pages, a.cols = table->cols, a.lengths = lengths, a.first = groups->first, a.shared = groups->shared;
  a.rows = (i32x4*)(at + space.rows_at), a.starts = (int32_t*)(at + space.starts_at), a.units = (int2*)(at + space.units_at), a.partial = (float*)(at + space.splits_at);
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.seqs = seqs, a.groups = groups->count, a.heads = cache->heads, a.share = q->heads / cache->heads, a.dim = cache->dim;
  a.pages = cache->pages, a.page_size = cache->page_size, a.max_len = max_len, a.max_shared = groups->max_shared;
  a.max_keys = (int)std::min<int64_t>((int64_t)table->cols * cache->page_size, INT32_MAX);
  a.wgs = kWgs, a.scale = opts->scale, a.softcap = opts->softcap;
  a.page_div = FastDiv((uint32_t)cache->page_size), a.share_div = FastDiv((uint32_t)a.share);
  const bool mx8 = cache->fmt == MX_E4M3;
  if (f == MX_F16 && mx8) launch_dim<_Float16, true>(a, st);
  else if (f == MX_F16) launch_dim<_Float16, false>(a, st);
  else if (mx8) launch_dim<__bf16, true>(a, st);
  else launch_dim<__bf16, false>(a, st);
  if (int s = launch_status()) return s;
  const Prefix prefix = {a.rows, a.units, a.partial};
  return sync_check(decode_launch(cache, f, q, out, lse, table, lengths, a.starts, max_len, opts, prefix, workspace, space.rows_at, st), st);
}
