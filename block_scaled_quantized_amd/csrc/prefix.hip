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
#include <algorithm>

#include "attention.h"

using namespace mx;

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 32 * kWaves;  // query rows of a workgroup
constexpr int kTile = 64;          // keys
constexpr int kMaxGroups = 1024, kMaxSplits = 64;
constexpr int kLeastTiles = 4;     // of a split
constexpr int kGroupsOfThread = kMaxGroups / kThreads;

struct Args {
  const uint8_t *k, *v, *ks, *vs;
  const void* q;
  const int32_t *table, *lengths, *first, *shared;
  i32x4* rows;       // written for the decode kernel, with starts
  int32_t* starts;
  float* partial;
  int64_t qt, qh, page_stride, head_stride, slot_stride;
  int seqs, groups, heads, share, dim, cols, pages, max_len, max_keys, max_shared, wgs, page_size;
  float scale, softcap;
  FastDiv page_div, share_div;
};

MX_DEV int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// What every workgroup works out for itself from the lengths: the groups' shared tiles and how they are split.
struct Plan {
  int first[kMaxGroups + 1];   // sequences
  int items[kMaxGroups + 1];   // work items before the group's
  int slots[kMaxGroups];       // slots before the group's
  int end[kMaxGroups];         // shared positions, whole tiles
  int members[kMaxGroups];     // with positions; then splits
  unsigned long long work;
  int falls;                   // whether the firsts do, which makes them no groups
  int wave_items[kWaves], wave_slots[kWaves];
};

MX_DEV int length_of(const Args& a, int b) { return max(0, min(min(a.lengths[b], a.max_len), a.max_keys)); }

// The group of sequence b, -1 if none.
MX_DEV int group_of(const Plan& p, int groups, int b) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= b) lo = mid;
    else hi = mid;
  }
  return p.first[lo] <= b && b < p.first[lo + 1] ? lo : -1;
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
  int rows, tiles, tiles32, keys, splits;  // of one group: query rows of a cache head, their tiles, tiles of keys
};
MX_DEV Shape shape_of(const Args& a, const Plan& p, int g) {
  Shape s;
  s.rows = max(0, p.first[g + 1] - p.first[g]) * a.share;
  s.tiles = ceil_div(s.rows, kRows), s.tiles32 = ceil_div(s.rows, kPrefixRows);
  s.keys = p.end[g] / kTile, s.splits = p.members[g];
  return s;
}

MX_DEV int plan(const Args& a, Plan& p) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  for (int g = t; g <= a.groups; g += kThreads) p.first[g] = max(0, min(a.first[g], a.seqs));
  for (int g = t; g < a.groups; g += kThreads) p.end[g] = max(0, min(a.shared[g], a.max_shared)), p.members[g] = 0;
  if (t == 0) p.work = 0, p.falls = 0;
  __syncthreads();
  for (int g = t; g < a.groups; g += kThreads)
    if (p.first[g + 1] < p.first[g]) p.falls = 1;
  // rows without positions do not count; a beginning that no two rows share is not worth its own pass
  for (int b = t; b < a.seqs; b += kThreads) {
    const int n = length_of(a, b), g = group_of(p, a.groups, b);
    if (g >= 0 && n > 0) atomicMin(&p.end[g], n), atomicAdd(&p.members[g], 1);
  }
  __syncthreads();
  unsigned long long work = 0;
  for (int g = t; g < a.groups; g += kThreads) {
    p.end[g] = p.members[g] < 2 || p.falls ? 0 : p.end[g] & ~(kTile - 1);
    const Shape s = shape_of(a, p, g);
    work += (unsigned long long)s.tiles * s.keys;
  }
  atomicAdd(&p.work, work * a.heads);
  __syncthreads();
  const unsigned long long per = max((unsigned long long)kLeastTiles, (p.work + a.wgs - 1) / a.wgs);
  int items[kGroupsOfThread], slots[kGroupsOfThread], all_items = 0, all_slots = 0;
#pragma unroll
  for (int i = 0; i < kGroupsOfThread; i++) {
    const int g = t * kGroupsOfThread + i;
    items[i] = all_items, slots[i] = all_slots;
    if (g >= a.groups) continue;
    const Shape s = shape_of(a, p, g);
    int splits = (int)min((unsigned long long)kMaxSplits, (s.keys + per - 1) / per);
    if (splits > 1) splits = ceil_div(s.keys, ceil_div(s.keys, splits));  // whole tiles each, none empty
    p.members[g] = splits;
    all_items += a.heads * s.tiles * splits, all_slots += a.heads * s.tiles32 * splits;
  }
  const int upto_items = (int)wave_scan((uint32_t)all_items), upto_slots = (int)wave_scan((uint32_t)all_slots);
  if (lane == 63) p.wave_items[wave] = upto_items, p.wave_slots[wave] = upto_slots;
  __syncthreads();
  int before_items = upto_items - all_items, before_slots = upto_slots - all_slots, total = 0;
  for (int w = 0; w < kWaves; w++) {
    if (w < wave) before_items += p.wave_items[w], before_slots += p.wave_slots[w];
    total += p.wave_items[w];
  }
#pragma unroll
  for (int i = 0; i < kGroupsOfThread; i++) {
    const int g = t * kGroupsOfThread + i;
    if (g < a.groups) p.items[g] = before_items + items[i], p.slots[g] = before_slots + slots[i];
  }
  if (t == 0) p.items[a.groups] = total;
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = t; b < a.seqs; b += kThreads) {
      const int g = group_of(p, a.groups, b);
      const bool in = g >= 0 && p.end[g] > 0 && length_of(a, b) > 0;
      const Shape s = shape_of(a, p, max(g, 0));
      a.starts[b] = in ? p.end[g] : 0;
      a.rows[b] = in ? (i32x4){p.slots[g], s.splits, s.tiles32, (b - p.first[g]) * a.share} : (i32x4){0, 0, 0, 0};
    }
  }
  return total;
}

// Two waves per SIMD, but for heads above 128, whose accumulators and queries are twice as many.
constexpr int waves_per_simd(int D) { return D == 256 ? 1 : 2; }

// D: 64, 128 or 256, the head size rounded up. T: type of q and the arithmetic. MX8: E4M3 cache.
template <int D, typename T, bool MX8>
__global__ __launch_bounds__(kThreads, waves_per_simd(D)) void prefix_kernel(Args a) {
  typedef typename Vec<T>::x8 x8;
  constexpr float kShift = Vec<T>::kShift;
  constexpr int kSteps = D / 16, kOut = D / 32;
  constexpr int kPieces = MX8 ? D / 16 : D / 8;                      // 16-byte pieces of a key's row in the cache
  constexpr int kLoads = kTile * kPieces / kThreads;                 // of a thread, of keys and of values
  constexpr int kPitch = 2 * D;                                      // bytes of a key's row in LDS
  __shared__ Plan groups;
  __shared__ __attribute__((aligned(16))) char lds_k[kTile * kPitch], lds_v[kTile * kPitch];
  __shared__ int64_t place[2][kTile];            // of the keys of two tiles, element offsets
  __shared__ unsigned long long there[2];        // which of them have a page
  __shared__ int chosen[8];

  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), c = lane & 31, h = lane >> 5;
  const int dim = a.dim;
  const int total = uniform(plan(a, groups));
  // each XCD takes a run of the items: those that read the same keys are next to each other
  int first_item = blockIdx.x;
  if (gridDim.x % 8 == 0) first_item = (blockIdx.x & 7) * (gridDim.x / 8) + (blockIdx.x >> 3);

  for (int item = first_item; item < total; item += gridDim.x) {
    __syncthreads();  // the one before is done with what is shared here
    if (t == 0) {
      int lo = 0, hi = a.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (groups.items[mid] <= item) lo = mid;
        else hi = mid;
      }
      const Shape s = shape_of(a, groups, lo);
      const int in = item - groups.items[lo], part = in / s.tiles;  // [head][split][tile]
      chosen[0] = groups.first[lo], chosen[1] = s.rows, chosen[2] = s.tiles32, chosen[3] = s.keys, chosen[4] = s.splits;
      chosen[5] = in - part * s.tiles, chosen[6] = part, chosen[7] = groups.slots[lo];
    }
    __syncthreads();
    const int first = uniform(chosen[0]), rows = uniform(chosen[1]), tiles32 = uniform(chosen[2]), keys = uniform(chosen[3]), splits = uniform(chosen[4]);
    const int row_tile = uniform(chosen[5]), part = uniform(chosen[6]), hk = part / splits, split = part - hk * splits;
    const int slot0 = uniform(chosen[7]) + (hk * tiles32 + row_tile * kWaves + wave) * splits + split;
    const int each = ceil_div(keys, splits), begin = split * each, end = min(keys, begin + each);
    const int64_t head_at = (int64_t)hk * a.head_stride;
    const int32_t* table = a.table + (int64_t)first * a.cols;
    const int row0 = row_tile * kRows + 32 * wave;
    const bool active = row0 < rows;

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
        q[s] = __builtin_bit_cast(x8, w);
      }
    }

    f32x16 acc[kOut];
#pragma unroll
    for (int i = 0; i < kOut; i++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][e] = 0.f;
    float m = -INFINITY, l = 0.f;

    const auto page_of = [&](int tile) -> int { return t < kTile ? table[min((int)a.page_div.div((uint32_t)(tile * kTile + t)), a.cols - 1)] : -1; };
    const auto put_place = [&](int tile, int page) {
      if (t >= kTile) return;
      const int key = tile * kTile + t;
      const bool ok = page >= 0 && page < a.pages;
      place[tile & 1][t] = ok ? head_at + page * a.page_stride + (key - (int)a.page_div.div((uint32_t)key) * a.page_size) * a.slot_stride : -1;
      const unsigned long long mask = __ballot(ok);
      if (t == 0) there[tile & 1] = mask;
    };
    // piece i of a thread: row (t + kThreads i) / kPieces, piece (t + kThreads i) % kPieces of it
    u32x4 next_k[kLoads], next_v[kLoads];
    uint32_t next_ke[kLoads], next_ve[kLoads];
    // (Offsets are worked out anew for each tile: kept in registers over the loop, they would be most of them.)
    const auto anew = [](int x) {
      asm volatile("" : "+v"(x));
      return x;
    };
    const auto load = [&](int tile) {
      const int t = anew(threadIdx.x), d = (t % kPieces) * (MX8 ? 16 : 8);
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const int64_t p = place[tile & 1][t / kPieces + i * (kThreads / kPieces)];
        // a key without a page has the cache's first row, and elements past dim that row's first: memory that is there
        const int64_t from = p >= 0 && d < dim ? p + d : 0;
        if constexpr (MX8) {
          next_k[i] = *reinterpret_cast<const u32x4*>(a.k + from), next_ke[i] = a.ks[from >> 5];
          next_v[i] = *reinterpret_cast<const u32x4*>(a.v + from), next_ve[i] = a.vs[from >> 5];
        } else {
          next_k[i] = *reinterpret_cast<const u32x4*>((const T*)a.k + from);
          next_v[i] = *reinterpret_cast<const u32x4*>((const T*)a.v + from);
        }
      }
    };
    // Chunk g (16 bytes) of key r stands at g ^ (r's low bits): a read of K takes one chunk of 16 rows, one of V 64 bytes of four.
    const auto k_swap = [](int r) { return (D == 64 ? (r >> 1) & 7 : r & 15) * 16; };
    const auto v_swap = [](int r) { return (D == 64 ? (r >> 1) & 1 : r & 3) * 64; };
    const auto stage = [&](unsigned long long mask) {
      const int t = anew(threadIdx.x), g = (t % kPieces) * (MX8 ? 32 : 16);
      const bool inside = g < 2 * dim;
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const int key = t / kPieces + i * (kThreads / kPieces), row = key * kPitch;
        const bool ok = inside && (mask >> key & 1);  // others: zeros, as 0 * NaN is NaN
        const auto put = [&](char* to, int at, u32x4 x) { *reinterpret_cast<u32x4*>(to + row + at) = ok ? x : (u32x4){0u, 0u, 0u, 0u}; };
        if constexpr (MX8) {
          const u32x4 x = next_k[i], y = next_v[i];
          put(lds_k, g ^ k_swap(key), widen<T>((u32x2){x[0], x[1]}, next_ke[i]));
          put(lds_k, (g + 16) ^ k_swap(key), widen<T>((u32x2){x[2], x[3]}, next_ke[i]));
          put(lds_v, g ^ v_swap(key), widen<T>((u32x2){y[0], y[1]}, next_ve[i]));
          put(lds_v, (g + 16) ^ v_swap(key), widen<T>((u32x2){y[2], y[3]}, next_ve[i]));
        } else {
          put(lds_k, g ^ k_swap(key), next_k[i]);
          put(lds_v, g ^ v_swap(key), next_v[i]);
        }
      }
    };
    // A lane's place in K: row c, chunk h of a step's two. In V by transposing reads: lane i of 16 names key i / 4 (and 4 h) and four of
    // its group's 16 columns, and gets column i of the four keys.
    const int v_key = 4 * h + (lane & 15) / 4;
    const int k_at = c * kPitch + ((16 * h) ^ k_swap(c)), v_at = v_key * kPitch + ((32 * ((lane >> 4) & 1) + 8 * (lane & 3)) ^ v_swap(v_key));

    put_place(begin, page_of(begin));
    if (begin + 1 < end) put_place(begin + 1, page_of(begin + 1));
    __syncthreads();
    load(begin);
    for (int tile = begin; tile < end; tile++) {
      const unsigned long long mask = there[tile & 1];
      const int page = tile + 2 < end ? page_of(tile + 2) : -1;
      __syncthreads();  // the tile before is used up, and this one's places are read
      stage(mask);
      if (tile + 2 < end) put_place(tile + 2, page);
      __syncthreads();
      if (tile + 1 < end) load(tile + 1);
      if (!active) continue;

      // S^T of both halves of 32 keys: element e of a lane is key 8 (e / 4) + 4 h + e % 4 of the half, row c
      f32x16 s[2];
      const int k_from = anew(k_at), v_from = anew(v_at);
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 16; e++) s[u][e] = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; st++) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const x8 w = *reinterpret_cast<const x8*>(lds_k + (k_from ^ (32 * st)) + 32 * kPitch * u);
          s[u] = Vec<T>::mfma(w, q[st], s[u]);
        }
        if (st % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // a few reads at a time: all of them at once would spill
      }
      if (a.softcap > 0.f) {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int e = 0; e < 16; e++) s[u][e] = kLog2e * soft_cap(s[u][e] * a.scale, a.softcap);
      } else {
        const float f = a.scale * kLog2e;
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int e = 0; e < 16; e++) s[u][e] *= f;
      }
      if (mask != ~0ull) {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int e = 0; e < 16; e++)
            if (!((uint32_t)(mask >> 32 * u) >> 4 * h >> (8 * (e / 4) + e % 4) & 1u)) s[u][e] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 16; e++) top = fmaxf(top, s[u][e]);
      if (__any(top > m)) {  // seldom after the first tiles
        const auto r = __builtin_amdgcn_permlane32_swap(fbits(top), fbits(top), false, false);
        top = fmaxf(fmaxf(bitsf(r[0]), bitsf(r[1])), m);
        const float f = __builtin_amdgcn_exp2f(m - finite_or_zero(top));
        l *= f, m = top;
#pragma unroll
        for (int i = 0; i < kOut; i++) acc[i] *= f;
      }
      const float ref = finite_or_zero(m) - kShift;
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
          s[u][e] = __builtin_amdgcn_exp2f(s[u][e] - ref);
          l += s[u][e];
        }
      // out^T += V^T P^T, 16 keys at a time: a lane's eight are 16 st + 4 h + {0 .. 3, 8 .. 11}
#pragma unroll
      for (int st = 0; st < 4; st++) {
        __builtin_amdgcn_sched_barrier(0);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = s[st / 2][8 * (st % 2) + e];
        const x8 p = __builtin_bit_cast(x8, (u32x4){Vec<T>::cut(x[0], x[1]), Vec<T>::cut(x[2], x[3]), Vec<T>::cut(x[4], x[5]), Vec<T>::cut(x[6], x[7])});
        x8 rest;
#pragma unroll
        for (int e = 0; e < 8; e++) rest[e] = (T)fmaxf(x[e] - (float)p[e], Vec<T>::kLeast);
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
              w[i].half[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds_v + (v_from ^ (64 * (i0 + i))) + (16 * st + 8 * j) * kPitch));
#pragma unroll
          for (int i = 0; i < kSome; i++) acc[i0 + i] = Vec<T>::mfma(w[i].whole, rest, acc[i0 + i]);
#pragma unroll
          for (int i = 0; i < kSome; i++) acc[i0 + i] = Vec<T>::mfma(w[i].whole, p, acc[i0 + i]);
        }
      }
    }

    if (active) {
      const auto r = __builtin_amdgcn_permlane32_swap(fbits(l), fbits(l), false, false);
      l = bitsf(r[0]) + bitsf(r[1]);
      float* out = a.partial + slot0 * prefix_slot_floats(dim);
      const int lane = anew(threadIdx.x) & 63, c = lane & 31, h = lane >> 5;
      if (row0 + c < rows) {
#pragma unroll
        for (int i = 0; i < kOut; i++)
#pragma unroll
          for (int g = 0; g < 4; g++) {
            const int d = 32 * i + 8 * g + 4 * h;
            const f32x4 v = {acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
            if (d < dim) *reinterpret_cast<f32x4*>(out + (d * (kPrefixRows / 4) + c) * 4) = v;
          }
        if (h == 0) out[kPrefixRows * dim + 2 * c] = m, out[kPrefixRows * dim + 2 * c + 1] = l;
      }
    }
  }
}

// ---- host -----------------------------------------------------------------------------------

constexpr int kCUs = 256;
int padded(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
int workgroups(int dim) { return kCUs * waves_per_simd(padded(dim)); }

// A workspace: the decode kernel's (its counters first, whatever the shape), the rows' places and starts, the slots.
struct Space {
  size_t rows_at, starts_at, slots_at, bytes;
};

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

bool sizes_ok(int groups, int max_shared) { return groups >= 0 && groups <= kMaxGroups && max_shared >= 0; }

// Whether there is anything to share.
bool worth(int seqs, int groups, int max_len, int max_shared) { return seqs >= 2 && groups > 0 && std::min(max_len, max_shared) >= kTile; }

Space space_for(const mxkv_cache* c, int seqs, int q_heads, int groups, int max_len) {
  Space s;
  s.rows_at = std::max(kDecodeCounterBytes, up16(decode_workspace(c, seqs, q_heads, max_len, 0)));
  s.starts_at = s.rows_at + 16 * (size_t)seqs;
  s.slots_at = up16(s.starts_at + 4 * (size_t)seqs);
  // Units (a group's cache head and 128 rows) are at most those of full tiles and one more of each group; their splits, as each but a
  // unit's last is full, at most the workgroups and the units. A split's 128 rows are at most four slots.
  const size_t share = q_heads / c->heads;
  const size_t units = (size_t)c->heads * ((size_t)seqs * share / kRows + groups);
  s.bytes = s.slots_at + (workgroups(c->dim) + units) * kWaves * (size_t)prefix_slot_floats(c->dim) * 4;
  return s;
}

template <int D, typename T>
void launch(const Args& a, bool mx8, hipStream_t st) {
  if (mx8) hipLaunchKernelGGL((prefix_kernel<D, T, true>), dim3((unsigned)a.wgs), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((prefix_kernel<D, T, false>), dim3((unsigned)a.wgs), dim3(kThreads), 0, st, a);
}

template <typename T>
void launch_dim(const Args& a, bool mx8, hipStream_t st) {
  const int D = padded(a.dim);
  if (D == 64) launch<64, T>(a, mx8, st);
  else if (D == 128) launch<128, T>(a, mx8, st);
  else launch<256, T>(a, mx8, st);
}

}  // namespace

extern "C" size_t mxattn_prefix_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int groups, int max_len, int max_shared) {
  if (!cache || check_geometry(cache) || !sizes_ok(groups, max_shared) || !decode_sizes_ok(cache, seqs, q_heads, max_len, 0) || seqs == 0) return 0;
  if (!worth(seqs, groups, max_len, max_shared)) return decode_workspace(cache, seqs, q_heads, max_len, 0);
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
  const bool sharing = workspace && worth(seqs, groups->count, max_len, groups->max_shared);
  const Space space = sharing ? space_for(cache, seqs, q->heads, groups->count, max_len) : Space{};
  if (!sharing || workspace_bytes < space.bytes)
    return sync_check(decode_launch(cache, f, q, out, lse, table, lengths, nullptr, max_len, opts, Prefix{}, workspace, workspace_bytes, st), st);
  uint8_t* at = (uint8_t*)workspace;
  Args a = {};
  a.k = (const uint8_t*)cache->k, a.v = (const uint8_t*)cache->v, a.ks = (const uint8_t*)cache->ks, a.vs = (const uint8_t*)cache->vs;
  a.q = q->data, a.qt = q->token_stride, a.qh = q->head_stride;
  a.table = table->pages, a.cols = table->cols, a.lengths = lengths, a.first = groups->first, a.shared = groups->shared;
  a.rows = (i32x4*)(at + space.rows_at), a.starts = (int32_t*)(at + space.starts_at), a.partial = (float*)(at + space.slots_at);
  a.page_stride = cache->page_stride, a.head_stride = kv_head_stride(cache), a.slot_stride = slot_stride(cache);
  a.seqs = seqs, a.groups = groups->count, a.heads = cache->heads, a.share = q->heads / cache->heads, a.dim = cache->dim;
  a.pages = cache->pages, a.page_size = cache->page_size, a.max_len = max_len, a.max_shared = groups->max_shared;
  a.max_keys = (int)std::min<int64_t>((int64_t)table->cols * cache->page_size, INT32_MAX);
  a.wgs = workgroups(cache->dim), a.scale = opts->scale, a.softcap = opts->softcap;
  a.page_div = FastDiv((uint32_t)cache->page_size), a.share_div = FastDiv((uint32_t)a.share);
  if (f == MX_F16) launch_dim<_Float16>(a, cache->fmt == MX_E4M3, st);
  else launch_dim<__bf16>(a, cache->fmt == MX_E4M3, st);
  if (int s = launch_status()) return s;
  const Prefix prefix = {a.rows, a.partial};
  return sync_check(decode_launch(cache, f, q, out, lse, table, lengths, a.starts, max_len, opts, prefix, workspace, space.rows_at, st), st);
}
