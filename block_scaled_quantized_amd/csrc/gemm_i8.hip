// gemm_i8.hip -- C = A B of 8-bit integers, A [M][K] with a scale per row (token), B stored [N][K] with a scale per row (output
// channel): C[m,n] = sa[m] sb[n] sum_k a[m,k] b[n,k] (+ bias[n], ReLU). The sums are exact 32-bit integers (K is bounded), so neither
// their order nor a split of K changes a result.
//
// Two kernels. For few rows the weights are read once and bound the time: a wave takes them from global memory straight to the
// matrix cores' registers (16x16x64), the waves of a workgroup share K. For more rows the matrix cores bound it: tiles go through LDS
// (direct global -> LDS copies, two slots of 128 bytes of K) to 32x32x32 instructions. K need not be a multiple of anything: bytes of A past
// K become zeros on the way, and a zero times whatever integer B holds there is zero.
#include <algorithm>

#include "kvcache.h"

using namespace mx;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kFar = 0x80000000u;  // an offset past every buffer: loads give 0
constexpr int kCounterBytes = 16384;    // of the workspace: a counter per tile that K is split of
constexpr int kMaxCounters = kCounterBytes / 4;
constexpr int kCUs = 256;

struct Args {
  const uint8_t *a, *b;
  const float *sa, *sb;
  const void* bias;
  void* c;
  uint32_t* counters;
  uint8_t* partial;
  int64_t lda, ldb, ldc;
  int M, N, K, relu, vector;  // vector: rows of C are 16-byte aligned
  int tiles_m, tiles_n, splits;
};

MX_DEV int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
MX_DEV rsrc_t resource(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, uniform((int)bytes), 0x00020000);
}
MX_DEV uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_ptr_t)p; }

// Bytes of rows first .. first + rows - 1, each up to its last 16-byte piece of K.
MX_DEV uint32_t extent(int rows, int64_t ld, int K) { return (uint32_t)((rows - 1) * ld + ((K + 15) & ~15)); }

template <typename T>
MX_DEV T finished(int sum, float scale, float bias, bool relu) {
  float v = (float)sum * scale + bias;
  if (relu) v = fmaxf(v, 0.f);
  return (T)v;
}

// Whether this workgroup is the last of n to arrive at a counter, which it takes back to zero. The caller's waves have written
// their partial sums past the caches; each waits for its stores before the barrier.
MX_DEV bool arrives_last(uint32_t* counter, int n, int* flag) {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) *flag = atomicInc(counter, (unsigned)(n - 1)) == (unsigned)(n - 1);
  __syncthreads();
  return uniform(*flag);
}
constexpr int kThrough = 17;  // sc0 sc1: partial sums cross XCDs

// ---- few rows ---------------------------------------------------------------------------------

// MT tiles of 16 rows of A, NT tiles of 16 rows of B. Lane l of a 16x16x64 instruction holds 16 bytes of row l % 16 of each
// operand, those of K-piece l / 16; B is the first operand, so that a lane ends with four neighbouring columns of C of one row.
template <typename T, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void rows_kernel(Args p) {
  constexpr int kStep = 64, kDeep = NT * MT >= 8 ? 1 : NT >= 4 ? 2 : 4;  // steps on their way
  __shared__ v4i sums[WAVES][MT * NT][64];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, rows = min(16 * NT, p.N - n0);
  const int steps = ceil_div(p.K, kStep), split = blockIdx.y;
  // K's steps split evenly; the waves take a split's steps in turn
  const int begin = (int)((int64_t)steps * split / p.splits), end = (int)((int64_t)steps * (split + 1) / p.splits);

  const rsrc_t ra = resource(p.a, extent(p.M, p.lda, p.K)), rb = resource(p.b + n0 * p.ldb, extent(rows, p.ldb, p.K));
  uint32_t at_a[MT], at_b[NT];
#pragma unroll
  for (int i = 0; i < MT; i++) at_a[i] = (uint32_t)(min(16 * i + r, p.M - 1) * p.lda) + 16u * q;  // rows past M repeat the last one, and are not written
#pragma unroll
  for (int i = 0; i < NT; i++) at_b[i] = (uint32_t)((16 * i + r) * p.ldb) + 16u * q;

  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = (v4i){0, 0, 0, 0};

  struct Step {
    v4i a[MT], b[NT];
  } ring[kDeep];
  const auto load = [&](Step& s, int step) {
    const uint32_t k = (uint32_t)step * kStep;
    const bool in = step < end && k + 16u * q < (uint32_t)p.K;
#pragma unroll
    for (int i = 0; i < NT; i++) s.b[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, in ? at_b[i] + k : kFar, 0, 2));
#pragma unroll
    for (int i = 0; i < MT; i++) s.a[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? at_a[i] + k : kFar, 0, 0));
  };
  const auto multiply = [&](Step& s, int step) {
    const int left = p.K - (step * kStep + 16 * q);  // bytes of this lane's piece that K has
    if (step * kStep + kStep > p.K && left < 16) {
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const int n = max(0, min(4, left - 4 * w));
          s.a[i][w] = n == 4 ? s.a[i][w] : (int)((uint32_t)s.a[i][w] & ((1u << (8 * n)) - 1u));
        }
    }
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.b[j], s.a[i], acc[i][j], 0, 0, 0);
  };
  int step = begin + wave;
#pragma unroll
  for (int d = 0; d < kDeep; d++) load(ring[d], step + d * WAVES);
  for (; step < end; step += kDeep * WAVES) {
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      multiply(ring[d], step + d * WAVES);  // a step past the end is of zeros
      load(ring[d], step + (d + kDeep) * WAVES);
    }
  }

#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) sums[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // item: four neighbouring columns of one row; neighbouring threads take neighbouring columns
  constexpr int kItems = MT * NT * 64, kThreads = 64 * WAVES, kEach = (kItems + kThreads - 1) / kThreads;
  v4i sum[kEach];
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    const int item = threadIdx.x + e * kThreads, quad = item % (4 * NT), m = item / (4 * NT);
    if (item >= kItems) break;
    const int tile = (m / 16) * NT + quad / 4, at = (quad % 4) * 16 + m % 16;
    sum[e] = sums[0][tile][at];
#pragma unroll
    for (int w = 1; w < WAVES; w++) sum[e] += sums[w][tile][at];
  }
  if (p.splits > 1) {
    const rsrc_t rp = resource(p.partial, (uint32_t)gridDim.x * p.splits * kItems * 16u);
    const uint32_t first = (uint32_t)blockIdx.x * p.splits * kItems * 16u;
#pragma unroll
    for (int e = 0; e < kEach; e++) {
      const int item = threadIdx.x + e * kThreads;
      if (item < kItems) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum[e]), rp, first + ((uint32_t)split * kItems + item) * 16u, 0, kThrough);
    }
    if (!arrives_last(p.counters + blockIdx.x, p.splits, &flag)) return;
    for (int o = 0; o < p.splits; o++) {
      if (o == split) continue;
#pragma unroll
      for (int e = 0; e < kEach; e++) {
        const int item = threadIdx.x + e * kThreads;
        if (item < kItems) sum[e] += __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rp, first + ((uint32_t)o * kItems + item) * 16u, 0, kThrough));
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    const int item = threadIdx.x + e * kThreads, quad = item % (4 * NT), m = item / (4 * NT), n = n0 + 4 * quad;
    if (item >= kItems || m >= p.M || n >= p.N) continue;
    const float sa = p.sa[m];
    T* c = (T*)p.c + m * p.ldc + n;
    typedef T x4 __attribute__((ext_vector_type(4)));
    x4 v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int at = min(n + i, p.N - 1);
      v[i] = finished<T>(sum[e][i], sa * p.sb[at], p.bias ? (float)((const T*)p.bias)[at] : 0.f, p.relu);
    }
    if (p.vector && n + 4 <= p.N) {
      *reinterpret_cast<x4*>(c) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < p.N) c[i] = v[i];
    }
  }
}

// ---- tiles ------------------------------------------------------------------------------------

// The fragments of one K-step of 32 bytes: FA tiles of 32 rows of A, FB of B, 4096 bytes apart. In one block with their wait, as the
// compiler would wait for every copy in flight before a read of LDS that it can see.
template <int FA, int FB>
MX_DEV void read_step(v4i (&a)[FA], v4i (&b)[FB], uint32_t at_a, uint32_t at_b) {
  static_assert(FA == 4 ? FB == 2 : FA == 2 && FB <= 2, "fragments");
  if constexpr (FA == 4) {
    asm volatile(
        "ds_read_b128 %4, %7\n"
        "ds_read_b128 %5, %7 offset:4096\n"
        "ds_read_b128 %0, %6\n"
        "ds_read_b128 %1, %6 offset:4096\n"
        "ds_read_b128 %2, %6 offset:8192\n"
        "ds_read_b128 %3, %6 offset:12288\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(a[2]), "=&v"(a[3]), "=&v"(b[0]), "=&v"(b[1])
        : "v"(at_a), "v"(at_b));
  } else if constexpr (FB == 2) {
    asm volatile(
        "ds_read_b128 %2, %5\n"
        "ds_read_b128 %3, %5 offset:4096\n"
        "ds_read_b128 %0, %4\n"
        "ds_read_b128 %1, %4 offset:4096\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(b[0]), "=&v"(b[1])
        : "v"(at_a), "v"(at_b));
  } else {
    asm volatile(
        "ds_read_b128 %2, %4\n"
        "ds_read_b128 %0, %3\n"
        "ds_read_b128 %1, %3 offset:4096\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(b[0])
        : "v"(at_a), "v"(at_b));
  }
}

// BM x BN tiles; WM x WN waves of (BM / WM) x (BN / WN) each. A slot holds 128 bytes of every row: chunk c (16 bytes) of row r at
// place c ^ ((r >> 1) & 7), so that the 16 rows that a quarter of a read touches lie on different banks.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, WM * WN == 8 ? 2 : 2) void tile_kernel(Args p) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, FA = BM / WM / 32, FB = BN / WN / 32;
  constexpr int kSlot = (BM + BN) * 128, kCopies = (BM + BN) / 8 / kWaves;  // copies of a wave: 8 rows each
  static_assert((BM / 8) % kWaves == 0, "a copy is of A or of B for all waves");
  constexpr int kCols = 32 * FB, kPitch = kCols * (int)sizeof(T) + 16;  // epilogue: 32 rows of a wave
  constexpr int kLds = std::max(2 * kSlot, kWaves * 32 * kPitch);
  __shared__ __attribute__((aligned(16))) char lds[kLds];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r32 = lane & 31, h = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;

  // Each XCD takes a run of tiles, in bands of 8 tile rows, so that what it runs at once shares operands in its L2.
  int id = blockIdx.x;
  const int wgs = gridDim.x, tiles = p.tiles_m * p.tiles_n;
  {
    const int each = wgs / 8, rest = wgs % 8, x = id & 7;
    id = x * each + min(x, rest) + (id >> 3);
  }
  const int split = id / tiles;
  id -= split * tiles;
  const int band = id / (8 * p.tiles_n), in_band = id - band * 8 * p.tiles_n, band_rows = min(8, p.tiles_m - 8 * band);
  const int tm = 8 * band + in_band % band_rows, tn = in_band / band_rows;
  const int m0 = tm * BM, n0 = tn * BN;

  const rsrc_t ra = resource(p.a + m0 * p.lda, extent(min(BM, p.M - m0), p.lda, p.K));
  const rsrc_t rb = resource(p.b + n0 * p.ldb, extent(min(BN, p.N - n0), p.ldb, p.K));
  const int slots = ceil_div(p.K, 128);
  const int begin = (int)((int64_t)slots * split / p.splits), end = (int)((int64_t)slots * (split + 1) / p.splits);

  // Copy j of a wave fills rows 8 (wave + kWaves j) .. + 7 of the slot; lane l chunk place l % 8 of row l / 8. Which chunk
  // that is depends on the row's bits 1 to 3, which all copies of a wave share.
  const int row8 = lane >> 3, chunk = (lane & 7) ^ (((8 * wave + row8) >> 1) & 7);
  const uint32_t at_a = (uint32_t)((8 * wave + row8) * p.lda) + 16u * chunk, at_b = (uint32_t)((8 * wave + row8) * p.ldb) + 16u * chunk;
  const uint32_t step_a = (uint32_t)(8 * kWaves * p.lda), step_b = (uint32_t)(8 * kWaves * p.ldb);
  const auto copy = [&](int slot) {
    char* to = lds + (slot & 1) * kSlot + wave * 1024;
    const uint32_t k = (uint32_t)slot * 128u;
    const bool in = k + 16u * chunk < (uint32_t)p.K;
#pragma unroll
    for (int j = 0; j < kCopies; j++) {
      const bool is_a = j < BM / 8 / kWaves;
      const uint32_t off = is_a ? at_a + j * step_a + k : at_b + (j - BM / 8 / kWaves) * step_b + k;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (lds_ptr_t)(to + j * kWaves * 1024), 16, in ? off : kFar, 0, 0, 1);
    }
  };

  v16i acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; i++)
#pragma unroll
    for (int j = 0; j < FB; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0;

  uint32_t read_a[4], read_b[4];
#pragma unroll
  for (int s = 0; s < 4; s++) {
    const uint32_t lo = lds_address(lds) + (uint32_t)r32 * 128u + 16u * (uint32_t)((2 * s + h) ^ ((r32 >> 1) & 7));
    read_a[s] = lo + wm * FA * 4096u;
    read_b[s] = lo + BM * 128u + wn * FB * 4096u;
  }

  if (begin < end) copy(begin);
  for (int slot = begin; slot < end; slot++) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's copies have landed; the barrier: everybody's, and the other slot is free
    asm volatile("s_barrier" ::: "memory");
    if (slot + 1 < end) copy(slot + 1);
    if ((slot + 1) * 128 > p.K && (p.K & 15)) {
      // the piece of A in which K ends: its other bytes become zeros
      const int c = (p.K & 127) >> 4, keep = p.K & 15;
      if (threadIdx.x < BM) {
        uint32_t* w = reinterpret_cast<uint32_t*>(lds + (slot & 1) * kSlot + threadIdx.x * 128 + 16 * (c ^ ((threadIdx.x >> 1) & 7)));
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int n = max(0, min(4, keep - 4 * i));
          if (n < 4) w[i] &= (1u << (8 * n)) - 1u;
        }
      }
      __syncthreads();
    }
    const uint32_t base = (uint32_t)(slot & 1) * kSlot;
#pragma unroll
    for (int s = 0; s < 4; s++) {
      v4i a[FA], b[FB];
      read_step<FA, FB>(a, b, read_a[s] + base, read_b[s] + base);
#pragma unroll
      for (int i = 0; i < FA; i++)
#pragma unroll
        for (int j = 0; j < FB; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  if (p.splits > 1) {
    constexpr uint32_t kPart = BM * BN * 4;
    const rsrc_t rp = resource(p.partial, (uint32_t)wgs * kPart);
    const auto place = [&](int o, int i, int j, int g) {
      return ((uint32_t)id * p.splits + o) * kPart + (uint32_t)(((i * FB + j) * 4 + g) * kThreads + threadIdx.x) * 16u;
    };
#pragma unroll
    for (int i = 0; i < FA; i++)
#pragma unroll
      for (int j = 0; j < FB; j++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const int x = acc[i][j][4 * g], y = acc[i][j][4 * g + 1], z = acc[i][j][4 * g + 2], w = acc[i][j][4 * g + 3];
          __builtin_amdgcn_raw_buffer_store_b128((u32x4){(uint32_t)x, (uint32_t)y, (uint32_t)z, (uint32_t)w}, rp, place(split, i, j, g), 0, kThrough);
        }
    if (!arrives_last(p.counters + id, p.splits, &flag)) return;
    for (int o = 0; o < p.splits; o++) {
      if (o == split) continue;
#pragma unroll
      for (int i = 0; i < FA; i++)
#pragma unroll
        for (int j = 0; j < FB; j++) {
          v4i w[4];
#pragma unroll
          for (int g = 0; g < 4; g++) w[g] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rp, place(o, i, j, g), 0, kThrough));
#pragma unroll
          for (int g = 0; g < 4; g++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][4 * g + e] += w[g][e];
        }
    }
  }
  __syncthreads();  // the slots become the waves' rows of C

  // Element e of a tile: column 8 (e / 4) + 4 h + e % 4, row r32. 32 rows at a time go through LDS, so that a store is of whole lines.
  char* mine = lds + wave * 32 * kPitch;
  const int c0 = n0 + wn * kCols;
  constexpr int kUnit = 16 / (int)sizeof(T), kPerRow = kCols / kUnit;
  typedef T x4 __attribute__((ext_vector_type(4)));
  typedef T unit __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
  for (int i = 0; i < FA; i++) {
    const int row0 = m0 + (wm * FA + i) * 32;
    const float sa = p.sa[min(row0 + r32, p.M - 1)];
#pragma unroll
    for (int j = 0; j < FB; j++)
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int col = 32 * j + 8 * g + 4 * h;
        x4 v;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int n = min(c0 + col + e, p.N - 1);
          v[e] = finished<T>(acc[i][j][4 * g + e], sa * p.sb[n], p.bias ? (float)((const T*)p.bias)[n] : 0.f, p.relu);
        }
        *reinterpret_cast<x4*>(mine + r32 * kPitch + col * (int)sizeof(T)) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (p.vector) {
#pragma unroll
      for (int u = 0; u < 32 * kPerRow / 64; u++) {
        const int at = u * 64 + lane, row = at / kPerRow, col = (at % kPerRow) * kUnit;
        const unit v = *reinterpret_cast<const unit*>(mine + row * kPitch + col * (int)sizeof(T));
        if (row0 + row >= p.M) continue;
        T* c = (T*)p.c + (row0 + row) * p.ldc + c0 + col;
        if (c0 + col + kUnit <= p.N) {
          __builtin_nontemporal_store(v, reinterpret_cast<unit*>(c));
        } else {
          for (int e = 0; e < kUnit; e++)
            if (c0 + col + e < p.N) c[e] = v[e];
        }
      }
    } else {
      for (int at = lane; at < 32 * kCols; at += 64) {
        const int row = at / kCols, col = at % kCols;
        if (row0 + row < p.M && c0 + col < p.N) ((T*)p.c)[(row0 + row) * p.ldc + c0 + col] = *reinterpret_cast<const T*>(mine + row * kPitch + col * (int)sizeof(T));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// ---- host -----------------------------------------------------------------------------------

struct Plan {
  int kind;  // 0: few rows; 1: 128 x 128 tiles; 2: 256 x 256 tiles
  int mt, nt, tiles_m, tiles_n, splits;
  size_t bytes;
};

Plan plan_for(int M, int N, int K, bool can_split) {
  Plan p = {};
  p.splits = 1;
  if (M <= 64) {
    p.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    p.nt = N >= 16 * 2 * 2 * kCUs ? 4 : N >= 16 * 2 * kCUs ? 2 : 1;
    p.tiles_m = 1, p.tiles_n = ceil_div(N, 16 * p.nt);
    const int steps = ceil_div(K, 64);
    if (can_split && p.tiles_n <= kCUs && steps >= 32) p.splits = std::max(1, std::min(2 * kCUs / p.tiles_n, steps / 16));
    if (p.splits > 1) p.bytes = kCounterBytes + (size_t)p.tiles_n * p.splits * p.mt * p.nt * 1024;
    return p;
  }
  const int64_t big = (int64_t)ceil_div(M, 256) * ceil_div(N, 256);
  p.kind = big >= kCUs * 3 / 4 ? 2 : 1;
  const int side = p.kind == 2 ? 256 : 128;
  p.tiles_m = ceil_div(M, side), p.tiles_n = ceil_div(N, side);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const int slots = ceil_div(K, 128);
  if (can_split && p.kind == 1 && tiles <= kCUs && slots >= 8) p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(2 * kCUs / tiles, slots / 4));
  if (p.splits > 1) p.bytes = kCounterBytes + (size_t)tiles * p.splits * side * side * 4;
  return p;
}

template <typename T, int MT, int WAVES>
void launch_rows(const Args& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.tiles_n, (unsigned)p.splits), block(64 * WAVES);
  if (p.nt == 1) hipLaunchKernelGGL((rows_kernel<T, MT, 1, WAVES>), grid, block, 0, st, a);
  else if (p.nt == 2) hipLaunchKernelGGL((rows_kernel<T, MT, 2, WAVES>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((rows_kernel<T, MT, 4, WAVES>), grid, block, 0, st, a);
}

template <typename T>
void launch(const Args& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.tiles_m * p.tiles_n * p.splits));
  if (p.kind == 2) hipLaunchKernelGGL((tile_kernel<T, 256, 256, 2, 4>), grid, dim3(512), 0, st, a);
  else if (p.kind == 1) hipLaunchKernelGGL((tile_kernel<T, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else if (p.mt == 1) launch_rows<T, 1, 8>(a, p, st);
  else if (p.mt == 2) launch_rows<T, 2, 4>(a, p, st);
  else launch_rows<T, 4, 4>(a, p, st);
}

int check_sizes(int M, int N, int K) {
  // 2^14 K below 2^31: the sum of K products of -128 by -128 stays an int
  return M < 0 || M > MX_MAX_DIM || N < 1 || N > MX_MAX_DIM || K < 1 || K > MXGEMM_I8_MAX_K ? MX_ERR_SHAPE : MX_OK;
}

}  // namespace

extern "C" size_t mxgemm_i8_workspace_size(int M, int N, int K) {
  if (check_sizes(M, N, K) || M == 0) return 0;
  return plan_for(M, N, K, true).bytes;
}

extern "C" int mxgemm_i8_run(int M, int N, int K, const mx_rows* A, const float* SA, const mx_rows* B, const float* SB, const void* bias, int fc,
                             const mx_rows* C, unsigned flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (fc != MX_F16 && fc != MX_BF16 && fc != MX_F32) return MX_ERR_FORMAT;
  if (flags & ~(unsigned)MXGEMM_RELU) return MX_ERR_FORMAT;
  if (int s = check_sizes(M, N, K)) return s;
  if (!A || !B || !C) return MX_ERR_NULL;
  if (M == 0) return MX_OK;
  if (!A->data || !SA || !B->data || !SB || !C->data) return MX_ERR_NULL;
  const int64_t most = (int64_t)MX_MAX_DIM;
  if (A->stride < K || A->stride % 16 || A->stride > most || B->stride < K || B->stride % 16 || B->stride > most || C->stride < N) return MX_ERR_SHAPE;
  if (!aligned16(A->data) || !aligned16(SA) || !aligned16(B->data) || !aligned16(SB) || !aligned16(C->data) || !aligned16(bias) || !aligned16(workspace))
    return MX_ERR_ALIGN;
  Plan p = plan_for(M, N, K, true);
  if (p.splits > 1 && (!workspace || workspace_bytes < p.bytes)) p = plan_for(M, N, K, false);
  Args a = {};
  a.a = (const uint8_t*)A->data, a.lda = A->stride, a.b = (const uint8_t*)B->data, a.ldb = B->stride;
  a.sa = SA, a.sb = SB, a.bias = bias, a.c = C->data, a.ldc = C->stride;
  a.M = M, a.N = N, a.K = K, a.relu = (flags & MXGEMM_RELU) != 0u;
  a.vector = C->stride * (fc == MX_F32 ? 4 : 2) % 16 == 0;
  a.tiles_m = p.tiles_m, a.tiles_n = p.tiles_n, a.splits = p.splits;
  if (p.splits > 1) a.counters = (uint32_t*)workspace, a.partial = (uint8_t*)workspace + kCounterBytes;
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  if (fc == MX_F16) launch<_Float16>(a, p, st);
  else if (fc == MX_BF16) launch<__bf16>(a, p, st);
  else launch<float>(a, p, st);
  return sync_check(launch_status(), st);
}
