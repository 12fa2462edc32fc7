// gemm_i8.hip -- C = A B of 8-bit integers, A [M][K] with a scale per row (token), B stored [N][K] with a scale per row (output
// channel): C[m,n] = sa[m] sb[n] sum_k a[m,k] b[n,k] (+ bias[n], ReLU). The sums are exact 32-bit integers (K is bounded), so neither
// their order nor a split of K changes a result.
//
// Two kernels. For up to 16 rows of few columns a call is the latency of a few loads: a wave takes the weights from global memory straight
// to the matrix cores' registers (16x16x64), the waves of a workgroup share K. For others tiles go through LDS (direct global -> LDS copies, a
// ring of slots of 128 bytes of K) to 32x32x32 instructions: 64 wide, where the weights' bytes bound the time (64 x 12288 x 4096: 12.6 to 13.2 us,
// 3.9 to 4.2 TB/s), to 256 wide, where the matrix cores and LDS do (2048 x 14336 x 4096: 113 to 119 us, 2.0 to 2.1 POP/s; a slot of a 256 wide tile
// takes 2048 clocks of the matrix cores, 1536 of LDS for the reads and 512 for what is copied into it). K need not be a multiple of
// anything: bytes of A past K become zeros on the way, and a zero times whatever integer B holds there is zero.
#include <algorithm>
#include <type_traits>

#include "kvcache.h"

using namespace mx;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kFar = 0x80000000u;  // an offset past every buffer: loads give 0
constexpr int kCounterBytes = 16384;    // of the workspace: a counter per tile that K is split of
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
// The same as four scalar registers, for assembly.
MX_DEV v4i resource_words(const void* base, uint32_t bytes) {
  const uint64_t at = (uint64_t)base;
  return (v4i){uniform((int)at), uniform((int)(at >> 32)) & 0xFFFF, uniform((int)bytes), 0x00020000};
}
MX_DEV uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_ptr_t)p; }

// Bytes of rows first .. first + rows - 1, each up to its last 16-byte piece of K.
MX_DEV uint32_t extent(int rows, int64_t ld, int K) { return (uint32_t)((rows - 1) * ld + ((K + 15) & ~15)); }

template <typename T>
MX_DEV T finished(int sum, float scale, float bias, bool relu) {
  float v = fmaf((float)sum, scale, bias);
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

// Up to 16 rows of A by 16 of B to a workgroup, whose waves take K's steps in turn: for weights that are too small to fill the chip with tiles, where the
// time is the latency of a few loads (1 x 4096 x 4096: 6.8 us, in 64 x 64 tiles 10.3). Lane l of a 16x16x64 instruction holds 16 bytes of
// row l % 16 of each operand, those of K-piece l / 16; B is the first operand, so that a lane ends with four neighbouring columns
// of C of one row.
template <typename T>
__global__ __launch_bounds__(512) void rows_kernel(Args p) {
  constexpr int kStep = 64, kWaves = 8, kDeep = 8;  // kDeep: steps of a wave on their way
  __shared__ v4i sums[kWaves][64];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, rows = min(16, p.N - n0);
  const int steps = ceil_div(p.K, kStep), split = blockIdx.y;
  const int begin = (int)((int64_t)steps * split / p.splits), end = (int)((int64_t)steps * (split + 1) / p.splits);

  const rsrc_t ra = resource(p.a, extent(p.M, p.lda, p.K)), rb = resource(p.b + n0 * p.ldb, extent(rows, p.ldb, p.K));
  const uint32_t at_a = (uint32_t)(min(r, p.M - 1) * p.lda) + 16u * q;  // rows past M repeat the last one, and are not written
  const uint32_t at_b = (uint32_t)(r * p.ldb) + 16u * q;
  v4i acc = {0, 0, 0, 0};
  struct Step {
    v4i a, b;
  } ring[kDeep];
  const auto load = [&](Step& s, int step) {
    const uint32_t k = (uint32_t)step * kStep;
    const bool in = step < end && k + 16u * q < (uint32_t)p.K;
    s.b = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, in ? at_b + k : kFar, 0, 2));  // weights: non-temporal
    s.a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? at_a + k : kFar, 0, 0));
  };
  const auto multiply = [&](Step& s, int step) {
    const int left = p.K - (step * kStep + 16 * q);  // bytes of this lane's piece that K has
    if (step * kStep + kStep > p.K && left < 16) {
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const int n = max(0, min(4, left - 4 * w));
        s.a[w] = n == 4 ? s.a[w] : (int)((uint32_t)s.a[w] & ((1u << (8 * n)) - 1u));
      }
    }
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.b, s.a, acc, 0, 0, 0);
  };
  int step = begin + wave;
#pragma unroll
  for (int d = 0; d < kDeep; d++) load(ring[d], step + d * kWaves);
  for (; step < end; step += kDeep * kWaves) {
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      multiply(ring[d], step + d * kWaves);  // a step past the end is of zeros
      load(ring[d], step + (d + kDeep) * kWaves);
    }
  }

  sums[wave][lane] = acc;
  __syncthreads();
  // thread: four neighbouring columns of one row; neighbouring threads take neighbouring columns
  const int quad = threadIdx.x % 4, m = threadIdx.x / 4, n = n0 + 4 * quad;
  const bool mine = threadIdx.x < 64;
  v4i sum = {0, 0, 0, 0};
  if (mine) {
#pragma unroll
    for (int w = 0; w < kWaves; w++) sum += sums[w][quad * 16 + m];
  }
  if (p.splits > 1) {
    const rsrc_t rp = resource(p.partial, (uint32_t)gridDim.x * p.splits * 1024u);
    const uint32_t first = (uint32_t)blockIdx.x * p.splits * 1024u + threadIdx.x * 16u;
    if (mine) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), rp, first + (uint32_t)split * 1024u, 0, kThrough);
    if (!arrives_last(p.counters + blockIdx.x, p.splits, &flag)) return;
    if (mine) {
      for (int o = 0; o < p.splits; o++)
        if (o != split) sum += __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rp, first + (uint32_t)o * 1024u, 0, kThrough));
    }
  }
  if (!mine || m >= p.M || n >= p.N) return;
  const float sa = p.sa[m];
  T* c = (T*)p.c + m * p.ldc + n;
  typedef T x4 __attribute__((ext_vector_type(4)));
  x4 v;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int at = min(n + i, p.N - 1);
    v[i] = finished<T>(sum[i], sa * p.sb[at], p.bias ? (float)((const T*)p.bias)[at] : 0.f, p.relu);
  }
  if (p.vector && n + 4 <= p.N) {
    *reinterpret_cast<x4*>(c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (n + i < p.N) c[i] = v[i];
  }
}

// ---- tiles ------------------------------------------------------------------------------------

// One wave's copy of 16 bytes per lane from memory to LDS, `to` and on; past the L1, as no CU reads a byte twice. (In assembly, as the compiler
// would wait for every copy on its way before a read of LDS that it can see; the kernel waits by counts. The instruction has no
// result, and M0 needs a state between.)
MX_DEV void copy16(uint32_t to, v4i from, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tbuffer_load_dwordx4 %1, %2, 0 offen sc0 lds" ::"s"(to), "v"(offset), "s"(from) : "m0");
}

// Waits until at most N of the wave's accesses to memory, the last ones, are outstanding.
template <int N>
MX_DEV void wait_memory() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0F70 | (N >> 4) << 14);
}

// BM x BN tiles; WM x WN waves of (BM / WM) x (BN / WN) each. A slot holds 128 bytes of every row: chunk c (16 bytes) of row r at
// place c ^ ((r >> 1) & 7), so that the 16 rows that a quarter of a read touches lie on different banks. SLOTS of them: one in use, the
// others on their way. A slot's copies are issued a few at a time between the matrix instructions, as a CU takes 64 bytes a clock and waves
// would wait to issue more.
template <typename T, int BM, int BN, int WM, int WN, int SLOTS>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_kernel(Args p) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, FA = BM / WM / 32, FB = BN / WN / 32;
  constexpr int kSlot = (BM + BN) * 128, kCopies = (BM + BN) / 8 / kWaves;  // copies of a wave: 8 rows each
  static_assert((BM / 8) % kWaves == 0, "a copy is of A or of B for all waves");
  constexpr int kCols = 32 * FB, kPitch = kCols * (int)sizeof(T) + 16;  // epilogue: 32 rows of a wave
  constexpr int kLds = std::max(SLOTS * kSlot, kWaves * 32 * kPitch);
  constexpr int kAtOnce = (kCopies + 2) / 3;  // copies of a step: a slot's are started in three
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

  const v4i ra = resource_words(p.a + m0 * p.lda, extent(min(BM, p.M - m0), p.lda, p.K));
  const v4i rb = resource_words(p.b + n0 * p.ldb, extent(min(BN, p.N - n0), p.ldb, p.K));
  const int slots = ceil_div(p.K, 128);
  const int begin = (int)((int64_t)slots * split / p.splits), end = (int)((int64_t)slots * (split + 1) / p.splits);

  // Copy j of a wave fills rows 8 (wave + kWaves j) .. + 7 of the slot; lane l chunk place l % 8 of row l / 8. Which chunk
  // that is depends on the row's bits 1 to 3, which all copies of a wave share.
  const int row8 = lane >> 3, chunk = (lane & 7) ^ (((8 * wave + row8) >> 1) & 7);
  const uint32_t at_a = (uint32_t)((8 * wave + row8) * p.lda) + 16u * chunk, at_b = (uint32_t)((8 * wave + row8) * p.ldb) + 16u * chunk;
  const uint32_t step_a = (uint32_t)(8 * kWaves * p.lda), step_b = (uint32_t)(8 * kWaves * p.ldb);
  const auto copy = [&](int slot, int at, int first, int last) {  // into slot place `at`
    const uint32_t to = lds_address(lds) + at * kSlot + wave * 1024, k = (uint32_t)slot * 128u;
    const bool in = k + 16u * chunk < (uint32_t)p.K;
#pragma unroll
    for (int j = 0; j < kCopies; j++) {
      if (j < first || j >= last) continue;
      const bool is_a = j < BM / 8 / kWaves;
      const uint32_t off = is_a ? at_a + j * step_a + k : at_b + (j - BM / 8 / kWaves) * step_b + k;
      copy16(to + j * kWaves * 1024, is_a ? ra : rb, in ? off : kFar);
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
    const uint32_t lo = (uint32_t)r32 * 128u + 16u * (uint32_t)((2 * s + h) ^ ((r32 >> 1) & 7));
    read_a[s] = lo + wm * FA * 4096u;
    read_b[s] = lo + BM * 128u + wn * FB * 4096u;
  }

  const auto mask = [&](int slot, const char* base) {  // the piece of A in which K ends: its other bytes become zeros
    if ((slot + 1) * 128 <= p.K || !(p.K & 15)) return;
    const int c = (p.K & 127) >> 4, keep = p.K & 15;
    if (threadIdx.x < BM) {
      uint32_t* w = (uint32_t*)(base + threadIdx.x * 128 + 16 * (c ^ ((threadIdx.x >> 1) & 7)));
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int n = max(0, min(4, keep - 4 * i));
        if (n < 4) w[i] &= (1u << (8 * n)) - 1u;
      }
    }
    __syncthreads();
  };
  constexpr int kMul = FA * FB, kBefore = kMul > 4 ? 2 : 0;
  constexpr int kFirst = kMul == 1 ? SLOTS - 1 : SLOTS;  // slots that are copied before the first is used
#pragma unroll
  for (int i = 0; i < kFirst; i++)
    if (begin + i < end) copy(begin + i, i, 0, kCopies);
  // Waits for this wave's copies of a slot, of which `later` more follow at most, then for everybody's. All reads of LDS have ended.
  const auto ready = [&](bool follow, auto later, int slot, const char* base) {
    if (follow) wait_memory<decltype(later)::value * kCopies>();
    else wait_memory<0>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    mask(slot, base);
  };
  int here = 0;
  if constexpr (kMul == 1) {
    // Small tiles wait for memory: a slot's fragments are read at once, the place of the slot before is filled meanwhile.
    for (int slot = begin; slot < end; slot++) {
      const char* const base = lds + here * kSlot;
      ready(slot + SLOTS - 2 < end, std::integral_constant<int, SLOTS - 2>(), slot, base);
      if (slot + SLOTS - 1 < end) copy(slot + SLOTS - 1, here == 0 ? SLOTS - 1 : here - 1, 0, kCopies);
      v4i a[4], b[4];
#pragma unroll
      for (int s = 0; s < 4; s++) b[s] = *reinterpret_cast<const v4i*>(base + read_b[s]), a[s] = *reinterpret_cast<const v4i*>(base + read_a[s]);
#pragma unroll
      for (int s = 0; s < 4; s++) acc[0][0] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[s], a[s], acc[0][0], 0, 0, 0);
      here = here + 1 == SLOTS ? 0 : here + 1;
    }
  } else {
    // A step's fragments are read, and copies started, between the instructions of the step before. Before a slot's last step
    // all of it is in registers: from there on the next slot is read, and its own place is filled with the one after the others.
    // (2048 x 14336 x 4096 in tiles of 256: 113 us; reads and copies before a step's instructions, a barrier after its last: 123.)
    v4i a[2][FA], b[2][FB];
    const auto read = [&](const char* base, int s, int i) {  // fragment i of step s
      if (i < FB) b[s % 2][i] = *reinterpret_cast<const v4i*>(base + read_b[s] + 4096 * i);
      else a[s % 2][i - FB] = *reinterpret_cast<const v4i*>(base + read_a[s] + 4096 * (i - FB));
    };
    ready(begin + SLOTS - 1 < end, std::integral_constant<int, SLOTS - 1>(), begin, lds);
#pragma unroll
    for (int i = 0; i < FA + FB; i++) read(lds, 0, i);
    for (int slot = begin; slot < end; slot++) {
      const int next = here + 1 == SLOTS ? 0 : here + 1, before = here == 0 ? SLOTS - 1 : here - 1;
      const char* const base = lds + here * kSlot;
      const char* const after = lds + next * kSlot;
      const bool more = slot + SLOTS < end, older = slot > begin && slot - 1 + SLOTS < end;  // copies to its place, to that of the one before
#pragma unroll
      for (int s = 0; s < 4; s++) {
#pragma unroll
        for (int m = 0; m < kMul; m++) {
          if (s == 3 && m == kBefore && slot + 1 < end) ready(slot + SLOTS - 1 < end, std::integral_constant<int, SLOTS - 2>(), slot + 1, after);
          acc[m / FB][m % FB] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[s % 2][m % FB], a[s % 2][m / FB], acc[m / FB][m % FB], 0, 0, 0);
          const int u = s < 3 ? m : m - kBefore, of = s < 3 ? kMul : kMul - kBefore;  // what follows instruction u of `of`
          if (u >= 0) {
#pragma unroll
            for (int i = 0; i < FA + FB; i++)
              if (i * of / (FA + FB) == u) read(s < 3 ? base : after, (s + 1) % 4, i);
            const int first = min(kCopies, (s + 1) % 4 * kAtOnce), n = min(kCopies - first, kAtOnce);
            if (s == 3 ? more : older) copy(s == 3 ? slot + SLOTS : slot - 1 + SLOTS, s == 3 ? here : before, first + n * u / of, first + n * (u + 1) / of);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      here = next;
    }
  }
  __syncthreads();

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
  int side;  // of the tiles; 0: few rows
  int tiles_m, tiles_n, splits;
  size_t bytes;
};

Plan plan_for(int M, int N, int K, bool can_split) {
  Plan p = {};
  p.splits = 1;
  // Up to 16 rows: 16 columns to a workgroup, if all run at once and the weights have 32 MB at most (16 x 4096 x 4096: 8.4 us, in tiles 10.3;
  // 1 x 8192 x 4096: 11.3 and 10.8; 16 x 4096 x 14336: 21 and 16). K is split to six steps of each wave (1 x 1024 x 14336: 8.6 us, whole 13.9).
  if (M <= 16 && N <= 16 * kCUs && (int64_t)N * K <= (int64_t)1 << 25) {
    p.tiles_m = 1, p.tiles_n = ceil_div(N, 16);
    if (can_split) p.splits = std::max(1, std::min(2 * kCUs / p.tiles_n, ceil_div(K, 64) / 48));
    if (p.splits > 1) p.bytes = kCounterBytes + (size_t)p.tiles_n * p.splits * 1024;
    return p;
  }
  // The largest tiles that fill three quarters of the CUs (1024 x 14336 x 4096: 256 wide 60 us, 128 wide 78; 256 x 12288 x 4096: 128 wide 22, 64 wide 32;
  // 512 x 4096 x 4096: 64 wide 17.5 us, 128 wide and K split 21), but none that the rows or columns would fill half at most: the time is then that of
  // the other operand's bytes (1 x 70000 x 4096, and 70000 x 16 x 4096: 64 wide 67 us, 256 wide 123 to 127; 64 x 128256 x 4096: 112 to 118 and 139 to 144;
  // 128 x 70000 x 4096: 128 wide 103, 256 wide 129, 64 wide 98).
  const auto tiles = [&](int side) { return (int64_t)ceil_div(M, side) * ceil_div(N, side); };
  const int most = std::min(M, N) <= 64 ? 64 : std::min(M, N) <= 128 ? 128 : 256;
  p.side = most >= 256 && tiles(256) >= kCUs * 3 / 4 ? 256 : most >= 128 && tiles(128) >= kCUs * 3 / 4 ? 128 : 64;
  p.tiles_m = ceil_div(M, p.side), p.tiles_n = ceil_div(N, p.side);
  const int64_t n = tiles(p.side);
  // Small tiles that leave CUs idle split K, four slots at least to a workgroup (64 x 4096 x 4096: 10.6 us in four, 10.5 in two, 13.8 in
  // eight; 128 x 4096 x 4096: 11.4 in two, 13.5 whole).
  if (can_split && p.side == 64 && n < kCUs) p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kCUs / n, ceil_div(K, 128) / 4));
  if (p.splits > 1) p.bytes = kCounterBytes + (size_t)n * p.splits * p.side * p.side * 4;
  return p;
}

template <typename T>
void launch(const Args& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.tiles_m * p.tiles_n * p.splits));
  if (p.side == 256) hipLaunchKernelGGL((tile_kernel<T, 256, 256, 2, 4, 2>), grid, dim3(512), 0, st, a);
  // one workgroup to a CU: eight waves and four slots; more: two to a CU, of four waves and two slots (1024 x 4096 x 4096: 24.5 us and 31;
  // 2048 x 4096 x 4096: 49 and 40)
  else if (p.side == 128 && grid.x <= kCUs) hipLaunchKernelGGL((tile_kernel<T, 128, 128, 2, 4, 4>), grid, dim3(512), 0, st, a);
  else if (p.side == 128) hipLaunchKernelGGL((tile_kernel<T, 128, 128, 2, 2, 2>), grid, dim3(256), 0, st, a);
  else if (p.side == 64) hipLaunchKernelGGL((tile_kernel<T, 64, 64, 2, 2, 4>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((rows_kernel<T>), dim3((unsigned)p.tiles_n, (unsigned)p.splits), dim3(512), 0, st, a);
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
