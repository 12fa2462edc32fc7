// norm.hip -- root-mean-square norm of rows, with the residual's addition before it and 8-bit outputs with scales after it, and
// the quantisation of rows alone.
//
// h = round(x + r),  y_i = h_i w_i / sqrt(mean h^2 + eps). With g_i = h_i w_i the row's factor is left out of what needs a whole row: the
// sum of squares and the largest |g| are one pass and one reduction, 8-bit integers are q = rint(g 127 / max |g|), whose scale alone
// has the factor, and the others are g times the factor, or h times the factor times w where they have the input's own type. So a row
// is read once, held in registers as it was rounded, and written once, what is as wide as the input by non-temporal stores (4096 x 4096, bf16 with
// residual to E4M3: 20.4 us, with plain ones 25.4). Memory bounds long calls: those 118 MB are at 5.8 TB/s; one row of 4096 takes 4.3 to 4.9 us, most
// of it the launch. A thread takes units of eight neighbouring elements (16 bytes of 16-bit ones); four lanes hold a block of 32.
#include <algorithm>
#include <type_traits>

#include "kvcache.h"
#include "quant_rules.h"

using namespace mx;

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Eight;
template <>
struct Eight<_Float16> { typedef f16x8 type; };
template <>
struct Eight<__bf16> { typedef bf16x8 type; };
template <>
struct Eight<float> { typedef f32x8 type; };

constexpr int kRowsOfWaves = 4;  // rows of a workgroup whose waves take one each

struct Args {
  const void *x, *residual, *weight;
  void *total, *out, *scales;
  int64_t x_stride, residual_stride, total_stride, out_stride;  // elements
  int rows, dim;
  float eps;
  double inv;  // 1 / dim
  int norm;
};

// Over the wave's lanes: exchanges of its halves and of rows of 16, rotations within a row. Every lane has the result.
template <typename F>
MX_DEV uint32_t wave_all(uint32_t x, F f) {
  auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = f(r[0], r[1]);
  r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(r[0], r[1]);
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xF, 0xF, false));  // row_ror 8, 4, 2, 1
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xF, 0xF, false));
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xF, 0xF, false));
  return f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xF, 0xF, false));
}
MX_DEV uint32_t add_bits(uint32_t a, uint32_t b) { return fbits(bitsf(a) + bitsf(b)); }
MX_DEV float wave_sum(float x) { return bitsf(wave_all(fbits(x), add_bits)); }
// The same in 64 bits, whose halves are exchanged each.
MX_DEV double wave_sum(double x) {
  const auto halves = [](double v) { return __builtin_bit_cast(u32x2, v); };
  const auto whole = [](uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, (u32x2){lo, hi}); };
  const auto swapped = [&](auto swap) {
    const u32x2 w = halves(x);
    const auto lo = swap(w[0]), hi = swap(w[1]);
    x = whole(lo[0], hi[0]) + whole(lo[1], hi[1]);
  };
  swapped([](uint32_t w) { return __builtin_amdgcn_permlane32_swap(w, w, false, false); });
  swapped([](uint32_t w) { return __builtin_amdgcn_permlane16_swap(w, w, false, false); });
  const auto turned = [&](auto turn) {
    const u32x2 w = halves(x);
    x += whole(turn(w[0]), turn(w[1]));
  };
  turned([](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x128, 0xF, 0xF, false); });
  turned([](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x124, 0xF, 0xF, false); });
  turned([](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x122, 0xF, 0xF, false); });
  turned([](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x121, 0xF, 0xF, false); });
  return x;
}
MX_DEV uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }  // of magnitudes: NaN above infinity above all
MX_DEV uint32_t magnitude(float x) { return fbits(x) & 0x7FFFFFFFu; }
constexpr double kNear = 0x1p-40;  // an element this near below a power of two counts as it: the row's factor in 64 bits is good for so much
constexpr uint32_t kInf = 0x7F800000u, kFew = 27u << 23, kSmall = 47u << 23;  // infinity, 2^-100, 2^-80
MX_DEV uint32_t quad_max(uint32_t x) {  // over four neighbouring lanes
  x = max_bits(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));  // quad_perm: 1 away, 2 away
  return max_bits(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
}

// The exponent e of a positive finite number, 2^e <= x (subnormal ones count as -127), and 2^-e in two factors.
MX_DEV int exponent_of(uint32_t bits) { return max(-126, (int)(bits >> 23) - 127); }
MX_DEV float pow2(int e) { return bitsf((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// W: waves of a row (1: each wave of the workgroup has its own row). U: units of a thread. LOOP: rows of any length, read again
// where they are longer than W waves hold.
template <typename T, int OUT, int W, int U, bool LOOP>
__global__ __launch_bounds__(W == 1 ? 64 * kRowsOfWaves : 64 * W) void norm_kernel(Args a) {
  typedef typename Eight<T>::type x8;
  typedef x8 stored __attribute__((aligned(16)));  // rows are 16-byte aligned
  constexpr int kLanes = 64 * W, kChunk = kLanes * U;
  // A block's scale jumps where its largest element passes a power of two, so that element counts to its last bits, and so do the row's sum and
  // factor: in 64 bits for blocks (4096 x 4096: 20.4 us; 19.9 with a sum in 32, which gave most rows of one size the wrong scale).
  constexpr bool kBlocks = OUT == MX_E4M3 || OUT == MX_E5M2;
  typedef std::conditional_t<kBlocks, double, float> Sum;
  __shared__ Sum sums[W];
  __shared__ uint32_t tops[W];
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, wave = threadIdx.x >> 6;
  const int row = W == 1 ? (int)blockIdx.x * kRowsOfWaves + __builtin_amdgcn_readfirstlane(wave) : (int)blockIdx.x;
  if (W == 1 && row >= a.rows) return;
  const int dim = a.dim, whole = dim / 8, tail = dim & 7, units = whole + (tail ? 1 : 0);
  const T* x = (const T*)a.x + row * a.x_stride;
  const T* r = a.residual ? (const T*)a.residual + row * a.residual_stride : nullptr;
  T* total = a.total ? (T*)a.total + row * a.total_stride : nullptr;
  const T* weight = (const T*)a.weight;

  const auto load = [&](const T* p, int i) -> x8 {
    if (i < whole) return *reinterpret_cast<const stored*>(p + 8 * (int64_t)i);
    x8 v = {};
    if (i < units) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < tail) v[e] = p[8 * (int64_t)i + e];
    }
    return v;
  };
  const auto store = [&](T* p, int i, x8 v) {
    if (i < whole) {
      __builtin_nontemporal_store(v, reinterpret_cast<stored*>(p + 8 * (int64_t)i));
    } else if (i < units) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < tail) p[8 * (int64_t)i + e] = v[e];
    }
  };
  const auto wide = [&](x8 v) -> f32x8 { return __builtin_convertvector(v, f32x8); };
  const auto weighted = [&](f32x8 h, int i) -> f32x8 { return weight ? h * wide(load(weight, i)) : h; };

  // unit i of the row, added up and rounded
  const auto fetch = [&](int i) -> x8 {
    if (total) return load(total, i);
    const x8 v = load(x, i);
    return r ? __builtin_convertvector(wide(v) + wide(load(r, i)), x8) : v;
  };
  // f(unit, its rounded h) over the row: what the registers hold, or read again
  x8 held[U];
  const auto each = [&](auto f) {
    if constexpr (!LOOP) {
#pragma unroll
      for (int u = 0; u < U; u++) f(t + u * kLanes, held[u]);
    } else {
      for (int c = 0; c < units; c += kChunk) {
        if (units > kChunk) {
#pragma unroll
          for (int u = 0; u < U; u++) held[u] = fetch(c + t + u * kLanes);
        }
#pragma unroll
        for (int u = 0; u < U; u++) f(c + t + u * kLanes, held[u]);
      }
    }
  };
  // the row's sum of squares and largest magnitude, from the threads' own (the waves' sums are added in 64 bits)
  const auto reduce = [&](Sum& sum, uint32_t& top) {
    sum = wave_sum(sum);
    top = wave_all(top, max_bits);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) sums[wave] = sum, tops[wave] = top;
      __syncthreads();
      double all = (double)sums[0];
      top = tops[0];
#pragma unroll
      for (int w = 1; w < W; w++) all += (double)sums[w], top = max_bits(top, tops[w]);
      sum = (Sum)all;
    }
  };

  Sum sum = 0;
  uint32_t top = 0u;  // of |g|
  const auto count = [&](f32x8 h, int i) {
    const f32x8 g = weighted(h, i);
#pragma unroll
    for (int e = 0; e < 8; e++) sum = __builtin_elementwise_fma((Sum)h[e], (Sum)h[e], sum);
    if constexpr (OUT == MX_INT8) {
#pragma unroll
      for (int e = 0; e < 8; e++) top = max_bits(top, magnitude(g[e]));
    }
  };
  for (int c = 0; c < (LOOP ? units : 1); c += kChunk) {
    x8 add[U];
#pragma unroll
    for (int u = 0; u < U; u++) held[u] = load(x, c + t + u * kLanes);
    if (r) {
#pragma unroll
      for (int u = 0; u < U; u++) add[u] = load(r, c + t + u * kLanes);
#pragma unroll
      for (int u = 0; u < U; u++) {
        held[u] = __builtin_convertvector(wide(held[u]) + wide(add[u]), x8);
        if (total) store(total, c + t + u * kLanes, held[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) count(wide(held[u]), c + t + u * kLanes);
  }
  // y = h pre pre2 before w factor, where one of `before` and `factor` is the row's: a product with the weight alone could leave fp32's
  // range where y does not. (exact: the factor in 64 bits, for blocks.)
  float before = 1.f, factor = 1.f, pre = 1.f, pre2 = 1.f;
  double exact = 1.0;
  if (a.norm || OUT == MX_INT8) reduce(sum, top);
  if (a.norm) {
    float eps = a.eps;
    const auto mean = [&] { return (float)(sum * (Sum)a.inv + (Sum)eps); };
    // Where squares leave fp32's range (sums that overflow, means under 2^-100 that lose bits), the row is scaled by a power of two that brings
    // its largest element, or the root of eps, to 1. A row with infinities or NaN stays.
    if (!(mean() >= 0x1p-100f && mean() < INFINITY)) {
      uint32_t most = 0u;
      Sum none = 0;
      each([&](int, x8 v) {
        const f32x8 h = wide(v);
#pragma unroll
        for (int e = 0; e < 8; e++) most = max_bits(most, magnitude(h[e]));
      });
      if constexpr (W > 1) __syncthreads();
      reduce(none, most);
      if (most < kInf && most > 0u) {
        const int e = eps > 0.f ? max(exponent_of(most), (exponent_of(fbits(eps)) - 1) / 2) : exponent_of(most);
        const int half = -e / 2, rest = -e - half;
        pre = pow2(half), pre2 = pow2(rest);
        eps = eps * pre * pre2 * pre * pre2;
        sum = 0, top = 0u;
        each([&](int i, x8 v) { count(wide(v) * pre * pre2, i); });
        if constexpr (W > 1) __syncthreads();
        reduce(sum, top);
      } else if (most == 0u && eps > 0.f) {
        eps = 1.f;  // zeros, whatever the root of a subnormal is
      }
    }
    factor = __builtin_amdgcn_rsqf(mean());
    exact = (double)factor;
    if (kBlocks && factor > 0.f && factor < INFINITY) {
      // one step of Newton's from the approximation, whose error of 2^-23 becomes 2^-45
      const double f = (double)factor, v = sum * a.inv + (double)eps, r = f * (1.5 - 0.5 * v * f * f);
      factor = (float)r, exact = r;
    }
    if constexpr (!kBlocks && OUT != MX_INT8) before = factor, factor = 1.f;
  }

  const auto g_of = [&](x8 v, int i) -> f32x8 {
    f32x8 h = wide(v);
    if (pre != 1.f || pre2 != 1.f) h = h * pre * pre2;
    return weighted(h * before, i);
  };
  if constexpr (OUT == MX_INT8) {
    if (a.norm && !(top >= kFew && top < kInf) && factor < INFINITY) {  // products that leave fp32's range, or vanish in it
      before = factor, factor = 1.f, top = 0u;
      Sum none = 0;
      each([&](int i, x8 v) {
        const f32x8 y = g_of(v, i);
#pragma unroll
        for (int e = 0; e < 8; e++) top = max_bits(top, magnitude(y[e]));
      });
      if constexpr (W > 1) __syncthreads();
      reduce(none, top);
    }
    const bool fine = top < kInf && factor < INFINITY;
    // small rows are lifted, as 127 / max |g| would overflow
    const float lift = bitsf(top) < 0x1p-60f ? 0x1p64f : 1.f;
    const float inv = fine && top > 0u ? 127.f / (bitsf(top) * lift) : 0.f;
    if (t == 0) ((float*)a.scales)[row] = fine ? bitsf(top) * factor / 127.f : bitsf(0x7FC00000u);
    int8_t* out = (int8_t*)a.out + row * a.out_stride;
    each([&](int i, x8 v) {
      const f32x8 g = g_of(v, i) * lift;
      uint32_t w[2] = {0u, 0u};
      if (fine) {
#pragma unroll
        for (int e = 0; e < 8; e++) w[e / 4] |= ((uint32_t)(int)rintf(g[e] * inv) & 255u) << (8 * (e % 4));
      }
      if (i < whole) {
        *reinterpret_cast<u32x2*>(out + 8 * (int64_t)i) = (u32x2){w[0], w[1]};
      } else if (i < units) {
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (e < tail) out[8 * (int64_t)i + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
      }
    });
  } else if constexpr (OUT == MX_E4M3 || OUT == MX_E5M2) {
    uint8_t* out = (uint8_t*)a.out + row * a.out_stride;
    uint8_t* scales = (uint8_t*)a.scales + (int64_t)row * (dim / 32);
    each([&](int i, x8 v) {
      f32x8 y = g_of(v, i) * factor;
      uint32_t amax = 0u;
#pragma unroll
      for (int e = 0; e < 8; e++) amax = max_bits(amax, magnitude(y[e]));
      amax = quad_max(amax);
      // In 64 bits: next to a power of two (y is off by three half steps at most), and where the product with the weight left fp32's range, or
      // vanished in it and the factor (at most 2^50) makes it larger again (binary16's cannot).
      bool closer = ((amax + 4u) & 0x7FFFFFu) < 8u && amax > 0u;
      if constexpr (!std::is_same_v<T, _Float16>) closer |= amax >= kInf || (amax < kSmall && factor > 1.f);
      if (a.norm && sum != 0 && __any(closer)) {  // (a row of zeros has none)
        x8 anew = v;
        asm("" : "+v"(anew));  // here, and not kept in 64 bits since the sum
        const f32x8 h = wide(anew);
        f32x8 w;
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = 1.f;
        if (weight) w = wide(load(weight, i));
        uint32_t most = 0u;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const double d = (double)h[e] * pre * pre2 * w[e] * exact;
          if (closer) y[e] = (float)d;
          // what was rounded up to a power of two has the scale of what is below
          most = max_bits(most, magnitude(y[e]) - (fabs(d) < (1.0 - kNear) * fabs((double)y[e]) ? 1u : 0u));
        }
        amax = closer ? quad_max(most) : amax;
      }
      int shift;
      const uint32_t E = mx_block_scale(amax, amax >= kInf, OUT, &shift);
      if (i >= units) return;
      uint32_t w[2] = {0u, 0u};
      if (amax < kInf) {
        // the scaled conversion divides by 2^(E - 127) and rounds to nearest even; what would pass the largest element is cut to
        // it before
        const float scale = bitsf(E << 23);
        const int exponent = (int)E - 127;
        const float most = OUT == MX_E4M3 ? 448.f : 57344.f;
        const float limit = exponent < -126 ? most * 0x1p-126f * 0.5f : most * pow2(exponent);  // at most 1.75 * 2^127
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = __builtin_amdgcn_fmed3f(y[e], -limit, limit);
#pragma unroll
        for (int p = 0; p < 2; p++) {
          s16x2 c = {0, 0};
          if constexpr (OUT == MX_E4M3) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, y[4 * p], y[4 * p + 1], scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, y[4 * p + 2], y[4 * p + 3], scale, true);
          } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, y[4 * p], y[4 * p + 1], scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, y[4 * p + 2], y[4 * p + 3], scale, true);
          }
          w[p] = __builtin_bit_cast(uint32_t, c);
        }
      }
      *reinterpret_cast<u32x2*>(out + 8 * (int64_t)i) = (u32x2){w[0], w[1]};
      if ((i & 3) == 0) scales[i / 4] = (uint8_t)E;
    });
  } else {
    T* out = (T*)a.out + row * a.out_stride;
    each([&](int i, x8 v) { store(out, i, __builtin_convertvector(g_of(v, i) * factor, x8)); });
  }
}

// ---- host -----------------------------------------------------------------------------------

template <typename T, int OUT, int W, int U, bool LOOP = false>
void launch(const Args& a, hipStream_t st) {
  const unsigned grid = W == 1 ? (unsigned)ceil_div(a.rows, kRowsOfWaves) : (unsigned)a.rows;
  hipLaunchKernelGGL((norm_kernel<T, OUT, W, U, LOOP>), dim3(grid), dim3(W == 1 ? 64 * kRowsOfWaves : 64 * W), 0, st, a);
}

// Short rows: a wave to each, which needs no barrier. Longer ones: as many waves as make a row's chain of latencies short and still let rows
// follow one another on a CU, so that some load while others store. With many rows a thread has two units on their way (4096
// x 4096, bf16 with residual to E4M3: 20.4 us of four waves, 26 of eight, 28 of one; 512 rows: 4.7 and 4.5 of eight).
template <typename T, int OUT>
void launch_shape(const Args& a, hipStream_t st) {
  const int units = ceil_div(a.dim, 8);
  if (units <= 64 * 2) launch<T, OUT, 1, 2>(a, st);
  else if (units <= 512 && a.rows >= 1024) launch<T, OUT, 4, 2>(a, st);
  else if (units <= 512) launch<T, OUT, 8, 1>(a, st);
  else if (units <= 1024) launch<T, OUT, 16, 1>(a, st);
  else if (units <= 1024 * 2) launch<T, OUT, 16, 2>(a, st);
  else launch<T, OUT, 16, 4, true>(a, st);
}

template <typename T, int SAME>
void launch_out(const Args& a, int fmt, hipStream_t st) {
  if (fmt == MX_INT8) launch_shape<T, MX_INT8>(a, st);
  else if (fmt == MX_E4M3) launch_shape<T, MX_E4M3>(a, st);
  else if (fmt == MX_E5M2) launch_shape<T, MX_E5M2>(a, st);
  else launch_shape<T, SAME>(a, st);
}

int check_rows(const mx_rows* m, int dim, int elem_bytes) {
  if (!m || !m->data) return MX_ERR_NULL;
  if (m->stride < dim || m->stride % (16 / elem_bytes)) return MX_ERR_SHAPE;
  return aligned16(m->data) ? MX_OK : MX_ERR_ALIGN;
}

int run(Args a, int f, int rows, int dim, const mx_rows* x, const mx_rows* residual, const mx_rows* total, const void* weight, int fmt,
        const mx_rows* out, void* scales, void* stream) {
  if (f != MX_F16 && f != MX_BF16 && f != MX_F32) return MX_ERR_FORMAT;
  const bool block = fmt == MX_E4M3 || fmt == MX_E5M2;
  if (fmt != MX_INT8 && !block && fmt != f) return MX_ERR_FORMAT;
  if (rows < 0 || rows > MX_MAX_DIM || dim < 1 || dim > MX_MAX_DIM || (block && dim % 32)) return MX_ERR_SHAPE;
  if (!x || !out) return MX_ERR_NULL;
  if (total && !residual) return MX_ERR_NULL;
  if (rows == 0) return MX_OK;
  const int bytes = f == MX_F32 ? 4 : 2, out_bytes = fmt == f ? bytes : 1;
  if (int s = check_rows(x, dim, bytes)) return s;
  if (residual)
    if (int s = check_rows(residual, dim, bytes)) return s;
  if (total)
    if (int s = check_rows(total, dim, bytes)) return s;
  if (int s = check_rows(out, dim, out_bytes)) return s;
  if (fmt != f && !scales) return MX_ERR_NULL;
  if (!aligned16(weight) || !aligned16(scales)) return MX_ERR_ALIGN;
  a.x = x->data, a.x_stride = x->stride, a.weight = weight, a.rows = rows, a.dim = dim;
  if (residual) a.residual = residual->data, a.residual_stride = residual->stride;
  if (total) a.total = total->data, a.total_stride = total->stride;
  a.out = out->data, a.out_stride = out->stride, a.scales = scales;
  a.inv = 1.0 / dim;
  if (int s = check_arch()) return s;
  const hipStream_t st = as_stream(stream);
  if (f == MX_F16) launch_out<_Float16, MX_F16>(a, fmt, st);
  else if (f == MX_BF16) launch_out<__bf16, MX_BF16>(a, fmt, st);
  else launch_out<float, MX_F32>(a, fmt, st);
  return sync_check(launch_status(), st);
}

}  // namespace

extern "C" int mxnorm_run(int f, int rows, int dim, const mx_rows* x, const mx_rows* residual, const mx_rows* total, const void* weight,
                          float eps, int fmt, const mx_rows* out, void* scales, void* stream) {
  if (!(eps >= 0.f) || !__builtin_isfinite(eps)) return MX_ERR_SHAPE;
  Args a = {};
  a.norm = 1, a.eps = eps;
  return run(a, f, rows, dim, x, residual, total, weight, fmt, out, scales, stream);
}

extern "C" int mxquant_rows_run(int f, int rows, int dim, const mx_rows* x, int fmt, const mx_rows* out, void* scales, void* stream) {
  if (fmt != MX_INT8 && fmt != MX_E4M3 && fmt != MX_E5M2) return MX_ERR_FORMAT;
  return run(Args{}, f, rows, dim, x, nullptr, nullptr, nullptr, fmt, out, scales, stream);
}
