// attention.h -- what the attention kernels share: the 16-bit types' matrix instructions and conversions, the score cap, and the
// partial results of shared positions that one kernel leaves for the other.
#pragma once
#include "kvcache.h"

namespace mx {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  typedef f16x8 x8;
  // A probability p = 2^(x - m) goes to the matrix cores as two values of T: p cut to T, and what that leaves rounded
  // to T. Together they hold 21 bits of p (bfloat16: 15). One value alone made the error against 64 bits 1.2 to 1.4
  // times that of the result's own rounding. The second is never 0 nor negative, as its product with an infinite value has
  // to be what the first one's is: kLeast, 2^-39 of the largest p (bfloat16: 2^-126), is far below a half step of any sum.
  // p is at most 1; binary16 would lose those under 2^-24, which can matter in number in a long row, so they
  // are scaled by 2^15 (which cancels in the division by their sum). bfloat16 has the range.
  static constexpr float kShift = 15.0f, kLeast = 0x1p-24f;
  static MX_DEV uint32_t cut(float a, float b) { return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b)); }
  // Eight probabilities as both values. (What is left is cut too, 2^-22 of p at most; it is not negative, so its bits compare as integers.)
  static MX_DEV void split(const float (&x)[8], x8& p, x8& rest) {
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const auto both = __builtin_amdgcn_cvt_pkrtz(x[2 * i], x[2 * i + 1]);
      hi[i] = __builtin_bit_cast(uint32_t, both);
      const uint32_t left = cut(x[2 * i] - (float)both[0], x[2 * i + 1] - (float)both[1]);
      lo[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, left), (s16x2){1, 1}));
    }
    p = __builtin_bit_cast(x8, hi), rest = __builtin_bit_cast(x8, lo);
  }
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static MX_DEV f32x16 mfma(x8 a, x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static MX_DEV uint32_t from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HI));
  }
};
template <>
struct Vec<__bf16> {
  typedef bf16x8 x8;
  static constexpr float kShift = 0.0f, kLeast = 0x1p-126f;
  static MX_DEV uint32_t cut(float a, float b) { return __builtin_amdgcn_perm(fbits(b), fbits(a), 0x07060302u); }
  static MX_DEV void split(const float (&x)[8], x8& p, x8& rest) {
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      hi[i] = cut(x[2 * i], x[2 * i + 1]);
      bf16x2 left;
#pragma unroll
      for (int e = 0; e < 2; e++) left[e] = (__bf16)(x[2 * i + e] - bitsf(fbits(x[2 * i + e]) & 0xFFFF0000u));
      lo[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, left), (s16x2){0x80, 0x80}));
    }
    p = __builtin_bit_cast(x8, hi), rest = __builtin_bit_cast(x8, lo);
  }
  static MX_DEV f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static MX_DEV f32x16 mfma(x8 a, x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
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

MX_DEV float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// c tanh(s / c): where |s / c| < 0.2 by its series, whose fifth term is below half a step, else by one
// exponential, whose error is relative to c. A cap that is far above every score leaves them as they are.
MX_DEV float soft_cap(float s, float c) {
  const float y = s * fminf(1.0f / c, 3.0e38f), z = y * y;
  const float near = s * fmaf(z, fmaf(z, fmaf(z, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
  const float far = fmaf(c, -2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.0f * kLog2e * y)), c);
  return fabsf(y) < 0.2f ? near : far;
}

// Partial results of positions that rows share, for the kernel that goes on with each row's own. A unit is 128 query rows of a group and
// cache head, in four slots of 32 for each of the splits of its keys, which are next to each other: the outputs [dim / 4][32] quads, then [32] {maximum,
// sum}, as the kernels hold them.
constexpr int kPrefixRows = 32, kPrefixSlots = 4, kPrefixUnit = kPrefixRows * kPrefixSlots;
struct Prefix {
  const i32x4* rows;      // of sequence b: {its group's first unit, units of a cache head, first row in its group, whether it shares}
  const int2* units;      // {first split, splits}
  const float* partial;   // NULL: no shared positions
};
MX_HD int64_t prefix_slot_floats(int dim) { return (int64_t)kPrefixRows * (dim + 2); }

// The launch behind mxattn_decode_run, whose checks the caller has made. starts: first attended positions on the device, or NULL.
int decode_launch(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse, const mxkv_table* table, const int32_t* lengths,
                  const int32_t* starts, int max_len, const mxattn_opts* opts, const Prefix& prefix, void* workspace, size_t workspace_bytes, hipStream_t st);
int check_attention(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, const mxkv_table* table, const int32_t* lengths, int max_len,
                    const mxattn_opts* opts);
bool decode_sizes_ok(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window);
size_t decode_workspace(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window);  // 0 for invalid sizes too
constexpr size_t kDecodeCounterBytes = 3 * 2 * 256 * 4;  // at a workspace's beginning, whatever the shape

}  // namespace mx
