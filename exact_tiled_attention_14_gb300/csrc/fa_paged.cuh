// fa_paged.cuh — a key/value cache in pages of 8-bit codes, as the append,
// read and decoding kernels see it.
//
// k and v are [pages, Hk, page_size, d] codes, their scales [pages, Hk]
// float32: an element's value is code * scale of its page and head.  The page
// table [B, per_seq] names the pages of each sequence in order; slot n of
// sequence b is row n % page_size of page page_table[b][n / page_size].  A
// table entry outside [0, pages) names no page: nothing is written for its
// slots, and they are read as if nobody saw them.
#pragma once

#include <cstdint>

#include "ptx_sm103.cuh"

namespace fa {

constexpr int kPageRows = 16;        // page sizes are multiples of it
constexpr int kMaxPage = 128;
constexpr float kMinPageScale = 7.8886090522101181e-31f;   // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// Two e4m3 codes (low byte first) as packed half-precision values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}
// Four int8 codes as two packed pairs of half-precision integers, exactly:
// code + 128 becomes the low byte of 1024 + x, from which 1152 is taken.
__device__ __forceinline__ void int8x4_to_f16x2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = four ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x4140);
  hi = __byte_perm(u, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}
template <bool kInt8>
__device__ __forceinline__ void codes4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    int8x4_to_f16x2(four, lo, hi);
  } else {
    lo = e4m3x2_to_f16x2(four);
    hi = e4m3x2_to_f16x2(four >> 16);
  }
}
template <bool kInt8>
__device__ __forceinline__ void codes4_float(uint32_t four, float* x) {
  uint32_t lo, hi;
  codes4<kInt8>(four, lo, hi);
  ptx::unpack2<false>(lo, x[0], x[1]);
  ptx::unpack2<false>(hi, x[2], x[3]);
}
// Four values as codes, to nearest even (NaN becomes a NaN code as e4m3, 0 as int8).
template <bool kInt8>
__device__ __forceinline__ uint32_t to_codes4(const float* x) {
  if constexpr (kInt8) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int c;
      asm("cvt.rni.s32.f32 %0, %1;" : "=r"(c) : "f"(x[i]));
      c = max(min(c, 127), -127);
      r |= static_cast<uint32_t>(c & 0xff) << (8 * i);
    }
    return r;
  } else {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
    return r;
  }
}

// A page's scale from the largest magnitude (as float bits) of its elements.
// e4m3: the smallest power of two s with top <= 448 s = 1.75 * 2^8 s, so that
// raising it later shifts exponents and rounds nothing but what falls below
// the normal range; int8: top / 127, which uses the codes' whole range.  A
// magnitude that is not finite gives NaN, which every reader of the page sees.
template <bool kInt8>
__host__ __device__ __forceinline__ float page_scale(uint32_t top_bits);
template <>
__host__ __device__ __forceinline__ float page_scale<false>(uint32_t top_bits) {
  uint32_t bits = 0x7fc00000u;
  if (top_bits < kInfBits) {
    // the exponent, one higher where the significand is above 1.75
    const int e = static_cast<int>((top_bits + 0x1fffffu) >> 23) - 127 - 8;
    bits = static_cast<uint32_t>((e < -100 ? -100 : e) + 127) << 23;
  }
#ifdef __CUDA_ARCH__
  return __uint_as_float(bits);
#else
  float f;
  __builtin_memcpy(&f, &bits, 4);
  return f;
#endif
}
template <>
__host__ __device__ __forceinline__ float page_scale<true>(uint32_t top_bits) {
#ifdef __CUDA_ARCH__
  if (top_bits >= kInfBits) return __uint_as_float(0x7fc00000u);
  return fmaxf(__fdiv_rn(__uint_as_float(top_bits), 127.0f), kMinPageScale);
#else
  float top;
  __builtin_memcpy(&top, &top_bits, 4);
  if (top_bits >= kInfBits) return __builtin_nanf("");
  const float s = top / 127.0f;
  return s > kMinPageScale ? s : kMinPageScale;
#endif
}

// Slots of a sequence after an append: its `count` new tokens are the last of
// its first `len` slots (both clamped to the capacity and to `T` tokens given);
// token i sits at slot first + i and tokens before `skip` have no slot.
struct AppendSpan {
  int first, skip, end;      // new slots: first + skip .. end - 1
};
__host__ __device__ __forceinline__ AppendSpan append_span(int len, int count, int T,
                                                           int capacity) {
  AppendSpan a;
  if (count < 0) count = 0;
  if (count > T) count = T;
  const int real = len < 0 ? 0 : len;
  a.first = real - count;                        // may be negative: those tokens have no slot
  a.skip = a.first < 0 ? -a.first : 0;
  a.end = real < capacity ? real : capacity;
  if (a.end < a.first + a.skip) a.end = a.first + a.skip;
  return a;
}
// Pages that `T` tokens in a row can touch at most.
__host__ __device__ __forceinline__ int append_pages(int T, int page) {
  return static_cast<int>((static_cast<long long>(T) + page - 2) / page) + 1;
}

}  // namespace fa
