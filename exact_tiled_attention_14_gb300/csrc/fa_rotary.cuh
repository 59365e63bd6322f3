// fa_rotary.cuh — rotation of query and key elements by their token's
// position, shared by the rotary kernels and the cache's append.
//
// A head's first `rot` elements are rot / 2 pairs; pair j of the token at
// position p is turned by the angle p * w_j:
//     (a, b) -> mscale * (a cos - b sin, b cos + a sin),
// and back (the gradient) by the negative angle.  Pairs are (2 j, 2 j + 1)
// (interleaved) or (j, j + rot / 2) (halves); elements from `rot` on stay.
//
// Angles.  w_j arrives as turns per position in units of 2^-64, so the
// product with the position, wrapped at 64 bits as integers wrap, is the
// angle's fraction of a turn, and whole turns cost no bits, where a float32 angle is
// off by up to a tenth of a radian at position 2^20.  What is off is the
// frequency: p * 2^-65 turns for one that is rounded to its unit, up to p * 2^-56 for
// the fastest pairs of one that comes from float64.  The fraction is cut to the
// nearest quarter turn; the rest, at most an eighth, is cut to 2^-34 turns and goes
// through the Taylor polynomials of sine and cosine in float32, of which the first
// terms left out are 2e-9 and 2.5e-8 there (about 30 operations a pair): cosine and
// sine are off by less than 2^-22, before the product with mscale.
#pragma once

#include <cstdint>

#include "ptx_sm103.cuh"

namespace fa {

__device__ __forceinline__ void rotary_cos_sin(int pos, unsigned long long freq, float mscale,
                                               float& c, float& s) {
  const unsigned long long turn =
      static_cast<unsigned long long>(static_cast<long long>(pos)) * freq;
  const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);
  // the rest in units of 2^-34 turns: the two top bits leave by themselves
  const int rest = static_cast<int>(static_cast<uint32_t>(turn >> 30));
  const float x = static_cast<float>(rest) * 3.6572954e-10f;      // 2 pi 2^-34
  const float y = x * x;
  // x - x^3 / 3! + x^5 / 5! - x^7 / 7! + x^9 / 9!
  float sn = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(y, sn, 1.f / 120.f);
  sn = fmaf(y, sn, -1.f / 6.f);
  sn = fmaf(x * y, sn, x);
  // 1 - x^2 / 2! + x^4 / 4! - x^6 / 6! + x^8 / 8!
  float cs = fmaf(y, 1.f / 40320.f, -1.f / 720.f);
  cs = fmaf(y, cs, 1.f / 24.f);
  cs = fmaf(y, cs, -0.5f);
  cs = fmaf(y, cs, 1.f);
  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
  const bool odd = quarter & 1u;
  const float u = (odd ? sn : cs) * mscale, v = (odd ? cs : sn) * mscale;
  c = __uint_as_float(__float_as_uint(u) ^ ((quarter + 1u & 2u) << 30));
  s = __uint_as_float(__float_as_uint(v) ^ ((quarter & 2u) << 30));
}

// Sixteen elements of a row that are turned together: eight pairs, or sixteen
// elements behind the rotated ones.  Unit u of a row covers vectors of eight
// elements that start at columns first(u) and second(u).
struct RotaryUnit {
  int first, second;
  bool turned;
};
__host__ __device__ __forceinline__ RotaryUnit rotary_unit(int u, int rot, bool interleaved) {
  RotaryUnit r;
  r.turned = u * 16 < rot;
  r.first = r.turned && !interleaved ? u * 8 : u * 16;
  r.second = r.turned && !interleaved ? u * 8 + rot / 2 : u * 16 + 8;
  return r;
}

// Turn a unit's values x[0..7] (first vector), x[8..15] (second), two pairs an
// instruction where their registers are neighbours.
template <bool kInterleaved>
__device__ __forceinline__ void rotary_turn(float* x, const float* c, const float* s) {
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = fmaf(a, c[i], -(b * s[i]));
      x[2 * i + 1] = fmaf(b, c[i], a * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t a = ptx::f2_pack(x[i], x[i + 1]), b = ptx::f2_pack(x[i + 8], x[i + 9]);
      const uint64_t c2 = ptx::f2_pack(c[i], c[i + 1]), s2 = ptx::f2_pack(s[i], s[i + 1]);
      const uint64_t n2 = ptx::f2_pack(-s[i], -s[i + 1]);
      ptx::f2_unpack(ptx::ffma2(a, c2, ptx::fmul2(b, n2)), x[i], x[i + 1]);
      ptx::f2_unpack(ptx::ffma2(b, c2, ptx::fmul2(a, s2)), x[i + 8], x[i + 9]);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4 v, float* x) {
  ptx::unpack2<kBf16>(v.x, x[0], x[1]);
  ptx::unpack2<kBf16>(v.y, x[2], x[3]);
  ptx::unpack2<kBf16>(v.z, x[4], x[5]);
  ptx::unpack2<kBf16>(v.w, x[6], x[7]);
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(ptx::pack2<kBf16>(x[0], x[1]), ptx::pack2<kBf16>(x[2], x[3]),
                    ptx::pack2<kBf16>(x[4], x[5]), ptx::pack2<kBf16>(x[6], x[7]));
}

}  // namespace fa
