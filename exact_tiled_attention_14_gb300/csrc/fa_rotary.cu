// fa_rotary.cu — the entry point fa_rotary of the C ABI declared in
// include/fa.h: rotation of queries and keys by their positions, and back.
//
// One pass over memory: each element of q and k is read once and written
// once, 4 bytes an element against about three operations, so HBM bounds it.
// A thread owns one unit (16 elements, see fa_rotary.cuh) of one token and
// walks over several heads with the unit's eight cosines and sines in
// registers, since every head of a token turns by the same angles: at about 30
// instructions a pair they cost as much as several heads' loads, products and
// stores.  16384 tokens of 32 + 8 heads, d = 128 (336 MB): 54 us a call, 6.2 TB/s
// of the 6.8 of a copy; 32 single tokens 6, which is the launch.  Rows are read through their strides, so that the slices of a fused
// projection's output go straight to the [B, H, N, d] layout that the
// attention kernels read.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.cuh"
#include "fa_rotary.cuh"

using namespace fa::host;

namespace fa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 4;      // heads whose loads are in flight together

// One tensor, strides in elements (batch, head, token).
struct RotaryTensor {
  const uint16_t* in;
  uint16_t* out;
  long long ib, ih, in_, ob, oh, on;
};

struct RotaryParams {
  RotaryTensor q, k;
  const unsigned long long* freqs;   // [rot / 2]
  const int* positions;              // [B, N] or NULL
  const int* seqlens;                // [B] or NULL
  long long units;                   // B * N * d / 16
  int N, H, heads, rot;              // heads: H + Hk
  int per_row;                       // log2 of a row's units
  int chunk;                         // heads of a thread
  float mscale;
  bool inverse;
};

template <bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads)
    fa_rotary_kernel(const __grid_constant__ RotaryParams p) {
  const long long at = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x;
  if (at >= p.units) return;
  const long long token = at >> p.per_row;
  const RotaryUnit u =
      rotary_unit(static_cast<int>(at) & ((1 << p.per_row) - 1), p.rot, kInterleaved);
  const long long b = token / p.N;
  const int n = static_cast<int>(token - b * p.N);
  float c[8], s[8];
  if (u.turned) {
    int pos = n;
    if (p.positions)
      pos = p.positions[token];
    else if (p.seqlens)     // (wraps as integers wrap, like the angle)
      pos = static_cast<int>(static_cast<uint32_t>(p.seqlens[b]) - p.N + n);
    const int pair = kInterleaved ? u.first / 2 : u.first;
    const ulonglong2* const f = reinterpret_cast<const ulonglong2*>(p.freqs + pair);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 w = __ldg(f + i);
      rotary_cos_sin(pos, w.x, p.mscale, c[2 * i], s[2 * i]);
      rotary_cos_sin(pos, w.y, p.mscale, c[2 * i + 1], s[2 * i + 1]);
    }
    if (p.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
  }
  const int end = min((static_cast<int>(blockIdx.y) + 1) * p.chunk, p.heads);
  for (int h0 = blockIdx.y * p.chunk; h0 < end; h0 += kRotBatch) {
    uint4 v[kRotBatch][2];
#pragma unroll
    for (int i = 0; i < kRotBatch; ++i) {
      if (h0 + i < end) {
        const bool is_q = h0 + i < p.H;
        const RotaryTensor& t = is_q ? p.q : p.k;
        const uint16_t* const row =
            t.in + b * t.ib + (is_q ? h0 + i : h0 + i - p.H) * t.ih + n * t.in_;
        v[i][0] = *reinterpret_cast<const uint4*>(row + u.first);
        v[i][1] = *reinterpret_cast<const uint4*>(row + u.second);
      }
    }
#pragma unroll
    for (int i = 0; i < kRotBatch; ++i) {
      if (h0 + i < end) {
        const bool is_q = h0 + i < p.H;
        const RotaryTensor& t = is_q ? p.q : p.k;
        uint16_t* const row =
            t.out + b * t.ob + (is_q ? h0 + i : h0 + i - p.H) * t.oh + n * t.on;
        if (u.turned) {
          float x[16];
          unpack8<kBf16>(v[i][0], x);
          unpack8<kBf16>(v[i][1], x + 8);
          rotary_turn<kInterleaved>(x, c, s);
          v[i][0] = pack8<kBf16>(x);
          v[i][1] = pack8<kBf16>(x + 8);
        }
        *reinterpret_cast<uint4*>(row + u.first) = v[i][0];
        *reinterpret_cast<uint4*>(row + u.second) = v[i][1];
      }
    }
  }
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_rotary(const void* q, const void* k, void* q_out, void* k_out, int B, int H, int Hk, int N,
              int d, const long long* strides, const unsigned long long* freqs, int rot,
              float mscale, int interleaved, int inverse, const int* positions, const int* seqlens,
              int dtype, cudaStream_t stream) {
  if (B < 0 || H < 0 || Hk < 0 || N < 0 || d <= 0) return FA_ERR_SHAPE;
  const long long tokens = static_cast<long long>(B) * N;
  const long long heads = static_cast<long long>(H) + Hk;
  if (tokens > (1 << 30) || heads > (1 << 30)) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_SHAPE;
  if (positions && seqlens) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!std::isfinite(mscale) || !(mscale > 0.0f)) return FA_ERR_SCALE;
  if (tokens == 0 || heads == 0) return FA_OK;
  if (!freqs || !strides || (H > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)))
    return FA_ERR_NULLPTR;
  auto misaligned = [](const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(q_out, 16) || misaligned(k_out, 16) ||
      misaligned(freqs, 16) || misaligned(positions, 4) || misaligned(seqlens, 4))
    return FA_ERR_ALIGN;
  for (int i = H > 0 ? 0 : 6; i < (Hk > 0 ? 12 : 6); ++i)
    if (strides[i] % 8 != 0) return FA_ERR_ALIGN;

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;
  fa::RotaryParams p{};
  auto tensor = [&](const void* in, void* out, const long long* st) {
    return fa::RotaryTensor{static_cast<const uint16_t*>(in), static_cast<uint16_t*>(out),
                            st[0], st[1], st[2], st[3], st[4], st[5]};
  };
  p.q = tensor(q, q_out, strides);
  p.k = tensor(k, k_out, strides + 6);
  p.freqs = freqs;
  p.positions = positions;
  p.seqlens = seqlens;
  p.per_row = d == 128 ? 3 : 2;
  p.units = tokens << p.per_row;
  p.N = N;
  p.H = H;
  p.heads = static_cast<int>(heads);
  p.rot = rot;
  p.mscale = mscale;
  p.inverse = inverse != 0;
  // Heads of a thread: as many as leave the GPU's thread slots filled once
  // over, so that a call of few tokens spreads and one of many shares angles.
  const long long slots = static_cast<long long>(info->sms) * 2048;
  p.chunk = static_cast<int>(std::min(std::max(p.units * heads / slots, 1ll), 8ll));
  if (p.chunk > fa::kRotBatch) p.chunk = 2 * fa::kRotBatch;
  while ((heads + p.chunk - 1) / p.chunk > 65535) p.chunk *= 2;
  const dim3 grid(static_cast<unsigned>((p.units + fa::kRotThreads - 1) / fa::kRotThreads),
                  static_cast<unsigned>((heads + p.chunk - 1) / p.chunk));
  if (dtype == FA_BF16) {
    if (interleaved)
      fa::fa_rotary_kernel<true, true><<<grid, fa::kRotThreads, 0, stream>>>(p);
    else
      fa::fa_rotary_kernel<true, false><<<grid, fa::kRotThreads, 0, stream>>>(p);
  } else {
    if (interleaved)
      fa::fa_rotary_kernel<false, true><<<grid, fa::kRotThreads, 0, stream>>>(p);
    else
      fa::fa_rotary_kernel<false, false><<<grid, fa::kRotThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
