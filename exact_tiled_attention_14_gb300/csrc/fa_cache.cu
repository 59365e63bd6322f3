// fa_cache.cu — the entry points fa_cache_append and fa_cache_read of the C
// ABI declared in include/fa.h: new keys and values into a paged 8-bit cache,
// and its tokens back as 16-bit keys and values.
//
// Both move bytes: an appended element is read in 16 bits and written in 8,
// a read one the other way round, so HBM bounds them; few tokens are bound by
// one launch and its chain of dependent loads (length, table, tokens).
//
// Append.  A page's scale needs the largest magnitude of all its new elements
// before the first one can be written, so a block takes whole pages: one page
// of a sequence, for several heads of k or of v, with the page's elements of
// one head in registers (a thread holds two units of 16, see fa_rotary.cuh;
// 32 to 1024 threads).  Nothing is read twice, and the cosines and sines of a
// thread's pairs serve all heads that its block walks over.  Only the page
// that the sequence's earlier tokens fill in part has codes to keep; when a
// new token raises its scale, the thread that owns their unit quantises them
// again.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.cuh"
#include "fa_paged.cuh"
#include "fa_rotary.cuh"

using namespace fa::host;

namespace fa {
namespace {

struct AppendParams {
  const uint16_t* in[2];      // k, v
  long long sb[2], sh[2], st[2];
  uint8_t* cache[2];
  float* scale[2];
  const int* table;
  const int* seqlens;
  const int* counts;          // [B] or NULL: T
  const int* positions;       // [B, T] or NULL: the slot
  const unsigned long long* freqs;   // NULL: no rotation
  int Hk, T, page, per_seq, pages, n_pages, rot, chunk, capacity;
  int per_row;                // log2 of a row's units
  float mscale;
};

template <bool kBf16, bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(512)
    fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ uint32_t top_s[2][16];
  const int b = blockIdx.x / p.n_pages, which = blockIdx.z;
  const int T = p.T, page = p.page;
  const AppendSpan a =
      append_span(p.seqlens[b], p.counts ? p.counts[b] : T, T, p.capacity);
  const int lo = a.first + a.skip;                            // first new slot
  const int nth = lo / page + (blockIdx.x - b * p.n_pages);   // page of the sequence
  const int slot0 = nth * page;
  if (slot0 >= a.end || lo >= a.end) return;
  const int id = p.table[static_cast<size_t>(b) * p.per_seq + nth];
  if (id < 0 || id >= p.pages) return;
  const int keep = lo - slot0;            // rows of earlier tokens (<= 0: none)

  const int width = 16 << p.per_row;      // d
  const int threads = blockDim.x;
  const bool turn = which == 0 && p.freqs != nullptr;
  int row[2];
  RotaryUnit u[2];
  float c[2][8], s[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int unit = threadIdx.x + i * threads;
    row[i] = unit >> p.per_row;
    u[i] = rotary_unit(unit & ((1 << p.per_row) - 1), turn ? p.rot : 0, kInterleaved);
    const int slot = slot0 + row[i];
    if (u[i].turned && row[i] < page && slot >= lo && slot < a.end) {
      const int pos =
          p.positions ? p.positions[static_cast<size_t>(b) * T + (slot - a.first)] : slot;
      const int pair = kInterleaved ? u[i].first / 2 : u[i].first;
      const ulonglong2* const f = reinterpret_cast<const ulonglong2*>(p.freqs + pair);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const ulonglong2 w = __ldg(f + j);
        rotary_cos_sin(pos, w.x, p.mscale, c[i][2 * j], s[i][2 * j]);
        rotary_cos_sin(pos, w.y, p.mscale, c[i][2 * j + 1], s[i][2 * j + 1]);
      }
    }
  }

  const uint16_t* const in = p.in[which] + b * p.sb[which];
  const int end = min((static_cast<int>(blockIdx.y) + 1) * p.chunk, p.Hk);
  for (int h = blockIdx.y * p.chunk; h < end; ++h) {
    float x[2][16];
    bool fresh[2];
    uint32_t top = 0;
    const size_t head = static_cast<size_t>(id) * p.Hk + h;
    const float before = keep > 0 ? p.scale[which][head] : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int slot = slot0 + row[i];
      fresh[i] = row[i] < page && slot >= lo && slot < a.end;
      if (fresh[i]) {
        const uint16_t* const src = in + h * p.sh[which] + (slot - a.first) * p.st[which];
        unpack8<kBf16>(*reinterpret_cast<const uint4*>(src + u[i].first), x[i]);
        unpack8<kBf16>(*reinterpret_cast<const uint4*>(src + u[i].second), x[i] + 8);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (fresh[i]) {
        if (u[i].turned) rotary_turn<kInterleaved>(x[i], c[i], s[i]);
        // magnitudes compared as bits: NaN is above everything
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    uint32_t* const shared = top_s[(h - blockIdx.y * p.chunk) & 1];   // one barrier a head
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = top;
    __syncthreads();
    top = shared[threadIdx.x & 15];
    top = __reduce_max_sync(0xffffffffu,
                            (threadIdx.x & 31) < (threads >> 5) ? top : 0u);
    float scale = page_scale<kInt8>(top);
    // a NaN on either side stays
    if (keep > 0 && !(before < scale)) scale = before == before && scale != scale ? scale : before;
    const float inverse = __frcp_rn(scale);
    uint8_t* const dst = p.cache[which] + head * page * width;
    if (threadIdx.x == 0) p.scale[which][head] = scale;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint8_t* const out = dst + row[i] * width;
      if (fresh[i]) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] *= inverse;
      } else if (row[i] < keep && before < scale) {
        // codes under the old scale, quantised under the new one
        const float f = before * inverse;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint2 w = *reinterpret_cast<const uint2*>(out + (half ? u[i].second : u[i].first));
          codes4_float<kInt8>(w.x, x[i] + 8 * half);
          codes4_float<kInt8>(w.y, x[i] + 8 * half + 4);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] *= f;
      } else {
        continue;
      }
      *reinterpret_cast<uint2*>(out + u[i].first) =
          make_uint2(to_codes4<kInt8>(x[i]), to_codes4<kInt8>(x[i] + 4));
      *reinterpret_cast<uint2*>(out + u[i].second) =
          make_uint2(to_codes4<kInt8>(x[i] + 8), to_codes4<kInt8>(x[i] + 12));
    }
  }
}

struct ReadParams {
  const uint8_t* cache[2];
  const float* scale[2];
  uint16_t* out[2];           // [B, Hk, N, d]
  const int* table;
  const int* seqlens;
  int Hk, N, page, per_seq, pages;
  int per_row;
  long long units;            // of one head of one sequence: N * d / 16
};

// A thread takes kReadUnits units of 16 elements, a block's width apart, of
// one head of one sequence.
constexpr int kReadThreads = 256, kReadUnits = 4;

template <bool kBf16, bool kInt8>
__global__ void __launch_bounds__(kReadThreads)
    fa_cache_read_kernel(const __grid_constant__ ReadParams p) {
  const int which = blockIdx.z & 1, b = blockIdx.z >> 1;
  const long long first =
      static_cast<long long>(blockIdx.x) * (kReadThreads * kReadUnits) + threadIdx.x;
  const int width = 16 << p.per_row;
  for (int h = blockIdx.y; h < p.Hk; h += gridDim.y) {
    const int len = min(p.seqlens[b], p.per_seq * p.page);
    uint16_t* const out =
        p.out[which] + (static_cast<size_t>(b) * p.Hk + h) * p.N * width;
    uint4 codes[kReadUnits];
    float scale[kReadUnits];
#pragma unroll
    for (int i = 0; i < kReadUnits; ++i) {
      const long long unit = first + i * kReadThreads;
      const int n = static_cast<int>(unit >> p.per_row);
      scale[i] = 0.0f;
      codes[i] = make_uint4(0, 0, 0, 0);
      if (unit < p.units && n < len) {
        const int nth = n / p.page;
        const int id = p.table[static_cast<size_t>(b) * p.per_seq + nth];
        if (id >= 0 && id < p.pages) {
          const size_t head = static_cast<size_t>(id) * p.Hk + h;
          scale[i] = p.scale[which][head];
          codes[i] = *reinterpret_cast<const uint4*>(
              p.cache[which] + (head * p.page + (n - nth * p.page)) * width +
              (static_cast<int>(unit) & ((1 << p.per_row) - 1)) * 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kReadUnits; ++i) {
      const long long unit = first + i * kReadThreads;
      if (unit >= p.units) continue;
      const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
      float x[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) codes4_float<kInt8>(w[j], x + 4 * j);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= scale[i];
      uint4* const dst = reinterpret_cast<uint4*>(out + unit * 16);
      dst[0] = pack8<kBf16>(x);
      dst[1] = pack8<kBf16>(x + 8);
    }
  }
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <bool kBf16, bool kInt8>
void append(const AppendParams& p, bool interleaved, dim3 grid, int threads, cudaStream_t stream) {
  if (interleaved)
    fa_cache_append_kernel<kBf16, kInt8, true><<<grid, threads, 0, stream>>>(p);
  else
    fa_cache_append_kernel<kBf16, kInt8, false><<<grid, threads, 0, stream>>>(p);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_cache_append(const void* k, const void* v, int B, int Hk, int T, int d,
                    const long long* strides, void* k_cache, void* v_cache, float* k_scale,
                    float* v_scale, int pages, int page_size, const int* page_table,
                    int pages_per_seq, const int* seqlens, const int* counts,
                    const unsigned long long* freqs, int rot, float mscale, int interleaved,
                    const int* positions, int dtype, int cache_dtype, cudaStream_t stream) {
  const int rc = check_paged(B, Hk, d, pages, page_size, pages_per_seq, cache_dtype);
  if (rc != FA_OK) return rc;
  if (T < 0 || static_cast<long long>(B) * T > (1 << 30)) return FA_ERR_SHAPE;
  if (freqs && (rot < 16 || rot > d || rot % 16 != 0)) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (freqs && (!std::isfinite(mscale) || !(mscale > 0.0f))) return FA_ERR_SCALE;
  if (B == 0 || Hk == 0 || T == 0) return FA_OK;
  const long long n_pages = fa::append_pages(T, page_size);
  if (n_pages * B > (1ll << 31) - 1) return FA_ERR_SHAPE;
  if (!k || !v || !strides || !k_cache || !v_cache || !k_scale || !v_scale || !page_table ||
      !seqlens)
    return FA_ERR_NULLPTR;
  using fa::misaligned;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_cache, 16) ||
      misaligned(v_cache, 16) || misaligned(k_scale, 4) || misaligned(v_scale, 4) ||
      misaligned(page_table, 4) || misaligned(seqlens, 4) || misaligned(counts, 4) ||
      misaligned(positions, 4) || misaligned(freqs, 16))
    return FA_ERR_ALIGN;
  for (int i = 0; i < 6; ++i)
    if (strides[i] % 8 != 0) return FA_ERR_ALIGN;

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;
  fa::AppendParams p{};
  const void* in[2] = {k, v};
  void* cache[2] = {k_cache, v_cache};
  float* scale[2] = {k_scale, v_scale};
  for (int i = 0; i < 2; ++i) {
    p.in[i] = static_cast<const uint16_t*>(in[i]);
    p.sb[i] = strides[3 * i];
    p.sh[i] = strides[3 * i + 1];
    p.st[i] = strides[3 * i + 2];
    p.cache[i] = static_cast<uint8_t*>(cache[i]);
    p.scale[i] = scale[i];
  }
  p.table = page_table;
  p.seqlens = seqlens;
  p.counts = counts;
  p.positions = positions;
  p.freqs = freqs;
  p.Hk = Hk;
  p.T = T;
  p.page = page_size;
  p.per_seq = pages_per_seq;
  p.pages = pages;
  p.capacity = pages_per_seq * page_size;
  p.n_pages = static_cast<int>(n_pages);
  p.rot = rot;
  p.mscale = mscale;
  p.per_row = d == 128 ? 3 : 2;
  const int threads = std::max(page_size * d / 32, 32);
  // Heads of a block: as many as leave the GPU's thread slots filled once over.
  const long long slots = static_cast<long long>(info->sms) * 2048;
  p.chunk = static_cast<int>(
      std::min(std::max(n_pages * B * 2 * threads * Hk / slots, 1ll), 8ll));
  while ((Hk + p.chunk - 1) / p.chunk > 65535) p.chunk *= 2;
  const dim3 grid(static_cast<unsigned>(n_pages * B),
                  static_cast<unsigned>((Hk + p.chunk - 1) / p.chunk), 2);
  const bool inter = interleaved != 0, bf16 = dtype == FA_BF16;
  if (cache_dtype == FA_INT8)
    bf16 ? fa::append<true, true>(p, inter, grid, threads, stream)
         : fa::append<false, true>(p, inter, grid, threads, stream);
  else
    bf16 ? fa::append<true, false>(p, inter, grid, threads, stream)
         : fa::append<false, false>(p, inter, grid, threads, stream);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                  const float* v_scale, void* k, void* v, int B, int Hk, int N, int d, int pages,
                  int page_size, const int* page_table, int pages_per_seq, const int* seqlens,
                  int dtype, int cache_dtype, cudaStream_t stream) {
  const int rc = check_paged(B, Hk, d, pages, page_size, pages_per_seq, cache_dtype);
  if (rc != FA_OK) return rc;
  if (N < 0 || N > (1 << 30) || B > 32767) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (B == 0 || Hk == 0 || N == 0) return FA_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !k || !v || !page_table || !seqlens)
    return FA_ERR_NULLPTR;
  using fa::misaligned;
  if (misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(k, 16) ||
      misaligned(v, 16) || misaligned(k_scale, 4) || misaligned(v_scale, 4) ||
      misaligned(page_table, 4) || misaligned(seqlens, 4))
    return FA_ERR_ALIGN;
  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;
  fa::ReadParams p{};
  p.cache[0] = static_cast<const uint8_t*>(k_cache);
  p.cache[1] = static_cast<const uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.out[0] = static_cast<uint16_t*>(k);
  p.out[1] = static_cast<uint16_t*>(v);
  p.table = page_table;
  p.seqlens = seqlens;
  p.Hk = Hk;
  p.N = N;
  p.page = page_size;
  p.per_seq = pages_per_seq;
  p.pages = pages;
  p.per_row = d == 128 ? 3 : 2;
  p.units = static_cast<long long>(N) << p.per_row;
  constexpr int kPer = fa::kReadThreads * fa::kReadUnits;
  const dim3 grid(static_cast<unsigned>((p.units + kPer - 1) / kPer),
                  static_cast<unsigned>(std::min(Hk, 65535)), static_cast<unsigned>(2 * B));
  const bool bf16 = dtype == FA_BF16;
  if (cache_dtype == FA_INT8) {
    bf16 ? fa::fa_cache_read_kernel<true, true><<<grid, fa::kReadThreads, 0, stream>>>(p)
         : fa::fa_cache_read_kernel<false, true><<<grid, fa::kReadThreads, 0, stream>>>(p);
  } else {
    bf16 ? fa::fa_cache_read_kernel<true, false><<<grid, fa::kReadThreads, 0, stream>>>(p)
         : fa::fa_cache_read_kernel<false, false><<<grid, fa::kReadThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
