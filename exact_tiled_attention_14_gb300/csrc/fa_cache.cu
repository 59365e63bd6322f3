// fa_cache.cu — the entry points fa_cache_append and fa_cache_read of the C
// ABI declared in include/fa.h: new keys and values into a paged 8-bit cache,
// and its tokens back as 16-bit keys and values.
//
// Both move bytes: an appended element is read in 16 bits and written in 8,
// a read one the other way round, so HBM bounds them; few tokens are bound by
// one launch and its chain of dependent loads (length, table, tokens).
//
// Append.  A page's scale needs the largest magnitude of all its new elements
// before the first one can be written, so each page is one worker's, with its
// new elements of one head in registers, and nothing is read twice.  Only the
// page that the sequence's earlier tokens fill in part has codes to keep; when
// a new token raises its scale, their owners quantise them again.
//  - Up to kFewTokens tokens: a warp takes one page and head of k or of v, four
//    elements a lane and token (64 sequences, 8 heads, d = 128: one token 6.2 us,
//    10.3 with the blocks below; eight tokens 8.2 and 8.9).
//  - More: a block of 64 to 1024 threads takes a page for up to four heads, a
//    thread holding one unit of 16 elements (see fa_rotary.cuh).  The tokens
//    of all heads are copied to shared memory at once, each thread's own, and
//    arrive while the cosines and sines, the same for all heads, are formed.
//    Four prompts of 2049 to 8192 tokens, 8 heads, d = 128 (84 MB in, 42 out): 38
//    us against 18.5 of their bytes, 43 as int8 codes.  15 instructions an element (angles,
//    unpacking, two reductions, the codes) take half of the issue slots, and
//    the blocks wait at a barrier for each head; one barrier for all four heads
//    (41 us) and equal runs of heads for persistent blocks (39) were slower.
// Read.  16 elements a thread and step, stored as 32 bytes at once so that every
// sector is written whole (where the outputs begin at one): four caches of 2048 to 16384 tokens 57 us (71 as two
// halves; int8 62), 6.1 TB/s with two thirds of it writes.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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

// A worker's place: the page's number in its sequence and first slot, whether it
// gets tokens, the new slots lo .. end - 1 of the sequence and token 0's slot.
struct AppendPage {
  int nth, slot0, lo, end, first;
  bool some;
};
__device__ __forceinline__ AppendPage append_page(const AppendParams& p, int b, int nth_new) {
  const AppendSpan a = append_span(p.seqlens[b], p.counts ? p.counts[b] : p.T, p.T, p.capacity);
  AppendPage x;
  x.first = a.first;
  x.lo = a.first + a.skip;
  x.end = a.end;
  x.nth = x.lo / p.page + nth_new;
  x.slot0 = x.nth * p.page;
  x.some = x.slot0 < a.end && x.lo < a.end;
  return x;
}
// The page itself (of a place that gets tokens), -1 where the table names none.
__device__ __forceinline__ int append_id(const AppendParams& p, int b, const AppendPage& pg) {
  const int id = p.table[static_cast<size_t>(b) * p.per_seq + pg.nth];
  return id < p.pages ? id : -1;
}
// The scale that a page goes on with: a page with earlier tokens keeps `before`
// unless `now` is larger; a NaN on either side stays.
__device__ __forceinline__ float append_scale(bool partly, float before, float now) {
  if (!partly || before < now) return now;
  return before == before && now != now ? now : before;
}
// New codes under a scale of NaN are 0, not NaN: a weight of 0 times a code must be
// 0 for the tokens that do not see the page.
__device__ __forceinline__ uint32_t append_mask(float scale) { return scale == scale ? ~0u : 0u; }
// Angles of a unit's pairs first .. first + kPairs - 1.
template <int kPairs>
__device__ __forceinline__ void append_angles(const AppendParams& p, int b, int token, int slot,
                                              int first, float* c, float* s) {
  const int pos = p.positions ? p.positions[static_cast<size_t>(b) * p.T + token] : slot;
  const ulonglong2* const f = reinterpret_cast<const ulonglong2*>(p.freqs + first);
#pragma unroll
  for (int j = 0; j < kPairs / 2; ++j) {
    const ulonglong2 w = __ldg(f + j);
    rotary_cos_sin(pos, w.x, p.mscale, c[2 * j], s[2 * j]);
    rotary_cos_sin(pos, w.y, p.mscale, c[2 * j + 1], s[2 * j + 1]);
  }
}

// One warp: a page and head of k or of v with up to kFewTokens new tokens.
constexpr int kFewTokens = 8, kFewThreads = 128;
template <bool kBf16, bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(kFewThreads)
    fa_cache_append_few_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31, width = 16 << p.per_row;
  const int h = blockIdx.y * (kFewThreads / 32) + (threadIdx.x >> 5), which = blockIdx.z;
  if (h >= p.Hk) return;
  const int b = blockIdx.x / p.n_pages;
  const AppendPage pg = append_page(p, b, blockIdx.x - b * p.n_pages);
  if (!pg.some) return;
  const int id = append_id(p, b, pg);
  if (id < 0) return;
  const int keep = pg.lo - pg.slot0;
  const int lo = max(pg.lo, pg.slot0), n = min(pg.end, pg.slot0 + p.page) - lo;
  const size_t head = static_cast<size_t>(id) * p.Hk + h;
  const float before = keep > 0 ? p.scale[which][head] : 0.0f;
  // four elements of a row: two pairs, or four behind the rotated ones
  const bool turned = which == 0 && p.freqs != nullptr && lane * 4 < p.rot;
  const bool halves = turned && !kInterleaved;
  const int c0 = halves ? lane * 2 : lane * 4, c1 = halves ? lane * 2 + p.rot / 2 : lane * 4 + 2;
  const bool on = lane * 4 < width;
  const uint16_t* const in = p.in[which] + b * p.sb[which] + h * p.sh[which];
  uint32_t raw[kFewTokens][2];
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    raw[i][0] = raw[i][1] = 0;
    if (i < n && on) {
      const uint16_t* const src = in + (lo + i - pg.first) * p.st[which];
      raw[i][0] = *reinterpret_cast<const uint32_t*>(src + c0);
      raw[i][1] = *reinterpret_cast<const uint32_t*>(src + c1);
    }
  }
  float x[kFewTokens][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    ptx::unpack2<kBf16>(raw[i][0], x[i][0], x[i][1]);
    ptx::unpack2<kBf16>(raw[i][1], x[i][2], x[i][3]);
    if (turned && i < n) {
      float c[2], s[2];
      append_angles<2>(p, b, lo + i - pg.first, lo + i, lane * 2, c, s);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ia = kInterleaved ? 2 * j : j, ib = kInterleaved ? 2 * j + 1 : j + 2;
        const float a = x[i][ia], e = x[i][ib];
        x[i][ia] = fmaf(a, c[j], -(e * s[j]));
        x[i][ib] = fmaf(e, c[j], a * s[j]);
      }
    }
    // magnitudes compared as bits: NaN is above everything
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const float scale = append_scale(keep > 0, before, page_scale<kInt8>(top));
  const float inverse = __frcp_rn(scale);
  const uint32_t written = append_mask(scale);
  uint8_t* const dst = p.cache[which] + head * p.page * width;
  if (lane == 0) p.scale[which][head] = scale;
  if (!on) return;
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    if (i < n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] *= inverse;
      const uint32_t codes = to_codes4<kInt8>(x[i]) & written;
      uint8_t* const row = dst + (lo + i - pg.slot0) * width;
      *reinterpret_cast<uint16_t*>(row + c0) = static_cast<uint16_t>(codes);
      *reinterpret_cast<uint16_t*>(row + c1) = static_cast<uint16_t>(codes >> 16);
    }
  }
  if (keep > 0 && before < scale) {
    // earlier codes under the old scale, quantised under the new one
    const float f = before * inverse;
    uint32_t* const col = reinterpret_cast<uint32_t*>(dst) + lane;
#pragma unroll 8
    for (int r = 0; r < keep; ++r) {
      float y[4];
      codes4_float<kInt8>(col[r * (width / 4)], y);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] *= f;
      col[r * (width / 4)] = to_codes4<kInt8>(y);
    }
  }
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

constexpr int kPageHeads = 4;      // heads of a block at most
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <bool kBf16, bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(1024)
    fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ uint4 tokens_s[];       // [head][vector of the thread][thread]
  __shared__ uint32_t top_s[2][32];
  const int b = blockIdx.x / p.n_pages, which = blockIdx.z;
  const int page = p.page, threads = blockDim.x;
  const AppendPage pg = append_page(p, b, blockIdx.x - b * p.n_pages);
  if (!pg.some) return;
  const int keep = pg.lo - pg.slot0;        // rows of earlier tokens (<= 0: none)
  const int width = 16 << p.per_row;        // d
  const bool turn = which == 0 && p.freqs != nullptr;
  const int h0 = blockIdx.y * p.chunk, heads = min(p.chunk, p.Hk - h0);
  const int row = threadIdx.x >> p.per_row, slot = pg.slot0 + row;
  const RotaryUnit u =
      rotary_unit(threadIdx.x & ((1 << p.per_row) - 1), turn ? p.rot : 0, kInterleaved);
  const bool fresh = slot >= pg.lo && slot < pg.end;
  const uint32_t mine = ptx::smem_u32(tokens_s + threadIdx.x);
  {
    const uint16_t* src =
        p.in[which] + b * p.sb[which] + h0 * p.sh[which] + (slot - pg.first) * p.st[which];
#pragma unroll
    for (int k = 0; k < kPageHeads; ++k) {
      if (k < heads && fresh) {
        copy16(mine + (2 * k * threads) * 16, src + u.first);
        copy16(mine + ((2 * k + 1) * threads) * 16, src + u.second);
        src += p.sh[which];
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  const int id = append_id(p, b, pg);
  float c[8], s[8];
  if (u.turned && fresh)
    append_angles<8>(p, b, slot - pg.first, slot, kInterleaved ? u.first / 2 : u.first, c, s);
  if (id < 0) {                             // no page: the copies land before the block ends
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    return;
  }

  float* const scale_at = p.scale[which] + static_cast<size_t>(id) * p.Hk + h0;
  uint8_t* out = p.cache[which] + ((static_cast<size_t>(id) * p.Hk + h0) * page + row) * width;
#pragma unroll 1
  for (int k = 0; k < heads; ++k, out += page * width) {
    // the thread's own copies of head k; those of later heads may be on their way
    if (k == 0)
      asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (k == 1)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (k == 2)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    float x[16], largest = 0.f;
    const float before = keep > 0 ? scale_at[k] : 0.0f;
    if (fresh) {
      unpack8<kBf16>(tokens_s[2 * k * threads + threadIdx.x], x);
      unpack8<kBf16>(tokens_s[(2 * k + 1) * threads + threadIdx.x], x + 8);
      if (u.turned) rotary_turn<kInterleaved>(x, c, s);
#pragma unroll
      for (int j = 0; j < 16; j += 2) largest = max3_nan(largest, fabsf(x[j]), fabsf(x[j + 1]));
    }
    // compared as bits: NaN is above everything
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(largest) & 0x7fffffffu);
    uint32_t* const shared = top_s[k & 1];  // one barrier a head
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = top;
    __syncthreads();
    top = (threadIdx.x & 31) < (threads >> 5) ? shared[threadIdx.x & 31] : 0u;
    top = __reduce_max_sync(0xffffffffu, top);
    const float scale = append_scale(keep > 0, before, page_scale<kInt8>(top));
    const float inverse = __frcp_rn(scale);
    const uint32_t written = append_mask(scale);
    if (threadIdx.x == 0) scale_at[k] = scale;
    if (fresh) {
      const uint64_t i2 = ptx::f2_pack(inverse, inverse);
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(x[j], x[j + 1]), i2), x[j], x[j + 1]);
    } else if (row < keep && before < scale) {
      // codes under the old scale, quantised under the new one
      const float f = before * inverse;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint2 w = *reinterpret_cast<const uint2*>(out + (half ? u.second : u.first));
        codes4_float<kInt8>(w.x, x + 8 * half);
        codes4_float<kInt8>(w.y, x + 8 * half + 4);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= f;
    } else {
      continue;
    }
    *reinterpret_cast<uint2*>(out + u.first) =
        make_uint2(to_codes4<kInt8>(x) & written, to_codes4<kInt8>(x + 4) & written);
    *reinterpret_cast<uint2*>(out + u.second) =
        make_uint2(to_codes4<kInt8>(x + 8) & written, to_codes4<kInt8>(x + 12) & written);
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
  bool sectors;               // both outputs begin at a multiple of 32 bytes
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
      const uint4 lo = pack8<kBf16>(x), hi = pack8<kBf16>(x + 8);
      if (p.sectors) {
        ptx::store32(out + unit * 16, lo, hi);
      } else {
        *reinterpret_cast<uint4*>(out + unit * 16) = lo;
        *reinterpret_cast<uint4*>(out + unit * 16 + 8) = hi;
      }
    }
  }
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <bool kBf16, bool kInt8, bool kInterleaved>
cudaError_t append_variant(const AppendParams& p, int rows, int threads, cudaStream_t stream) {
  if (p.T <= kFewTokens) {
    const int warps = kFewThreads / 32;
    const dim3 grid(rows, (p.Hk + warps - 1) / warps, 2);
    fa_cache_append_few_kernel<kBf16, kInt8, kInterleaved><<<grid, kFewThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  static std::atomic<uint64_t> done{0};   // devices on which the smem limit was raised
  auto kernel = fa_cache_append_kernel<kBf16, kInt8, kInterleaved>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPageHeads * 1024 * 32);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  const dim3 grid(rows, (p.Hk + p.chunk - 1) / p.chunk, 2);
  kernel<<<grid, threads, p.chunk * threads * 32, stream>>>(p);
  return cudaGetLastError();
}
template <bool kBf16, bool kInt8>
cudaError_t append(const AppendParams& p, bool interleaved, int rows, int threads,
                   cudaStream_t stream) {
  return interleaved ? append_variant<kBf16, kInt8, true>(p, rows, threads, stream)
                     : append_variant<kBf16, kInt8, false>(p, rows, threads, stream);
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
  if (T < 0 || static_cast<long long>(B) * T > (1 << 30) || Hk > 65535) return FA_ERR_SHAPE;
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
  const int threads = page_size * d / 16;   // 64 .. 1024
  // Heads of a block: as many as leave the GPU's thread slots filled once over.
  const long long slots = static_cast<long long>(info->sms) * 1024;
  p.chunk = static_cast<int>(std::min<long long>(
      std::max(n_pages * B * 2 * threads * Hk / slots, 1ll), fa::kPageHeads));
  const int rows = static_cast<int>(n_pages * B);
  const bool inter = interleaved != 0, bf16 = dtype == FA_BF16;
  cudaError_t e;
  if (cache_dtype == FA_INT8)
    e = bf16 ? fa::append<true, true>(p, inter, rows, threads, stream)
             : fa::append<false, true>(p, inter, rows, threads, stream);
  else
    e = bf16 ? fa::append<true, false>(p, inter, rows, threads, stream)
             : fa::append<false, false>(p, inter, rows, threads, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
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
  p.sectors = !misaligned(k, 32) && !misaligned(v, 32);
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
