// cache_sm100.cuh -- the paged key/value cache: addressing shared by every
// kernel that touches it, and the kernels that move tokens in and out.
//
// Position n of sequence b is token n % page_size of page table[b][n / page_size].
// Quantised rows (e4m3 codes, one fp32 scale per token and kv head): with a =
// max |x| clamped to [2^-100, FLT_MAX], scale = a / 448, code = rn(x * (448 / a)),
// value = code * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>
#include <stdint.h>

#include "layout.cuh"

namespace fa {

struct CacheParams {
  uint8_t* k;  // pages, bf16 or e4m3
  uint8_t* v;
  float* ks;  // scales (e4m3)
  float* vs;
  const int* table;
  const int* seqlens;
  Strides pages, scales;  // elements; b = page, h = kv head, n = token
  long long table_stride;
  int B, Hkv, num_pages, page_size, max_pages;
  uint32_t page_mul;  // ceil(2^(31 + page_shift) / page_size), page_shift = ceil(log2 page_size)
  int page_shift;
};

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxLo = 7.888609052210118e-31f;  // 2^-100: 448 / a stays finite

__device__ __forceinline__ int cache_length(const CacheParams& c, int b) {
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  return static_cast<int>(max(0LL, min(static_cast<long long>(c.seqlens[b]), cap)));
}

// pos / page_size for 0 <= pos < 2^31: with e = page_mul * page_size - 2^(31 +
// page_shift) < page_size <= 2^page_shift, pos * e / 2^(31 + page_shift) < 1.
__device__ __forceinline__ int page_of(const CacheParams& c, int pos) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(pos)) * c.page_mul) >> (31 + c.page_shift));
}

// Page of position pos (0 <= pos < cache_length) of sequence b, or -1; *slot:
// the token inside the page.
__device__ __forceinline__ int cache_page(const CacheParams& c, int b, int pos, int* slot) {
  const int i = page_of(c, pos);
  *slot = pos - i * c.page_size;
  const int page = c.table[b * c.table_stride + i];
  return page >= 0 && page < c.num_pages ? page : -1;
}

// Two e4m3 codes (the low one first) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(x, __NV_E4M3);
  return __half22float2(__half2(h));
}

// ---------------------------------------------------------------- moving tokens
struct MoveParams {
  CacheParams c;
  uint8_t* k;  // dense tokens [T, Hkv, D] bf16: read by the write kernel, written by the read kernel
  uint8_t* v;
  long long k_row, k_head, v_row, v_head;  // elements
  const int* cu;                           // [B + 1] offsets of the sequences' rows
  int T;
};

// Sequence b with cu[b] <= t < cu[b + 1], or -1: a search by the whole warp, 32
// offsets a step (two dependent loads for up to 1024 sequences).
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t, int lane) {
  int lo = 0, hi = B;  // the answer is the number of b in [0, B) with cu[b + 1] <= t
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;
    const unsigned m = __ballot_sync(0xffffffffu, i < hi && cu[i + 1] <= t);
    lo += __popc(m) * step;
    hi = min(hi, lo + step);
  }
  const unsigned m = __ballot_sync(0xffffffffu, lo + lane < hi && cu[lo + lane + 1] <= t);
  const int b = lo + __popc(m);
  return b < B && cu[b] <= t && t < cu[b + 1] ? b : -1;
}

constexpr int kMoveWarps = 8;
constexpr int kMoveUnroll = 4;  // loads of 512 bytes that a warp has in flight

// A warp moves kMoveUnroll * 32 / (D / 8) rows of one token (its K and V rows,
// alternating, head after head); D / 8 lanes hold a row, 16 bytes of bf16 each.
template <int D, bool kQuant, bool kWrite>
__global__ void __launch_bounds__(32 * kMoveWarps) cache_move_kernel(const MoveParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int chunks = (2 * p.c.Hkv + kRows * kMoveUnroll - 1) / (kRows * kMoveUnroll);
  const long long task = static_cast<long long>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(task / chunks);
  if (t >= p.T) return;
  const int r0 = static_cast<int>(task % chunks) * kRows * kMoveUnroll + lane / kLanes;
  const int col = (lane % kLanes) * 8;

  const int b = find_sequence(p.cu, p.c.B, t, lane);
  if (b < 0) return;
  const int pos = cache_length(p.c, b) - (p.cu[b + 1] - t);
  int slot = 0;
  const int page = pos >= 0 ? cache_page(p.c, b, pos, &slot) : -1;
  if (kWrite && page < 0) return;

  uint4 x[kMoveUnroll];
  float sc[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int r = r0 + u * kRows, h = r >> 1;
    x[u] = make_uint4(0, 0, 0, 0);
    sc[u] = 0.f;
    if (h >= p.c.Hkv) continue;
    if (kWrite) {
      const uint8_t* src = (r & 1) ? p.v : p.k;
      const long long at = (r & 1) ? t * p.v_row + h * p.v_head : t * p.k_row + h * p.k_head;
      x[u] = __ldg(reinterpret_cast<const uint4*>(src + (at + col) * 2));
    } else if (page >= 0) {
      const uint8_t* src = (r & 1) ? p.c.v : p.c.k;
      const long long at = p.c.pages.row(page, h, slot) + col;
      if (kQuant) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + at);
        x[u].x = w.x;
        x[u].y = w.y;
        sc[u] = ((r & 1) ? p.c.vs : p.c.ks)[p.c.scales.row(page, h, slot)];
      } else {
        x[u] = *reinterpret_cast<const uint4*>(src + at * 2);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int r = r0 + u * kRows, h = r >> 1;
    if (kWrite && kQuant) {
      // |x| as integers: NaN > infinity > finite, so one maximum finds both
      uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                            __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float amax = m > 0x7f80u ? __uint_as_float(0x7fc00000u)
                                     : fminf(fmaxf(__uint_as_float(m << 16), kAmaxLo), FLT_MAX);
      const float inv = __fdiv_rn(kE4m3Max, amax);
      if (h >= p.c.Hkv) continue;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint16_t code[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        code[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[i] << 16) * inv,
                                                       __uint_as_float(w[i] & 0xffff0000u) * inv),
                                           __NV_SATFINITE, __NV_E4M3);
      const uint2 out = make_uint2(code[0] | (static_cast<uint32_t>(code[1]) << 16),
                                   code[2] | (static_cast<uint32_t>(code[3]) << 16));
      uint8_t* dst = (r & 1) ? p.c.v : p.c.k;
      *reinterpret_cast<uint2*>(dst + p.c.pages.row(page, h, slot) + col) = out;
      if (col == 0) ((r & 1) ? p.c.vs : p.c.ks)[p.c.scales.row(page, h, slot)] = __fdiv_rn(amax, kE4m3Max);
    } else if (h < p.c.Hkv) {
      if (kWrite) {
        uint8_t* dst = (r & 1) ? p.c.v : p.c.k;
        *reinterpret_cast<uint4*>(dst + (p.c.pages.row(page, h, slot) + col) * 2) = x[u];
      } else {
        if (kQuant) {
          const uint32_t w[2] = {x[u].x, x[u].y};
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
            const __nv_bfloat162 y = __floats2bfloat162_rn(f.x * sc[u], f.y * sc[u]);
            out[i] = *reinterpret_cast<const uint32_t*>(&y);
          }
          // a place without a page reads as zero, whatever 0 * 0 above
          x[u] = make_uint4(out[0], out[1], out[2], out[3]);
        }
        uint8_t* dst = (r & 1) ? p.v : p.k;
        const long long at = (r & 1) ? t * p.v_row + h * p.v_head : t * p.k_row + h * p.k_head;
        *reinterpret_cast<uint4*>(dst + (at + col) * 2) = x[u];
      }
    }
  }
}

}  // namespace fa
