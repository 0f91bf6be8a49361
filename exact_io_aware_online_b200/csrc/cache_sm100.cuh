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

// Every kernel here is launched to begin while the one before it ends, and
// waits for that one's results (and for its reads of what is written) with this.
// Loads behind it are plain ones: the read-only path (ld.global.nc) wants memory
// that nobody writes from this kernel's first block on, and the kernel before,
// which may still run then, writes tokens, pages and queries.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may begin (and wait) once every block has said this.
__device__ __forceinline__ void let_successor_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- moving tokens
struct MoveParams {
  CacheParams c;
  uint8_t* k;  // dense tokens [T, Hkv, D] bf16: read by the write kernel, written by the read kernel
  uint8_t* v;
  long long k_row, k_head, v_row, v_head;  // elements
  const int* cu;                           // [B + 1] offsets of the sequences' rows
  int T;
  uint32_t row_mul;  // row / (2 * Hkv), as CacheParams::page_mul
  int row_shift;
};

// The number of sequences b with cu[b + 1] <= t: the one that t belongs to, if
// to any.  A search by the whole warp, 32 offsets a step (two dependent loads
// for up to 1024 sequences).
__device__ __forceinline__ int first_sequence(const int* cu, int B, int t, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;
    const unsigned m = __ballot_sync(0xffffffffu, i < hi && cu[i + 1] <= t);
    lo += __popc(m) * step;
    hi = min(hi, lo + step);
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && cu[lo + lane + 1] <= t));
}

// Rows of the dense side in the order token, K then V, head.  Four lanes hold a
// row (D / 4 values each, 8 at a time, interleaved, so that 4 lanes' loads and
// stores fill sectors) and a warp 8 * kMoveUnroll rows, which may belong to
// several tokens.  Few lanes a row keep what a row costs once -- the join of
// the maximum, two divisions, addresses -- small beside its bytes (sixteen lanes
// a row: writing 131072 quantised tokens 199 us against 127 us then); a write loads
// its rows before it looks up where they go.  Bound by HBM from a few thousand
// tokens on, by the launch and four dependent loads below.  Measured, of the
// copy rate of 6561 GB/s: that write 129 us (96%), reading a ragged quantised batch back
// 118 us (96%), 256 short bf16 sequences at d = 64 53 us (93%), one token each of 64
// sequences 2.8 us (11 us a call with the host's side).
constexpr int kMoveWarps = 4;
constexpr int kMoveUnroll = 2;
constexpr int kMoveRows = 8 * kMoveUnroll;  // of a warp

template <int D, bool kQuant, bool kWrite>
__global__ void __launch_bounds__(32 * kMoveWarps) cache_move_kernel(const MoveParams p) {
  constexpr int N = D / 32;  // groups of 8 values that a lane holds of a row
  const int lane = threadIdx.x & 31, q = lane & 3;
  const uint32_t rows = 2u * p.c.Hkv * p.T;
  const uint32_t first = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * kMoveRows;
  if (first >= rows) return;
  auto token_of = [&](uint32_t row) {
    return static_cast<int>((static_cast<unsigned long long>(row) * p.row_mul) >> (31 + p.row_shift));
  };

  uint4 x[kMoveUnroll][N];
  int token[kMoveUnroll], head[kMoveUnroll];
  bool isv[kMoveUnroll], on[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const uint32_t row = first + 8 * u + (lane >> 2);
    on[u] = row < rows;
    token[u] = token_of(on[u] ? row : first);
    const int h = static_cast<int>((on[u] ? row : first) - 2u * p.c.Hkv * token[u]);
    isv[u] = h >= p.c.Hkv;
    head[u] = isv[u] ? h - p.c.Hkv : h;
  }
  auto dense = [&](int u) {
    return (isv[u] ? p.v + 2 * (token[u] * p.v_row + head[u] * p.v_head) : p.k + 2 * (token[u] * p.k_row + head[u] * p.k_head)) +
           q * 16;
  };
  wait_for_predecessor();
  if (kWrite) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const uint8_t* src = dense(u);
#pragma unroll
      for (int i = 0; i < N; ++i) x[u][i] = *reinterpret_cast<const uint4*>(src + i * 64);
    }
  }

  let_successor_begin();
  // ---- where the rows live: the sequence of the warp's first token, from which each lane goes on to its own
  const int t0 = token_of(first);
  const int b0 = first_sequence(p.cu, p.c.B, t0, lane);
  int page[kMoveUnroll], slot[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    int b = b0;
    while (b < p.c.B && p.cu[b + 1] <= token[u]) ++b;
    on[u] = on[u] && b < p.c.B && p.cu[b] <= token[u];
    page[u] = -1;
    slot[u] = 0;
    if (on[u]) {
      const int pos = cache_length(p.c, b) - (p.cu[b + 1] - token[u]);
      if (pos >= 0) page[u] = cache_page(p.c, b, pos, &slot[u]);
    }
    if (kWrite) on[u] = on[u] && page[u] >= 0;
  }

  float sc[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    sc[u] = 0.f;
    if (!kWrite) {
      const bool there = on[u] && page[u] >= 0;  // a place without a page reads as zero
      const uint8_t* src = there ? (isv[u] ? p.c.v : p.c.k) + p.c.pages.row(page[u], head[u], slot[u]) * (kQuant ? 1 : 2) : p.c.k;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[u][i] = make_uint4(0, 0, 0, 0);
        if (there && kQuant) {
          const uint2 w = *reinterpret_cast<const uint2*>(src + q * 8 + i * 32);
          x[u][i].x = w.x;
          x[u][i].y = w.y;
        } else if (there) {
          x[u][i] = *reinterpret_cast<const uint4*>(src + q * 16 + i * 64);
        }
      }
      if (kQuant && there) sc[u] = (isv[u] ? p.c.vs : p.c.ks)[p.c.scales.row(page[u], head[u], slot[u])];
    }
  }
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    if (kWrite && kQuant) {
      // |x| as integers: NaN > infinity > finite, so one maximum finds both
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[u][i].x & 0x7fff7fffu, x[u][i].y & 0x7fff7fffu),
                                 __vmaxu2(x[u][i].z & 0x7fff7fffu, x[u][i].w & 0x7fff7fffu)));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      if (!on[u]) continue;
      const float amax = m > 0x7f80u ? __uint_as_float(0x7fc00000u)
                                     : fminf(fmaxf(__uint_as_float(m << 16), kAmaxLo), FLT_MAX);
      const float inv = __fdiv_rn(kE4m3Max, amax);
      uint8_t* dst = (isv[u] ? p.c.v : p.c.k) + p.c.pages.row(page[u], head[u], slot[u]) + q * 8;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
        uint16_t code[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          code[y] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[y] << 16) * inv,
                                                         __uint_as_float(w[y] & 0xffff0000u) * inv),
                                             __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(dst + i * 32) = make_uint2(code[0] | (static_cast<uint32_t>(code[1]) << 16),
                                                             code[2] | (static_cast<uint32_t>(code[3]) << 16));
      }
      if (q == 0) (isv[u] ? p.c.vs : p.c.ks)[p.c.scales.row(page[u], head[u], slot[u])] = __fdiv_rn(amax, kE4m3Max);
    } else if (on[u]) {
      uint8_t* dst = kWrite ? (isv[u] ? p.c.v : p.c.k) + 2 * p.c.pages.row(page[u], head[u], slot[u]) + q * 16 : dense(u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (kQuant) {
          const uint32_t w[2] = {x[u][i].x, x[u][i].y};
          uint32_t out[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[y >> 1] >> (16 * (y & 1))));
            const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * sc[u], f.y * sc[u]);
            out[y] = *reinterpret_cast<const uint32_t*>(&v);
          }
          x[u][i] = make_uint4(out[0], out[1], out[2], out[3]);
        }
        *reinterpret_cast<uint4*>(dst + i * 64) = x[u][i];
      }
    }
  }
}

}  // namespace fa
