// paged_sm100.cuh -- attention of each sequence's newest Nq tokens over the
// paged key/value cache (cache_sm100.cuh), forward only.
//
// Query row i of sequence b sits at position p = L_b - Nq + i; it sees the keys
// j < L_b that the causal / window predicate on (p, j) allows:
//   s_j = scale * q . k_j,  O = sum_j e^{s_j} v_j / sum_j e^{s_j},  LSE = ln sum_j e^{s_j}.
#pragma once

#include "cache_sm100.cuh"

namespace fa {

struct PagedParams {
  CacheParams c;
  const uint8_t* q;  // [B, H, Nq, D] bf16
  uint8_t* o;
  float* lse;
  Strides sq, so;
  int H, Nq, g;  // g = H / Hkv
  float scale_log2;
  int causal, window;
};

// One warp per query row, one key at a time, the online softmax in base 2.
template <int D, bool kQuant>
__global__ void __launch_bounds__(128) paged_row_kernel(const PagedParams p) {
  constexpr int E = D / 32;  // elements of a row that a lane holds
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.c.B) * p.H * p.Nq) return;
  const int i = static_cast<int>(row % p.Nq), h = static_cast<int>(row / p.Nq % p.H),
            b = static_cast<int>(row / p.Nq / p.H), kh = h / p.g;
  const int L = cache_length(p.c, b), pos = L - p.Nq + i;
  int lo = 0, hi = pos < 0 ? 0 : (p.causal ? pos + 1 : L);
  if (p.window >= 0) {
    lo = max(0, pos - p.window);
    hi = static_cast<int>(min(static_cast<long long>(hi), static_cast<long long>(pos) + p.window + 1));
  }
  float q[E], acc[E];
  const __nv_bfloat16* qr = reinterpret_cast<const __nv_bfloat16*>(p.q) + p.sq.row(b, h, i) + lane * E;
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    int slot;
    const int page = cache_page(p.c, b, j, &slot);
    if (page < 0) continue;
    const long long at = p.c.pages.row(page, kh, slot) + lane * E;
    float k[E], v[E];
    if (kQuant) {
      const long long sa = p.c.scales.row(page, kh, slot);
      const float ks = p.c.ks[sa], vs = p.c.vs[sa];
      for (int e = 0; e < E; e += 2) {
        const float2 a = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.c.k + at + e));
        const float2 c = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.c.v + at + e));
        k[e] = a.x * ks;
        k[e + 1] = a.y * ks;
        v[e] = c.x * vs;
        v[e + 1] = c.y * vs;
      }
    } else {
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.k)[at + e]);
        v[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.v)[at + e]);
      }
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * k[e];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - mu), w = exp2f(s - mu);
    m = mn;
    l = l * a + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * v[e];
  }
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + p.so.row(b, h, i) + lane * E;
  for (int e = 0; e < E; ++e) o[e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] / l);
  if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace fa
