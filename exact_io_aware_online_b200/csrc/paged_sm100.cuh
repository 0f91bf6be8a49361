// paged_sm100.cuh -- attention of each sequence's newest Nq tokens over the
// paged key/value cache (cache_sm100.cuh), forward only.
//
// Query row i of sequence b sits at position p = L_b - Nq + i; it sees the keys
// j < L_b that the causal / window predicate on (p, j) allows:
//   s_j = scale * q . k_j,  O = sum_j e^{s_j} v_j / sum_j e^{s_j},  LSE = ln sum_j e^{s_j},
// in one pass over the keys with a running maximum m, sum l and accumulator
// (base 2, rescaled only when the maximum grows by more than 2^8).
//
// What bounds it: every key and value crosses HBM once and meets the g * Nq
// rows that share its kv head, 2 * rows flops a byte (bf16): below 64 rows far
// under what mma.sync delivers, so the kernel is laid out for bytes in flight,
// not for the tensor pipe.  Rows are padded to 16 for m16n8k16 products.
//
// Work: the keys that some row of a unit (sequence, kv head, block of rows) may
// see are cut into tiles of 64.  All tiles of all units form one list, and CTA
// c of G takes its c-th even share, whatever the lengths: it walks its tiles
// through a cp.async ring that runs on from one unit into the next.  A unit
// that lies in one share is finished by its CTA; one that several share leaves
// a partial (m, l, accumulator) per CTA -- at most two per CTA, so the
// workspace does not grow with the batch -- for paged_combine_kernel.
#pragma once

#include "cache_sm100.cuh"

namespace fa {

constexpr int kPagedTile = 64;      // keys of a tile
constexpr int kPagedThreads = 128;  // 4 warps
constexpr int kPagedMaxCtas = 296;  // two on each of 148 SMs
constexpr int kPagedCombineRows = 8;
constexpr int kPagedRing = 8;       // descriptions of tiles: those staged, the one computed and the next one

struct PagedParams {
  CacheParams c;
  const uint8_t* q;  // [B, H, Nq, D] bf16
  uint8_t* o;
  float* lse;
  Strides sq, so;
  int H, Nq, g;  // g = H / Hkv
  float scale_log2;
  int causal, window;
  int R, nblk;     // rows of a kv head (g * Nq), blocks of 16 * RB rows they make
  int prow;        // rows of a partial: min(R, 16 * RB)
  float* part_o;   // [2 * G][prow][D]
  float4* part_m;  // [2 * G][prow]: m, l, sum of the weights as the second product saw them
  int4* split;     // [G]: the unit that starts in CTA c and goes on in later ones: b, unit, CTAs it spans (or 0)
};

template <int D, bool kQuant, int RB>
struct PagedCfg {
  static constexpr int kRowBytes = kQuant ? D : 2 * D;
  static constexpr int kTileBytes = kPagedTile * kRowBytes;
  static constexpr int kScaleBytes = kQuant ? kPagedTile * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kScaleBytes;
  // stages: as many as two CTAs of an SM have room for
  static constexpr int kStages = kStageBytes >= 32768 ? 3 : 5;
  static constexpr int kMerge = 4 * 16 * 8 * 16;  // 4 warps x 16 rows x 8 groups of 4 floats
  static constexpr int kOffsBytes = kPagedRing * kPagedTile * 8;
  static constexpr int kSmemBytes =
      kStages * kStageBytes + kMerge + 4 * 16 * 16 + (kQuant ? 2 : 1) * kOffsBytes + kPagedRing * 32;
  static_assert(kStages + 2 <= kPagedRing, "a tile's description outlives its copies");
};

__device__ __forceinline__ uint32_t paged_smem(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 4) bytes to shared memory, zeros when !on.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes as two bf16 numbers (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t x) {
  const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(x));
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// 16-byte unit `chunk` of key row `key` of a staged tile.  The exponent-or
// spreads both access patterns over all banks: keys (2m, 2m + 1) x 4 units (K)
// and keys (2q + const, q = 0..3) x 2 units (V).
template <int kRowBytes>
__device__ __forceinline__ uint32_t paged_at(int key, int chunk) {
  const int hi = (((key >> 2) ^ key) & 1) << 2;
  if (kRowBytes == 256) return key * 256 + ((chunk ^ (((key >> 1) & 1) | hi)) << 4);
  if (kRowBytes == 128) return key * 128 + ((chunk ^ ((((key >> 1) & 1) << 1) | hi)) << 4);
  return key * 64 + ((chunk ^ (((key >> 1) & 1) << 1)) << 4);
}

// First key that some row of a sequence of length L may see, and its tiles.
__device__ __forceinline__ int paged_first_key(const PagedParams& p, int L) {
  return p.window < 0 ? 0 : max(0, max(L - p.Nq, 0) - p.window);
}
__device__ __forceinline__ int paged_tiles(const PagedParams& p, int L) {
  return (L - paged_first_key(p, L) + kPagedTile - 1) / kPagedTile;
}

struct PagedDesc {  // a tile, as the front of the pipeline describes it to the rest
  int b, unit, key0, flags, L;
  uint32_t valid[2];  // keys that exist: in range and on a page
  int pad;
};
constexpr int kFlagUnitStart = 1, kFlagUnitEnd = 2, kFlagSegEnd = 4;

template <int D, bool kQuant, int RB>
__global__ void __launch_bounds__(kPagedThreads, 2) paged_kernel(const PagedParams p) {
  using C = PagedCfg<D, kQuant, RB>;
  constexpr int KW = 4 / RB;           // warps that share a row block's keys
  constexpr int NT = D / 8;            // output column tiles
  constexpr int QS = D / 16;           // k-steps of the score product
  constexpr int ST = C::kStages;
  constexpr int ES = kQuant ? 1 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* merge = reinterpret_cast<float4*>(smem + ST * C::kStageBytes);
  float4* stat = merge + 4 * 16 * 8;                                   // [4 warps][16 rows]: m, l, lb
  long long* offs = reinterpret_cast<long long*>(stat + 4 * 16);       // [ring][64] element offset of a row, -1: none
  long long* soffs = offs + kPagedRing * kPagedTile;                   // [ring][64] offset of its scale
  PagedDesc* desc = reinterpret_cast<PagedDesc*>(kQuant ? soffs + kPagedRing * kPagedTile : soffs);  // [ring]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, B = p.c.B;
  const long long U = static_cast<long long>(p.c.Hkv) * p.nblk;  // units of a sequence

  // ---- this CTA's share [t0, t1) of the tile list
  long long* red = reinterpret_cast<long long*>(merge);
  long long sum = 0;
  for (int b = tid; b < B; b += kPagedThreads) sum += paged_tiles(p, cache_length(p.c, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  const long long W = (red[0] + red[1] + red[2] + red[3]) * U;
  const long long G = min(static_cast<long long>(gridDim.x), W);  // CTAs with a share: at least one tile each
  const long long t0 = cta < G ? cta * W / G : 0, t1 = cta < G ? (cta + 1) * W / G : 0;
  const int cnt = static_cast<int>(t1 - t0);

  // rows of sequences without keys
  for (int b = cta; b < B; b += gridDim.x) {
    if (paged_tiles(p, cache_length(p.c, b)) != 0) continue;
    for (long long r = tid; r < static_cast<long long>(p.H) * p.Nq; r += kPagedThreads) {
      const int h = static_cast<int>(r / p.Nq), i = static_cast<int>(r % p.Nq);
      uint4* o = reinterpret_cast<uint4*>(p.o + 2 * p.so.row(b, h, i));
#pragma unroll
      for (int x = 0; x < D / 8; ++x) o[x] = make_uint4(0, 0, 0, 0);
      p.lse[static_cast<long long>(b) * p.H * p.Nq + r] = -INFINITY;
    }
  }
  if (cnt == 0) {
    if (tid == 0) p.split[cta] = make_int4(0, 0, 0, 0);
    return;
  }

  // ---- the front cursor: sequence, unit and tile of t0
  int fb = 0, fu = 0, ft = 0, fL, fnt, fLnext;
  {
    long long base = 0;
    for (int at = 0;; at += kPagedThreads) {
      const int b = at + tid;
      const long long mine = b < B ? paged_tiles(p, cache_length(p.c, b)) * U : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) red[warp] = incl;
      __syncthreads();
      long long before = base;
      for (int w = 0; w < warp; ++w) before += red[w];
      const long long lo = before + incl - mine, hi = before + incl;
      if (lo <= t0 && t0 < hi) {
        red[4] = b;
        red[5] = t0 - lo;
      }
      base += red[0] + red[1] + red[2] + red[3];
      if (t0 < base) break;  // found (uniform)
    }
    __syncthreads();
    fb = static_cast<int>(red[4]);
    const long long off = red[5];
    __syncthreads();
    fL = cache_length(p.c, fb);
    fnt = paged_tiles(p, fL);
    fu = static_cast<int>(off / fnt);
    ft = static_cast<int>(off % fnt);
    fLnext = fb + 1 < B ? cache_length(p.c, fb + 1) : 0;
  }
  // what fetch() leaves for store()
  int n_page = -1, n_slot = 0, n_b = 0, n_u = 0, n_key0 = 0, n_flags = 0, n_L = 0;
  const int frow = tid & (kPagedTile - 1);

  // fetch(n): loads the page of this thread's row of tile n and advances the cursor
  auto fetch = [&](int n) {
    if (n >= cnt) return;
    n_b = fb;
    n_u = fu;
    n_L = fL;
    n_key0 = paged_first_key(p, fL) + ft * kPagedTile;
    n_flags = (ft == 0 ? kFlagUnitStart : 0) | (ft == fnt - 1 ? kFlagUnitEnd | kFlagSegEnd : 0) |
              (n == cnt - 1 ? kFlagSegEnd : 0);
    const int pos = n_key0 + frow;
    n_page = -1;
    if (pos < fL) {
      const int i = pos / p.c.page_size;
      n_slot = pos - i * p.c.page_size;
      n_page = p.c.table[fb * p.c.table_stride + i];
    }
    if (++ft == fnt) {
      ft = 0;
      if (++fu == static_cast<int>(U)) {
        fu = 0;
        if (n + 1 < cnt) {  // the next sequence with keys (there is one: tiles are left)
          do {
            ++fb;
            fL = fLnext;
            fLnext = fb + 1 < B ? cache_length(p.c, fb + 1) : 0;
            fnt = paged_tiles(p, fL);
          } while (fnt == 0 && fb < B - 1);
        }
      }
    }
  };
  // store(n): the row's offsets and the tile's description, for issue() and compute()
  auto store = [&](int n) {
    if (n >= cnt) return;
    const bool on = n_page >= 0 && n_page < p.c.num_pages;
    const int kh = n_u / p.nblk;
    if (tid < kPagedTile) {
      offs[(n % kPagedRing) * kPagedTile + frow] = on ? p.c.pages.row(n_page, kh, n_slot) : -1;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      PagedDesc& t = desc[n % kPagedRing];
      if (lane == 0) t.valid[warp] = m;
      if (tid == 0) {
        t.b = n_b;
        t.unit = n_u;
        t.key0 = n_key0;
        t.flags = n_flags;
        t.L = n_L;
      }
    } else if (kQuant) {
      soffs[(n % kPagedRing) * kPagedTile + frow] = on ? p.c.scales.row(n_page, kh, n_slot) : -1;
    }
  };
  const uint32_t smem0 = paged_smem(smem);
  // issue(n): the copies of tile n into its stage (always one group, empty past the end)
  auto issue = [&](int n) {
    if (n < cnt) {
      constexpr int CPR = C::kRowBytes / 16, RPI = kPagedThreads / CPR;  // units of a row, rows of a pass
      const uint32_t dst = smem0 + (n % ST) * C::kStageBytes;
      const int chunk = tid % CPR;
#pragma unroll
      for (int i = 0; i < kPagedTile / RPI; ++i) {
        const int row = tid / CPR + i * RPI;
        const long long off = offs[(n % kPagedRing) * kPagedTile + row];
        const bool on = off >= 0;
        const long long at = (on ? off * ES : 0) + chunk * 16;
        const uint32_t to = dst + paged_at<C::kRowBytes>(row, chunk);
        cp_async16(to, p.c.k + at, on);
        cp_async16(to + C::kTileBytes, p.c.v + at, on);
      }
      if (kQuant) {
        const long long off = soffs[(n % kPagedRing) * kPagedTile + frow];
        const float* src = (tid < kPagedTile ? p.c.ks : p.c.vs) + (off >= 0 ? off : 0);
        cp_async4(dst + 2 * C::kTileBytes + tid * 4, src, off >= 0);
      }
    }
    cp_async_commit();
  };

  // ---- a warp's rows and its share of a tile's keys
  const int rb = warp / KW, kw = warp % KW, qd = lane & 3, rq = lane >> 2;
  uint32_t qa[QS][4];
  float acc[NT][4];
  float m[2], l[2], lb[2];
  int rlo[2], rhi[2];          // keys that the thread's two rows may see
  int free_lo = 0, free_hi = 0;  // keys that every row of the unit may see
  bool seg_starts_unit = false;
  int seg_first = 0;
  bool fresh = true;  // the next tile begins a segment

  for (int n = 0; n < ST; ++n) {
    fetch(n);
    store(n);
  }
  fetch(ST);
  __syncthreads();
  for (int n = 0; n < ST - 1; ++n) issue(n);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int n = 0; n < cnt; ++n) {
    cp_async_wait<ST - 2>();
    store(n + ST);
    __syncthreads();  // tile n has landed; everyone is done with tile n - 1
    issue(n + ST - 1);
    fetch(n + ST + 1);

    const PagedDesc& t = desc[n % kPagedRing];
    const int b = t.b, unit = t.unit, key0 = t.key0, flags = t.flags;
    const int kh = unit / p.nblk, row0 = (unit % p.nblk) * 16 * RB;
    if (fresh) {
      fresh = false;
      seg_starts_unit = flags & kFlagUnitStart;
      seg_first = n;
      const int L = t.L;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[x] = -INFINITY;
        l[x] = lb[x] = 0.f;
        const int r = row0 + rb * 16 + rq + 8 * x;
        const int h = r / p.Nq, i = r - h * p.Nq, pos = L - p.Nq + i;
        const bool on = r < p.R;
        rlo[x] = 0;
        rhi[x] = 0x7fffffff;  // padding rows: never stored
        if (on) {
          rlo[x] = p.window < 0 ? 0 : max(0, pos - p.window);
          rhi[x] = pos < 0 ? 0 : (p.causal ? pos + 1 : (p.window < 0 ? L : min(L, pos + p.window + 1)));
        }
        const uint8_t* qr = p.q + 2 * (on ? p.sq.row(b, kh * p.g + h, i) : 0);
        // the k index of the score product is permuted so that a key's row is
        // read in 16-byte units; the queries take the same order
        constexpr int W2 = kQuant ? 8 : 4;  // words of q that belong to one 16-byte unit of k
#pragma unroll
        for (int i2 = 0; i2 < D / (8 * W2); ++i2) {
          uint32_t w[W2];
#pragma unroll
          for (int y = 0; y < W2; y += 4) {
            const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(qr + (qd + 4 * i2) * W2 * 4 + y * 4))
                               : make_uint4(0, 0, 0, 0);
            w[y] = v.x;
            w[y + 1] = v.y;
            w[y + 2] = v.z;
            w[y + 3] = v.w;
          }
#pragma unroll
          for (int y = 0; y < W2 / 2; ++y) {
            qa[i2 * (W2 / 2) + y][x] = w[2 * y];
            qa[i2 * (W2 / 2) + y][2 + x] = w[2 * y + 1];
          }
        }
      }
#pragma unroll
      for (int x = 0; x < NT; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
      free_lo = p.window < 0 ? 0 : max(0, L - 1 - p.window);
      free_hi = L < p.Nq ? 0 : (p.causal ? L - p.Nq + 1 : (p.window < 0 ? L : min(L, L - p.Nq + p.window + 1)));
    }

    const uint32_t sK = smem0 + (n % ST) * C::kStageBytes, sV = sK + C::kTileBytes;
    const float* scl = reinterpret_cast<const float*>(smem + (n % ST) * C::kStageBytes + 2 * C::kTileBytes);
    const bool edge = key0 < free_lo || key0 + kPagedTile > free_hi || (t.valid[0] & t.valid[1]) != 0xffffffffu;
#pragma unroll 1
    for (int s = 0; s < RB; ++s) {
      const int kb = (kw * RB + s) * 16;
      // ---- scores of 16 keys
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const int key = kb + nt * 8 + rq;
        if (kQuant) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const uint4 w = lds128(sK + paged_at<C::kRowBytes>(key, qd + 4 * i));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_bf16(sc[nt], qa[i * 4 + x], e4m3x2_to_bf16x2(ww[x]), e4m3x2_to_bf16x2(ww[x] >> 16));
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 w = lds128(sK + paged_at<C::kRowBytes>(key, qd + 4 * i));
            mma_bf16(sc[nt], qa[2 * i], w.x, w.y);
            mma_bf16(sc[nt], qa[2 * i + 1], w.z, w.w);
          }
        }
      }
      float2 vs[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float2 f = make_float2(p.scale_log2, p.scale_log2);
        if (kQuant) {
          const float2 ks = *reinterpret_cast<const float2*>(scl + kb + nt * 8 + 2 * qd);
          vs[nt] = *reinterpret_cast<const float2*>(scl + kPagedTile + kb + nt * 8 + 2 * qd);
          f.x *= ks.x;
          f.y *= ks.y;
        }
        sc[nt][0] *= f.x;
        sc[nt][1] *= f.y;
        sc[nt][2] *= f.x;
        sc[nt][3] *= f.y;
      }
      uint32_t allowed = 0xff;  // bit nt * 4 + e
      if (edge) {
        allowed = 0;
        const uint32_t vm = t.valid[kb >> 5] >> (kb & 31);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = nt * 8 + 2 * qd + (e & 1), j = key0 + kb + k;
            if (((vm >> k) & 1) && j >= rlo[e >> 1] && j < rhi[e >> 1])
              allowed |= 1u << (nt * 4 + e);
            else
              sc[nt][e] = -INFINITY;
          }
      }
      // ---- running maximum: moved only when it grows by more than 8 (weights stay below 2^8)
      float mx[2] = {fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])),
                     fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]))};
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
          const float mn = mx[x] > m[x] + 8.f ? mx[x] : m[x];
          f[x] = m[x] == mn ? 1.f : exp2_fast(m[x] - mn);
          m[x] = mn;
          l[x] *= f[x];
          lb[x] *= f[x];
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          acc[x][0] *= f[0];
          acc[x][1] *= f[0];
          acc[x][2] *= f[1];
          acc[x][3] *= f[1];
        }
      }
      const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = exp2_fast(sc[nt][e] - mu[e >> 1]);
          l[e >> 1] += w[e];
          if (kQuant) w[e] = edge && !((allowed >> (nt * 4 + e)) & 1) ? 0.f : w[e] * ((e & 1) ? vs[nt].y : vs[nt].x);
        }
        // the weights are rounded to bf16 for the second product (half a step,
        // 2^-8 of a weight); unquantised rows are normalised by the sum of the
        // rounded weights, so that O stays a mean of value rows
        pa[nt * 2] = pack_bf16(w[0], w[1]);
        pa[nt * 2 + 1] = pack_bf16(w[2], w[3]);
        if (!kQuant)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            lb[x] += __uint_as_float(pa[nt * 2 + x] << 16) + __uint_as_float(pa[nt * 2 + x] & 0xffff0000u);
      }
      // ---- O += P V: output column x + NT * rq of thread column pair is tile x, so that a
      // thread reads D / 8 consecutive values of each of its four keys
      const int vk[4] = {kb + 2 * qd, kb + 2 * qd + 1, kb + 2 * qd + 8, kb + 2 * qd + 9};
      uint32_t bad = 0;
      if (kQuant) {
        uint32_t w[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (D == 128) {
            const uint4 v = lds128(sV + paged_at<C::kRowBytes>(vk[k], rq));
            w[k][0] = v.x;
            w[k][1] = v.y;
            w[k][2 % (D / 32)] = v.z;
            w[k][3 % (D / 32)] = v.w;
          } else {
            const uint2 v = lds64(sV + paged_at<C::kRowBytes>(vk[k], rq >> 1) + (rq & 1) * 8);
            w[k][0] = v.x;
            w[k][1] = v.y;
          }
        }
        uint32_t vb[2][NT];
#pragma unroll
        for (int x = 0; x < NT / 2; ++x) {  // codes 2x, 2x + 1 of the thread's columns
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t z = __byte_perm(w[2 * y][x >> 1], w[2 * y + 1][x >> 1], (x & 1) ? 0x7362 : 0x5140);
            vb[y][2 * x] = e4m3x2_to_bf16x2(z);
            vb[y][2 * x + 1] = e4m3x2_to_bf16x2(z >> 16);
          }
        }
        if (edge)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              bad |= ((vb[y][x] & 0x7f80u) == 0x7f80u) | ((vb[y][x] & 0x7f800000u) == 0x7f800000u);
        if (!edge || !__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int x = 0; x < NT; ++x) mma_bf16(acc[x], pa, vb[0][x], vb[1][x]);
          continue;
        }
      } else {
        uint32_t w[4][D / 16];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int y = 0; y < D / 64; ++y) {
            const uint4 v = lds128(sV + paged_at<C::kRowBytes>(vk[k], rq * (D / 64) + y));
            w[k][4 * y] = v.x;
            w[k][4 * y + 1] = v.y;
            w[k][4 * y + 2] = v.z;
            w[k][4 * y + 3] = v.w;
          }
        if (edge)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
              bad |= ((w[k][y] & 0x7f80u) == 0x7f80u) | ((w[k][y] & 0x7f800000u) == 0x7f800000u);
        if (!edge || !__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            const uint32_t sel = (x & 1) ? 0x7632 : 0x5410;
            mma_bf16(acc[x], pa, __byte_perm(w[0][x >> 1], w[1][x >> 1], sel),
                     __byte_perm(w[2][x >> 1], w[3][x >> 1], sel));
          }
          continue;
        }
      }
      // An infinity or NaN among the values of a tile that some rows see only in
      // part: 0 * infinity would reach rows that may not see that key, so the
      // products are formed one by one and weights of zero are left out.
#pragma unroll 1
      for (int k = 0; k < 16; ++k) {
        const int src = (lane & ~3) | ((k & 7) >> 1);
        const uint32_t w0 = __shfl_sync(0xffffffffu, k < 8 ? pa[0] : pa[2], src);
        const uint32_t w1 = __shfl_sync(0xffffffffu, k < 8 ? pa[1] : pa[3], src);
        const float f0 = __uint_as_float((k & 1) ? w0 & 0xffff0000u : w0 << 16);
        const float f1 = __uint_as_float((k & 1) ? w1 & 0xffff0000u : w1 << 16);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = (2 * qd + e) * NT + x;
            const uint32_t at = sV + paged_at<C::kRowBytes>(kb + k, col * ES / 16) + (col * ES) % 16;
            float v;
            if (kQuant) {
              uint32_t z;
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z) : "r"(at));
              v = e4m3x2_to_float2(static_cast<uint16_t>(z)).x;
            } else {
              uint32_t z;
              asm volatile("ld.shared.u16 %0, [%1];" : "=r"(z) : "r"(at));
              v = __uint_as_float(z << 16);
            }
            if (f0 != 0.f) acc[x][e] += f0 * v;
            if (f1 != 0.f) acc[x][2 + e] += f1 * v;
          }
      }
    }

    if (!(flags & kFlagSegEnd)) continue;
    // ---- the segment's end: the KW warps of a row block join their states
    fresh = true;
    const bool whole = seg_starts_unit && (flags & kFlagUnitEnd);
    const int slot = 2 * cta + (seg_starts_unit ? 1 : 0);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], o);
        lb[x] += __shfl_xor_sync(0xffffffffu, lb[x], o);
      }
      if (qd == 0) stat[warp * 16 + rq + 8 * x] = make_float4(m[x], l[x], kQuant ? l[x] : lb[x], 0.f);
    }
    float out[RB][NT];  // thread: row tid / 8 (+ 16 per item), columns NT * (tid % 8) + 0..NT-1
    const int orow = tid >> 3, ogrp = tid & 7;
    float fw[RB][KW], mt[RB], lt[RB], lbt[RB];
#pragma unroll
    for (int ps = 0; ps < NT / 4; ++ps) {
      if (ps) __syncthreads();
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          merge[(warp * 16 + rq + 8 * x) * 8 + ((2 * qd + e) ^ ((rq >> 1) & 3))] =
              make_float4(acc[4 * ps][2 * x + e], acc[4 * ps + 1][2 * x + e], acc[4 * ps + 2][2 * x + e],
                          acc[4 * ps + 3][2 * x + e]);
      __syncthreads();
#pragma unroll
      for (int it = 0; it < RB; ++it) {
        const int w0 = it * KW;
        if (ps == 0) {
          mt[it] = -INFINITY;
#pragma unroll
          for (int w = 0; w < KW; ++w) mt[it] = fmaxf(mt[it], stat[(w0 + w) * 16 + orow].x);
          lt[it] = lbt[it] = 0.f;
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const float4 s4 = stat[(w0 + w) * 16 + orow];
            fw[it][w] = s4.x == -INFINITY ? (s4.y == 0.f ? 0.f : 1.f) : exp2_fast(s4.x - mt[it]);
            lt[it] += fw[it][w] * s4.y;
            lbt[it] += fw[it][w] * s4.z;
          }
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const float4 v = merge[((w0 + w) * 16 + orow) * 8 + (ogrp ^ ((orow >> 1) & 3))];
          const float f = fw[it][w];
          if (f != 0.f) {
            a.x += f * v.x;
            a.y += f * v.y;
            a.z += f * v.z;
            a.w += f * v.w;
          }
        }
        out[it][4 * ps] = a.x;
        out[it][4 * ps + 1] = a.y;
        out[it][4 * ps + 2] = a.z;
        out[it][4 * ps + 3] = a.w;
      }
    }
#pragma unroll
    for (int it = 0; it < RB; ++it) {
      const int rloc = it * 16 + orow, r = row0 + rloc;
      if (r >= p.R) continue;
      if (whole) {
        const int h = kh * p.g + r / p.Nq, i = r % p.Nq;
        const float inv = lt[it] == 0.f ? 0.f : 1.f / lbt[it];
        uint4* o = reinterpret_cast<uint4*>(p.o + 2 * (p.so.row(b, h, i) + ogrp * NT));
#pragma unroll
        for (int x = 0; x < NT; x += 8)
          o[x / 8] = make_uint4(pack_bf16(out[it][x] * inv, out[it][x + 1] * inv),
                                pack_bf16(out[it][x + 2] * inv, out[it][x + 3] * inv),
                                pack_bf16(out[it][x + 4] * inv, out[it][x + 5] * inv),
                                pack_bf16(out[it][x + 6] * inv, out[it][x + 7] * inv));
        if (ogrp == 0)
          p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i] =
              lt[it] == 0.f ? -INFINITY : (mt[it] + log2f(lt[it])) * 0.69314718055994531f;
      } else {
        const long long pr = static_cast<long long>(slot) * p.prow + rloc;
        float4* o = reinterpret_cast<float4*>(p.part_o + pr * D + ogrp * NT);
#pragma unroll
        for (int x = 0; x < NT; x += 4)
          o[x / 4] = make_float4(out[it][x], out[it][x + 1], out[it][x + 2], out[it][x + 3]);
        if (ogrp == 0) p.part_m[pr] = make_float4(mt[it], lt[it], lbt[it], 0.f);
      }
    }
    if (n == cnt - 1 && tid == 0) {
      int4 s = make_int4(0, 0, 0, 0);
      if (seg_starts_unit && !(flags & kFlagUnitEnd)) {  // goes on in the next CTAs
        const long long end = t1 - (n - seg_first + 1) + paged_tiles(p, t.L);  // one past the unit's last tile
        s = make_int4(b, unit, static_cast<int>((end * G - 1) / W) - cta + 1, 0);
      }
      p.split[cta] = s;
    }
    __syncthreads();  // merge and stat are free again
  }
  cp_async_wait<0>();
}

// Joins the partials of the units that several CTAs share: block (c, y) the
// unit that starts in CTA c, 8 rows of it, a warp each.  Partial 0 is CTA c's
// second slot, the others are the following CTAs' first.
template <int D>
__global__ void __launch_bounds__(32 * kPagedCombineRows) paged_combine_kernel(const PagedParams p, int rows_unit) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 s = p.split[blockIdx.x];
  const int parts = s.z;
  if (parts == 0) return;
  const int lane = threadIdx.x & 31;
  const int rloc = blockIdx.y * kPagedCombineRows + (threadIdx.x >> 5);
  const int kh = s.y / p.nblk, r = (s.y % p.nblk) * rows_unit + rloc;
  if (rloc >= rows_unit || r >= p.R) return;
  auto at = [&](int i) {
    return (static_cast<long long>(2) * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.prow + rloc;
  };
  float m = -INFINITY, l = 0.f, lb = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float4 st = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (i0 + lane < parts) st = p.part_m[at(i0 + lane)];
    float mn = fmaxf(m, st.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    const float old = m == -INFINITY ? 0.f : exp2_fast(m - mn);
    const float w = st.x == -INFINITY ? (st.y == 0.f ? 0.f : 1.f) : exp2_fast(st.x - mn);
    m = mn;
    l *= old;
    lb *= old;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    float ls = w == 0.f ? 0.f : w * st.y, lbs = w == 0.f ? 0.f : w * st.z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ls += __shfl_xor_sync(0xffffffffu, ls, o);
      lbs += __shfl_xor_sync(0xffffffffu, lbs, o);
    }
    l += ls;
    lb += lbs;
    const int cnt = min(32, parts - i0);
#pragma unroll 8
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.part_o + at(i0 + i) * D + lane * E;
      float v[E];
      if (E == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[0] = f.x;
        v[1] = f.y;
        v[2 % E] = f.z;
        v[3 % E] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[0] = f.x;
        v[1] = f.y;
      }
      if (wi != 0.f)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wi * v[e];
    }
  }
  const int h = kh * p.g + r / p.Nq, i = r % p.Nq;
  const float inv = l == 0.f ? 0.f : 1.f / lb;
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + 2 * (p.so.row(s.x, h, i) + lane * E));
#pragma unroll
  for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0)
    p.lse[(static_cast<long long>(s.x) * p.H + h) * p.Nq + i] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace fa
