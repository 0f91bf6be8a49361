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
// rows that share its kv head, 2 * rows flops a byte (bf16): up to 16 rows far
// under what mma.sync delivers, so the kernel is laid out for bytes in flight
// and few instructions, not for the tensor pipe.  Both products are formed
// transposed, S^T = K Q^T and O^T = V^T P^T, so that the 16 of m16n8k16 is
// filled by keys and by columns of V and only the rows are padded, to 8.
// Quantised pages cost two conversions for four codes besides, each a quarter
// of a warp instruction's rate: they and the rows' exponentials bound the
// kernel from 16 rows on.
//
// Work: the keys that some row of a unit (sequence, 1 to 4 kv heads, block of
// rows) may see are cut into tiles of 32 to 128, about 32 KB.  The CTAs form
// groups of `lanes`, a lane for each unit of a sequence (or every lanes-th), so
// that a group reads the same tokens' heads at the same time: heads inside
// tokens are then whole DRAM rows, the 32-byte sectors of the scales are read
// from DRAM once, and blocks of rows share their keys in L2.  The tiles of all
// sequences form one list, and group c of G takes its c-th even share, whatever
// the lengths (beginning a unit counts as much as a tile: with tiles alone 64
// ragged sequences took 168 us against 141 us).  In each CTA one warp walks the
// share, looks pages up and keeps a ring of tiles loading (TMA boxes of 8 to 32
// tokens, each inside a page, over the unit's kv heads; scales by cp.async), on
// from one unit into the next; four warps compute, where the kv heads allow it
// each its own head or rows, so that they never meet; otherwise they share a
// tile's keys and join their states at a unit's end.  A unit that lies in one
// share is finished by its CTA; one that several share leaves a partial (m, l,
// accumulator) per CTA -- at most two per CTA, so the workspace does not grow
// with the batch -- for paged_combine_kernel (joining by the last warp to arrive
// instead, four rows at a time, was slower wherever many units are shared, the
// registers of both phases in one kernel: 128 ragged quantised sequences 111 us
// against 97 us, four tokens of 16 sequences 71 us against 49 us).  Where no
// unit can have more than a few tiles, none is shared: its group is the one its
// first tile falls to, and there is nothing to combine.
//
// Positions inside the kernel are padded: a page counts as page_size rounded up
// to 8 tokens, so that a box never spans two pages; the slots that do not exist
// are zero-filled by the TMA and masked.
//
// Measured (one call among others, 32 query heads on 8 kv heads, d = 128, of the
// copy rate of 6561 GB/s): one token over 8 x 32768 tokens, bf16, 168 us (97%); 64
// ragged sequences, bf16, 119 us (93%); 128 ragged sequences, e4m3, 64 query heads,
// 100 us (80%); four tokens each of 16 sequences, e4m3, 51 us (48%); 256 sequences, 16 heads,
// d = 64, window 255, 32 us (58%).
#pragma once

#include <type_traits>

#include "cache_sm100.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kPagedWarps = 4;      // that compute; one more loads
constexpr int kPagedThreads = 32 * (kPagedWarps + 1);
constexpr int kPagedMaxCtas = 444;  // three on each of 148 SMs
constexpr int kPagedCombineWarps = 8;
constexpr int kPagedWhole = 4;      // tiles: one CTA takes them in about the time of the second kernel

struct PagedParams {
  CacheParams c;
  const uint8_t* q;  // [B, H, Nq, D] bf16
  uint8_t* o;
  float* lse;
  Strides sq, so;
  int H, Nq, g;  // g = H / Hkv
  float scale_log2;
  int causal, window;
  int R, nblk;     // rows of a kv head (g * Nq), blocks they make
  int lanes;       // CTAs of a group: a divisor of a sequence's units
  int whole;       // no unit is shared
  int pad_page;    // page_size rounded up to a multiple of 8
  uint32_t pad_mul;  // pos / pad_page, as CacheParams::page_mul
  int pad_shift;
  int box_log;     // log2 of the tokens of a TMA box: 3 to 5
  int scale_rows;  // the scales of a unit's kv heads lie in line, aligned to their size
  int prow;        // rows of a partial: min(R, rows of a unit)
  float* part_o;   // [2 * G][kv heads of a unit][prow][D]
  float4* part_m;  // [2 * G][kv heads of a unit][prow]: m, l, unit of the accumulator
  int4* split;     // [CTAs]: the unit that starts in CTA c and goes on in its lane: b, unit, CTAs it spans (or 0)
};

// A unit has HG kv heads and up to 8 * NB * RG rows of each: a warp holds NB
// blocks of 8 rows of one head, and KW = 4 / (HG * RG) warps share each tile's
// keys.
template <int D, bool kQuant, int NB, int RG, int HG>
struct PagedCfg {
  static constexpr int kRows = 8 * NB * RG;
  static constexpr int KW = kPagedWarps / (HG * RG);
  static constexpr int kRowBytes = kQuant ? D : 2 * D;
  // keys: 32 KB of K and V, which two stages of three CTAs have room for; half of it where four warps share the keys
  // of a quantised tile (128 ragged sequences 109 us against 121 us: more, smaller steps of the ring)
  static constexpr int kTile = (kRowBytes == 256 || (kQuant && KW == 4 && D == 128) ? 64 : 128) / HG;
  static constexpr int kPart = kRowBytes == 256 ? 128 : kRowBytes;  // bytes of a row in a TMA box (its swizzle's width)
  static constexpr int kTileBytes = HG * kTile * kRowBytes;
  static constexpr int kScaleBytes = kQuant ? HG * kTile * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + (kQuant ? 1024 : 0);  // K, V, scales of K and of V
  static constexpr int kCtas = D == 128 && NB == 2 ? 2 : 3;  // of an SM
  static constexpr int kStages = (226 * 1024 / kCtas - 2048) / kStageBytes < 4 ? (226 * 1024 / kCtas - 2048) / kStageBytes : 4;
  static constexpr int kMergeStride = D + 4;  // floats; 2 * stride = 8 mod 32: a warp's stores meet every bank once
  static constexpr int kStatBytes = KW > 1 ? kPagedWarps * 8 * NB * 16 : 0;
  static constexpr int kSmemBytes = kStages * (kStageBytes + 16 + 48) + kStatBytes + 16 + 128;
  static_assert(kStages >= 2, "a tile loads while another is computed");
  static_assert(kTile >= 32, "a warp's lanes load the scales of 32 keys");
  static_assert(2 * kScaleBytes <= 1024, "both tiles' scales fit behind the values");
  static_assert(KW == 1 || (HG == 1 && kPagedWarps * 8 * kMergeStride * 4 <= kStageBytes),
                "the warps' accumulators are joined in a stage");
};

// N = 4, 8 or 16 bytes to shared memory, zeros when !on.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0) : "memory");
}
// The barrier counts an arrival once this thread's cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 y = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}
// c[16 x 8] += a[16 x 16] b[16 x 8]; a, b both f16 or both bf16.
template <bool kHalf>
__device__ __forceinline__ void mma16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t* b) {
  if (kHalf)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// The transpose of an 8 x 8 matrix of 16-bit values, a row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// mbar_wait() that first polls without a look at the clock and the limit (in
// global memory): most waits here are shorter than that.
__device__ __forceinline__ bool paged_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(a, parity)) return true;
  return mbar_wait(bar, parity, abort);
}
// What a state (m, l) counts for in one whose maximum is mt.  A state without a
// key has no weight; one of NaN alone (its maximum still -infinity) passes on.
__device__ __forceinline__ float paged_weight(float m, float l, float mt) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2_fast(m - mt);
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}
// The smaller magnitude of two f16 pairs, each half by itself.
__device__ __forceinline__ uint32_t min_abs_f16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("{\n .reg .b32 a;\n abs.f16x2 a, %1;\n min.f16x2 %0, a, %2;\n}" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
// Four e4m3 codes (the lowest first) as f16 numbers (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(x));
}
// Padded positions: pos + (pad_page - page_size) for every page before it.
__device__ __forceinline__ int paged_pad(const PagedParams& p, int pos) {
  return p.pad_page == p.c.page_size ? pos : pos + page_of(p.c, pos) * (p.pad_page - p.c.page_size);
}
// The padded positions [x, y) of a sequence of length L that some row may see;
// x is the beginning of a box.
__device__ __forceinline__ int2 paged_span(const PagedParams& p, int L) {
  if (L == 0) return make_int2(0, 0);
  const int first = p.window < 0 ? 0 : max(0, max(L - p.Nq, 0) - p.window);
  return make_int2(paged_pad(p, first) >> p.box_log << p.box_log, paged_pad(p, L - 1) + 1);
}
template <int kTile>
__device__ __forceinline__ int paged_tiles(const PagedParams& p, int L) {
  const int2 s = paged_span(p, L);
  return (s.y - s.x + kTile - 1) / kTile;
}

__device__ __forceinline__ int pad_page_of(const PagedParams& p, int padded) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(padded)) * p.pad_mul) >> (31 + p.pad_shift));
}
__device__ __forceinline__ int paged_slot(const PagedParams& p, int padded) {  // the token inside its page
  return padded - pad_page_of(p, padded) * p.pad_page;
}

// a / b for a >= 0, b > 0: in 32 bits where they do, a fraction of the 64-bit division's instructions.
__device__ __forceinline__ long long paged_div(long long a, long long b) {
  return (a | b) >> 32 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Adds what rounding to f16 took from products below 2^-14 of 16 keys.  In parts: a row's rests down to 2^-28 of its
// largest, scaled by a power of two that puts that one into [2^14, 2^15), then those that are left (those below 2^-111
// share the last part).  A function of its own, whose accumulators pass through memory: inside the loop it costs every
// path registers (128 ragged quantised sequences 106 us against 101 us).
template <int D, int NB>
struct PagedRests {
  float acc[NB][D / 16][4], p[NB][4];  // as in the kernel; the products
  uint32_t rows[4];  // this lane's D / 8 codes of keys 2 qd, + 1, + 8, + 9
};
template <int D, int NB>
__device__ __noinline__ void paged_add_rests(PagedRests<D, NB>& t, uint32_t at) {
  float r[NB][4];
  bool left = false;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = t.p[nb][e];
      r[nb][e] = fabsf(x) < 0x1p-14f ? x - __half2float(__float2half_rn(x)) : 0.f;
      left |= r[nb][e] != 0.f;
    }
  while (__any_sync(0xffffffffu, left)) {
    left = false;
    uint32_t pp[NB][2];
    float back[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float part[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t mx = max(__float_as_uint(r[nb][c]) & 0x7fffffffu, __float_as_uint(r[nb][2 + c]) & 0x7fffffffu);
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const uint32_t e = max(mx >> 23, 15u);
        const float up = __uint_as_float((268u - e) << 23);
        back[nb][c] = __uint_as_float((e - 14u) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float& x = r[nb][2 * h + c];
          const float y = x * up;
          const bool now = !(fabsf(y) < 0x1p-14f) || e == 15u;
          part[2 * h + c] = now ? y : 0.f;
          x = now ? 0.f : x;
          left |= x != 0.f;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) pp[nb][h] = transpose8x8(pack_f16(part[2 * h], part[2 * h + 1]));
    }
#pragma unroll
    for (int x = 0; x < D / 16; x += 2) {  // columns 2x, 2x + 1; 2x + 2, 2x + 3 of the lane's D / 8
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) w[y] = ld_shared_u32(t.rows[y] + at + 2 * x);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t sel = z ? 0x7362 : 0x5140;
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16(__byte_perm(w[0], w[1], sel), &a0, &a1);
        e4m3x4_to_f16(__byte_perm(w[2], w[3], sel), &a2, &a3);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float y[4] = {0.f, 0.f, 0.f, 0.f};
          mma16<true>(y, a0, a1, a2, a3, pp[nb]);
#pragma unroll
          for (int i = 0; i < 4; ++i) t.acc[nb][x + z][i] = fmaf(y[i], back[nb][i & 1], t.acc[nb][x + z][i]);
        }
      }
    }
  }
}

struct PagedDesc {  // a tile, as the loading warp describes it to the others
  int b, unit, key0, end;
  int flags, L;
  uint32_t boxes;         // those that are on a page
  int next_b, next_unit;  // of the tile after it
  int pad[3];
};
constexpr int kFlagUnitStart = 1, kFlagUnitEnd = 2, kFlagSegEnd = 4;

template <int D, bool kQuant, int NB, int RG, int HG>
__global__ void __launch_bounds__(kPagedThreads, PagedCfg<D, kQuant, NB, RG, HG>::kCtas)
    paged_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, kQuant, NB, RG, HG>;
  constexpr int KW = C::KW;                   // warps that share a tile's keys
  constexpr int DT = D / 16;                  // row tiles of O^T = V^T P^T
  constexpr int QS = D / 16;                  // k-steps of S^T = K Q^T
  constexpr int ST = C::kStages, RB = C::kRowBytes, PB = C::kPart, TK = C::kTile;
  // groups of 16 keys that a warp takes together: two, but where their registers spill (quantised, 16 rows a warp:
  // 115 us with two, 112 us with one, at 64 rows on 16384 tokens of 8 sequences)
  constexpr int KS = TK / KW >= 32 && !(kQuant && NB == 2) ? 2 : 1;
  constexpr int ES = kQuant ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* stat = reinterpret_cast<float4*>(smem + ST * C::kStageBytes);     // [warps][8 * NB rows]: m, l, unit
  PagedDesc* desc = reinterpret_cast<PagedDesc*>(smem + ST * C::kStageBytes + C::kStatBytes);  // [ST]
  uint64_t* full = reinterpret_cast<uint64_t*>(desc + ST);                  // [ST]
  uint64_t* empty = full + ST;                                              // [ST]
  uint64_t* joined = empty + ST;
  volatile int* abort = reinterpret_cast<int*>(joined + 1);
  long long* red = reinterpret_cast<long long*>(joined + 2);                // [16]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, B = p.c.B;
  const int group = cta / p.lanes, ulane = cta - group * p.lanes, groups = gridDim.x / p.lanes;
  const int U = p.c.Hkv / HG * p.nblk / p.lanes;  // units of a sequence in a lane: ulane + lanes * (0 .. U - 1)
  int stall = 0;
  if (warp == kPagedWarps) {  // what the loading warp needs from far away, while the share is found
    stall = *static_cast<volatile int*>(&g_debug_stall);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + i, kQuant ? 33 : 1);
      mbar_init(empty + i, kPagedWarps);
    }
    mbar_init(joined, kPagedWarps);
    *abort = 0;
    fence_mbar_init();
  }

  wait_for_predecessor();
  // nothing to join, until this CTA has come to its end: one that gives up leaves it at that
  if (tid == 0 && !p.whole) p.split[cta] = make_int4(0, 0, 0, 0);

  // ---- this group's share [s0, s1) of the list, in which a unit counts its tiles and c0
  auto tiles_of = [&](int b) { return b < B ? paged_tiles<TK>(p, cache_length(p.c, b)) : 0; };
  auto packed = [](int nt) { return (static_cast<long long>(nt) << 32) + (nt != 0); };  // tiles, sequences with keys
  const int per = (B + kPagedThreads - 1) / kPagedThreads;  // sequences of a thread: per * tid ...
  long long mine = 0, incl, sum = 0;
  for (int i = 0; i < per; ++i) mine += packed(tiles_of(per * tid + i));
  incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
#pragma unroll
  for (int w = 0; w < kPagedThreads / 32; ++w) {
    if (w < warp) before += red[w];
    sum += red[w];
  }
  const int c0 = p.whole || (sum >> 32) * U >= 2LL * groups ? 1 : 0;  // few tiles: one for each CTA
  auto cost = [&](long long x) { return ((x >> 32) + (x & 0xffffffffLL) * c0) * U; };
  const long long W = cost(sum);
  // groups with a share: c0 + 1 or more, so that each holds a tile
  const long long G = min(static_cast<long long>(groups), c0 ? W >> 1 : W);
  const long long s0 = group < G ? paged_div(group * W, G) : 0, s1 = group < G ? paged_div((group + 1) * W, G) : 0;

  // rows of sequences without keys
  for (int b = cta; b < B; b += gridDim.x) {
    if (tiles_of(b) != 0) continue;
    for (long long r = tid; r < static_cast<long long>(p.H) * p.Nq; r += kPagedThreads) {
      const int h = static_cast<int>(r / p.Nq), i = static_cast<int>(r % p.Nq);
      uint4* o = reinterpret_cast<uint4*>(p.o + 2 * p.so.row(b, h, i));
#pragma unroll
      for (int x = 0; x < D / 8; ++x) o[x] = make_uint4(0, 0, 0, 0);
      p.lse[static_cast<long long>(b) * p.H * p.Nq + r] = -INFINITY;
    }
  }
  if (group >= G) return;

  // ---- the front cursor: sequence, unit and tile of s0; the tiles up to s1
  int fb, fu, ft, cnt;
  long long last_end;  // where the unit that s1 lies in ends, on the list
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const long long at = e ? s1 : s0;
    if (e && tid == 0 && s1 == W) red[12] = (sum >> 32) * U, red[13] = W;
    if (at < cost(before) || at >= cost(before + mine)) continue;
    long long from = before;
    for (int b = per * tid;; ++b) {  // found before this thread's sequences end
      const int nt = tiles_of(b);
      if (at >= cost(from + packed(nt))) {
        from += packed(nt);
        continue;
      }
      const long long in = at - cost(from);
      int u = static_cast<int>(paged_div(in, nt + c0)), t = 0;
      const int off = static_cast<int>(in - static_cast<long long>(u) * (nt + c0));
      if (!p.whole)
        t = max(0, off - c0);
      else if (off != 0)
        ++u;  // the next unit; behind the last, the next sequence's first
      const long long done = (from >> 32) * U + static_cast<long long>(u) * nt + t;  // tiles before it
      while (u == U && b < B) {
        ++b;
        if (tiles_of(b) != 0) u = 0;
      }
      if (e) {
        red[12] = done;
        red[13] = at - off + nt + c0;
      } else {
        red[8] = b;
        red[9] = u;
        red[10] = t;
        red[11] = done;
      }
      break;
    }
  }
  __syncthreads();
  fb = static_cast<int>(red[8]);
  fu = static_cast<int>(red[9]);
  ft = static_cast<int>(red[10]);
  cnt = static_cast<int>(red[12] - red[11]);
  last_end = red[13];
  if (cnt == 0) return;  // p.whole: no unit starts in the share
  let_successor_begin();

  if (warp == kPagedWarps) {
    // ---- the loading warp
    if (stall) return;
    const int box = 1 << p.box_log;
    int fL = cache_length(p.c, fb), fLnext = fb + 1 < B ? cache_length(p.c, fb + 1) : 0;
    int2 span = paged_span(p, fL);
    int fnt = paged_tiles<TK>(p, fL);
    struct Tile {
      int b, u, key0, end, flags, L;
      int page, slot;  // of box `lane`
    };
    // the page table's entries for the sequence after this one on their way into L2
    auto prefetch = [&] {
      if (fLnext == 0 || lane >= TK >> p.box_log) return;
      const int2 s = paged_span(p, fLnext);
      const int pos = s.x + (lane << p.box_log);
      if (pos < s.y)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + (fb + 1) * p.c.table_stride + pad_page_of(p, pos)));
    };
    // the n-th tile; moves the cursor on
    auto fetch = [&](int n) {
      Tile t = {0, 0, 0, 0, 0, 0, -1, 0};
      if (n >= cnt) return t;
      t.b = fb;
      t.u = fu * p.lanes + ulane;
      t.L = fL;
      t.key0 = span.x + ft * TK;
      t.end = span.y;
      t.flags = (ft == 0 ? kFlagUnitStart : 0) | (ft == fnt - 1 ? kFlagUnitEnd | kFlagSegEnd : 0) |
                (n == cnt - 1 ? kFlagSegEnd : 0);
      const int pos = t.key0 + (lane << p.box_log);
      if (lane < TK >> p.box_log && pos < t.end) {
        const int i = pad_page_of(p, pos);
        t.slot = pos - i * p.pad_page;
        t.page = p.c.table[fb * p.c.table_stride + i];
      }
      if (++ft == fnt) {
        ft = 0;
        if (++fu == U) {
          fu = 0;
          if (n + 1 < cnt) {  // the next sequence with keys (there is one: tiles are left)
            do {
              ++fb;
              fL = fLnext;
              fLnext = fb + 1 < B ? cache_length(p.c, fb + 1) : 0;
              fnt = paged_tiles<TK>(p, fL);
            } while (fnt == 0 && fb < B - 1);
            span = paged_span(p, fL);
            prefetch();
          }
        }
      }
      return t;
    };
    prefetch();
    Tile cur = fetch(0);
    int st = 0, ph = 1;
    int n = 0;
    for (; n < cnt; ++n) {
      const Tile next = fetch(n + 1);
      if (!__all_sync(0xffffffffu, n < ST || paged_wait(empty + st, ph, abort))) break;
      const bool on = cur.page >= 0 && cur.page < p.c.num_pages;
      const uint32_t boxes = __ballot_sync(0xffffffffu, on);
      // boxes up to the end of the last group of 32 keys; those on no page are filled with zeros
      const int live = min(TK, (cur.end - cur.key0 + 31) & ~31) >> p.box_log;
      const int kh = (p.nblk == 1 ? cur.u : cur.u / p.nblk) * HG;
      uint8_t* dst = smem + st * C::kStageBytes;
      if (lane == 0) {
        int4* t = reinterpret_cast<int4*>(desc + st);
        t[0] = make_int4(cur.b, cur.u, cur.key0, cur.end);
        t[1] = make_int4(cur.flags, cur.L, static_cast<int>(boxes), next.b);
        t[2] = make_int4(next.u, 0, 0, 0);
        mbar_arrive_expect_tx(full + st, (live << p.box_log) * 2 * RB * HG);
      }
      const int page = on ? cur.page : p.c.num_pages;
      for (int i0 = 0; i0 < live; i0 += 4) {
        int pg[4], slot[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pg[i] = __shfl_sync(0xffffffffu, page, i0 + i);
          slot[i] = __shfl_sync(0xffffffffu, cur.slot, i0 + i);
        }
        if (lane != 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i0 + i >= live) break;
          uint8_t* to = dst + ((i0 + i) << p.box_log) * HG * PB;
#pragma unroll
          for (int h = 0; h < RB / PB; ++h) {
            tma_load_4d(&map_k, full + st, to + h * HG * TK * PB, h * PB / ES, slot[i], kh, pg[i]);
            tma_load_4d(&map_v, full + st, to + h * HG * TK * PB + C::kTileBytes, h * PB / ES, slot[i], kh, pg[i]);
          }
        }
      }
      if (kQuant) {
        const long long at = on ? p.c.scales.row(cur.page, kh, cur.slot) : -1;
        const uint32_t to = smem_u32(dst + 2 * C::kTileBytes);
        long long off[TK / 32];  // a head's entries, in groups of 32
        bool here[TK / 32];
#pragma unroll
        for (int i = 0; i < TK / 32; ++i) {
          const int src = (i * 32 + lane) >> p.box_log, in = lane & (box - 1);
          off[i] = __shfl_sync(0xffffffffu, at, src);
          const int slot = __shfl_sync(0xffffffffu, cur.slot, src) + in;
          here[i] = off[i] >= 0 && slot < p.c.page_size;
          off[i] += in * p.c.scales.n;
        }
        if (p.scale_rows) {  // [keys][heads]: the unit's heads in one copy
#pragma unroll
          for (int i = 0; i < TK / 32; ++i) {
            const uint32_t at = to + (i * 32 + lane) * HG * 4;
            const long long from = here[i] ? off[i] : 0;
            cp_async<HG * 4>(at, p.c.ks + from, here[i]);
            cp_async<HG * 4>(at + C::kScaleBytes, p.c.vs + from, here[i]);
          }
        } else {  // [heads][keys]
#pragma unroll
          for (int h = 0; h < HG; ++h)
#pragma unroll
            for (int i = 0; i < TK / 32; ++i) {
              const uint32_t at = to + (h * TK + i * 32 + lane) * 4;
              const long long from = here[i] ? off[i] + h * p.c.scales.h : 0;
              cp_async<4>(at, p.c.ks + from, here[i]);
              cp_async<4>(at + C::kScaleBytes, p.c.vs + from, here[i]);
            }
        }
        cp_async_arrive(full + st);
      }
      cur = next;
      if (++st == ST) st = 0, ph ^= 1;
    }
    if (kQuant) cp_async_wait_all();
    for (int i = max(0, n - ST); i < n; ++i)  // the copies under way end before the CTA does
      mbar_wait_drain(full + i % ST, (i / ST) & 1);
    return;
  }

  // ---- a computing warp's rows and its share of a tile's keys
  const int hg = warp / (RG * KW), rg = warp / KW % RG, kw = warp % KW, qd = lane & 3, rq = lane >> 2;
  uint32_t qb[NB][QS][2];  // Q^T: row rq of each block, the k index in the order of the K fragments
  float acc[NB][DT][4];    // O^T: columns dcol(x, 0), dcol(x, 1) of V for rows 2 qd, 2 qd + 1
  float mneg[NB][2], lim[NB][2], l[NB][2], rowf[NB][2], vref[NB][2], vinv[NB][2], vtop = 0.f;
  int rlo[NB][2], rhi[NB][2];  // padded positions that the thread's rows may see
  int free_lo = 0, free_hi = 0;  // those that every row of the unit may see
  bool settled = false;          // quantised: every row's accumulator has something large
  bool seg_starts_unit = false, fresh = true;  // fresh: the next tile begins a segment
  auto dcol = [&](int x, int e) { return kQuant ? rq * (D / 8) + 2 * x + e : 16 * x + 8 * e + rq; };
  // the queries of a unit, as they are in memory: words (8 s + qd, + 4) of a row, or its words 8 s + 2 qd, + 1 where
  // the K fragments are taken from 16 codes at a time
  auto load_q = [&](int b, int unit) {
    const int ku = p.nblk == 1 ? unit : unit / p.nblk, row0 = (unit - ku * p.nblk) * C::kRows + rg * 8 * NB;
    const int kh = ku * HG + hg;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = row0 + nb * 8 + rq;
      const int h = p.Nq == 1 ? r : r / p.Nq;
      const uint32_t* qr = reinterpret_cast<const uint32_t*>(p.q + 2 * (r < p.R ? p.sq.row(b, kh * p.g + h, r - h * p.Nq) : 0));
#pragma unroll
      for (int s = 0; s < QS; ++s) {
        uint2 v = make_uint2(0, 0);
        if (r < p.R)
          v = kQuant ? *reinterpret_cast<const uint2*>(qr + 8 * s + 2 * qd) : make_uint2(qr[8 * s + qd], qr[8 * s + 4 + qd]);
        qb[nb][s][0] = v.x;
        qb[nb][s][1] = v.y;
      }
    }
  };
  int jph = 0;
  auto join = [&] {  // the computing warps meet; false: given up
    __syncwarp();
    if (lane == 0) mbar_arrive(joined);
    const bool ok = paged_wait(joined, jph, abort);
    jph ^= 1;
    return __all_sync(0xffffffffu, ok) != 0;
  };
  int st = 0, ph = 0;
  auto release = [&] {  // this warp is done with the stage
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + st);
    if (++st == ST) st = 0, ph ^= 1;
  };
  // A stage holds [part of a row][box][head][token of the box][part bytes], the
  // 16-byte units swizzled by the TMA: unit ^ (token & 7) (parts of 128 bytes),
  // unit ^ (token / 2 & 3) (64).  Keys 16 i + (0 .. 15) are in one box or two.
  auto swz = [](int key) { return PB == 128 ? key & 7 : (key >> 1) & 3; };
  auto part = [](int i) { return i * 32 / PB * HG * TK * PB; };
  const int half = p.box_log == 3 ? HG * 8 * PB : 8 * PB;  // from key 16 i to 16 i + 8
  auto group_at = [&](int key) {  // key = 16 i, of this warp's head
    return (((key >> p.box_log) * HG + hg) << p.box_log) * PB + (key & ((1 << p.box_log) - 1)) * PB;
  };
  // a lane's row in a fragment of 16 keys x 32 bytes of K, of V (transposed)
  const uint32_t kat = (lane & 7) * PB + ((lane >> 3) & 1) * half + (((lane >> 4) ^ swz(lane & 7)) << 4);
  const uint32_t vat = (lane & 7) * PB + (lane >> 4) * half + ((((lane >> 3) & 1) ^ swz(lane & 7)) << 4);
  auto v_at = [&](int key, int byte) {  // of row key = 0 .. 15 of a group of V
    return byte / PB * HG * TK * PB + (key & 7) * PB + (key >> 3) * half + ((((byte % PB) >> 4) ^ swz(key)) << 4) + (byte & 15);
  };

  const int scl_step = p.scale_rows ? HG : 1, scl_at = p.scale_rows ? rq * HG + hg : hg * TK + rq;

  load_q(fb, fu * p.lanes + ulane);
  for (int n = 0; n < cnt; ++n) {
    if (!__all_sync(0xffffffffu, paged_wait(full + st, ph, abort))) return;
    const PagedDesc& t = desc[st];
    const int key0 = t.key0, flags = t.flags, left = t.end - t.key0;
    const uint32_t boxes = t.boxes, all_boxes = 0xffffffffu >> (32 - (TK >> p.box_log));
    if (fresh) {
      fresh = false;
      seg_starts_unit = flags & kFlagUnitStart;
      const int L = t.L, row0 = (p.nblk == 1 ? 0 : t.unit % p.nblk * C::kRows) + rg * 8 * NB;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float back = p.scale_log2;  // what a product of the scaled queries is multiplied by
        if (kQuant) {
          // bf16 queries as f16: scaled by a power of two that puts the row's
          // largest into [2^14, 2^15); exact down to 2^-31 of it
          uint32_t mx = 0;
#pragma unroll
          for (int s = 0; s < QS; ++s)
            mx = __vmaxu2(mx, __vmaxu2(qb[nb][s][0] & 0x7fff7fffu, qb[nb][s][1] & 0x7fff7fffu));
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const uint32_t e = min(max(mx >> 7, 27u), 254u);
          const float up = __uint_as_float((268u - e) << 23);
          back *= __uint_as_float((e - 14u) << 23);
#pragma unroll
          for (int s = 0; s < QS; ++s)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              qb[nb][s][y] = pack_f16(__uint_as_float(qb[nb][s][y] << 16) * up,
                                      __uint_as_float(qb[nb][s][y] & 0xffff0000u) * up);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mneg[nb][c] = 0.f;
          lim[nb][c] = -INFINITY;
          l[nb][c] = 0.f;
          vref[nb][c] = 0x1p-126f;
          vinv[nb][c] = 0.f;
          rowf[nb][c] = back;
          // neither zero nor infinite: times a masked key's -infinity, or times a score of zero, those make NaN.  (A factor
          // that underflows is that of scores of at most 2^-95 times the key's scale.)
          if (kQuant) rowf[nb][c] = fminf(fmaxf(__shfl_sync(0xffffffffu, back, (2 * qd + c) * 4), 0x1p-149f), FLT_MAX);
          const int r = row0 + nb * 8 + 2 * qd + c;
          const int i = p.Nq == 1 ? 0 : r % p.Nq, pos = L - p.Nq + i;
          rlo[nb][c] = 0;
          rhi[nb][c] = 0;  // padding rows see nothing
          if (r < p.R && pos >= 0) {
            rlo[nb][c] = p.window < 0 ? 0 : paged_pad(p, max(0, pos - p.window));
            rhi[nb][c] = paged_pad(p, (p.causal ? pos : (p.window < 0 ? L - 1 : min(L - 1, pos + p.window)))) + 1;
          }
        }
#pragma unroll
        for (int x = 0; x < DT; ++x) acc[nb][x][0] = acc[nb][x][1] = acc[nb][x][2] = acc[nb][x][3] = 0.f;
      }
      vtop = 0.f;
      settled = false;
      free_lo = p.window < 0 ? 0 : paged_pad(p, max(0, L - 1 - p.window));
      free_hi = 0;
      if (L >= p.Nq)
        free_hi = paged_pad(p, (p.causal ? L - p.Nq : (p.window < 0 ? L - 1 : min(L - 1, L - p.Nq + p.window)))) + 1;
    }

    const uint8_t* pV = smem + st * C::kStageBytes + C::kTileBytes;
    const uint32_t kaddr = smem_u32(smem + st * C::kStageBytes) + kat, vaddr = smem_u32(pV) + vat;
    const float* scl = reinterpret_cast<const float*>(pV + C::kTileBytes) + scl_at;  // K's, HG * TK further V's
    // the steps of a tile; kEdge: some row may not see some key of it
    auto steps = [&](auto edge_tile) {
      constexpr bool edge = decltype(edge_tile)::value;
#pragma unroll 1
      for (int s = 0; s < TK / KW / (16 * KS); ++s) {
        const int kb = (kw * (TK / KW / (16 * KS)) + s) * 16 * KS;
        if (edge && kb >= left) break;  // behind the end
        // ---- S^T of keys 16 k + rq (elements 0, 1) and 16 k + rq + 8 (2, 3), rows 2 qd and 2 qd + 1
        float sc[KS][NB][4];
        int at[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          at[k] = group_at(kb + 16 * k);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) sc[k][nb][0] = sc[k][nb][1] = sc[k][nb][2] = sc[k][nb][3] = 0.f;
          constexpr int NL = RB / 32;  // 32 bytes of 16 keys a load
          uint32_t a[NL][4];
#pragma unroll
          for (int i = 0; i < NL; ++i) ldmatrix_x4(a[i], (kaddr + at[k] + part(i)) ^ ((i << 5) & (PB - 1)));
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            if (kQuant) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(a[i][2 * y], &a0, &a2);
                e4m3x4_to_f16(a[i][2 * y + 1], &a1, &a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16<true>(sc[k][nb], a0, a1, a2, a3, qb[nb][(2 * i + y) % QS]);
              }
            } else {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16<false>(sc[k][nb], a[i][0], a[i][1], a[i][2], a[i][3], qb[nb][i % QS]);
            }
          }
        }
        float vs[KS][2];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float ks = kQuant ? scl[(kb + 16 * k + 8 * h) * scl_step] : 1.f;
            vs[k][h] = kQuant ? scl[HG * TK + (kb + 16 * k + 8 * h) * scl_step] : 1.f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (kQuant) sc[k][nb][2 * h + c] *= ks;
          }
        uint32_t allowed = 0xffffffffu;  // bit 4 (k NB + nb) + e
        if (edge) {
          allowed = 0;
          const int j0 = key0 + kb + rq;
          bool here[KS][2];  // key 16 k + 8 h + rq exists (8 keys in line are in one box)
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              here[k][h] = (boxes >> ((kb + 16 * k + 8 * h) >> p.box_log)) & 1;
              if (p.pad_page != p.c.page_size) here[k][h] &= paged_slot(p, j0 + 16 * k + 8 * h) < p.c.page_size;
            }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int lo = rlo[nb][c] - j0, hi = rhi[nb][c] - j0;
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (here[k][h] && 16 * k + 8 * h >= lo && 16 * k + 8 * h < hi)
                    allowed |= 1u << (4 * (k * NB + nb) + 2 * h + c);
                  else
                    sc[k][nb][2 * h + c] = -INFINITY;
            }
        }
        auto on = [&](int k, int nb, int e) { return !edge || ((allowed >> (4 * (k * NB + nb) + e)) & 1) != 0; };
        // ---- running maximum: moved only when it grows by more than 8 (weights
        // stay below 2^8).  Quantised: a key reaches the second product as f16(weight
        // * value scale / vref), and a row's accumulator counts in units of its vref,
        // a power of two 2^7 below (the power of two above) the largest value scale
        // so far: products stay below 2^15, and those of a key with that scale are
        // normal numbers of f16 down to weights of 2^-20.  Scales below vtop leave all
        // of a thread's rows as they are; a row that has seen scales of zero alone has
        // no vref yet (vinv = 0), and any other scale gives it one.
        float arg[KS][NB][4];  // exponents: score - maximum, or the score itself before a row's first key (lim = -infinity)
        bool grow = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int e = c; e < 4; e += 2) {
                arg[k][nb][e] = fmaf(sc[k][nb][e], rowf[nb][c], mneg[nb][c]);
                mx = fmaxf(mx, arg[k][nb][e]);
              }
            grow |= mx > lim[nb][c];
          }
        if (kQuant)
#pragma unroll
          for (int k = 0; k < KS; ++k) grow |= fmaxf(fabsf(vs[k][0]), fabsf(vs[k][1])) >= vtop;
        if (__any_sync(0xffffffffu, grow)) {
          vtop = INFINITY;
          settled = false;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = -INFINITY;
              uint32_t vb = 0;  // the largest scale, as bits of its magnitude
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  mx = fmaxf(mx, sc[k][nb][2 * h + c] * rowf[nb][c]);
                  if (kQuant && on(k, nb, 2 * h + c)) vb = max(vb, __float_as_uint(vs[k][h]) & 0x7fffffffu);
                }
#pragma unroll
              for (int o = 4; o <= 16; o <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (kQuant) vb = max(vb, __shfl_xor_sync(0xffffffffu, vb, o));
              }
              const float mo = lim[nb][c] == -INFINITY ? -INFINITY : -mneg[nb][c];
              const float mn = mx > mo + 8.f ? mx : mo;
              float f = mo == mn ? 1.f : exp2_fast(mo - mn);
              if (mn != -INFINITY) {
                mneg[nb][c] = -mn;
                lim[nb][c] = 8.f;
              }
              l[nb][c] *= f;
              if (kQuant) {
                if (vb != 0) {
                  const float vn = fmaxf(vref[nb][c], __uint_as_float(max(vb >> 23, 7u) - 6u << 23));
                  vinv[nb][c] = __uint_as_float((254u << 23) - __float_as_uint(vn));
                  f *= vref[nb][c] * vinv[nb][c];
                  vref[nb][c] = vn;
                }
                if (vinv[nb][c] > 0.f)
                  vtop = fminf(vtop, vref[nb][c] * 0x1p7f);
                else if (lim[nb][c] > 0.f)
                  vtop = 0x1p-149f;
              }
#pragma unroll
              for (int x = 0; x < DT; ++x) {
                acc[nb][x][c] *= f;
                acc[nb][x][2 + c] *= f;
              }
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = c; e < 4; e += 2) arg[k][nb][e] = fmaf(sc[k][nb][e], rowf[nb][c], mneg[nb][c]);
            }
        }
        // The weights are rounded to 16 bits for the second product: bf16 (half a
        // step is 2^-8 of a weight), or f16 of the product above, 2^-11 of it down to
        // 2^-14.  Products below that (`low`) may be all that counts, beside a key of
        // more weight whose value is zero: see behind the second product.
        uint32_t pb[KS][NB][2];
        bool low = false;
        uint32_t least = 0x7bff7bffu;  // f16 pairs; a step without masks looks at what was rounded (zeros count as low)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float w = exp2_fast(arg[k][nb][e]);
              l[nb][e & 1] += w;
              sc[k][nb][e] = w;
              if (kQuant) {
                sc[k][nb][e] = on(k, nb, e) ? w * (vs[k][e >> 1] * vinv[nb][e & 1]) : 0.f;
                if (edge) low |= fabsf(sc[k][nb][e]) < 0x1p-14f && sc[k][nb][e] != 0.f;
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = kQuant ? pack_f16(sc[k][nb][2 * h], sc[k][nb][2 * h + 1])
                                        : pack_bf16(sc[k][nb][2 * h], sc[k][nb][2 * h + 1]);
              if (kQuant && !edge) least = min_abs_f16x2(x, least);
              pb[k][nb][h] = transpose8x8(x);
            }
          }
        }
        if (kQuant && !edge) low = ((least - 0x04000400u) & 0x80008000u) != 0;
        // The slow form of columns dcol(x0 .. x0 + 3, .): products one by one in
        // fp32, weights of zero left out.  For an infinity or NaN among the values
        // of a tile that some rows see only in part (0 * infinity would reach rows
        // that may not see that key).
        auto one_by_one = [&](int k, int x0) {
#pragma unroll 1
          for (int y = 0; y < 16; ++y)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const int src = (y & 7) * 4 + qd;
              const float f0 = __shfl_sync(0xffffffffu, y < 8 ? sc[k][nb][0] : sc[k][nb][2], src);
              const float f1 = __shfl_sync(0xffffffffu, y < 8 ? sc[k][nb][1] : sc[k][nb][3], src);
#pragma unroll
              for (int x = x0; x < x0 + 4; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint8_t* from = pV + at[k] + v_at(y, dcol(x, e) * ES);
                  const float v = kQuant ? e4m3x2_to_float2(*from).x
                                         : __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(from)) << 16);
                  if (f0 != 0.f) acc[nb][x][2 * e] += f0 * v;
                  if (f1 != 0.f) acc[nb][x][2 * e + 1] += f1 * v;
                }
            }
        };
        // ---- O^T += V^T P^T
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if (kQuant) {
            uint32_t w[4][D / 32];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint8_t* v = pV + at[k] + v_at(2 * qd + (y & 1) + 8 * (y >> 1), rq * (D / 8));
              if (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(v);
                w[y][0] = x.x;
                w[y][1] = x.y;
                w[y][2 % (D / 32)] = x.z;
                w[y][3 % (D / 32)] = x.w;
              } else {
                const uint2 x = *reinterpret_cast<const uint2*>(v);
                w[y][0] = x.x;
                w[y][1] = x.y;
              }
            }
            uint32_t bad = 0;
            if (edge) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int z = 0; z < D / 32; ++z) bad |= (w[y][z] & 0x7f7f7f7fu) + 0x01010101u;
              bad &= 0x80808080u;  // a NaN's code
            }
            if (edge && __any_sync(0xffffffffu, bad)) {
#pragma unroll
              for (int x0 = 0; x0 < DT; x0 += 4) one_by_one(k, x0);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) sc[k][nb][0] = sc[k][nb][1] = sc[k][nb][2] = sc[k][nb][3] = 0.f;  // no rest
              continue;
            }
#pragma unroll
            for (int x = 0; x < DT; ++x) {  // columns 2x, 2x + 1 of the thread's D / 8
              const uint32_t sel = (x & 1) ? 0x7362 : 0x5140;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(w[0][x >> 1], w[1][x >> 1], sel), &a0, &a1);
              e4m3x4_to_f16(__byte_perm(w[2][x >> 1], w[3][x >> 1], sel), &a2, &a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16<true>(acc[nb][x], a0, a1, a2, a3, pb[k][nb]);
            }
          } else {
            const uint32_t from = vaddr + at[k];
#pragma unroll
            for (int x0 = 0; x0 < DT; x0 += 4) {
              uint32_t a[4][4];
#pragma unroll
              for (int x = 0; x < 4; ++x) ldmatrix_x4_trans(a[x], (from + part(x0 + x)) ^ (((x0 + x) << 5) & (PB - 1)));
              bool bad = false;
              if (edge) {  // value * 0 is a zero for finite values, NaN for others
                __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f), t = z;
#pragma unroll
                for (int x = 0; x < 16; ++x) t = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a[x >> 2][x & 3]), z, t);
                bad = (*reinterpret_cast<const uint32_t*>(&t) & 0x7fff7fffu) != 0;
              }
              if (edge && __any_sync(0xffffffffu, bad)) {
                one_by_one(k, x0);
                continue;
              }
#pragma unroll
              for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16<false>(acc[nb][x0 + x], a[x][0], a[x][1], a[x][2], a[x][3], pb[k][nb]);
            }
          }
        }
        // What rounding takes from low products is at most 2^-25 of each: it does not matter beside a row's accumulator that
        // has 2^10 in some column (2^15 keys: below 2^-11 of that).  Rows that have less get it added: 64 sequences of 8192
        // tokens, four rows a kv head, take 175 us however the scores are spread, 215 us where a tenth of the values are
        // zero and the scores' spread is 3, 405 us where it is 12.
        if constexpr (kQuant) {
          if (!settled && __any_sync(0xffffffffu, low)) {
            bool large = true;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float mx = rhi[nb][c] == 0 ? INFINITY : 0.f;  // rows that see nothing do not matter
#pragma unroll
                for (int x = 0; x < DT; ++x) mx = fmaxf(mx, fmaxf(fabsf(acc[nb][x][c]), fabsf(acc[nb][x][2 + c])));
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                large &= mx >= 0x1p10f;
              }
            settled = __all_sync(0xffffffffu, large);
          }
          if (!settled && __any_sync(0xffffffffu, low)) {
            PagedRests<D, NB> t;
#pragma unroll
            for (int y = 0; y < 4; ++y) t.rows[y] = smem_u32(pV + v_at(2 * qd + (y & 1) + 8 * (y >> 1), rq * (D / 8)));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int x = 0; x < DT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) t.acc[nb][x][e] = acc[nb][x][e];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              // (the scales are loaded again: kept in registers they cost four rows a head 2%; the smallest that a write
              // gives belongs to rows of zeros)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float v = __uint_as_float(ld_shared_u32(smem_u32(scl + HG * TK + (kb + 16 * k + 8 * (e >> 1)) * scl_step)));
                  t.p[nb][e] = fabsf(v) > kAmaxLo / kE4m3Max ? sc[k][nb][e] : 0.f;
                }
              paged_add_rests<D, NB>(t, at[k]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int x = 0; x < DT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nb][x][e] = t.acc[nb][x][e];
          }
        }
      }
    };
    if (key0 < free_lo || key0 + TK > free_hi || boxes != all_boxes || p.pad_page != p.c.page_size)
      steps(std::true_type{});
    else
      steps(std::false_type{});

    if (!(flags & kFlagSegEnd)) {
      release();
      continue;
    }
    // ---- the segment's end
    fresh = true;
    const int b = t.b, unit = t.unit;
    const int ku = p.nblk == 1 ? unit : unit / p.nblk, row0 = (unit - ku * p.nblk) * C::kRows, kh = ku * HG + hg;
    const bool whole = seg_starts_unit && (flags & kFlagUnitEnd);
    const int slot = 2 * cta + (seg_starts_unit ? 1 : 0);
    if (n + 1 < cnt) load_q(t.next_b, t.next_unit);  // the next unit's queries, on their way meanwhile
    if (n == cnt - 1 && tid == 0 && seg_starts_unit && !(flags & kFlagUnitEnd))  // the unit goes on in the next CTAs
      p.split[cta] = make_int4(b, unit, static_cast<int>(paged_div(last_end * G - 1, W)) - group + 1, 0);
    float m[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nb][c] = lim[nb][c] == -INFINITY ? -INFINITY : -mneg[nb][c];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], o);
      }
    if constexpr (KW == 1) {  // the warp's rows are its own
      release();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int rloc0 = (rg * NB + nb) * 8;
        if (row0 + rloc0 >= p.R) break;
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int rloc = rloc0 + 2 * qd + c;
            if (row0 + rloc >= p.R) continue;
            const long long pr = (static_cast<long long>(slot) * HG + hg) * p.prow + rloc;
            float* o = p.part_o + pr * D;
#pragma unroll
            for (int x = 0; x < DT; ++x)
              if (kQuant) {
                *reinterpret_cast<float2*>(o + dcol(x, 0)) = make_float2(acc[nb][x][c], acc[nb][x][2 + c]);
              } else {
                o[dcol(x, 0)] = acc[nb][x][c];
                o[dcol(x, 1)] = acc[nb][x][2 + c];
              }
            if (rq == 0) p.part_m[pr] = make_float4(m[nb][c], l[nb][c], vref[nb][c], 0.f);
          }
          continue;
        }
        float inv[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          inv[c] = l[nb][c] == 0.f ? 0.f : 1.f / l[nb][c];
          const int r = row0 + rloc0 + 2 * qd + c;
          if (r >= p.R) continue;
          const int hq = p.Nq == 1 ? r : r / p.Nq, h = kh * p.g + hq, i = r - hq * p.Nq;
          if (rq == 0)
            p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i] =
                l[nb][c] == 0.f ? -INFINITY : (m[nb][c] + log2f(l[nb][c])) * 0.69314718055994531f;
          if (kQuant) {  // D / 8 columns in line
            const float u = vref[nb][c];
            uint32_t w[DT];
#pragma unroll
            for (int x = 0; x < DT; ++x) w[x] = pack_bf16(acc[nb][x][c] * inv[c] * u, acc[nb][x][2 + c] * inv[c] * u);
            uint4* o = reinterpret_cast<uint4*>(p.o + 2 * (p.so.row(b, h, i) + rq * (D / 8)));
#pragma unroll
            for (int x = 0; x < DT; x += 4) o[x / 4] = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
          }
        }
        if (!kQuant) {  // 8 x 8 blocks of columns and rows, turned so that a lane has two columns of row rq
          const int r = row0 + rloc0 + rq;
          const int hq = p.Nq == 1 ? r : r / p.Nq, h = kh * p.g + hq, i = r - hq * p.Nq;
          uint32_t* o = reinterpret_cast<uint32_t*>(p.o + 2 * (r < p.R ? p.so.row(b, h, i) : 0)) + qd;
#pragma unroll
          for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = transpose8x8(pack_bf16(acc[nb][x][2 * e] * inv[0], acc[nb][x][2 * e + 1] * inv[1]));
              if (r < p.R) o[8 * x + 4 * e] = w;
            }
        }
      }
    } else {
      // the KW warps of a row group join their states in tile n's stage
      float* merge = reinterpret_cast<float*>(smem + st * C::kStageBytes);  // [warps][8 rows][kMergeStride]
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // tile n is read; the block before this one is joined, and so is the segment before: its readers of stat,
        // which no stage's barrier waits for, are behind it too
        if (!join()) return;
        float* mine = merge + (warp * 8 + 2 * qd) * C::kMergeStride;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (rq == 0) stat[(warp * NB + nb) * 8 + 2 * qd + c] = make_float4(m[nb][c], l[nb][c], vref[nb][c], 0.f);
          if (row0 + (rg * NB + nb) * 8 + 2 * qd + c >= p.R) continue;
#pragma unroll
          for (int x = 0; x < DT; ++x)
            if (kQuant) {
              *reinterpret_cast<float2*>(mine + c * C::kMergeStride + dcol(x, 0)) =
                  make_float2(acc[nb][x][c], acc[nb][x][2 + c]);
            } else {
              mine[c * C::kMergeStride + dcol(x, 0)] = acc[nb][x][c];
              mine[c * C::kMergeStride + dcol(x, 1)] = acc[nb][x][2 + c];
            }
        }
        if (!join()) return;
        constexpr int LPR = D / 4, RPP = 32 * kPagedWarps / LPR;  // threads of a row, rows of a pass
        const int col = tid % LPR * 4;
#pragma unroll
        for (int it = 0; it < RG * 8 / RPP; ++it) {
          const int rr = tid / LPR + it * RPP, g = rr >> 3, r8 = rr & 7;  // row r8 of group g
          const int rloc = (g * NB + nb) * 8 + r8, r = row0 + rloc;
          if (r >= p.R) continue;
          float mt = -INFINITY, vt = 0.f, lt = 0.f;
          float4 st[KW], a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            st[w] = stat[((g * KW + w) * NB + nb) * 8 + r8];
            mt = fmaxf(mt, st[w].x);
            vt = fmaxf(vt, st[w].z);
          }
          const float vti = __uint_as_float((254u << 23) - __float_as_uint(vt));
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            float f = paged_weight(st[w].x, st[w].y, mt);
            lt += f * st[w].y;
            if (kQuant) f *= st[w].z * vti;
            const float4 v = *reinterpret_cast<const float4*>(merge + ((g * KW + w) * 8 + r8) * C::kMergeStride + col);
            if (f != 0.f) {
              a.x += f * v.x;
              a.y += f * v.y;
              a.z += f * v.z;
              a.w += f * v.w;
            }
          }
          if (whole) {
            const int hq = p.Nq == 1 ? r : r / p.Nq, h = kh * p.g + hq, i = r - hq * p.Nq;
            const float inv = lt == 0.f ? 0.f : 1.f / lt, u = kQuant ? vt : 1.f;
            *reinterpret_cast<uint2*>(p.o + 2 * (p.so.row(b, h, i) + col)) =
                make_uint2(pack_bf16(a.x * inv * u, a.y * inv * u), pack_bf16(a.z * inv * u, a.w * inv * u));
            if (col == 0)
              p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i] =
                  lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.69314718055994531f;
          } else {
            const long long pr = static_cast<long long>(slot) * p.prow + rloc;
            *reinterpret_cast<float4*>(p.part_o + pr * D + col) = a;
            if (col == 0) p.part_m[pr] = make_float4(mt, lt, vt, 0.f);
          }
        }
      }
      fence_proxy_async_smem();  // the stage was written here; the TMA writes it next
      release();
    }
  }
}

// Joins the partials of the units that several CTAs share: block (c, y) the
// unit that starts in CTA c, 8 / CW rows of its heads.  Partial 0 is CTA c's
// second slot, the others are the lane's following CTAs' first.  CW warps take
// every CW-th partial of a row each: what bounds this is the latency of the
// loads, of which a warp has eight on their way.
template <int D, bool kQuant, int CW>
__global__ void __launch_bounds__(32 * kPagedCombineWarps)
    paged_combine_kernel(const PagedParams p, int rows_unit, int heads_unit) {
  constexpr int E = D / 32, kRows = kPagedCombineWarps / CW;
  __shared__ float4 stat[kRows][CW];
  __shared__ float part[CW > 1 ? kRows : 1][CW][D];
  wait_for_predecessor();
  const int4 s = p.split[blockIdx.x];
  const int parts = s.z;
  if (parts == 0) return;
  const int lane = threadIdx.x & 31, brow = threadIdx.x / (32 * CW), cw = (threadIdx.x >> 5) % CW;
  const int row = blockIdx.y * kRows + brow, hg = row / p.prow, rloc = row - hg * p.prow;
  const int ku = s.y / p.nblk, kh = ku * heads_unit + hg, r = (s.y - ku * p.nblk) * rows_unit + rloc;
  const bool on = hg < heads_unit && r < p.R;
  float m = -INFINITY, l = 0.f, u = 0x1p-126f, acc[E];  // u: the accumulators' unit, the largest so far
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (on) {
    const int mine = (parts - cw + CW - 1) / CW;  // partials cw, cw + CW, ...
    auto at = [&](int i) {
      i = cw + i * CW;
      return ((static_cast<long long>(2) * (blockIdx.x + i * p.lanes) + (i == 0 ? 1 : 0)) * heads_unit + hg) * p.prow + rloc;
    };
    constexpr int kAhead = 8;
    float v[kAhead][E];
    auto load = [&](int i, int cnt) {
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[y][e] = 0.f;
        if (y < cnt) {
          const float* src = p.part_o + at(i + y) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(src + e);
            v[y][e] = f.x;
            v[y][e + 1] = f.y;
          }
        }
      }
    };
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const int cnt = min(32, mine - i0);
      load(i0, cnt);  // on their way while the weights are formed
      float4 st = make_float4(-INFINITY, 0.f, 0x1p-126f, 0.f);
      if (lane < cnt) st = p.part_m[at(i0 + lane)];
      float mn = fmaxf(m, st.x), un = fmaxf(u, st.z);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        un = fmaxf(un, __shfl_xor_sync(0xffffffffu, un, o));
      }
      const float ui = __uint_as_float((254u << 23) - __float_as_uint(un));
      float old = paged_weight(m, l, mn), w = paged_weight(st.x, st.y, mn);
      float ls = w == 0.f ? 0.f : w * st.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      l = l * old + ls;
      old *= u * ui;
      w *= st.z * ui;
      m = mn;
      u = un;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= old;
      for (int i = 0; i < cnt; i += kAhead) {
        if (i != 0) load(i0 + i, cnt - i);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const float wi = __shfl_sync(0xffffffffu, w, (i + y) & 31);
          if (i + y < cnt && wi != 0.f)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += wi * v[y][e];
        }
      }
    }
    if (CW > 1) {
      if (lane == 0) stat[brow][cw] = make_float4(m, l, u, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) part[CW > 1 ? brow : 0][cw][lane * E + e] = acc[e];
    }
  }
  if (CW > 1) {
    __syncthreads();
    if (!on || cw != 0) return;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      m = fmaxf(m, stat[brow][w].x);
      u = fmaxf(u, stat[brow][w].z);
    }
    const float ui = __uint_as_float((254u << 23) - __float_as_uint(u));
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      const float4 st = stat[brow][w];
      float f = paged_weight(st.x, st.y, m);
      if (f == 0.f) continue;
      l += f * st.y;
      f *= st.z * ui;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * part[CW > 1 ? brow : 0][w][lane * E + e];
    }
  } else if (!on) {
    return;
  }
  const int h = kh * p.g + r / p.Nq, i = r % p.Nq;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (!kQuant) u = 1.f;
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + 2 * (p.so.row(s.x, h, i) + lane * E));
#pragma unroll
  for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16(acc[e] * inv * u, acc[e + 1] * inv * u);
  if (lane == 0)
    p.lse[(static_cast<long long>(s.x) * p.H + h) * p.Nq + i] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace fa
