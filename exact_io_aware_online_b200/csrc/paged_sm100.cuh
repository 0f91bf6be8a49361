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
// under what mma.sync delivers, so the kernel is laid out for bytes in flight
// and few instructions, not for the tensor pipe.  Both products are formed
// transposed, S^T = K Q^T and O^T = V^T P^T, so that the 16 of m16n8k16 is
// filled by keys and by columns of V and only the rows are padded, to 8.
//
// Work: the keys that some row of a unit (sequence, kv head, block of rows) may
// see are cut into tiles of 64 or 128.  The CTAs form groups of `lanes`, a lane
// for each unit of a sequence (or every lanes-th), so that a group reads the
// same tokens' heads at the same time: heads inside tokens are then whole DRAM
// rows, the 32-byte sectors of the scales are read from DRAM once, and blocks
// of rows share their keys in L2.  The tiles of all sequences form one list, and
// group c of G takes its c-th even share, whatever the lengths (beginning a
// unit counts as much as a tile): each CTA walks its tiles through a cp.async
// ring that runs on from one unit into the next.  A unit that lies in one share
// is finished by its CTA; one that several share leaves a partial (m, l,
// accumulator) per CTA -- at most two per CTA, so the workspace does not grow
// with the batch -- for paged_combine_kernel.
#pragma once

#include <type_traits>

#include "cache_sm100.cuh"

namespace fa {

constexpr int kPagedThreads = 128;  // 4 warps
constexpr int kPagedMaxCtas = 444;  // three on each of 148 SMs
constexpr int kPagedCombineRows = 8;
constexpr int kPagedRing = 8;       // descriptions of tiles: those staged, the one computed and the next one
constexpr int kPagedOffs = 4;       // tiles' row offsets, from store() to issue()

struct PagedParams {
  CacheParams c;
  const uint8_t* q;  // [B, H, Nq, D] bf16
  uint8_t* o;
  float* lse;
  Strides sq, so;
  int H, Nq, g;  // g = H / Hkv
  float scale_log2;
  int causal, window;
  int R, nblk;     // rows of a kv head (g * Nq), units they make
  int lanes;       // CTAs of a group: a divisor of Hkv * nblk
  int prow;        // rows of a partial: min(R, rows of a unit)
  float* part_o;   // [2 * G][prow][D]
  float4* part_m;  // [2 * G][prow]: m, l, unit of the accumulator
  int4* split;     // [CTAs]: the unit that starts in CTA c and goes on in its lane: b, unit, CTAs it spans (or 0)
};

// A warp holds NB blocks of 8 rows; RG groups of warps hold different rows, the
// 4 / RG warps of a group share each tile's keys.
template <int D, bool kQuant, int NB, int RG>
struct PagedCfg {
  static constexpr int kRows = 8 * NB * RG;  // rows of a unit
  static constexpr int kRowBytes = kQuant ? D : 2 * D;
  static constexpr int kTile = kRowBytes == 256 ? 64 : 128;  // keys
  static constexpr int kTileBytes = kTile * kRowBytes;
  static constexpr int kScaleBytes = kQuant ? kTile * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kScaleBytes;
  static constexpr int kCtas = kStageBytes >= 32768 || (D == 128 && NB == 2) ? 2 : 3;  // of an SM
  static constexpr int kStages = 3;
  static constexpr int kMergeStride = D + 4;  // floats; 2 * stride = 8 mod 32: a warp's stores meet every bank once
  static constexpr int kStatBytes = 4 * 8 * NB * 16;
  static constexpr int kOffsBytes = kPagedOffs * kTile * 8;
  static constexpr int kSmemBytes = kStages * kStageBytes + kStatBytes + (kQuant ? 2 : 1) * kOffsBytes + kPagedRing * 48;
  static_assert(kStages + 2 <= kPagedRing && kStages <= kPagedOffs, "a tile's description outlives its copies");
  static_assert(4 * 8 * kMergeStride * 4 <= kStageBytes, "the warps' accumulators are joined in a stage");
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
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Four e4m3 codes (the lowest first) as f16 numbers (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(x));
}
// Byte of the 16-byte unit `chunk` of key row `key` in a staged tile.  K: eight
// lanes read keys (2m, 2m + 1) x 4 consecutive units.  V: bf16, eight keys x
// one unit (ldmatrix); e4m3, keys (0, 2, 4, 6) + const x units (2c, 2c + 1).
// The exclusive-or puts each such set into different banks (but for V rows of
// 64 bytes, which are read in pairs).
template <int kRowBytes>
__device__ __forceinline__ uint32_t k_at(int key, int chunk) {
  return key * kRowBytes + (kRowBytes == 64 ? chunk << 4 : (chunk ^ ((key & 1) << 2)) << 4);
}
template <int kRowBytes, bool kQuant>
__device__ __forceinline__ uint32_t v_at(int key, int chunk) {
  const int x = !kQuant ? key & 7 : kRowBytes == 128 ? key & 6 : key & 2;
  return key * kRowBytes + ((chunk ^ x) << 4);
}

// First key that some row of a sequence of length L may see, and its tiles.
__device__ __forceinline__ int paged_first_key(const PagedParams& p, int L) {
  return p.window < 0 ? 0 : max(0, max(L - p.Nq, 0) - p.window);
}
template <int kTile>
__device__ __forceinline__ int paged_tiles(const PagedParams& p, int L) {
  return (L - paged_first_key(p, L) + kTile - 1) / kTile;
}

struct PagedDesc {  // a tile, as the front of the pipeline describes it to the rest
  int b, unit, key0, flags, L;
  uint32_t valid[4];  // keys that exist: in range and on a page
  int pad[3];
};
constexpr int kFlagUnitStart = 1, kFlagUnitEnd = 2, kFlagSegEnd = 4;

template <int D, bool kQuant, int NB, int RG>
__global__ void __launch_bounds__(kPagedThreads, PagedCfg<D, kQuant, NB, RG>::kCtas)
    paged_kernel(const PagedParams p) {
  using C = PagedCfg<D, kQuant, NB, RG>;
  constexpr int KW = 4 / RG;                  // warps that share a tile's keys
  constexpr int DT = D / 16;                  // row tiles of O^T = V^T P^T
  constexpr int QS = D / 16;                  // k-steps of S^T = K Q^T
  constexpr int ST = C::kStages, RB = C::kRowBytes, TK = C::kTile;
  constexpr int KS = TK / KW >= 32 ? 2 : 1;   // groups of 16 keys that a warp takes together
  constexpr int ES = kQuant ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* stat = reinterpret_cast<float4*>(smem + ST * C::kStageBytes);  // [4 warps][8 * NB rows]: m, l, unit
  long long* offs = reinterpret_cast<long long*>(stat + 4 * 8 * NB);     // [kPagedOffs][TK] byte offset of a row, -1: none
  long long* soffs = offs + kPagedOffs * TK;                         // [kPagedOffs][TK] element offset of its scale
  PagedDesc* desc = reinterpret_cast<PagedDesc*>(kQuant ? soffs + kPagedOffs * TK : soffs);  // [ring]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, B = p.c.B;
  const int group = cta / p.lanes, ulane = cta - group * p.lanes, groups = gridDim.x / p.lanes;
  const int U = p.c.Hkv * p.nblk / p.lanes;  // units of a sequence in a lane: ulane + lanes * (0 .. U - 1)

  // ---- this group's share [s0, s1) of the list, in which a unit counts its tiles and c0
  long long* red = reinterpret_cast<long long*>(smem);
  auto tiles_of = [&](int b) { return b < B ? paged_tiles<TK>(p, cache_length(p.c, b)) : 0; };
  auto packed = [](int nt) { return (static_cast<long long>(nt) << 32) + (nt != 0); };  // tiles, sequences with keys
  long long sum = 0;
  for (int b = tid; b < B; b += kPagedThreads) sum += packed(tiles_of(b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = red[0] + red[1] + red[2] + red[3];
  const int c0 = (sum >> 32) * U >= 2LL * groups ? 1 : 0;  // few tiles: one for each CTA
  auto cost = [&](long long x) { return ((x >> 32) + (x & 0xffffffffLL) * c0) * U; };
  const long long W = cost(sum);
  // groups with a share: c0 + 1 or more, so that each holds a tile
  const long long G = min(static_cast<long long>(groups), W / (c0 + 1));
  const long long s0 = group < G ? group * W / G : 0, s1 = group < G ? (group + 1) * W / G : 0;

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
  if (group >= G) {
    if (tid == 0) p.split[cta] = make_int4(0, 0, 0, 0);
    return;
  }

  // ---- the front cursor: sequence, unit and tile of s0; the tiles up to s1
  int fb, fu, ft, fL, fnt, fLnext, cnt;
  long long last_end;  // where the unit that s1 lies in ends
  {
    long long base = 0;
    __syncthreads();
    if (tid == 0) red[8] = (sum >> 32) * U, red[9] = W;  // s1 at the very end
    for (int at = 0;; at += kPagedThreads) {
      const int b = at + tid, nt = tiles_of(b);
      long long incl = packed(nt);
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
      const long long first = before + incl - packed(nt), lo = cost(first), hi = cost(before + incl);
      if (nt != 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const long long at_s = e ? s1 : s0;
          if (lo > at_s || at_s >= hi) continue;
          const int u = static_cast<int>((at_s - lo) / (nt + c0)), off = static_cast<int>((at_s - lo) % (nt + c0));
          const int t = max(0, off - c0);
          const long long done = (first >> 32) * U + static_cast<long long>(u) * nt + t;  // tiles before it
          if (e) {
            red[8] = done;
            red[9] = at_s - off + nt + c0;
          } else {
            red[4] = b;
            red[5] = u;
            red[6] = t;
            red[7] = done;
          }
        }
      }
      base += red[0] + red[1] + red[2] + red[3];
      if (s1 < cost(base) || at + kPagedThreads >= B) break;  // found (uniform)
    }
    __syncthreads();
    fb = static_cast<int>(red[4]);
    fu = static_cast<int>(red[5]);
    ft = static_cast<int>(red[6]);
    cnt = static_cast<int>(red[8] - red[7]);
    last_end = red[9];
    __syncthreads();
    fL = cache_length(p.c, fb);
    fnt = paged_tiles<TK>(p, fL);
    fLnext = fb + 1 < B ? cache_length(p.c, fb + 1) : 0;
  }
  const int frow = tid & (TK - 1);
  struct Tile {  // a tile as fetch() leaves it for store(): this thread's row
    int page, slot, b, u, key0, flags, L;
  };

  // fetch(n): loads the page of this thread's row of tile n and advances the cursor
  auto fetch = [&](int n) {
    Tile t = {-1, 0, 0, 0, 0, 0, 0};
    if (n >= cnt) return t;
    t.b = fb;
    t.u = fu * p.lanes + ulane;
    t.L = fL;
    t.key0 = paged_first_key(p, fL) + ft * TK;
    t.flags = (ft == 0 ? kFlagUnitStart : 0) | (ft == fnt - 1 ? kFlagUnitEnd | kFlagSegEnd : 0) |
              (n == cnt - 1 ? kFlagSegEnd : 0);
    const int pos = t.key0 + frow;
    if (tid < TK && pos < fL) {
      const int i = page_of(p.c, pos);
      t.slot = pos - i * p.c.page_size;
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
        }
      }
    }
    return t;
  };
  // store(n): the row's offsets and the tile's description, for issue() and compute()
  auto store = [&](int n, const Tile& f) {
    if (n >= cnt) return;
    const bool on = f.page >= 0 && f.page < p.c.num_pages;
    const int kh = p.nblk == 1 ? f.u : f.u / p.nblk;
    if (tid < TK) {
      offs[(n % kPagedOffs) * TK + tid] = on ? p.c.pages.row(f.page, kh, f.slot) * ES : -1;
      if (kQuant) soffs[(n % kPagedOffs) * TK + tid] = on ? p.c.scales.row(f.page, kh, f.slot) : -1;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      PagedDesc& t = desc[n % kPagedRing];
      if (lane == 0) t.valid[warp] = m;
      if (tid == 0) {
        t.b = f.b;
        t.unit = f.u;
        t.key0 = f.key0;
        t.flags = f.flags;
        t.L = f.L;
      }
    }
  };
  const uint32_t smem0 = paged_smem(smem);
  // issue(n): the copies of tile n into its stage (always one group, empty past the end)
  constexpr int CPR = RB / 16, RPI = kPagedThreads / CPR;  // 16-byte units of a row, rows of a pass
  const int chunk = tid % CPR, crow = tid / CPR;
  auto issue = [&](int n) {
    if (n < cnt) {
      const uint32_t dst = smem0 + (n % ST) * C::kStageBytes;
      const long long* src = offs + (n % kPagedOffs) * TK + crow;
#pragma unroll
      for (int i = 0; i < TK / RPI; ++i) {
        const int row = crow + i * RPI;
        const long long off = src[i * RPI];
        const bool on = off >= 0;
        const long long at = (on ? off : 0) + chunk * 16;
        cp_async16(dst + k_at<RB>(row, chunk), p.c.k + at, on);
        cp_async16(dst + C::kTileBytes + v_at<RB, kQuant>(row, chunk), p.c.v + at, on);
      }
      if (kQuant) {
        const long long off = soffs[(n % kPagedOffs) * TK + tid], at = off >= 0 ? off : 0;
        cp_async4(dst + 2 * C::kTileBytes + tid * 4, p.c.ks + at, off >= 0);
        cp_async4(dst + 2 * C::kTileBytes + (TK + tid) * 4, p.c.vs + at, off >= 0);
      }
    }
    cp_async_commit();
  };

  // ---- a warp's rows and its share of a tile's keys
  const int rg = warp / KW, kw = warp % KW, qd = lane & 3, rq = lane >> 2;
  uint32_t qb[NB][QS][2];  // Q^T: row rq of each block, the k index in the order in which a key's 16-byte units come
  float acc[NB][DT][4];    // O^T: columns dcol(x, 0), dcol(x, 1) of V for rows 2 qd, 2 qd + 1
  float m[NB][2], l[NB][2], rowf[NB][2], vref[NB][2], vinv[NB][2];
  int rlo[NB][2], rhi[NB][2];  // keys that the thread's rows may see
  int free_lo = 0, free_hi = 0;  // keys that every row of the unit may see
  bool seg_starts_unit = false, fresh = true;  // fresh: the next tile begins a segment
  auto dcol = [&](int x, int e) { return kQuant ? rq * (D / 8) + 2 * x + e : 16 * x + 8 * e + rq; };
  // the queries of unit t, as they are in memory
  auto load_q = [&](const PagedDesc& t) {
    const int kh = p.nblk == 1 ? t.unit : t.unit / p.nblk, row0 = (t.unit - kh * p.nblk) * C::kRows + rg * 8 * NB;
    constexpr int W2 = kQuant ? 8 : 4;  // words of q that belong to one 16-byte unit of k
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = row0 + nb * 8 + rq;
      const int h = p.Nq == 1 ? r : r / p.Nq;
      const uint8_t* qr = p.q + 2 * (r < p.R ? p.sq.row(t.b, kh * p.g + h, r - h * p.Nq) : 0);
#pragma unroll
      for (int i = 0; i < D / 2 / W2 / 4; ++i)
#pragma unroll
        for (int y = 0; y < W2; y += 4) {
          const uint4 v = r < p.R ? __ldg(reinterpret_cast<const uint4*>(qr + (qd + 4 * i) * W2 * 4 + y * 4))
                                  : make_uint4(0, 0, 0, 0);
          const int s = i * (W2 / 2) + y / 2;
          qb[nb][s][0] = v.x;
          qb[nb][s][1] = v.y;
          qb[nb][s + 1][0] = v.z;
          qb[nb][s + 1][1] = v.w;
        }
    }
  };

  {
    Tile t[ST];
#pragma unroll
    for (int n = 0; n < ST; ++n) t[n] = fetch(n);
#pragma unroll
    for (int n = 0; n < ST; ++n) store(n, t[n]);
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < ST - 1; ++n) issue(n);
  load_q(desc[0]);
  Tile next = fetch(ST);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int n = 0; n < cnt; ++n) {
    cp_async_wait<ST - 2>();
    store(n + ST, next);
    __syncthreads();  // tile n has landed; everyone is done with tile n - 1
    issue(n + ST - 1);
    next = fetch(n + ST + 1);

    const PagedDesc& t = desc[n % kPagedRing];
    const int key0 = t.key0, flags = t.flags;
    if (fresh) {
      fresh = false;
      seg_starts_unit = flags & kFlagUnitStart;
      const int L = t.L, row0 = (p.nblk == 1 ? 0 : t.unit % p.nblk * C::kRows) + rg * 8 * NB;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float back = p.scale_log2;  // what a product of the scaled queries is multiplied by
        if (kQuant) {
          // bf16 queries as f16: scaled by a power of two that puts the row's
          // largest into [2^14, 2^15); exact down to 2^-32 of it
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
          m[nb][c] = -INFINITY;
          l[nb][c] = 0.f;
          vref[nb][c] = __uint_as_float(1u << 23);   // 2^-126
          vinv[nb][c] = __uint_as_float(253u << 23);
          rowf[nb][c] = kQuant ? __shfl_sync(0xffffffffu, back, (2 * qd + c) * 4) : back;
          const int r = row0 + nb * 8 + 2 * qd + c;
          const int i = p.Nq == 1 ? 0 : r % p.Nq, pos = L - p.Nq + i;
          rlo[nb][c] = 0;
          rhi[nb][c] = 0;  // padding rows see nothing
          if (r < p.R) {
            rlo[nb][c] = p.window < 0 ? 0 : max(0, pos - p.window);
            rhi[nb][c] = pos < 0 ? 0 : (p.causal ? pos + 1 : (p.window < 0 ? L : min(L, pos + p.window + 1)));
          }
        }
#pragma unroll
        for (int x = 0; x < DT; ++x) acc[nb][x][0] = acc[nb][x][1] = acc[nb][x][2] = acc[nb][x][3] = 0.f;
      }
      free_lo = p.window < 0 ? 0 : max(0, L - 1 - p.window);
      free_hi = L < p.Nq ? 0 : (p.causal ? L - p.Nq + 1 : (p.window < 0 ? L : min(L, L - p.Nq + p.window + 1)));
    }

    const uint8_t* pK = smem + (n % ST) * C::kStageBytes;
    const uint8_t* pV = pK + C::kTileBytes;
    const uint32_t sV = paged_smem(pV);
    const float* scl = reinterpret_cast<const float*>(pV + C::kTileBytes);
    bool some = key0 < free_lo || key0 + TK > free_hi;
#pragma unroll
    for (int i = 0; i < TK / 32; ++i) some |= t.valid[i] != 0xffffffffu;
    // the steps of a tile; kEdge: some row may not see some key of it
    auto steps = [&](auto edge_tile) {
      constexpr bool edge = decltype(edge_tile)::value;
#pragma unroll 1
    for (int s = 0; s < TK / KW / (16 * KS); ++s) {
      const int kb = (kw * (TK / KW / (16 * KS)) + s) * 16 * KS;
      uint32_t vm = 0xffffffffu;
      if (edge) {
        vm = t.valid[kb >> 5] >> (kb & 31);
        if ((KS == 2 ? vm : vm & 0xffffu) == 0) continue;  // behind the end
      }
      // ---- S^T of keys 16 k + rq (elements 0, 1) and 16 k + rq + 8 (2, 3), rows 2 qd and 2 qd + 1
      float sc[KS][NB][4];
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[k][nb][0] = sc[k][nb][1] = sc[k][nb][2] = sc[k][nb][3] = 0.f;
#pragma unroll
      for (int i = 0; i < (kQuant ? D / 64 : D / 32); ++i)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint4 a = *reinterpret_cast<const uint4*>(pK + k_at<RB>(kb + 16 * k + rq, qd + 4 * i)),
                      b = *reinterpret_cast<const uint4*>(pK + k_at<RB>(kb + 16 * k + rq + 8, qd + 4 * i));
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
          if (kQuant) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(aw[x], &a0, &a2);
              e4m3x4_to_f16(bw[x], &a1, &a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16<true>(sc[k][nb], a0, a1, a2, a3, qb[nb][(i * 4 + x) % QS]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16<false>(sc[k][nb], aw[2 * x], bw[2 * x], aw[2 * x + 1], bw[2 * x + 1], qb[nb][(2 * i + x) % QS]);
          }
        }
      float vs[KS][2];
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ks = kQuant ? scl[kb + 16 * k + 8 * h + rq] : 1.f;
          vs[k][h] = kQuant ? scl[TK + kb + 16 * k + 8 * h + rq] : 1.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              sc[k][nb][2 * h + c] *= rowf[nb][c];
              if (kQuant) sc[k][nb][2 * h + c] *= ks;
            }
        }
      uint32_t allowed = 0xffffffffu;  // bit 4 (k NB + nb) + e
      if (edge) {
        allowed = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = 16 * k + rq + 8 * (e >> 1), j = key0 + kb + key;
              if (((vm >> key) & 1) && j >= rlo[nb][e & 1] && j < rhi[nb][e & 1])
                allowed |= 1u << (4 * (k * NB + nb) + e);
              else
                sc[k][nb][e] = -INFINITY;
            }
      }
      auto on = [&](int k, int nb, int e) { return !edge || ((allowed >> (4 * (k * NB + nb) + e)) & 1) != 0; };
      // ---- running maximum: moved only when it grows by more than 8 (weights
      // stay below 2^8).  Quantised: weights reach the second product as f16
      // multiples of the largest value scale so far (vref, a power of two above
      // it); a row's accumulator counts in units of its vref.
      bool grow = false;
      float mx[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[nb][c] = fmaxf(sc[0][nb][c], sc[0][nb][2 + c]);
          if (KS == 2) mx[nb][c] = fmaxf(mx[nb][c], fmaxf(sc[KS - 1][nb][c], sc[KS - 1][nb][2 + c]));
          grow |= mx[nb][c] > m[nb][c] + 8.f;
          if (kQuant)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) grow |= fabsf(vs[k][h]) >= vref[nb][c] && on(k, nb, 2 * h + c);
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t ve = 0;
            if (kQuant)
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (on(k, nb, 2 * h + c)) ve = max(ve, (__float_as_uint(vs[k][h]) >> 23) & 0xffu);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
              mx[nb][c] = fmaxf(mx[nb][c], __shfl_xor_sync(0xffffffffu, mx[nb][c], o));
              if (kQuant) ve = max(ve, __shfl_xor_sync(0xffffffffu, ve, o));
            }
            const float mn = mx[nb][c] > m[nb][c] + 8.f ? mx[nb][c] : m[nb][c];
            float f = m[nb][c] == mn ? 1.f : exp2_fast(m[nb][c] - mn);
            m[nb][c] = mn;
            l[nb][c] *= f;
            if (kQuant) {
              const float vn = fmaxf(vref[nb][c], __uint_as_float(min(ve + 1u, 253u) << 23));
              vinv[nb][c] = __uint_as_float((254u << 23) - __float_as_uint(vn));
              f *= vref[nb][c] * vinv[nb][c];
              vref[nb][c] = vn;
            }
#pragma unroll
            for (int x = 0; x < DT; ++x) {
              acc[nb][x][c] *= f;
              acc[nb][x][2 + c] *= f;
            }
          }
      }
      // The weights are rounded to 16 bits for the second product: bf16 (half a
      // step is 2^-8 of a weight), or f16 of weight * value scale / vref, 2^-11
      // of it down to 2^-14; keys whose scale is below 2^-12 vref take the slow
      // form below.
      uint32_t pb[KS][NB][2];
      bool slow[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        slow[k] = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mu = m[nb][e & 1] == -INFINITY ? 0.f : m[nb][e & 1];
            const float w = exp2_fast(sc[k][nb][e] - mu);
            l[nb][e & 1] += w;
            sc[k][nb][e] = w;
            if (kQuant) {
              const float u = vs[k][e >> 1] * vinv[nb][e & 1];
              slow[k] |= on(k, nb, e) && fabsf(u) < 0x1p-12f && fabsf(vs[k][e >> 1]) > 0x1p-90f;
              sc[k][nb][e] = on(k, nb, e) ? w * u : 0.f;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pb[k][nb][h] = transpose8x8(kQuant ? pack_f16(sc[k][nb][2 * h], sc[k][nb][2 * h + 1])
                                               : pack_bf16(sc[k][nb][2 * h], sc[k][nb][2 * h + 1]));
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int kk = kb + 16 * k;
        uint32_t bad = slow[k];
        if (kQuant) {
          uint32_t w[4][D / 32];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int key = kk + 2 * qd + (y & 1) + 8 * (y >> 1);
            if (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(pV + v_at<RB, kQuant>(key, rq));
              w[y][0] = v.x;
              w[y][1] = v.y;
              w[y][2 % (D / 32)] = v.z;
              w[y][3 % (D / 32)] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(pV + v_at<RB, kQuant>(key, rq >> 1) + (rq & 1) * 8);
              w[y][0] = v.x;
              w[y][1] = v.y;
            }
          }
          if (edge)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int z = 0; z < D / 32; ++z) bad |= ((w[y][z] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // NaN codes
          if (!__any_sync(0xffffffffu, bad)) {
#pragma unroll
            for (int x = 0; x < DT; ++x) {  // columns 2x, 2x + 1 of the thread's D / 8
              const uint32_t sel = (x & 1) ? 0x7362 : 0x5140;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(w[0][x >> 1], w[1][x >> 1], sel), &a0, &a1);
              e4m3x4_to_f16(__byte_perm(w[2][x >> 1], w[3][x >> 1], sel), &a2, &a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16<true>(acc[nb][x], a0, a1, a2, a3, pb[k][nb]);
            }
            continue;
          }
        } else {
          const int key = kk + (lane & 7) + ((lane >> 4) << 3);
          const uint32_t at = sV + v_at<RB, kQuant>(key, (lane >> 3) & 1);
          if (edge) {
#pragma unroll
            for (int x = 0; x < DT; ++x) {
              uint32_t a[4];
              ldmatrix_x4_trans(a, at ^ (x << 5));
#pragma unroll
              for (int y = 0; y < 4; ++y)
                bad |= ((a[y] & 0x7f80u) == 0x7f80u) | ((a[y] & 0x7f800000u) == 0x7f800000u);
            }
          }
          if (!edge || !__any_sync(0xffffffffu, bad)) {
#pragma unroll
            for (int x0 = 0; x0 < DT; x0 += 4) {
              uint32_t a[4][4];
#pragma unroll
              for (int x = 0; x < 4; ++x) ldmatrix_x4_trans(a[x], at ^ ((x0 + x) << 5));
#pragma unroll
              for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16<false>(acc[nb][x0 + x], a[x][0], a[x][1], a[x][2], a[x][3], pb[k][nb]);
            }
            continue;
          }
        }
        // The slow form: products one by one in fp32, weights of zero left out.
        // For an infinity or NaN among the values of a tile that some rows see
        // only in part (0 * infinity would reach rows that may not see that key),
        // and for value scales too far apart for f16.
#pragma unroll 1
        for (int y = 0; y < 16; ++y)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int src = (y & 7) * 4 + qd;
            const float f0 = __shfl_sync(0xffffffffu, y < 8 ? sc[k][nb][0] : sc[k][nb][2], src);
            const float f1 = __shfl_sync(0xffffffffu, y < 8 ? sc[k][nb][1] : sc[k][nb][3], src);
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int col = dcol(x, e);
                const uint32_t at = sV + v_at<RB, kQuant>(kk + y, col * ES / 16) + (col * ES) % 16;
                uint32_t z;
                float v;
                if (kQuant) {
                  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z) : "r"(at) : "memory");
                  v = e4m3x2_to_float2(static_cast<uint16_t>(z)).x;
                } else {
                  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(z) : "r"(at) : "memory");
                  v = __uint_as_float(z << 16);
                }
                if (f0 != 0.f) acc[nb][x][2 * e] += f0 * v;
                if (f1 != 0.f) acc[nb][x][2 * e + 1] += f1 * v;
              }
          }
      }
    }

    };
    if (some)
      steps(std::true_type{});
    else
      steps(std::false_type{});

    if (!(flags & kFlagSegEnd)) continue;
    // ---- the segment's end: the KW warps of a row group join their states in tile n's stage
    fresh = true;
    const int b = t.b, unit = t.unit;
    const int kh = p.nblk == 1 ? unit : unit / p.nblk, row0 = (unit - kh * p.nblk) * C::kRows;
    const bool whole = seg_starts_unit && (flags & kFlagUnitEnd);
    const int slot = 2 * cta + (seg_starts_unit ? 1 : 0);
    if (n + 1 < cnt) load_q(desc[(n + 1) % kPagedRing]);  // the next unit's queries, on their way meanwhile
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], o);
        if (rq == 0) stat[(warp * NB + nb) * 8 + 2 * qd + c] = make_float4(m[nb][c], l[nb][c], vref[nb][c], 0.f);
      }
    float* merge = reinterpret_cast<float*>(smem + (n % ST) * C::kStageBytes);  // [4 warps][8 rows][kMergeStride]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __syncthreads();  // tile n is read, the block before this one joined
      float* mine = merge + (warp * 8 + 2 * qd) * C::kMergeStride;
#pragma unroll
      for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (kQuant) {
            *reinterpret_cast<float2*>(mine + c * C::kMergeStride + dcol(x, 0)) =
                make_float2(acc[nb][x][c], acc[nb][x][2 + c]);
          } else {
            mine[c * C::kMergeStride + dcol(x, 0)] = acc[nb][x][c];
            mine[c * C::kMergeStride + dcol(x, 1)] = acc[nb][x][2 + c];
          }
      __syncthreads();
      constexpr int LPR = D / 4, RPP = kPagedThreads / LPR;  // threads of a row, rows of a pass
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
          float f = st[w].x == -INFINITY ? (st[w].y == 0.f ? 0.f : 1.f) : exp2_fast(st[w].x - mt);
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
    if (n == cnt - 1 && tid == 0) {
      int4 s = make_int4(0, 0, 0, 0);
      if (seg_starts_unit && !(flags & kFlagUnitEnd)) {  // goes on in the next CTAs
        s = make_int4(b, unit, static_cast<int>((last_end * G - 1) / W) - group + 1, 0);
      }
      p.split[cta] = s;
    }
  }
  cp_async_wait<0>();
}

// Joins the partials of the units that several CTAs share: block (c, y) the
// unit that starts in CTA c, 8 rows of it, a warp each.  Partial 0 is CTA c's
// second slot, the others are the lane's following CTAs' first.
template <int D, bool kQuant>
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
    return (static_cast<long long>(2) * (blockIdx.x + i * p.lanes) + (i == 0 ? 1 : 0)) * p.prow + rloc;
  };
  float m = -INFINITY, l = 0.f, u = 0x1p-126f, acc[E];  // u: the accumulators' unit, the largest so far
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float4 st = make_float4(-INFINITY, 0.f, 0x1p-126f, 0.f);
    if (i0 + lane < parts) st = p.part_m[at(i0 + lane)];
    float mn = fmaxf(m, st.x), un = fmaxf(u, st.z);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      un = fmaxf(un, __shfl_xor_sync(0xffffffffu, un, o));
    }
    const float ui = __uint_as_float((254u << 23) - __float_as_uint(un));
    float old = m == -INFINITY ? 0.f : exp2_fast(m - mn);
    float w = st.x == -INFINITY ? (st.y == 0.f ? 0.f : 1.f) : exp2_fast(st.x - mn);
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
