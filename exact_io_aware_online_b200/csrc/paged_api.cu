// paged_api.cu -- the paged-cache part of libfa.so's C ABI (include/fa.h):
// argument checking and kernel launches.  A translation unit of its own, so
// that the dense kernels' sources (which their captured profiles are keyed by)
// do not depend on it.  Like there, every entry point validates on the host
// first and enqueues nothing when an argument is bad.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/fa.h"
#include "cache_sm100.cuh"
#include "paged_sm100.cuh"

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The kernels run on the current device: a stream of another one is an
// argument error (NULL is the current device's legacy stream).  A capturing
// stream cannot be asked for its device without ending the capture; there the
// launch itself fails on a foreign stream.
fa_status check_stream(void* stream) {
  int cur = 0, sdev = 0;
  if (cudaGetDevice(&cur) != cudaSuccess) return FA_ERR_CUDA;
  if (stream == nullptr) return FA_OK;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &capturing) != cudaSuccess) return FA_ERR_INVALID_ARG;
  if (capturing != cudaStreamCaptureStatusNone) return FA_OK;
  if (cudaStreamGetDevice(static_cast<cudaStream_t>(stream), &sdev) != cudaSuccess) return FA_ERR_INVALID_ARG;
  return sdev == cur ? FA_OK : FA_ERR_INVALID_ARG;
}

// The kernel may begin while the one before it in the stream ends; it waits for that one itself.
template <typename... KArgs, typename... Args>
fa_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Strides of an [n0, n1, n2, inner] tensor of esize-byte elements: positive,
// below 2^40 bytes and multiples of `align` bytes; an axis of extent 1 is never
// stepped, so its stride is replaced.  `output`: the layout must be one-to-one
// (sorted by stride, each axis steps past the extent of the axes inside it).
fa_status check_strides(const fa_strides& in, long long n0, long long n1, long long n2, int inner, int esize, int align,
                        bool output, fa::Strides* out) {
  struct Axis {
    long long stride, extent;
  } ax[3] = {{in.batch, n0}, {in.head, n1}, {in.row, n2}};
  const long long lim = (1LL << 40) / esize;
  for (Axis& a : ax) {
    if (a.extent == 1) a.stride = 16;  // any aligned value
    if (a.stride <= 0 || a.stride >= lim) return FA_ERR_INVALID_ARG;
    if ((a.stride * esize) % align != 0) return FA_ERR_MISALIGNED;
  }
  *out = fa::Strides{ax[0].stride, ax[1].stride, ax[2].stride};
  if (output) {
    std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
    long long span = inner;
    for (const Axis& a : ax) {
      if (a.extent == 1) continue;
      if (a.stride < span) return FA_ERR_INVALID_ARG;
      span = a.stride * a.extent;
    }
  }
  return FA_OK;
}

void magic(int divisor, uint32_t* mul, int* shift) {  // see page_of()
  *shift = 0;
  while ((1LL << *shift) < divisor) ++*shift;
  *mul = static_cast<uint32_t>(((1ULL << (31 + *shift)) + divisor - 1) / divisor);
}

// `written`: the pages are an output.
fa_status check_cache(const fa_paged_cache* c, fa_dtype dtype, bool written, fa::CacheParams* p) {
  if (!c || !c->k_pages || !c->v_pages || !c->page_table || !c->seqlens) return FA_ERR_INVALID_ARG;
  if (c->B < 1 || c->Hkv < 1 || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_CACHE_BF16 && c->dtype != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (c->B > 1 && c->table_stride < c->max_pages) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  // positions are 32-bit
  if (static_cast<long long>(c->page_size) * c->max_pages > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  const bool quant = c->dtype == FA_CACHE_E4M3;
  if (quant && (!c->k_scale || !c->v_scale)) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return FA_ERR_MISALIGNED;
  p->scales = fa::Strides{0, 0, 0};
  fa_status s = check_strides(c->pages, c->num_pages, c->Hkv, c->page_size, c->d, quant ? 1 : 2, 16, written, &p->pages);
  if (s != FA_OK) return s;
  if (quant) {
    if (((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u) != 0)
      return FA_ERR_MISALIGNED;
    s = check_strides(c->scales, c->num_pages, c->Hkv, c->page_size, 1, 4, 4, written, &p->scales);
    if (s != FA_OK) return s;
  }
  p->k = static_cast<uint8_t*>(c->k_pages);
  p->v = static_cast<uint8_t*>(c->v_pages);
  p->ks = c->k_scale;
  p->vs = c->v_scale;
  p->table = c->page_table;
  p->seqlens = c->seqlens;
  p->table_stride = c->B > 1 ? c->table_stride : 0;
  p->B = c->B;
  p->Hkv = c->Hkv;
  p->num_pages = c->num_pages;
  p->page_size = c->page_size;
  p->max_pages = c->max_pages;
  magic(c->page_size, &p->page_mul, &p->page_shift);
  return FA_OK;
}

template <bool kWrite>
fa_status move_tokens(const fa_paged_cache* cache, void* k, void* v, const fa_strides* strides, const int* cu, int T,
                      fa_dtype dtype, void* stream) {
  fa::MoveParams p{};
  fa_status s = check_cache(cache, dtype, kWrite, &p.c);
  if (s != FA_OK) return s;
  if (T < 0 || !cu) return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (!k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return FA_ERR_MISALIGNED;
  const int d = cache->d, Hkv = cache->Hkv;
  const fa_strides packed{1, d, static_cast<long long>(Hkv) * d};
  fa::Strides sk, sv;
  if ((s = check_strides(strides ? strides[0] : packed, 1, Hkv, T, d, 2, 16, !kWrite, &sk)) != FA_OK) return s;
  if ((s = check_strides(strides ? strides[1] : packed, 1, Hkv, T, d, 2, 16, !kWrite, &sv)) != FA_OK) return s;
  const long long rows = 2LL * Hkv * T;
  if (rows > (1LL << 31) - fa::kMoveWarps * fa::kMoveRows) return FA_ERR_UNSUPPORTED;  // counted in 32 bits
  if ((s = check_stream(stream)) != FA_OK) return s;
  p.k = static_cast<uint8_t*>(k);
  p.v = static_cast<uint8_t*>(v);
  p.k_row = sk.n;
  p.k_head = sk.h;
  p.v_row = sv.n;
  p.v_head = sv.h;
  p.cu = cu;
  p.T = T;
  magic(2 * Hkv, &p.row_mul, &p.row_shift);
  const long long blocks = (rows + fa::kMoveWarps * fa::kMoveRows - 1) / (fa::kMoveWarps * fa::kMoveRows);
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * fa::kMoveWarps);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool quant = cache->dtype == FA_CACHE_E4M3;
  if (d == 64)
    return quant ? launch(fa::cache_move_kernel<64, true, kWrite>, grid, block, 0, st, p)
                 : launch(fa::cache_move_kernel<64, false, kWrite>, grid, block, 0, st, p);
  return quant ? launch(fa::cache_move_kernel<128, true, kWrite>, grid, block, 0, st, p)
               : launch(fa::cache_move_kernel<128, false, kWrite>, grid, block, 0, st, p);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(f)
               : nullptr;
  }();
  return fn;
}

// Pages [num_pages, Hkv, page_size, d] in boxes of `box` tokens of one page and
// `heads` heads: rows of 128 bytes (64 where a row has no more) with the swizzle of that
// width.  Tokens behind the page's end and a page number of num_pages read as zero.
bool page_map(CUtensorMap* m, const void* base, const fa::CacheParams& c, int d, bool quant, int box, int heads) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const int es = quant ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.pages.n) * es, static_cast<cuuint64_t>(c.pages.h) * es,
                                 static_cast<cuuint64_t>(c.pages.b) * es};
  const int inner = std::min(d * es, 128);
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(inner / es), static_cast<cuuint32_t>(box),
                               static_cast<cuuint32_t>(heads), 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return enc(m, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The workspace: split[CTAs] (int4), part_m[2 * CTAs][rows] (float4), part_o[2 * CTAs][rows][d] (float)
struct PagedOffsets {
  size_t part_m, part_o, bytes;
};
PagedOffsets paged_offsets(int rows, int d) {
  PagedOffsets w;
  w.part_m = fa::kPagedMaxCtas * sizeof(int4);
  w.part_o = w.part_m + sizeof(float4) * 2 * fa::kPagedMaxCtas * rows;
  w.bytes = w.part_o + sizeof(float) * 2 * fa::kPagedMaxCtas * rows * d;
  return w;
}

int paged_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : R <= 32 ? 32 : 64; }  // rows of a kv head in a unit
// kv heads of a unit: as many as leave each warp rows of its own, where they
// divide Hkv.  One for few sequences, whose units all CTAs would share (one
// token over 4000 in bf16, B = 1: 23 us against 29 us with four; B = 8, 32768:
// the same), and where a tile of 32 KB would be 16 keys (rows of 256 bytes: 64
// ragged sequences 125 us against 130 us; rows of 128 bytes, pages of 16: 107 us
// with four against 123 us).
int paged_heads(int B, int R, int Hkv, int row_bytes) {
  if (B * static_cast<long long>(Hkv) < 64) return 1;
  if (R <= 8 && row_bytes < 256 && Hkv % 4 == 0) return 4;
  return R > 8 && R <= 16 && Hkv % 2 == 0 ? 2 : 1;
}

template <int D, bool kQuant, int NB, int RG, int HG>
fa_status launch_paged(const fa_paged_cache* cache, fa::PagedParams p, cudaStream_t st) {
  using C = fa::PagedCfg<D, kQuant, NB, RG, HG>;
  const auto kernel = fa::paged_kernel<D, kQuant, NB, RG, HG>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static std::atomic<uint64_t> ready{0};  // devices on which this kernel may use its shared memory
  const uint64_t bit = dev < 64 ? 1ULL << dev : 0;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
      return FA_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  p.box_log = 3;
  while (p.box_log < 5 && p.pad_page % (2 << p.box_log) == 0 && C::kTile % (2 << p.box_log) == 0) ++p.box_log;
  CUtensorMap mk, mv;
  if (!page_map(&mk, cache->k_pages, p.c, D, kQuant, 1 << p.box_log, HG) ||
      !page_map(&mv, cache->v_pages, p.c, D, kQuant, 1 << p.box_log, HG))
    return FA_ERR_CUDA;
  p.scale_rows = kQuant && (HG == 1 || p.c.scales.h == 1) && p.c.scales.n % HG == 0 && p.c.scales.b % HG == 0 &&
                 ((reinterpret_cast<uintptr_t>(p.c.ks) | reinterpret_cast<uintptr_t>(p.c.vs)) & (4 * HG - 1)) == 0;
  // lanes: the largest divisor of a sequence's units that leaves at most one CTA in sixteen without work
  const int units = p.c.Hkv / HG * p.nblk, most = 148 * C::kCtas;
  p.lanes = std::min(units, most);
  while (units % p.lanes != 0 || most % p.lanes > most / 16) --p.lanes;
  // no more groups than the lengths could give tiles
  const long long cap = static_cast<long long>(p.c.max_pages) * p.pad_page;
  const double tiles = static_cast<double>((cap + C::kTile - 1) / C::kTile) * p.c.B;  // of one unit of each sequence
  // tiles of a unit at most: of the table's tokens, or of a window's and the pages and boxes it cuts
  long long keys = cap;
  if (p.window >= 0) {
    const long long seen = static_cast<long long>(p.window) + p.Nq;
    keys = std::min(cap, (seen + 2 * p.c.page_size - 2) / p.c.page_size * p.pad_page);
  }
  // units of up to kPagedWhole tiles are never shared, and of up to twice as many where one for each group keeps a
  // quarter of the groups or more at work (device time, shared against whole: 32 x 500 tokens in bf16 24.0 and 18.9 us,
  // 100 x 250 at d = 64 27.8 and 22.0 us; but one sequence of 500 10.3 and 14.8 us, 128 x 500 51.8 and 53.9 us)
  const long long most_tiles = (keys + C::kTile - 1) / C::kTile, in_lane = static_cast<long long>(p.c.B) * (units / p.lanes),
                  groups = most / p.lanes;
  p.whole = most_tiles <= fa::kPagedWhole || (most_tiles <= 2 * fa::kPagedWhole && 4 * in_lane >= groups && in_lane <= groups);
  const int ctas = p.lanes * static_cast<int>(std::min<double>(most / p.lanes, tiles * (units / p.lanes)));
  const fa_status s = launch(kernel, dim3(ctas), dim3(fa::kPagedThreads), C::kSmemBytes, st, mk, mv, p);
  if (s != FA_OK || p.whole) return s;
  // four warps a row where there are few rows (a wave of warps, and few blocks without work)
  const bool few = HG * p.prow <= 8 && static_cast<long long>(p.c.B) * p.H * p.Nq <= 148 * 16;
  const int rows = fa::kPagedCombineWarps / (few ? 4 : 1);
  const dim3 grid(ctas, (HG * p.prow + rows - 1) / rows), block(32 * fa::kPagedCombineWarps);
  return few ? launch(fa::paged_combine_kernel<D, kQuant, 4>, grid, block, 0, st, p, C::kRows, HG)
             : launch(fa::paged_combine_kernel<D, kQuant, 1>, grid, block, 0, st, p, C::kRows, HG);
}

template <int D, bool kQuant>
fa_status launch_paged_rows(const fa_paged_cache* cache, const fa::PagedParams& p, cudaStream_t st) {
  const int heads = paged_heads(p.c.B, p.R, p.c.Hkv, kQuant ? D : 2 * D);
  switch (paged_rows(p.R)) {
    case 8:
      if constexpr (kQuant || D == 64)  // rows of less than 256 bytes
        if (heads == 4) return launch_paged<D, kQuant, 1, 1, 4>(cache, p, st);
      return launch_paged<D, kQuant, 1, 1, 1>(cache, p, st);
    case 16:
      return heads == 2 ? launch_paged<D, kQuant, 1, 2, 2>(cache, p, st) : launch_paged<D, kQuant, 1, 2, 1>(cache, p, st);
    case 32: return launch_paged<D, kQuant, 1, 4, 1>(cache, p, st);
    default: return launch_paged<D, kQuant, 2, 4, 1>(cache, p, st);
  }
}

bool paged_sizes_ok(int B, int H, int Hkv, int Nq) {
  return B >= 1 && H >= 1 && Hkv >= 1 && Nq >= 1 && H % Hkv == 0 &&
         static_cast<long long>(B) * H <= 0x7fffffffLL / Nq;
}

}  // namespace

// This translation unit's copies of the device status word and the debugging
// switches, for the entry points that report and set them (fa_api.cu).
namespace fa {

cudaError_t paged_take_status(unsigned int* v) {
  const unsigned int zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(v, g_status, sizeof(*v));
  return e != cudaSuccess || *v == 0 ? e : cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}
cudaError_t paged_set_wait_limit(unsigned long long ns) { return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)); }
cudaError_t paged_set_stall(int on) { return cudaMemcpyToSymbol(g_debug_stall, &on, sizeof(on)); }

}  // namespace fa

extern "C" {

fa_status fa_cache_write(const fa_paged_cache* cache, const void* k, const void* v, const fa_strides* strides,
                         const int* cu_seqlens_dev, int T, fa_dtype dtype, void* stream) {
  return move_tokens<true>(cache, const_cast<void*>(k), const_cast<void*>(v), strides, cu_seqlens_dev, T, dtype,
                           stream);
}

fa_status fa_cache_read(const fa_paged_cache* cache, void* k, void* v, const fa_strides* strides,
                        const int* cu_seqlens_dev, int T, fa_dtype dtype, void* stream) {
  return move_tokens<false>(cache, k, v, strides, cu_seqlens_dev, T, dtype, stream);
}

size_t fa_fwd_paged_workspace_size(int B, int H, int Hkv, int Nq, int d) {
  if (!paged_sizes_ok(B, H, Hkv, Nq) || (d != 64 && d != 128)) return 0;
  const long long R = static_cast<long long>(H / Hkv) * Nq;
  const int r = static_cast<int>(std::min(R, 64LL));
  return paged_offsets(paged_heads(B, r, Hkv, d) * r, d).bytes;  // of a quantised cache: the most heads
}

fa_status fa_fwd_paged(const fa_paged_cache* cache, const void* q, void* o, float* lse, const fa_strides* strides,
                       int H, int Nq, float scale, int causal, int window, void* workspace, size_t ws_bytes,
                       fa_dtype dtype, void* stream) {
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !std::isfinite(scale_log2) || window < -1) return FA_ERR_INVALID_ARG;
  fa::PagedParams p{};
  fa_status s = check_cache(cache, dtype, false, &p.c);
  if (s != FA_OK) return s;
  const int B = cache->B, Hkv = cache->Hkv, d = cache->d;
  if (!paged_sizes_ok(B, H, Hkv, Nq)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const fa_strides dense{static_cast<long long>(H) * Nq * d, static_cast<long long>(Nq) * d, d};
  if ((s = check_strides(strides ? strides[0] : dense, B, H, Nq, d, 2, 16, false, &p.sq)) != FA_OK) return s;
  if ((s = check_strides(strides ? strides[1] : dense, B, H, Nq, d, 2, 16, true, &p.so)) != FA_OK) return s;
  if (!workspace || ws_bytes < fa_fwd_paged_workspace_size(B, H, Hkv, Nq, d)) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_MISALIGNED;
  p.pad_page = (cache->page_size + 7) & ~7;
  p.R = H / Hkv * Nq;
  const int block = paged_rows(p.R);
  p.nblk = (p.R + block - 1) / block;
  // positions are 32-bit with pages rounded up too, and so are the counts of tiles (of 16 keys or more): those of all
  // sequences and of a CTA
  const long long cap = static_cast<long long>(cache->max_pages) * p.pad_page;
  const double tiles = static_cast<double>(cap) / 16 * B;
  if (cap > (1LL << 30) || tiles > 2e9 || tiles / 296 * Hkv * p.nblk > 2e9) return FA_ERR_UNSUPPORTED;
  if ((s = check_stream(stream)) != FA_OK) return s;
  p.q = static_cast<const uint8_t*>(q);
  p.o = static_cast<uint8_t*>(o);
  p.lse = lse;
  p.H = H;
  p.Nq = Nq;
  p.g = H / Hkv;
  p.scale_log2 = scale_log2;
  p.causal = causal ? 1 : 0;
  p.window = window < (1 << 30) ? window : -1;  // positions stay below 2^30
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  p.prow = std::min(p.R, block);
  const bool quant = cache->dtype == FA_CACHE_E4M3;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const PagedOffsets at = paged_offsets(paged_heads(B, p.R, Hkv, quant ? d : 2 * d) * p.prow, d);
  p.split = reinterpret_cast<int4*>(ws);
  p.part_m = reinterpret_cast<float4*>(ws + at.part_m);
  p.part_o = reinterpret_cast<float*>(ws + at.part_o);
  magic(p.pad_page, &p.pad_mul, &p.pad_shift);
  if (d == 64) return quant ? launch_paged_rows<64, true>(cache, p, st) : launch_paged_rows<64, false>(cache, p, st);
  return quant ? launch_paged_rows<128, true>(cache, p, st) : launch_paged_rows<128, false>(cache, p, st);
}

}  // extern "C"
