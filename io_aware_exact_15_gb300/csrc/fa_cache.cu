// Paged key/value cache: writing new tokens (quantised on the way in) and
// reading a range of positions back as bf16.
//
// A page holds page_size positions of every key/value head: k_cache and
// v_cache are [num_pages, Hkv, page_size, d], so one (page, head) is one
// contiguous tile.  Position p of sequence b lives in page
// page_table[b][p / page_size], row p mod page_size.  Number formats and
// the scale rule: fa_quant.cuh.
//
// Both directions are bound by memory (bf16 on one side, the stored format
// on the other), or by the launch when a step writes one token per
// sequence.  8 elements per lane: a row is d / 8 lanes, its largest element
// a shuffle reduction, and a warp's rows are consecutive positions of one
// (sequence, head), so that data and scale bytes land next to each other.
// Measured: 16 x 4096 tokens of 4 heads of 128, appended as int8 and read
// back, ragged: 54.9 us, 4.8 TB/s (the bytes at a plain copy's rate: 39.1
// us).  Full rows: append bf16 6.5, e4m3 5.2, int8 4.9 TB/s, read 6.4, 6.1, 6.0:
// finding the scale and rounding is what the 8-bit append adds (int8 by
// conversions to integers: 4.3), the rest latency: lengths, then the page,
// then rows, one wave of blocks after the other.  Persistent warps that ask
// for the next rows before they finish these took 60 instead of 47 us.
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_quant.cuh"

namespace fa {
namespace {

struct CacheParams {
  void *kc, *vc;             // caches
  uint8_t *ks, *vs;          // scale bytes [num_pages, Hkv, page]
  const int *page_table, *start, *counts;
  void *k, *v;               // bf16 rows: read (append) or written (read)
  Strides sk, sv;
  int B, Hkv, N, num_pages, log_page, max_pages;
};

// Index of (page, head, row) for token n of sequence b, or -1: past the
// sequence's count, outside the table, or a page id outside the pool.
FA_DEV long long cache_row(const CacheParams& p, int b, int h, uint32_t n, int start,
                           uint32_t count) {
  const long long pos = static_cast<long long>(start) + n;
  if (n >= count || start < 0 || (pos >> p.log_page) >= p.max_pages) return -1;
  const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + (pos >> p.log_page)];
  if (page < 0 || page >= p.num_pages) return -1;
  return (((static_cast<long long>(page) * p.Hkv + h)) << p.log_page) +
         (pos & ((1 << p.log_page) - 1));
}

// One block: blockDim / 32 * RPW * U consecutive tokens of one (sequence,
// k or v, head).
template <int D, int FMT, bool WRITE, int U>
__global__ void __launch_bounds__(256) fa_cache_kernel(const CacheParams p) {
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = warps * RPW * U, chunks = (p.N - 1) / per + 1;
  const int bkh = blockIdx.x / chunks, chunk = blockIdx.x - bkh * chunks;
  const int b = bkh / (2 * p.Hkv), kh = bkh - b * 2 * p.Hkv;
  const bool isk = kh < p.Hkv;
  const int h = isk ? kh : kh - p.Hkv;
  const int start = p.start[b], l = lane % LPR;
  // (unsigned: N may be close to 2^31, and the last block reaches past it)
  const uint32_t count = p.counts ? max(min(p.counts[b], p.N), 0) : p.N;
  const uint32_t n0 = static_cast<uint32_t>(chunk) * per + warp * RPW * U + lane / LPR;
  const Strides s = isk ? p.sk : p.sv;
  uint16_t* x0 = static_cast<uint16_t*>(isk ? p.k : p.v) + b * s.b + h * s.h + 8 * l;
  uint8_t* cache = static_cast<uint8_t*>(isk ? p.kc : p.vc);
  uint8_t* scales = isk ? p.ks : p.vs;
  constexpr int EB = FMT == kCacheBf16 ? 2 : 1;  // bytes per stored element
  if (n0 - lane / LPR >= count) return;          // no token of this warp exists

  long long row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) row[u] = cache_row(p, b, h, n0 + u * RPW, start, count);
  if (WRITE) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[u] = n0 + u * RPW < count ? *reinterpret_cast<const uint4*>(x0 + (n0 + u * RPW) * s.n)
                                  : make_uint4(0, 0, 0, 0);  // does not wait for the page
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (FMT == kCacheBf16) {
        if (row[u] >= 0) *reinterpret_cast<uint4*>(cache + (row[u] * D + 8 * l) * EB) = x[u];
        continue;
      }
      uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      // |x| as bf16 bits orders like an integer, NaN above infinity
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t byte = row_scale<FMT>(m);
      uint2 y = make_uint2(0, 0);
      if (byte != kScaleNan) {
        const float f = inverse_scale(byte);
        // bf16's largest number is 127.5 steps of int8's largest scale
        if (FMT == kCacheInt8 && m == 0x7F7Fu)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = __vminu2(w[i] & 0x7FFF7FFFu, 0x7F7E7F7Eu) | (w[i] & 0x80008000u);
        y.x = quantise4<FMT>(bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1]), f);
        y.y = quantise4<FMT>(bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3]), f);
      } else {
        // any number times the NaN scale is NaN; a one keeps the byte a number
        y = make_uint2(0x01010101u, 0x01010101u);
      }
      if (row[u] >= 0) {
        *reinterpret_cast<uint2*>(cache + row[u] * D + 8 * l) = y;
        if (l == 0) scales[row[u]] = static_cast<uint8_t>(byte);
      }
    }
  } else {
    uint4 y[U];
    uint32_t byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      y[u] = make_uint4(0, 0, 0, 0);
      byte[u] = 127;
      if (row[u] >= 0) {
        if (FMT == kCacheBf16) {
          y[u] = *reinterpret_cast<const uint4*>(cache + (row[u] * D + 8 * l) * EB);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(cache + row[u] * D + 8 * l);
          y[u].x = w.x;
          y[u].y = w.y;
          byte[u] = scales[row[u]];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (FMT != kCacheBf16) {
        const RowScale sc = widen_scale<FMT>(byte[u]);
        const uint2 w = make_uint2(y[u].x, y[u].y);
        widen4<FMT>(w.x, sc, y[u].x, y[u].y);
        widen4<FMT>(w.y, sc, y[u].z, y[u].w);
      }
      // a position that no page holds reads as zeros
      if (n0 + u * RPW < count) *reinterpret_cast<uint4*>(x0 + (n0 + u * RPW) * s.n) = y[u];
    }
  }
}

template <int D, int FMT, bool WRITE>
cudaError_t launch_cache(const CacheParams& p, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 8);
  // Up to 8 RPW tokens (a decode step, a tree): one block per (sequence, k or
  // v, head), one row per lane.  More: blocks of 4 warps of eight rows in
  // flight per lane (16 x 4096 tokens, int8, append and read, before the
  // rounding by addition: 59.7 us; 8 warps 62.0, 2 warps 60.7, four rows per
  // lane 65.7).
  const bool wide = p.N > 8 * RPW;
  const int warps = wide ? 4 : (p.N + RPW - 1) / RPW, per = warps * RPW * (wide ? 8 : 1);
  const long long blocks = static_cast<long long>(p.B) * 2 * p.Hkv * ((p.N - 1) / per + 1);
  if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(warps * 32);
  return wide ? launch_pdl(fa_cache_kernel<D, FMT, WRITE, 8>, grid, block, 0, stream, p)
              : launch_pdl(fa_cache_kernel<D, FMT, WRITE, 1>, grid, block, 0, stream, p);
}

template <bool WRITE>
fa_status dispatch(const CacheParams& p, int format, int d, cudaStream_t stream) {
  cudaError_t e;
  if (d == 64)
    e = format == kCacheBf16   ? launch_cache<64, kCacheBf16, WRITE>(p, stream)
        : format == kCacheE4m3 ? launch_cache<64, kCacheE4m3, WRITE>(p, stream)
                               : launch_cache<64, kCacheInt8, WRITE>(p, stream);
  else
    e = format == kCacheBf16   ? launch_cache<128, kCacheBf16, WRITE>(p, stream)
        : format == kCacheE4m3 ? launch_cache<128, kCacheE4m3, WRITE>(p, stream)
                               : launch_cache<128, kCacheInt8, WRITE>(p, stream);
  FA_CUDA(e);
  return FA_OK;
}

// Everything but the pointers to rows; fills the common part of p.
fa_status cache_params(void* kc, void* vc, uint8_t* ks, uint8_t* vs, const int* page_table,
                       const int* start, const int* counts, int format, int B, int Hkv, int N,
                       int d, int num_pages, int page_size, int max_pages, CacheParams* p) {
  if (B < 1 || N < 1) return FA_ERR_INVALID_ARG;
  FA_TRY(check_cache(kc, vc, ks, vs, page_table, format, Hkv, d, num_pages, page_size, max_pages));
  FA_TRY(check_ptr4(start));
  if (counts) FA_TRY(check_ptr4(counts));
  if (static_cast<long long>(B) * Hkv > (1 << 28)) return FA_ERR_UNSUPPORTED;
  // a block takes at least two tokens of one key or value head
  if (static_cast<long long>(B) * Hkv * ((static_cast<long long>(N) + 1) / 2) >= (1LL << 30))
    return FA_ERR_UNSUPPORTED;
  p->kc = kc;
  p->vc = vc;
  p->ks = ks;
  p->vs = vs;
  p->page_table = page_table;
  p->start = start;
  p->counts = counts;
  p->B = B;
  p->Hkv = Hkv;
  p->N = N;
  p->num_pages = num_pages;
  p->log_page = log2_page(page_size);
  p->max_pages = max_pages;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_append(const void* k, const void* v, const int* page_table, const int* start,
                          const int* counts, void* k_cache, void* v_cache, uint8_t* k_scale,
                          uint8_t* v_scale, int format, int B, int Hkv, int N, int d,
                          int num_pages, int page_size, int max_pages, const long long* strides,
                          cudaStream_t stream) {
  using namespace fa;
  CacheParams p = {};
  FA_TRY(cache_params(k_cache, v_cache, k_scale, v_scale, page_table, start, counts, format, B,
                      Hkv, N, d, num_pages, page_size, max_pages, &p));
  FA_TRY(check_ptr16(k));
  FA_TRY(check_ptr16(v));
  FA_TRY(read_strides(strides, B, Hkv, N, d, &p.sk));
  FA_TRY(read_strides(strides ? strides + 3 : nullptr, B, Hkv, N, d, &p.sv));
  p.k = const_cast<void*>(k);
  p.v = const_cast<void*>(v);
  return dispatch<true>(p, format, d, stream);
}

fa_status fa_cache_read(const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                        const uint8_t* v_scale, const int* page_table, const int* start,
                        const int* counts, void* k, void* v, int format, int B, int Hkv, int N,
                        int d, int num_pages, int page_size, int max_pages, cudaStream_t stream) {
  using namespace fa;
  CacheParams p = {};
  FA_TRY(cache_params(const_cast<void*>(k_cache), const_cast<void*>(v_cache),
                      const_cast<uint8_t*>(k_scale), const_cast<uint8_t*>(v_scale), page_table,
                      start, counts, format, B, Hkv, N, d, num_pages, page_size, max_pages, &p));
  FA_TRY(check_ptr16(k));
  FA_TRY(check_ptr16(v));
  FA_TRY(read_strides(nullptr, B, Hkv, N, d, &p.sk));
  p.sv = p.sk;
  p.k = k;
  p.v = v;
  return dispatch<false>(p, format, d, stream);
}

}  // extern "C"
