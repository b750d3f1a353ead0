// Argument checks shared by the C entry points (host side).
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"

namespace fa {

// Status word of the current device (nullptr and *st on error) and the time
// limit of device-side waits (fa_api.cu).
int* status_word(fa_status* st);
unsigned long long wait_limit_ns();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline fa_status check_ptr16(const void* p) {
  if (!p) return FA_ERR_INVALID_ARG;
  if (!aligned(p, 16)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

inline fa_status check_ptr4(const void* p) {
  if (!p) return FA_ERR_INVALID_ARG;
  if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

inline fa_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return FA_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return FA_ERR_MISALIGNED;
  if (have < need) return FA_ERR_WORKSPACE;
  return FA_OK;
}

#define FA_TRY(x)                    \
  do {                               \
    const fa_status _s = (x);        \
    if (_s != FA_OK) return _s;      \
  } while (0)

#define FA_CUDA(x)                                \
  do {                                            \
    if ((x) != cudaSuccess) return FA_ERR_CUDA;   \
  } while (0)

// log2 of a cache page's positions (16, 32, 64 or 128), -1 for others
inline int log2_page(int page_size) {
  for (int l = 4; l <= 7; ++l)
    if (page_size == 1 << l) return l;
  return -1;
}

// Arguments that describe a paged key/value cache.  A row index
// (page, head, row) stays below 2^38; a sequence's positions stay below 2^30,
// so that sums of two of them, and a tile more, fit in 32 bits.
inline fa_status check_cache(const void* k_cache, const void* v_cache, const void* k_scale,
                             const void* v_scale, const void* page_table, int format, int Hkv,
                             int d, int num_pages, int page_size, int max_pages) {
  if (Hkv < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (format < FA_CACHE_BF16 || format > FA_CACHE_INT8) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (log2_page(page_size) < 0) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * Hkv >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  FA_TRY(check_ptr16(k_cache));
  FA_TRY(check_ptr16(v_cache));
  FA_TRY(check_ptr4(page_table));
  if (format != FA_CACHE_BF16) {
    FA_TRY(check_ptr16(k_scale));
    FA_TRY(check_ptr16(v_scale));
  }
  return FA_OK;
}

// Element strides (batch, head, row) of a [B, H, N, d] tensor whose d
// elements are contiguous.
struct Strides {
  long long b, h, n;
};

// `s` (three strides) or, when it is null, those of a contiguous tensor.
// Rows start on 16-byte boundaries: strides are multiples of 8 elements.
// Strides of axes of length 1 are not looked at (and not used).
inline fa_status read_strides(const long long* s, int B, int H, int N, int d, Strides* out) {
  if (!s) {
    *out = Strides{static_cast<long long>(H) * N * d, static_cast<long long>(N) * d, d};
    return FA_OK;
  }
  const int n[3] = {B, H, N};
  long long v[3];
  for (int i = 0; i < 3; ++i) {
    v[i] = n[i] > 1 ? s[i] : 0;
    if (v[i] < 0) return FA_ERR_INVALID_ARG;
    if (v[i] % 8 != 0) return FA_ERR_MISALIGNED;
    // no offset passes 2^48 elements (more than any memory holds)
    if (v[i] > 0 && n[i] - 1 > (1LL << 46) / v[i]) return FA_ERR_INVALID_ARG;
  }
  *out = Strides{v[0], v[1], v[2]};
  return FA_OK;
}

// Rows of a tensor that is written must not overlap: by ascending stride,
// each axis steps over everything the axes below it span.
inline fa_status check_disjoint(const Strides& s, int B, int H, int N, int d) {
  struct Axis {
    long long stride;
    int n;
  } a[3] = {{s.b, B}, {s.h, H}, {s.n, N}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (a[j].stride > a[j + 1].stride) {
        const Axis t = a[j];
        a[j] = a[j + 1];
        a[j + 1] = t;
      }
  long long span = d;
  for (const Axis& x : a) {
    if (x.n == 1) continue;
    if (x.stride < span) return FA_ERR_INVALID_ARG;
    span += x.stride * (x.n - 1);
  }
  return FA_OK;
}

}  // namespace fa
