// Attention of drafted tokens over a paged key/value cache.
//
// Sequence b has hist_lens[b] accepted tokens and draft_lens[b] <= T drafted
// ones whose keys and values stand behind them in the cache.  Draft i sees
// every accepted token and the drafts whose bit is set in its mask row (its
// ancestors and itself in a tree; all drafts up to itself without a mask):
//   o_i = sum_j p_ij v_j,  p_i = softmax over the seen j of scale q_i k_j.
//
// One warp per (sequence, head, draft): the query row lives in registers
// (D / 32 elements per lane), keys are taken one by one with a running max
// and sum.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_quant.cuh"

namespace fa {
namespace {

struct TreeParams {
  const void* q;                 // bf16 [B, H, T, d]
  const void *kc, *vc;           // caches [num_pages, Hkv, page, d]
  const uint8_t *ks, *vs;        // scale bytes [num_pages, Hkv, page]
  const int *page_table, *hist, *drafts;
  const uint32_t* mask;          // [B, T, words] or null
  void* o;                       // bf16 [B, H, T, d]
  float* lse;                    // [B, H, T]
  int B, H, Hkv, T, num_pages, log_page, max_pages, words;
  float scale;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// D / 32 elements of a cache row as fp32
template <int D, int FMT>
FA_DEV void cache_elements(const void* cache, const uint8_t* scales, long long row, int lane,
                           float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if (FMT == kCacheBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(cache) + row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(cache) + row * D + lane * E;
    uint32_t w = 0, lo, hi;
#pragma unroll
    for (int i = 0; i < E; ++i) w |= static_cast<uint32_t>(p[i]) << (8 * i);
    widen4<FMT>(w, widen_scale<FMT>(scales[row]), lo, hi);
    x[0] = bf16_lo(lo);
    x[1] = bf16_hi(lo);
    if (E == 4) {
      x[E - 2] = bf16_lo(hi);
      x[E - 1] = bf16_hi(hi);
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(128) fa_tree_kernel(const TreeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= static_cast<long long>(p.B) * p.H * p.T) return;
  const int t = static_cast<int>(r % p.T), h = static_cast<int>(r / p.T % p.H),
            b = static_cast<int>(r / p.T / p.H), hkv = h / (p.H / p.Hkv);
  const int cap = p.max_pages << p.log_page;
  const int hist = min(max(p.hist[b], 0), cap);
  const int nd = min(p.drafts ? min(max(p.drafts[b], 0), p.T) : p.T, cap - hist);
  float q[E], o[E], x[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __uint_as_float(
        static_cast<uint32_t>(static_cast<const uint16_t*>(p.q)[r * D + lane * E + i]) << 16);
    o[i] = 0.f;
  }
  for (int j = 0; t < nd && j < hist + nd; ++j) {
    if (j >= hist) {
      const int i = j - hist;
      const bool seen =
          p.mask ? (p.mask[(static_cast<size_t>(b) * p.T + t) * p.words + i / 32] >> (i % 32)) & 1u
                 : i <= t;
      if (!seen) continue;
    }
    int page = p.page_table[static_cast<size_t>(b) * p.max_pages + (j >> p.log_page)];
    page = min(max(page, 0), p.num_pages - 1);
    const long long row = ((static_cast<long long>(page) * p.Hkv + hkv) << p.log_page) +
                          (j & ((1 << p.log_page) - 1));
    cache_elements<D, FMT>(p.kc, p.ks, row, lane, x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.scale * kLog2e;
    const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
    const float a = ex2(m - mu), e = ex2(s - mu);
    cache_elements<D, FMT>(p.vc, p.vs, row, lane, x);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(e, x[i], o[i] * a);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is 0
  uint16_t* out = static_cast<uint16_t*>(p.o) + r * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) = pack_bf16(o[i] * inv, o[i + 1] * inv);
  if (lane == 0) p.lse[r] = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
}

template <int D, int FMT>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.T;
  return launch_pdl(fa_tree_kernel<D, FMT>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128),
                    0, stream, p);
}

size_t tree_ws_bytes(int B, int H, int Hkv, int T, int d) { return 256; }

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_tree_attention_workspace_size(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || T < 1 || d < 1) return 0;
  return fa::tree_ws_bytes(B, H, Hkv, T, d);
}

fa_status fa_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                            const uint8_t* k_scale, const uint8_t* v_scale, const int* page_table,
                            const int* hist_lens, const int* draft_lens, const uint32_t* tree_mask,
                            void* o, float* lse, int format, int B, int H, int Hkv, int T, int d,
                            int num_pages, int page_size, int max_pages, float scale,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace fa;
  if (B < 1 || H < 1 || T < 1) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || Hkv > H || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  FA_TRY(check_cache(k_cache, v_cache, k_scale, v_scale, page_table, format, Hkv, d, num_pages,
                     page_size, max_pages));
  if (T > 1024 || static_cast<long long>(B) * H * T * d >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  FA_TRY(check_ptr16(q));
  FA_TRY(check_ptr16(o));
  FA_TRY(check_ptr4(lse));
  FA_TRY(check_ptr4(hist_lens));
  if (draft_lens) FA_TRY(check_ptr4(draft_lens));
  if (tree_mask) FA_TRY(check_ptr4(tree_mask));
  FA_TRY(check_ws(workspace, workspace_bytes, tree_ws_bytes(B, H, Hkv, T, d)));
  TreeParams p = {};
  p.q = q;
  p.kc = k_cache;
  p.vc = v_cache;
  p.ks = k_scale;
  p.vs = v_scale;
  p.page_table = page_table;
  p.hist = hist_lens;
  p.drafts = draft_lens;
  p.mask = tree_mask;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.T = T;
  p.num_pages = num_pages;
  p.log_page = log2_page(page_size);
  p.max_pages = max_pages;
  p.words = (T + 31) / 32;
  p.scale = scale;
  if (d == 64)
    FA_CUDA(format == kCacheBf16   ? (launch_tree<64, kCacheBf16>(p, stream))
            : format == kCacheE4m3 ? (launch_tree<64, kCacheE4m3>(p, stream))
                                   : (launch_tree<64, kCacheInt8>(p, stream)));
  else
    FA_CUDA(format == kCacheBf16   ? (launch_tree<128, kCacheBf16>(p, stream))
            : format == kCacheE4m3 ? (launch_tree<128, kCacheE4m3>(p, stream))
                                   : (launch_tree<128, kCacheInt8>(p, stream)));
  return FA_OK;
}

}  // extern "C"
