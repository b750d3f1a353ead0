// What the tree attention kernels share: the arguments, the lengths of the
// sequences, the split of the work into runs, and which keys a draft sees.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_quant.cuh"

namespace fa {

// CTAs, at most (the workspace holds two parts of each); up to 8 rows twice
// as many
constexpr int kMaxGrid = 192;

struct TreeParams {
  const void* q;           // bf16 [B, H, T, d]
  const void *kc, *vc;     // caches [num_pages, Hkv, page, d]
  const uint8_t *ks, *vs;  // scale bytes [num_pages, Hkv, page]
  const int *page_table, *hist, *drafts;
  const uint32_t* mask;    // [B, T, words] or null
  void* o;                 // bf16 [B, H, T, d]
  float* lse;              // [B, H, T]
  // Parts of problems that several CTAs work on.  CTA c has two places: 2 c
  // for the part that begins its run inside a problem, 2 c + 1 for the one
  // that ends it inside a problem begun there.
  float2* part_ml;         // [2 * grid][slot_rows] (max in log2 units, sum)
  float* part_o;           // [2 * grid][slot_rows][d]
  int2* joins;             // [grid] the problem begun and not ended by CTA c
                           // ((b * Hkv + head) * groups + group) and its parts, or 0 parts
  int B, Hkv, T, rows;     // rows = H / Hkv * T
  int groups, slot_rows;   // row groups per key/value head; rows of a part
  int pair;                // 256-row groups
  int num_pages, log_page, max_pages, words;
  float scale;
  int* err;
  uint64_t wait_ns;
};

// Lengths of a sequence, clamped to what the page table can hold.
struct SeqLen {
  int hist, nd, tiles;
  FA_DEV int len() const { return hist + nd; }
};
FA_DEV SeqLen seq_len(const TreeParams& p, int b) {
  SeqLen s;
  const int cap = p.max_pages << p.log_page;
  s.hist = min(max(p.hist[b], 0), cap);
  s.nd = min(p.drafts ? min(max(p.drafts[b], 0), p.T) : p.T, cap - s.hist);
  // one unit even without a key: somebody has to write the rows
  s.tiles = max(1, (s.len() + kTile - 1) / kTile);
  return s;
}

// Units of sequence b: its tiles for each key/value head and row group.  All
// sequences together have less than 2^31 (checked on the host).
FA_DEV uint32_t seq_units(const TreeParams& p, int b) {
  return b < p.B ? static_cast<uint32_t>(seq_len(p, b).tiles) * (p.Hkv * p.groups) : 0u;
}

// A CTA's run of units.
struct Run {
  int b, hr, t;         // first unit: sequence, key/value head x group, tile
  uint32_t first, left; // its number, units
  uint32_t total;       // units of all sequences
  int n;                // CTAs that have some
};

// First unit of CTA c of n: floor(total c / n).
FA_DEV uint32_t run_begin(uint32_t total, uint32_t c, uint32_t n) {
  const uint32_t q = total / n, r = total - q * n;
  return q * c + r * c / n;
}

// Run of CTA c: with n = the grid's CTAs, or the units if there are fewer (no
// run between two others is empty).  Whole warp.
FA_DEV Run find_run(const TreeParams& p, int c, int grid, int lane) {
  const uint32_t mine = seq_units(p, lane);  // the first 32 sequences
  uint32_t total = __reduce_add_sync(0xffffffffu, mine);
  for (int b0 = 32; b0 < p.B; b0 += 32)
    total += __reduce_add_sync(0xffffffffu, seq_units(p, b0 + lane));
  const int n = total < static_cast<uint32_t>(grid) ? static_cast<int>(total) : grid;
  Run r = {0, 0, 0, 0, 0, total, n};
  if (c >= n) return r;
  r.first = run_begin(total, c, n);
  r.left = run_begin(total, c + 1, n) - r.first;
  uint32_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const uint32_t u = b0 == 0 ? mine : seq_units(p, b0 + lane);
    uint32_t incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > r.first);
    if (hit) {
      const int w = __ffs(hit) - 1;
      const uint32_t rem = __shfl_sync(0xffffffffu, r.first - (base + incl - u), w);
      const uint32_t tiles = __shfl_sync(0xffffffffu, u, w) / (p.Hkv * p.groups);
      r.b = b0 + w;
      r.hr = static_cast<int>(rem / tiles);
      r.t = static_cast<int>(rem - r.hr * tiles);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// The parts of problems in a run, in order; every role of the CTA walks it.
struct PartIter {
  SeqLen s;
  int b, hr, t0, t1;  // tiles [t0, t1) of problem (b, hr)
  int next_t;
  uint32_t left;
  FA_DEV void init(const TreeParams& p, const Run& r) {
    b = r.b;
    hr = r.hr;
    next_t = r.t;
    left = r.left;
    s = seq_len(p, b);
  }
  FA_DEV bool next(const TreeParams& p) {
    if (left == 0) return false;
    if (next_t == s.tiles) {
      next_t = 0;
      if (++hr == p.Hkv * p.groups) {
        hr = 0;
        ++b;
        s = seq_len(p, b);
      }
    }
    t0 = next_t;
    const int n = min(left, static_cast<uint32_t>(s.tiles - t0));
    t1 = next_t = t0 + n;
    left -= n;
    return true;
  }
};

// The problem that this CTA begins and does not end, for the second kernel;
// `it` after the last part of the run (one thread; idle CTAs too, with no
// part).
FA_DEV void note_join(const TreeParams& p, const Run& r, const PartIter& it, int c) {
  int2 j = make_int2(0, 0);
  if (r.left > 0 && it.t0 == 0 && it.t1 < it.s.tiles) {
    // unit u belongs to CTA floor(((u + 1) n - 1) / total)
    const uint64_t last = static_cast<uint64_t>(r.first) + r.left + (it.s.tiles - it.t1) - 1;
    const int c1 = static_cast<int>(((last + 1) * r.n - 1) / r.total);
    j = make_int2(it.b * p.Hkv * p.groups + it.hr, c1 - c + 1);
  }
  p.joins[c] = j;
}

// The tiles of a run, in order.
struct TileIter {
  PartIter it;
  int t = 0, part = -1;
  bool first = false, last = false;
  FA_DEV bool next(const TreeParams& p) {
    first = part < 0 || t + 1 >= it.t1;
    if (first) {
      if (!it.next(p)) return false;
      ++part;
      t = it.t0;
    } else {
      ++t;
    }
    last = t + 1 == it.t1;
    return true;
  }
};

// bits 0 .. n-1
FA_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Which of the 32 keys from position `pos` on draft t of a sequence sees.
FA_DEV uint32_t seen_bits(const TreeParams& p, const uint32_t* mask_row, const SeqLen& s, int t,
                          int pos) {
  const int d0 = pos - s.hist;  // draft index of bit 0
  uint32_t w;
  if (!mask_row) {
    w = low_bits(t + 1 - d0);
  } else if (d0 >= 0) {
    const int i = d0 >> 5;
    w = __funnelshift_r(i < p.words ? mask_row[i] : 0u, i + 1 < p.words ? mask_row[i + 1] : 0u,
                        d0 & 31);
  } else {
    w = d0 > -32 ? mask_row[0] << -d0 : 0u;
  }
  return (w & low_bits(s.nd - d0)) | low_bits(-d0);
}

FA_DEV uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
FA_DEV uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// untiled bulk copy (16-byte aligned, a multiple of 16 bytes)
FA_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// a NaN or an infinity in a packed bf16 pair
FA_DEV bool not_finite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
// the pair with NaN and infinities replaced by zero
FA_DEV uint32_t finite2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

// Adds the NaN and infinite values among the drafts of positions [lo, hi)
// that draft t sees to its written row of O (they were zeroed in the tiles):
// `o` (bf16) or `part` (fp32).  Rare.
template <int D, int FMT>
static __device__ __noinline__ void add_not_finite(const TreeParams& p, int b, int hkv, SeqLen s, int t,
                                            int lo, int hi, uint16_t* o, float* part) {
  const uint32_t* mr = p.mask ? p.mask + (static_cast<size_t>(b) * p.T + t) * p.words : nullptr;
  for (int pos = lo; pos < hi; ++pos) {
    if (!(seen_bits(p, mr, s, t, pos) & 1u)) continue;
    int page = p.page_table[static_cast<size_t>(b) * p.max_pages + (pos >> p.log_page)];
    page = min(max(page, 0), p.num_pages - 1);
    const long long row = ((static_cast<long long>(page) * p.Hkv + hkv) << p.log_page) +
                          (pos & ((1 << p.log_page) - 1));
    if (FMT != kCacheBf16 && p.vs[row] != kScaleNan) continue;
    for (int j = 0; j < D; ++j) {
      const float v = FMT != kCacheBf16
                          ? __uint_as_float(0x7FFFFFFFu)
                          : __uint_as_float(static_cast<uint32_t>(
                                                static_cast<const uint16_t*>(p.vc)[row * D + j])
                                            << 16);
      if (isfinite(v)) continue;
      if (part)
        part[j] += v;
      else
        o[j] = static_cast<uint16_t>(
            pack_bf16(__uint_as_float(static_cast<uint32_t>(o[j]) << 16) + v, 0.f) & 0xFFFFu);
    }
  }
}

// Few query rows per key/value head: fa_tree_few.cu (warp MMAs) up to 16 rows
// for bf16 and up to 24 for 8 bits, else fa_tree.cu.  The rule sees sizes,
// not the lengths of the histories, which are on the device.  us by
// fa_tree_few.cu | fa_tree.cu, 4 key/value heads, sequences x keys:
//   d = 128           16 x 8192      256 x 500      1024 x 120     1 x 512
//   bf16   9 rows   53.8 | 54.4    79.8 | 83.4    191 | 226    11.0 | 12.9
//         12        54.7 | 54.5    86.5 | 80.1    218 | 227    11.3 | 12.7
//         16        55.1 | 55.0    89.1 | 101     221 | 227    11.5 | 12.7
//   e4m3  16        47.1 | 68.0    89.6 | 139     226 | 248    12.2 | 12.1
//         24        59.2 | 68.6     115 | 140     301 | 254    13.8 | 12.4
//   int8  16        51.0 | 69.5    94.4 | 142     231 | 251    12.3 | 12.1
//         24        63.6 | 70.2     120 | 142     309 | 256    14.0 | 12.4
//   d = 64
//   bf16  16        33.5 | 37.5    59.7 | 92.5    141 | 176     9.2 | 10.7
//   e4m3  24        43.5 | 54.1    80.0 | 114     205 | 220    11.3 | 10.7
//   int8  24        45.6 | 55.9    82.6 | 116     207 | 219    11.4 | 10.7
// At the rule's edge the two are equal for long histories of bf16, d = 128,
// and 17 to 24 rows of 8 bits gain on long histories and lose on short ones
// (a tile each, or one sequence alone).  Beyond it (16 x 8192 keys): bf16, d = 128, 24 rows 73.2 |
// 56.8; e4m3 32 rows 149 | 69.6; int8 157 | 71.0; d = 64 bf16 24 rows 50.8 |
// 40.0; e4m3 32 rows 55.6 | 55.6.
// tk, tv: maps of whole pages (make_cache_map).
inline bool tree_few_rows(int rows, int format) { return rows <= (format == kCacheBf16 ? 16 : 24); }
// CTAs of it on an SM: two up to 8 rows, but for bf16 of d = 128, whose ring
// takes the whole shared memory.  Two (8 warps each) | one (16 warps), e4m3,
// 4 rows of 4 heads of 128, us: 4096 sequences of 60 keys 288 | 453, 256 of
// 500 keys 47.7 | 55.4, 32 of up to 8192 keys 40.8 | 41.1, of 8191 keys each
// 54.0 | 53.3.
constexpr int few_ctas(int rows, int format, int d) {
  return rows <= 8 && (format != kCacheBf16 || d == 64) ? 2 : 1;
}
cudaError_t launch_tree_few(const TreeParams& p, int format, int d, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream);

}  // namespace fa
