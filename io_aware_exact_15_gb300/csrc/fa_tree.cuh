// What the tree attention kernels share: the lengths of the sequences, the split of the work into runs, and which keys a draft sees.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_quant.cuh"
#include "fa_tree_host.h"

namespace fa {

// Lengths of a sequence, clamped to what the page table can hold.
//
// WIN: a draft with c drafts before it on its path sees the positions below
// `sinks` and those from hist + c - window + 1 on (of the drafts those that
// its mask row or the chain's order has).  So positions fall into three
// classes: those that every draft sees (below `sinks`, or in [edge, hist)),
// those that none sees (in [sinks, lo), and past the end), and those that are
// a matter of the draft.  Tiles of which no draft sees anything are left out:
// the t-th of a sequence's tiles is the t-th of the table before `sunk`, the
// (t + skip)-th from there on.
template <bool WIN>
struct SeqLen {
  int hist, nd, tiles;
  FA_DEV int len() const { return hist + nd; }
  FA_DEV int key_tile(int t) const { return t; }
  FA_DEV bool nobody(int pos) const { return pos >= len(); }
  FA_DEV bool everybody(int pos) const { return pos < hist; }
  // whether n positions from pos on are not all everybody's, and are all nobody's
  FA_DEV bool mixed(int pos, int n) const { return pos + n > hist; }
  FA_DEV bool nothing(int pos, int) const { return pos >= len(); }
};
template <>
struct SeqLen<true> {
  int hist, nd, tiles;
  int sinks, lo, edge, sunk, skip;
  FA_DEV int len() const { return hist + nd; }
  FA_DEV int key_tile(int t) const { return t >= sunk ? t + skip : t; }
  FA_DEV bool nobody(int pos) const { return pos >= len() || (pos >= sinks && pos < lo); }
  FA_DEV bool everybody(int pos) const { return pos < hist && (pos < sinks || pos >= edge); }
  FA_DEV bool mixed(int pos, int n) const {
    return pos + n > hist || (pos < edge && pos + n > sinks);
  }
  FA_DEV bool nothing(int pos, int n) const {
    return pos >= len() || (pos >= sinks && pos + n <= lo);
  }
};
template <bool WIN>
FA_DEV SeqLen<WIN> seq_len(const TreeParams& p, int b) {
  SeqLen<WIN> s;
  const int cap = p.max_pages << p.log_page;
  s.hist = min(max(p.hist[b], 0), cap);
  s.nd = min(p.drafts ? min(max(p.drafts[b], 0), p.T) : p.T, cap - s.hist);
  int tiles = (s.len() + kTile - 1) / kTile;
  if constexpr (WIN) {
    s.sinks = p.sinks;
    s.lo = max(s.hist - p.window + 1, 0);
    s.edge = max(s.hist - p.window + max(s.nd, 1), 0);
    s.sunk = min((min(p.sinks, s.len()) + kTile - 1) / kTile, s.lo / kTile);
    s.skip = s.lo / kTile - s.sunk;
    tiles -= min(s.skip, tiles);
  }
  // one unit even without a key: somebody has to write the rows
  s.tiles = max(1, tiles);
  return s;
}

// Units of sequence b: its tiles for each key/value head and row group.  All
// sequences together have less than 2^31 (checked on the host).
template <bool WIN>
FA_DEV uint32_t seq_units(const TreeParams& p, int b) {
  return b < p.B ? static_cast<uint32_t>(seq_len<WIN>(p, b).tiles) * (p.Hkv * p.groups) : 0u;
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
template <bool WIN>
FA_DEV Run find_run(const TreeParams& p, int c, int grid, int lane) {
  if (WIN && p.whole) {  // an equal number of problems each
    const uint32_t per_b = p.Hkv * p.groups, problems = p.B * per_b;
    const uint32_t n = min(problems, static_cast<uint32_t>(grid));
    Run r = {0, 0, 0, 0, 0, 0, static_cast<int>(n)};
    if (c >= static_cast<int>(n)) return r;
    const uint32_t p0 = run_begin(problems, c, n), p1 = run_begin(problems, c + 1, n);
    r.b = p0 / per_b;
    r.hr = p0 - r.b * per_b;
    for (uint32_t i = p0; i < p1; i += 32)
      r.left += __reduce_add_sync(
          0xffffffffu, i + lane < p1 ? seq_len<WIN>(p, (i + lane) / per_b).tiles : 0);
    return r;
  }
  if (WIN && p.cluster) {  // CTA c: its share of the tiles of problem c / cluster
    const int problem = c / p.cluster, i = c - problem * p.cluster;
    Run r = {problem / (p.Hkv * p.groups), 0, 0, 0, 0, 0, grid};
    r.hr = problem - r.b * (p.Hkv * p.groups);
    const int tiles = seq_len<WIN>(p, r.b).tiles;
    r.t = tiles * i / p.cluster;
    r.left = tiles * (i + 1) / p.cluster - r.t;
    return r;
  }
  const uint32_t mine = seq_units<WIN>(p, lane);  // the first 32 sequences
  uint32_t total = __reduce_add_sync(0xffffffffu, mine);
  for (int b0 = 32; b0 < p.B; b0 += 32)
    total += __reduce_add_sync(0xffffffffu, seq_units<WIN>(p, b0 + lane));
  const int n = total < static_cast<uint32_t>(grid) ? static_cast<int>(total) : grid;
  Run r = {0, 0, 0, 0, 0, total, n};
  if (c >= n) return r;
  r.first = run_begin(total, c, n);
  r.left = run_begin(total, c + 1, n) - r.first;
  uint32_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const uint32_t u = b0 == 0 ? mine : seq_units<WIN>(p, b0 + lane);
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
template <bool WIN>
struct PartIter {
  SeqLen<WIN> s;
  int b, hr, t0, t1;  // tiles [t0, t1) of problem (b, hr)
  int next_t;
  uint32_t left;
  FA_DEV void init(const TreeParams& p, const Run& r) {
    b = r.b;
    hr = r.hr;
    next_t = r.t;
    left = r.left;
    s = seq_len<WIN>(p, b);
  }
  FA_DEV bool next(const TreeParams& p) {
    if (left == 0) return false;
    if (next_t == s.tiles) {
      next_t = 0;
      if (++hr == p.Hkv * p.groups) {
        hr = 0;
        ++b;
        s = seq_len<WIN>(p, b);
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
template <bool WIN>
FA_DEV void note_join(const TreeParams& p, const Run& r, const PartIter<WIN>& it, int c) {
  int2 j = make_int2(0, 0);
  if (r.left > 0 && it.t0 == 0 && it.t1 < it.s.tiles) {
    // unit u belongs to CTA floor(((u + 1) n - 1) / total)
    const uint64_t last = static_cast<uint64_t>(r.first) + r.left + (it.s.tiles - it.t1) - 1;
    const int c1 = static_cast<int>(((last + 1) * r.n - 1) / r.total);
    j = make_int2(it.b * p.Hkv * p.groups + it.hr, c1 - c + 1);
  }
  p.joins[c] = j;
}

// Row `row` of problem bh from its n <= 8 parts, whose rows in part_ml and
// part_o `at` says (fa_tree_join_kernel's sum).  Whole warp.  The parts are of
// other SMs of the cluster: L1 may hold what stood there before.
template <int D, class At>
FA_DEV void join_row(const TreeParams& p, int bh, int row, int n, const At& at, int lane) {
  constexpr int E = D / 32;
  float v[8][E];
#pragma unroll
  for (int k = 0; k < 8; ++k) {  // all on their way together
    const float* y = p.part_o + at(min(k, n - 1)) * D + lane * E;
    if (E == 4)
      *reinterpret_cast<float4*>(v[k]) = __ldcg(reinterpret_cast<const float4*>(y));
    else
      *reinterpret_cast<float2*>(v[k]) = __ldcg(reinterpret_cast<const float2*>(y));
  }
  const float2 x = lane < n ? __ldcg(p.part_ml + at(lane)) : make_float2(-INFINITY, 0.f);
  float M = x.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  // a part in which the row saw nothing counts nothing, whatever it holds
  const float a = x.y == 0.f ? 0.f : ex2(x.x - (M == -INFINITY ? 0.f : M));
  const uint32_t use = __ballot_sync(0xffffffffu, x.y != 0.f);
  float l = x.y * a, o[E];
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float ak = __shfl_sync(0xffffffffu, a, k);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (use >> k) & 1u ? fmaf(v[k][e], ak, o[e]) : o[e];
  }
  const bool has = !(l == 0.f);
  const float inv = has ? 1.f / l : 0.f;
  const size_t gr = static_cast<size_t>(bh) * p.rows + row;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + gr * D + lane * E);
#pragma unroll
  for (int i = 0; i < E; i += 2) dst[i / 2] = has ? pack_bf16(o[i] * inv, o[i + 1] * inv) : 0u;
  if (lane == 0) p.lse[gr] = has ? (M + lg2(l)) * 0.6931471805599453f : -INFINITY;
}

// The tiles of a run, in order.
template <bool WIN>
struct TileIter {
  PartIter<WIN> it;
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

// The first position of draft t's window: behind the drafts that it sees
// beside itself.
FA_DEV int window_begin(const TreeParams& p, const uint32_t* mask_row, const SeqLen<true>& s,
                        int t) {
  int c = t;
  if (mask_row) {
    c = 0;
    for (int i = 0; i < p.words; ++i) {
      uint32_t w = mask_row[i] & low_bits(s.nd - 32 * i);
      if (i == t >> 5) w &= ~(1u << (t & 31));
      c += __popc(w);
    }
  }
  return s.hist + c - p.window + 1;
}

// Which of the 32 keys from position `pos` on draft t of a sequence sees; its
// window begins at `begin` (WIN).  (A mask goes with windows no shorter than
// the drafts: `begin` is then at most hist, and cuts no draft off.)
template <bool WIN>
FA_DEV uint32_t seen_bits(const TreeParams& p, const uint32_t* mask_row, const SeqLen<WIN>& s,
                          int t, int pos, int begin) {
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
  w = (w & low_bits(s.nd - d0)) | low_bits(-d0);
  if constexpr (WIN) w &= ~low_bits(begin - pos) | low_bits(s.sinks - pos);
  return w;
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

// Adds the NaN and infinite values among the positions of tiles [t0, t1) that
// not every draft sees and draft t does to its written row of O (they were
// zeroed in the tiles): `o` (bf16) or `part` (fp32).  Rare.
template <int D, int FMT, bool WIN>
static __device__ __noinline__ void add_not_finite(const TreeParams& p, int b, int hkv,
                                                   SeqLen<WIN> s, int t, int t0, int t1,
                                                   uint16_t* o, float* part) {
  const uint32_t* mr = p.mask ? p.mask + (static_cast<size_t>(b) * p.T + t) * p.words : nullptr;
  int begin = 0;
  if constexpr (WIN) begin = window_begin(p, mr, s, t);
  const int first = WIN ? t0 * kTile : max(s.hist, t0 * kTile);
  for (int at = first; at < (WIN ? t1 * kTile : min(s.len(), t1 * kTile)); ++at) {
    const int pos = s.key_tile(at / kTile) * kTile + at % kTile;
    if (WIN && (s.everybody(pos) || s.nobody(pos))) continue;
    if (!(seen_bits<WIN>(p, mr, s, t, pos, begin) & 1u)) continue;
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

// tk, tv: maps of whole pages (make_cache_map).
// (with p.window: the kernels with a window)
cudaError_t launch_tree_few(const TreeParams& p, int format, int d, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream);

}  // namespace fa
