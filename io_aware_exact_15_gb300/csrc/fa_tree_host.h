// Tree attention on the host: the arguments, and how the work is cut and which
// kernel takes it, by sizes alone.
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {

// CTAs, at most (the workspace holds two parts of each); up to 8 rows twice
// as many
constexpr int kMaxGrid = 192;
inline int most_ctas(int rows) { return rows <= 8 ? 2 * kMaxGrid : kMaxGrid; }

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
  int whole;               // (windows) CTAs take whole problems: nothing to join
  int cluster;             // (windows, few rows) CTAs of a cluster share a problem and join it
  int num_pages, log_page, max_pages, words;
  int window, sinks;       // kernels with a window: at least 1, at least 0
  float scale;
  int* err;
  uint64_t wait_ns;
};

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
inline bool tree_few_rows(int rows, int format) {
  return rows <= (format == FA_CACHE_BF16 ? 16 : 24);
}
// CTAs of it on an SM: two up to 8 rows, but for bf16 of d = 128, whose ring
// takes the whole shared memory.  Two (8 warps each) | one (16 warps), e4m3,
// 4 rows of 4 heads of 128, us: 4096 sequences of 60 keys 288 | 453, 256 of
// 500 keys 47.7 | 55.4, 32 of up to 8192 keys 40.8 | 41.1, of 8191 keys each
// 54.0 | 53.3.
constexpr int few_ctas(int rows, int format, int d) {
  return rows <= 8 && (format != FA_CACHE_BF16 || d == 64) ? 2 : 1;
}

// Tiles of the longest sequence that the page table can hold (with a window:
// the sinks', and those that window + T - 1 positions can touch).
inline long long most_tiles(const TreeParams& p) {
  const long long all = ((static_cast<long long>(p.max_pages) << p.log_page) + kTile - 1) / kTile;
  if (!p.window) return all;
  const long long near = (static_cast<long long>(p.window) + p.T + kTile - 3) / kTile + 1 +
                         (p.sinks + kTile - 1) / kTile;
  return near < all ? near : all;
}

// CTAs: one for each of `places` (SMs times the CTAs that fit on one), no more
// than there can be units (0 without a device).
inline int tree_grid(const TreeParams& p, int places) {
  if (p.cluster) return p.B * p.Hkv * p.cluster;
  const long long most = static_cast<long long>(p.B) * p.Hkv * p.groups * most_tiles(p);
  const int grid = places < most_ctas(p.rows) ? places : most_ctas(p.rows);
  return most < grid ? static_cast<int>(most) : grid;
}

// Windows make problems of about the same length, known to the host, so CTAs
// can take whole ones: no parts to store, no second kernel, and no CTA reads
// the lengths of others' sequences.  That leaves SMs idle when there are fewer
// problems than SMs, or a last round of them.  It is done where the estimates
// say so: us per tile, and what cutting costs beside it (4 where each CTA has
// one tile at most, else 10, 24 with 256-row groups, whose parts are 128 KB).
// With more than 128 rows, whole problems are 128-row groups if the SMs have
// one each.  A third way, for few rows and fewer problems than SMs: 2, 4 or 8
// CTAs of a cluster share a problem and join its parts themselves behind a
// cluster barrier (2 us), where a second kernel takes 4 at least.  (8 CTAs that
// have an SM each leave SMs of a GPC idle: only for a quarter of the SMs.)
// cut or whole, the better | shared, us, 1 token, 4 key/value heads:
//   d = 128, bf16  x 1, window 512 13.2 | 10.4; x 8, 512 19.0 | 12.0, 4096 31.6 |
//   21.0; x 16, 4096 38.0 | 29.4; e4m3 x 1, 512 10.5 | 8.4; x 16, 1024 14.3 | 11.2
//   d = 64, bf16  x 1, 512 10.7 | 8.3; x 8, 4096 19.4 | 15.9; e4m3 x 8, 4096
//   13.9 | 12.5; (4 rows a token: bf16, d = 128, x 8, 512 22.6 | 15.9)
// cut | whole, us, 4 key/value heads of 128 but for drafts:
//   1 token x 16 sequences, bf16, window 128 27.3 | 17.0, 1024 33.4 | 27.3
//   1 token x 1, bf16, window 128 19.1 | 15.0, 512 19.1 | 21.1
//   1 token x 64, e4m3, window 4096 70.3 | 66.2
//   23 drafts, 12 heads of 64, x 8, window 1024 31.4 | 23.2, x 16 45.7 | 39.6
//   92 rows, bf16, x 32, window 1024 49.8 | 35.5; e4m3 55.9 | 37.5
//   256 rows, bf16, x 16, window 1024 51.8 | 33.4, x 4, 4096 45.7 | 51.8
//   256 rows, int8, x 16, window 1024 53.9 | 37.5, 4096 82.6 | 86.7
// On any device there are no more CTAs than the workspace has parts for.
inline void split_window(TreeParams* p, int format, int d, int device_sms) {
  const bool few = tree_few_rows(p->rows, format);
  const int places = device_sms * (few ? few_ctas(p->rows, format, d) : 1);
  const int sms = places < most_ctas(p->rows) ? places : most_ctas(p->rows);
  if (sms <= 0) return;
  const double us = few                       ? 0.9
                    : format != FA_CACHE_BF16 ? (d == 64 ? 1.1 : 2.0)
                                              : (d == 64 ? 0.7 : 1.2);
  const double mt = static_cast<double>(most_tiles(*p));
  const double bh = static_cast<double>(p->B) * p->Hkv;
  const double units = bh * p->groups * mt;  // if cut
  const double per_cta = units / sms > 1 ? units / sms : 1;
  const double cut = per_cta * us * (p->pair ? 1.45 : 1.0) +
                     (units <= sms ? 4 : p->pair ? 24 : 10);
  if (few && mt > 1) {
    int n = 2;
    const bool two = few_ctas(p->rows, format, d) == 2;
    while (n < 8 && n < mt && bh * 2 * n <= (n < 4 || two ? sms : sms / 2)) n *= 2;
    const double shared = ceil(mt / n) * us + 2;
    if (bh * n <= sms && shared < cut && shared < mt * us) {
      p->cluster = n;
      return;
    }
  }
  const int groups = (p->rows + kTile - 1) / kTile;
  if (ceil(bh * groups / sms) * mt * us > cut || (p->pair && bh * groups > sms)) return;
  p->whole = 1;
  p->pair = 0;
  p->groups = groups;
}

}  // namespace fa
