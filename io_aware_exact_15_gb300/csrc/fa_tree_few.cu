// Tree attention for few query rows per key/value head (a decode step, a
// small tree): R = G T <= 32 rows.
//
// With so few rows the work is reading the cache: per 128 keys a
// 128-row tensor-core tile would compute (and its softmax walk) mostly
// padding.  So here the rows are the M = 16 side of warp-level MMAs and
// every warp keeps its own running softmax over its own keys:
//   A CTA has 8 warps and a run of units as in fa_tree.cu (a unit is 128 keys
//   of a (sequence, key/value head)); warp w takes keys 16 w .. 16 w + 15 of
//   each unit through its own ring of TMA slots (K and V of 16 keys each) and
//   meets the other warps only at the end of a problem, where their O and
//   (m, l) are added.  16 keys never cross a page.
//   S = Q K^T and O += P V stay in registers: the accumulator layout of S is
//   the operand layout of P.
//
// Contraction indices and key columns may be permuted freely as long as both
// operands agree, which gives every lane whole 16-byte pieces of a row:
//   * lane (g = lane / 4, c = lane % 4) reads for the key in column n = g of
//     an 8-key tile the pieces c (and c + 4) of the row; Q's fragments are the
//     same pieces of rows g and g + 8;
//   * column n stands for key n / 2 (n even) or (n / 2) ^ 5 (n odd), which
//     keeps the eight lanes of a shared-memory access on different banks;
//   * 8-bit V: lane (g, c) reads one piece (d / 8 elements) of the rows of
//     keys c and c ^ 5 and pairs them byte by byte, so tile t of the output
//     holds element t of the pieces.
//
// 8-bit caches: the stored numbers go to the MMA as f16 (exact), the scales
// stay outside: a key's scale multiplies its score, a value's is added to
// the exponent of its weight, P' = 2^(s + e_v - M + 7) with M the running max
// of s + e_v, so P' <= 2^15, rounded to f16: by half a step (2^-11 of it), or
// for weights below 2^-21 of the largest by 2^-32 of the largest; l keeps
// its own max of s.  Q goes in as f16 with each row scaled by a power
// of two to [2^14, 2^15): exact but for elements 2^-31 below the row's
// largest.  No value is widened to bf16, which would cost five integer
// operations per two elements against one or two.
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "fa_internal.h"
#include "fa_quant.cuh"
#include "fa_tree.cuh"

namespace fa {
namespace {

constexpr int kFewWarps = 8;
constexpr int kFewKeys = 16;  // keys per warp and unit
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;  // O is rescaled when the max grew by more than 2^8
constexpr float kLift = 7.0f;  // f16 weights: 2^7 above the max, 2^15 at most

template <int D, int FMT, int MT>
struct FewSmem {
  static constexpr bool Q8 = FMT != kCacheBf16;
  static constexpr int EB = Q8 ? 1 : 2;
  static constexpr int KBYTES = kFewKeys * D * EB;  // 16 keys or values
  static constexpr int SLOT = 2 * KBYTES;
  static constexpr int R = Q8 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 6);  // slots per warp
  static constexpr int ROWS = 16 * MT;
  static constexpr int CW = 64 / MT;                // columns added up at a time
  static constexpr int RING = 0;
  static constexpr int SUM = RING + kFewWarps * R * SLOT;  // [8][ROWS][CW] fp32; (m, l) first
  static constexpr int SC = SUM + kFewWarps * ROWS * CW * 4;  // scale bytes: 16 + 16 per slot
  static constexpr int FIN = SC + (Q8 ? kFewWarps * R * 32 : 0);  // (m, l) of the rows
  static constexpr int BAR = FIN + ROWS * 8;
  static constexpr int MISC = BAR + kFewWarps * R * 8;  // abort flag, bad part
  static constexpr int ALLOC = MISC + 16 + 1024;        // + slack for 1024-byte alignment
  static_assert(ALLOC <= 232448, "shared memory budget");
};

template <bool F16>
FA_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                     uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

FA_DEV void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

FA_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// four stored bytes as f16 pairs (bytes 0, 1) and (2, 3), exact
template <int FMT>
FA_DEV void stored_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kCacheE4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // x + 128 under the exponent of 1024, less 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}

// 2^(byte - 127); NaN for the scale of a bad row
FA_DEV float scale_value(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte << 23);
}
// byte - 127
FA_DEV float scale_exponent(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7FFFFFFFu) : static_cast<float>(static_cast<int>(byte) - 127);
}

FA_DEV uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
FA_DEV uint2 lds_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

FA_DEV float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
FA_DEV float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// The 16-key pieces of one warp, in the order of its run.
struct PieceIter {
  PartIter it;
  int t = 0;
  bool in_part = false;
  // next piece with a key; false at the end of the run
  FA_DEV bool next(const TreeParams& p, int w) {
    for (;;) {
      if (in_part && t + 1 < it.t1) {
        ++t;
      } else {
        if (!it.next(p)) return false;
        in_part = true;
        t = it.t0;
      }
      if (pos(w) < it.s.len()) return true;
    }
  }
  FA_DEV int pos(int w) const { return t * kTile + w * kFewKeys; }
};

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kFewWarps * 32, 1)
    fa_tree_few_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const void* q, const TreeParams p) {
  using L = FewSmem<D, FMT, MT>;
  constexpr bool Q8 = L::Q8;
  constexpr int NT = D / 8;   // 8-column tiles of O
  constexpr int QR = D / 8;   // packed registers of a row's share of a lane (2 elements each)
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC);
  // whether part p has NaN or infinite draft values: entry p % 2 says p
  volatile int* bad_parts = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  const uint32_t ring = sb + L::RING + w * L::R * L::SLOT;
  const uint32_t scales = sb + L::SC + w * L::R * 32;
  const uint32_t bars = sb + L::BAR + w * L::R * 8;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    bad_parts[0] = bad_parts[1] = -1;
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (lane == 0) {
    for (int i = 0; i < L::R; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  const Run run = find_run(p, blockIdx.x, gridDim.x, lane);
  __syncthreads();
  if (run.left == 0) return;
  const WaitCtl wc{abort_flag, p.err, p.wait_ns};

  // ---- loads: this warp's next piece to fetch, its page already looked up
  PieceIter ld;
  ld.it.init(p, run);
  bool more = ld.next(p, w);
  int page = 0;
  auto look_up = [&]() {
    if (more)
      page = p.page_table[static_cast<size_t>(ld.it.b) * p.max_pages + (ld.pos(w) >> p.log_page)];
  };
  look_up();
  uint32_t sent = 0;
  auto fetch = [&]() {
    if (!more) return;
    if (lane == 0) {
      const int slot = sent % L::R;
      const uint32_t bar = bars + 8 * slot, dst = ring + slot * L::SLOT;
      const int id = min(max(page, 0), p.num_pages - 1);
      const int hkv = ld.it.hr;
      const int row = ld.pos(w) & ((1 << p.log_page) - 1), z = id * p.Hkv + hkv;
      mbar_arrive_expect_tx(bar, L::SLOT + (Q8 ? 32 : 0));
      constexpr int CH = Q8 ? 1 : D / 64;
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        tma_load_3d(dst + h * kFewKeys * 128, &tk, bar, 64 * h, row, z);
        tma_load_3d(dst + L::KBYTES + h * kFewKeys * 128, &tv, bar, 64 * h, row, z);
      }
      if (Q8) {
        const size_t at = (static_cast<size_t>(z) << p.log_page) + row;
        bulk_load(scales + slot * 32, p.ks + at, 16, bar);
        bulk_load(scales + slot * 32 + 16, p.vs + at, 16, bar);
      }
    }
    ++sent;
    more = ld.next(p, w);
    look_up();
  };
  for (int i = 0; i < L::R; ++i) fetch();

  const float sl2 = p.scale * kLog2e;
  // key of column n in an 8-key tile: lanes read column n = g
  const int krow = (g & 1) ? (g >> 1) ^ 5 : g >> 1;
  const int k0 = c, k1 = c ^ 5;  // keys of columns 2c, 2c + 1
  PartIter it;
  it.init(p, run);
  uint32_t used = 0;
  int part = -1;
  bool ok = true;  // false: a wait gave up; the warp still meets the others
  while (it.next(p)) {
    ++part;
    // ---- Q of this part: rows g and g + 8 of each 16-row tile
    uint32_t qf[MT][2][QR];
    float frow[MT][2];          // score factor of a row (log2 units)
    uint32_t vis[MT][2];
    int trow[MT][2];            // draft of a row, -1 for none
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * mt + 8 * r + g;
        const bool in = row < p.rows;
        const int t = row % p.T;
        trow[mt][r] = in && t < it.s.nd ? t : -1;
        const uint16_t* qrow = static_cast<const uint16_t*>(q) +
                               ((static_cast<size_t>(it.b) * p.Hkv + it.hr) * p.rows + row) * D;
        // pieces of 16 bytes: bf16 keys pair with pieces c, c + 4 of each 64
        // elements; 8-bit keys have 16 elements to a piece, two of these
#pragma unroll
        for (int i = 0; i < QR / 4; ++i) {
          const int piece = Q8 ? 2 * (c + 4 * (i >> 1)) + (i & 1) : 8 * (i >> 1) + c + 4 * (i & 1);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in) v = *reinterpret_cast<const uint4*>(qrow + 8 * piece);
          qf[mt][r][4 * i] = v.x;
          qf[mt][r][4 * i + 1] = v.y;
          qf[mt][r][4 * i + 2] = v.z;
          qf[mt][r][4 * i + 3] = v.w;
        }
        frow[mt][r] = sl2;
        if (Q8) {
          uint32_t m2 = 0;
#pragma unroll
          for (int i = 0; i < QR; ++i) m2 = __vmaxu2(m2, qf[mt][r][i] & 0x7FFF7FFFu);
          uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          // 2^E <= max < 2^(E+1); times 2^(14 - E).  E >= -100 keeps both
          // factors normal.
          const int E = max(static_cast<int>(m >> 7) - 127, -100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - max(E, -100)) << 23);
          frow[mt][r] = sl2 * __uint_as_float(static_cast<uint32_t>(127 + E - 14) << 23);
#pragma unroll
          for (int i = 0; i < QR; ++i)
            qf[mt][r][i] = pack_f16(bf16_lo(qf[mt][r][i]) * up, bf16_hi(qf[mt][r][i]) * up);
        }
      }
    float o[MT][NT][4];
    float M[MT][2], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][t][e] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) M[mt][r] = m[mt][r] = -INFINITY, l[mt][r] = 0.f;
    }
    bool bad = false;
#pragma unroll 1
    for (int tile = it.t0; ok && tile < it.t1; ++tile) {
      const int pos = tile * kTile + w * kFewKeys;
      if (pos >= it.s.len()) break;  // this warp's keys end in front of the tile's
      const int slot = used % L::R;
      ok = __all_sync(0xffffffffu, wait_bar(bars + 8 * slot, (used / L::R) & 1, wc));
      if (!ok) break;
      const uint32_t ka = ring + slot * L::SLOT, va = ka + L::KBYTES;
      const bool tail = pos + kFewKeys > it.s.hist;
      // ---- S = Q K^T
      float s[MT][2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
        const int row = 8 * j + krow;
        if (!Q8) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {  // pieces of 8 elements
            const int chunk = c + 4 * (i & 1);
            const uint4 k = ld_shared_v4(ka + (i >> 1) * kFewKeys * 128 + sw128_offset(row, chunk));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<false>(s[mt][j], qf[mt][0][4 * i], qf[mt][1][4 * i], qf[mt][0][4 * i + 1],
                              qf[mt][1][4 * i + 1], k.x, k.y);
              mma16816<false>(s[mt][j], qf[mt][0][4 * i + 2], qf[mt][1][4 * i + 2],
                              qf[mt][0][4 * i + 3], qf[mt][1][4 * i + 3], k.z, k.w);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {  // pieces of 16 elements
            const uint32_t at = D == 128 ? sw128_offset(row, c + 4 * i)
                                         : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
            const uint4 k = ld_shared_v4(ka + at);
            const uint32_t kw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              stored_f16<FMT>(kw[x], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma16816<true>(s[mt][j], qf[mt][0][8 * i + 2 * x], qf[mt][1][8 * i + 2 * x],
                               qf[mt][0][8 * i + 2 * x + 1], qf[mt][1][8 * i + 2 * x + 1], b0, b1);
            }
          }
        }
      }
      // ---- softmax step; keys of s[.][j][e]: 8 j + (e & 1 ? k1 : k0)
      float fk[4], ev[4];
      if (Q8) {
        const uint32_t sc = scales + slot * 32;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 8 * (x >> 1) + ((x & 1) ? k1 : k0);
          fk[x] = scale_value(lds_u8(sc + key));
          ev[x] = scale_exponent(lds_u8(sc + 16 + key));
        }
      }
      if (tail) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t = trow[mt][r];
            vis[mt][r] =
                t < 0 ? 0u
                      : seen_bits(p,
                                  p.mask ? p.mask + (static_cast<size_t>(it.b) * p.T + t) * p.words
                                         : nullptr,
                                  it.s, t, pos);
          }
      }
      uint32_t pf[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x[4], y[4];  // scores, and with the value's exponent (log2 units)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = s[mt][i >> 1][2 * r + (i & 1)] * frow[mt][r];
            y[i] = x[i];
            if (Q8) {
              x[i] *= fk[i];
              y[i] = x[i] + ev[i];
            }
          }
          if (tail)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((vis[mt][r] >> (8 * (i >> 1) + ((i & 1) ? k1 : k0))) & 1u))
                x[i] = y[i] = -INFINITY;
          const float ymax = quad_max(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
          float alpha = 1.f;
          if (ymax > M[mt][r] + kLazy) {
            alpha = ex2(M[mt][r] - ymax);
            M[mt][r] = ymax;
          }
          const float Mu = M[mt][r] == -INFINITY ? 0.f : M[mt][r] - (Q8 ? kLift : 0.f);
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(y[i] - Mu);
          if (!Q8) {
            l[mt][r] = l[mt][r] * alpha + ((e[0] + e[1]) + (e[2] + e[3]));
            m[mt][r] = M[mt][r];
            pf[mt][r] = pack_bf16(e[0], e[1]);
            pf[mt][2 + r] = pack_bf16(e[2], e[3]);
          } else {
            // the sum is the lane's own: its four keys of each piece
            const float xmax = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            if (xmax > m[mt][r] + kLazy) {
              l[mt][r] *= ex2(m[mt][r] - xmax);
              m[mt][r] = xmax;
            }
            const float mu = m[mt][r] == -INFINITY ? 0.f : m[mt][r];
            l[mt][r] += (ex2(x[0] - mu) + ex2(x[1] - mu)) + (ex2(x[2] - mu) + ex2(x[3] - mu));
            pf[mt][r] = pack_f16(e[0], e[1]);
            pf[mt][2 + r] = pack_f16(e[2], e[3]);
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              o[mt][t][2 * r] *= alpha;
              o[mt][t][2 * r + 1] *= alpha;
            }
          }
        }
      // ---- O += P V
      const int nval = it.s.len() - pos, ndraft = it.s.hist - pos;
      if (!Q8) {
        // rows of the four 8 x 8 pieces: keys 0-7 and 8-15 of two column tiles
        const int j = lane & 7, vrow = 8 * ((lane >> 3) & 1) + ((j & 1) ? (j >> 1) ^ 5 : j >> 1);
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          const int cc = t + (lane >> 4);
          uint32_t b[4];
          ldmatrix_x4_trans(va + (cc >> 3) * kFewKeys * 128 + sw128_offset(vrow, cc & 7), b);
          if (tail) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int ka0 = 8 * (x & 1) + k0, ka1 = 8 * (x & 1) + k1;
              if (ka0 >= nval) b[x] &= 0xFFFF0000u;  // past the last token
              if (ka1 >= nval) b[x] &= 0x0000FFFFu;
              const uint32_t f = finite2(b[x]);  // drafts: back at the end of the part
              if (f != b[x] && (ka0 >= ndraft || ka1 >= ndraft)) {
                const uint32_t keep = (ka0 < ndraft ? 0x0000FFFFu : 0u) |
                                      (ka1 < ndraft ? 0xFFFF0000u : 0u);
                const uint32_t n = (f & ~keep) | (b[x] & keep);
                bad |= n != b[x];
                b[x] = n;
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<false>(o[mt][t], pf[mt][0], pf[mt][1], pf[mt][2], pf[mt][3], b[0], b[1]);
            mma16816<false>(o[mt][t + 1], pf[mt][0], pf[mt][1], pf[mt][2], pf[mt][3], b[2], b[3]);
          }
        }
      } else {
        constexpr int WV = D / 32;  // words of a lane's piece: 16 or 8 elements
        uint32_t v[4][WV];          // rows k0, k1, 8 + k0, 8 + k1
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 8 * (x >> 1) + ((x & 1) ? k1 : k0);
          if (D == 128) {
            const uint4 y = ld_shared_v4(va + sw128_offset(row, (g >> 1) + 4 * (g & 1)));
            v[x][0] = y.x, v[x][1] = y.y, v[x][WV - 2] = y.z, v[x][WV - 1] = y.w;
          } else {
            const int u = (g & 1) + 4 * ((g >> 1) & 1) + 2 * (g >> 2);
            const uint2 y = lds_v2(va + row * 64 + (((u >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (u & 1));
            v[x][0] = y.x, v[x][1] = y.y;
          }
          if (tail && row >= nval)
#pragma unroll
            for (int i = 0; i < WV; ++i) v[x][i] = 0;
        }
#pragma unroll
        for (int i = 0; i < WV; ++i) {
          // bytes (key a, key b) of two columns to a word
          uint32_t b[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            stored_f16<FMT>(__byte_perm(v[2 * h][i], v[2 * h + 1][i], 0x5140), b[h][0], b[h][1]);
            stored_f16<FMT>(__byte_perm(v[2 * h][i], v[2 * h + 1][i], 0x7362), b[h][2], b[h][3]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma16816<true>(o[mt][4 * i + x], pf[mt][0], pf[mt][1], pf[mt][2], pf[mt][3], b[0][x],
                             b[1][x]);
        }
      }
      ++used;
      __syncwarp();  // every lane has read the slot
      fetch();
    }
    // ---- end of the part: the warps' rows are added in a fixed order
    if (bad) bad_parts[part & 1] = part;
    float2* ml = reinterpret_cast<float2*>(smem + L::SUM);
    float2* fin = reinterpret_cast<float2*>(smem + L::FIN);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mq = Q8 ? quad_max(m[mt][r]) : m[mt][r];
        const float mu = mq == -INFINITY ? 0.f : mq;
        const float lq = quad_sum(l[mt][r] * ex2(m[mt][r] - mu));
        if (c == 0) ml[w * L::ROWS + 16 * mt + 8 * r + g] = make_float2(mq, lq);
      }
    __syncthreads();
    if (threadIdx.x < L::ROWS) {
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < kFewWarps; ++i) mm = fmaxf(mm, ml[i * L::ROWS + threadIdx.x].x);
      const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int i = 0; i < kFewWarps; ++i) {
        const float2 x = ml[i * L::ROWS + threadIdx.x];
        ll = fmaf(x.y, ex2(x.x - mu), ll);
      }
      fin[threadIdx.x] = make_float2(mm, ll);
    }
    __syncthreads();
    const bool whole = it.t0 == 0 && it.t1 == it.s.tiles;
    const size_t orow0 = (static_cast<size_t>(it.b) * p.Hkv + it.hr) * p.rows;
    const size_t prow0 =
        (2 * static_cast<size_t>(blockIdx.x) + (it.t0 == 0 ? 1 : 0)) * p.slot_rows;
    float* sum = reinterpret_cast<float*>(smem + L::SUM);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // O in units of 2^m; the factor in two steps (M - m reaches 128)
        const float mm = fin[16 * mt + 8 * r + g].x;
        const float a = mm == -INFINITY ? 0.f : ex2(0.5f * (M[mt][r] - (Q8 ? kLift : 0.f) - mm));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) o[mt][t][2 * r + e] = o[mt][t][2 * r + e] * a * a;
      }
#pragma unroll
    for (int pass = 0; pass < D / L::CW; ++pass) {
      const int lo = pass * L::CW;
      // column of o[.][t][e]; rows 8 apart share a bank pattern, turned by g
      auto put = [&](int mt, int r, int col, float v) {
        const int row = 16 * mt + 8 * r + g;
        sum[(w * L::ROWS + row) * L::CW + ((col - lo) ^ (8 * (g & 3)))] = v;
      };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              int col;
              if (!Q8) {
                col = 8 * t + 2 * c + e;
              } else if (D == 128) {
                col = 64 * e + 16 * c + t;
              } else {
                col = 32 * (c & 1) + 16 * (c >> 1) + 8 * e + t;
              }
              if (col >= lo && col < lo + L::CW) put(mt, r, col, o[mt][t][2 * r + e]);
            }
      __syncthreads();
      constexpr int TPR = L::CW / 4;  // threads per row, four columns each
      const int row = threadIdx.x / TPR, col = 4 * (threadIdx.x % TPR);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kFewWarps; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(
            &sum[(i * L::ROWS + row) * L::CW + (col ^ (8 * (row & 3)))]);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      if (row < p.rows) {
        const bool valid = row % p.T < it.s.nd;
        const float2 f = fin[row];
        if (whole) {
          const bool has = valid && !(f.y == 0.f);  // a NaN sum stays one
          const float inv = has ? 1.f / f.y : 0.f;
          uint2 out = make_uint2(0, 0);
          if (has)
            out = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + (orow0 + row) * D + lo + col) = out;
          if (pass == 0 && col == 0)
            p.lse[orow0 + row] = has ? (f.x + lg2(f.y)) * kLn2 : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(p.part_o + (prow0 + row) * D + lo + col) = v;
          if (pass == 0 && col == 0)
            p.part_ml[prow0 + row] = make_float2(valid ? f.x : -INFINITY, valid ? f.y : 0.f);
        }
      }
      __syncthreads();
    }
    if (!Q8 && bad_parts[part & 1] == part) {  // after the barrier: the rows are written
      const int row = threadIdx.x, t = row % p.T;
      if (row < p.rows && t < it.s.nd)
        add_not_finite<D, FMT>(p, it.b, it.hr, it.s, t, max(it.s.hist, it.t0 * kTile),
                               min(it.s.len(), it.t1 * kTile),
                               whole ? static_cast<uint16_t*>(p.o) + (orow0 + row) * D : nullptr,
                               whole ? nullptr : p.part_o + (prow0 + row) * D);
    }
  }
  // copies still in flight (only after a wait gave up) land before the CTA exits
  for (uint32_t i = used; i < sent; ++i) drain_bar(bars + 8 * (i % L::R), (i / L::R) & 1, p.wait_ns);
}

template <int D, int FMT, int MT>
cudaError_t launch_few_rows(const TreeParams& p, const void* q, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream) {
  using L = FewSmem<D, FMT, MT>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = smem_attr_once(
      attr_done, reinterpret_cast<const void*>(fa_tree_few_kernel<D, FMT, MT>), L::ALLOC);
  if (e != cudaSuccess) return e;
  return launch_pdl(fa_tree_few_kernel<D, FMT, MT>, dim3(grid), dim3(kFewWarps * 32), L::ALLOC,
                    stream, tk, tv, q, p);
}

template <int D, int FMT>
cudaError_t launch_few_fmt(const TreeParams& p, const void* q, const CUtensorMap& tk,
                           const CUtensorMap& tv, int grid, cudaStream_t stream) {
  return p.rows <= 16 ? launch_few_rows<D, FMT, 1>(p, q, tk, tv, grid, stream)
                      : launch_few_rows<D, FMT, 2>(p, q, tk, tv, grid, stream);
}

}  // namespace

cudaError_t launch_tree_few(const TreeParams& p, int format, int d, const void* q,
                            const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                            cudaStream_t stream) {
  if (d == 64)
    return format == kCacheBf16   ? launch_few_fmt<64, kCacheBf16>(p, q, tk, tv, grid, stream)
           : format == kCacheE4m3 ? launch_few_fmt<64, kCacheE4m3>(p, q, tk, tv, grid, stream)
                                  : launch_few_fmt<64, kCacheInt8>(p, q, tk, tv, grid, stream);
  return format == kCacheBf16   ? launch_few_fmt<128, kCacheBf16>(p, q, tk, tv, grid, stream)
         : format == kCacheE4m3 ? launch_few_fmt<128, kCacheE4m3>(p, q, tk, tv, grid, stream)
                                : launch_few_fmt<128, kCacheInt8>(p, q, tk, tv, grid, stream);
}

}  // namespace fa
