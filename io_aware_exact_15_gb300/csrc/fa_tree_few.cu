// Tree attention for few query rows per key/value head (a decode step, a
// small tree): R = G T up to 16 rows, 24 for 8-bit caches (fa_tree_host.h has the
// rule and both sides' times).
//
// With so few rows the work is reading the cache: per 128 keys a
// 128-row tensor-core tile would compute (and its softmax walk) mostly
// padding.  So here the keys are the M = 16 side of warp-level MMAs, the rows
// the N = 8 side (these MMAs take 32 cycles each, so a 16-row side would
// already cost more than the memory), and every warp keeps its own running
// softmax over its own keys:
//   A CTA has a run of units as in fa_tree.cu (a unit is 128 keys of a
//   (sequence, key/value head)).  Two warps load whole units into a ring of
//   stages, one K and one V; the others take the units' 16-key chunks in turn
//   and meet only at the end of a problem, where their O and (m, l) are
//   added.  A chunk is a chain of dependent steps of some 1500 cycles and a
//   unit costs a loading warp 1700, so many warps of both kinds are needed to
//   follow the memory: two CTAs per SM where their rings and registers fit
//   (few_ctas), which also hides the ends of short problems, a chain of
//   barriers and sums, behind each other.
//   S^T = K Q^T (16 keys x 8 rows) and O^T += V^T P^T (16 columns x 8 rows)
//   stay in registers; P^T becomes an operand by an 8 x 8 transpose.
//
// Contraction indices, keys and columns may be permuted freely as long as
// both operands agree, which gives every lane whole 16-byte pieces of a row:
//   * lane (g = lane / 4, c = lane % 4) reads the pieces c (and c + 4) of its
//     keys' rows; Q's fragments are the same pieces of row g;
//   * index m of 8 keys stands for key m / 2 (m even) or (m / 2) ^ 5 (m odd),
//     which keeps the eight lanes of a shared-memory access on different
//     banks;
//   * 8-bit V: lane (g, c) reads one piece (d / 8 elements) of the rows of
//     keys c and c ^ 5 and pairs them byte by byte, so column tile i of the
//     output holds elements 2 i and 2 i + 1 of the pieces.
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
//
// Measured: 32 sequences x 1 token, 16 + 4 heads of 128, up to 8192 e4m3
// keys: 40.8 us, 4.2 TB/s (the bytes at a plain copy's rate: 25.8); 256
// sequences of 500 keys 47.7 (20.0).  Issue slots are 44 % busy, the
// ALU 46 %; the rest is the chain of a chunk and the ends of problems.
// With a window of 4096: 64 sequences x 1 token of up to 32768 e4m3 keys 55.1 us, 4.9
// TB/s (40.0); 1 sequence x 1 token, window 512, bf16: 10.4 us, one launch of
// clusters whose CTAs share a problem (split_window in fa_tree_host.h).
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "fa_internal.h"
#include "fa_quant.cuh"
#include "fa_tree.cuh"

namespace fa {
namespace {

constexpr int kFewKeys = 16;   // keys of a chunk
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;  // O is rescaled when the max grew by more than 2^8
constexpr float kLift = 7.0f;  // f16 weights: 2^7 above the max, 2^15 at most

// RT: 8-row tiles of the query rows
template <int D, int FMT, int RT>
struct FewSmem {
  static constexpr bool Q8 = FMT != kCacheBf16;
  static constexpr int ROWS = 8 * RT;
  static constexpr int EB = Q8 ? 1 : 2;
  static constexpr int CH = Q8 ? 1 : D / 64;            // column chunks of a tile
  static constexpr int CHUNK = kTile * (Q8 ? D : 128);  // bytes of one: [128 rows x 128 or D B]
  static constexpr int KBYTES = CH * CHUNK;             // 128 keys or values
  static constexpr int STAGE = 2 * KBYTES;
  static constexpr int CTAS = few_ctas(ROWS, FMT, D);   // per SM
  static constexpr int R = CTAS == 2 ? (STAGE == 16384 ? 6 : 3)  // stages
                           : Q8      ? (D == 128 ? 6 : 8)
                                     : (D == 128 ? 3 : 6);
  static constexpr int NL = 2;  // warps that load
  // warps that compute; 128, 168 or 255 registers for each of an SM's
  static constexpr int NC = CTAS == 2 ? 6 : RT == 1 ? 14 : RT == 2 ? 10 : 6;
  static constexpr int THREADS = 32 * (NC + NL);
  // columns added up at a time: at most 32 KB of the warps' rows
  static constexpr int CW = RT == 1 ? 64 : 32;
  static constexpr int RING = 0;
  static constexpr int SUM = RING + R * STAGE;            // [NC][ROWS][CW] fp32; (m, l) first
  static constexpr int SC = SUM + NC * ROWS * CW * 4;     // scale bytes: 128 + 128 per stage
  static constexpr int FIN = SC + (Q8 ? R * 256 : 0);     // (m, l) of the rows
  static constexpr int BAR = FIN + ROWS * 8;              // full, empty of each stage
  static constexpr int RUN = BAR + R * 16;
  static constexpr int MISC = RUN + 32;                   // abort flag, bad parts
  static constexpr int ALLOC = MISC + 16 + 1024;          // + slack for 1024-byte alignment
  static_assert((ALLOC + 1024) * CTAS <= 233472, "shared memory budget");
};

FA_DEV void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

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

// 8 x 8 transpose of 16-bit elements: lane (g, c) gives (g, 2c), (g, 2c + 1)
// and gets (2c, g), (2c + 1, g)
FA_DEV uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// over the eight lanes of a row (the same lane % 4)
FA_DEV float lanes_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
FA_DEV float lanes_sum(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, int FMT, int RT, bool WIN>
__global__ void __launch_bounds__(FewSmem<D, FMT, RT>::THREADS, FewSmem<D, FMT, RT>::CTAS)
    fa_tree_few_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const TreeParams p) {
  using L = FewSmem<D, FMT, RT>;
  constexpr bool Q8 = L::Q8;
  constexpr int MT = D / 16;  // 16-column tiles of O
  constexpr int QR = D / 8;   // packed registers of a row's share of a lane (2 elements each)
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC);
  // whether part p has NaN or infinite draft values: entry p % 2 says p
  volatile int* bad_parts = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  Run* run_slot = reinterpret_cast<Run*>(smem + L::RUN);
  auto full = [&](int stage) { return sb + L::BAR + 16 * stage; };
  auto empty = [&](int stage) { return sb + L::BAR + 16 * stage + 8; };

  if (warp == 0) {
    const Run r = find_run<WIN>(p, blockIdx.x, gridDim.x, lane);
    if (lane == 0) *run_slot = r;
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < L::R; ++i) {
      mbar_init(full(i), 2);  // K and V
      mbar_init(empty(i), L::NC);
    }
    *abort_flag = 0;
    bad_parts[0] = bad_parts[1] = -1;
    fence_mbar_init();
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  __syncthreads();
  const Run run = *run_slot;
  // WIN: the CTAs of a cluster each have a part of one problem; once all parts
  // are written (every thread of the cluster comes here), the first one joins them
  auto parts_written = [&]() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  };
  if (run.left == 0) {
    if (WIN && p.cluster)
      parts_written();
    else if (threadIdx.x == 0)
      note_join(p, run, PartIter<WIN>(), blockIdx.x);
    return;
  }
  const WaitCtl wc{abort_flag, p.err, p.wait_ns};

  if (warp < L::NL) {
    // ------------------------------------------------------ loads
    // warp 0: K, warp 1: V
    const bool isv = warp == 1;
    const CUtensorMap* map = isv ? &tv : &tk;
    const uint8_t* sc = isv ? p.vs : p.ks;
    const int psize = 1 << p.log_page;
    TileIter<WIN> ti;
    ti.it.init(p, run);
    uint32_t n = 0;
    bool ok = true;
    bool have = ti.next(p);
    // pages of the next tile that hold a token (that a draft sees), one per lane
    int np = 0, id = 0;
    bool want = false;
    auto look_up = [&]() {
      const int kb = ti.it.s.key_tile(ti.t) * kTile;
      const int nval = min(max(ti.it.s.len() - kb, 0), kTile);
      np = (nval + psize - 1) >> p.log_page;
      want = lane < np && !(WIN && ti.it.s.nothing(kb + lane * psize, psize));
      if (WIN) np = __popc(__ballot_sync(0xffffffffu, want));
      id = 0;
      if (want)
        id = p.page_table[static_cast<size_t>(ti.it.b) * p.max_pages + (kb >> p.log_page) + lane];
    };
    if (have) look_up();
    while (have) {
      const int stage = n % L::R;
      if (!isv && ti.first) {  // Q of a part that the others are still to begin
        const char* q = static_cast<const char*>(p.q) +
                        (static_cast<size_t>(ti.it.b) * p.Hkv + ti.it.hr) * p.rows * (2 * D);
        if (lane < p.rows * (D / 64)) prefetch_l1(q + 128 * lane);
      }
      if (n >= L::R) ok = __all_sync(0xffffffffu, wait_bar(empty(stage), (n / L::R - 1) & 1, wc));
      if (!ok) break;
      if (lane == 0)
        mbar_arrive_expect_tx(full(stage), np * psize * (D * L::EB + (Q8 ? 1 : 0)));
      __syncwarp();
      if (want) {
        const int z = min(max(id, 0), p.num_pages - 1) * p.Hkv + ti.it.hr;
        const uint32_t dst = sb + L::RING + stage * L::STAGE + (isv ? L::KBYTES : 0) +
                             lane * psize * (Q8 ? D : 128);
#pragma unroll
        for (int h = 0; h < L::CH; ++h)
          tma_load_3d(dst + h * L::CHUNK, map, full(stage), 64 * h, 0, z);
        if (Q8)
          bulk_load(sb + L::SC + stage * 256 + (isv ? 128 : 0) + lane * psize,
                    sc + (static_cast<size_t>(z) << p.log_page), psize, full(stage));
      }
      ++n;
      have = ti.next(p);
      if (have) look_up();
    }
    // let copies still in flight land before the CTA can exit
    for (uint32_t j = n > L::R ? n - L::R : 0; j < n; ++j)
      drain_bar(full(j % L::R), (j / L::R) & 1, p.wait_ns);
    if (WIN && p.cluster) parts_written();
    return;
  }

  // -------------------------------------------------------- attention
  const int w = warp - L::NL, tid = threadIdx.x - 32 * L::NL;
  auto meet = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * L::NC) : "memory"); };
  const float sl2 = p.scale * kLog2e;
  const int k_own = (g & 1) ? (g >> 1) ^ 5 : g >> 1;  // key of index g
  const int k0 = c, k1 = c ^ 5;                       // keys of indices 2c, 2c + 1
  PartIter<WIN> it;
  it.init(p, run);
  uint32_t n = 0;  // tiles of the run
  int part = -1;
  bool ok = true;  // false: a wait gave up; the warp still meets the others
  while (it.next(p)) {
    ++part;
    // ---- Q of this part: row 8 rt + g of each tile
    uint32_t qf[RT][QR];
    float frow[RT][2];  // score factor of rows 8 rt + 2c, + 1 (log2 units)
    int trow[RT][2];    // their drafts, -1 for none
    int begin[RT][2];   // WIN: where their windows begin
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = 8 * rt + g;
      const uint16_t* qrow = static_cast<const uint16_t*>(p.q) +
                             ((static_cast<size_t>(it.b) * p.Hkv + it.hr) * p.rows + row) * D;
      // pieces of 16 bytes: bf16 keys pair with pieces c, c + 4 of each 64
      // elements; 8-bit keys have 16 elements to a piece, two of these
#pragma unroll
      for (int i = 0; i < QR / 4; ++i) {
        const int piece = Q8 ? 2 * (c + 4 * (i >> 1)) + (i & 1) : 8 * (i >> 1) + c + 4 * (i & 1);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < p.rows) v = *reinterpret_cast<const uint4*>(qrow + 8 * piece);
        qf[rt][4 * i] = v.x;
        qf[rt][4 * i + 1] = v.y;
        qf[rt][4 * i + 2] = v.z;
        qf[rt][4 * i + 3] = v.w;
      }
      float f = sl2;
      if (Q8) {
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < QR; ++i) m2 = __vmaxu2(m2, qf[rt][i] & 0x7FFF7FFFu);
        uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^E <= max < 2^(E+1); times 2^(14 - E).  E >= -100 keeps both
        // factors normal.
        const int E = max(static_cast<int>(m >> 7) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - E) << 23);
        f = sl2 * __uint_as_float(static_cast<uint32_t>(127 + E - 14) << 23);
#pragma unroll
        for (int i = 0; i < QR; ++i)
          qf[rt][i] = pack_f16(bf16_lo(qf[rt][i]) * up, bf16_hi(qf[rt][i]) * up);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        frow[rt][r] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + r));
        const int row2 = 8 * rt + 2 * c + r, t = row2 % p.T;
        trow[rt][r] = row2 < p.rows && t < it.s.nd ? t : -1;
        begin[rt][r] = 0;
        if constexpr (WIN)
          if (trow[rt][r] >= 0)
            begin[rt][r] = window_begin(
                p, p.mask ? p.mask + (static_cast<size_t>(it.b) * p.T + t) * p.words : nullptr,
                it.s, t);
      }
    }
    float o[RT][MT][4];  // column tile: (element 0, rows 2c, 2c + 1), (element 1, ...)
    float M[RT][2], m[RT][2], l[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[rt][i][e] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) M[rt][r] = m[rt][r] = -INFINITY, l[rt][r] = 0.f;
    }
    bool bad = false;
    int chunk = w;  // of the part; this warp's next one
#pragma unroll 1
    for (int tile = it.t0; tile < it.t1; ++tile, ++n) {
     const int stage = n % L::R;
     // every warp waits for every tile and gives every stage back, also
     // without a chunk of its own there: a barrier's parity tells two loads of
     // a stage apart, not three, so nobody may fall two loads behind
     ok = ok && __all_sync(0xffffffffu, wait_bar(full(stage), (n / L::R) & 1, wc));
     if (!ok) continue;
#pragma unroll 1
     for (; chunk < 8 * (tile - it.t0 + 1); chunk += L::NC) {
      const int sub = chunk & 7, pos = it.s.key_tile(tile) * kTile + sub * kFewKeys;
      if (it.s.nothing(pos, kFewKeys)) continue;
      const uint32_t ka = sb + L::RING + stage * L::STAGE + sub * kFewKeys * (Q8 ? D : 128);
      const uint32_t va = ka + L::KBYTES;
      const bool tail = it.s.mixed(pos, kFewKeys);
      // ---- S^T = K Q^T: s[rt] = (key g, rows 2c, 2c + 1), (key 8 + g, ...)
      float s[RT][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[rt][e] = 0.f;
      if (!Q8) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // pieces of 8 elements
          const uint32_t at = (i >> 1) * L::CHUNK + sw128_offset(k_own, c + 4 * (i & 1));
          const uint4 a = ld_shared_v4(ka + at), b = ld_shared_v4(ka + at + 8 * 128);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            mma16816<false>(s[rt], a.x, b.x, a.y, b.y, qf[rt][4 * i], qf[rt][4 * i + 1]);
            mma16816<false>(s[rt], a.z, b.z, a.w, b.w, qf[rt][4 * i + 2], qf[rt][4 * i + 3]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // pieces of 16 elements
          const uint32_t at = D == 128 ? sw128_offset(k_own, c + 4 * i)
                                       : k_own * 64 + ((c ^ ((k_own >> 1) & 3)) << 4);
          const uint4 a = ld_shared_v4(ka + at), b = ld_shared_v4(ka + at + 8 * D);
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t a0, a2, a1, a3;
            stored_f16<FMT>(aw[x], a0, a2);
            stored_f16<FMT>(bw[x], a1, a3);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              mma16816<true>(s[rt], a0, a1, a2, a3, qf[rt][8 * i + 2 * x],
                             qf[rt][8 * i + 2 * x + 1]);
          }
        }
      }
      // ---- softmax step over keys k_own and 8 + k_own
      float fk[2], ev[2];
      if (Q8) {
        const uint32_t sc = sb + L::SC + stage * 256 + sub * kFewKeys;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          fk[x] = scale_value(ld_shared_u8(sc + 8 * x + k_own));
          ev[x] = scale_exponent(ld_shared_u8(sc + 128 + 8 * x + k_own));
        }
      }
      uint32_t pf[RT][2];  // P^T operands: keys 0-7, 8-15
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float x[2][2], y[2][2];  // [row][key]: scores, and with the value's exponent (log2 units)
        bool over = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[r][i] = s[rt][2 * i + r] * frow[rt][r];
            if (Q8) x[r][i] *= fk[i];
            y[r][i] = Q8 ? x[r][i] + ev[i] : x[r][i];
          }
          if (tail) {
            const int t = trow[rt][r];
            const uint32_t vis =
                t < 0 ? 0u
                      : seen_bits<WIN>(
                            p,
                            p.mask ? p.mask + (static_cast<size_t>(it.b) * p.T + t) * p.words
                                   : nullptr,
                            it.s, t, pos, begin[rt][r]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (!((vis >> (8 * i + k_own)) & 1u)) x[r][i] = y[r][i] = -INFINITY;
          }
          over |= fmaxf(y[r][0], y[r][1]) > M[rt][r] + kLazy;
          if (Q8) over |= fmaxf(x[r][0], x[r][1]) > m[rt][r] + kLazy;
        }
        // The maxima are looked for (over the row's lanes) only when a score
        // passes one by more than 2^8: rarely after the first chunks.
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float ymax = lanes_max(fmaxf(y[r][0], y[r][1]));
            if (ymax > M[rt][r] + kLazy) {
              const float alpha = ex2(M[rt][r] - ymax);
              M[rt][r] = ymax;
              if (!Q8) l[rt][r] *= alpha;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[rt][i][r] *= alpha;
                o[rt][i][2 + r] *= alpha;
              }
            }
            if (Q8) {
              const float xmax = fmaxf(x[r][0], x[r][1]);  // the lane's own sum
              if (xmax > m[rt][r] + kLazy) {
                l[rt][r] *= ex2(m[rt][r] - xmax);
                m[rt][r] = xmax;
              }
            }
          }
        }
        float e[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float Mu = M[rt][r] == -INFINITY ? 0.f : M[rt][r] - (Q8 ? kLift : 0.f);
          e[r][0] = ex2(y[r][0] - Mu);
          e[r][1] = ex2(y[r][1] - Mu);
          if (Q8) {
            const float mu = m[rt][r] == -INFINITY ? 0.f : m[rt][r];
            l[rt][r] += ex2(x[r][0] - mu) + ex2(x[r][1] - mu);
          } else {
            l[rt][r] += e[r][0] + e[r][1];
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          pf[rt][i] =
              transpose8(Q8 ? pack_f16(e[0][i], e[1][i]) : pack_bf16(e[0][i], e[1][i]));
      }
      // ---- O^T += V^T P^T
      if (!Q8) {
        // rows of the four 8 x 8 pieces: keys 0-7 and 8-15 of two column halves
        const int j = lane & 7, vrow = 8 * (lane >> 4) + ((j & 1) ? (j >> 1) ^ 5 : j >> 1);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int cc = 2 * i + ((lane >> 3) & 1);
          uint32_t a[4];  // (keys 0-7, columns 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
          ldmatrix_x4_trans(va + (cc >> 3) * L::CHUNK + sw128_offset(vrow, cc & 7), a);
          if (tail) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int ka0 = 8 * (x >> 1) + k0, ka1 = 8 * (x >> 1) + k1;
              if (it.s.nobody(pos + ka0)) a[x] &= 0xFFFF0000u;  // past the last token, say
              if (it.s.nobody(pos + ka1)) a[x] &= 0x0000FFFFu;
              // NaN and infinities of drafts (of what not every draft sees):
              // back at the end of the part
              const uint32_t f = finite2(a[x]);
              const uint32_t history = (it.s.everybody(pos + ka0) ? 0x0000FFFFu : 0u) |
                                       (it.s.everybody(pos + ka1) ? 0xFFFF0000u : 0u);
              const uint32_t n = (f & ~history) | (a[x] & history);
              bad |= n != a[x];
              a[x] = n;
            }
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            mma16816<false>(o[rt][i], a[0], a[1], a[2], a[3], pf[rt][0], pf[rt][1]);
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
            const uint2 y = ld_shared_v2(va + row * 64 + (((u >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (u & 1));
            v[x][0] = y.x, v[x][1] = y.y;
          }
          if (tail && it.s.nobody(pos + row))
#pragma unroll
            for (int i = 0; i < WV; ++i) v[x][i] = 0;
          // Not every draft sees it: no e4m3 number that is a NaN, which a weight
          // of zero would not stop.  (A row that is NaN has a scale that says
          // so, and those that see it get theirs from that.)
          if (WIN && FMT == kCacheE4m3 && tail && !it.s.everybody(pos + row))
#pragma unroll
            for (int i = 0; i < WV; ++i) {
              const uint32_t n = ((v[x][i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              v[x][i] &= ~((n >> 7) * 0xFFu);
            }
        }
#pragma unroll
        for (int i = 0; i < WV; ++i) {
          // bytes (key a, key b) of two columns to a word
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            stored_f16<FMT>(__byte_perm(v[2 * h][i], v[2 * h + 1][i], 0x5140), a[h][0], a[h][1]);
            stored_f16<FMT>(__byte_perm(v[2 * h][i], v[2 * h + 1][i], 0x7362), a[h][2], a[h][3]);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              mma16816<true>(o[rt][2 * i + x], a[0][2 * x], a[0][2 * x + 1], a[1][2 * x],
                             a[1][2 * x + 1], pf[rt][0], pf[rt][1]);
        }
      }
     }
     __syncwarp();  // every lane has read this warp's chunks
     if (lane == 0) mbar_arrive(empty(stage));
    }
    // ---- end of the part: the warps' rows are added in a fixed order
    if (bad) bad_parts[part & 1] = part;
    float2* ml = reinterpret_cast<float2*>(smem + L::SUM);
    float2* fin = reinterpret_cast<float2*>(smem + L::FIN);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mq = Q8 ? lanes_max(m[rt][r]) : M[rt][r];
        const float mu = mq == -INFINITY ? 0.f : mq;
        const float lq = lanes_sum(Q8 ? l[rt][r] * ex2(m[rt][r] - mu) : l[rt][r]);
        if (g == 0) ml[w * L::ROWS + 8 * rt + 2 * c + r] = make_float2(mq, lq);
      }
    meet();
    if (tid < L::ROWS) {
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < L::NC; ++i) mm = fmaxf(mm, ml[i * L::ROWS + tid].x);
      const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int i = 0; i < L::NC; ++i) {
        const float2 x = ml[i * L::ROWS + tid];
        ll = fmaf(x.y, ex2(x.x - mu), ll);
      }
      fin[tid] = make_float2(mm, ll);
    }
    meet();
    const bool whole = it.t0 == 0 && it.t1 == it.s.tiles;
    const size_t orow0 = (static_cast<size_t>(it.b) * p.Hkv + it.hr) * p.rows;
    const size_t prow0 =
        (2 * static_cast<size_t>(blockIdx.x) + (it.t0 == 0 ? 1 : 0)) * p.slot_rows;
    float* sum = reinterpret_cast<float*>(smem + L::SUM);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // O in units of 2^m; the factor in two steps (M - m reaches 128)
        const float mm = fin[8 * rt + 2 * c + r].x;
        const float a = mm == -INFINITY ? 0.f : ex2(0.5f * (M[rt][r] - (Q8 ? kLift : 0.f) - mm));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[rt][i][r] = o[rt][i][r] * a * a;
          o[rt][i][2 + r] = o[rt][i][2 + r] * a * a;
        }
      }
    // Column tile i, element hi of lane g goes to place 8 (2 i + hi) + g of a
    // row (with rows 2c turned by 8 c places: 32 banks); the place of a
    // column is its own for bf16, element x of lane g's piece for 8 bits.
#pragma unroll
    for (int pass = 0; pass < D / L::CW; ++pass) {
      constexpr int IW = L::CW / 16;  // column tiles of a pass
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < IW; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 8 * rt + 2 * c + (e & 1), at = 8 * (2 * i + (e >> 1)) + g;
            sum[(w * L::ROWS + row) * L::CW + (at ^ (8 * c))] = o[rt][pass * IW + i][e];
          }
      meet();
#pragma unroll 1
      for (int x = tid; x < L::ROWS * L::CW; x += 32 * L::NC) {
        const int row = x / L::CW, at = x % L::CW;
        if (row >= p.rows) break;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < L::NC; ++i)
          v += sum[(i * L::ROWS + row) * L::CW + (at ^ (8 * ((row >> 1) & 3)))];
        const int el = 2 * pass * IW + (at >> 3), gl = at & 7;
        const int col = !Q8        ? 8 * el + gl
                        : D == 128 ? 16 * ((gl >> 1) + 4 * (gl & 1)) + el
                                   : 8 * ((gl & 1) + 4 * ((gl >> 1) & 1) + 2 * (gl >> 2)) + el;
        const bool valid = row % p.T < it.s.nd;
        const float2 f = fin[row];
        if (whole) {
          const bool has = valid && !(f.y == 0.f);  // a NaN sum stays one
          static_cast<uint16_t*>(p.o)[(orow0 + row) * D + col] =
              has ? static_cast<uint16_t>(pack_bf16(v / f.y, 0.f)) : 0;
          if (pass == 0 && at == 0)
            p.lse[orow0 + row] = has ? (f.x + lg2(f.y)) * kLn2 : -INFINITY;
        } else {
          p.part_o[(prow0 + row) * D + col] = v;
          if (pass == 0 && at == 0)
            p.part_ml[prow0 + row] = make_float2(valid ? f.x : -INFINITY, valid ? f.y : 0.f);
        }
      }
      meet();
    }
    if (!Q8 && bad_parts[part & 1] == part) {  // after the barrier: the rows are written
      const int row = tid, t = row % p.T;
      if (row < p.rows && t < it.s.nd)
        add_not_finite<D, FMT, WIN>(
            p, it.b, it.hr, it.s, t, it.t0, it.t1,
            whole ? static_cast<uint16_t*>(p.o) + (orow0 + row) * D : nullptr,
            whole ? nullptr : p.part_o + (prow0 + row) * D);
    }
  }
  if (WIN && p.cluster) {
    const int tiles = it.s.tiles;
    parts_written();
    if (it.t0 > 0 || it.t1 == tiles) return;  // not the first part, or all there is
    // the k-th part is CTA k's, or with fewer tiles than CTAs that of the k-th one with a tile
    const int n = min(tiles, p.cluster);
    const size_t c0 = blockIdx.x - blockIdx.x % p.cluster;
#pragma unroll 1
    for (int row = w; row < p.rows; row += L::NC) {
      auto at = [&](int k) {
        const int i = n == p.cluster ? k : ((k + 1) * p.cluster + tiles - 1) / tiles - 1;
        return (2 * (c0 + i) + (k == 0 ? 1 : 0)) * p.slot_rows + row;
      };
      join_row<D>(p, it.b * p.Hkv + it.hr, row, n, at, lane);
    }
    return;
  }
  if (tid == 0) note_join(p, run, it, blockIdx.x);
}

template <int D, int FMT, int RT, bool WIN>
cudaError_t launch_few_win(const TreeParams& p, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream) {
  using L = FewSmem<D, FMT, RT>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = smem_attr_once(
      attr_done, reinterpret_cast<const void*>(fa_tree_few_kernel<D, FMT, RT, WIN>), L::ALLOC);
  if (e != cudaSuccess) return e;
  if (WIN && p.cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::ALLOC;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fa_tree_few_kernel<D, FMT, RT, WIN>, tk, tv, p);
  }
  return launch_pdl(fa_tree_few_kernel<D, FMT, RT, WIN>, dim3(grid), dim3(L::THREADS), L::ALLOC,
                    stream, tk, tv, p);
}

template <int D, int FMT, int RT>
cudaError_t launch_few_rows(const TreeParams& p, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream) {
  return p.window ? launch_few_win<D, FMT, RT, true>(p, tk, tv, grid, stream)
                  : launch_few_win<D, FMT, RT, false>(p, tk, tv, grid, stream);
}

template <int D, int FMT>
cudaError_t launch_few_fmt(const TreeParams& p, const CUtensorMap& tk,
                           const CUtensorMap& tv, int grid, cudaStream_t stream) {
  if (p.rows <= 8) return launch_few_rows<D, FMT, 1>(p, tk, tv, grid, stream);
  if (p.rows <= 16) return launch_few_rows<D, FMT, 2>(p, tk, tv, grid, stream);
  if constexpr (FMT != kCacheBf16)
    if (p.rows <= 24) return launch_few_rows<D, FMT, 3>(p, tk, tv, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree_few(const TreeParams& p, int format, int d, const CUtensorMap& tk,
                            const CUtensorMap& tv, int grid, cudaStream_t stream) {
  if (d == 64)
    return format == kCacheBf16   ? launch_few_fmt<64, kCacheBf16>(p, tk, tv, grid, stream)
           : format == kCacheE4m3 ? launch_few_fmt<64, kCacheE4m3>(p, tk, tv, grid, stream)
                                  : launch_few_fmt<64, kCacheInt8>(p, tk, tv, grid, stream);
  return format == kCacheBf16   ? launch_few_fmt<128, kCacheBf16>(p, tk, tv, grid, stream)
         : format == kCacheE4m3 ? launch_few_fmt<128, kCacheE4m3>(p, tk, tv, grid, stream)
                                : launch_few_fmt<128, kCacheInt8>(p, tk, tv, grid, stream);
}

}  // namespace fa
