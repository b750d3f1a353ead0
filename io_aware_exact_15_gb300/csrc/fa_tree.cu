// Attention of drafted tokens over a paged key/value cache.
//
// Sequence b has hist_lens[b] accepted tokens and draft_lens[b] <= T drafted
// ones whose keys and values stand behind them in the cache.  Draft i sees
// every accepted token and the drafts whose bit is set in its mask row (its
// ancestors and itself in a tree; all drafts up to itself without a mask):
//   o_i = sum_j p_ij v_j,  p_i = softmax over the seen j of scale q_i k_j.
//
// The G = H / Hkv query heads of a key/value head and the T drafts make
// R = G T query rows that read the same keys, so the work is a matrix
// product of R rows per (sequence, key/value head).  It is bound by reading
// the cache: 4 d flops per row and key against 4 d bytes per key (bf16), so
// up to about 290 rows the tensor cores can follow the memory.
//
// Work split.  A problem is (sequence, key/value head, group of rows), a unit
// one 128-key tile of a problem.  The units of all problems form one line,
// cut into equal runs, one per CTA (one CTA per SM): every SM reads the same
// number of bytes whatever the lengths are.  A run may end inside a problem;
// such a part leaves its unnormalised O and its (m, l) per row in the
// workspace, and a second kernel joins the parts.  The lengths live on the
// device, so the kernel finds its run itself (a sum over the sequences).
//
// CTA (warp 0 loads K and Q, warp 10 V, warp 1 issues the MMAs, warps 2-5 and
// 6-9 do softmax):
//   up to 128 rows ("split"): the tiles of the run alternate between the two
//     softmax warpgroups, each with its own S and O in tensor memory, so that
//     one tile's softmax overlaps the other's MMAs; the two are added at the
//     end of each problem.
//   more rows ("pair"): each warpgroup has 128 of 256 rows, every tile
//     serves both.
// bf16 caches: TMA brings each page's rows into the 128-byte-swizzled tile
// the MMA reads.  8-bit caches: bulk copies bring the stored bytes, and 8 more
// warps widen them to the same bf16 tile (exact, see fa_quant.cuh), so the
// products are those of the values that fa_cache_read returns.
//
// Measured (ragged lengths, heads of 128; the bytes at a plain copy's rate in
// brackets): 8 x 23 drafts of 16 + 4 heads over up to 16384 keys, bf16, 92
// rows: 47.6 us (27.0), 3.8 TB/s; what is left are the ends of parts and the
// join.  2 x 16 drafts over up to 131072 keys, e4m3, 64 rows: 115 us (33.0);
// 16 x 64 drafts over up to 8192 keys, int8, 256 rows: 79.1 us (15.2, by the
// products); both wait for widened tiles: issue slots 52 and 42 % busy.
//
// With a window (WIN, fa_tree_attention_window) units are the tiles that some
// draft sees something of; a problem has few of them (window / 128 and two or
// three), so its ends weigh more, and whole problems go to the CTAs where
// there are enough of them (split_window, fa_tree_host.h).  8 x 23 drafts of 12 heads of 64,
// window 2048, 64 first positions, bf16: 24.9 us (the bytes: 7.8); 16 x 64
// drafts of 16 + 4 heads of 128, window 1024, int8: 32.4 us (3.9): the
// launch, the search for the run, and one problem's chain of tiles.
//
// Keys that nobody may see are never left to chance: scores are replaced by
// -inf, values of rows past the last token are zeroed in shared memory, and
// so are NaN and infinite values of drafts, which the rows that do see them
// get back at the end (0 x NaN would reach every row otherwise).
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_quant.cuh"
#include "fa_tree.cuh"

namespace fa {
namespace {

static_assert(kCacheBf16 == static_cast<int>(FA_CACHE_BF16) &&
                  kCacheE4m3 == static_cast<int>(FA_CACHE_E4M3) &&
                  kCacheInt8 == static_cast<int>(FA_CACHE_INT8),
              "the public formats are the kernels'");

// Warps that widen 8-bit tiles, half of them K and half V (19 in all: 96
// registers).  One tile is a chain of some 2000 cycles for its warps.
constexpr int kConvWarps = 8, kConvTeam = kConvWarps / 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;  // O is rescaled when the max grew by more than 2^8

// Place of K or V of the run's tile g of `total` in the ring of bf16 tiles,
// which is the order in which the MMAs consume them.  pair: K0 V0 K1 V1 ...;
// split, where a tile's scores are formed before the previous tile's weights
// are used: K0 K1 V0 K2 V1 ... V(n-1).
// K and V are brought by warps of their own.  A barrier's parity tells one
// load of a slot from the next, not from the one after it, so nobody may wait
// two loads ahead of the slot's state.  A bringer waits for the consumption
// of the slot's last tile, NS places back; for its own previous tile, at most
// two places back, it had waited for the place NS before that one, and the
// MMAs consume in order, so everything 2 NS places back is gone.  The MMAs
// take every place in turn.  (The ring of stored 8-bit tiles has no such
// order, two teams empty it, so it is a ring for K and one for V.)
template <bool PAIR>
FA_DEV uint32_t ring_place(uint32_t g, uint32_t total, bool isv) {
  if (PAIR) return 2 * g + (isv ? 1 : 0);
  if (isv) return g + 1 == total ? 2 * g + 1 : 2 * g + 2;
  return g ? 2 * g - 1 : 0;
}

template <int D, int FMT, bool PAIR>
struct TreeSmem {
  static constexpr bool Q8 = FMT != kCacheBf16;
  static constexpr int GROUP = PAIR ? 2 * kTile : kTile;  // query rows of a problem
  static constexpr int CH = D / 64;             // 128-byte column chunks per row
  static constexpr int CHUNK = kTile * 128;     // [128 rows x 128 B] = 16 KB
  static constexpr int TILE = CH * CHUNK;       // one 128 x D bf16 tile
  static constexpr int RAW = kTile * D;         // one 128 x D tile of stored bytes
  // bf16 K/V tiles, and stored tiles (half K, half V).  d = 128, pair, 256
  // rows: 4 and 2 take 106.6 us where 3 and 4 take 110.4 (16 x 8192 e4m3
  // keys, 4 heads); split, 64 rows, 4 and 4 take 115 where 5 and 2 take 142.
  static constexpr int NS = D == 64 ? (Q8 ? 6 : 8) : 4;
  static constexpr int NR = !Q8 ? 0 : D == 64 ? 8 : PAIR ? 2 : 4;
  // Q: pair: two row tiles; split: the tiles of two parts, or of one where
  // the stored tiles need the room
  static constexpr int QB = PAIR || Q8 ? 1 : 2;  // parts whose Q has a place
  static constexpr int Q = 0;
  static constexpr int KV = (PAIR ? 2 : QB) * TILE;
  static constexpr int RW = KV + NS * TILE;
  // bf16: each softmax warp's 32 rows x 32 columns of O on their way out (8-bit
  // tiles leave no room)
  static constexpr int OUT = RW + NR * RAW;
  static constexpr int SC = OUT + (Q8 ? 0 : 8 * 4096);  // scale bytes of the stored tiles
  static constexpr int NOTE = SC + NR * kTile;  // what a stored tile holds: two int4 each
  static constexpr int ML = NOTE + NR * 32;     // (m, l) of the second warpgroup's rows
  static constexpr int BAR = ML + (PAIR ? 0 : kTile * 8);
  static constexpr int B_QF = 0, B_QE = 2, B_KVF = 4, B_KVE = B_KVF + NS, B_RF = B_KVE + NS,
                       B_RE = B_RF + NR, B_SF = B_RE + NR, B_PF = B_SF + 2, B_OF = B_PF + 2,
                       B_X1 = B_OF + 1, B_X2 = B_X1 + 1, B_DONE = B_X2 + 1,
                       B_OF1 = B_DONE + 1, NBAR = B_OF1 + (PAIR ? 1 : 0);
  static constexpr int RUN = BAR + NBAR * 8;    // Run
  static constexpr int MISC = RUN + 32;
  static constexpr int ALLOC = MISC + 40 + 1024;  // + slack for 1024-byte alignment
  static constexpr int THREADS = 352 + (Q8 ? 32 * kConvWarps : 0);
  // tensor memory columns: S0, S1 (128 each), O0, O1 (D each)
  static constexpr int T_O = 2 * kTile;
  // P (bf16) takes the upper half of its S: from the last keys to the first,
  // the scores are in registers when weights are stored over them
  static constexpr int T_P = 64;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

template <int D, int FMT, bool PAIR, bool WIN>
__global__ void __launch_bounds__(TreeSmem<D, FMT, PAIR>::THREADS, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const TreeParams p) {
  using L = TreeSmem<D, FMT, PAIR>;
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + L::BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  // part p has NaN or infinite draft values if entry p % 8 says p (whoever
  // finds them is less than 8 parts ahead of the end of a part)
  volatile int* bad_parts = reinterpret_cast<volatile int*>(smem + L::MISC + 8);
  Run* run_slot = reinterpret_cast<Run*>(smem + L::RUN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    const Run r = find_run<WIN>(p, blockIdx.x, gridDim.x, lane);
    if (lane == 0) {
      *run_slot = r;
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(L::B_QF + i), 1);
        mbar_init(bar(L::B_QE + i), 1);
        mbar_init(bar(L::B_SF + i), 1);
        mbar_init(bar(L::B_PF + i), 4);
      }
      for (int i = 0; i < L::NS; ++i) {
        mbar_init(bar(L::B_KVF + i), L::Q8 ? kConvTeam : 1);
        mbar_init(bar(L::B_KVE + i), 1);
      }
      for (int i = 0; i < L::NR; ++i) {
        mbar_init(bar(L::B_RF + i), 1);
        mbar_init(bar(L::B_RE + i), kConvTeam);
      }
      mbar_init(bar(L::B_OF), 1);
      if (PAIR) mbar_init(bar(L::B_OF1), 1);
      mbar_init(bar(L::B_X1), 4);
      mbar_init(bar(L::B_X2), 4);
      mbar_init(bar(L::B_DONE), 1);
      *abort_flag = 0;
      for (int i = 0; i < 8; ++i) bad_parts[i] = -1;
      fence_mbar_init();
      prefetch_tmap(&tq);
      if (!L::Q8) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Run run = *run_slot;
  const WaitCtl wc{abort_flag, p.err, p.wait_ns};
  auto uwait = [&](uint32_t b, uint32_t ph) {
    return __all_sync(0xffffffffu, wait_bar(b, ph, wc));
  };
  TileIter<WIN> tiles0;
  if (run.left > 0) tiles0.it.init(p, run);
  else tiles0.it.left = 0;

  if (warp == 0 || warp == 10) {
    // ------------------------------------------------------ loads
    const bool isv = warp == 10;
    TileIter<WIN> ti = tiles0;
    uint32_t g = 0;
    int parts = 0;
    bool ok = true;
    const int page = 1 << p.log_page;
    // pages of the next tile that hold a token (that a draft sees), one per
    // lane: looked up one tile ahead
    bool have = ti.next(p);
    int np = 0, id = 0;
    bool want = false;
    auto look_up = [&]() {
      const int kb = ti.it.s.key_tile(ti.t) * kTile;
      const int nval = min(max(ti.it.s.len() - kb, 0), kTile);
      np = (nval + page - 1) >> p.log_page;
      want = lane < np && !(WIN && ti.it.s.nothing(kb + lane * page, page));
      if (WIN) np = __popc(__ballot_sync(0xffffffffu, want));
      id = 0;
      if (want)
        id = p.page_table[static_cast<size_t>(ti.it.b) * p.max_pages + (kb >> p.log_page) + lane];
    };
    if (have) look_up();
    constexpr uint32_t N = L::Q8 ? L::NR / 2 : L::NS;
    constexpr int B_FULL = L::Q8 ? L::B_RF : L::B_KVF, B_FREE = L::Q8 ? L::B_RE : L::B_KVE;
    while (have) {
      const int hkv = ti.it.hr / p.groups;
      if (!isv && ti.first) {
        const int qb = L::QB == 1 ? 0 : ti.part & 1, use = L::QB == 1 ? ti.part : ti.part >> 1;
        if (use > 0) ok = uwait(bar(L::B_QE + qb), (use - 1) & 1);
        if (!ok) break;
        ++parts;
        if (lane == 0) {
          const int r0 = PAIR || WIN ? (ti.it.hr - hkv * p.groups) * L::GROUP : 0;
          const bool two = PAIR && r0 + kTile < p.rows;
          mbar_arrive_expect_tx(bar(L::B_QF + qb), (two ? 2 : 1) * L::TILE);
          for (int i = 0; i < (two ? 2 : 1); ++i)
#pragma unroll
            for (int c = 0; c < L::CH; ++c)
              tma_load_3d(sb + L::Q + (qb + i) * L::TILE + c * L::CHUNK, &tq, bar(L::B_QF + qb),
                          64 * c, r0 + i * kTile, ti.it.b * p.Hkv + hkv);
        }
      }
      const uint32_t idx = L::Q8 ? g : ring_place<PAIR>(g, run.left, isv);
      const uint32_t slot = idx % N + (L::Q8 && isv ? N : 0);
      if (idx >= N) ok = uwait(bar(B_FREE + slot), (idx / N - 1) & 1);
      if (!ok) break;
      const uint32_t full = bar(B_FULL + slot);
      if (lane == 0) {
        if (L::Q8) {
          const int kb = ti.it.s.key_tile(ti.t) * kTile;
          int4* note = reinterpret_cast<int4*>(smem + L::NOTE + slot * 32);
          note[0] = make_int4(ti.it.s.len() - kb, ti.it.s.hist - kb, ti.part, 0);
          if constexpr (WIN)
            note[1] = make_int4(ti.it.s.sinks - kb, ti.it.s.lo - kb, ti.it.s.edge - kb, 0);
        }
        mbar_arrive_expect_tx(full, np * page * (L::Q8 ? D + 1 : 2 * D));
      }
      __syncwarp();
      if (want) {
        const int z = min(max(id, 0), p.num_pages - 1) * p.Hkv + hkv;
        if (!L::Q8) {
#pragma unroll
          for (int c = 0; c < L::CH; ++c)
            tma_load_3d(sb + L::KV + slot * L::TILE + c * L::CHUNK + lane * page * 128,
                        isv ? &tv : &tk, full, 64 * c, 0, z);
        } else {
          const size_t row = static_cast<size_t>(z) << p.log_page;
          bulk_load(sb + L::RW + slot * L::RAW + lane * page * D,
                    static_cast<const uint8_t*>(isv ? p.vc : p.kc) + row * D, page * D, full);
          bulk_load(sb + L::SC + slot * kTile + lane * page, (isv ? p.vs : p.ks) + row, page, full);
        }
      }
      ++g;
      have = ti.next(p);
      if (have) look_up();
    }
    // let copies still in flight land before the CTA can exit
    for (int i = max(0, parts - L::QB); i < parts; ++i)
      drain_bar(bar(L::B_QF + (L::QB == 1 ? 0 : i & 1)), (L::QB == 1 ? i : i >> 1) & 1, p.wait_ns);
    for (uint32_t j = g > N ? g - N : 0; j < g; ++j) {
      const uint32_t idx = L::Q8 ? j : ring_place<PAIR>(j, run.left, isv);
      // (an earlier load has been replaced in its slot, so it has landed)
      if (L::Q8 || idx + N >= 2 * g)
        drain_bar(bar(B_FULL + idx % N + (L::Q8 && isv ? N : 0)), (idx / N) & 1, p.wait_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    auto ecommit = [&](uint32_t b) {
      if (elect_one()) mma_commit(b);
    };
    constexpr uint32_t idS = idesc_bf16(128, kTile, false, false);
    constexpr uint32_t idO = idesc_bf16(128, D, false, true);
    const uint64_t dq0 = desc_sw128(sb + L::Q, 16, 1024);
    const uint64_t dk0 = desc_sw128(sb + L::KV, 16, 1024);
    const uint64_t dv0 = desc_sw128(sb + L::KV, L::CHUNK, 1024);
    auto issue_s = [&](int s, int qtile, int slot) {
      const uint64_t qa = desc_advance(dq0, qtile * L::TILE);
      const uint64_t kb = desc_advance(dk0, slot * L::TILE);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = (kk >> 2) * L::CHUNK + (kk & 3) * 32;
        const uint64_t da = desc_advance(qa, at), db = desc_advance(kb, at);
        if (elect_one()) mma_bf16_ss(tmem + s * kTile, da, db, idS, kk > 0);
      }
    };
    auto issue_pv = [&](int s, int slot, bool acc) {
      const uint64_t vb = desc_advance(dv0, slot * L::TILE);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint64_t db = desc_advance(vb, kk * 2048);
        if (elect_one())
          mma_bf16_ts(tmem + L::T_O + s * D, tmem + s * kTile + L::T_P + kk * 8, db, idO,
                      (acc || kk > 0) ? 1u : 0u);
      }
    };
    TileIter<WIN> ti = tiles0;
    uint32_t idx = 0;  // tiles taken from the ring
    auto wait_kv = [&]() {
      return uwait(bar(L::B_KVF + idx % L::NS), (idx / L::NS) & 1);
    };
    auto wait_q = [&](int part) {
      return L::QB == 1 ? uwait(bar(L::B_QF), part & 1)
                        : uwait(bar(L::B_QF + (part & 1)), (part >> 1) & 1);
    };
    // which warpgroups a pair tile serves
    auto members = [&](const TileIter<WIN>& x) {
      return (x.it.hr % p.groups) * 2 * kTile + kTile < p.rows ? 3 : 1;
    };
    bool ok = true;
    bool have = ti.next(p);
    uint32_t g = 0, cnt0 = 0, cnt1 = 0;  // tiles; PVs of each warpgroup
    bool acc0 = false, acc1 = false;
    int mem = PAIR && have ? members(ti) : 1;
    int part = ti.part;
    bool last = ti.last;
    if (have) {
      ok = wait_q(part) && wait_kv();
      if (ok) {
        tc_fence_after();
        const int slot = idx % L::NS;
        issue_s(0, L::QB == 1 ? 0 : part & 1, slot);
        ecommit(bar(L::B_SF));
        if (PAIR && (mem & 2)) {
          issue_s(1, 1, slot);
          ecommit(bar(L::B_SF + 1));
        }
        ecommit(bar(L::B_KVE + slot));
        if (last) ecommit(bar(L::B_QE + (L::QB == 1 ? 0 : part & 1)));
        ++idx;
      }
    }
    while (ok && have) {
      const bool have_n = ti.next(p);
      const int mem_n = have_n && PAIR ? members(ti) : 1;
      if (!PAIR) {
        const int s = g & 1;
        if (have_n) {  // the next tile's scores go to the other warpgroup
          if (ti.first) ok = wait_q(ti.part);
          if (ok) ok = wait_kv();
          if (!ok) break;
          tc_fence_after();
          const int slot = idx % L::NS;
          issue_s(s ^ 1, L::QB == 1 ? 0 : ti.part & 1, slot);
          ecommit(bar(L::B_SF + (s ^ 1)));
          ecommit(bar(L::B_KVE + slot));
          if (ti.last) ecommit(bar(L::B_QE + (L::QB == 1 ? 0 : ti.part & 1)));
          ++idx;
        }
        ok = wait_kv() && uwait(bar(L::B_PF + s), (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const int slot = idx % L::NS;
        issue_pv(s, slot, s ? acc1 : acc0);
        (s ? acc1 : acc0) = true;
        ecommit(bar(L::B_KVE + slot));
        ++idx;
      } else {
        ok = wait_kv();
        if (!ok) break;
        const int vslot = idx % L::NS;
        ++idx;
        bool ready = false;  // the next tile's K (and Q)
        for (int s = 0; s < 2 && ok; ++s) {
          if (mem & (1 << s)) {
            uint32_t& cnt = s ? cnt1 : cnt0;
            ok = uwait(bar(L::B_PF + s), cnt & 1);
            if (!ok) break;
            tc_fence_after();
            issue_pv(s, vslot, s ? acc1 : acc0);
            (s ? acc1 : acc0) = true;
            ++cnt;
          }
          if (have_n && (mem_n & (1 << s))) {
            if (!ready) {
              if (ti.first) ok = wait_q(ti.part);
              if (ok) ok = wait_kv();
              if (!ok) break;
              tc_fence_after();
              ready = true;
            }
            issue_s(s, s, idx % L::NS);
            ecommit(bar(L::B_SF + s));
          }
        }
        if (!ok) break;
        ecommit(bar(L::B_KVE + vslot));
        if (ready) {
          ecommit(bar(L::B_KVE + idx % L::NS));
          if (ti.last) ecommit(bar(L::B_QE));
          ++idx;
        }
      }
      if (last) {
        // pair: a barrier for each warpgroup, and only for parts in which it
        // has rows.  The issuer needs nothing of the second one for the
        // others, and on a shared barrier it could be two phases ahead of a
        // warp that still waits for the part before.
        ecommit(bar(L::B_OF));
        if (PAIR && (mem & 2)) ecommit(bar(L::B_OF1));
        acc0 = acc1 = false;
      }
      ++g;
      have = have_n;
      mem = mem_n;
      part = ti.part;
      last = ti.last;
    }
    // every MMA issued above completes before the CTA gives its memory back
    ecommit(bar(L::B_DONE));
    drain_bar(bar(L::B_DONE), 0, p.wait_ns);
  } else if (warp < 10) {
    // ------------------------------------------------------ softmax
    const int s = (warp - 2) >> 2;
    const int q4 = warp & 3;  // tensor memory lanes this warp may access
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + s * kTile;
    const uint32_t tO = tmem + lane_off + L::T_O + s * D;
    const uint32_t tP = tS + L::T_P;
    const float sl2 = p.scale * kLog2e;
    float2* ml = reinterpret_cast<float2*>(smem + L::ML);
    PartIter<WIN> it = tiles0.it;
    uint32_t g = 0, cnt = 0;  // tiles; parities of own tiles (bit 0) and parts (bit 1)
    const uint32_t total = run.left;
    int part = -1;
    bool ok = true, owe_x2 = false;
    while (ok && it.next(p)) {
      ++part;
      const int hkv = it.hr / p.groups;
      const int row0 = PAIR || WIN ? (it.hr - hkv * p.groups) * L::GROUP + (PAIR ? s * kTile : 0)
                                   : 0;  // (only windows have several 128-row groups)
      const bool mine_all = row0 < p.rows;             // pair: this warpgroup has rows
      const bool busy = row0 + q4 * 32 < p.rows;       // this warp has rows
      const int row = row0 + r, t = row % p.T;
      const bool valid = row < p.rows && t < it.s.nd;
      const uint32_t* mask_row =
          p.mask ? p.mask + (static_cast<size_t>(it.b) * p.T + t) * p.words : nullptr;
      int begin = 0;  // WIN: where the row's window begins
      if constexpr (WIN)
        if (valid) begin = window_begin(p, mask_row, it.s, t);
      float m = -INFINITY, l = 0.f;
      int mine = 0;               // tiles of this part done by this warpgroup
      for (int tile = it.t0; tile < it.t1 && ok; ++tile, ++g) {
        if (PAIR ? !mine_all : static_cast<int>(g & 1) != s) continue;
        const int kb = it.s.key_tile(tile) * kTile;
        // drafts or the end in this tile (WIN: or an edge of the window)
        const bool tail = it.s.mixed(kb, kTile);
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        auto look = [&]() {
          if (tail && busy) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              vis[w] = valid ? seen_bits<WIN>(p, mask_row, it.s, t, kb + 32 * w, begin) : 0u;
          }
        };
        // bf16: the mask's words come while the scores are formed (8 bits:
        // there are no registers for them)
        if (!L::Q8) look();
        ok = uwait(bar(L::B_SF + s), cnt & 1);
        if (!ok) break;
        tc_fence_after();
        if (L::Q8) look();
        if (busy) {
          // the scores of a row: all 128 in registers (bf16), or a quarter at
          // a time, read again for the weights (8-bit: the widening warps
          // leave fewer registers)
          constexpr int NH = L::Q8 ? 4 : 1, C = 4 / NH;
          uint32_t sr[C][32];
          auto load_scores = [&](int half) {
#pragma unroll
            for (int c = 0; c < C; ++c) tmem_ld32(tS + 32 * C * half + 32 * c, sr[c]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C; ++c) reg_fence(sr[c]);
            if (tail) {
#pragma unroll
              for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((vis[C * half + c] >> j) & 1u)) sr[c][j] = __float_as_uint(-INFINITY);
            }
          };
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = -INFINITY;
#pragma unroll
          for (int half = 0; half < NH; ++half) {
            load_scores(half);
#pragma unroll
            for (int j = 0; j < 32; j += 2)
#pragma unroll
              for (int c = 0; c < C; ++c) {
                float& x = mx[C == 1 ? (j >> 1) & 3 : c];
                x = fmax3(x, __uint_as_float(sr[c][j]), __uint_as_float(sr[c][j + 1]));
              }
          }
          const float mxa = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
          const float m_new = fmaxf(m, mxa * sl2);
          const bool resc = m_new > m + kRescaleLog2;
          const float alpha = resc ? ex2(m - m_new) : 1.f;
          if (resc) {
            l *= alpha;
            m = m_new;
          }
          const bool rescale_o = mine > 0 && __any_sync(0xffffffffu, resc);
          const float mu = (m == -INFINITY) ? 0.f : m;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nmux2 = f2_pack(-mu, -mu);
          uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            const int half = NH - 1 - k;  // the last ones are in registers
            if (k > 0) load_scores(half);
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                float a, b;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c][j]), __uint_as_float(sr[c][j + 1])),
                                 sl2x2, nmux2),
                          a, b);
                a = ex2(a);
                b = ex2(b);
                // the sum takes the fp32 weights; P is rounded to bf16 for
                // the MMA (half a step, 2^-8, of each weight)
                uint64_t& lx = (j & 2) ? lb : la;
                lx = f2_add(lx, f2_pack(a, b));
                sr[c][j / 2] = pack_bf16(a, b);
              }
              tmem_st16(tP + 16 * (C * half + c),
                        *reinterpret_cast<const uint32_t(*)[16]>(&sr[c][0]));
            }
          }
          {
            float a, b;
            f2_unpack(f2_add(la, lb), a, b);
            l += a + b;
          }
          if (rescale_o) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * c, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st32(tO + 32 * c, o);
            }
          }
          tmem_st_wait();
        }
        if (!L::Q8 && tail && !(PAIR && s == 1)) {
          // One V row per thread: zero past the last token, zero NaN and
          // infinities of drafts.  (Not before this tile's scores: only they
          // show that the ring slot's last tile has come and gone.)
          const uint32_t vi = PAIR ? 2 * g + 1 : g + 1 == total ? 2 * g + 1 : 2 * g + 2;
          ok = uwait(bar(L::B_KVF + vi % L::NS), (vi / L::NS) & 1);
          if (!ok) break;
          const uint32_t v0 = sb + L::KV + (vi % L::NS) * L::TILE;
          const int pos = kb + r;
          if (!it.s.everybody(pos)) {
            const bool past = it.s.nobody(pos);
#pragma unroll 1
            for (int c0 = 0; c0 < L::CH * 8; c0 += 4) {
              uint4 v[4];
              uint32_t at[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                at[k] = v0 + (c0 >> 3) * L::CHUNK + sw128_offset(r, (c0 & 7) + k);
                v[k] = past ? make_uint4(0, 0, 0, 0) : ld_shared_v4(at[k]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool bad = not_finite2(v[k].x) || not_finite2(v[k].y) ||
                                 not_finite2(v[k].z) || not_finite2(v[k].w);
                if (bad) bad_parts[part & 7] = part;
                if (bad || past)
                  st_shared_v4(at[k], finite2(v[k].x), finite2(v[k].y), finite2(v[k].z),
                               finite2(v[k].w));
              }
            }
          }
          fence_async_smem();
        }
        if (owe_x2) {  // O of the last part has been read
          ok = uwait(bar(L::B_X2), (part - 1) & 1);
          if (!ok) break;
          owe_x2 = false;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_PF + s));
        cnt ^= 1;
        ++mine;
      }
      if (!ok) break;
      // ---------------------------------------------------- end of a part
      if (!PAIR && s == 1) {
        if (owe_x2) ok = uwait(bar(L::B_X2), (part - 1) & 1);
        if (!ok) break;
        ml[r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_X1));
        owe_x2 = true;
        continue;
      }
      if (!PAIR) {
        ok = uwait(bar(L::B_OF), part & 1);
      } else if (mine_all) {
        ok = uwait(bar(s ? L::B_OF1 : L::B_OF), (cnt >> 1) & 1);
        cnt ^= 2;
      }
      if (ok && !PAIR) ok = uwait(bar(L::B_X1), part & 1);
      if (!ok) break;
      tc_fence_after();
      if (busy) {
        int other = 0;  // the other warpgroup's tiles of this part
        float a0 = 1.f, a1 = 0.f;
        if (!PAIR) {
          other = it.t1 - it.t0 - mine;
          const float2 x = ml[r];
          const float mm = fmaxf(m, x.x), mu = mm == -INFINITY ? 0.f : mm;
          a0 = ex2(m - mu);
          a1 = ex2(x.x - mu);
          l = l * a0 + x.y * a1;
          m = mm;
        }
        const bool whole = it.t0 == 0 && it.t1 == it.s.tiles;
        const bool has = valid && !(l == 0.f);  // a NaN sum stays one
        const float inv = has ? 1.f / l : 0.f;
        const size_t orow = (static_cast<size_t>(it.b) * p.Hkv + hkv) * p.rows + row;
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (it.t0 == 0 ? 1 : 0);
        const size_t prow = slot * p.slot_rows + (PAIR ? s * kTile : 0) + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0.f;
          if (mine > 0) {
            tmem_ld32(tO + 32 * c, x);
            tmem_ld_wait();
            reg_fence(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(x[j]) * a0;
          }
          if (other > 0) {
            tmem_ld32(tO + D + 32 * c, x);
            tmem_ld_wait();
            reg_fence(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(x[j]), a1, o[j]);
          }
          if (!L::Q8) {
            // through shared memory, so that a store writes whole pieces of
            // rows: 4 rows of 128 bytes (parts) or 8 of 64 (results)
            const uint32_t out = sb + L::OUT + (warp - 2) * 4096;
            const int rows_here = min(32, p.rows - row0 - q4 * 32);
            if (whole) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const float* y = &o[8 * v];
                st_shared_v4(out + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4),
                             has ? pack_bf16(y[0] * inv, y[1] * inv) : 0u,
                             has ? pack_bf16(y[2] * inv, y[3] * inv) : 0u,
                             has ? pack_bf16(y[4] * inv, y[5] * inv) : 0u,
                             has ? pack_bf16(y[6] * inv, y[7] * inv) : 0u);
              }
              __syncwarp();
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const int j = 8 * v + (lane >> 2), piece = lane & 3;
                const uint4 y = ld_shared_v4(out + j * 64 + ((piece ^ ((j >> 1) & 3)) << 4));
                if (j < rows_here)
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (orow - lane + j) * D +
                                            32 * c + 8 * piece) = y;
              }
            } else {
#pragma unroll
              for (int v = 0; v < 8; ++v)
                st_shared_v4(out + sw128_offset(lane, v), __float_as_uint(o[4 * v]),
                             __float_as_uint(o[4 * v + 1]), __float_as_uint(o[4 * v + 2]),
                             __float_as_uint(o[4 * v + 3]));
              __syncwarp();
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                const int j = 4 * v + (lane >> 3), piece = lane & 7;
                const uint4 y = ld_shared_v4(out + sw128_offset(j, piece));
                if (j < rows_here)
                  *reinterpret_cast<uint4*>(p.part_o + (prow - lane + j) * D + 32 * c + 4 * piece) = y;
              }
            }
            __syncwarp();
          } else if (row < p.rows) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * D + 32 * c);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const float* y = &o[8 * v];
                uint4 w = make_uint4(0, 0, 0, 0);
                if (has)
                  w = make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                                 pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
                dst[v] = w;
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + 32 * c);
#pragma unroll
              for (int v = 0; v < 8; ++v)
                dst[v] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
          }
        }
        if (row < p.rows) {
          if (whole)
            p.lse[orow] = has ? (m + lg2(l)) * kLn2 : -INFINITY;
          else
            p.part_ml[prow] = make_float2(valid ? m : -INFINITY, valid ? l : 0.f);
        }
        __syncwarp();  // rows were written by other lanes of the warp
        if (valid && bad_parts[part & 7] == part)
          add_not_finite<D, FMT, WIN>(p, it.b, hkv, it.s, t, it.t0, it.t1,
                                      whole ? static_cast<uint16_t*>(p.o) + orow * D : nullptr,
                                      whole ? nullptr : p.part_o + prow * D);
      }
      if (!PAIR) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_X2));
      }
    }
    if (warp == 2 && lane == 0) note_join(p, run, it, blockIdx.x);
  } else if (L::Q8) {
    // ------------------------------------------------------ widening
    // 16 stored bytes per lane and step: two 8-byte loads, two 16-byte
    // stores.  Which half comes first alternates (`sel`) so that the lanes
    // of an access fall on different banks.
    constexpr int LPR = D / 16, RPI = 32 / LPR;  // lanes per row, rows per step
    constexpr int BATCH = 4;                     // rows of a lane on their way together
    const int cw = (warp - 11) % kConvTeam, u = lane % LPR, rl = lane / LPR;
    const bool isv = warp - 11 >= kConvTeam;
    bool ok = true;
    constexpr uint32_t N = L::Q8 ? L::NR / 2 : 1;
    const uint32_t total = run.left;
    for (uint32_t g = 0; ok && g < total; ++g) {
      const uint32_t idx = ring_place<PAIR>(g, total, isv);
      const uint32_t rs = g % N + (isv ? N : 0), ds = idx % L::NS, dr = idx / L::NS;
      ok = uwait(bar(L::B_RF + rs), (g / N) & 1);
      if (ok && dr > 0) ok = uwait(bar(L::B_KVE + ds), (dr - 1) & 1);
      if (!ok) break;
      const uint32_t raw = sb + L::RW + rs * L::RAW, sc = sb + L::SC + rs * kTile;
      const uint32_t dst = sb + L::KV + ds * L::TILE + (D == 128 ? (u >> 2) * L::CHUNK : 0);
      const uint4 note = ld_shared_v4(sb + L::NOTE + rs * 32);
      uint4 edges = make_uint4(0, 0, 0, 0);  // sinks, lo, edge (see SeqLen) from the tile's first key
      if (WIN) edges = ld_shared_v4(sb + L::NOTE + rs * 32 + 16);
      const int sinks = static_cast<int>(edges.x), lo = static_cast<int>(edges.y),
                edge = static_cast<int>(edges.z);
      const int nval = static_cast<int>(note.x), ndraft = static_cast<int>(note.y);
      const int part = static_cast<int>(note.z), c0 = 2 * (u & 3);
      // drafts or the end in this tile (WIN: or an edge of the window)
      const bool check = isv && (ndraft < kTile || (WIN && edge > 0 && sinks < kTile));
#pragma unroll 1
      for (int r0 = cw * RPI; r0 < kTile; r0 += BATCH * kConvTeam * RPI) {
        uint2 w[BATCH][2];
        uint32_t byte[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int row = r0 + i * kConvTeam * RPI + rl;
          const int sel = D == 128 ? ((u >> 2) ^ row) & 1 : (row >> 1) & 1;
          const uint32_t a = raw + row * D + 16 * u;
          w[i][0] = ld_shared_v2(a + 8 * sel);
          w[i][1] = ld_shared_v2(a + 8 * (sel ^ 1));
          byte[i] = ld_shared_u8(sc + row);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int row = r0 + i * kConvTeam * RPI + rl;
          const int sel = D == 128 ? ((u >> 2) ^ row) & 1 : (row >> 1) & 1;
          const RowScale scale = widen_scale<FMT>(byte[i]);
          uint4 y0, y1;
          widen4<FMT>(w[i][0].x, scale, y0.x, y0.y);
          widen4<FMT>(w[i][0].y, scale, y0.z, y0.w);
          widen4<FMT>(w[i][1].x, scale, y1.x, y1.y);
          widen4<FMT>(w[i][1].y, scale, y1.z, y1.w);
          if (check && (row >= ndraft || (WIN && row >= sinks && row < edge))) {
            const bool past = row >= nval || (WIN && row >= sinks && row < lo);
            const bool bad = !past && byte[i] == kScaleNan;
            if (bad) bad_parts[part & 7] = part;
            if (bad || past) y0 = y1 = make_uint4(0, 0, 0, 0);
          }
          st_shared_v4(dst + sw128_offset(row, c0 + sel), y0.x, y0.y, y0.z, y0.w);
          st_shared_v4(dst + sw128_offset(row, c0 + (sel ^ 1)), y1.x, y1.y, y1.z, y1.w);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::B_KVF + ds));
        mbar_arrive(bar(L::B_RE + rs));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of problems that more than one CTA worked on: one warp per
// row, one row of blocks per CTA of the main kernel, for the problem that
// CTA began and did not end (its parts are its own last and the first ones
// of the CTAs behind it).
// O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the parts i.
template <int D>
__global__ void __launch_bounds__(256) fa_tree_join_kernel(const TreeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, c = blockIdx.y;
  const int2 j = p.joins[c];
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int bh = j.x / p.groups, row = (j.x - bh * p.groups) * 2 * kTile + r;
  if (j.y == 0 || r >= p.slot_rows || row >= p.rows) return;
  auto at = [&](int i) {  // row of part i
    return static_cast<size_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * p.slot_rows + r;
  };
  float2 first = make_float2(-INFINITY, 0.f);  // part `lane`
  if (lane < j.y) first = p.part_ml[at(lane)];
  float M = first.x;
  for (int i = 32 + lane; i < j.y; i += 32) M = fmaxf(M, p.part_ml[at(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  float l = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  for (int i0 = 0; i0 < j.y; i0 += 32) {
    float2 x = first;
    if (i0 > 0) {
      x = make_float2(-INFINITY, 0.f);
      if (i0 + lane < j.y) x = p.part_ml[at(i0 + lane)];
    }
    // a part in which the row saw nothing counts nothing, whatever it holds
    const float a = x.y == 0.f ? 0.f : ex2(x.x - mu);
    l = fmaf(x.y, a, l);  // summed over the lanes below
    const uint32_t use = __ballot_sync(0xffffffffu, x.y != 0.f);
    const int m = min(32, j.y - i0);
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float ai = __shfl_sync(0xffffffffu, a, i);
      const float* y = p.part_o + at(i0 + i) * D + lane * E;
      float v[E];
      if (E == 4)
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(y);
      else
        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(y);
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] = (use >> i) & 1u ? fmaf(v[k], ai, o[k]) : o[k];
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const bool has = !(l == 0.f);
  const float inv = has ? 1.f / l : 0.f;
  const size_t gr = static_cast<size_t>(bh) * p.rows + row;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + gr * D + lane * E);
#pragma unroll
  for (int i = 0; i < E; i += 2) dst[i / 2] = has ? pack_bf16(o[i] * inv, o[i + 1] * inv) : 0u;
  if (lane == 0) p.lse[gr] = has ? (M + lg2(l)) * kLn2 : -INFINITY;
}

// Rows of a part: one group of up to 128 (split) or 256 (pair) rows.
int slot_rows(int rows) {
  const int most = rows > kTile ? 2 * kTile : kTile;
  return rows < most ? rows : most;
}

constexpr size_t kJoinBytes = 2 * kMaxGrid * sizeof(int2);  // a multiple of 256
size_t tree_ml_bytes(int rows) {
  return align256(2ull * most_ctas(rows) * slot_rows(rows) * sizeof(float2));
}
size_t tree_ws_bytes(int H, int Hkv, int T, int d) {
  const int rows = H / Hkv * T;
  return kJoinBytes + tree_ml_bytes(rows) +
         align256(2ull * most_ctas(rows) * slot_rows(rows) * d * sizeof(float));
}

cudaError_t launch_join(const TreeParams& p, int d, int grid, cudaStream_t stream) {
  // tables of one tile: every problem is one unit, nothing to join
  if (p.whole || p.cluster || most_tiles(p) == 1) return cudaSuccess;
  const dim3 blocks((p.slot_rows + 7) / 8, grid);
  return d == 64 ? launch_pdl(fa_tree_join_kernel<64>, blocks, dim3(256), 0, stream, p)
                 : launch_pdl(fa_tree_join_kernel<128>, blocks, dim3(256), 0, stream, p);
}

template <int D, int FMT, bool PAIR, bool WIN>
cudaError_t launch_tree_mode(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t stream) {
  using L = TreeSmem<D, FMT, PAIR>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_attr_once(
      attr_done, reinterpret_cast<const void*>(fa_tree_kernel<D, FMT, PAIR, WIN>), L::ALLOC);
  if (e != cudaSuccess) return e;
  const int grid = tree_grid(p, sm_count());
  if (grid <= 0) return cudaErrorInvalidDevice;
  e = launch_pdl(fa_tree_kernel<D, FMT, PAIR, WIN>, dim3(grid), dim3(L::THREADS), L::ALLOC, stream,
                 tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  return launch_join(p, D, grid, stream);
}

template <int D, int FMT>
cudaError_t launch_tree(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t stream) {
  if (p.window)
    return p.pair ? launch_tree_mode<D, FMT, true, true>(p, tq, tk, tv, stream)
                  : launch_tree_mode<D, FMT, false, true>(p, tq, tk, tv, stream);
  return p.pair ? launch_tree_mode<D, FMT, true, false>(p, tq, tk, tv, stream)
                : launch_tree_mode<D, FMT, false, false>(p, tq, tk, tv, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_tree_attention_workspace_size(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || T < 1 || d < 1 || Hkv > H || H % Hkv != 0) return 0;
  return fa::tree_ws_bytes(H, Hkv, T, d);
}

}  // extern "C"

namespace fa {
namespace {
// Both entry points; window 0: none.
fa_status tree_attention(const void* q, const void* k_cache, const void* v_cache,
                         const uint8_t* k_scale, const uint8_t* v_scale, const int* page_table,
                         const int* hist_lens, const int* draft_lens, const uint32_t* tree_mask,
                         void* o, float* lse, int format, int B, int H, int Hkv, int T, int d,
                         int num_pages, int page_size, int max_pages, float scale, int window,
                         int sinks, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
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
  FA_TRY(check_ws(workspace, workspace_bytes, tree_ws_bytes(H, Hkv, T, d)));
  TreeParams p = {};
  p.kc = k_cache;
  p.vc = v_cache;
  p.ks = k_scale;
  p.vs = v_scale;
  p.page_table = page_table;
  p.hist = hist_lens;
  p.drafts = draft_lens;
  p.mask = tree_mask;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hkv = Hkv;
  p.T = T;
  p.rows = H / Hkv * T;
  p.pair = p.rows > kTile ? 1 : 0;
  p.groups = p.pair ? (p.rows + 2 * kTile - 1) / (2 * kTile) : 1;
  p.slot_rows = slot_rows(p.rows);
  char* ws = static_cast<char*>(workspace);
  p.joins = reinterpret_cast<int2*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + kJoinBytes);
  p.part_o = reinterpret_cast<float*>(ws + kJoinBytes + tree_ml_bytes(p.rows));
  p.num_pages = num_pages;
  p.log_page = log2_page(page_size);
  p.max_pages = max_pages;
  p.words = (T + 31) / 32;
  p.window = window;
  p.sinks = sinks;
  p.scale = scale;
  if (window) split_window(&p, format, d, sm_count());
  // units (TreeParams, find_run) are counted in 32 bits
  if (static_cast<long long>(B) * Hkv * p.groups > ((1LL << 31) - 1) / most_tiles(p))
    return FA_ERR_UNSUPPORTED;
  fa_status st = FA_OK;
  p.err = status_word(&st);
  if (!p.err) return st;
  p.wait_ns = wait_limit_ns();
  CUtensorMap tq, tk, tv;
  if (tree_few_rows(p.rows, format)) {
    if (!make_cache_map(&tk, k_cache, num_pages * Hkv, page_size, d, format != kCacheBf16) ||
        !make_cache_map(&tv, v_cache, num_pages * Hkv, page_size, d, format != kCacheBf16))
      return FA_ERR_CUDA;
    const int grid = tree_grid(p, sm_count() * few_ctas(p.rows, format, d));
    if (grid <= 0) return FA_ERR_CUDA;
    FA_CUDA(launch_tree_few(p, format, d, tk, tv, grid, stream));
    FA_CUDA(launch_join(p, d, grid, stream));
    return FA_OK;
  }
  if (!make_tile_map(&tq, q, B * Hkv, p.rows, d)) return FA_ERR_CUDA;
  if (format == kCacheBf16) {
    if (!make_tile_map(&tk, k_cache, num_pages * Hkv, page_size, d, page_size) ||
        !make_tile_map(&tv, v_cache, num_pages * Hkv, page_size, d, page_size))
      return FA_ERR_CUDA;
  } else {
    tk = tv = tq;  // not read: stored bytes come by untiled copies
  }
  if (d == 64)
    FA_CUDA(format == kCacheBf16   ? (launch_tree<64, kCacheBf16>(p, tq, tk, tv, stream))
            : format == kCacheE4m3 ? (launch_tree<64, kCacheE4m3>(p, tq, tk, tv, stream))
                                   : (launch_tree<64, kCacheInt8>(p, tq, tk, tv, stream)));
  else
    FA_CUDA(format == kCacheBf16   ? (launch_tree<128, kCacheBf16>(p, tq, tk, tv, stream))
            : format == kCacheE4m3 ? (launch_tree<128, kCacheE4m3>(p, tq, tk, tv, stream))
                                   : (launch_tree<128, kCacheInt8>(p, tq, tk, tv, stream)));
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                            const uint8_t* k_scale, const uint8_t* v_scale, const int* page_table,
                            const int* hist_lens, const int* draft_lens, const uint32_t* tree_mask,
                            void* o, float* lse, int format, int B, int H, int Hkv, int T, int d,
                            int num_pages, int page_size, int max_pages, float scale,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return fa::tree_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, hist_lens,
                            draft_lens, tree_mask, o, lse, format, B, H, Hkv, T, d, num_pages,
                            page_size, max_pages, scale, 0, 0, workspace, workspace_bytes, stream);
}

fa_status fa_tree_attention_window(const void* q, const void* k_cache, const void* v_cache,
                                   const uint8_t* k_scale, const uint8_t* v_scale,
                                   const int* page_table, const int* hist_lens,
                                   const int* draft_lens, const uint32_t* tree_mask, void* o,
                                   float* lse, int format, int B, int H, int Hkv, int T, int d,
                                   int num_pages, int page_size, int max_pages, float scale,
                                   int window, int sinks, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  // a mask's drafts all lie within the window
  if (sinks > 1024 || (tree_mask && T > window)) return FA_ERR_UNSUPPORTED;
  // positions stay below 2^30: no window is longer
  return fa::tree_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, hist_lens,
                            draft_lens, tree_mask, o, lse, format, B, H, Hkv, T, d, num_pages,
                            page_size, max_pages, scale, window < (1 << 30) ? window : 1 << 30,
                            sinks, workspace, workspace_bytes, stream);
}

}  // extern "C"
