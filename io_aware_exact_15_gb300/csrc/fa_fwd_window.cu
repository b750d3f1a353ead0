// Forward pass over long batches with a sliding window: the two-tile form of
// fa_fwd.cu as a persistent kernel.
//
// A window's walk is short (window / 128 + 2 key tiles), so a CTA that does
// one walk spends much of its life starting and ending: tensor memory, first
// loads, the last product, O on its way out.  Here one CTA per SM takes
// units (two 128-row query tiles of a head) in turn and nothing stops between
// them: the loading warp runs ahead into the next unit's Q, K and V, the
// issuing warp puts its first products behind this one's last, and while one
// softmax warpgroup writes O the other's products keep the tensor core busy.
//   warp 0      TMA: Q_s of each unit as soon as the last S_s product has read
//               the previous one, K_j and V_j through a ring
//   warp 1      issues S_s = Q_s K_j^T and O_s += P_s V_j (as fa_fwd.cu)
//   warps 2-5   softmax and output of the unit's query tile 0, warps 6-9 of 1
// An O_s that has been read is known by the next unit's first P_s, whose
// threads read it.  Rows go out through 2 KB of shared memory per warp, whole
// 64-byte pieces.
//MEASURED
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_sched.cuh"
#include "fa_window.cuh"

namespace fa {
namespace {

template <int D>
struct FwdWinSmem {
  static constexpr int CH = D / 64;          // 128-byte column chunks per row
  static constexpr int CHUNK = kTile * 128;  // [128 rows x 128 B] = 16 KB
  static constexpr int TILE = CH * CHUNK;    // one 128 x D bf16 tile
  static constexpr int NS = D == 64 ? 8 : 4;  // ring of K and V tiles
  static constexpr int THREADS = 320;
  static constexpr int Q = 0;
  static constexpr int KV = Q + 2 * TILE;
  static constexpr int OUT = KV + NS * TILE;  // 32 rows x 64 B of each softmax warp
  static constexpr int BAR = OUT + 8 * 2048;
  static constexpr int B_QF = 0, B_QE = 2, B_SF = 4, B_PF = 6, B_OF = 8, B_FIN = 10, B_KVF = 11,
                       B_KVE = B_KVF + NS, NBAR = B_KVE + NS;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int T_O = 2 * kTile;           // TMEM: S0 S1 O0 O1
  static constexpr int ALLOC = MISC + 16 + 1024;  // + slack for 1024-byte alignment
  static_assert(ALLOC <= 232448, "shared memory budget");
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;  // lazy rescale threshold (factor 256)

// The units of a CTA, tile by tile: every role walks the same.
struct UnitWalk {
  FwdScheduleT<kTile, true> sch;
  int u, N, row0, zq, zkv;
  int seen;  // query tiles that have had a key tile
  FA_DEV void begin() { u = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x); }
  FA_DEV bool unit(const FwdParams& p) {
    const int BH = p.B * p.H, npairs = ((p.N + kTile - 1) / kTile + 1) / 2;
    while ((u += gridDim.x) < npairs * BH) {
      // the pairs at a sequence's begin, whose walks are short, come last
      const int v = u / BH, bh = u - v * BH, pair = npairs - 1 - v, b = bh / p.H;
      const int head = bh - b * p.H;
      N = p.N;
      row0 = 0;
      zq = bh;
      if (p.cu_seqlens) {
        const int a = min(max(p.cu_seqlens[b], 0), p.total);
        const int e = min(max(p.cu_seqlens[b + 1], a), p.total);
        row0 = a;
        N = min(e - a, p.N);
        zq = head;
        if (2 * pair * kTile >= N) continue;
      }
      zkv = zq / (p.H / p.Hkv);
      sch.init(pair, (N + kTile - 1) / kTile, true, p.lists, 0);
      sch.reach(p.window, p.sinks, N);
      seen = 0;
      return true;
    }
    return false;
  }
};

// One key tile of a walk: `mem` has the query tiles that it is for, `first`
// those for which it is their first, `last` their last.
struct Step {
  int kt, mem, first, last;
};
FA_DEV bool next_step(UnitWalk& w, Step& t) {
  if (!w.sch.next(t.kt, t.mem)) return false;
  t.first = t.mem & ~w.seen;
  w.seen |= t.mem;
  t.last = t.mem & ((t.kt == w.sch.qt[0] ? 1 : 0) | (t.kt == w.sch.qt[1] ? 2 : 0));
  return true;
}

template <int D>
__global__ void __launch_bounds__(FwdWinSmem<D>::THREADS, 1)
    fa_fwd_window_kernel(const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const FwdParams p) {
  using L = FwdWinSmem<D>;
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + L::BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::B_QF + s), 1);
      mbar_init(bar(L::B_QE + s), 1);
      mbar_init(bar(L::B_SF + s), 1);
      mbar_init(bar(L::B_PF + s), 128);
      mbar_init(bar(L::B_OF + s), 1);
    }
    mbar_init(bar(L::B_FIN), 1);
    for (int s = 0; s < L::NS; ++s) {
      mbar_init(bar(L::B_KVF + s), 1);
      mbar_init(bar(L::B_KVE + s), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err, p.wait_ns};
  UnitWalk w;
  w.begin();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t idx = 0, nq[2] = {0, 0};
      bool ok = true;
      auto load_q = [&](int s) {
        if (nq[s] > 0 && !wait_bar(bar(L::B_QE + s), (nq[s] - 1) & 1, wc)) return false;
        mbar_arrive_expect_tx(bar(L::B_QF + s), L::TILE);
#pragma unroll
        for (int c = 0; c < L::CH; ++c)
          tma_load_3d(sb + L::Q + s * L::TILE + c * L::CHUNK, &tq, bar(L::B_QF + s), 64 * c,
                      w.row0 + w.sch.qt[s] * kTile, w.zq);
        ++nq[s];
        return true;
      };
      auto load_kv = [&](const CUtensorMap* m, int kt) {
        const int pos = idx % L::NS;
        const uint32_t round = idx / L::NS;
        if (round > 0 && !wait_bar(bar(L::B_KVE + pos), (round - 1) & 1, wc)) return false;
        mbar_arrive_expect_tx(bar(L::B_KVF + pos), L::TILE);
#pragma unroll
        for (int c = 0; c < L::CH; ++c)
          tma_load_3d(sb + L::KV + pos * L::TILE + c * L::CHUNK, m, bar(L::B_KVF + pos), 64 * c,
                      w.row0 + kt * kTile, w.zkv);
        ++idx;
        return true;
      };
      while (ok && w.unit(p)) {
        // in the order of their use: Q_0, the first K, Q_1, the first V
        bool begin = true;
        Step t;
        while (ok && next_step(w, t)) {
          if (begin) ok = load_q(0);
          ok = ok && load_kv(&tk, t.kt);
          if (begin && w.sch.act[1]) ok = ok && load_q(1);
          ok = ok && load_kv(&tv, t.kt);
          begin = false;
        }
      }
      // let copies still in flight land before the CTA can exit
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) drain_bar(bar(L::B_QF + s), (nq[s] - 1) & 1, p.wait_ns);
      for (uint32_t j = idx > static_cast<uint32_t>(L::NS) ? idx - L::NS : 0; j < idx; ++j)
        drain_bar(bar(L::B_KVF + j % L::NS), (j / L::NS) & 1, p.wait_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    // (the whole warp: waits are votes, so that control flow is uniform)
    auto uwait = [&](uint32_t b, uint32_t ph) {
      return __all_sync(0xffffffffu, wait_bar(b, ph, wc));
    };
    auto ecommit = [&](uint32_t b) {
      if (elect_one()) mma_commit(b);
    };
    constexpr uint32_t idS = idesc_bf16(128, kTile, false, false);
    constexpr uint32_t idO = idesc_bf16(128, D, false, true);
    const uint64_t dq0 = desc_sw128(sb + L::Q, 16, 1024);
    const uint64_t dkv0 = desc_sw128(sb + L::KV, 16, 1024);       // K-major ring slot 0
    const uint64_t dv0 = desc_sw128(sb + L::KV, L::CHUNK, 1024);  // MN-major ring slot 0
    uint32_t nq[2] = {0, 0}, np[2] = {0, 0};  // Q tiles, P tiles waited for
    uint32_t idx = 0;
    // S_s of step t, K in ring slot kpos
    auto issue_s = [&](int s, const Step& t, int kpos) {
      if (t.first & (1 << s)) {
        if (!uwait(bar(L::B_QF + s), nq[s] & 1)) return false;
        ++nq[s];
        tc_fence_after();
      }
      const uint64_t qa = desc_advance(dq0, s * L::TILE);
      const uint64_t kb = desc_advance(dkv0, kpos * L::TILE);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * L::CHUNK + (kk & 3) * 32;
        if (elect_one())
          mma_bf16_ss(tmem + s * kTile, desc_advance(qa, off), desc_advance(kb, off), idS, kk > 0);
      }
      ecommit(bar(L::B_SF + s));
      if (t.last & (1 << s)) ecommit(bar(L::B_QE + s));
      return true;
    };
    // O_s += P_s V: P_s in TMEM over S_s, V MN-major in shared memory
    auto issue_pv = [&](int s, int vpos, bool acc) {
      const uint64_t vb = desc_advance(dv0, vpos * L::TILE);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        if (elect_one())
          mma_bf16_ts(tmem + L::T_O + s * D, tmem + s * kTile + kk * 8,
                      desc_advance(vb, kk * 2048), idO, (acc || kk > 0) ? 1u : 0u);
    };
    // the next step, of the next unit where this one is at its end
    auto next = [&](Step& t) {
      if (next_step(w, t)) return true;
      return w.unit(p) && next_step(w, t);
    };
    Step t, tn;
    bool ok = true, have = w.unit(p) && next_step(w, t);
    if (have) {
      ok = uwait(bar(L::B_KVF), 0);
      tc_fence_after();
      for (int s = 0; s < 2; ++s)
        if (ok && (t.mem & (1 << s))) ok = issue_s(s, t, 0);
      ecommit(bar(L::B_KVE));
      ++idx;
    }
    while (ok && have) {
      const bool have_n = next(tn);
      const int vpos = idx % L::NS;
      if (!(ok = uwait(bar(L::B_KVF + vpos), (idx / L::NS) & 1))) break;
      ++idx;
      tc_fence_after();
      int kpos = -1;
      for (int s = 0; s < 2; ++s) {
        if (t.mem & (1 << s)) {
          if (!(ok = uwait(bar(L::B_PF + s), np[s] & 1))) break;
          ++np[s];
          tc_fence_after();
          issue_pv(s, vpos, !(t.first & (1 << s)));
          if (t.last & (1 << s)) ecommit(bar(L::B_OF + s));
        }
        if (have_n && (tn.mem & (1 << s))) {
          if (kpos < 0) {
            kpos = idx % L::NS;
            if (!(ok = uwait(bar(L::B_KVF + kpos), (idx / L::NS) & 1))) break;
            tc_fence_after();
          }
          if (!(ok = issue_s(s, tn, kpos))) break;
        }
      }
      if (!ok) break;
      ecommit(bar(L::B_KVE + vpos));
      if (kpos >= 0) {
        ecommit(bar(L::B_KVE + kpos));
        ++idx;
      }
      t = tn;
      have = have_n;
    }
    // every MMA issued above completes before this fires
    ecommit(bar(L::B_FIN));
    drain_bar(bar(L::B_FIN), 0, p.wait_ns);
  } else {
    // ------------------------------------------------------ softmax warps
    const int s = (warp - 2) >> 2;
    const int q4 = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + s * kTile;
    const uint32_t tO = tmem + lane_off + L::T_O + s * D;
    const float sl2 = p.scale * kLog2e;
    const size_t slice_rows = p.cu_seqlens ? p.total : p.N;
    const uint32_t stg = sb + L::OUT + (warp - 2) * 2048;
    uint32_t cnt = 0, units = 0;
    bool ok = true;
    while (ok && w.unit(p)) {
      if (!w.sch.act[s]) continue;
      const int N = w.N, qt = w.sch.qt[s], qrow = qt * kTile + q4 * 32 + lane;
      float m = -INFINITY, l = 0.f;
      Step t;
      while (next_step(w, t)) {
        if (!(t.mem & (1 << s))) continue;
        ok = __all_sync(0xffffffffu, wait_bar(bar(L::B_SF + s), cnt & 1, wc));
        if (!ok) break;
        ++cnt;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence(sr[c]);
        const int kbase = t.kt * kTile;
        // the diagonal, the end, or some row's window begins behind the
        // tile's first key and not all are sinks
        if (kbase + kTile > N || t.kt == qt ||
            (kbase < qt * kTile + kTile - p.window && kbase + kTile > p.sinks)) {
          const int lim = min(N, qrow + 1) - kbase, lo = qrow - p.window + 1 - kbase;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t vis = reach_bits(lim - 32 * c, lo - 32 * c, p.sinks - kbase - 32 * c);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((vis >> j) & 1u)) sr[c][j] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; j += 2)  // two scores per three-input max
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mx[c] = fmax3(mx[c], __uint_as_float(sr[c][j]), __uint_as_float(sr[c][j + 1]));
        const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2);
        const bool resc = m_new > m + kRescaleLog2;
        const float alpha = resc ? ex2(m - m_new) : 1.f;
        if (resc) {
          l *= alpha;
          m = m_new;
        }
        const bool rescale_o = !(t.first & (1 << s)) && __any_sync(0xffffffffu, resc);
        const float mu = (m == -INFINITY) ? 0.f : m;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nmux2 = f2_pack(-mu, -mu);
        uint64_t lw[2] = {0ull, 0ull};  // row sums of the fp32 weights
        // P (bf16) overwrites the first 64 columns of S, which are in registers
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[q][2 * i]),
                                     __uint_as_float(sr[q][2 * i + 1])),
                             sl2x2, nmux2),
                      a, b);
            a = ex2(a);
            b = ex2(b);
            lw[i & 1] = f2_add(lw[i & 1], f2_pack(a, b));
            sr[q][i] = pack_bf16(a, b);
          }
          tmem_st16(tS + 16 * q, *reinterpret_cast<const uint32_t(*)[16]>(&sr[q][0]));
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
        float l0, l1;
        f2_unpack(f2_add(lw[0], lw[1]), l0, l1);
        l += l0 + l1;
        tc_fence_before();
        mbar_arrive(bar(L::B_PF + s));
      }
      // ---------------------------------------------------- epilogue
      if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(L::B_OF + s), units & 1, wc));
      ++units;
      if (!ok) break;
      tc_fence_after();
      const int qrow0 = qrow - lane, nrows = min(32, N - qrow0);  // this warp's rows
      const size_t first = static_cast<size_t>(w.zq) * slice_rows + w.row0;
      uint8_t* obase = static_cast<uint8_t*>(p.o) + (first + qrow0) * D * 2;
      const bool store = qrow < N, has = l > 0.f;
      const float inv = has ? 1.f / l : 0.f;
      float odd = 0.f;  // NaN once a number of the row is not finite
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_ld_wait();
        reg_fence(o);
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          x[j] = __uint_as_float(o[j]) * inv;
          odd = fmaf(x[j], 0.f, odd);
        }
        // row `lane`, 16-byte piece v; 8 lanes on 8 different bank groups
#pragma unroll
        for (int v = 0; v < 4; ++v)
          st_shared_v4(stg + 64 * lane + 16 * (v ^ ((lane >> 1) & 3)),
                       pack_bf16(x[8 * v], x[8 * v + 1]), pack_bf16(x[8 * v + 2], x[8 * v + 3]),
                       pack_bf16(x[8 * v + 4], x[8 * v + 5]),
                       pack_bf16(x[8 * v + 6], x[8 * v + 7]));
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int j = 8 * it + (lane >> 2), v = lane & 3;
          const uint4 y = ld_shared_v4(stg + 64 * j + 16 * (v ^ ((j >> 1) & 3)));
          if (j < nrows)
            *reinterpret_cast<uint4*>(obase + static_cast<size_t>(j) * D * 2 + c * 64 + v * 16) = y;
        }
        __syncwarp();
      }
      tc_fence_before();  // (ordered before the next unit's P)
      const float lse2 = m + lg2(l);
      if (store) p.lse[first + qrow] = has ? lse2 * kLn2 : -INFINITY;
      // (a NaN logsumexp: the row sees a key whose score is one)
      uint32_t again = __ballot_sync(0xffffffffu, store && has && odd != 0.f && lse2 == lse2);
      for (; again; again &= again - 1) {  // the rows were written by all lanes
        const int j = __ffs(again) - 1;
        __syncwarp();
        window_row_o<D>(p.q, p.k, p.v, p.o, first, static_cast<size_t>(w.zkv) * slice_rows + w.row0,
                        qrow0 + j, p.window, p.sinks, sl2, __shfl_sync(0xffffffffu, lse2, j));
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

template <int D>
cudaError_t launch(const FwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tv, cudaStream_t stream) {
  using L = FwdWinSmem<D>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_attr_once(attr_done, reinterpret_cast<const void*>(fa_fwd_window_kernel<D>),
                                 L::ALLOC);
  if (e != cudaSuccess) return e;
  const long long units =
      static_cast<long long>(((p.N + kTile - 1) / kTile + 1) / 2) * p.B * p.H;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return launch_pdl(fa_fwd_window_kernel<D>, dim3(static_cast<unsigned>(units < sms ? units : sms)),
                    dim3(L::THREADS), L::ALLOC, stream, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_forward_window(const FwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, cudaStream_t stream) {
  return p.d == 64 ? launch<64>(p, tq, tk, tv, stream) : launch<128>(p, tq, tk, tv, stream);
}

}  // namespace fa
