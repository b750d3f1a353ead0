// Per-head RMS norm of queries and keys with the position rotation, in one
// pass, and its backward.
//
// For a row x of d elements with norm weights w, at position p:
//   r = (mean(x^2) + eps)^(-1/2),  y = x r w,
//   (a, b) -> (a c - b s, b c + a s) for each pair of the first `rot`
//   elements of y, c and s the cosine and sine of row p of the tables.
// Backward, with G the gradient of the result turned back by the same
// angles (the rotation's transpose) and xh = x r:
//   dw = sum over rows of G xh,   dx = r (G w - xh mean(G w xh)).
// Everything between the bf16 loads and the one bf16 rounding of the result
// is fp32; the backward forms r again from x, so the forward stores nothing.
//
// Both are bound by memory: 4 bytes per element forward (bf16 in, bf16 out),
// 6 backward.  Layout: 8 elements (16 bytes) per lane, so a row is d / 8
// lanes and a warp holds 2 (d = 128) or 4 (d = 64) rows.  The rows of a warp
// are heads of one token: they share the position, so a lane loads its
// cosines and sines once for all its rows.  The input strides are free (a
// packed [B, N, heads, d] projection is read in place) and the result is
// [B, H, N, d], which the attention entry points take.
//
// A warp takes whole tokens, eight consecutive ones to a block (so that each
// head's rows are written in longer pieces), and walks their heads a few rows
// at a time.  Loads go through a queue in shared memory (asynchronous
// copies, each lane its own 16 bytes, so nothing has to be synchronised):
// loads that wait in registers kept at most 64 KB of an SM in flight and
// lost the time between a block's loads.
//
// Measured, packed input, 16 + 4 heads of 128: forward of 4 x 4096 tokens
// 34.6 us, 5.1 TB/s (8 x 8192: 122.6 us, 5.5 TB/s; a plain copy of the 4 x
// 4096 tokens' bytes takes 29.0); backward of 4 x 4096 tokens 49.6 us,
// 5.3 TB/s.  What is left is the instructions: without the arithmetic, the
// same loads and stores take 32.5 us, and a warp's step is a chain (load,
// sum over the lanes, scale, store) that 4 warps of a scheduler do not
// cover; a third block per SM has no registers.  Addresses are stepped, not
// formed anew, and pieces behind the last head left out (39.2 us without
// both); 16 elements a lane took 35.4 us forward, and the backward spilled.
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;          // warps per block
constexpr int kMaxPartials = 1024; // blocks of the backward, at most
constexpr int kQueue = 3;          // steps of a warp on their way or in use

struct RopeTables {
  const float* cos;
  const float* sin;
  const int* positions;  // [B, N] or null (0 .. N-1)
  int rows;              // of cos and sin
  int rot;
};

struct RopeParams {
  const void *q, *k;              // bf16, strided
  Strides sq, sk;
  const float *wq, *wk;
  RopeTables t;
  void *oq, *ok;                  // forward: bf16 [B, H, N, d]
  const void *gq, *gk;            // backward: gradients of the results, [B, H, N, d]
  void *dq, *dk;                  // backward: bf16, strided
  Strides sdq, sdk;
  float* part;                    // backward: [blocks][2][d] sums of dwq, dwk
  int B, H, Hkv, N;
  float eps;
};

// 8 bf16 elements as four fp32 pairs (exact), and back (one rounding)
FA_DEV void widen(const uint4& v, uint64_t (&x)[4]) {
  x[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x));
  x[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
  x[2] = f2_pack(bf16_lo(v.z), bf16_hi(v.z));
  x[3] = f2_pack(bf16_lo(v.w), bf16_hi(v.w));
}
FA_DEV uint32_t narrow(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_bf16(a, b);
}
FA_DEV uint4 narrow(const uint64_t (&x)[4]) {
  return make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
}
// sum of the products of two rows' pieces
FA_DEV float dot8(const uint64_t (&x)[4], const uint64_t (&y)[4]) {
  float a, b;
  f2_unpack(f2_fma(x[3], y[3], f2_fma(x[2], y[2], f2_fma(x[1], y[1], f2_mul(x[0], y[0])))), a, b);
  return a + b;
}

// sums over the LPR lanes of each of U rows (step by step for all of them:
// one row's five exchanges are a chain of latencies)
template <int LPR, int U>
FA_DEV void row_sums(float (&v)[U]) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
}

// 8 fp32 numbers of shared memory as pairs
FA_DEV void load8(uint32_t at, uint64_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = ld_shared_v4(at + 16 * i);
    x[2 * i] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    x[2 * i + 1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
}

// wq, wk into shared memory (whole block)
template <int D>
FA_DEV void stage_weights(float (&w)[2][D], const float* wq, const float* wk) {
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) w[i / D][i % D] = i < D ? wq[i] : wk[i - D];
  __syncthreads();
}

// The rotation of one lane's 8 elements: y_i = c_i x_i + s_i x'_i, where x'
// is the other element of the pair and s carries the sign.  Adjacent pairs:
// x' is the neighbour in the same packed word.  Half pairs (i, i + rot / 2):
// x' sits `hop` lanes away (rot is a multiple of 16, so a half is a whole
// number of lanes).  Elements from `rot` on are their own x' with
// c = s = 1/2 (x w / 2 twice is x w to the bit; with s = 0 an infinite x'
// would make them NaN).
template <int D, bool INTER>
struct Turn {
  uint64_t c[4], s[4];
  bool in, upper;
  int partner;  // lane of x'
  int other;    // first of the elements x' (to find their weights)

  FA_DEV Turn(int rot, int lane) {
    constexpr int LPR = D / 8;
    const int e0 = 8 * (lane % LPR), hop = rot / 16;
    in = e0 < rot;
    upper = !INTER && e0 >= rot / 2;
    partner = !in || INTER ? lane : upper ? lane - hop : lane + hop;
    other = e0 + 8 * (partner - lane);
  }

  // from this lane's numbers of the tables: 8 cosines and 8 sines (adjacent
  // pairs: 4 and 4), 16 bytes at a time, `pitch` bytes apart
  template <bool BACK>
  FA_DEV void load(uint32_t at, uint32_t pitch) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = s[i] = f2_pack(0.5f, 0.5f);
    if (!in) return;
    auto four = [&](int i, uint64_t& a, uint64_t& b) {
      const uint4 v = ld_shared_v4(at + i * pitch);
      a = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
      b = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
    };
    if (INTER) {
      four(0, c[0], c[2]);
      four(1, s[0], s[2]);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float a, b;
        f2_unpack(c[i], a, b);
        c[i] = f2_pack(a, a), c[i + 1] = f2_pack(b, b);
        f2_unpack(s[i], a, b);
        if (BACK) a = -a, b = -b;
        s[i] = f2_pack(-a, a), s[i + 1] = f2_pack(-b, b);
      }
    } else {
      four(0, c[0], c[1]);
      four(1, c[2], c[3]);
      four(2, s[0], s[1]);
      four(3, s[2], s[3]);
      if (upper == BACK) {  // a' = a c - b s in the lower half, b' = b c + a s
        const uint64_t m = f2_pack(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = f2_mul(s[i], m);
      }
    }
  }

  // x' of a packed piece; all lanes of the warp
  FA_DEV uint4 swap(const uint4& v) const {
    if (INTER) {
      const uint32_t sel = in ? 0x1032u : 0x3210u;
      return make_uint4(__byte_perm(v.x, 0, sel), __byte_perm(v.y, 0, sel),
                        __byte_perm(v.z, 0, sel), __byte_perm(v.w, 0, sel));
    }
    return make_uint4(__shfl_sync(0xffffffffu, v.x, partner), __shfl_sync(0xffffffffu, v.y, partner),
                      __shfl_sync(0xffffffffu, v.z, partner),
                      __shfl_sync(0xffffffffu, v.w, partner));
  }

  // c, s times the weights of the element that each multiplies
  FA_DEV void weigh(uint32_t w, int e0) {
    uint64_t own[4], others[4];
    load8(w + 4 * e0, own);
    load8(w + 4 * other, others);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = f2_mul(c[i], own[i]);
      if (INTER && in) {
        float a, b;
        f2_unpack(own[i], a, b);
        others[i] = f2_pack(b, a);
      }
      s[i] = f2_mul(s[i], others[i]);
    }
  }
};

FA_DEV void copy16(uint32_t dst, const void* src, bool real) {
  // no bytes are read, and zeros written, where `real` is false
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
FA_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
FA_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a warp is in its tokens, `stride` apart: token (b, n), and the step
// (group of U * RPW heads, of q first).
struct Walk {
  uint32_t token, stride;
  int b, n, db, dn, step;
  FA_DEV Walk(const RopeParams& p)
      : token(blockIdx.x * kWarps + (threadIdx.x >> 5)), stride(gridDim.x * kWarps), step(0) {
    b = token / p.N;
    n = token - static_cast<uint32_t>(b) * p.N;
    db = stride / p.N;
    dn = stride - static_cast<uint32_t>(db) * p.N;
  }
  FA_DEV void advance(int N) {
    // (the sum stays below 2^32: tokens and grid are far smaller)
    token += stride;
    b += db;
    n += dn;
    if (n >= N) n -= N, ++b;
  }
};

// The queue of a warp: kQueue steps of x (and, backward, of the gradient), and
// the numbers of the tables of the last two tokens.
template <int D, bool INTER, bool BACK, int U>
struct Queue {
  static constexpr int LPR = D / 8, RPW = 32 / LPR, GRP = U * RPW;
  static constexpr int PIECES = U * (BACK ? 2 : 1);
  static constexpr int TAB = INTER ? 2 : 4;
  static constexpr int BYTES = (kQueue * PIECES + 2 * TAB) * 512;  // of a warp
  const RopeParams& p;
  uint32_t at;     // shared memory of this lane
  int nq, steps, lane, e0, sub;
  uint32_t tokens;
  Walk next;       // step to send
  uint32_t sent = 0, turn = 0;
  int pos_next = 0;            // position of the next token to send (given ones)
  int left = 0;                // heads of q or of k from this step on
  const uint16_t *x, *g;       // this lane's first piece of the step; RPW heads
  long long xh, gh;            // further on is `xh` (gradients `gh`) elements away

  FA_DEV int position(uint32_t token) const {
    return p.t.positions && token < tokens ? __ldg(p.t.positions + token) : 0;
  }

  FA_DEV Queue(const RopeParams& p_, uint32_t smem) : p(p_), next(p_) {
    lane = threadIdx.x & 31;
    at = smem + (threadIdx.x >> 5) * BYTES + lane * 16;
    e0 = 8 * (lane % LPR);
    sub = lane / LPR;
    nq = (p.H + GRP - 1) / GRP;
    steps = nq + (p.Hkv + GRP - 1) / GRP;
    tokens = static_cast<uint32_t>(p.B) * p.N;
    pos_next = position(next.token);
#pragma unroll 1
    for (int i = 0; i < kQueue - 1; ++i) send();
  }

  FA_DEV uint32_t piece(uint32_t step, int i) const {
    return at + ((step % kQueue) * PIECES + i) * 512;
  }
  FA_DEV uint32_t tables(uint32_t t) const { return at + (kQueue * PIECES + (t & 1) * TAB) * 512; }

  FA_DEV void send_tables() {
    const int pos = min(max(p.t.positions ? pos_next : next.n, 0), p.t.rows - 1);
    pos_next = position(tokens - next.token > next.stride ? next.token + next.stride : tokens);
    if (e0 < p.t.rot) {
      const size_t row = static_cast<size_t>(pos) * (p.t.rot / 2);
      const int i0 = INTER ? e0 / 2 : e0 >= p.t.rot / 2 ? e0 - p.t.rot / 2 : e0;
#pragma unroll
      for (int i = 0; i < TAB / 2; ++i) {
        copy16(tables(turn) + i * 512, p.t.cos + row + i0 + 4 * i, true);
        copy16(tables(turn) + (TAB / 2 + i) * 512, p.t.sin + row + i0 + 4 * i, true);
      }
    }
    ++turn;
  }

  // sends one step (or an empty one behind the last)
  FA_DEV void send() {
    if (next.token < tokens) {
      if (next.step == 0) send_tables();
      if (next.step == 0 || next.step == nq) {
        const bool isq = next.step == 0;
        left = isq ? p.H : p.Hkv;
        const Strides s = isq ? p.sq : p.sk;
        x = static_cast<const uint16_t*>(isq ? p.q : p.k) + next.b * s.b + next.n * s.n + e0 +
            sub * s.h;
        xh = RPW * s.h;
        if (BACK) {
          gh = static_cast<long long>(p.N) * D;
          g = static_cast<const uint16_t*>(isq ? p.gq : p.gk) +
              (static_cast<size_t>(next.b) * left * p.N + next.n) * D + e0 + sub * gh;
          gh *= RPW;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!BACK && u * RPW >= left) break;  // nobody takes the pieces behind the last head
        const bool real = u * RPW + sub < left;
        if (BACK) {  // heads past the last: zeros, for the sums
          copy16(piece(sent, u), real ? x + u * xh : p.q, real);
          copy16(piece(sent, U + u), real ? g + u * gh : p.q, real);
        } else if (real) {
          copy16(piece(sent, u), x + u * xh, true);
        }
      }
      x += U * xh;
      if (BACK) g += U * gh;
      left -= GRP;
      if (++next.step == steps) {
        next.step = 0;
        next.advance(p.N);
      }
    }
    ++sent;
    copy_commit();
  }
  FA_DEV uint4 take(uint32_t step, int i) const { return ld_shared_v4(piece(step, i)); }
};

// C pieces of a step, from piece u0: their heads' rows normed and turned.
// `o` is this lane's place in the first one's result, `oh` RPW heads.
template <int C, class Q, class T>
FA_DEV void norm_pieces(const Q& q, const T& turn, uint32_t step, int u0, uint16_t* o, size_t oh,
                        int left, float inv_d, float eps) {
  uint4 raw[C];
  uint64_t x[C][4], y[C][4];
  float r[C];
#pragma unroll
  for (int u = 0; u < C; ++u) raw[u] = q.take(step, u0 + u);
#pragma unroll
  for (int u = 0; u < C; ++u) {
    widen(raw[u], x[u]);
    r[u] = dot8(x[u], x[u]);
    widen(turn.swap(raw[u]), y[u]);
  }
  row_sums<Q::LPR>(r);
#pragma unroll
  for (int u = 0; u < C; ++u) {
    r[u] = rsqrtf(r[u] * inv_d + eps);
    const uint64_t r2 = f2_pack(r[u], r[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[u][i] = f2_mul(f2_fma(y[u][i], turn.s[i], f2_mul(x[u][i], turn.c[i])), r2);
    if ((u0 + u) * Q::RPW + q.sub < left)
      *reinterpret_cast<uint4*>(o + (u0 + u) * oh) = narrow(x[u]);
  }
}

template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32) fa_norm_rope_kernel(const RopeParams p) {
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  using Q = Queue<D, INTER, false, U>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  __shared__ __align__(16) float weights[2][D];
  Q q(p, smem_u32(rope_smem));
  stage_weights(weights, p.wq, p.wk);
  Turn<D, INTER> turn(p.t.rot, q.lane);
  Walk w(p);
  uint32_t step = 0, token_no = 0;
  const size_t oh = static_cast<size_t>(p.N) * D;
  for (; w.token < q.tokens; w.advance(p.N), ++token_no) {
    uint16_t* o = nullptr;
    int left = 0;
#pragma unroll 1
    for (w.step = 0; w.step < q.steps; ++w.step, ++step) {
      q.send();
      copy_wait<kQueue - 1>();  // this step has come
      // the weights go into the rotation's factors: out = r (c w x + s w' x')
      if (w.step == 0 || w.step == q.nq) {
        const bool isq = w.step == 0;
        turn.template load<false>(q.tables(token_no), 512);
        turn.weigh(smem_u32(weights[isq ? 0 : 1]), q.e0);
        left = isq ? p.H : p.Hkv;
        o = static_cast<uint16_t*>(isq ? p.oq : p.ok) + static_cast<size_t>(w.b) * left * oh +
            static_cast<size_t>(w.n) * D + q.e0 + q.sub * oh;
      }
      constexpr float inv_d = 1.f / D;
      if (left > (U - 1) * Q::RPW) {
        norm_pieces<U>(q, turn, step, 0, o, Q::RPW * oh, left, inv_d, p.eps);
      } else {
#pragma unroll 1
        for (int u = 0; u * Q::RPW < left; u += 2)
          norm_pieces<2>(q, turn, step, u, o, Q::RPW * oh, left, inv_d, p.eps);
      }
      o += Q::GRP * oh;
      left -= Q::GRP;
    }
  }
}

template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32) fa_norm_rope_back_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  using Q = Queue<D, INTER, true, U>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  __shared__ float sums[kWarps][D];
  __shared__ __align__(16) float staged[2][D];
  const int warp = threadIdx.x >> 5;
  Q q(p, smem_u32(rope_smem));
  stage_weights(staged, p.wq, p.wk);
  Turn<D, INTER> turn(p.t.rot, q.lane);
  Walk w(p);
  uint32_t step = 0, token_no = 0;
  uint64_t acc[2][4] = {};  // dwq, dwk of this warp's rows: pairs of fp32 zeros
  uint64_t weights[4];
  auto rows = [&](uint64_t (&sum)[4], uint16_t* d0, long long sh, int h0, int H) {
    uint4 rx[U], rg[U];
    uint64_t x[U][4], g[U][4], y[4];
    float r[U], mean[U];
#pragma unroll
    for (int u = 0; u < U; ++u) rx[u] = q.take(step, u), rg[u] = q.take(step, U + u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      widen(rx[u], x[u]);
      r[u] = dot8(x[u], x[u]);
      widen(rg[u], g[u]);
      widen(turn.swap(rg[u]), y);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        g[u][i] = f2_fma(y[i], turn.s[i], f2_mul(g[u][i], turn.c[i]));  // G
    }
    row_sums<Q::LPR>(r);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = rsqrtf(r[u] * (1.f / D) + p.eps);
      const uint64_t r2 = f2_pack(r[u], r[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[u][i] = f2_mul(x[u][i], r2);                // xh
        sum[i] = f2_fma(g[u][i], x[u][i], sum[i]);    // rows past H hold zeros
        g[u][i] = f2_mul(g[u][i], weights[i]);
      }
      mean[u] = dot8(g[u], x[u]) * (-1.f / D);
    }
    row_sums<Q::LPR>(mean);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * Q::RPW + q.sub;
      const uint64_t r2 = f2_pack(r[u], r[u]), m2 = f2_pack(mean[u], mean[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[u][i] = f2_mul(f2_fma(x[u][i], m2, g[u][i]), r2);
      if (h < H) *reinterpret_cast<uint4*>(d0 + h * sh) = narrow(g[u]);
    }
  };
  for (; w.token < q.tokens; w.advance(p.N), ++token_no) {
#pragma unroll 1
    for (w.step = 0; w.step < q.steps; ++w.step, ++step) {
      q.send();
      copy_wait<kQueue - 1>();  // this step has come
      if (w.step == 0) {
        turn.template load<true>(q.tables(token_no), 512);
        load8(smem_u32(staged[0]) + 4 * q.e0, weights);
      } else if (w.step == q.nq) {
        load8(smem_u32(staged[1]) + 4 * q.e0, weights);
      }
      if (w.step < q.nq)
        rows(acc[0], static_cast<uint16_t*>(p.dq) + w.b * p.sdq.b + w.n * p.sdq.n + q.e0, p.sdq.h,
             w.step * Q::GRP, p.H);
      else
        rows(acc[1], static_cast<uint16_t*>(p.dk) + w.b * p.sdk.b + w.n * p.sdk.n + q.e0, p.sdk.h,
             (w.step - q.nq) * Q::GRP, p.Hkv);
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(acc[kind][i], a[2 * i], a[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = Q::LPR; o < 32; o <<= 1) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
    if (q.lane < Q::LPR)
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[warp][8 * q.lane + i] = a[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += sums[i][threadIdx.x];
      p.part[(static_cast<size_t>(blockIdx.x) * 2 + kind) * D + threadIdx.x] = t;
    }
    __syncthreads();
  }
}

// dwq, dwk = sums of the blocks' partial sums, in a fixed order.  One block
// of 32 x 32 threads per 32 columns of [dwq | dwk].
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const float* part, int blocks, int d,
                                                               float* dwq, float* dwk) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float t[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
  float s = 0.f;
#pragma unroll 4
  for (int i = ty; i < blocks; i += 32) s += part[static_cast<size_t>(i) * 2 * d + col];
  t[ty][tx] = s;
  __syncthreads();
  s = t[tx][ty];  // partial tx of column ty
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tx == 0) {
    const int c = blockIdx.x * 32 + ty;
    (c < d ? dwq : dwk)[c < d ? c : c - d] = s;
  }
}

// Blocks: a warp per token, at most as many as the SMs hold at once (0 on
// error).
int rope_grid(const RopeParams& p, int per_sm) {
  const long long blocks = (static_cast<long long>(p.B) * p.N + kWarps - 1) / kWarps;
  const long long most = static_cast<long long>(per_sm) * sm_count();
  return static_cast<int>(blocks < most ? blocks : most);
}

template <int D, bool INTER>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  constexpr int U = 4;
  constexpr int bytes = kWarps * Queue<D, INTER, false, U>::BYTES;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = smem_attr_once(
      attr_done, reinterpret_cast<const void*>(fa_norm_rope_kernel<D, INTER, U>), bytes);
  if (e != cudaSuccess) return e;
  const int grid = rope_grid(p, 2);
  if (grid <= 0) return cudaErrorInvalidDevice;
  return launch_pdl(fa_norm_rope_kernel<D, INTER, U>, dim3(grid), dim3(kWarps * 32), bytes, stream,
                    p);
}

template <int D, bool INTER>
cudaError_t launch_rope_back(const RopeParams& p, float* dwq, float* dwk, cudaStream_t stream) {
  constexpr int U = 2;
  constexpr int bytes = kWarps * Queue<D, INTER, true, U>::BYTES;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_attr_once(
      attr_done, reinterpret_cast<const void*>(fa_norm_rope_back_kernel<D, INTER, U>), bytes);
  if (e != cudaSuccess) return e;
  int grid = rope_grid(p, 2);
  if (grid <= 0) return cudaErrorInvalidDevice;
  if (grid > kMaxPartials) grid = kMaxPartials;
  e = launch_pdl(fa_norm_rope_back_kernel<D, INTER, U>, dim3(grid), dim3(kWarps * 32), bytes,
                 stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(fa_norm_rope_dw_kernel, dim3(2 * D / 32), dim3(1024), 0, stream,
                    static_cast<const float*>(p.part), grid, D, dwq, dwk);
}

size_t rope_ws_bytes(int d) { return static_cast<size_t>(kMaxPartials) * 2 * d * sizeof(float); }

fa_status check_rope(const void* wq, const void* wk, const void* cos, const void* sin,
                     const int* positions, int B, int H, int Hkv, int N, int d, int rot,
                     int table_rows, float eps) {
  if (B < 1 || H < 1 || Hkv < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (!(isfinite(eps) && eps > 0.f)) return FA_ERR_INVALID_ARG;
  if (table_rows < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  // tokens and blocks are counted in 31 bits
  if (static_cast<long long>(B) * N >= (1LL << 31) / (static_cast<long long>(H) + Hkv))
    return FA_ERR_UNSUPPORTED;
  for (const void* p : {wq, wk, cos, sin}) FA_TRY(check_ptr16(p));
  if (positions) FA_TRY(check_ptr4(positions));
  return FA_OK;
}

RopeParams rope_params(const void* q, const void* k, const float* wq, const float* wk,
                       const float* cos, const float* sin, const int* positions, int B, int H,
                       int Hkv, int N, int rot, int table_rows, float eps) {
  RopeParams p = {};
  p.q = q;
  p.k = k;
  p.wq = wq;
  p.wk = wk;
  p.t = RopeTables{cos, sin, positions, table_rows, rot};
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.eps = eps;
  return p;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const void* k, const float* wq, const float* wk,
                          const float* cos, const float* sin, const int* positions, void* q_out,
                          void* k_out, int B, int H, int Hkv, int N, int d, int rot,
                          int table_rows, int interleaved, float eps, const long long* strides,
                          cudaStream_t stream) {
  using namespace fa;
  FA_TRY(check_rope(wq, wk, cos, sin, positions, B, H, Hkv, N, d, rot, table_rows, eps));
  for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    FA_TRY(check_ptr16(x));
  RopeParams p =
      rope_params(q, k, wq, wk, cos, sin, positions, B, H, Hkv, N, rot, table_rows, eps);
  FA_TRY(read_strides(strides, B, H, N, d, &p.sq));
  FA_TRY(read_strides(strides ? strides + 3 : nullptr, B, Hkv, N, d, &p.sk));
  p.oq = q_out;
  p.ok = k_out;
  if (d == 64)
    FA_CUDA(interleaved ? (launch_rope<64, true>(p, stream)) : (launch_rope<64, false>(p, stream)));
  else
    FA_CUDA(interleaved ? (launch_rope<128, true>(p, stream))
                        : (launch_rope<128, false>(p, stream)));
  return FA_OK;
}

size_t fa_qk_norm_rope_workspace_size(int d) {
  if (d < 1) return 0;
  return fa::rope_ws_bytes(d);
}

fa_status fa_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                                   const void* k, const float* wq, const float* wk,
                                   const float* cos, const float* sin, const int* positions,
                                   void* dq, void* dk, float* dwq, float* dwk, int B, int H,
                                   int Hkv, int N, int d, int rot, int table_rows,
                                   int interleaved, float eps, const long long* strides,
                                   const long long* grad_strides, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  using namespace fa;
  FA_TRY(check_rope(wq, wk, cos, sin, positions, B, H, Hkv, N, d, rot, table_rows, eps));
  for (const void* x : {dq_out, dk_out, q, k, static_cast<const void*>(dq),
                        static_cast<const void*>(dk)})
    FA_TRY(check_ptr16(x));
  FA_TRY(check_ptr4(dwq));
  FA_TRY(check_ptr4(dwk));
  RopeParams p =
      rope_params(q, k, wq, wk, cos, sin, positions, B, H, Hkv, N, rot, table_rows, eps);
  FA_TRY(read_strides(strides, B, H, N, d, &p.sq));
  FA_TRY(read_strides(strides ? strides + 3 : nullptr, B, Hkv, N, d, &p.sk));
  FA_TRY(read_strides(grad_strides, B, H, N, d, &p.sdq));
  FA_TRY(read_strides(grad_strides ? grad_strides + 3 : nullptr, B, Hkv, N, d, &p.sdk));
  FA_TRY(check_disjoint(p.sdq, B, H, N, d));
  FA_TRY(check_disjoint(p.sdk, B, Hkv, N, d));
  FA_TRY(check_ws(workspace, workspace_bytes, rope_ws_bytes(d)));
  p.gq = dq_out;
  p.gk = dk_out;
  p.dq = dq;
  p.dk = dk;
  p.part = static_cast<float*>(workspace);
  if (d == 64)
    FA_CUDA(interleaved ? (launch_rope_back<64, true>(p, dwq, dwk, stream))
                        : (launch_rope_back<64, false>(p, dwq, dwk, stream)));
  else
    FA_CUDA(interleaved ? (launch_rope_back<128, true>(p, dwq, dwk, stream))
                        : (launch_rope_back<128, false>(p, dwq, dwk, stream)));
  return FA_OK;
}

}  // extern "C"
