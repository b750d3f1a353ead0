// Rows of windowed attention that are computed again, by one warp each, from
// the definition.
//
// The tile kernels multiply masked weights as zeros, and 0 x NaN is NaN: a NaN
// or an infinity in a row of v (k, q, dO in the backward) reaches every row
// that shares a 128 x 128 tile with it, also the rows that do not see it, rows
// of the next sequence of a packed batch and what stands behind the last one
// among them.  Checking tiles on their way in would cost every tile; a row
// that caught something shows it in its result.  So results are looked at as
// they are written, and the columns of a row that hold a NaN or an infinity are
// formed again here from the keys (or queries) that belong to it and nothing
// else.  Where such a number does belong to the row, that ends as soon as all of
// these columns have one again, since no sum brings them back.  A query with
// the logsumexp -infinity (all its scores are) has no weights: its sums are
// empty, whatever numbers its keys have.
#pragma once

#include <stdint.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

// The window backward's weights are 2^15 P (fa_bwd.cu), and so is what they are
// summed to before the outputs.
constexpr float kPLift = 32768.f;

// A lane's elements of a row: E = D / 32 from E * lane on.
template <int D>
struct RowPiece {
  static constexpr int E = D / 32;
  float x[E];
  FA_DEV void zero() {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = 0.f;
  }
  FA_DEV void load(const void* rows, size_t row, int lane) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(rows) +
                                                          row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t y = __ldg(w + i);
      x[2 * i] = bf16_lo(y);
      x[2 * i + 1] = bf16_hi(y);
    }
  }
  FA_DEV void store(void* rows, size_t row, int lane, float f) const {
    uint32_t* w =
        reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(rows) + row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16(x[2 * i] * f, x[2 * i + 1] * f);
  }
  FA_DEV void add(float f, const RowPiece& y) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = fmaf(f, y.x[i], x[i]);
  }
  FA_DEV float dot(const RowPiece& y) const {  // this lane's share
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(x[i], y.x[i], s);
    return s;
  }
};

// Rows taken at a time: their loads and sums over the lanes overlap.
constexpr int kRowBatch = 4;
FA_DEV void sum_lanes(float (&s)[kRowBatch]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
}
FA_DEV bool not_finite(float x) { return !(fabsf(x) <= 3.402823466e38f); }

// The columns of row `row` that are to be formed again, the others as they are.
template <int D>
struct Mend {
  static constexpr int E = RowPiece<D>::E;
  RowPiece<D> old, acc;
  FA_DEV void begin(const void* rows, size_t row, int lane) {
    // (written by this warp, or by an earlier kernel)
    const volatile uint32_t* w = reinterpret_cast<const volatile uint32_t*>(
        static_cast<const uint16_t*>(rows) + row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t y = w[i];
      old.x[2 * i] = bf16_lo(y);
      old.x[2 * i + 1] = bf16_hi(y);
    }
    acc.zero();
  }
  FA_DEV bool done() const {  // none of them can become finite any more
    bool d = true;
#pragma unroll
    for (int i = 0; i < E; ++i) d = d && (!not_finite(old.x[i]) || not_finite(acc.x[i]));
    return __all_sync(0xffffffffu, d);
  }
  FA_DEV void end(void* rows, size_t row, int lane, float f) {
#pragma unroll
    for (int i = 0; i < E; ++i) acc.x[i] = not_finite(old.x[i]) ? acc.x[i] * f : old.x[i];
    acc.store(rows, row, lane, 1.f);
  }
};

// o of query i of a sequence: rows q0 + i of q, o and k0 + j of k, v; lse2 is
// its logsumexp in log2 units.  Whole warp.
template <int D>
static __device__ __noinline__ void window_row_o(const void* q, const void* k, const void* v,
                                                 void* o, size_t q0, size_t k0, int i, int window,
                                                 int sinks, float sl2, float lse2) {
  const int lane = threadIdx.x & 31;
  RowPiece<D> qi;
  Mend<D> m;
  qi.load(q, q0 + i, lane);
  m.begin(o, q0 + i, lane);
  const int lo = max(i - window + 1, 0), first = min(sinks, lo);
  const int total = lse2 == -INFINITY ? 0 : first + i + 1 - lo;
#pragma unroll 1
  for (int n = 0; n < total && !m.done(); n += kRowBatch) {
    RowPiece<D> kj[kRowBatch], vj[kRowBatch];
    float s[kRowBatch];
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      const int x = min(n + u, total - 1);
      const size_t j = k0 + (x < first ? x : lo + x - first);
      kj[u].load(k, j, lane);
      vj[u].load(v, j, lane);
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) s[u] = qi.dot(kj[u]);
    sum_lanes(s);
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u)
      if (n + u < total) m.acc.add(ex2(fmaf(s[u], sl2, -lse2)), vj[u]);
  }
  m.end(o, q0 + i, lane, 1.f);
}

// dq of query i: rows q0 + i of q, dO and dq.
template <int D>
static __device__ __noinline__ void window_row_dq(const WindowFinish& w, size_t q0, size_t k0,
                                                  int i, float lse2, float delta) {
  const int lane = threadIdx.x & 31;
  const float sl2 = w.b.scale * 1.4426950408889634f;
  RowPiece<D> qi, gi;
  Mend<D> m;
  qi.load(w.q, q0 + i, lane);
  gi.load(w.dO, q0 + i, lane);
  m.begin(w.dq, q0 + i, lane);
  const int lo = max(i - w.b.window + 1, 0), first = min(w.b.sinks, lo);
  const int total = lse2 == -INFINITY ? 0 : first + i + 1 - lo;
#pragma unroll 1
  for (int n = 0; n < total && !m.done(); n += kRowBatch) {
    RowPiece<D> kj[kRowBatch], vj[kRowBatch];
    float s[kRowBatch], t[kRowBatch];
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      const int x = min(n + u, total - 1);
      const size_t j = k0 + (x < first ? x : lo + x - first);
      kj[u].load(w.k, j, lane);
      vj[u].load(w.v, j, lane);
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      s[u] = qi.dot(kj[u]);
      t[u] = gi.dot(vj[u]);
    }
    sum_lanes(s);
    sum_lanes(t);
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u)
      if (n + u < total) m.acc.add(ex2(fmaf(s[u], sl2, -lse2)) * (t[u] - delta), kj[u]);
  }
  m.end(w.dq, q0 + i, lane, w.b.scale);
}

// dv (or dk) of key j of a sequence of N rows, over G query heads whose slices
// are `slice` rows apart: rows q0 + i of q, dO, lse and delta, k0 + j of k, v.
template <int D>
static __device__ __noinline__ void window_row_dkv(const WindowFinish& w, bool dv, size_t q0,
                                                   size_t slice, int G, size_t k0, int j, int N) {
  const int lane = threadIdx.x & 31;
  const float sl2 = w.b.scale * 1.4426950408889634f;
  void* out = dv ? w.b.dv : w.b.dk;
  RowPiece<D> kj, vj;
  Mend<D> m;
  kj.load(w.k, k0 + j, lane);
  vj.load(w.v, k0 + j, lane);
  m.begin(out, k0 + j, lane);
  const int end = j < w.b.sinks || N - j < w.b.window ? N : j + w.b.window;
#pragma unroll 1
  for (int g = 0; g < G; ++g, q0 += slice) {
#pragma unroll 1
    for (int i = j; i < end && !m.done(); i += kRowBatch) {
      RowPiece<D> qi[kRowBatch], gi[kRowBatch];
      float s[kRowBatch], t[kRowBatch], l[kRowBatch], dl[kRowBatch];
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        const size_t row = q0 + min(i + u, end - 1);
        qi[u].load(w.q, row, lane);
        gi[u].load(w.dO, row, lane);
        l[u] = w.b.lse[row];
        dl[u] = w.b.delta[row];
      }
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        s[u] = kj.dot(qi[u]);
        t[u] = vj.dot(gi[u]);
      }
      sum_lanes(s);
      if (!dv) sum_lanes(t);
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        if (i + u >= end || l[u] == -INFINITY) continue;
        const float pij = ex2(fmaf(s[u], sl2, -l[u] * 1.4426950408889634f));
        if (dv)
          m.acc.add(pij, gi[u]);
        else
          m.acc.add(pij * (t[u] - dl[u]), qi[u]);
      }
    }
  }
  m.end(out, k0 + j, lane, dv ? 1.f : w.b.scale);
}

}  // namespace fa
