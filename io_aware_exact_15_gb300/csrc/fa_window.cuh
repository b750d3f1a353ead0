// Rows of windowed attention that are computed again, by one warp each, from
// the definition.
//
// The tile kernels multiply masked weights as zeros, and 0 x NaN is NaN: a NaN
// or an infinity in a row of v (k, q, dO in the backward) reaches every row
// that shares a 128 x 128 tile with it, also the rows that do not see it, rows
// of the next sequence of a packed batch and what stands behind the last one
// among them.  Checking tiles on their way in would cost every tile; a row
// that caught something shows it in its result.  So results are looked at as
// they are written, and a row with a NaN or an infinity in it is formed again
// here from the keys (or queries) that belong to it and nothing else.  Rows to
// which such a number belongs end as soon as every column is NaN.
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
  // the same sum in every lane
  FA_DEV float dot(const RowPiece& y) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(x[i], y.x[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
  FA_DEV bool all_nan() const {
    bool n = true;
#pragma unroll
    for (int i = 0; i < E; ++i) n = n && x[i] != x[i];
    return __all_sync(0xffffffffu, n);
  }
};

// o of query i of a sequence: rows q0 + i of q, o and k0 + j of k, v; lse2 is
// its logsumexp in log2 units.  Whole warp.
template <int D>
static __device__ __noinline__ void window_row_o(const void* q, const void* k, const void* v,
                                                 void* o, size_t q0, size_t k0, int i, int window,
                                                 int sinks, float sl2, float lse2) {
  const int lane = threadIdx.x & 31;
  RowPiece<D> qi, kj, vj, acc;
  qi.load(q, q0 + i, lane);
  acc.zero();
  const int lo = max(i - window + 1, 0), first = min(sinks, lo);
#pragma unroll 1
  for (int n = 0; n < first + i + 1 - lo; ++n) {
    const int j = n < first ? n : lo + n - first;
    kj.load(k, k0 + j, lane);
    vj.load(v, k0 + j, lane);
    acc.add(ex2(fmaf(qi.dot(kj), sl2, -lse2)), vj);
    if (acc.all_nan()) break;
  }
  acc.store(o, q0 + i, lane, 1.f);
}

// dq of query i: rows q0 + i of q, dO and dq.
template <int D>
static __device__ __noinline__ void window_row_dq(const WindowFinish& w, size_t q0, size_t k0,
                                                  int i, float lse2, float delta) {
  const int lane = threadIdx.x & 31;
  const float sl2 = w.b.scale * 1.4426950408889634f;
  RowPiece<D> qi, gi, kj, vj, acc;
  qi.load(w.q, q0 + i, lane);
  gi.load(w.dO, q0 + i, lane);
  acc.zero();
  const int lo = max(i - w.b.window + 1, 0), first = min(w.b.sinks, lo);
#pragma unroll 1
  for (int n = 0; n < first + i + 1 - lo; ++n) {
    const int j = n < first ? n : lo + n - first;
    kj.load(w.k, k0 + j, lane);
    vj.load(w.v, k0 + j, lane);
    acc.add(ex2(fmaf(qi.dot(kj), sl2, -lse2)) * (gi.dot(vj) - delta), kj);
    if (acc.all_nan()) break;
  }
  acc.store(w.dq, q0 + i, lane, w.b.scale);
}

// dv (or dk) of key j of a sequence of N rows, over G query heads whose slices
// are `slice` rows apart: rows q0 + i of q, dO, lse and delta, k0 + j of k, v.
template <int D>
static __device__ __noinline__ void window_row_dkv(const WindowFinish& w, bool dv, size_t q0,
                                                   size_t slice, int G, size_t k0, int j, int N) {
  const int lane = threadIdx.x & 31;
  const float sl2 = w.b.scale * 1.4426950408889634f;
  RowPiece<D> kj, vj, qi, gi, acc;
  kj.load(w.k, k0 + j, lane);
  vj.load(w.v, k0 + j, lane);
  acc.zero();
  const int end = j < w.b.sinks || N - j < w.b.window ? N : j + w.b.window;
#pragma unroll 1
  for (int g = 0; g < G; ++g, q0 += slice) {
#pragma unroll 1
    for (int i = j; i < end; ++i) {
      qi.load(w.q, q0 + i, lane);
      gi.load(w.dO, q0 + i, lane);
      const float pij = ex2(fmaf(qi.dot(kj), sl2, -w.b.lse[q0 + i] * 1.4426950408889634f));
      if (dv)
        acc.add(pij, gi);
      else
        acc.add(pij * (gi.dot(vj) - w.b.delta[q0 + i]), qi);
      if (acc.all_nan()) break;
    }
  }
  acc.store(dv ? w.b.dv : w.b.dk, k0 + j, lane, dv ? 1.f : w.b.scale);
}

}  // namespace fa
