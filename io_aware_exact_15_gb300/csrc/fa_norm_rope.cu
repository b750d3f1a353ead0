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

FA_DEV uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

FA_DEV void widen(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
FA_DEV uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// sum over the LPR lanes of a row
template <int LPR>
FA_DEV float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The angles of one lane's 8 elements.  Adjacent pairs: c, s hold 4 values.
// Half pairs (i, i + rot / 2): 8 values, and the partner element sits `hop`
// lanes away (rot is a multiple of 16, so a half is a whole number of lanes).
template <int D, bool INTER>
struct Turn {
  float c[8], s[8];
  bool in, upper;
  int partner;  // lane that holds the other half's elements

  FA_DEV void load(const RopeTables& t, int b, int n, int N, int lane) {
    constexpr int LPR = D / 8;
    const int l = lane % LPR, e0 = 8 * l, hop = t.rot / 16;
    in = e0 < t.rot;
    upper = !INTER && e0 >= t.rot / 2;
    partner = in ? (upper ? lane - hop : lane + hop) : lane;
    int pos = t.positions ? t.positions[static_cast<size_t>(b) * N + n] : n;
    pos = min(max(pos, 0), t.rows - 1);
    const size_t row = static_cast<size_t>(pos) * (t.rot / 2);
    constexpr int V = INTER ? 1 : 2;
    const int i0 = INTER ? e0 / 2 : (upper ? e0 - t.rot / 2 : e0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float4 a = make_float4(1.f, 1.f, 1.f, 1.f), z = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        a = __ldg(reinterpret_cast<const float4*>(t.cos + row + i0) + v);
        z = __ldg(reinterpret_cast<const float4*>(t.sin + row + i0) + v);
      }
      c[4 * v] = a.x, c[4 * v + 1] = a.y, c[4 * v + 2] = a.z, c[4 * v + 3] = a.w;
      s[4 * v] = z.x, s[4 * v + 1] = z.y, s[4 * v + 2] = z.z, s[4 * v + 3] = z.w;
    }
  }

  // y turned by the angles (BACK: against them); all lanes of the warp
  template <bool BACK>
  FA_DEV void apply(float (&y)[8]) const {
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], b = y[2 * i + 1], z = BACK ? -s[i] : s[i];
        y[2 * i] = in ? a * c[i] - b * z : a;
        y[2 * i + 1] = in ? b * c[i] + a * z : b;
      }
    } else {
      const bool minus = upper == BACK;  // lower half forward, upper half backward
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, y[i], partner);
        y[i] = in ? y[i] * c[i] + (minus ? -o : o) * s[i] : y[i];
      }
    }
  }
};

FA_DEV void load_weights(const float* w, int e0, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + e0));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + e0) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// One block = eight consecutive tokens (a warp each) x one group of U * RPW
// heads of q or of k: reads run along a token's heads, writes along a head's
// tokens, both in pieces of 2 KB (d = 128).  All loads of a warp are in
// flight together.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32) fa_norm_rope_kernel(const RopeParams p) {
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  grid_dep_launch();
  constexpr int LPR = D / 8, RPW = 32 / LPR, GRP = U * RPW;
  const int lane = threadIdx.x & 31, e0 = 8 * (lane % LPR), sub = lane / LPR;
  const uint32_t nq = (p.H + GRP - 1) / GRP, groups = nq + (p.Hkv + GRP - 1) / GRP;
  const uint32_t block = blockIdx.x / groups, group = blockIdx.x - block * groups;
  const uint32_t token = block * kWarps + (threadIdx.x >> 5);
  if (token >= static_cast<uint32_t>(p.B) * p.N) return;
  const int b = token / p.N, n = token - static_cast<uint32_t>(b) * p.N;
  const bool isq = group < nq;
  const int h0 = (isq ? group : group - nq) * GRP, H = isq ? p.H : p.Hkv;
  const Strides s = isq ? p.sq : p.sk;
  const uint16_t* x0 = static_cast<const uint16_t*>(isq ? p.q : p.k) + b * s.b + n * s.n + e0;
  uint16_t* o0 = static_cast<uint16_t*>(isq ? p.oq : p.ok) +
                 (static_cast<size_t>(b) * H * p.N + n) * D + e0;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPW + sub;
    raw[u] = h < H ? ld16(x0 + h * s.h) : make_uint4(0, 0, 0, 0);
  }
  Turn<D, INTER> turn;
  turn.load(p.t, b, n, p.N, lane);
  float w[8];
  load_weights(isq ? p.wq : p.wk, e0, w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPW + sub;
    float x[8];
    widen(raw[u], x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    turn.template apply<false>(x);
    if (h < H) *reinterpret_cast<uint4*>(o0 + static_cast<size_t>(h) * p.N * D) = narrow(x);
  }
}

// Backward of U rows per lane group: acc += G xh, the rows' gradients are
// written to d0 (+ h * sh).
template <int D, bool INTER, int U>
FA_DEV void norm_rope_back_rows(const uint4 (&rx)[U], const uint4 (&rg)[U], const float* weights,
                                const Turn<D, INTER>& turn, float eps, uint16_t* d0, long long sh,
                                int h0, int H, float (&acc)[8]) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  float w[8];
  load_weights(weights, 8 * (lane % LPR), w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPW + sub;
    float x[8], g[8];
    widen(rx[u], x);
    widen(rg[u], g);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + eps);
    turn.template apply<true>(g);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= r;
      acc[i] = fmaf(g[i], x[i], acc[i]);  // rows past H hold zeros
      g[i] *= w[i];
      dot = fmaf(g[i], x[i], dot);
    }
    const float mean = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = r * (g[i] - x[i] * mean);
    if (h < H) *reinterpret_cast<uint4*>(d0 + h * sh) = narrow(g);
  }
}

// A warp takes whole tokens (dealt round-robin to the grid's warps) and walks
// their heads U * RPW at a time, the next rows already on their way; the
// sums of dw stay in registers until the end.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32, 3) fa_norm_rope_back_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int LPR = D / 8, RPW = 32 / LPR, GRP = U * RPW;
  __shared__ float sums[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = 8 * (lane % LPR), sub = lane / LPR;
  const int nq = (p.H + GRP - 1) / GRP, steps = nq + (p.Hkv + GRP - 1) / GRP;
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.N, stride = gridDim.x * kWarps;
  float acc[2][8] = {};
  uint4 rx[U], rg[U];
  auto fetch = [&](uint32_t token, int step) {
    const int b = token / p.N, n = token - static_cast<uint32_t>(b) * p.N;
    const bool isq = step < nq;
    const int h0 = (isq ? step : step - nq) * GRP, H = isq ? p.H : p.Hkv;
    const Strides s = isq ? p.sq : p.sk;
    const uint16_t* x0 = static_cast<const uint16_t*>(isq ? p.q : p.k) + b * s.b + n * s.n + e0;
    const uint16_t* g0 = static_cast<const uint16_t*>(isq ? p.gq : p.gk) +
                         (static_cast<size_t>(b) * H * p.N + n) * D + e0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RPW + sub;
      rx[u] = rg[u] = make_uint4(0, 0, 0, 0);
      if (h < H) {
        rx[u] = ld16(x0 + h * s.h);
        rg[u] = ld16(g0 + static_cast<size_t>(h) * p.N * D);
      }
    }
  };
  uint32_t token = blockIdx.x * kWarps + warp;
  if (token < tokens) fetch(token, 0);
  for (; token < tokens; token += stride) {
    const int b = token / p.N, n = token - static_cast<uint32_t>(b) * p.N;
    Turn<D, INTER> turn;
    turn.load(p.t, b, n, p.N, lane);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      uint4 cx[U], cg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) cx[u] = rx[u], cg[u] = rg[u];
      if (step + 1 < steps)
        fetch(token, step + 1);
      else if (tokens - token > stride)
        fetch(token + stride, 0);
      if (step < nq)
        norm_rope_back_rows<D, INTER, U>(
            cx, cg, p.wq, turn, p.eps,
            static_cast<uint16_t*>(p.dq) + b * p.sdq.b + n * p.sdq.n + e0, p.sdq.h, step * GRP,
            p.H, acc[0]);
      else
        norm_rope_back_rows<D, INTER, U>(
            cx, cg, p.wk, turn, p.eps,
            static_cast<uint16_t*>(p.dk) + b * p.sdk.b + n * p.sdk.n + e0, p.sdk.h,
            (step - nq) * GRP, p.Hkv, acc[1]);
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1)
        acc[kind][i] += __shfl_xor_sync(0xffffffffu, acc[kind][i], o);
    if (lane < LPR)
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[warp][8 * lane + i] = acc[kind][i];
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

template <int D, bool INTER>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 8);
  // Few tokens: one row per lane group, so that the heads of a token spread
  // over as many warps as there are.  Many: four rows in flight per lane.
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const bool wide = tokens * (p.H + p.Hkv) >= 32LL * 1024;
  const int grp = wide ? 4 * RPW : RPW;
  const long long groups = (p.H + grp - 1) / grp + (p.Hkv + grp - 1) / grp;
  const dim3 grid(static_cast<unsigned>((tokens + kWarps - 1) / kWarps * groups));
  return wide ? launch_pdl(fa_norm_rope_kernel<D, INTER, 4>, grid, dim3(kWarps * 32), 0, stream, p)
              : launch_pdl(fa_norm_rope_kernel<D, INTER, 1>, grid, dim3(kWarps * 32), 0, stream, p);
}

template <int D, bool INTER>
cudaError_t launch_rope_back(const RopeParams& p, float* dwq, float* dwk, cudaStream_t stream) {
  constexpr int U = 2;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  long long blocks = (static_cast<long long>(p.B) * p.N + kWarps - 1) / kWarps;
  if (blocks > 3LL * sms) blocks = 3LL * sms;
  if (blocks > kMaxPartials) blocks = kMaxPartials;
  cudaError_t e = launch_pdl(fa_norm_rope_back_kernel<D, INTER, U>,
                             dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(fa_norm_rope_dw_kernel, dim3(2 * D / 32), dim3(1024), 0, stream,
                    static_cast<const float*>(p.part), static_cast<int>(blocks), D, dwq, dwk);
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
