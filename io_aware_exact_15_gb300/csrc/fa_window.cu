// Causal attention over a sliding window with a few first tokens that stay
// visible: query i sees key j when j <= i and (i - j < window or j < sinks).
// Entry points of the forward and the backward, and the backward's last kernel.
//
// Both passes are the tile kernels of fa_fwd.cu and fa_bwd.cu (kind kWindow)
// with schedules that visit only tiles with a visible pair, and masks by bits
// on the tiles that the diagonal, the window's edge, the last first token or
// the sequence's end crosses.  Their work is about window / 128 + 1 tiles of
// 128 keys per 128 rows and the first tokens' tiles, so they are bound by the
// tensor cores and the exponentials as the causal kernels are.
//
// The backward is three kernels: D = <dO, O> and a cleared dQ accumulator;
// the tiles; and what is here.  All but the second are bound by memory: of
// 533 us for 2 x 16 heads (4 of K and V) of 8192 rows of 128, window 1024, 4
// first keys, the first takes 40 and the last 36 (134 MB of fp32 accumulator in,
// 67 of bf16 out, half of that not yet in DRAM when it ends: 4.9 TB/s of DRAM
// traffic), of 193 us for 6 packed sequences of up to 4096 rows, 12 heads
// of 64, window 512, 16 first keys, 17 and 21.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_sched.cuh"
#include "fa_window.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kUnroll = 4;

// A sequence of the batch: its rows in a slice and its length.
struct Seq {
  int row0, n;
};
FA_DEV Seq sequence(const BwdParams& p, int b) {
  if (!p.cu_seqlens) return Seq{0, p.N};
  const int a = min(max(p.cu_seqlens[b], 0), p.total);
  const int e = min(max(p.cu_seqlens[b + 1], a), p.total);
  return Seq{a, min(e - a, p.N)};
}

// The backward's last kernel: dq = bf16(scale * accumulator); the parts of the
// first key tiles added up in their order; rows with a NaN or an infinity
// formed again.  Blocks [0, nsum): a warp per 4 (d = 64) or 2 rows of a first
// key tile's dV or dK; [nsum, nsum + nbad): a warp per 32 words of `bad`; the rest: dq.
template <int D>
__global__ void __launch_bounds__(256) fa_window_finish_kernel(const WindowFinish w, int nsum,
                                                               int nbad) {
  grid_dep_wait();  // the previous kernel's writes are visible from here on
  const BwdParams& p = w.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.H / p.Hkv, ntmax = (p.N + kTile - 1) / kTile;
  const size_t slice = p.cu_seqlens ? p.total : p.N;
  // first rows of key/value head bkv's slices, sequence s: queries and keys
  auto origin = [&](int bkv, const Seq& s, size_t& q0, size_t& k0) {
    const int zkv = p.cu_seqlens ? bkv % p.Hkv : bkv;
    const int zq = p.cu_seqlens ? zkv * G : (bkv / p.Hkv) * p.H + (bkv % p.Hkv) * G;
    q0 = zq * slice + s.row0;
    k0 = zkv * slice + s.row0;
  };
  if (static_cast<int>(blockIdx.x) < nsum) {
    // ------------------------------------------------ sums of parts
    constexpr int LPR = D / 8, RPW = 32 / LPR;    // lanes per row, 8 columns each
    const int t = (blockIdx.x * 8 + warp) * RPW;  // ((bkv, tile), dV or dK, first row)
    const int r = (t & (kTile - 1)) + lane / LPR, side = (t >> 7) & 1, unit = t >> 8;
    const int tiles = p.group_parts > 1 ? ntmax : p.sink_tiles;
    // packed: a sequence with parts is longer than L = 128 part_tiles rows, so
    // it has a multiple of L among them, and is looked for at its first
    const int L = p.part_tiles * kTile, marks = p.packed ? p.total / L + 1 : 1;
    if (unit >= (p.packed ? p.Hkv * marks : p.B * p.Hkv) * tiles) return;
    int bkv = unit / tiles;
    const int kt = unit - bkv * tiles;
    if (p.packed) {
      const int head = bkv / marks, mark = (bkv - head * marks) * L;
      const int b = packed_find(p.cu_seqlens, p.B, p.total, mark, 1, 0);
      const int a = min(max(p.cu_seqlens[b], 0), p.total);
      if (a > mark || a <= mark - L) return;
      bkv = b * p.Hkv + head;
    }
    const Seq s = sequence(p, bkv / p.Hkv);
    const int nT = (s.n + kTile - 1) / kTile, j = kt * kTile + r;
    // no such rows, or written whole
    if (j - lane / LPR >= s.n || (p.group_parts == 1 && kt + p.part_tiles >= nT)) return;
    const bool sunk = kt < p.sink_tiles;
    const int parts =
        (sunk ? (nT - kt + p.part_tiles - 1) / p.part_tiles : 1) * p.group_parts;
    const size_t slot =
        p.packed ? static_cast<size_t>(bkv % p.Hkv * tiles + kt) * p.slot_units + 2 * (s.row0 / L)
                 : static_cast<size_t>(bkv) * p.slot_units +
                       (sunk ? kt * p.sink_parts : p.sink_tiles * (p.sink_parts - 1) + kt) *
                           p.group_parts;
    const float* src = p.part + ((slot * 2 + side) * kTile + r) * D + 8 * (lane % LPR);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float4* x = reinterpret_cast<const float4*>(src + static_cast<size_t>(i) * 2 * kTile * D);
      const float4 y = x[0], z = x[1];
      a = make_float4(a.x + y.x, a.y + y.y, a.z + y.z, a.w + y.w);
      b = make_float4(b.x + z.x, b.y + z.y, b.z + z.z, b.w + z.w);
    }
    float odd = fmaf(a.x, 0.f, fmaf(a.y, 0.f, fmaf(a.z, 0.f, a.w * 0.f)));
    odd = fmaf(b.x, 0.f, fmaf(b.y, 0.f, fmaf(b.z, 0.f, fmaf(b.w, 0.f, odd))));
    size_t q0, k0;
    origin(bkv, s, q0, k0);
    const float f = side == 0 ? 1.f / kPLift : p.scale;
    if (j < s.n)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(side == 0 ? p.dv : p.dk) + (k0 + j) * D +
                                8 * (lane % LPR)) =
          make_uint4(pack_bf16(a.x * f, a.y * f), pack_bf16(a.z * f, a.w * f),
                     pack_bf16(b.x * f, b.y * f), pack_bf16(b.z * f, b.w * f));
    uint32_t again = __ballot_sync(0xffffffffu, j < s.n && odd != 0.f);
    while (again) {  // (rare) the lanes of one row at a time
      const int first = (__ffs(again) - 1) / LPR * LPR;
      again &= ~(((1u << LPR) - 1u) << first);
      __syncwarp();  // the row was written by its lanes
      window_row_dkv<D>(w, side == 0, q0, slice, G, k0, __shfl_sync(0xffffffffu, j, first), s.n);
    }
    return;
  }
  if (static_cast<int>(blockIdx.x) < nsum + nbad) {
    // ------------------------------------------------ rows that caught something
    const int per = p.packed ? p.total / kTile + p.B : p.B * ntmax;  // tiles of a head
    const long long total = 8LL * p.Hkv * per;
    const long long t = (static_cast<long long>(blockIdx.x - nsum) * 8 + warp) * 32 + lane;
    uint32_t word = 0;
    int bkv = 0, kt = 0;
    Seq s = {0, 0};
    if (t < total) {
      const int unit = static_cast<int>(t >> 3);
      if (p.packed) {
        const int head = unit / per, v = unit - head * per;
        const int b = packed_find(p.cu_seqlens, p.B, p.total, v, kTile, 1);
        bkv = b * p.Hkv + head;
        kt = v - (min(max(p.cu_seqlens[b], 0), p.total) / kTile + b);
      } else {
        bkv = unit / ntmax;
        kt = unit - bkv * ntmax;
      }
      s = sequence(p, bkv / p.Hkv);
      const int nT = (s.n + kTile - 1) / kTile;
      // tiles that were written whole
      if (p.group_parts == 1 && kt >= 0 && kt < nT && !(kt < p.sink_tiles && kt + p.part_tiles < nT))
        // (rows of the sequence alone: after a wait that gave up, anything may stand there)
        word = p.bad[t] & low_bits(s.n - kt * kTile - 32 * static_cast<int>(t & 3));
    }
    for (uint32_t some = __ballot_sync(0xffffffffu, word != 0); some; some &= some - 1) {
      const int from = __ffs(some) - 1;
      uint32_t rows = __shfl_sync(0xffffffffu, word, from);
      const int b0 = __shfl_sync(0xffffffffu, bkv, from), k = __shfl_sync(0xffffffffu, kt, from);
      const Seq q = {__shfl_sync(0xffffffffu, s.row0, from), __shfl_sync(0xffffffffu, s.n, from)};
      const int which = static_cast<int>((t - lane + from) & 7);  // dV or dK, quarter of the tile
      size_t q0, k0;
      origin(b0, q, q0, k0);
      for (; rows; rows &= rows - 1)
        window_row_dkv<D>(w, which < 4, q0, slice, G, k0,
                          k * kTile + 32 * (which & 3) + __ffs(rows) - 1, q.n);
    }
    return;
  }
  // -------------------------------------------------- dq
  constexpr int TPR = D / 8;  // lanes per row, 8 elements each
  const int blocks = gridDim.x - nsum - nbad, block = blockIdx.x - nsum - nbad;
  const int nslices = p.cu_seqlens ? p.H : p.B * p.H;
  const long long total = static_cast<long long>(slice) * nslices * TPR;
  const long long stride = static_cast<long long>(blocks) * blockDim.x;
  // packed: rows before the first sequence and behind the last are left alone
  uint32_t from = 0, to = static_cast<uint32_t>(slice);
  if (p.cu_seqlens) {
    from = min(max(p.cu_seqlens[0], 0), p.total);
    const Seq s = sequence(p, p.B - 1);
    to = s.row0 + s.n;
  }
  const float4* acc = reinterpret_cast<const float4*>(p.dq_acc);
  for (long long i0 = static_cast<long long>(block) * blockDim.x + threadIdx.x; i0 - lane < total;
       i0 += kUnroll * stride) {
    float4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = i0 + u * stride;
      if (i < total) {
        a[u] = acc[2 * i];
        b[u] = acc[2 * i + 1];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = i0 + u * stride;
      const uint32_t row = static_cast<uint32_t>(i / TPR), in = row % static_cast<uint32_t>(slice);
      const bool live = i < total && in >= from && in < to;
      float odd = 0.f;
      if (live) {
        odd = fmaf(a[u].x, 0.f, fmaf(a[u].y, 0.f, fmaf(a[u].z, 0.f, a[u].w * 0.f)));
        odd = fmaf(b[u].x, 0.f, fmaf(b[u].y, 0.f, fmaf(b[u].z, 0.f, fmaf(b[u].w, 0.f, odd))));
        reinterpret_cast<uint4*>(w.dq)[i] =
            make_uint4(pack_bf16(a[u].x * p.scale, a[u].y * p.scale),
                       pack_bf16(a[u].z * p.scale, a[u].w * p.scale),
                       pack_bf16(b[u].x * p.scale, b[u].y * p.scale),
                       pack_bf16(b[u].z * p.scale, b[u].w * p.scale));
      }
      uint32_t again = __ballot_sync(0xffffffffu, odd != 0.f);
      while (again) {  // (rare) the lanes of one row at a time
        const int first = (__ffs(again) - 1) / TPR * TPR;
        again &= ~(((1u << TPR) - 1u) << first);
        __syncwarp();  // the row was written by its lanes
        const uint32_t at = __shfl_sync(0xffffffffu, row, first);
        const uint32_t z = at / static_cast<uint32_t>(slice);
        int x = static_cast<int>(at - z * static_cast<uint32_t>(slice));  // row in its slice
        int bq = z / p.H;
        const int h = z - bq * p.H;
        Seq s = {0, p.N};
        if (p.cu_seqlens) {  // its sequence: the last that begins at or before it
          int lo = 0, hi = p.B;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            (p.cu_seqlens[mid] <= x ? lo : hi) = mid;
          }
          bq = lo;
          s = sequence(p, lo);
        }
        x -= s.row0;
        if (x < 0 || x >= s.n) continue;  // (offsets that break the rules)
        const int zkv = p.cu_seqlens ? h / G : bq * p.Hkv + h / G;
        window_row_dq<D>(w, static_cast<size_t>(z) * slice + s.row0, zkv * slice + s.row0, x,
                         p.lse[at] * kLog2e, p.delta[at]);
      }
    }
  }
}

template <int D>
cudaError_t launch_finish(const WindowFinish& w, cudaStream_t stream) {
  const BwdParams& p = w.b;
  const long long bkv = static_cast<long long>(p.B) * p.Hkv, nT = (p.N + kTile - 1) / kTile;
  const long long rows = p.cu_seqlens ? static_cast<long long>(p.H) * p.total
                                      : static_cast<long long>(p.B) * p.H * p.N;
  const long long marks = p.total / (p.part_tiles * kTile) + 1;
  const long long nsum = (p.group_parts > 1    ? bkv * nT
                          : p.sink_parts == 1  ? 0
                          : p.packed           ? p.Hkv * marks * p.sink_tiles
                                               : bkv * p.sink_tiles) *
                         (2 * kTile * (D / 8) / 256);
  const long long tiles = p.packed ? p.Hkv * packed_units(p.B, p.total, kTile) : bkv * nT;
  const long long nbad = (8 * tiles + 255) / 256;
  const long long want = (rows * (D / 8) + 256 * kUnroll - 1) / (256 * kUnroll);
  const long long most = 8LL * sm_count();
  if (most <= 0) return cudaErrorInvalidDevice;
  const long long blocks = nsum + nbad + (want < most ? want : most);
  return launch_pdl(fa_window_finish_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                    stream, w, static_cast<int>(nsum), static_cast<int>(nbad));
}

}  // namespace

cudaError_t launch_window_finish(const WindowFinish& w, cudaStream_t stream) {
  return w.b.d == 64 ? launch_finish<64>(w, stream) : launch_finish<128>(w, stream);
}

namespace {

// How walks are cut.  The first key tiles': parts as long as the other tiles'
// walks, of 8 query tiles at least (a part ends with 128 KB of fp32 sums at
// d = 128, about what three tiles' products cost), or 2 where there are fewer
// key tiles than SMs.  Then the heads of a group go apart too, as far as
// there are SMs: 1024 rows of 16 heads (4 of K and V), window 256, 114 -> 45 us.
struct WalkSplit {
  int tiles, parts, part_tiles, group_parts;
  bool packed;           // units, slots and flags by where the sequences begin
  int slot_units;        // slots of a head (packed: of its first tiles each)
  long long slots;       // all of them
  long long bad_tiles;   // tiles with flags
};
// total: rows of a packed batch, else 0
WalkSplit walk_split(int B, int H, int Hkv, int N, int total, int d, int window, int sinks) {
  constexpr int kSms = 152;  // (not the device's: workspaces are sized without one)
  const long long nT = (N + kTile - 1) / kTile, units = static_cast<long long>(B) * Hkv * nT;
  const long long live = total > 0 ? Hkv * packed_units(B, total, kTile) : units;
  WalkSplit s;
  s.tiles = ((sinks < N ? sinks : N) + kTile - 1) / kTile;
  const int walk = (window - 2 + kTile) / kTile + 1;
  const int least = (live < units ? live : units) <= kSms ? 2 : 8;
  s.part_tiles = walk > least ? walk : least;
  s.parts = s.tiles ? (nT + s.part_tiles - 1) / s.part_tiles : 1;
  s.group_parts = 1;
  for (int g = 2; g <= H / Hkv && units * g <= kSms; ++g)
    if (H / Hkv % g == 0) s.group_parts = g;
  // Packed batches: units by where their sequences begin if they would mostly be
  // of tiles that do not exist, or if the walks of all sequences at once read
  // more of Q and dO than L2 keeps.  Else tile by tile, all sequences together:
  // the longest walks come first.  16 heads (4 of K and V), tile by tile | by
  // begin, us: 64 sequences of up to 2027 rows of 128, window 512, 1437 | 1241;
  // 16 of up to 4045, window 1024, 989 | 976; 64 of up to 509 rows of 64, window
  // 256, 135 | 147; one of 14000 among 63 of up to 199 (8 heads, 2) 386 | 313.
  const long long tiles_q = static_cast<long long>(B) * H * walk, all_q = H * (total / kTile + 1LL);
  const long long near = (tiles_q < all_q ? tiles_q : all_q) * 4 * kTile * d;
  s.packed = total > 0 && s.group_parts == 1 && (units > 3 * live || near > (96LL << 20));
  const long long L = static_cast<long long>(s.part_tiles) * kTile;
  const long long per = s.group_parts > 1 ? (nT + s.tiles * (s.parts - 1LL)) * s.group_parts
                        : s.parts == 1    ? 0
                        : s.packed        ? 2 * (total / L)
                                          : static_cast<long long>(s.tiles) * s.parts;
  s.slot_units = static_cast<int>(per);
  s.slots = per * Hkv * (s.packed ? s.tiles : B);
  s.bad_tiles = s.packed ? live : units;
  return s;
}

struct WindowWorkspace {
  float *delta, *dq_acc, *part;
  uint32_t* bad;
  int* unit_counter;  // [1]
  size_t bytes;
};
// rows: of all query slices
WindowWorkspace window_ws(void* ws, size_t rows, int d, const WalkSplit& s) {
  char* base = static_cast<char*>(ws);
  WindowWorkspace w;
  size_t at = 0;
  auto take = [&](size_t n) {
    char* x = base + at;
    at += align256(n);
    return x;
  };
  w.delta = reinterpret_cast<float*>(take(rows * sizeof(float)));
  w.dq_acc = reinterpret_cast<float*>(take(rows * d * sizeof(float)));
  w.part = reinterpret_cast<float*>(take(s.slots * 2 * kTile * d * sizeof(float)));
  w.bad = reinterpret_cast<uint32_t*>(take(s.bad_tiles * 8 * sizeof(uint32_t)));
  w.unit_counter = reinterpret_cast<int*>(take(sizeof(int)));
  w.bytes = at;
  return w;
}

constexpr int kMaxSinks = 1024;

// Sizes of both passes; a packed batch (cu_seqlens) has `total` rows.
fa_status check_window(bool packed, int B, int H, int Hkv, int N, int total, int d, float scale,
                       int window, int sinks) {
  if (B < 1 || H < 1 || total < 0) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || Hkv > H || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (sinks > kMaxSinks) return FA_ERR_UNSUPPORTED;
  if (packed) {
    if (total == 0) return FA_OK;
    if (N < 1 || N > total) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(H) * total * d >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  } else {
    if (N < 1 || total != 0) return FA_ERR_INVALID_ARG;
    // (step by step: the product of four ints passes 64 bits)
    const long long rows = static_cast<long long>(B) * H;
    if (rows >= (1LL << 31) || rows * N >= (1LL << 31) || rows * N * d >= (1LL << 31))
      return FA_ERR_UNSUPPORTED;
  }
  const long long bh = static_cast<long long>(B) * H, nT = (N + kTile - 1) / kTile;
  if (bh >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  const WalkSplit s =
      walk_split(B, H, Hkv, N, packed ? total : 0, d, window < N ? window : N, sinks);
  const long long units = bh * (nT + static_cast<long long>(s.tiles) * s.parts);
  // units, and a row of the last kernel's 256 each, are counted in 32 bits
  const long long some = !s.packed ? units
                                 : H * (packed_units(B, total, kTile) +
                                        s.tiles * packed_units(B, total, s.part_tiles * kTile));
  if (some >= (1LL << 23) || units >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_forward_window(const void* q, const void* k, const void* v, void* o, float* lse,
                            const int* cu_seqlens, int B, int H, int Hkv, int N, int total, int d,
                            float scale, int window, int sinks, cudaStream_t stream) {
  using namespace fa;
  FA_TRY(check_window(cu_seqlens != nullptr, B, H, Hkv, N, total, d, scale, window, sinks));
  if (cu_seqlens) {
    FA_TRY(check_ptr4(cu_seqlens));
    if (total == 0) return FA_OK;  // every sequence empty: nothing to write
  }
  for (const void* x : {q, k, v, static_cast<const void*>(o)}) FA_TRY(check_ptr16(x));
  FA_TRY(check_ptr4(lse));
  fa_status st = FA_OK;
  int* err = status_word(&st);
  if (!err) return st;
  const int zq = cu_seqlens ? H : B * H, zkv = cu_seqlens ? Hkv : B * Hkv;
  const int rows = cu_seqlens ? total : N;
  CUtensorMap tq, tk, tv;
  if (!make_tile_map(&tq, q, zq, rows, d) || !make_tile_map(&tk, k, zkv, rows, d) ||
      !make_tile_map(&tv, v, zkv, rows, d))
    return FA_ERR_CUDA;
  FwdParams p;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.scale = scale;
  p.causal = 1;
  p.cu_seqlens = cu_seqlens;
  p.total = total;
  p.window = window < N ? window : N;
  p.sinks = sinks;
  p.q = q;
  p.k = k;
  p.v = v;
  p.err = err;
  p.wait_ns = wait_limit_ns();
  FA_CUDA(launch_forward(p, tq, tk, tv, stream));
  return FA_OK;
}

size_t fa_backward_window_workspace_size(int B, int H, int Hkv, int N, int total, int d,
                                         int window, int sinks) {
  using namespace fa;
  if (check_window(total > 0, B, H, Hkv, N, total, d, 1.f, window, sinks) != FA_OK) return 0;
  const size_t rows = total > 0 ? static_cast<size_t>(H) * total : static_cast<size_t>(B) * H * N;
  return window_ws(nullptr, rows, d,
                   walk_split(B, H, Hkv, N, total, d, window < N ? window : N, sinks))
      .bytes;
}

fa_status fa_backward_window(const void* q, const void* k, const void* v, const void* o,
                             const void* dO, const float* lse, void* dq, void* dk, void* dv,
                             const int* cu_seqlens, int B, int H, int Hkv, int N, int total, int d,
                             float scale, int window, int sinks, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  using namespace fa;
  FA_TRY(check_window(cu_seqlens != nullptr, B, H, Hkv, N, total, d, scale, window, sinks));
  if (cu_seqlens) {
    FA_TRY(check_ptr4(cu_seqlens));
    if (total == 0) return FA_OK;  // every sequence empty: nothing to write
  }
  for (const void* x : {q, k, v, o, dO, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    FA_TRY(check_ptr16(x));
  FA_TRY(check_ptr4(lse));
  if (window > N) window = N;
  const WalkSplit split = walk_split(B, H, Hkv, N, total, d, window, sinks);
  const int zq = cu_seqlens ? H : B * H, zkv = cu_seqlens ? Hkv : B * Hkv;
  const int rows = cu_seqlens ? total : N;
  const long long qrows = static_cast<long long>(zq) * rows;
  const WindowWorkspace ws = window_ws(workspace, qrows, d, split);
  FA_TRY(check_ws(workspace, workspace_bytes, ws.bytes));
  fa_status st = FA_OK;
  int* err = status_word(&st);
  if (!err) return st;
  CUtensorMap tq, tk, tv, tdo, tdq;
  if (!make_tile_map(&tq, q, zq, rows, d) || !make_tile_map(&tk, k, zkv, rows, d) ||
      !make_tile_map(&tv, v, zkv, rows, d) || !make_tile_map(&tdo, dO, zq, rows, d) ||
      !make_acc_map(&tdq, ws.dq_acc, zq, rows, d))
    return FA_ERR_CUDA;
  FA_CUDA(launch_bwd_preprocess(o, dO, ws.delta, ws.dq_acc, ws.unit_counter, 1, qrows, d,
                                stream));
  WindowFinish w;
  BwdParams& p = w.b;
  p.lse = lse;
  p.delta = ws.delta;
  p.dq_acc = ws.dq_acc;
  p.dk = dk;
  p.dv = dv;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.scale = scale;
  p.causal = 1;
  p.cu_seqlens = cu_seqlens;
  p.total = total;
  p.part = ws.part;
  p.window = window;
  p.sinks = sinks;
  p.sink_tiles = split.tiles;
  p.sink_parts = split.parts;
  p.part_tiles = split.part_tiles;
  p.group_parts = split.group_parts;
  p.slot_units = split.slot_units;
  p.packed = split.packed;
  p.bad = ws.bad;
  p.unit_counter = ws.unit_counter;
  p.err = err;
  p.wait_ns = wait_limit_ns();
  FA_CUDA(launch_backward_main(p, tq, tk, tv, tdo, tdq, stream));
  w.q = q;
  w.k = k;
  w.v = v;
  w.dO = dO;
  w.dq = dq;
  FA_CUDA(launch_window_finish(w, stream));
  return FA_OK;
}

}  // extern "C"
