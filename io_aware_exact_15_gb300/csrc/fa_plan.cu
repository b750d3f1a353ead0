// Page tables, slots and positions of a serving step, from the requests'
// lengths: what the host would otherwise work out and copy over.
//
// Integer work on a few words per request, bound by latency: a chain of
// dependent loads (lengths, table entries, line of free pages) and prefix sums
// over the requests, so everything but long lists of slots happens in one
// launch of one cluster: its blocks exchange their sums through distributed
// shared memory and order pushes before pops with cluster barriers, where
// separate kernels would cost a launch each.
//
// Order of events, the same on every run: the pages that go back join the end
// of the line, by request and position; then missing pages are taken from its
// front, by request and position.  A request is a lane's matter while it
// touches up to 4 table entries (a decode step), the whole warp's beyond.
//
// Measured, a call among others, on a table where no page is missing or behind
// the window: 64 requests of one token, window 1024: 6.0 us; 512 prompts of up
// to 2048 tokens: 9.9 us with the second kernel (8 MB of slots and positions:
// 1.2 us at a plain copy's rate).  Both are a launch's time, four or five
// dependent loads and two cluster barriers.  On tables that miss the new
// tokens' pages (and hold some behind the window), in a graph, such | the
// above: 5.0 | 4.4 us, and 11.9 | 10.5 (10648 pages taken).
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kPlanWarps = 32;      // warps of a block
constexpr int kPlanCluster = 8;     // blocks of the cluster, at most
constexpr int kMaxRequests = 32 * kPlanWarps * kPlanCluster;
constexpr int kFew = 4;             // table entries, tokens that a lane does itself

struct PlanParams {
  const int *lens, *counts;
  int *table, *line, *state;
  long long* slots;
  int *positions, *cu, *granted;
  int B, max_tokens, num_pages, log_page, max_pages, window, sinks;
  int per_warp;   // requests of a warp
  int expand;     // 1: this kernel writes slots and positions too
};

FA_DEV void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
FA_DEV void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
FA_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
FA_DEV void st_cluster_u64(uint32_t smem, uint32_t rank, unsigned long long v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// exclusive sum over the lanes
template <class T>
FA_DEV T lanes_before(T v, int lane) {
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  return incl - v;
}

// tokens n of a request: slot and position; `off` its first place in the list
FA_DEV void write_token(const PlanParams& p, const int* row, long long off, int n, int len,
                        int granted) {
  const long long at = off + n;
  if (at >= p.max_tokens) return;
  const int pos = len + n;
  long long slot = -1;
  if (n < granted)
    slot = (static_cast<long long>(row[pos >> p.log_page]) << p.log_page) |
           (pos & ((1 << p.log_page) - 1));
  p.slots[at] = slot;
  p.positions[at] = pos;
}

__global__ void __launch_bounds__(32 * kPlanWarps, 1) fa_plan_kernel(const PlanParams p) {
  __shared__ unsigned long long warp_sum[3][kPlanWarps];     // tokens, pages back, pages missing
  __shared__ unsigned long long block_sum[3][kPlanCluster];  // of every block, written by each
  cluster_arrive();  // this block runs: its shared memory can be written
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), blocks = gridDim.x;
  const int num = p.num_pages, cap = p.max_pages << p.log_page;
  const int b = (rank * kPlanWarps + warp) * p.per_warp + lane;
  const bool mine = lane < p.per_warp && b < p.B;
  const unsigned head = static_cast<unsigned>(p.state[0]) % static_cast<unsigned>(num);
  const int count = min(max(p.state[1], 0), num);
  auto page_ok = [&](int id) { return id >= 0 && id < num; };
  auto row_of = [&](int r) { return p.table + static_cast<size_t>(r) * p.max_pages; };
  auto place = [&](long long i) {  // i-th place of the line, i < num
    const unsigned x = head + static_cast<unsigned>(i);
    return p.line + (x >= static_cast<unsigned>(num) ? x - num : x);
  };

  // ------------------------------------------------ what each request needs
  int len = 0, tok = 0, fit = 0;
  bool ended = false;
  if (mine) {
    len = min(max(p.lens[b], 0), cap);
    const int c = p.counts[b];
    ended = c < 0;
    tok = max(c, 0);
    fit = min(tok, cap - len);
  }
  int* row = row_of(mine ? b : 0);
  // pages [back0, back1) go back: the run of pages below the window's edge
  // (ended requests: every page of the row)
  const int edge = p.window ? max(len - p.window + 1, 0) >> p.log_page : 0;
  const int keep = static_cast<int>(((static_cast<long long>(p.sinks) - 1) >> p.log_page) + 1);
  const int first = len >> p.log_page, last = fit > 0 ? (len + fit - 1) >> p.log_page : first - 1;
  int back = 0, missing = 0;
  bool more = ended;
  if (mine && !ended) {
    int id[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) id[i] = edge - 1 - i >= keep ? row[edge - 1 - i] : -1;
    bool run = true;
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      run = run && page_ok(id[i]);
      back += run;
    }
    more = run && edge - kFew > keep;
    if (last - first < kFew) {
#pragma unroll
      for (int i = 0; i < kFew; ++i) id[i] = first + i <= last ? row[first + i] : 0;
#pragma unroll
      for (int i = 0; i < kFew; ++i) missing += first + i <= last && !page_ok(id[i]);
    }
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, more); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    const int* r = row_of(__shfl_sync(0xffffffffu, b, from));
    const int e = __shfl_sync(0xffffffffu, edge, from);
    int n = 0;
    if (__shfl_sync(0xffffffffu, ended, from)) {
      for (int i = 0; i < p.max_pages; i += 32)
        n += __popc(__ballot_sync(0xffffffffu, i + lane < p.max_pages && page_ok(r[i + lane])));
    } else {
      for (int i = e - 1; i >= keep; i -= 32) {
        const uint32_t gone =
            ~__ballot_sync(0xffffffffu, i - lane >= keep && page_ok(r[i - lane]));
        n += gone ? __ffs(gone) - 1 : 32;
        if (gone) break;
      }
    }
    if (lane == from) back = n;
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, last - first >= kFew); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    const int* r = row_of(__shfl_sync(0xffffffffu, b, from));
    const int i0 = __shfl_sync(0xffffffffu, first, from), i1 = __shfl_sync(0xffffffffu, last, from);
    int n = 0;
#pragma unroll 2
    for (int i = i0; i <= i1; i += 32)
      n += __popc(__ballot_sync(0xffffffffu, i + lane <= i1 && !page_ok(r[i + lane])));
    if (lane == from) missing = n;
  }

  // ------------------------------------------------ sums over the requests
  long long off[3] = {tok, back, missing};  // then: of the requests before
  {
    long long before[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      before[i] = lanes_before(off[i], lane);
      if (lane == 31) warp_sum[i][warp] = before[i] + off[i];
      off[i] = before[i];
    }
  }
  __syncthreads();
  cluster_wait();
  if (warp < 3) {
    const unsigned long long x = warp_sum[warp][lane], at = lanes_before(x, lane);
    warp_sum[warp][lane] = at;
    const unsigned long long all = __shfl_sync(0xffffffffu, at + x, 31);
    if (lane < blocks) st_cluster_u64(smem_u32(&block_sum[warp][rank]), lane, all);
  }
  cluster_arrive();
  cluster_wait();
  long long total[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    off[i] += warp_sum[i][warp];
    for (int r = 0; r < blocks; ++r) {
      const long long x = block_sum[i][r];
      total[i] += x;
      if (r < rank) off[i] += x;
    }
  }
  const long long pushed = min(total[1], static_cast<long long>(num - count));
  const long long avail = count + pushed;
  const long long taken = min(total[2], avail);

  // ------------------------------------------------ pages go back
  // (a line that would hold more than every page, from a table with a page in
  // it twice, loses the rest)
  if (mine && !ended && back <= kFew) {
    for (int i = 0; i < back; ++i) {
      int* e = row + edge - back + i;
      if (count + off[1] + i < num) *place(count + off[1] + i) = *e;
      *e = -1;
    }
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, mine && (ended || back > kFew)); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    int* r = row_of(__shfl_sync(0xffffffffu, b, from));
    const bool all = __shfl_sync(0xffffffffu, ended, from);
    const int i1 = all ? p.max_pages : __shfl_sync(0xffffffffu, edge, from);
    const int i0 = all ? 0 : i1 - __shfl_sync(0xffffffffu, back, from);
    long long at = count + __shfl_sync(0xffffffffu, off[1], from);
    for (int i = i0; i < i1; i += 32) {
      const int id = i + lane < i1 ? r[i + lane] : -1;
      const uint32_t some = __ballot_sync(0xffffffffu, page_ok(id));
      const long long to = at + __popc(some & low_bits(lane));
      if (page_ok(id) && to < num) *place(to) = id;
      if (i + lane < i1) r[i + lane] = -1;
      at += __popc(some);
    }
  }
  // pops need to see the pushes only where they reach them
  if (total[2] > count) {
    cluster_arrive();
    cluster_wait();
  }

  // ------------------------------------------------ missing pages are taken
  // granted: tokens up to the first page that the line could not give
  int granted = fit;
  if (mine && missing && last - first < kFew) {
    long long at = off[2];
    bool dry = false;
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      if (first + i > last || page_ok(row[first + i]) || dry) continue;
      if (at < avail) {
        row[first + i] = __ldcg(place(at));
        ++at;
      } else {
        dry = true;
        granted = min(fit, max(((first + i) << p.log_page) - len, 0));
      }
    }
  }
  __syncwarp();
  for (uint32_t m = __ballot_sync(0xffffffffu, missing && last - first >= kFew); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    int* r = row_of(__shfl_sync(0xffffffffu, b, from));
    const int i0 = __shfl_sync(0xffffffffu, first, from), i1 = __shfl_sync(0xffffffffu, last, from);
    long long at = __shfl_sync(0xffffffffu, off[2], from);
    int dry = -1;  // the first page without one
    for (int i = i0; i <= i1 && dry < 0; i += 32) {
      const bool want = i + lane <= i1 && !page_ok(r[i + lane]);
      const uint32_t some = __ballot_sync(0xffffffffu, want);
      const long long k = at + __popc(some & low_bits(lane));
      if (want && k < avail) r[i + lane] = __ldcg(place(k));
      const uint32_t none = __ballot_sync(0xffffffffu, want && k >= avail);
      if (none) dry = i + __ffs(none) - 1;
      at += __popc(some);
    }
    if (lane == from && dry >= 0) granted = min(fit, max((dry << p.log_page) - len, 0));
  }
  __syncwarp();
  if (mine) {
    granted = static_cast<int>(
        min(static_cast<long long>(granted), max(p.max_tokens - off[0], 0LL)));
    p.granted[b] = granted;
    p.cu[b] = static_cast<int>(min(off[0], static_cast<long long>(p.max_tokens)));
  }
  const int listed = static_cast<int>(min(total[0], static_cast<long long>(p.max_tokens)));
  if (rank == 0 && threadIdx.x == 0) {
    p.cu[p.B] = listed;
    p.state[0] = static_cast<int>((head + static_cast<unsigned long long>(taken)) %
                                  static_cast<unsigned>(num));
    p.state[1] = static_cast<int>(avail - taken);
  }
  if (!p.expand) return;

  // ------------------------------------------------ slots and positions
  if (mine && tok <= kFew)
    for (int n = 0; n < tok; ++n) write_token(p, row, off[0], n, len, granted);
  for (uint32_t m = __ballot_sync(0xffffffffu, tok > kFew); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    const int* r = row_of(__shfl_sync(0xffffffffu, b, from));
    const long long at = __shfl_sync(0xffffffffu, off[0], from);
    const int l = __shfl_sync(0xffffffffu, len, from), g = __shfl_sync(0xffffffffu, granted, from);
    const int n = static_cast<int>(min(static_cast<long long>(__shfl_sync(0xffffffffu, tok, from)),
                                       max(p.max_tokens - at, 0LL)));
#pragma unroll 4
    for (int i = lane; i < n; i += 32) write_token(p, r, at, i, l, g);
  }
  for (int i = listed + rank * blockDim.x + threadIdx.x; i < p.max_tokens;
       i += blocks * blockDim.x) {
    p.slots[i] = -1;
    p.positions[i] = 0;
  }
}

// The last of cu[lo .. hi - 1] (ascending) that is <= t, with cu[lo] <= t: 32
// places looked at together.  Whole warp.
FA_DEV int last_begin(const int* cu, int lo, int hi, int t, int lane) {
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
    const int last = 31 - __clz(le);  // lane 0 always is
    hi = min(hi, lo + (last + 1) * step);
    lo += last * step;
  }
  return lo;
}

// Slots and positions of long lists, over the whole GPU: a warp takes 32
// kTokens consecutive ones, finds the requests of its first and last token,
// and each lane those of its own between them (in a prompt they are the same).
constexpr int kTokens = 4;
__global__ void __launch_bounds__(256) fa_plan_tokens_kernel(const PlanParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long t0 =
      (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x - lane) * kTokens;
  const int listed = p.cu[p.B], cap = p.max_pages << p.log_page;
  int b0 = 0, b1 = 0;
  if (t0 < listed) {
    const int t1 = static_cast<int>(min(t0 + 32 * kTokens, static_cast<long long>(listed))) - 1;
    b0 = last_begin(p.cu, 0, p.B, static_cast<int>(t0), lane);
    b1 = p.cu[b0 + 1] > t1 ? b0 : last_begin(p.cu, b0, p.B, t1, lane);
  }
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const long long at = t0 + 32 * k + lane;
    if (at >= p.max_tokens) return;
    const int t = static_cast<int>(at);
    if (t >= listed) {
      p.slots[t] = -1;
      p.positions[t] = 0;
      continue;
    }
    int b = b0, hi = b1 + 1;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      (p.cu[mid] <= t ? b : hi) = mid;
    }
    const int begin = p.cu[b];
    write_token(p, p.table + static_cast<size_t>(b) * p.max_pages, begin, t - begin,
                min(max(p.lens[b], 0), cap), p.granted[b]);
  }
}

// Up to this many tokens the cluster writes their slots itself.
constexpr int kExpandHere = 8192;

cudaError_t launch_plan(PlanParams p, cudaStream_t stream) {
  // one request per warp while the cluster has warps for them
  int blocks = (p.B + kPlanWarps - 1) / kPlanWarps;
  blocks = blocks >= kPlanCluster ? kPlanCluster : blocks > 4 ? 8 : blocks > 2 ? 4 : blocks;
  p.per_warp = (p.B + blocks * kPlanWarps - 1) / (blocks * kPlanWarps);
  p.expand = p.max_tokens <= kExpandHere;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(32 * kPlanWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_plan_kernel, p);
  if (e != cudaSuccess || p.expand) return e;
  const long long threads = (static_cast<long long>(p.max_tokens) + kTokens - 1) / kTokens;
  return launch_pdl(fa_plan_tokens_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)),
                    dim3(256), 0, stream, p);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_plan(const int* lens, const int* counts, int* page_table, int* free_pages,
                        int* free_state, long long* slots, int* positions, int* cu_seqlens,
                        int* granted, int B, int max_tokens, int num_pages, int page_size,
                        int max_pages, int window, int sinks, cudaStream_t stream) {
  using namespace fa;
  if (B < 1 || max_tokens < 0 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (log2_page(page_size) < 0 || B > kMaxRequests) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (max_tokens > (1 << 30)) return FA_ERR_UNSUPPORTED;  // (positions fit in 31 bits)
  for (const void* x : {static_cast<const void*>(lens), static_cast<const void*>(counts),
                        static_cast<const void*>(page_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(free_state),
                        static_cast<const void*>(cu_seqlens), static_cast<const void*>(granted)})
    FA_TRY(check_ptr4(x));
  if (max_tokens > 0) {
    FA_TRY(check_ptr4(positions));
    if (!slots) return FA_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return FA_ERR_MISALIGNED;
  }
  PlanParams p = {};
  p.lens = lens;
  p.counts = counts;
  p.table = page_table;
  p.line = free_pages;
  p.state = free_state;
  p.slots = slots;
  p.positions = positions;
  p.cu = cu_seqlens;
  p.granted = granted;
  p.B = B;
  p.max_tokens = max_tokens;
  p.num_pages = num_pages;
  p.log_page = log2_page(page_size);
  p.max_pages = max_pages;
  // positions stay below 2^30: no window is longer
  p.window = window < (1 << 30) ? window : 1 << 30;
  p.sinks = sinks;
  FA_CUDA(launch_plan(p, stream));
  return FA_OK;
}

}  // extern "C"
