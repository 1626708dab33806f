// Bookkeeping of the paged cache: fa_cache_plan (pages, slot map, positions and tree
// masks from request lengths) and fa_cache_commit (the accepted path moved forward).
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_cache.h"
#include "tma_host.h"

namespace fa {
namespace {

// ------------------------------------------------------------------ plan
//
// Latency bound: the floor is a launch and the loads that wait for one another (lengths, free
// pages, table). Measured, back to back and with every page already held: 4.3 us for 8 requests' next
// tokens, 6.4 for 256 trees of up to 64 tokens (16.5 with pages by a warp per request and the trees
// behind them in the same CTAs). The pages are handed out by one cluster of 8 CTAs, so that the two
// places where all requests meet (pages given back, if there are any, before any is taken; tables
// written before slots are read) are cluster barriers and the whole plan is one launch. Every CTA reads
// all lengths and scans the needs itself, one load's latency, which is cheaper than handing prefix sums
// around; pages are then given out a thread per page and slots a thread per row.
//
// Tree masks need no pages: further clusters build them at the same time. The set of a token's
// ancestors by pointer doubling: with A_t the mask known so far and up_t the first token not in
// it, A_t |= A_{up_t}, up_t = up_{up_t} doubles the covered path each round, so
// ceil(log2(max_new)) rounds suffice; the depth is the number of bits minus one. One thread per
// token, groups of threads (a power of two >= max_new) per request.

constexpr int kPlanThreads = 512;
constexpr int kPlanCtas = 8;
constexpr int kPlanPer = kCacheMaxB / kPlanThreads;  // requests scanned by a thread
constexpr int kPlanRows = 4;                         // rows a thread has in flight

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sums of x and y over the CTA; `all_x`, `all_y` get the sums. `sums` holds two
// words per warp.
__device__ __forceinline__ void scan_exclusive(int& x, int& y, int* sums, int& all_x, int& all_y) {
  constexpr int kWarps = kPlanThreads / 32;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int s = x, t = y;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, k), v = __shfl_up_sync(0xffffffffu, t, k);
    if (lane >= k) {
      s += u;
      t += v;
    }
  }
  if (lane == 31) {
    sums[warp] = s;
    sums[kWarps + warp] = t;
  }
  __syncthreads();
  all_x = all_y = 0;
  int before_x = 0, before_y = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int u = sums[i], v = sums[kWarps + i];
    before_x += i < warp ? u : 0;
    before_y += i < warp ? v : 0;
    all_x += u;
    all_y += v;
  }
  x = before_x + s - x;
  y = before_y + t - y;
}

// The last b of [0, B) with first[b] <= x (first[0] <= x; `first` does not fall).
__device__ __forceinline__ int find_last(const int* first, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Pages, state, slots (and positions, without trees) by the first cluster.
__device__ __forceinline__ void plan_pages(const PlanArgs& p, int* smem) {
  __shared__ int sums[2 * kPlanThreads / 32];
  int* s_cu = smem;               // [B + 1]
  int* s_need = s_cu + p.B + 1;   // [B] pages taken by the requests before b
  int* s_give = s_need + p.B;     // [B] pages given back before b
  int* s_held = s_give + p.B;     // [B]
  int* s_want = s_held + p.B;     // [B] -1: takes no part
  int* s_ctx = s_want + p.B;      // [B]
  const int tid = threadIdx.x, rank = blockIdx.x;
  constexpr int kAll = kPlanCtas * kPlanThreads;
  const int me = rank * kPlanThreads + tid;
  const int free0 = min(max(*p.free_count, 0), p.num_pages);

  // Thread t scans requests t * per .. t * per + per - 1.
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  int need = 0, give = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.B) {
      const int ctx = p.ctx_len[b], cu = p.cu_new[b];
      const long long n = static_cast<long long>(p.cu_new[b + 1]) - cu;
      const int held = min(max(p.n_pages[b], 0), p.max_pages);
      const long long pages = (static_cast<long long>(ctx) + n + (1 << p.page_shift) - 1) >> p.page_shift;
      // New rows behind the buffers get no slot and so are never written: none of the request's are then.
      const bool inside = (n == 0) | ((cu >= 0) & (cu + n <= p.rows));
      const bool ok = (ctx >= 0) & (n >= 0) & (n <= p.max_new) & inside & (pages <= p.max_pages);
      const int want = ok ? static_cast<int>(pages) : -1;
      s_cu[b] = cu;
      s_ctx[b] = ctx;
      s_held[b] = held;
      s_want[b] = want;
      s_need[b] = ok ? max(want - held, 0) : 0;
      s_give[b] = ok ? max(held - want, 0) : 0;
      need += s_need[b];
      give += s_give[b];
    }
  }
  if (tid == 0) s_cu[p.B] = p.cu_new[p.B];
  int need_all, give_all;
  scan_exclusive(need, give, sums, need_all, give_all);
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.B) {
      const int x = s_need[b], y = s_give[b];
      s_need[b] = need;
      s_give[b] = give;
      need += x;
      give += y;
    }
  }
  __syncthreads();
  auto need_upto = [&](int b) { return b + 1 < p.B ? s_need[b + 1] : need_all; };  // by requests 0 .. b
  const int free1 = min(free0 + give_all, p.num_pages);

  // Pages given back, then (behind them) pages taken, a thread per page. give_all is the same in
  // all CTAs of the cluster, so they agree on the barrier.
  if (give_all > 0) {
    for (int k = me; k < give_all; k += kAll) {
      const int b = find_last(s_give, p.B, k);
      int32_t* entry = p.block_table + static_cast<size_t>(b) * p.max_pages + s_want[b] + (k - s_give[b]);
      if (free0 + k < p.num_pages) p.free_list[free0 + k] = *entry;
      *entry = -1;
    }
    cluster_barrier();
  }
  for (int k = me; k < min(need_all, free1); k += kAll) {
    const int b = find_last(s_need, p.B, k);
    if (need_upto(b) <= free1)
      p.block_table[static_cast<size_t>(b) * p.max_pages + s_held[b] + (k - s_need[b])] = p.free_list[free1 - 1 - k];
  }
  cluster_barrier();  // the tables are written, and every CTA has read the state

  auto granted = [&](int b) { return s_want[b] >= 0 && (s_want[b] <= s_held[b] || need_upto(b) <= free1); };
  for (int b = me; b < p.B; b += kAll) {
    const bool yes = granted(b);
    if (yes) p.n_pages[b] = s_want[b];
    p.seq_len[b] = yes ? s_ctx[b] + (s_cu[b + 1] - s_cu[b]) : 0;
  }
  if (me == 0) {
    // The needs' sums grow, so the granted ones are the first of them.
    int b = p.B - 1;
    while (b >= 0 && need_upto(b) > free1) --b;
    *p.free_count = free1 - (b >= 0 ? need_upto(b) : 0);
  }

  // Slots, a thread per row, a few rows at a time.
  const int page_mask = (1 << p.page_shift) - 1;
  for (int t0 = me; t0 < p.rows; t0 += kPlanRows * kAll) {
    int at[kPlanRows], page[kPlanRows];
    bool inside[kPlanRows], few[kPlanRows];
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      const int t = t0 + k * kAll;
      at[k] = 0;
      page[k] = -1;
      inside[k] = few[k] = false;
      if (t < p.rows) {
        const int b = find_last(s_cu, p.B, t);
        const int i = t - s_cu[b], n = s_cu[b + 1] - s_cu[b];
        inside[k] = i >= 0 && i < n;
        few[k] = n <= p.max_new;
        at[k] = inside[k] ? s_ctx[b] + i : 0;
        if (inside[k] && granted(b)) page[k] = p.block_table[static_cast<size_t>(b) * p.max_pages + (at[k] >> p.page_shift)];
      }
    }
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      const int t = t0 + k * kAll;
      if (t < p.rows) {
        const bool there = page[k] >= 0 && page[k] < p.num_pages;
        p.slot[t] = there ? (page[k] << p.page_shift) + (at[k] & page_mask) : -1;
        if (p.parent == nullptr || !inside[k] || !few[k]) p.position[t] = at[k];
      }
    }
  }
}

// Masks and positions of drafted trees, by the CTAs behind the first cluster.
__device__ __forceinline__ void plan_trees(const PlanArgs& p, int* smem, int cta, int ctas) {
  int group = 32;
  while (group < p.max_new) group <<= 1;
  unsigned long long* s_mask = reinterpret_cast<unsigned long long*>(smem);              // [threads][words]
  int* s_up = reinterpret_cast<int*>(s_mask + static_cast<size_t>(kPlanThreads) * p.words);  // [threads]
  const int tid = threadIdx.x, groups = kPlanThreads / group;
  const int g = tid / group, i = tid % group, base = g * group;
  const int rounds = 32 - __clz(max(p.max_new - 1, 1));
  for (int b0 = cta * groups; b0 < p.B; b0 += ctas * groups) {
    const int b = b0 + g;
    const int start = b < p.B ? p.cu_new[b] : 0;
    const long long n = b < p.B ? static_cast<long long>(p.cu_new[b + 1]) - start : 0;
    const bool mine = n <= p.max_new && i < n && start >= 0 && start < p.rows - i;
    int up = -1, ctx = 0;
    if (mine) {
      ctx = p.ctx_len[b];
      up = p.parent[start + i];
      if (up < 0 || up >= i) up = -1;
    }
    unsigned long long m[FA_TREE_MAX / 64];
#pragma unroll
    for (int w = 0; w < FA_TREE_MAX / 64; ++w) {
      m[w] = (w == i / 64) ? 1ull << (i % 64) : 0ull;
      if (w < p.words) s_mask[tid * p.words + w] = m[w];
    }
    s_up[tid] = up;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
      int next = up;
      if (up >= 0) {
        next = s_up[base + up];
#pragma unroll
        for (int w = 0; w < FA_TREE_MAX / 64; ++w)
          if (w < p.words) m[w] |= s_mask[(base + up) * p.words + w];
      }
      __syncthreads();
      up = next;
      s_up[tid] = up;
#pragma unroll
      for (int w = 0; w < FA_TREE_MAX / 64; ++w)
        if (w < p.words) s_mask[tid * p.words + w] = m[w];
      __syncthreads();
    }
    if (mine) {
      int bits = 0;
#pragma unroll
      for (int w = 0; w < FA_TREE_MAX / 64; ++w) {
        if (w < p.words) {
          p.tree_mask[static_cast<size_t>(start + i) * p.words + w] = m[w];
          bits += __popcll(m[w]);
        }
      }
      p.position[start + i] = ctx + bits - 1;
    }
  }
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    fa_cache_plan_kernel(const __grid_constant__ PlanArgs p) {
  extern __shared__ __align__(8) int plan_smem[];
  if (blockIdx.x < kPlanCtas) plan_pages(p, plan_smem);
  else plan_trees(p, plan_smem, blockIdx.x - kPlanCtas, gridDim.x - kPlanCtas);
}

// ------------------------------------------------------------------ commit
//
// A CTA per request; a thread owns one 16-byte column of K or V of one head and moves
// it along the whole path, a batch of rows at a time (all loads of a batch before its
// stores). The indices are strictly increasing, so a row's target never lies behind
// the source of a later one and no order between threads is needed. It moves a few
// rows of each request and is bound by latency: lengths, then the table, then the rows (256
// requests, about 6 rows of 2 x 8 heads of 128 each: 6.1 us, 13.6 MB).

constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 8;
constexpr int kCommitChunk = 128;  // path entries whose addresses are held at a time

__global__ void __launch_bounds__(kCommitThreads) fa_cache_commit_kernel(const CommitArgs p) {
  __shared__ long long s_src[kCommitChunk], s_dst[kCommitChunk];
  __shared__ int s_stop;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int ctx = p.ctx_len[b];
  const int count = min(max(p.n_accepted[b], 0), p.max_accept);
  const int32_t* acc = p.accepted + static_cast<size_t>(b) * p.max_accept;
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  const int mask = (1 << p.page_shift) - 1;
  const int vecs = p.d / 8, columns = p.H_kv * vecs;
  if (tid == 0) s_stop = ctx < 0 ? 0 : count;
  __syncthreads();
  int kept = 0;
  for (int j0 = 0; j0 < count; j0 += kCommitChunk) {
    const int j = j0 + tid;
    if (tid < kCommitChunk && j < count) {
      const int from = acc[j], before = j > 0 ? acc[j - 1] : -1;
      long long src = -1, dst = -1;
      const long long rs = static_cast<long long>(ctx) + from, rd = static_cast<long long>(ctx) + j;
      if (from > before && from >= 0 && ctx >= 0 && (rs >> p.page_shift) < p.max_pages) {
        const int ps = table[rs >> p.page_shift], pd = table[rd >> p.page_shift];  // rd <= rs
        if (ps >= 0 && ps < p.num_pages && pd >= 0 && pd < p.num_pages) {
          src = ps * p.page_stride + (rs & mask) * p.row_stride;
          dst = pd * p.page_stride + (rd & mask) * p.row_stride;
        }
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
      if (src < 0) atomicMin(&s_stop, j);
    }
    __syncthreads();
    const int stop = min(s_stop, j0 + kCommitChunk);
    for (int c = tid; c < 2 * columns; c += kCommitThreads) {
      const int col = c % columns;
      uint16_t* base = (c < columns ? p.k : p.v) + (col / vecs) * p.head_stride + (col % vecs) * 8;
      for (int e = j0; e < stop; e += kCommitBatch) {
        uint4 x[kCommitBatch];
#pragma unroll
        for (int u = 0; u < kCommitBatch; ++u)
          if (e + u < stop) x[u] = *reinterpret_cast<const uint4*>(base + s_src[e + u - j0]);
#pragma unroll
        for (int u = 0; u < kCommitBatch; ++u)
          if (e + u < stop && s_src[e + u - j0] != s_dst[e + u - j0])
            *reinterpret_cast<uint4*>(base + s_dst[e + u - j0]) = x[u];
      }
    }
    kept = min(stop, count);
    __syncthreads();
    if (s_stop < j0 + kCommitChunk) break;
  }
  if (tid == 0) p.new_len[b] = ctx + (count > 0 ? kept : 0);
}

}  // namespace

int launch_cache_plan(const PlanArgs& a, cudaStream_t stream) {
  size_t bytes = static_cast<size_t>(6 * a.B + 1) * 4;
  unsigned clusters = 1;
  if (a.parent != nullptr) {
    const size_t trees = static_cast<size_t>(kPlanThreads) * (8 * a.words + 4);
    bytes = bytes > trees ? bytes : trees;
    int group = 32;
    while (group < a.max_new) group <<= 1;
    const int ctas = (a.B + kPlanThreads / group - 1) / (kPlanThreads / group);
    const int more = (ctas + kPlanCtas - 1) / kPlanCtas;
    clusters += more < 17 ? more : 17;  // 18 clusters of 8 fill the SMs
  }
  if (bytes > 48 * 1024) {
    const cudaError_t e = host::ensure_dynamic_smem(reinterpret_cast<const void*>(fa_cache_plan_kernel), 100 * 1024);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  fa_cache_plan_kernel<<<clusters * kPlanCtas, kPlanThreads, bytes, stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

int launch_cache_commit(const CommitArgs& a, cudaStream_t stream) {
  fa_cache_commit_kernel<<<static_cast<unsigned>(a.B), kCommitThreads, 0, stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
