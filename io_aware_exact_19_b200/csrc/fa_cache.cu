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
// One cluster of 8 CTAs, so that the two places where all requests meet (pages given
// back before any is taken, tables written before slots are read) are cluster barriers
// and the whole plan is one launch. It is latency bound: the floor is a launch and a
// handful of dependent loads. Every CTA reads all lengths and scans the needs itself
// (a few loads a thread), which is cheaper than handing prefix sums around.
//
// Tree masks: the set of a token's ancestors by pointer doubling. With A_t the mask
// known so far and up_t the first token not in it, A_t |= A_{up_t}, up_t = up_{up_t}
// doubles the covered path each round, so ceil(log2(max_new)) rounds suffice; the
// depth is the number of bits minus one. One thread per token, groups of threads
// (a power of two >= max_new) per request.

constexpr int kPlanThreads = 512;
constexpr int kPlanCtas = 8;
constexpr int kPlanPer = kCacheMaxB / kPlanThreads;  // requests scanned by a thread

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum of x over the CTA; `total` gets the sum. `warp_sums` holds a word per warp.
__device__ __forceinline__ int scan_exclusive(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int s = x;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, k);
    if (lane >= k) s += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  const int w = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    const int v = __shfl_sync(0xffffffffu, w, i);
    before += i < warp ? v : 0;
    all += v;
  }
  total = all;
  return before + s - x;
}

// What the lengths say of request b, before anything is written.
struct Wish {
  int ctx, n, held, want;  // want < 0: takes no part
};

__device__ __forceinline__ Wish wish_of(const PlanArgs& p, int b) {
  Wish w;
  w.ctx = p.ctx_len[b];
  const long long n = static_cast<long long>(p.cu_new[b + 1]) - p.cu_new[b];
  w.held = min(max(p.n_pages[b], 0), p.max_pages);
  const long long want =
      (static_cast<long long>(w.ctx) + n + (1 << p.page_shift) - 1) >> p.page_shift;
  const bool ok = w.ctx >= 0 && n >= 0 && n <= p.max_new && want <= p.max_pages;
  w.n = ok ? static_cast<int>(n) : 0;
  w.want = ok ? static_cast<int>(want) : -1;
  return w;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    fa_cache_plan_kernel(const PlanArgs p) {
  extern __shared__ int plan_smem[];
  __shared__ int warp_sums[32];
  int* s_cu = plan_smem;                  // [B + 1]
  int* s_need = s_cu + p.B + 1;           // [B] pages taken by the requests before b
  int* s_give = s_need + p.B;             // [B] pages given back before b
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = blockIdx.x;
  constexpr int kWarps = kPlanThreads / 32;
  const int free0 = min(max(*p.free_count, 0), p.num_pages);

  // Thread t scans requests t * per .. t * per + per - 1.
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  int need_mine = 0, give_mine = 0;
  int need_b[kPlanPer], give_b[kPlanPer];
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    need_b[k] = give_b[k] = 0;
    const int b = tid * per + k;
    if (k < per && b < p.B) {
      const Wish w = wish_of(p, b);
      if (w.want >= 0) {
        need_b[k] = max(w.want - w.held, 0);
        give_b[k] = max(w.held - w.want, 0);
      }
      s_cu[b] = p.cu_new[b];
      need_mine += need_b[k];
      give_mine += give_b[k];
    }
  }
  if (tid == 0) s_cu[p.B] = p.cu_new[p.B];
  int need_all, give_all;
  int need_at = scan_exclusive(need_mine, warp_sums, need_all);
  int give_at = scan_exclusive(give_mine, warp_sums, give_all);
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.B) {
      s_need[b] = need_at;
      s_give[b] = give_at;
      need_at += need_b[k];
      give_at += give_b[k];
    }
  }
  __syncthreads();
  const int free1 = min(free0 + give_all, p.num_pages);

  // Pages given back, a warp per request. (give_all is the same in all CTAs.)
  if (give_all > 0) {
    for (int b = rank * kWarps + warp; b < p.B; b += kPlanCtas * kWarps) {
      const Wish w = wish_of(p, b);
      if (w.want < 0 || w.held <= w.want) continue;
      int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
      for (int i = w.want + lane; i < w.held; i += 32) {
        const int at = free0 + s_give[b] + (i - w.want);
        if (at < p.num_pages) p.free_list[at] = row[i];
        row[i] = -1;
      }
    }
  }
  cluster_barrier();  // every CTA has read the state; the pages given back are in the list

  // Pages taken and the new state, a warp per request.
  for (int b = rank * kWarps + warp; b < p.B; b += kPlanCtas * kWarps) {
    const Wish w = wish_of(p, b);
    const int need = w.want < 0 ? 0 : max(w.want - w.held, 0);
    const bool granted = w.want >= 0 && (need == 0 || static_cast<long long>(s_need[b]) + need <= free1);
    if (granted) {
      int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
      for (int i = lane; i < need; i += 32) row[w.held + i] = p.free_list[free1 - 1 - (s_need[b] + i)];
    }
    __syncwarp();
    if (lane == 0) {
      if (granted) p.n_pages[b] = w.want;
      p.seq_len[b] = granted ? w.ctx + w.n : 0;
    }
  }
  if (rank == 0 && tid == 0) {
    // The needs are a growing sequence of sums, so the granted ones are its first part.
    int used = 0;
    for (int b = p.B - 1; b >= 0; --b) {
      const int upto = b + 1 < p.B ? s_need[b + 1] : need_all;
      if (upto <= free1) {
        used = upto;
        break;
      }
    }
    *p.free_count = free1 - used;
  }
  cluster_barrier();  // tables and seq_len are written

  // Slots (and, without trees, positions), a thread per row.
  for (int t = rank * kPlanThreads + tid; t < p.rows; t += kPlanCtas * kPlanThreads) {
    int lo = 0, hi = p.B;  // the last b with cu[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int i = t - s_cu[lo];
    const int n = s_cu[lo + 1] - s_cu[lo];
    const bool inside = i >= 0 && i < n;
    const int ctx = p.ctx_len[lo];
    int slot = -1;
    if (inside && p.seq_len[lo] > 0) {
      const int at = ctx + i;
      const int page = p.block_table[static_cast<size_t>(lo) * p.max_pages + (at >> p.page_shift)];
      if (page >= 0 && page < p.num_pages)
        slot = (page << p.page_shift) + (at & ((1 << p.page_shift) - 1));
    }
    p.slot[t] = slot;
    if (p.parent == nullptr || !inside || n > p.max_new) p.position[t] = inside ? ctx + i : 0;
  }
  if (p.parent == nullptr) return;

  // Trees.
  int group = 32;
  while (group < p.max_new) group <<= 1;
  unsigned long long* s_mask = reinterpret_cast<unsigned long long*>(
      plan_smem + ((3 * p.B + 1 + 1) / 2) * 2);                     // [threads][words]
  int* s_up = reinterpret_cast<int*>(s_mask + static_cast<size_t>(kPlanThreads) * p.words);  // [threads]
  const int groups = kPlanThreads / group;
  const int g = tid / group, i = tid % group, base = g * group;
  const int rounds = 32 - __clz(max(p.max_new - 1, 1));
  for (int b0 = rank * groups; b0 < p.B; b0 += kPlanCtas * groups) {
    const int b = b0 + g;
    const int start = b < p.B ? s_cu[b] : 0;
    const int n = b < p.B ? s_cu[b + 1] - start : 0;
    const bool mine = n <= p.max_new && i < n && start + i >= 0 && start + i < p.rows;
    int up = -1;
    if (mine) {
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
      p.position[start + i] = p.ctx_len[b] + bits - 1;
    }
  }
}

// ------------------------------------------------------------------ commit
//
// A CTA per request; a thread owns one 16-byte column of K or V of one head and moves
// it along the whole path, a batch of rows at a time (all loads of a batch before its
// stores). The indices are strictly increasing, so a row's target never lies behind
// the source of a later one and no order between threads is needed. It moves a few
// rows of each request and is bound by latency: lengths, then the table, then the rows.

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
  size_t bytes = static_cast<size_t>(((3 * a.B + 1 + 1) / 2) * 2) * 4;
  if (a.parent != nullptr) bytes += static_cast<size_t>(kPlanThreads) * (8 * a.words + 4);
  if (bytes > 48 * 1024) {
    const cudaError_t e = host::ensure_dynamic_smem(reinterpret_cast<const void*>(fa_cache_plan_kernel), 96 * 1024);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  fa_cache_plan_kernel<<<kPlanCtas, kPlanThreads, bytes, stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

int launch_cache_commit(const CommitArgs& a, cudaStream_t stream) {
  fa_cache_commit_kernel<<<static_cast<unsigned>(a.B), kCommitThreads, 0, stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
