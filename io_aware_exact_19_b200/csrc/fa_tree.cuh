// Attention of a ragged batch's new rows over a paged key/value cache, on the tensor
// cores (tcgen05), split over the keys and the requests alike.
//
// The rows of one request that share a cache head (its new tokens times the group of
// query heads) are few: 1 x 4 in decoding, 16 x 4 for a drafted tree, against
// thousands of keys. So the tiles are turned around: keys are the MMA's 128 rows and
// the N = 16, 32 or 64 query rows its columns, and nothing is padded to 128:
//   S^T = K_j Q^T      A = K tile (K-major), B = Q; fp32 in TMEM, lane = key
//   P^T = exp2(S^T * scale*log2(e) - m)   thread = key, column = query row
//   O^T += V_j^T P^T   A = V tile read MN-major, B = P^T [key][row] in shared memory;
//                      fp32 in TMEM, lane = head-dimension index
// The softmax of a column runs over the lanes. Its reference m is kept in shared memory
// and moves only when some score exceeds it by more than 8 (in log2 units; P stays
// below 2^8, and O and the sums, kept in 32 bits, are consistent): one barrier with an
// OR per tile decides that, and only then the column maxima are reduced across the
// lanes. Each thread sums its own keys' P; the sums meet once, at the end.
// P is rounded to the element type once (the tensor cores take 16 bits); the sums are of
// the unrounded P. (More rows than 64: fa_tree_wide.cuh.)
//
// Work: a unit is (request, cache head, N query rows); its key tiles of 128 are laid
// end to end with those of all other units, and each CTA (one per SM, persistent) takes
// an equal run of them, whatever the lengths. A unit that is cut leaves partial
// (O, log2-sum-exp) pairs which fa_tree_merge_kernel joins (the update of the interview
// explainer, section 3.2, applied to runs of keys), in the order of the keys, so the
// result does not depend on which CTA ends first. Prompt chunks, whose units are many and
// long, are not cut: each CTA takes whole units, request by request as they stand in the batch,
// and of a request the last row tiles, which see the most keys, first (see by_unit in fa_tree.cu).
//
// Warp roles: a softmax warpgroup for every 32 columns (a thread holds its key's scores for
// them), then a TMA producer warp for K, the MMA warp, and a producer warp for V.
//
// What bounds it: reading K and V once, with few rows (64 requests of 0.8K to 8K keys, one row
// each, H_kv = 8, groups of 4, d = 128, pages of 16: 1.05 GB in 167 us, 6.3 TB/s; the SMs finish
// between 131 and 161 us, since they do not get equal shares of the bandwidth). With 64 rows and
// d = 64 a tile's 32 KB arrive in 1400 cycles and its softmax and the MMAs' issue take 1600 (a
// 64-row tree over 64K keys, 16 heads: 65 us, 4.1 TB/s). Small calls are bound by their way through
// the roles: 1000 keys, one row, 9300 cycles, 2900 of them until the first load is on its way.
#pragma once

#include "fa_cache.h"
#include "sm100.cuh"

namespace fa {
namespace tree {

using namespace fa::sm100;

constexpr int kKeys = 128;  // keys per tile
constexpr int kMaxWorkers = 148;
constexpr float kRescale = 8.0f;
constexpr uint64_t kDrainNs = 2000000000ull;  // limit of the waits on the abort path
constexpr float kNoKey = 1e30f;  // minus the reference of a column that has seen no key

// Division of x in [0, 2^31) by a number known at launch: q = (hi32(x * mul) + x) >> shift.
struct Divider {
  uint32_t by, mul, shift;
  static Divider of(int d) {
    Divider r{static_cast<uint32_t>(d), 0, 0};
    while ((1ull << r.shift) < r.by) ++r.shift;
    r.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << r.shift) - r.by)) / r.by + 1);
    return r;
  }
  __device__ __forceinline__ int operator()(int x) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(x), mul) + static_cast<uint32_t>(x)) >> shift);
  }
};

struct Params {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  long long q_row, q_head, o_row, o_head;
  int B, rows, Hq, H_kv, G, d, num_pages, max_pages, page_shift, words;
  Divider by_group;  // G
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seq_len;
  const unsigned long long* tree_mask;
  float scale_log2;
  int by_unit;      // no cuts: CTA c takes units c, c + gridDim.x, ...
  int workers;      // CTAs the key tiles are cut among
  float* part_o;    // fp32 [2 * workers][N][D]
  float* part_lse;  // fp32 [2 * workers][N], log2 units
  int4* cuts;       // [workers][2]: the unit whose first cut piece worker w holds
  int* status;
  uint64_t timeout_ns;
  int withhold;  // debug: the producers issue no load
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void group_barrier(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, r;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred r, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return any != 0;
}

// A run of key tiles of one unit.
struct Item {
  int ctx;             // rows of the request before its new ones (negative: not all are there)
  int b, q0, n, len;   // request, its first row, its rows (those there), its keys
  int h, r0;           // cache head, first query row (token * G + head in group) of the unit
  int t0, t1;          // key tiles to visit
  int clean;           // tiles before this one are seen whole by every row
  int take, tiles;     // tiles of this run and of the unit, before the causal reach
  int valid;
};

// x / y for x >= 0, y > 0: below 2^22 by a reciprocal (the quotient is then off by at most one),
// else in 32 bits where they suffice.
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 22) == 0) {
    const int a = static_cast<int>(x), b = static_cast<int>(y);
    int q = __float2int_rz(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    const int rest = a - q * b;
    q += rest >= b ? 1 : (rest < 0 ? -1 : 0);
    return q;
  }
  return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}

// `total` tiles in equal runs: worker w takes begin(w) .. begin(w + 1) - 1. Every worker up to
// the total has one tile at least.
struct Share {
  long long base, more, total;
  __device__ __forceinline__ void set(long long tiles, long long workers) {
    const long long w = max(min(workers, tiles), 1ll);
    total = tiles;
    base = divide(tiles, w);
    more = tiles - base * w;  // the first workers take one tile more
  }
  __device__ __forceinline__ long long begin(long long w) const { return min(w * base + min(w, more), total); }
  __device__ __forceinline__ int worker(long long tile) const {
    const long long long_runs = more * (base + 1);
    return static_cast<int>(tile < long_runs ? divide(tile, base + 1) : more + divide(tile - long_runs, base));
  }
};

// Walks the runs of a CTA. Units of request b: h-major over (cache head, N-row tile).
template <int N>
struct Cursor {
  long long pos, end, off;
  int b;

  // Tiles request b counts for; also its rows and keys.
  static __device__ __forceinline__ long long weight(const Params& p, int b, int& q0, int& n, int& len, int& units,
                                                     int& tiles) {
    return weight(p, p.cu_q[b], p.cu_q[b + 1], p.seq_len[b], q0, n, len, units, tiles);
  }
  static __device__ __forceinline__ long long weight(const Params& p, int cu0, int cu1, int seq, int& q0, int& n, int& len,
                                                     int& units, int& tiles) {
    q0 = min(max(cu0, 0), p.rows);
    n = max(min(cu1, p.rows) - q0, 0);
    const long long held = min(static_cast<long long>(p.max_pages) << p.page_shift, 0x7FFFFF00ll);  // keys stay ints
    len = static_cast<int>(min(static_cast<long long>(max(seq, 0)), held));
    units = static_cast<int>((static_cast<long long>(n) * p.G + N - 1) / N);
    tiles = p.by_unit ? 1 : max((len + kKeys - 1) / kKeys, 1);
    return static_cast<long long>(p.H_kv) * units * tiles;
  }

  // The item at the cursor, in request b whose rows, keys, units and tiles are given.
  __device__ __forceinline__ void take(const Params& p, Item& it, int q0, int n, int len, int units, int tiles) {
    const long long u = divide(off, tiles);
    const int t = static_cast<int>(off - u * tiles);
    // Cut: head by head, its row tiles in order. By unit: under a chain the last rows see the most
    // keys, so the last row tile of every head, then the one before, and so on.
    int h = static_cast<int>(divide(u, p.by_unit ? p.H_kv : units));
    int rt = static_cast<int>(u - static_cast<long long>(h) * (p.by_unit ? p.H_kv : units));
    if (p.by_unit) {
      const int back = h;
      h = rt;
      rt = units - 1 - back;
    }
    // All of the request's rows count for their places, also those behind p.rows.
    const int r0 = rt * N, ctx = max(p.seq_len[b], 0) - (p.cu_q[b + 1] - q0);
    const int taken = static_cast<int>(min(static_cast<long long>(tiles - t), end - pos));
    int t1 = (len + kKeys - 1) / kKeys;
    if (!p.by_unit) t1 = min(t + taken, t1);
    int whole_to = ctx;  // keys that every row sees
    if (p.tree_mask == nullptr) {
      // The chain's reach: the unit's last token sees keys up to its own. (seq_len may say
      // more than the pages hold; the tokens' places follow seq_len.)
      const int reach = ctx + min(p.by_group(r0 + N - 1), n - 1) + 1;
      t1 = min(t1, reach <= 0 ? 0 : (reach - 1) / kKeys + 1);
      whole_to += p.by_group(r0) + 1;
    }
    it.ctx = ctx;
    it.b = b;
    it.q0 = q0;
    it.n = n;
    it.len = len;
    it.h = h;
    it.r0 = r0;
    it.t0 = t;
    it.t1 = max(t1, t);
    it.clean = max(min(whole_to, len), 0) / kKeys;
    it.take = taken;
    it.tiles = tiles;
    it.valid = 1;
    pos += p.by_unit ? gridDim.x : taken;
    off += p.by_unit ? gridDim.x : taken;
  }

  __device__ __forceinline__ void next(const Params& p, Item& it) {
    it.valid = 0;
    while (pos < end && b < p.B) {
      int q0, n, len, units, tiles;
      const long long w = weight(p, b, q0, n, len, units, tiles);
      if (off >= w) {
        off -= w;
        ++b;
        continue;
      }
      take(p, it, q0, n, len, units, tiles);
      return;
    }
  }
};

// Where the softmax warps stand, kept in shared memory rather than in every thread's registers:
// their first thread walks on, an item ahead. Three slots: one warpgroup may still finish
// item k while the walker, past the barrier behind item k's tiles, writes item k + 2.
template <int N>
struct Walk {
  Cursor<N> cur;
  long long unit_at[3];  // where the item's unit begins in the run of all tiles
  Item item[3];
};

// Addresses of the barriers: q_full, drain, s_full[2], p_full[2], pv_done[2] (of tile n the one
// n % 2: a warpgroup may be a tile ahead of another), then k_full, k_empty, v_full, v_empty of
// each of S stages.
template <int S>
struct Bars {
  static constexpr int kCount = 8 + 4 * S;
  uint32_t base;
  __device__ __forceinline__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ __forceinline__ uint32_t q_full() const { return at(0); }
  __device__ __forceinline__ uint32_t drain() const { return at(1); }
  __device__ __forceinline__ uint32_t s_full(int n) const { return at(2 + (n & 1)); }
  __device__ __forceinline__ uint32_t p_full(int n) const { return at(4 + (n & 1)); }
  __device__ __forceinline__ uint32_t pv_done(int n) const { return at(6 + (n & 1)); }
  __device__ __forceinline__ uint32_t k_full(int s) const { return at(8 + s); }
  __device__ __forceinline__ uint32_t k_empty(int s) const { return at(8 + S + s); }
  __device__ __forceinline__ uint32_t v_full(int s) const { return at(8 + 2 * S + s); }
  __device__ __forceinline__ uint32_t v_empty(int s) const { return at(8 + 3 * S + s); }
};

// What follows the tiles in shared memory, at the same places for both kernels.
template <int N, int S>
struct Tail {
  Walk<N> walk;
  Cursor<N> first_cur;  // the CTA's first run and where it goes on
  Item first_item;
  uint64_t bars[Bars<S>::kCount];
  // Whether a tile has a page index outside the cache. While the softmax looks at tile n, S of
  // tile n + 1 may have let go of its K, and the flag of tile n + 1 + S be written.
  int bad_page[S + 2];
  uint32_t tmem;
  int abort_flag;
};

template <int D, int N>
struct Smem {
  static_assert(N == 16 || N == 32 || N == 64, "the wide kernel takes more");
  static constexpr int kCols = N < 32 ? N : 32;            // columns of a softmax thread
  static constexpr int kGroups = N / kCols;                // softmax warpgroups
  static constexpr int kTile = kKeys * D * 2;              // one K or V tile
  static constexpr int kChunk = kKeys * 128;               // its 64-column chunk
  static constexpr int kQ = N * D * 2;
  // P of a tile while P V still reads the last one's: two buffers, of up to 32 columns side by
  // side in one chunk; one where shared memory is better spent on a third stage of K and V.
  static constexpr int kPBufs = D == 128 && N == 64 ? 1 : 2;
  static constexpr int kPStep = N <= 32 ? 64 : kKeys * 128;  // bytes from one to the other
  static constexpr int kP = (N == 64 ? kPBufs : 1) * kKeys * 128;
  static constexpr int kStages = D == 256 ? 1 : (D == 128 ? 3 : (N == 64 ? 5 : 6));
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + (kQ + 1023) / 1024 * 1024;
  static constexpr int kKOff = kPOff + kP;
  static constexpr int kVOff = kKOff + kStages * kTile;
  static constexpr int kRefOff = kVOff + kStages * kTile;  // minus the reference of each column
  static constexpr int kRedOff = kRefOff + 4 * N;          // [group][4 warps][columns]
  static constexpr int kTailOff = kRedOff + 4 * 4 * N;
  static constexpr int kAlloc = kTailOff + static_cast<int>(sizeof(Tail<N, kStages>));
  static_assert(kAlloc <= 232448, "shared memory");
};

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sum v[c] over the 32 lanes for each of C columns: lane l ends with column l (C = 32) or
// l / 2 (C = 16) in v[0].
template <int C>
__device__ __forceinline__ void sum_columns(float (&v)[C]) {
  const int lane = lane_id();
#pragma unroll
  for (int o = 16, cnt = C / 2; o > 0; o >>= 1, cnt >>= 1) {
    if (cnt > 0) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < cnt; ++i) {
        const float send = up ? v[i] : v[i + cnt], keep = up ? v[i + cnt] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

template <int C>
__device__ __forceinline__ void load_scores(uint32_t t, float (&s)[C]) {
  if constexpr (C == 16) tmem_ld16(t, reinterpret_cast<uint32_t(&)[16]>(s));
  else tmem_ld32(t, reinterpret_cast<uint32_t(&)[32]>(s));
  tmem_ld_wait();
}

// A softmax warp's wait. Its result does not matter: after one has run out, the abort flag
// lets every later one return at once and the warp goes on through the same steps.
__device__ __forceinline__ void wait_tile(uint32_t bar, uint32_t parity, const WaitCtx& ctx) {
  mbar_wait(bar, parity, ctx);
  __syncwarp();
}

// (a, b) * (s, s) + (c, d) in one instruction.
__device__ __forceinline__ void fma2(float& a, float& b, float s, float c, float d) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %4};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(c), "f"(d));
}

__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

// Where a CTA begins: the first tile of its run, how the tiles are shared out, its TMEM.
struct Start {
  long long lo;
  Share share;
  uint32_t tmem;
};

// The start of both kernels: barriers, TMEM, and the CTA's run of tiles. `ring` is shared memory
// that nothing is loaded into yet (33 KB).
template <int N, int S, int kThreads, int kSoftWarps>
__device__ __forceinline__ Start begin(const Params& p, Tail<N, S>& tail, const Bars<S>& bar, uint8_t* ring) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The first requests' lengths, asked for before anything else is set up.
  const int mine_b = min(tid, p.B - 1);
  const int cu0 = p.cu_q[mine_b], cu1 = p.cu_q[mine_b + 1], seq = p.seq_len[mine_b];
  if (tid == 0) {
    tail.abort_flag = 0;
    tail.first_item.valid = 0;
    tail.first_cur.pos = tail.first_cur.end = 0;
    mbar_init(bar.q_full(), kSoftWarps);
    mbar_init(bar.drain(), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.s_full(i), 2);  // the commit, and the issuer (for what it has seen)
      mbar_init(bar.p_full(i), kSoftWarps);
      mbar_init(bar.pv_done(i), 1);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(bar.k_full(s), 1);
      mbar_init(bar.k_empty(s), 1);
      mbar_init(bar.v_full(s), 1);
      mbar_init(bar.v_empty(s), 1);
    }
    fence_barrier_init();
  }
  if (warp == kSoftWarps + 1) {
    tmem_alloc(smem_u32(&tail.tmem), 512);
    tmem_relinquish();
  }

  long long lo, total = 0;
  Share share;
  // The CTA's run of tiles: sums of the requests' weights (kept in the ring, which is
  // still empty); the thread that has the request in which the run begins finds the first item.
  {
    long long* before = reinterpret_cast<long long*>(ring);  // [B]
    long long* warp_sum = before + kCacheMaxB;
    constexpr int kWarps = kThreads / 32;
    long long mine = 0, w = 0;  // of this thread's last request: the weights before it, its own
    int q0 = 0, n = 0, len = 0, units = 1, tiles = 1;
    for (int base = 0; base < p.B; base += kThreads) {
      const int b = base + tid;
      if (base == 0) w = Cursor<N>::weight(p, cu0, cu1, seq, q0, n, len, units, tiles);
      else if (b < p.B) w = Cursor<N>::weight(p, b, q0, n, len, units, tiles);
      if (b >= p.B) w = 0;
      long long s = w;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += y;
      }
      if (lane == 31) warp_sum[warp] = s;
      __syncthreads();
      mine = total + s - w;
      for (int i = 0; i < kWarps; ++i) {
        const long long x = warp_sum[i];
        mine += i < warp ? x : 0;
        total += x;
      }
      if (p.B > kThreads && b < p.B) before[b] = mine;
      __syncthreads();
    }
    share.set(total, p.by_unit ? max(total, 1ll) : p.workers);
    lo = share.begin(blockIdx.x);
    const long long hi = p.by_unit ? total : share.begin(static_cast<long long>(blockIdx.x) + 1);
    if (p.B <= kThreads) {
      if (lo < hi && mine <= lo && lo < mine + w) {
        Cursor<N> c{lo, hi, lo - mine, tid};
        c.take(p, tail.first_item, q0, n, len, units, tiles);
        tail.first_cur = c;
      }
    } else {
      for (int b = tid; b < p.B && lo < hi; b += kThreads) {
        const long long from = before[b], to = b + 1 < p.B ? before[b + 1] : total;
        if (from <= lo && lo < to) {
          Cursor<N> c{lo, hi, lo - from, b};
          Cursor<N>::weight(p, b, q0, n, len, units, tiles);
          c.take(p, tail.first_item, q0, n, len, units, tiles);
          tail.first_cur = c;
        }
      }
    }
  }
  fence_proxy_async_smem();  // TMA writes where the sums were
  tc_fence_before();
  __syncthreads();  // behind every read of the sums
  tc_fence_after();
  return {lo, share, tail.tmem};
}

// The loading warps, one for K and one for V: every tile of the CTA's runs, in order.
template <int D, int N, int S>
__device__ __forceinline__ void load_tiles(const Params& p, Tail<N, S>& tail, const Bars<S>& bar, bool is_v,
                                           const CUtensorMap* map_k, const CUtensorMap* map_v, uint8_t* k_ring,
                                           uint8_t* v_ring, const WaitCtx& ctx) {
  constexpr int kTile = kKeys * D * 2;
  const int lane = threadIdx.x % 32;
  // A copy takes about 80 cycles to issue whatever its size, so with small pages (16 rows:
  // 32 copies a tile) one warp for both would be slower than the memory.
  const CUtensorMap* map = is_v ? map_v : map_k;
  const uint32_t ring = smem_u32(is_v ? v_ring : k_ring);
  const uint32_t full0 = is_v ? bar.v_full(0) : bar.k_full(0), empty0 = is_v ? bar.v_empty(0) : bar.k_empty(0);
  const int per_tile = p.page_shift >= 7 ? 1 : kKeys >> p.page_shift;  // pages of a tile
  const int box_rows = kKeys / per_tile;
  constexpr int kChunks = D / 64;
  if (lane == 0) prefetch_tmap(map);
  int issued = 0, s = 0, ph = 1;
  bool ok = true;
  Cursor<N> cur = tail.first_cur;
  Item it = tail.first_item;
  for (; ok && it.valid && !p.withhold; cur.next(p, it)) {
    const int32_t* table = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
    const int head = __shfl_sync(0xffffffffu, it.h, 0);
    // A lane's page of tile t; none (behind the length, or a bad index) is a page past the last,
    // which TMA fills with zeros.
    auto page_of = [&](int t) {
      const long long key = static_cast<long long>(t) * kKeys + lane * box_rows;
      return lane < per_tile && key < it.len ? table[key >> p.page_shift] : p.num_pages;
    };
    int ahead = it.t0 < it.t1 ? page_of(it.t0) : 0;
    for (int t = it.t0; t < it.t1; ++t) {
      int page = ahead;
      if (t + 1 < it.t1) ahead = page_of(t + 1);
      const int first_row = per_tile == 1 ? (t * kKeys) & ((1 << p.page_shift) - 1) : 0;
      bool bad = page < 0 || page >= p.num_pages;
      if (bad) page = p.num_pages;
      bad = __any_sync(0xffffffffu, bad && lane < per_tile && static_cast<long long>(t) * kKeys + lane * box_rows < it.len);
      if (!(ok = mbar_wait_warp(empty0 + 8 * s, ph, ctx))) break;
      if (lane == 0) {
        if (!is_v) tail.bad_page[issued % (S + 2)] = bad;
        mbar_arrive_expect_tx(full0 + 8 * s, kTile);
      }
      __syncwarp();
      // One elected lane issues every page's boxes: their operands are then the same in all lanes.
      for (int i = 0; i < per_tile; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_4d(ring + s * kTile + i * box_rows * 128 + c * kKeys * 128, map, full0 + 8 * s, c * 64, first_row,
                        head, pg);
        }
      }
      __syncwarp();
      ++issued;
      if (++s == S) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  if (tail.abort_flag) {
    // Aborting: what is in flight lands before the CTA exits; the last load into a stage
    // completes that stage's phase.
    for (int i = 0; i < S; ++i)
      if (issued > i) mbar_wait_bounded(full0 + 8 * i, ((issued - 1 - (issued - 1 - i) % S) / S) & 1, kDrainNs);
  }
}

// The issuing warp: S of the next tile, then P V of this one. The whole warp walks and waits; one
// elected lane issues (in issue_s and issue_o), so the operands of each MMA are the same in all
// lanes and sit in uniform registers.
template <int N, int S, typename IssueS, typename IssueO>
__device__ __forceinline__ void issue_tiles(const Params& p, Tail<N, S>& tail, const Bars<S>& bar, const WaitCtx& ctx,
                                            const IssueS& issue_s, const IssueO& issue_o) {
  int n = 0, q_count = 0;
  int s = 0, ph = 0;            // stage and phase of tile n
  bool ok = true, issued = false;
  Cursor<N> cur = tail.first_cur;
  Item it = tail.first_item;
  for (; ok && it.valid; cur.next(p, it)) {
    const int tiles = __shfl_sync(0xffffffffu, it.t1 - it.t0, 0);
    if (tiles == 0) continue;
    if (!(ok = mbar_wait_warp(bar.q_full(), q_count & 1, ctx))) break;
    ++q_count;
    if (!(ok = mbar_wait_warp(bar.k_full(s), ph, ctx))) break;
    tc_fence_after();
    issue_s(n, s);
    issued = true;
    for (int j = 0; j < tiles; ++j, ++n) {
      const int s1 = s + 1 == S ? 0 : s + 1, ph1 = s + 1 == S ? ph ^ 1 : ph;
      if (j + 1 < tiles) {
        // The other S buffer was read before P of tile n - 1 arrived.
        if (!(ok = mbar_wait_warp(bar.k_full(s1), ph1, ctx))) break;
        tc_fence_after();
        issue_s(n + 1, s1);
      }
      if (!(ok = mbar_wait_warp(bar.v_full(s), ph, ctx))) break;
      if (!(ok = mbar_wait_warp(bar.p_full(n), (n >> 1) & 1, ctx))) break;
      tc_fence_after();
      issue_o(n, s, j > 0);
      s = s1;
      ph = ph1;
    }
  }
  if (!ok && issued) {
    // Aborting: everything issued completes before TMEM and the operands go.
    if (elect_one()) {
      umma_commit(bar.drain());
      mbar_wait_bounded(bar.drain(), 0, kDrainNs);
    }
    __syncwarp();
  }
}

template <int D, bool BF16, int N>
__global__ void __launch_bounds__(128 * (N > 32 ? N / 32 : 1) + 96, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                   const __grid_constant__ Params p) {
  using L = Smem<D, N>;
  constexpr int S = L::kStages, C = L::kCols, kSoftWarps = 4 * L::kGroups;
  constexpr int kThreads = 128 * L::kGroups + 96;
  extern __shared__ __align__(1024) uint8_t smem[];  // the tiles' swizzle counts from 1024-byte boundaries
  Tail<N, S>& tail = *reinterpret_cast<Tail<N, S>*>(smem + L::kTailOff);
  float* minus_ref = reinterpret_cast<float*>(smem + L::kRefOff);
  const Bars<S> bar{smem_u32(tail.bars)};
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr uint32_t kTmemO = 256;  // O^T columns; S^T buffers at 0 and N
  for (int c = tid; c < N; c += kThreads) minus_ref[c] = kNoKey;
  const Start start = begin<N, S, kThreads, kSoftWarps>(p, tail, bar, smem + L::kKOff);
  const uint32_t tmem = start.tmem;
  const WaitCtx ctx{&tail.abort_flag, p.status, p.timeout_ns};

  if (warp == kSoftWarps || warp == kSoftWarps + 2) {
    load_tiles<D>(p, tail, bar, warp != kSoftWarps, &tmap_k, &tmap_v, smem + L::kKOff, smem + L::kVOff, ctx);
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_f16(BF16, kKeys, N, false, false);
    constexpr int kM = D == 64 ? 64 : 128;
    constexpr uint32_t idesc_o = idesc_f16(BF16, kM, N, true, true);
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
    const uint64_t dK = sdesc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
    const uint64_t dV = sdesc_sw128(smem_u32(smem + L::kVOff), L::kChunk, 1024);
    const uint64_t dP = sdesc_sw128(smem_u32(smem + L::kPOff), kKeys * 128, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto issue_s = [&](int n, int s) {
      const uint64_t a = sdesc_add(dK, static_cast<uint32_t>(s) * L::kTile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t in = (k % 4) * 32;
          umma_ss(tm + (n & 1) * N, sdesc_add(a, (k / 4) * L::kChunk + in), sdesc_add(dQ, (k / 4) * N * 128 + in),
                  idesc_s, k > 0);
        }
        umma_commit(bar.s_full(n));
        umma_commit(bar.k_empty(s));
        mbar_arrive(bar.s_full(n));
      }
      __syncwarp();
    };
    auto issue_o = [&](int n, int s, uint32_t add) {
      const uint64_t a = sdesc_add(dV, static_cast<uint32_t>(s) * L::kTile);
      const uint64_t b = sdesc_add(dP, static_cast<uint32_t>(n % L::kPBufs) * L::kPStep);
      if (elect_one()) {
#pragma unroll
        for (int half = 0; half < (D == 256 ? 2 : 1); ++half)
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            umma_ss(tm + kTmemO + half * N, sdesc_add(a, half * 2 * L::kChunk + k * 2048), sdesc_add(b, k * 2048),
                    idesc_o, k > 0 ? 1u : add);
        umma_commit(bar.pv_done(n));
        umma_commit(bar.v_empty(s));
      }
      __syncwarp();
    };
    issue_tiles(p, tail, bar, ctx, issue_s, issue_o);
  } else {
    // ------------------------------------------------------------ softmax
    // After a wait ran out every later one returns at once (the abort flag), and the
    // threads go on through the same barriers to the end; the status word tells.
    const int group = warp / 4, quarter = warp % 4, r = quarter * 32 + lane, gt = tid % 128;
    const int bar_id = 1 + group, col0 = group * C;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    // Minus the references of this group's columns (the fp16 P is taken 2^7 larger, so that
    // small ones stay in its normal range: 2^7 * 2^8 < 65504).
    constexpr float kBias = BF16 ? 0.0f : 7.0f;
    float* ref = minus_ref + col0;
    float* red = reinterpret_cast<float*>(smem + L::kRedOff) + group * 4 * C;  // [4][C]
    float* factor = red;  // [C], each written over the column by the thread that has read it
    // Row r of P: the group's half of the 64 columns, 16-byte pieces swizzled.
    const uint32_t p_row = smem_u32(smem + L::kPOff) + r * 128;
    const int piece0 = group * 4;
    int n = 0;          // tiles seen
    float l[C];

    auto load_q = [&](const Item& it) {
      // Query rows r0 .. r0 + N - 1 of the unit, swizzled as TMA would, copied without passing
      // through registers; rows past the last and columns past d are zero.
      constexpr int kVecs = N * D / 8;
      const int r0 = it.r0, rows = it.n * p.G - r0;
      const uint16_t* from = p.q + it.q0 * p.q_row + it.h * p.G * p.q_head;
      const uint32_t sq = smem_u32(smem + L::kQOff);
#pragma unroll 2
      for (int v = tid; v < kVecs; v += 128 * L::kGroups) {
        const int row = v / (D / 8), c = v % (D / 8);
        const bool there = row < rows && 8 * c < p.d;
        const int tok = p.by_group(r0 + row), g = (r0 + row) - tok * p.G;
        const uint16_t* src = there ? from + tok * p.q_row + g * p.q_head + 8 * c : p.q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + (c / 8) * (N * 128) + row * 128 +
                                                                           ((c % 8) ^ (row % 8)) * 16),
                     "l"(src), "r"(there ? 16 : 0)
                     : "memory");
      }
    };
    auto q_loaded = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.q_full());
    };

    Walk<N>& walk = tail.walk;
    auto soft_barrier = [] { asm volatile("bar.sync 8, %0;" ::"n"(128 * L::kGroups) : "memory"); };
    auto advance = [&](int to) {
      Item& it = walk.item[to];
      walk.cur.next(p, it);
      walk.unit_at[to] = walk.cur.pos - it.take - it.t0;
    };
    if (tid == 0) {
      walk.cur = tail.first_cur;
      walk.item[0] = tail.first_item;
      walk.unit_at[0] = walk.cur.pos - walk.item[0].take - walk.item[0].t0;
    }
    soft_barrier();
    if (walk.item[0].valid && walk.item[0].t1 > walk.item[0].t0) {
      load_q(walk.item[0]);
      q_loaded();
    }
    int which = 0, then = 1;
    if (gt == 0 && group == 0 && !p.by_unit) p.cuts[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    while (walk.item[which].valid) {
      const Item& it = walk.item[which];
      const int t1 = it.t1, len = it.len, clean = it.clean;
      if (tid == 0) advance(then);
      if (p.tree_mask != nullptr && t1 > clean) {
        // The last tiles' mask words, a token a lane, are near when their turn comes.
        const int tok = p.by_group(it.r0 + col0) + lane;
        if (tok < it.n) {
          const unsigned long long* m = p.tree_mask + static_cast<size_t>(it.q0 + tok) * p.words;
          asm volatile("prefetch.global.L1 [%0];" ::"l"(m));
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.0f;
      const int n_first = n;
      for (int t = it.t0; t < t1; ++t, ++n) {
        const int key = t * kKeys + r;
        // Columns that see this thread's key (bit c: column col0 + c).
        uint32_t seen = ~0u;
        if (t >= clean) {
        const bool alive = key < len;
        seen = alive ? ~0u : 0u;
        const long long own = static_cast<long long>(key) - it.ctx;  // its index among the new tokens
        const int first_row = it.r0 + col0;
        if (p.tree_mask == nullptr) {
          if (alive && own >= 0) {
            const long long c = own * p.G - first_row;  // rows of token `own` and later
            seen = c <= 0 ? ~0u : (c >= 32 ? 0u : ~0u << c);
          }
        } else if (own - lane + 31 >= 0) {
          // Lane i fetches the bits of token first + i for the warp's 32 keys; then each key
          // collects its bit of every token.
          const int first = p.by_group(first_row), last = min(p.by_group(first_row + C - 1), it.n - 1);
          const long long base = own - lane;  // of the warp's first key; the context's keys are seen
          uint32_t bits = 0;
          if (first + lane <= last) {
            const unsigned long long* m = p.tree_mask + static_cast<size_t>(it.q0 + first + lane) * p.words;
            auto word = [&](long long i) { return i >= 0 && i < p.words ? m[i] : 0ull; };
            if (base < 0) {
              bits = ~0u >> (32 + base) | static_cast<uint32_t>(word(0) << -base);
            } else {
              const long long w = base / 64;
              const int at = static_cast<int>(base % 64);
              bits = static_cast<uint32_t>(word(w) >> at);
              if (at > 32) bits |= static_cast<uint32_t>(word(w + 1) << (64 - at));
            }
          }
          uint32_t mine = 0;
          for (int tok = first; tok <= last; ++tok) {
            const uint32_t b = __shfl_sync(0xffffffffu, bits, tok - first);
            const int from = max(tok * p.G - first_row, 0), to = min((tok + 1) * p.G - first_row, 32);
            if ((b >> lane) & 1u) mine |= (~0u >> (32 - to)) & (~0u << from);  // 0 <= from < to
          }
          if (alive) seen = mine;
        }
        }
        wait_tile(bar.s_full(n), (n >> 1) & 1, ctx);
        tc_fence_after();
        bool masked = t >= clean;
        if (tail.bad_page[n % (S + 2)]) {
          // A page index outside the cache: its keys are not there.
          masked = true;
          if (key < len) {
            const int page = p.block_table[static_cast<size_t>(it.b) * p.max_pages + (key >> p.page_shift)];
            if (page < 0 || page >= p.num_pages) seen = 0u;
          }
        }
        const uint32_t t_s = tmem + lanes + (n & 1) * N + col0;
        float x[C];
        load_scores<C>(t_s, x);
        auto against_ref = [&]() {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 f = lds128(smem_u32(ref + c));
            fma2(x[c], x[c + 1], sl2, f.x, f.y);
            fma2(x[c + 2], x[c + 3], sl2, f.z, f.w);
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (!((seen >> c) & 1u)) x[c] = -INFINITY;
          }
        };
        const bool first = n == n_first;
        if (first) {
          // The run's first reference of each column: the largest of four of its scores. Any score
          // within 2^8 of the largest will do, and the vote below catches the rest.
          if (lane == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) red[quarter * C + c] = ((seen >> c) & 1u) ? x[c] * sl2 : -INFINITY;
          }
          group_barrier(bar_id);
          if (gt < C) {
            const float high = fmaxf(fmaxf(red[gt], red[C + gt]), fmaxf(red[2 * C + gt], red[3 * C + gt])) - kBias;
            if (high > -kNoKey) ref[gt] = -high;
          }
          group_barrier(bar_id);
        }
        against_ref();
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < C; c += 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], x[c + i]);
        }
        if (group_any(bar_id, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kRescale + kBias)) {
          // Some column's reference moves. P V of the tile before, which adds to O, must be complete.
          if (!first) {
            wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
            tc_fence_after();
          }
          load_scores<C>(t_s, x);
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = ((seen >> c) & 1u) ? x[c] * sl2 : -INFINITY;
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = warp_max(x[c]);
          if (lane == 0) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
              *reinterpret_cast<float4*>(red + quarter * C + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
          }
          group_barrier(bar_id);
          if (gt < C) {
            const float high = fmaxf(fmaxf(red[gt], red[C + gt]), fmaxf(red[2 * C + gt], red[3 * C + gt])) - kBias;
            const float old = -ref[gt];
            const float now = high > old + kRescale ? high : old;
            factor[gt] = ex2(old - now);
            ref[gt] = -now;
          }
          group_barrier(bar_id);
          if (!first) {
#pragma unroll 1
            for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {
              const uint32_t t_o = tmem + lanes + kTmemO + h * N + col0;
#pragma unroll 1
              for (int c = 0; c < C; c += 16) {
                uint32_t o[16];
                tmem_ld16(t_o + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor[c + i]);
                tmem_st16(t_o + c, o);
              }
            }
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < C; ++c) l[c] *= factor[c];
          }
          load_scores<C>(t_s, x);
          against_ref();
        }
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          x[c] = ex2(x[c]);
          x[c + 1] = ex2(x[c + 1]);
          add2(l[c], l[c + 1], x[c], x[c + 1]);
        }
        // P V that read this buffer of P last is complete: with two buffers that of tile n - 2, which
        // was issued before S of this tile, whose commit covers it.
        if (L::kPBufs == 1 && !first) wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
        const int buf = n % L::kPBufs;
        const uint32_t p_at = p_row + (N <= 32 ? 0 : buf * L::kPStep);
        const int piece = piece0 + (N <= 32 ? 4 * buf : 0);
#pragma unroll
        for (int c = 0; c < C; c += 8)
          sts128(p_at + (((piece + c / 8) ^ (r % 8)) * 16), pack2<BF16>(x[c], x[c + 1]),
                 pack2<BF16>(x[c + 2], x[c + 3]), pack2<BF16>(x[c + 4], x[c + 5]), pack2<BF16>(x[c + 6], x[c + 7]));
        if (t >= clean && t * kKeys + (kKeys - 1) >= len) {
          // The last tile: what the page holds behind the last key may be anything, and 0 * NaN is
          // not 0, so those rows of V are cleared. (The stage's phase before this tile's must be over,
          // or the wait would take it for this one: S of this tile says so of tile n - 2, and with a
          // single stage it is tile n - 1 whose P V must have ended.)
          if (S == 1 && !first) wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
          wait_tile(bar.v_full(n % S), (n / S) & 1, ctx);
          if (key >= len && group == 0) {
            const uint32_t row = smem_u32(smem + L::kVOff + (n % S) * L::kTile) + r * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) sts128(row + c * L::kChunk + i * 16, 0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.p_full(n));
      }
      // Every S of this unit is read, so Q may be replaced.
      soft_barrier();  // every warp is done with them, and the item that follows is known
      const bool more = walk.item[then].valid && walk.item[then].t1 > walk.item[then].t0;
      if (more) load_q(walk.item[then]);  // arrives while the sums are joined

      // ---------------------------------------------------------- the run's result
      const bool some = n > n_first;
      sum_columns<C>(l);
      red[quarter * C + (C == 32 ? lane : lane / 2)] = l[0];
      group_barrier(bar_id);
      const bool whole = it.take == it.tiles;
      const long long unit_at = walk.unit_at[which];
      const int slot = 2 * static_cast<int>(blockIdx.x) + (unit_at > start.lo ? 1 : 0);
      const int left = it.n * p.G - it.r0 - col0;  // columns of this group that are rows
      if (gt < C) {
        const float sum = (red[gt] + red[C + gt]) + (red[2 * C + gt] + red[3 * C + gt]);
        const float lse2 = sum > 0.0f ? lg2(sum) - ref[gt] : (sum == 0.0f ? -INFINITY : sum);
        factor[gt] = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
        ref[gt] = kNoKey;
        if (whole) {
          if (gt < left) {
            const int rr = it.r0 + col0 + gt, tok = p.by_group(rr);
            p.lse[static_cast<size_t>(it.q0 + tok) * p.Hq + it.h * p.G + rr - tok * p.G] = lse2 * 0.6931471805599453f;
          }
        } else {
          p.part_lse[static_cast<size_t>(slot) * N + col0 + gt] = lse2;
        }
      }
      if (more) q_loaded();
      group_barrier(bar_id);
      if (some) {
        wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
        tc_fence_after();
      }
      constexpr int kOutBytes = D == 64 ? 128 : 256, kOutRows = kOutBytes / 64;
      // Byte `at` of column c's output: in the group's own pieces of P, since the other group may be
      // writing P of the next item's first tile already.
      auto staged = [&](int c, int at) {
        const int row = c * kOutRows + at / 64;
        return smem + L::kPOff + row * 128 + ((piece0 + at % 64 / 16) ^ (row % 8)) * 16 + at % 16;
      };
#pragma unroll 1
      for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
        const uint32_t t_o = tmem + lanes + kTmemO + half * N + col0;
        // M = 64 keeps row i in lane 32 * (i / 16) + i % 16.
        const int e = D == 64 ? quarter * 16 + lane : half * 128 + r;
        const bool mine = (D != 64 || lane < 16) && e < p.d;
        float* part = p.part_o + (static_cast<size_t>(slot) * N + col0) * D + e;
#pragma unroll 1
        for (int c = 0; c < C; c += 16, part += 16 * D) {
          uint32_t o[16];
          if (some) {
            tmem_ld16(t_o + c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = factor[c + i];
            o[i] = some && f != 0.0f ? __float_as_uint(__uint_as_float(o[i]) * f) : 0u;
          }
          if (!mine) continue;
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < left) part[i * D] = __uint_as_float(o[i]);
          } else {
            // Turned around through the group's part of P, free by now: its four pieces of each of
            // the 128 rows, kOutRows rows for a column's kOutBytes.
            const int at = e % (kOutBytes / 2) * 2;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint16_t*>(staged(c + i, at)) =
                  static_cast<uint16_t>(pack2<BF16>(__uint_as_float(o[i]), 0.0f));
          }
        }
        if (whole) {
          group_barrier(bar_id);
          constexpr int kVecs = kOutBytes / 16;
#pragma unroll 2
          for (int v = gt; v < C * kVecs; v += 128) {
            const int c = v / kVecs, at = v % kVecs * 16, rr = it.r0 + col0 + c;
            const uint4 y = *reinterpret_cast<const uint4*>(staged(c, at));
            const int d0 = half * 128 + at / 2;
            if (c < left && d0 < p.d) {
              const int tok = p.by_group(rr), g = rr - tok * p.G;
              *reinterpret_cast<uint4*>(p.o + (it.q0 + tok) * p.o_row + (it.h * p.G + g) * p.o_head + d0) = y;
            }
          }
          if (D == 256) group_barrier(bar_id);  // the second half takes the same place
        }
      }
      tc_fence_before();
      // The unit that goes on in the next CTAs (at most the last one): what the merge needs to know.
      if (!whole && it.t0 == 0 && gt == 0 && group == 0) {
        p.cuts[2 * blockIdx.x] = make_int4(1, slot, start.share.worker(unit_at + it.tiles - 1), it.q0);
        p.cuts[2 * blockIdx.x + 1] = make_int4(it.h, it.r0, it.n, 0);
      }
      group_barrier(bar_id);  // the scratch is read
      which = then;
      then = then == 2 ? 0 : then + 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of a cut unit: lse = log sum_s exp(lse_s), O = sum_s exp(lse_s - lse) O_s.
// Block (w, y): rows 8y .. 8y + 7 of the unit whose first piece worker w holds, a warp a row.
template <int D, bool BF16, int N>
__global__ void __launch_bounds__(256) fa_tree_merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x, lane = threadIdx.x % 32, c = blockIdx.y * 8 + threadIdx.x / 32;
  const int4 a = p.cuts[2 * w], u = p.cuts[2 * w + 1];  // u: cache head, first row, rows of the request
  if (a.x == 0 || c >= N) return;
  const int rr = u.y + c;
  if (rr >= u.z * p.G) return;
  const int pieces = a.z - w + 1;
  auto row_of = [&](int i) { return static_cast<size_t>(i == 0 ? a.y : 2 * (w + i)) * N + c; };
  // A lane holds the lse of one piece, of 32 at a time, and kPer consecutive elements of O, of kAhead
  // pieces at a time; the first are asked for together with the lse's, before their weights are known.
  // (Many rows come in few pieces: 16 trees of 48 x 7 rows took 60 us with eight ahead, 57 with four; four
  // rows to a warp, in a quarter of the blocks, 57 there and 38 for 33 in a tree over 30000 keys.)
  constexpr int kPer = D / 32, kAhead = N >= 64 ? 4 : 8;
  float o[kAhead][kPer];
  auto load_o = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i < pieces) {
        const float* src = p.part_o + row_of(i0 + i) * D + lane * kPer;
        if constexpr (kPer == 2) {
          const float2 y = *reinterpret_cast<const float2*>(src);
          o[i][0] = y.x, o[i][1] = y.y;
        } else {
#pragma unroll
          for (int k = 0; k < kPer; k += 4) {
            const float4 y = *reinterpret_cast<const float4*>(src + k);
            o[i][k] = y.x, o[i][k + 1] = y.y, o[i][k + 2] = y.z, o[i][k + 3] = y.w;
          }
        }
      }
    }
  };
  float x = lane < pieces ? p.part_lse[row_of(lane)] : -INFINITY;
  load_o(0);
  float m = x;
  bool nan = x != x;
  for (int i = lane + 32; i < pieces; i += 32) {
    const float y = p.part_lse[row_of(i)];
    nan |= y != y;
    m = fmaxf(m, y);
  }
  m = warp_max(m);
  nan = __any_sync(0xffffffffu, nan);
  float z = 0.0f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
  for (int i0 = 0; i0 < pieces; i0 += kAhead) {
    if (i0 > 0) {
      load_o(i0);
      if (i0 % 32 == 0) x = i0 + lane < pieces ? p.part_lse[row_of(i0 + lane)] : -INFINITY;
    }
    const float weight = x == -INFINITY ? 0.0f : ex2(x - m);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float f = __shfl_sync(0xffffffffu, weight, (i0 + i) % 32);
      if (i0 + i < pieces) {
        z += f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = fmaf(f, o[i][k], acc[k]);
      }
    }
  }
  const float inv = z > 0.0f ? 1.0f / z : z;
  const int tok = p.by_group(rr), head = u.x * p.G + rr - tok * p.G;
  uint16_t* dst = p.o + (a.w + tok) * p.o_row + head * p.o_head + lane * kPer;
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    if (lane * kPer + k < p.d) *reinterpret_cast<uint32_t*>(dst + k) = pack2<BF16>(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0)
    p.lse[static_cast<size_t>(a.w + tok) * p.Hq + head] = z > 0.0f ? (m + lg2(z)) * 0.6931471805599453f
                                                                    : (nan ? z : -INFINITY);
}

}  // namespace tree
}  // namespace fa
