// Attention of a ragged batch's new rows over a paged key/value cache, on the tensor
// cores (tcgen05), split over the keys and the requests alike.
//
// The rows of one request that share a cache head (its new tokens times the group of
// query heads) are few: 1 x 4 in decoding, 48 x 7 for a drafted tree, against
// thousands of keys. So the tiles are turned around: keys are the MMA's 128 rows and
// the N = 16, 32, 64 or 128 query rows its columns, and nothing is padded to 128:
//   S^T = K_j Q^T      A = K tile (K-major), B = Q; fp32 in TMEM, lane = key
//   P^T = exp2(S^T * scale*log2(e) - m)   thread = key, column = query row
//   O^T += V_j^T P^T   A = V tile read MN-major, B = P^T [key][row] in shared memory;
//                      fp32 in TMEM, lane = head-dimension index
// The softmax of a column runs over the lanes. Its reference m is kept in shared memory
// and moves only when some score exceeds it by more than 8 (in log2 units; P stays
// below 2^8, and O and the sums, kept in 32 bits, are consistent): one barrier with an
// OR per tile decides that, and only then the column maxima are reduced across the
// lanes. Each thread sums its own keys' P; the sums meet once, at the end.
//
// Work: a unit is (request, cache head, N query rows); its key tiles of 128 are laid
// end to end with those of all other units, and each CTA (one per SM, persistent) takes
// an equal run of them, whatever the lengths. A unit that is cut leaves partial
// (O, log2-sum-exp) pairs which fa_tree_merge_kernel joins (the update of the interview
// explainer, section 3.2, applied to runs of keys). Prompt chunks, whose units are many
// and long, are not cut: a CTA per unit, the longest first.
//
// Warp roles: 4 (N <= 64) or 8 softmax warps (warpgroup w owns columns 64w .. 64w+63),
// then a TMA producer warp, whose lanes each fetch pages of the tile, and an MMA warp.
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

struct Params {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  long long q_row, q_head, o_row, o_head;
  int B, rows, Hq, H_kv, G, d, num_pages, max_pages, page_shift, words;
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seq_len;
  const unsigned long long* tree_mask;
  float scale_log2;
  int by_unit;      // a CTA per unit (no cuts)
  int workers;      // CTAs the key tiles are cut among
  float* part_o;    // fp32 [2 * workers][N][D]
  float* part_lse;  // fp32 [2 * workers][N], log2 units
  int4* cuts;       // [workers][2]: the unit whose first cut piece worker w holds
  int* status;
  uint64_t timeout_ns;
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

template <int D, int N>
struct Smem {
  static constexpr int kGroups = N == 128 ? 2 : 1;        // softmax warpgroups
  static constexpr int kCols = N / kGroups;                // columns of a thread
  static constexpr int kTile = kKeys * D * 2;              // one K or V tile
  static constexpr int kChunk = kKeys * 128;               // its 64-column chunk
  static constexpr int kQ = N * D * 2;
  static constexpr int kP = kGroups * kKeys * 128;         // [group][key][64 columns]
  static constexpr int kStages = D == 256 ? 1 : (D == 128 ? (N == 128 ? 2 : 3) : (N == 128 ? 5 : 6));
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + (kQ + 1023) / 1024 * 1024;
  static constexpr int kKOff = kPOff + kP;
  static constexpr int kVOff = kKOff + kStages * kTile;
  static constexpr int kRefOff = kVOff + kStages * kTile;  // minus the reference of each column
  static constexpr int kBarOff = kRefOff + 4 * N;
  // q_full, p_full, pv_done, drain, s_full[2], then k_full, k_empty, v_full, v_empty of each stage
  static constexpr int kNumBars = 6 + 4 * kStages;
  static constexpr int kMiscOff = kBarOff + 8 * kNumBars;  // TMEM base, abort flag, first request, its offset
  static constexpr int kBytes = kMiscOff + 32;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
  static_assert(4 * 4 * kCols + 8 * kCols <= kKeys * 128, "the reductions' scratch lies in P");
};

// A run of key tiles of one unit.
struct Item {
  int b, q0, n, len;   // request, its first row, its rows, its keys
  int h, r0;           // cache head, first query row (token * G + head in group) of the unit
  int t0, t1;          // key tiles to visit
  int whole;           // the unit is not cut
  int take, tiles;     // tiles of this run and of the unit, before the causal reach
};

// Walks the runs of a CTA. Units of request b: h-major over (cache head, N-row tile).
template <int N>
struct Cursor {
  long long pos, end, off;
  int b;

  // Tiles request b counts for; also its rows and keys.
  static __device__ __forceinline__ long long weight(const Params& p, int b, int& q0, int& n, int& len, int& units,
                                                     int& tiles) {
    q0 = min(max(p.cu_q[b], 0), p.rows);
    n = max(min(p.cu_q[b + 1], p.rows) - q0, 0);
    len = static_cast<int>(
        min(static_cast<long long>(max(p.seq_len[b], 0)), static_cast<long long>(p.max_pages) << p.page_shift));
    units = static_cast<int>((static_cast<long long>(n) * p.G + N - 1) / N);
    tiles = p.by_unit ? 1 : max((len + kKeys - 1) / kKeys, 1);
    return static_cast<long long>(p.H_kv) * units * tiles;
  }

  __device__ __forceinline__ bool next(const Params& p, Item& it) {
    while (pos < end && b < p.B) {
      int units, tiles;
      const long long w = weight(p, b, it.q0, it.n, it.len, units, tiles);
      if (off >= w) {
        off -= w;
        ++b;
        continue;
      }
      const unsigned long long u = static_cast<unsigned long long>(off) / static_cast<unsigned>(tiles);
      const int t = static_cast<int>(off - static_cast<long long>(u) * tiles);
      it.b = b;
      it.h = static_cast<int>(u / static_cast<unsigned>(units));
      int rt = static_cast<int>(u - static_cast<unsigned long long>(it.h) * units);
      if (p.by_unit) rt = units - 1 - rt;  // under a chain the last rows see the most keys
      it.r0 = rt * N;
      it.take = static_cast<int>(min(static_cast<long long>(tiles - t), end - pos));
      it.tiles = tiles;
      it.whole = it.take == tiles;
      it.t0 = t;
      it.t1 = p.by_unit ? (it.len + kKeys - 1) / kKeys : min(t + it.take, (it.len + kKeys - 1) / kKeys);
      if (p.tree_mask == nullptr) {
        // The chain's reach: the unit's last token sees keys up to its own. (seq_len may say
        // more than the pages hold; the tokens' places follow seq_len.)
        const int last = min((it.r0 + N - 1) / p.G, it.n - 1);
        const long long reach = static_cast<long long>(p.seq_len[b]) - it.n + last + 1;
        const int lim = reach <= 0 ? 0 : static_cast<int>((reach + kKeys - 1) / kKeys);
        it.t1 = min(it.t1, lim);
      }
      it.t1 = max(it.t1, it.t0);
      pos += it.take;
      off += it.take;
      return true;
    }
    return false;
  }
};

// Reduce v[c] over the 32 lanes for each of C columns: lane l ends with columns
// C/32 * l .. (C = 64: two, v[0] and v[1]; C = 32: one; C = 16: column l / 2).
template <int C, bool kMax>
__device__ __forceinline__ void reduce_columns(float (&v)[C]) {
  const int lane = lane_id();
  int cnt = C;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (cnt > 1) {
      cnt >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        if (i < cnt) {
          const float send = up ? v[i] : v[i + cnt], keep = up ? v[i + cnt] : v[i];
          const float got = __shfl_xor_sync(0xffffffffu, send, o);
          v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
      }
    } else {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
  }
}

template <int C>
__device__ __forceinline__ void store_columns(float* dst, const float (&v)[C]) {
  const int lane = lane_id();
  if constexpr (C == 64) {
    dst[2 * lane] = v[0];
    dst[2 * lane + 1] = v[1];
  } else if constexpr (C == 32) {
    dst[lane] = v[0];
  } else {
    if (lane % 2 == 0) dst[lane / 2] = v[0];
  }
}

template <int C>
__device__ __forceinline__ void load_scores(uint32_t t, float (&s)[C]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(s);
  if constexpr (C == 16) {
    tmem_ld16(t, *reinterpret_cast<uint32_t(*)[16]>(r));
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 32) tmem_ld32(t + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
  }
  tmem_ld_wait();
}

template <int D, bool BF16, int N>
__global__ void __launch_bounds__(128 * (N == 128 ? 2 : 1) + 64, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                   const Params p) {
  using L = Smem<D, N>;
  constexpr int S = L::kStages, C = L::kCols, kSoftWarps = 4 * L::kGroups;
  constexpr int kThreads = 128 * L::kGroups + 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int* first_b = reinterpret_cast<int*>(smem + L::kMiscOff + 8);
  long long* first_off = reinterpret_cast<long long*>(smem + L::kMiscOff + 16);
  float* minus_ref = reinterpret_cast<float*>(smem + L::kRefOff);
  const uint32_t q_full = smem_u32(&bars[0]), p_full = smem_u32(&bars[1]), pv_done = smem_u32(&bars[2]),
                 drain = smem_u32(&bars[3]);
  auto s_full = [&](int i) { return smem_u32(&bars[4 + i]); };
  auto k_full = [&](int s) { return smem_u32(&bars[6 + s]); };
  auto k_empty = [&](int s) { return smem_u32(&bars[6 + S + s]); };
  auto v_full = [&](int s) { return smem_u32(&bars[6 + 2 * S + s]); };
  auto v_empty = [&](int s) { return smem_u32(&bars[6 + 3 * S + s]); };
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr uint32_t kTmemO = 256;  // O^T columns; S^T buffers at 0 and N

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    *abort_flag = 0;
    *first_b = p.B;
    mbar_init(q_full, 128 * L::kGroups);
    mbar_init(p_full, 128 * L::kGroups);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) mbar_init(s_full(i), 1);
    for (int s = 0; s < S; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    fence_barrier_init();
  }
  for (int c = tid; c < N; c += kThreads) minus_ref[c] = kNoKey;
  if (warp == kSoftWarps + 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  // The CTA's run of tiles: sums of the requests' weights (kept in the ring, which is
  // still empty), then the request in which the run begins.
  long long lo, hi, workers, total = 0;
  {
    long long* before = reinterpret_cast<long long*>(smem + L::kKOff);  // [B]
    long long* warp_sum = before + kCacheMaxB;
    constexpr int kWarps = kThreads / 32;
    for (int base = 0; base < p.B; base += kThreads) {
      const int b = base + tid;
      long long w = 0;
      int q0, n, len, units, tiles;
      if (b < p.B) w = Cursor<N>::weight(p, b, q0, n, len, units, tiles);
      long long s = w;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += y;
      }
      if (lane == 31) warp_sum[warp] = s;
      __syncthreads();
      long long ahead = total;
      for (int i = 0; i < kWarps; ++i) {
        const long long x = warp_sum[i];
        ahead += i < warp ? x : 0;
        total += x;
      }
      if (b < p.B) before[b] = ahead + s - w;
      __syncthreads();
    }
    const long long me = blockIdx.x;
    workers = min(static_cast<long long>(p.workers), max(total, 1ll));  // each has a tile at least
    lo = p.by_unit ? me : min(me * total / workers, total);
    hi = p.by_unit ? min(me + 1, total) : min((me + 1) * total / workers, total);
    for (int b = tid; b < p.B; b += kThreads) {
      const long long from = before[b], to = b + 1 < p.B ? before[b + 1] : total;
      if (from <= lo && lo < to) {
        *first_b = b;
        *first_off = lo - from;
      }
    }
  }
  fence_proxy_async_smem();  // TMA writes where the sums were
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx ctx{abort_flag, p.status, p.timeout_ns};
  Cursor<N> cur;
  cur.pos = lo;
  cur.end = hi;
  cur.b = *first_b;
  cur.off = cur.b < p.B ? *first_off : 0;
  // (The prefix sums in the ring are not read any more: the barrier above is behind every read.)

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ TMA producer
    const int per_tile = p.page_shift >= 7 ? 1 : kKeys >> p.page_shift;  // pages of a tile
    const int box_rows = kKeys / per_tile;
    constexpr int kChunks = D / 64;
    if (lane == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
    int n = 0, k_issued = 0, v_issued = 0;
    bool ok = true;
    Item it;
    while (ok && cur.next(p, it)) {
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
      for (int t = it.t0; ok && t < it.t1; ++t, ++n) {
        const int s = n % S;
        const uint32_t ph = ((n / S) & 1) ^ 1;
        // A lane's page; none (behind the length, or a bad index) is a page past the last, which TMA
        // fills with zeros.
        int page = p.num_pages, row = 0;
        if (lane < per_tile) {
          const long long key = static_cast<long long>(t) * kKeys + lane * box_rows;
          if (key < it.len) {
            page = table[key >> p.page_shift];
            row = static_cast<int>(key & ((1 << p.page_shift) - 1));
            if (page < 0 || page >= p.num_pages) page = p.num_pages;
          }
        }
        auto fetch = [&](const CUtensorMap* map, uint32_t full, int ring) {
          if (lane == 0) mbar_arrive_expect_tx(full, L::kTile);
          __syncwarp();
          if (lane < per_tile) {
            const uint32_t dst = smem_u32(smem + ring + s * L::kTile) + lane * box_rows * 128;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(dst + c * L::kChunk, map, full, c * 64, row, it.h, page);
          }
          __syncwarp();
        };
        if (!(ok = mbar_wait_warp(k_empty(s), ph, ctx))) break;
        fetch(&tmap_k, k_full(s), L::kKOff);
        ++k_issued;
        if (!(ok = mbar_wait_warp(v_empty(s), ph, ctx))) break;
        fetch(&tmap_v, v_full(s), L::kVOff);
        ++v_issued;
      }
    }
    if (*abort_flag) {
      // Aborting: what is in flight lands before the CTA exits; the last load into a stage
      // completes that stage's phase.
      for (int s = 0; s < S; ++s) {
        if (k_issued > s)
          mbar_wait_bounded(k_full(s), ((k_issued - 1 - (k_issued - 1 - s) % S) / S) & 1, kDrainNs);
        if (v_issued > s)
          mbar_wait_bounded(v_full(s), ((v_issued - 1 - (v_issued - 1 - s) % S) / S) & 1, kDrainNs);
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16(BF16, kKeys, N, false, false);
      constexpr int kM = D == 64 ? 64 : 128;
      constexpr uint32_t idesc_o = idesc_f16(BF16, kM, N, true, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(smem + L::kVOff), L::kChunk, 1024);
      const uint64_t dP = sdesc_sw128(smem_u32(smem + L::kPOff), kKeys * 128, 1024);
      auto issue_s = [&](int n) {
        const int s = n % S;
        const uint64_t a = sdesc_add(dK, static_cast<uint32_t>(s) * L::kTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t in = (k % 4) * 32;
          umma_ss(tmem + (n & 1) * N, sdesc_add(a, (k / 4) * L::kChunk + in), sdesc_add(dQ, (k / 4) * N * 128 + in),
                  idesc_s, k > 0);
        }
        umma_commit(s_full(n & 1));
        umma_commit(k_empty(s));
      };
      auto issue_o = [&](int n, bool first) {
        const uint64_t a = sdesc_add(dV, static_cast<uint32_t>(n % S) * L::kTile);
#pragma unroll
        for (int half = 0; half < (D == 256 ? 2 : 1); ++half)
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            umma_ss(tmem + kTmemO + half * N, sdesc_add(a, half * 2 * L::kChunk + k * 2048), sdesc_add(dP, k * 2048),
                    idesc_o, !first || k > 0);
        umma_commit(pv_done);
        umma_commit(v_empty(n % S));
      };
      int n = 0, q_count = 0;
      bool ok = true, issued = false;
      Item it;
      while (ok && cur.next(p, it)) {
        const int tiles = it.t1 - it.t0;
        if (tiles == 0) continue;
        if (!(ok = mbar_wait(q_full, q_count & 1, ctx))) break;
        ++q_count;
        if (!(ok = mbar_wait(k_full(n % S), (n / S) & 1, ctx))) break;
        tc_fence_after();
        issue_s(n);
        issued = true;
        for (int j = 0; j < tiles; ++j, ++n) {
          if (j + 1 < tiles) {
            // The other S buffer was read before P of tile n - 1 arrived.
            if (!(ok = mbar_wait(k_full((n + 1) % S), ((n + 1) / S) & 1, ctx))) break;
            tc_fence_after();
            issue_s(n + 1);
          }
          if (!(ok = mbar_wait(v_full(n % S), (n / S) & 1, ctx))) break;
          if (!(ok = mbar_wait(p_full, n & 1, ctx))) break;
          tc_fence_after();
          issue_o(n, j == 0);
        }
      }
      if (!ok && issued) {
        // Aborting: everything issued completes before TMEM and the operands go.
        umma_commit(drain);
        mbar_wait_bounded(drain, 0, kDrainNs);
      }
    }
    __syncwarp();
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
    uint8_t* sP = smem + L::kPOff + group * (kKeys * 128);
    float* red = reinterpret_cast<float*>(sP);       // [4][C], then
    float* factor = red + 4 * C;                      // [C]
    const uint32_t p_row = smem_u32(sP) + r * 128;
    int n = 0;          // tiles seen
    float l[C];

    auto load_q = [&](const Item& it) {
      // Query rows r0 .. r0 + N - 1 of the unit, swizzled as TMA would; rows past the last and
      // columns past d are zero.
      constexpr int kVecs = N * D / 8;
      const int rows = it.n * p.G - it.r0;
      for (int v = tid; v < kVecs; v += 128 * L::kGroups) {
        const int row = v / (D / 8), c = v % (D / 8);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < rows && 8 * c < p.d) {
          const int tok = (it.r0 + row) / p.G, g = (it.r0 + row) - tok * p.G;
          x = *reinterpret_cast<const uint4*>(p.q + (it.q0 + tok) * p.q_row + (it.h * p.G + g) * p.q_head + 8 * c);
        }
        sts128(smem_u32(smem + L::kQOff) + (c / 8) * (N * 128) + row * 128 + ((c % 8) ^ (row % 8)) * 16, x.x, x.y, x.z,
               x.w);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    };

    Item it, following;
    bool have = cur.next(p, it);
    if (have && it.t1 > it.t0) load_q(it);
    int4 cut0 = make_int4(0, 0, 0, 0), cut1 = cut0;
    while (have) {
      const long long unit_at = cur.pos - it.take - it.t0;  // where the unit begins in the run of all tiles
      const bool more = cur.next(p, following);
      const long long ctx_len = static_cast<long long>(p.seq_len[it.b]) - it.n;
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.0f;
      const int n_first = n;
      auto page_of = [&](int t) {
        const long long key = static_cast<long long>(t) * kKeys + r;
        return key < it.len ? table[key >> p.page_shift] : -1;
      };
      int page = it.t1 > it.t0 ? page_of(it.t0) : 0;
      for (int t = it.t0; t < it.t1; ++t, ++n) {
        const long long key = static_cast<long long>(t) * kKeys + r;
        const bool alive = page >= 0 && page < p.num_pages;  // key < len included
        if (t + 1 < it.t1) page = page_of(t + 1);
        // Columns that see this thread's key (bit c: column col0 + c).
        unsigned long long seen = alive ? ~0ull : 0ull;
        const long long own = key - ctx_len;  // its index among the new tokens
        const int first_row = it.r0 + col0;
        if (alive && own >= 0) {
          if (p.tree_mask == nullptr) {
            const long long c = own * p.G - first_row;  // rows of token `own` and later
            seen = c <= 0 ? ~0ull : (c >= 64 ? 0ull : ~0ull << c);
          } else {
            seen = 0ull;
            const int last = min((first_row + C - 1) / p.G, it.n - 1);
            if (own < 64ll * p.words) {
              const unsigned long long* m = p.tree_mask + static_cast<size_t>(it.q0) * p.words + own / 64;
#pragma unroll 4
              for (int tok = first_row / p.G; tok <= last; ++tok) {
                const unsigned long long bit = (m[static_cast<size_t>(tok) * p.words] >> (own % 64)) & 1ull;
                const int from = max(tok * p.G - first_row, 0), to = min((tok + 1) * p.G - first_row, 64);
                if (bit) seen |= (~0ull >> (64 - to)) & (~0ull << from);  // its group's columns; 0 <= from < to
              }
            }
          }
        }
        const bool masked = __any_sync(0xffffffffu, seen != ~0ull);

        mbar_wait_warp(s_full(n & 1), (n >> 1) & 1, ctx);
        tc_fence_after();
        const uint32_t t_s = tmem + lanes + (n & 1) * N + col0;
        float x[C];
        load_scores<C>(t_s, x);
        auto against_ref = [&]() {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 f = lds128(smem_u32(ref + c));
            x[c] = fmaf(x[c], sl2, f.x);
            x[c + 1] = fmaf(x[c + 1], sl2, f.y);
            x[c + 2] = fmaf(x[c + 2], sl2, f.z);
            x[c + 3] = fmaf(x[c + 3], sl2, f.w);
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (!((seen >> c) & 1ull)) x[c] = -INFINITY;
          }
        };
        against_ref();
        float top = x[0];
#pragma unroll
        for (int c = 1; c < C; ++c) top = fmaxf(top, x[c]);
        if (group_any(bar_id, top > kRescale + kBias)) {
          // Some column's reference moves. P V of the tile before must be complete: it adds to O,
          // and the scratch lies where it reads P.
          if (n > n_first) {
            mbar_wait_warp(pv_done, (n - 1) & 1, ctx);
            tc_fence_after();
          }
          load_scores<C>(t_s, x);
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = ((seen >> c) & 1ull) ? x[c] * sl2 : -INFINITY;
          reduce_columns<C, true>(x);
          store_columns<C>(red + quarter * C, x);
          group_barrier(bar_id);
          if (gt < C) {
            const float high = fmaxf(fmaxf(red[gt], red[C + gt]), fmaxf(red[2 * C + gt], red[3 * C + gt])) - kBias;
            const float old = -ref[gt];
            const float now = high > old + kRescale ? high : old;
            factor[gt] = ex2(old - now);
            ref[gt] = -now;
          }
          group_barrier(bar_id);
          if (n > n_first) {
#pragma unroll
            for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
              const uint32_t t_o = tmem + lanes + kTmemO + half * N + col0;
#pragma unroll
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
          }
#pragma unroll
          for (int c = 0; c < C; ++c) l[c] *= factor[c];
          load_scores<C>(t_s, x);
          against_ref();
          group_barrier(bar_id);  // the scratch is read; P may be written
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          x[c] = ex2(x[c]);
          l[c] += x[c];
        }
        // P V of the tile before has read its P.
        if (n > n_first) mbar_wait_warp(pv_done, (n - 1) & 1, ctx);
#pragma unroll
        for (int c = 0; c < C; c += 8)
          sts128(p_row + (((c / 8) ^ (r % 8)) * 16), pack2<BF16>(x[c], x[c + 1]), pack2<BF16>(x[c + 2], x[c + 3]),
                 pack2<BF16>(x[c + 4], x[c + 5]), pack2<BF16>(x[c + 6], x[c + 7]));
        if (static_cast<long long>(t + 1) * kKeys > it.len) {
          // The last tile: what the page holds behind the last key may be anything, and 0 * NaN is
          // not 0, so those rows of V are cleared.
          mbar_wait_warp(v_full(n % S), (n / S) & 1, ctx);
          if (key >= it.len && group == 0) {
            const uint32_t row = smem_u32(smem + L::kVOff + (n % S) * L::kTile) + r * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) sts128(row + c * L::kChunk + i * 16, 0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(p_full);
      }
      // Every S of this unit is read, so Q may be replaced.
      if (more && following.t1 > following.t0) load_q(following);

      // ---------------------------------------------------------- the run's result
      const bool some = n > n_first;
      if (some) {
        mbar_wait_warp(pv_done, (n - 1) & 1, ctx);
        tc_fence_after();
      }
      reduce_columns<C, false>(l);
      store_columns<C>(red + quarter * C, l);
      group_barrier(bar_id);
      const int slot = 2 * static_cast<int>(blockIdx.x) + (unit_at > lo ? 1 : 0);
      const int left = it.n * p.G - it.r0 - col0;  // columns of this group that are rows
      if (gt < C) {
        const float sum = (red[gt] + red[C + gt]) + (red[2 * C + gt] + red[3 * C + gt]);
        const float lse2 = sum > 0.0f ? lg2(sum) - ref[gt] : (sum == 0.0f ? -INFINITY : sum);
        factor[gt] = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
        ref[gt] = kNoKey;
        if (it.whole) {
          if (gt < left) {
            const int rr = it.r0 + col0 + gt, tok = rr / p.G;
            p.lse[static_cast<size_t>(it.q0 + tok) * p.Hq + it.h * p.G + rr - tok * p.G] = lse2 * 0.6931471805599453f;
          }
        } else {
          p.part_lse[static_cast<size_t>(slot) * N + col0 + gt] = lse2;
        }
      }
      group_barrier(bar_id);
#pragma unroll
      for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
        const uint32_t t_o = tmem + lanes + kTmemO + half * N + col0;
        // M = 64 keeps row i in lane 32 * (i / 16) + i % 16.
        const int e = D == 64 ? quarter * 16 + lane : half * 128 + r;
        const bool mine = (D != 64 || lane < 16) && e < p.d;
        int tok = (it.r0 + col0) / p.G, g = (it.r0 + col0) - tok * p.G;
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          uint32_t o[16];
          if (some) {
            tmem_ld16(t_o + c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = factor[c + i];
            const float y = some ? (f == 0.0f ? 0.0f : __uint_as_float(o[i]) * f) : 0.0f;
            if (it.whole) {
              if (mine && c + i < left)
                p.o[(it.q0 + tok) * p.o_row + (it.h * p.G + g) * p.o_head + e] =
                    static_cast<uint16_t>(pack2<BF16>(y, 0.0f));
              if (++g == p.G) {
                g = 0;
                ++tok;
              }
            } else if (mine) {
              p.part_o[(static_cast<size_t>(slot) * N + col0 + c + i) * D + e] = y;
            }
          }
        }
      }
      tc_fence_before();
      // The unit that goes on in the next CTAs: what the merge needs to know.
      if (!it.whole && it.t0 == 0) {
        const long long last = (unit_at + it.tiles) * workers;  // rounded up: the last worker with a tile of it
        cut0 = make_int4(1, slot, static_cast<int>((last + total - 1) / total) - 1, it.q0);
        cut1 = make_int4(it.h, it.r0, it.n, 0);
      }
      group_barrier(bar_id);  // factor is read; the scratch may become P again
      it = following;
      have = more;
    }
    if (tid == 0 && !p.by_unit) {
      p.cuts[2 * blockIdx.x] = cut0;
      p.cuts[2 * blockIdx.x + 1] = cut1;
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
__global__ void __launch_bounds__(256) fa_tree_merge_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x, lane = threadIdx.x % 32, c = blockIdx.y * 8 + threadIdx.x / 32;
  const int4 a = p.cuts[2 * w];
  if (a.x == 0 || c >= N) return;
  const int4 u = p.cuts[2 * w + 1];  // cache head, first row, rows of the request
  const int rr = u.y + c;
  if (rr >= u.z * p.G) return;
  const int pieces = a.z - w + 1;
  auto slot_of = [&](int i) { return i == 0 ? a.y : 2 * (w + i); };
  float m = -INFINITY;
  bool nan = false;
  for (int i = lane; i < pieces; i += 32) {
    const float x = p.part_lse[static_cast<size_t>(slot_of(i)) * N + c];
    nan |= x != x;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  nan = __any_sync(0xffffffffu, nan);
  constexpr int kPer = D / 32;  // elements of a lane, consecutive
  float z = 0.0f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
  if (m != -INFINITY || nan) {
    for (int i = 0; i < pieces; ++i) {
      const size_t row = static_cast<size_t>(slot_of(i)) * N + c;
      const float x = p.part_lse[row];
      if (x == -INFINITY) continue;
      const float f = ex2(x - m);
      z += f;
      const float* src = p.part_o + row * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 y = *reinterpret_cast<const float2*>(src + k);
        acc[k] = fmaf(f, y.x, acc[k]);
        acc[k + 1] = fmaf(f, y.y, acc[k + 1]);
      }
    }
  }
  const float inv = z > 0.0f ? 1.0f / z : z;
  const int tok = rr / p.G, head = u.x * p.G + rr - tok * p.G;
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
