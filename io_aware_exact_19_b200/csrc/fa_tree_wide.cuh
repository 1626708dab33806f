// The paged tree attention for units of more than 64 query rows (prompt chunks, large trees),
// d <= 128: 128 rows as the MMA's rows.
//
// With that many columns the turned-around product of fa_tree.cuh is bound by shared memory: its
// MMAs read K and Q, V and P from there (16 KB for 128 cycles' work at 128 bytes a cycle), next to
// P written and the tiles loaded. Here Q and P stay in TMEM, as the A operands of
//   S = Q K_j^T      O += P V_j          (lane = query row)
// so shared memory holds and feeds K and V alone, half the traffic, and a row's reference, sum
// and mask belong to one lane: nothing is reduced across lanes.
//
// Sixteen softmax warps: warpgroup g takes keys 32g .. 32g + 31 of every tile, so a row is worked
// on by four warps (one of each warpgroup, the same TMEM lanes). They agree on the row's
// reference: it moves only when a score exceeds it by more than 8 (log2 units), which one barrier
// of the four warps with an OR decides per tile; the first tile's maximum, and a moved one, goes
// through shared memory.
//
// TMEM (512 columns): S of tiles n, n + 1 at 0 and 128 (P over the first 64 of them, in 16 bits),
// O at 256, Q at 384.
//
// A tile of 128 keys takes 2100 cycles at d = 128 (the MMAs 1024, the exponentials 1024): two chunks of
// 2048 rows behind 8192 keys, H_kv = 8, groups of 4: 583 us, 988 TFLOP/s (of 1653 measured for a plain
// product; under the power cap, back to back, 630 to 670 us); one prompt of 8192 rows 566 us, 930
// TFLOP/s. Tried and slower: two sets of eight warps taking the tiles in turn, each with its own O (1960
// cycles a tile, but more to join at the end: the same on chunks, 64 for 60 us on 16 trees of 48 x 7
// rows); P computed before the vote; a quarter to a half of the exponentials as polynomials on the FMA
// pipes (592, 597, 620 us).
#pragma once

#include "fa_tree.cuh"

namespace fa {
namespace tree {

template <int D>
struct WideSmem {
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kChunk = kKeys * 128;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kStages * kTile;
  static constexpr int kRedOff = kVOff + kStages * kTile;  // float [4 warpgroups][128 rows]
  static constexpr int kTailOff = kRedOff + 4 * 4 * 128;
  static constexpr int kAlloc = kTailOff + static_cast<int>(sizeof(Tail<128, kStages>));
  static_assert(kAlloc <= 232448, "shared memory");
};

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 bytes to global memory (32-byte aligned).
__device__ __forceinline__ void stg256(float* p, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(long long n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(608, 1)
    fa_tree_wide_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ Params p) {
  using L = WideSmem<D>;
  constexpr int N = 128, S = L::kStages, kSoftWarps = 16, kThreads = 608;
  constexpr int kSlice = D / 4;  // elements of Q and of O that a warpgroup moves
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail<N, S>& tail = *reinterpret_cast<Tail<N, S>*>(smem + L::kTailOff);
  float* red = reinterpret_cast<float*>(smem + L::kRedOff);
  const Bars<S> bar{smem_u32(tail.bars)};
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr uint32_t kTmemO = 256, kTmemQ = 384;
  const Start start = begin<N, S, kThreads, kSoftWarps>(p, tail, bar, smem + L::kKOff);
  const uint32_t tmem = start.tmem;
  const WaitCtx ctx{&tail.abort_flag, p.status, p.timeout_ns};

  if (warp == kSoftWarps || warp == kSoftWarps + 2) {
    load_tiles<D>(p, tail, bar, warp != kSoftWarps, &tmap_k, &tmap_v, smem + L::kKOff, smem + L::kVOff, ctx);
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_f16(BF16, N, kKeys, false, false);
    constexpr uint32_t idesc_o = idesc_f16(BF16, N, D, false, true);
    const uint64_t dK = sdesc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
    const uint64_t dV = sdesc_sw128(smem_u32(smem + L::kVOff), L::kChunk, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto issue_s = [&](int n, int s) {
      // S of tile n goes where P of tile n - 2 was; its P V was issued before.
      const uint64_t b = sdesc_add(dK, static_cast<uint32_t>(s) * L::kTile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ts(tm + (n & 1) * 128, tm + kTmemQ + 8 * k, sdesc_add(b, (k / 4) * L::kChunk + (k % 4) * 32), idesc_s, k > 0);
        umma_commit(bar.s_full(n));
        umma_commit(bar.k_empty(s));
        mbar_arrive(bar.s_full(n));
      }
      __syncwarp();
    };
    auto issue_o = [&](int n, int s, uint32_t add) {
      const uint64_t b = sdesc_add(dV, static_cast<uint32_t>(s) * L::kTile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          umma_ts(tm + kTmemO, tm + (n & 1) * 128 + 8 * k, sdesc_add(b, k * 2048), idesc_o, k > 0 ? 1u : add);
        umma_commit(bar.pv_done(n));
        umma_commit(bar.v_empty(s));
      }
      __syncwarp();
    };
    issue_tiles(p, tail, bar, ctx, issue_s, issue_o);
  } else {
    // ------------------------------------------------------------ softmax
    // (After a wait ran out the threads go on through the same barriers to the end; see fa_tree.cuh.)
    const int group = warp / 4, quarter = warp % 4, r = quarter * 32 + lane;
    const int bar_id = 1 + quarter;  // of the four warps that share these rows
    const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = p.scale_log2;
    constexpr float kBias = BF16 ? 0.0f : 7.0f;  // keeps the fp16 P in its normal range (see fa_tree.cuh)
    int n = 0;  // tiles seen

    // Q: a thread's slice of its row, from memory to registers, then to TMEM.
    uint4 qv[kSlice / 8];
    auto fetch_q = [&](const Item& it) {
      const int rr = it.r0 + r, tok = p.by_group(rr), g = rr - tok * p.G;
      const uint16_t* src = p.q + (it.q0 + tok) * p.q_row + (it.h * p.G + g) * p.q_head + kSlice * group;
#pragma unroll
      for (int k = 0; k < kSlice / 8; ++k) {
        qv[k] = make_uint4(0, 0, 0, 0);
        if (tok < it.n && kSlice * group + 8 * k < p.d) qv[k] = *reinterpret_cast<const uint4*>(src + 8 * k);
      }
    };
    auto store_q = [&] {
      const uint32_t to = base + kTmemQ + (kSlice / 2) * group;
#pragma unroll
      for (int k = 0; k < kSlice / 8; k += 2) {
        const uint32_t w[8] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w, qv[k + 1].x, qv[k + 1].y, qv[k + 1].z, qv[k + 1].w};
        tmem_st8(to + 4 * k, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.q_full());
    };

    Walk<N>& walk = tail.walk;
    auto soft_barrier = [] { asm volatile("bar.sync 8, 512;" ::: "memory"); };
    auto advance = [&](int to) {
      Item& it = walk.item[to];
      walk.cur.next(p, it);
      walk.unit_at[to] = walk.cur.pos - it.take - it.t0;
    };
    if (tid == 0) {
      walk.cur = tail.first_cur;
      walk.item[0] = tail.first_item;
      walk.unit_at[0] = walk.cur.pos - walk.item[0].take - walk.item[0].t0;
      if (!p.by_unit) p.cuts[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    soft_barrier();
    if (walk.item[0].valid && walk.item[0].t1 > walk.item[0].t0) {
      fetch_q(walk.item[0]);
      store_q();
    }
    int which = 0, then = 1;
    while (walk.item[which].valid) {
      const Item& it = walk.item[which];
      const int t1 = it.t1, len = it.len, clean = it.clean;
      const int tok = p.by_group(it.r0 + r);  // of this row; past the last row: >= it.n
      if (tid == 0) advance(then);
      const unsigned long long* mask_row = nullptr;
      if (p.tree_mask != nullptr && tok < it.n) {
        mask_row = p.tree_mask + static_cast<size_t>(it.q0 + tok) * p.words;
        if (t1 > clean) asm volatile("prefetch.global.L1 [%0];" ::"l"(mask_row));
      }
      float ref = -kNoKey, l0 = 0.0f, l1 = 0.0f;
      const int n_first = n;
      for (int t = it.t0; t < t1; ++t, ++n) {
        const int key0 = t * kKeys + 32 * group;
        uint32_t seen = ~0u;  // bit c: the row sees key key0 + c
        if (t >= clean) {
          const long long own = static_cast<long long>(key0) - it.ctx;  // index of key0 among the new tokens
          if (p.tree_mask == nullptr) {
            seen = low_bits(tok + 1 - own);
          } else {
            seen = low_bits(-own);  // the context
            if (mask_row != nullptr && own > -32) {
              auto word = [&](long long i) { return i >= 0 && i < p.words ? mask_row[i] : 0ull; };
              if (own < 0) {
                seen |= static_cast<uint32_t>(word(0) << -own);
              } else {
                const long long w = own / 64;
                const int at = static_cast<int>(own % 64);
                seen |= static_cast<uint32_t>(word(w) >> at);
                if (at > 32) seen |= static_cast<uint32_t>(word(w + 1) << (64 - at));
              }
            }
          }
          seen &= low_bits(static_cast<long long>(len) - key0);
        }
        wait_tile(bar.s_full(n), (n >> 1) & 1, ctx);
        tc_fence_after();
        bool masked = t >= clean;
        if (tail.bad_page[n % (S + 2)]) {
          // A page index outside the cache: its keys are not there.
          masked = true;
          const int step = min(1 << p.page_shift, 32);
          for (int k = 0; k < 32 && key0 + k < len; k += step) {
            const int page = p.block_table[static_cast<size_t>(it.b) * p.max_pages + ((key0 + k) >> p.page_shift)];
            if (page < 0 || page >= p.num_pages) seen &= ~(low_bits(step) << k);
          }
        }
        const uint32_t t_s = base + (n & 1) * 128;
        float x[32];
        load_scores<32>(t_s + 32 * group, x);
        auto apply_mask = [&] {
          if (masked) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((seen >> c) & 1u)) x[c] = -INFINITY;
          }
        };
        auto largest = [&] {
          float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 32; c += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], x[c + i]);
          }
          return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        };
        const bool first = n == n_first;
        bool move = first;
        if (!first) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) fma2(x[c], x[c + 1], sl2, -ref, -ref);
          apply_mask();
          // Also: behind this barrier all four warps have read their scores, and P may go over them.
          move = group_any(bar_id, largest() > kRescale + kBias);
        }
        if (move) {
          // Some row's reference moves, or is set by the run's first tile. P V of the tile before,
          // which adds to O, must be complete.
          if (!first) {
            wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
            tc_fence_after();
            load_scores<32>(t_s + 32 * group, x);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] *= sl2;
          apply_mask();
          red[group * 128 + r] = largest();
          group_barrier(bar_id);
          const float high = fmaxf(fmaxf(red[r], red[128 + r]), fmaxf(red[256 + r], red[384 + r])) - kBias;
          const float now = high > ref + kRescale ? high : ref;
          if (!first) {
            const float f = ex2(ref - now);
            l0 *= f;
            l1 *= f;
#pragma unroll 1
            for (int c = 0; c < kSlice; c += 16) {
              uint32_t o[16];
              tmem_ld16(base + kTmemO + kSlice * group + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(base + kTmemO + kSlice * group + c, o);
            }
            tmem_st_wait();
          }
          ref = now;
#pragma unroll
          for (int c = 0; c < 32; c += 2) add2(x[c], x[c + 1], -ref, -ref);
        }
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          x[c] = ex2(x[c]);
          x[c + 1] = ex2(x[c + 1]);
          add2(l0, l1, x[c], x[c + 1]);
          w[c / 2] = pack2<BF16>(x[c], x[c + 1]);
        }
        tmem_st16(t_s + 16 * group, w);
        tmem_st_wait();
        if (t >= clean && t * kKeys + (kKeys - 1) >= len) {
          // The last tile: what the page holds behind the last key may be anything, and 0 * NaN is
          // not 0, so those rows of V are cleared (a thread a row, two 16-byte pieces of each chunk).
          wait_tile(bar.v_full(n % S), (n / S) & 1, ctx);
          const int row = tid % 128;
          if (t * kKeys + row >= len) {
            const uint32_t to = smem_u32(smem + L::kVOff + (n % S) * L::kTile) + row * 128 + group * 32;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              sts128(to + c * L::kChunk, 0, 0, 0, 0);
              sts128(to + c * L::kChunk + 16, 0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.p_full(n));
      }
      // Every S of this unit is read, so Q may be replaced.
      soft_barrier();  // the item that follows is known
      const bool more = walk.item[then].valid && walk.item[then].t1 > walk.item[then].t0;
      if (more) fetch_q(walk.item[then]);  // arrives while the sums are joined

      // ---------------------------------------------------------- the run's result
      const bool some = n > n_first;
      red[group * 128 + r] = l0 + l1;
      group_barrier(bar_id);
      const float sum = (red[r] + red[128 + r]) + (red[256 + r] + red[384 + r]);
      if (more) store_q();
      const bool whole = it.take == it.tiles;
      const long long unit_at = walk.unit_at[which];
      const int slot = 2 * static_cast<int>(blockIdx.x) + (unit_at > start.lo ? 1 : 0);
      const float lse2 = sum > 0.0f ? lg2(sum) + ref : (sum == 0.0f ? -INFINITY : sum);
      const float f = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
      const int g = it.r0 + r - tok * p.G;
      const size_t out_row = static_cast<size_t>(it.q0) + tok;
      if (group == 0 && tok < it.n) {
        if (whole) p.lse[out_row * p.Hq + it.h * p.G + g] = lse2 * 0.6931471805599453f;
        else p.part_lse[static_cast<size_t>(slot) * N + r] = lse2;
      }
      if (some) {
        wait_tile(bar.pv_done(n - 1), ((n - 1) >> 1) & 1, ctx);
        tc_fence_after();
      }
      uint16_t* dst = p.o + out_row * p.o_row + (it.h * p.G + g) * p.o_head + kSlice * group;
      float* part = p.part_o + (static_cast<size_t>(slot) * N + r) * D + kSlice * group;
#pragma unroll 1
      for (int c = 0; c < kSlice; c += 16) {
        uint32_t o[16];
        if (some) {
          tmem_ld16(base + kTmemO + kSlice * group + c, o);
          tmem_ld_wait();
        }
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = some && f != 0.0f ? __uint_as_float(o[i]) * f : 0.0f;
        if (tok < it.n) {
          if (!whole) {
            stg256(part + c, y);
            stg256(part + c + 8, y + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              if (kSlice * group + c + i < p.d)
                *reinterpret_cast<uint4*>(dst + c + i) =
                    make_uint4(pack2<BF16>(y[i], y[i + 1]), pack2<BF16>(y[i + 2], y[i + 3]), pack2<BF16>(y[i + 4], y[i + 5]),
                               pack2<BF16>(y[i + 6], y[i + 7]));
          }
        }
      }
      tc_fence_before();
      // The unit that goes on in the next CTAs (at most the last one): what the merge needs to know.
      if (!whole && it.t0 == 0 && tid == 0) {
        p.cuts[2 * blockIdx.x] = make_int4(1, slot, start.share.worker(unit_at + it.tiles - 1), it.q0);
        p.cuts[2 * blockIdx.x + 1] = make_int4(it.h, it.r0, it.n, 0);
      }
      group_barrier(bar_id);  // the sums are read
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

}  // namespace tree
}  // namespace fa
