// Rotary positions over several axes: fa_rope (training, both directions) and
// fa_rope_append (a serving step's q and k, with k and v written to the paged cache).
//
// Pair i of token t turns by the angle positions[axis[i]][t] * inv_freq[i]. A CTA takes a
// few tokens and all heads (or, with few tokens, a run of them): its threads compute the
// tokens' cosines and sines into shared memory, two each, while their first loads are on
// the way, and a thread then keeps those of its eight pairs of one token for all its heads.
// The angle is reduced to a fraction of a turn in 64 bits (position times frequency over
// 2 pi, minus the nearest whole number) before sincospif takes it in 32: the fraction's
// rounding is at most 2^-25 of a turn whatever the position.
//
// It moves each byte once in and once out and is bound by HBM: a thread takes two
// 16-byte pieces of a row (the eight x and the eight y of its pairs or, past the rotated
// elements and for V, 32 bytes to copy) of four heads at a time, so that eight loads are
// in flight. Measured: 16384 rows of 32 + 2 x 8 heads of 128 rotated and written to the cache
// (403 MB) in 66 us, 6.1 TB/s of the 6.5 a copy reaches; the two gradients of B=4 H=16 N=4096 d=128
// (134 MB each, a launch each) in 52 us. Each CTA computing its cosines in registers, and so again
// for every run of heads, took 72 and 58; 256 threads a CTA 68 and 55.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_cache.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;   // heads whose loads are in flight
constexpr int kHeadGroups = 4;  // threads that share a token's pairs, each with every fourth head

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

// (x, y) -> (x cos - y sin, x sin + y cos) of eight pairs: a holds the x and c the y, or with
// kPairs a and c hold four pairs each, x and y in turn.
template <bool BF16, bool kPairs>
__device__ __forceinline__ void rotate(uint4& a, uint4& c, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpack2<BF16>(wa[k]), y = unpack2<BF16>(wc[k]);
    if constexpr (kPairs) {
      wa[k] = sm100::pack2<BF16>(x.x * cs[k] - x.y * sn[k], x.x * sn[k] + x.y * cs[k]);
      wc[k] = sm100::pack2<BF16>(y.x * cs[4 + k] - y.y * sn[4 + k], y.x * sn[4 + k] + y.y * cs[4 + k]);
    } else {
      wa[k] = sm100::pack2<BF16>(x.x * cs[2 * k] - y.x * sn[2 * k], x.y * cs[2 * k + 1] - y.y * sn[2 * k + 1]);
      wc[k] = sm100::pack2<BF16>(x.x * sn[2 * k] + y.x * cs[2 * k], x.y * sn[2 * k + 1] + y.y * cs[2 * k + 1]);
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  c = make_uint4(wc[0], wc[1], wc[2], wc[3]);
}

// Grid: token tiles x runs of `heads_per` of all parts' heads. UNITS = d / 16 threads a token
// and head group.
template <int UNITS, bool BF16, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads, 6) fa_rope_kernel(const __grid_constant__ RopeArgs p, int heads_per) {
  constexpr int kTile = kRopeThreads / (UNITS * kHeadGroups);  // tokens of a CTA
  constexpr int kHalf = UNITS * 8;                              // pairs of a row, at most
  __shared__ __align__(16) float s_cos[kTile * kHalf], s_sin[kTile * kHalf];
  const int u = threadIdx.x % UNITS, tt = threadIdx.x / UNITS % kTile, g = threadIdx.x / (UNITS * kTile);
  const long long tokens = static_cast<long long>(p.B) * p.N, t0 = static_cast<long long>(blockIdx.x) * kTile;
  const long long t = t0 + tt;
  const bool live = g < kHeadGroups && t < tokens;
  const long long b = p.B == 1 ? 0 : t / p.N, n = t - b * p.N;
  const int half = p.rot / 2;
  const bool turned = 16 * u < p.rot;
  const int o0 = turned && !kPairs ? 8 * u : 16 * u;
  const int o1 = turned && !kPairs ? half + 8 * u : 16 * u + 8;
  bool ready = false;  // the tokens' cosines and sines are in registers
  float cs[8], sn[8];
  auto angles = [&] {
    for (int e = threadIdx.x; e < kTile * half; e += kRopeThreads) {
      const int i = e % half;
      const long long te = t0 + e / half, be = p.B == 1 ? 0 : te / p.N;
      const int ax = p.axis[i];
      float c = 1.0f, s = 0.0f;
      if (ax < p.n_axes && te < tokens) {
        const int pos = p.positions[ax * p.pos_axis + be * p.pos_b + (te - be * p.N)];
        const double turns = static_cast<double>(pos) * (static_cast<double>(p.inv_freq[i]) * 0.15915494309189535);
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
      }
      s_cos[(e / half) * kHalf + i] = c;
      s_sin[(e / half) * kHalf + i] = p.inverse ? -s : s;
    }
    __syncthreads();
    if (turned) {
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float4 c = *reinterpret_cast<const float4*>(&s_cos[tt * kHalf + 8 * u + k]);
        const float4 s = *reinterpret_cast<const float4*>(&s_sin[tt * kHalf + 8 * u + k]);
        cs[k] = c.x, cs[k + 1] = c.y, cs[k + 2] = c.z, cs[k + 3] = c.w;
        sn[k] = s.x, sn[k + 1] = s.y, sn[k + 2] = s.z, sn[k + 3] = s.w;
      }
    }
  };
  int first = blockIdx.y * heads_per, left = heads_per;  // in the part at hand; heads to do
  for (int i = 0; i < p.n_parts && left > 0; ++i) {
    const RopePart& r = p.part[i];
    if (first >= r.heads) {
      first -= r.heads;
      continue;
    }
    const int count = min(r.heads - first, left);
    left -= count;
    const uint16_t* src = r.src + b * r.src_b + n * r.src_n + first * r.src_h;
    uint16_t* dst = r.dst + first * r.dst_h;
    bool there = live;
    if (r.to_cache) {
      const long long slot = live ? p.slot[t] : -1;
      there = slot >= 0 && slot < p.cache_rows;
      dst += (slot >> p.page_shift) * r.dst_b + (slot & ((1 << p.page_shift) - 1)) * r.dst_n;
    } else {
      dst += b * r.dst_b + n * r.dst_n;
    }
    first = 0;
    for (int h0 = 0; h0 < count; h0 += kRopeAhead * kHeadGroups) {
      uint4 a[kRopeAhead], c[kRopeAhead];
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        const int h = h0 + g + k * kHeadGroups;
        if (there && h < count) {
          a[k] = *reinterpret_cast<const uint4*>(src + h * r.src_h + o0);
          c[k] = *reinterpret_cast<const uint4*>(src + h * r.src_h + o1);
        }
      }
      if (r.rotate && !ready) {  // the same for all threads of the CTA
        angles();
        ready = true;
      }
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        const int h = h0 + g + k * kHeadGroups;
        if (there && h < count) {
          if (r.rotate && turned) rotate<BF16, kPairs>(a[k], c[k], cs, sn);
          *reinterpret_cast<uint4*>(dst + h * r.dst_h + o0) = a[k];
          *reinterpret_cast<uint4*>(dst + h * r.dst_h + o1) = c[k];
        }
      }
    }
  }
}

template <int UNITS, bool BF16>
int launch_units(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kTile = kRopeThreads / (UNITS * kHeadGroups);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long tiles = (tokens + kTile - 1) / kTile;
  int heads = 0;
  for (int i = 0; i < a.n_parts; ++i) heads += a.part[i].heads;
  // Few tokens: the heads are cut into runs until there are about six CTAs an SM; each run
  // computes its tokens' cosines again.
  const long long want = heads * tiles / (6 * 148);
  int per = static_cast<int>(want < kHeadGroups ? kHeadGroups : (want > heads ? heads : want));
  const int runs = (heads + per - 1) / per;
  per = (heads + runs - 1) / runs;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + per - 1) / per));
  if (a.pairs) fa_rope_kernel<UNITS, BF16, true><<<grid, kRopeThreads, 0, stream>>>(a, per);
  else fa_rope_kernel<UNITS, BF16, false><<<grid, kRopeThreads, 0, stream>>>(a, per);
  return static_cast<int>(cudaGetLastError());
}

template <bool BF16>
int launch_type(const RopeArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_units<2, BF16>(a, stream);
    case 64: return launch_units<4, BF16>(a, stream);
    case 96: return launch_units<6, BF16>(a, stream);
    case 128: return launch_units<8, BF16>(a, stream);
    default: return launch_units<16, BF16>(a, stream);
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace fa
