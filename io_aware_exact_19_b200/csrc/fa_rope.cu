// Rotary positions over several axes: fa_rope (training, both directions) and
// fa_rope_append (a serving step's q and k, with k and v written to the paged cache).
//
// Pair i of token t turns by the angle positions[axis[i]][t] * inv_freq[i]. A CTA takes
// a tile of tokens: its threads compute the tile's cosines and sines once into shared
// memory and apply them to all heads, so their cost is shared by Hq + H_kv rows. The
// angle is reduced to a fraction of a turn in 64 bits (position times frequency over
// 2 pi, minus the nearest whole number) before sincospif takes it in 32: the fraction's
// rounding is at most 2^-25 of a turn whatever the position.
//
// It moves each byte once in and once out and is bound by HBM; a thread takes two
// 16-byte pieces of a row, the eight x and the eight y of eight pairs (or, past the
// rotated elements and for V, 32 bytes to copy).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_cache.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTile = 16;  // tokens per CTA
constexpr int kRopeMaxPairs = 128;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeArgs p, int tile) {
  __shared__ float2 turn[kRopeMaxTile * kRopeMaxPairs];  // cos, sin of [token][pair]
  const int tid = threadIdx.x;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const long long t0 = static_cast<long long>(blockIdx.x) * tile;
  const int here = static_cast<int>(min(static_cast<long long>(tile), tokens - t0));
  const int half = p.rot / 2;
  for (int e = tid; e < here * half; e += kRopeThreads) {
    const int i = e % half;
    const long long t = t0 + e / half;
    const long long b = t / p.N;
    const int ax = p.axis[i];
    float c = 1.0f, s = 0.0f;
    if (ax < p.n_axes) {
      const int pos = p.positions[ax * p.pos_axis + b * p.pos_b + (t - b * p.N)];
      const double turns = static_cast<double>(pos) * static_cast<double>(p.inv_freq[i]) * 0.15915494309189535;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
    }
    turn[e] = make_float2(c, p.inverse ? -s : s);
  }
  __syncthreads();
  const int units = p.d / 16, turned = p.rot / 16;  // 32-byte tasks of a row; the first `turned` rotate
  for (int part = 0; part < p.n_parts; ++part) {
    const RopePart& r = p.part[part];
    const int tasks = r.heads * here * units;
    for (int e = tid; e < tasks; e += kRopeThreads) {
      const int u = e % units, rest = e / units;
      const int tt = rest % here, h = rest / here;
      const long long t = t0 + tt, b = t / p.N, n = t - b * p.N;
      const uint16_t* src = r.src + b * r.src_b + h * r.src_h + n * r.src_n;
      uint16_t* dst;
      if (r.to_cache) {
        const long long slot = p.slot[t];
        if (slot < 0 || slot >= p.cache_rows) continue;
        dst = r.dst + (slot >> p.page_shift) * r.dst_b + h * r.dst_h + (slot & ((1 << p.page_shift) - 1)) * r.dst_n;
      } else {
        dst = r.dst + b * r.dst_b + h * r.dst_h + n * r.dst_n;
      }
      const bool rotate = r.rotate && u < turned;
      // Elements of the two pieces: eight x and eight y of pairs 8u .. 8u + 7, or 16 in a row.
      const int o0 = rotate && !p.pairs ? 8 * u : 16 * u;
      const int o1 = rotate && !p.pairs ? half + 8 * u : 16 * u + 8;
      uint4 a = *reinterpret_cast<const uint4*>(src + o0);
      uint4 c = *reinterpret_cast<const uint4*>(src + o1);
      if (rotate) {
        uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
        const float2* cs = turn + tt * half + 8 * u;
        if (p.pairs) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = unpack2<BF16>(wa[k]), y = unpack2<BF16>(wc[k]);
            const float2 f = cs[k], g = cs[4 + k];
            wa[k] = sm100::pack2<BF16>(x.x * f.x - x.y * f.y, x.x * f.y + x.y * f.x);
            wc[k] = sm100::pack2<BF16>(y.x * g.x - y.y * g.y, y.x * g.y + y.y * g.x);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = unpack2<BF16>(wa[k]), y = unpack2<BF16>(wc[k]);
            const float2 f = cs[2 * k], g = cs[2 * k + 1];
            wa[k] = sm100::pack2<BF16>(x.x * f.x - y.x * f.y, x.y * g.x - y.y * g.y);
            wc[k] = sm100::pack2<BF16>(x.x * f.y + y.x * f.x, x.y * g.y + y.y * g.x);
          }
        }
        a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
        c = make_uint4(wc[0], wc[1], wc[2], wc[3]);
      }
      *reinterpret_cast<uint4*>(dst + o0) = a;
      *reinterpret_cast<uint4*>(dst + o1) = c;
    }
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const long long tokens = static_cast<long long>(a.B) * a.N;
  if (tokens == 0) return 0;
  const int tile = 1;
  const unsigned grid = static_cast<unsigned>((tokens + tile - 1) / tile);
  if (a.bf16)
    fa_rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, tile);
  else
    fa_rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, tile);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
