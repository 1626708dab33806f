// Attention of a ragged batch's new rows over the paged cache (fa_tree_fwd).
//
// One CTA per row and head, a warp per key in turn, each warp with its own running
// maximum, sum and O (the online-softmax recurrence), merged at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_cache.h"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  else return __half2float(*reinterpret_cast<const __half*>(&x));
}

template <bool BF16>
__global__ void __launch_bounds__(32 * kWarps) fa_tree_simple_kernel(const TreeArgs p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][256];
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int b = -1;
  for (int k = 0; k < p.B; ++k)
    if (p.cu_q[k] <= t && t < p.cu_q[k + 1]) {
      b = k;
      break;
    }
  if (b < 0) return;
  const int d = p.cache.d, i = t - p.cu_q[b], n = p.cu_q[b + 1] - p.cu_q[b];
  const int len = min(static_cast<long long>(p.seq_len[b]), static_cast<long long>(p.max_pages) << p.page_shift);
  const int ctx = p.seq_len[b] - n, kvh = h / (p.Hq / p.cache.H_kv);
  const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + t * p.q.row_stride + h * p.q.head_stride;
  float qv[8], acc[8], m = -INFINITY, l = 0.0f;
  for (int c = 0; c < d / 32; ++c) {
    qv[c] = widen<BF16>(q[lane + 32 * c]) * p.scale;
    acc[c] = 0.0f;
  }
  for (int j = warp; j < len; j += kWarps) {
    bool seen = p.tree_mask == nullptr ? j <= i + ctx : j < ctx;
    if (p.tree_mask != nullptr && j >= ctx && j - ctx < 64 * p.words)
      seen = (p.tree_mask[static_cast<size_t>(t) * p.words + (j - ctx) / 64] >> ((j - ctx) % 64)) & 1;
    const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + (j >> p.page_shift)];
    if (!seen || page < 0 || page >= p.cache.num_pages) continue;
    const long long off = page * p.cache.page_stride + kvh * p.cache.head_stride +
                          (j & ((1 << p.page_shift) - 1)) * p.cache.row_stride;
    const uint16_t* k = static_cast<const uint16_t*>(p.cache.k) + off;
    const uint16_t* v = static_cast<const uint16_t*>(p.cache.v) + off;
    float s = 0.0f;
    for (int c = 0; c < d / 32; ++c) s = fmaf(qv[c], widen<BF16>(k[lane + 32 * c]), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float nm = fmaxf(m, s), a = m == -INFINITY ? 0.0f : expf(m - nm), e = expf(s - nm);
    m = nm;
    l = l * a + e;
    for (int c = 0; c < d / 32; ++c) acc[c] = acc[c] * a + e * widen<BF16>(v[lane + 32 * c]);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int c = 0; c < d / 32; ++c) s_o[warp][lane + 32 * c] = acc[c];
  __syncthreads();
  float mx = -INFINITY, z = 0.0f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
  for (int w = 0; w < kWarps; ++w) z += s_m[w] == -INFINITY ? 0.0f : s_l[w] * expf(s_m[w] - mx);
  for (int c = threadIdx.x; c < d; c += 32 * kWarps) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += s_m[w] == -INFINITY ? 0.0f : s_o[w][c] * expf(s_m[w] - mx);
    x = z > 0.0f ? x / z : 0.0f;
    uint16_t* o = static_cast<uint16_t*>(p.o.data) + t * p.o.row_stride + h * p.o.head_stride + c;
    if constexpr (BF16) *reinterpret_cast<__nv_bfloat16*>(o) = __float2bfloat16_rn(x);
    else *reinterpret_cast<__half*>(o) = __float2half_rn(x);
  }
  if (threadIdx.x == 0) p.lse[static_cast<size_t>(t) * p.Hq + h] = z > 0.0f ? mx + logf(z) : -INFINITY;
}

}  // namespace

size_t tree_fwd_workspace(int, int, int, int, int, int) { return 256; }

int launch_tree_fwd(const TreeArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return 0;
  dim3 grid(static_cast<unsigned>(a.rows), static_cast<unsigned>(a.Hq));
  if (a.cache.dtype == FA_BF16) fa_tree_simple_kernel<true><<<grid, 32 * kWarps, 0, stream>>>(a);
  else fa_tree_simple_kernel<false><<<grid, 32 * kWarps, 0, stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
