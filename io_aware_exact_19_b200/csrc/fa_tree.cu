// Host launcher of the paged tree attention.
#include "fa_tree.cuh"
#include "fa_tree_wide.cuh"

#include "fa_cache.h"
#include "tma_host.h"

namespace fa {
namespace {

// Query rows of a unit: the smallest tile that holds a request's rows of one cache head, since a
// wider one costs as if it were full (a tree of 64 rows over 64K keys, d = 64: 65 us with 64, 75
// with 128; 96 rows over 4000 keys: 54 us with 128, 68 as two of 64). With head dimension 256
// shared memory holds no more than 64 rows next to one stage of K and V.
int row_tile(int max_q, int group, int D) {
  const long long rows = static_cast<long long>(max_q) * group;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 || D == 256 ? 64 : 128));
}

int padded_dim(int d) { return d <= 64 ? 64 : (d <= 128 ? 128 : 256); }

// Prompt chunks with at least a unit for every SM are not cut. (H_kv = 8, groups of 4, d = 128: one
// prompt of 1024 rows 44 us cut and 27 not, 2048 rows 90 and 62, 8192 rows 970 and 566; 8 x 128 rows over
// 3000 keys 78 and 71; 40 of 300 rows behind 0 to 30000 keys 4700 and 3500; 64 single rows over 1000 to
// 8000 keys next to a prompt of 1024 230 and 210.) The rule counts units, since only the device knows their
// lengths, and loses where few units are long: where the last wave of them is nearly empty (just above
// 148 units: 600 rows behind 20000 keys at d = 64 188 us cut and 335 not, 330 x 7 behind 25000 245 and 437,
// 2 x 300 behind 3000 57 and 69; 312 units behind 20000 445 and 550), and where a long request stands next
// to a prompt (one row over 64K keys, 1024 rows over none: 89 and 549).
bool by_unit(int rows, int max_q, int Hq, int H_kv, int tile) {
  const long long units = static_cast<long long>(H_kv) * ((static_cast<long long>(rows) * (Hq / H_kv) + tile - 1) / tile);
  return static_cast<long long>(max_q) * (Hq / H_kv) >= 512 && units >= tree::kMaxWorkers;
}

struct Workspace {
  size_t part_lse, cuts, total;
};

Workspace layout(int tile, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.part_lse = up(static_cast<size_t>(2) * tree::kMaxWorkers * tile * D * 4);
  w.cuts = w.part_lse + up(static_cast<size_t>(2) * tree::kMaxWorkers * tile * 4);
  w.total = w.cuts + up(static_cast<size_t>(2) * tree::kMaxWorkers * sizeof(int4));
  return w;
}

bool make_map(CUtensorMap* map, const fa_kv_cache& c, const void* base) {
  host::EncodeTiledFn fn = host::encode_tiled_fn();
  if (!fn) return false;
  const CUtensorMapDataType dt = c.dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.H_kv), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.row_stride) * 2, static_cast<cuuint64_t>(c.head_stride) * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(c.page_size < tree::kKeys ? c.page_size : tree::kKeys), 1, 1};
  const cuuint32_t unit[4] = {1, 1, 1, 1};
  return fn(map, dt, 4, const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, int N>
int launch_t(const TreeArgs& a, cudaStream_t stream) {
  CUtensorMap tk, tv;
  if (!make_map(&tk, a.cache, a.cache.k) || !make_map(&tv, a.cache, a.cache.v))
    return static_cast<int>(cudaErrorInvalidValue);
  const Workspace ws = layout(N, D);
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  tree::Params p{};
  p.q = static_cast<const uint16_t*>(a.q.data);
  p.o = static_cast<uint16_t*>(a.o.data);
  p.lse = a.lse;
  p.q_row = a.q.row_stride;
  p.q_head = a.q.head_stride;
  p.o_row = a.o.row_stride;
  p.o_head = a.o.head_stride;
  p.B = a.B;
  p.rows = a.rows;
  p.Hq = a.Hq;
  p.H_kv = a.cache.H_kv;
  p.G = a.Hq / a.cache.H_kv;
  p.by_group = tree::Divider::of(p.G);
  p.d = a.cache.d;
  p.num_pages = a.cache.num_pages;
  p.max_pages = a.max_pages;
  p.page_shift = a.page_shift;
  p.words = a.words;
  p.block_table = a.block_table;
  p.cu_q = a.cu_q;
  p.seq_len = a.seq_len;
  p.tree_mask = a.tree_mask;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.by_unit = by_unit(a.rows, a.max_q, a.Hq, a.cache.H_kv, N);
  const int sms = host::sm_count();
  p.workers = sms > 0 && sms < tree::kMaxWorkers ? sms : tree::kMaxWorkers;
  p.part_o = reinterpret_cast<float*>(base);
  p.part_lse = reinterpret_cast<float*>(base + ws.part_lse);
  p.cuts = reinterpret_cast<int4*>(base + ws.cuts);
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  p.withhold = a.withhold;

  // More than 64 rows a unit: the kernel with query rows as the MMA's rows.
  void (*kern)(CUtensorMap, CUtensorMap, tree::Params);
  int kSmem;
  unsigned kThreads;
  if constexpr (N == 128) {
    kern = tree::fa_tree_wide_kernel<D, BF16>;
    kSmem = tree::WideSmem<D>::kAlloc;
    kThreads = 608;
  } else {
    kern = tree::fa_tree_kernel<D, BF16, N>;
    kSmem = tree::Smem<D, N>::kAlloc;
    kThreads = 128 * tree::Smem<D, N>::kGroups + 96;
  }
  cudaError_t e = host::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return static_cast<int>(e);
  // By unit: request b has at most H_kv * (its rows / N rounded up) units. With eight units a worker and
  // more, the workers take them in turn, which spares each unit a CTA's start (39 prompts of 485 rows x 7
  // behind 36, H_kv = 3, d = 128: 226 us with a CTA for each, 174; 45 of 471 x 4, d = 64: 135 and 101; one of
  // 8192 rows 585 and 561; 24 of 500 x 4 behind up to 4000 443 and 417); with fewer, of any lengths, whichever
  // CTA is free takes the next (10 of 300 x 4 behind up to 4000, four a worker: 131 us, in turn 143; 16 behind
  // up to 6000, seven a worker: 270 and 285).
  long long grid = p.workers;
  if (p.by_unit) {
    const long long whole = static_cast<long long>(p.H_kv) * ((static_cast<long long>(a.rows) * p.G + N - 1) / N);
    const long long most = whole + static_cast<long long>(p.H_kv) * a.B;
    if (whole < 8ll * p.workers) grid = most;
  }
  kern<<<static_cast<unsigned>(grid), kThreads, kSmem, stream>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.by_unit) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.workers), N / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tree::fa_tree_merge_kernel<D, BF16, N>, p));
}

template <int D, bool BF16>
int launch_d(const TreeArgs& a, cudaStream_t stream) {
  switch (row_tile(a.max_q, a.Hq / a.cache.H_kv, D)) {
    case 16: return launch_t<D, BF16, 16>(a, stream);
    case 32: return launch_t<D, BF16, 32>(a, stream);
    case 64: return launch_t<D, BF16, 64>(a, stream);
    default: return launch_t<D, BF16, D == 256 ? 64 : 128>(a, stream);
  }
}

template <bool BF16>
int launch_type(const TreeArgs& a, cudaStream_t stream) {
  switch (padded_dim(a.cache.d)) {
    case 64: return launch_d<64, BF16>(a, stream);
    case 128: return launch_d<128, BF16>(a, stream);
    default: return launch_d<256, BF16>(a, stream);
  }
}

}  // namespace

size_t tree_fwd_workspace(int, int, int max_q, int Hq, int H_kv, int d) {
  return layout(row_tile(max_q, Hq / H_kv, padded_dim(d)), padded_dim(d)).total;
}

int launch_tree_fwd(const TreeArgs& a, cudaStream_t stream) {
  return a.cache.dtype == FA_BF16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace fa
