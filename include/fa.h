/*
 * fa.h — C ABI of the B200 (sm_100a) exact attention library (libfa.so).
 *
 * The operation is exact scaled-dot-product attention as FlashAttention
 * computes it:
 *   S = scale * Q K^T, P = softmax(S) row by row, O = P V
 * ("FlashAttention" interview explainer, mstx.cn/posts/485, section 2.1,
 * standard attention; the 1/sqrt(d) scale as in the nanhubrain.csdn.net
 * FlashAttention essay, section 2). The forward streams K/V tiles past each
 * resident Q tile with the online-softmax recurrence (same explainer, section
 * 3.2) and writes only O and the per-row logsumexp. The backward recomputes P
 * from Q, K and the saved logsumexp instead of storing it ("FlashAttention"
 * concept card, lukebest.github.io, "反向：重算而非存储").
 *
 * Conventions shared by every entry point
 *   - Tensors q, k, v, o, dout, dq, dk, dv are contiguous [B, H, N, d] in the
 *     element type given by `dtype` (fp16 or bf16); lse is contiguous fp32
 *     [B, H, N]. All are DEVICE pointers, 16-byte aligned.
 *   - lse_i = ln sum_j exp(scale * q_i . k_j) over the keys row i may see
 *     (natural log, in the units of the scaled scores).
 *   - d must be 32, 64, 96 or 128, or 256 for the forward entry points
 *     (fa_fwd, fa_fwd_qk, fa_blocksparse_fwd, fa_fwd_splitkv; the backward,
 *     dropout and 8-bit entry points return FA_ERR_UNSUPPORTED for it). 32 and
 *     96 run in the 64 and 128 kernels with the missing columns zero-filled, at
 *     the cost of the padded width; 256 runs one query tile per CTA;
 *     N >= 1 (any value; ragged last tiles are handled); B, H >= 1 and
 *     B*H <= 65535.
 *   - causal != 0 masks key j > query i (top-left aligned; the essay's
 *     section 3.1 causal mask P_ij = 0 for j > i).
 *   - The caller owns all memory. The library allocates no device memory; the
 *     backward takes a caller-provided workspace of fa_bwd_workspace_size()
 *     bytes. Host-side tensor-map descriptors are built per call.
 *   - Every call is asynchronous on `stream` and never synchronises. Argument
 *     errors are reported before any launch; a failed launch returns
 *     FA_ERR_CUDA. Device-side time-outs (a wait that could not complete) are
 *     recorded in a device status word read by fa_device_status().
 *   - A row with no allowed key (possible only with a block mask) gets O = 0,
 *     lse = -inf and contributes zero gradients.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, non-positive size, bad dtype */
  FA_ERR_UNSUPPORTED = 2, /* valid but unsupported shape (head dimension, size limits) */
  FA_ERR_CUDA = 3,        /* a CUDA runtime call or kernel launch failed */
  FA_ERR_TIMEOUT = 4      /* a device-side wait gave up (see fa_device_status) */
} fa_status;

typedef enum { FA_FP16 = 0, FA_BF16 = 1 } fa_dtype;

/* Human-readable name of a status code (static string). */
const char* fa_status_string(fa_status s);

/*
 * Forward. Writes o [B,H,N,d] (dtype) and lse [B,H,N] (fp32).
 * q, k, v are read only. softmax_scale is usually 1/sqrt(d).
 */
fa_status fa_fwd(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float softmax_scale, int causal, cudaStream_t stream);

/*
 * Bytes of device workspace fa_bwd / fa_blocksparse_bwd need for these sizes:
 * two fp32 row vectors [B,H,ceil(N/128)*128] (D = rowsum(dO o O) and lse in
 * log2 units). Linear in N. Returns 0 for invalid sizes.
 */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward. Given the forward's inputs, its outputs o and lse, and the
 * incoming gradient dout = dL/dO, writes dq, dk, dv [B,H,N,d] (dtype):
 *   D = rowsum(dO o O), P = exp(scale*Q K^T - lse), dV = P^T dO,
 *   dP = dO V^T, dS = P o (dP - D), dQ = scale*dS K, dK = scale*dS^T Q.
 * P is recomputed from Q, K and lse rather than stored ("FlashAttention"
 * concept card, lukebest.github.io, "反向：重算而非存储"). dS is the softmax
 * Jacobian applied to dP: the softmax gradient printed in the cloud.baidu.com
 * explainer ("梯度计算优化") is dimensionally inconsistent, so the textbook
 * form above is used; D_i = rowsum(P o dP)_i equals rowsum(dO o O)_i.
 * workspace: device buffer of at least fa_bwd_workspace_size() bytes, 256-byte
 * aligned; its contents on entry do not matter and are overwritten.
 */
fa_status fa_bwd(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dout, void* dq, void* dk, void* dv, void* workspace, int B, int H, int N, int d,
                 float softmax_scale, int causal, cudaStream_t stream);

/*
 * fa_bwd without a workspace argument, for callers that cannot allocate device
 * memory (a host application that owns every byte of device memory and gives
 * this library no allocator, or a latency-critical loop where cudaMalloc is
 * not allowed). The pages describe no such variant; it has no counterpart
 * there. Arguments and results are those of fa_bwd (without block mask).
 * Scratch: a fixed array of FA_BWD_NOALLOC_SCRATCH_BYTES bytes in the
 * library's static device memory, held by every GPU that loads the library
 * until the process exits. If fa_bwd_workspace_size(B, H, N, d) exceeds it the
 * call returns FA_ERR_UNSUPPORTED and launches nothing. All calls on a device
 * share that array: calls whose kernels may overlap on the GPU race and must be
 * ordered by the caller. Nothing in it needs to start at zero: every call's
 * first kernel rewrites all the entries (D and lse in log2 units) its second
 * kernel reads. Every other limit is that of fa_bwd. The first call on a device
 * looks up the array's device address (cudaGetSymbolAddress) and caches it;
 * make that first call before any stream capture. Allocates nothing.
 */
#define FA_BWD_NOALLOC_SCRATCH_BYTES (32u << 20)
fa_status fa_bwd_noalloc(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv, int B, int H, int N,
                         int d, float softmax_scale, int causal, cudaStream_t stream);

/*
 * Block-sparse forward ("FlashAttention" concept card, "Block-Sparse
 * FlashAttention": a fixed block mask whose zero blocks are skipped).
 * block_mask: DEVICE pointer to uint8 [N/128][N/128], row-major, shared by all
 * (b, h); entry (I, J) != 0 lets query tile I (rows 128I..128I+127) attend to
 * key tile J. Zero tiles are never loaded. Composes with `causal` by AND.
 * Requires N % 128 == 0 and N/128 <= 2048 (else FA_ERR_UNSUPPORTED).
 */
fa_status fa_blocksparse_fwd(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse,
                             int B, int H, int N, int d, float softmax_scale, int causal,
                             const uint8_t* block_mask, cudaStream_t stream);

/* Block-sparse backward; arguments as fa_bwd plus block_mask as in fa_blocksparse_fwd. */
fa_status fa_blocksparse_bwd(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                             int B, int H, int N, int d, float softmax_scale, int causal,
                             const uint8_t* block_mask, cudaStream_t stream);

/*
 * Forward with Nq query rows and Nk key/value rows (a query block that is the
 * last Nq positions of a longer key sequence, cross-attention, decoding). The
 * pages treat the square case; this generalises the same computation:
 * q, o [B,H,Nq,d]; k, v [B,H,Nk,d]; lse [B,H,Nq]. The causal mask is
 * bottom-right aligned: query i attends to key j iff j <= i + Nk - Nq (for
 * Nq = Nk the rule j <= i). A query row with no key gets O = 0, lse = -inf.
 * block_mask may be NULL; otherwise it is a DEVICE uint8 [Nq/128][Nk/128] as
 * in fa_blocksparse_fwd and needs Nq, Nk multiples of 128 (at most 2048 tiles
 * each). With Nq = Nk this computes exactly what fa_fwd / fa_blocksparse_fwd do.
 * Errors, ownership and stream semantics as fa_fwd.
 */
fa_status fa_fwd_qk(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                    int Nq, int Nk, int d, float softmax_scale, int causal, const uint8_t* block_mask,
                    cudaStream_t stream);

/*
 * Backward of fa_fwd_qk: dq [B,H,Nq,d]; dk, dv [B,H,Nk,d]; o, dout [B,H,Nq,d];
 * workspace of at least fa_bwd_workspace_size(B, H, Nq, d) bytes (256-byte
 * aligned). Rows without keys contribute nothing. Otherwise as fa_bwd.
 */
fa_status fa_bwd_qk(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o, const float* lse,
                    const void* dout, void* dq, void* dk, void* dv, void* workspace, int B, int H, int Nq, int Nk,
                    int d, float softmax_scale, int causal, const uint8_t* block_mask, cudaStream_t stream);

/*
 * Split-KV forward (FlashDecoding, the "FlashAttention" concept card's lineage
 * table: partial softmax per key range, then a synchronising merge). Computes
 * exactly what fa_fwd_qk computes, with more parallelism when B*H*ceil(Nq/128)
 * is small next to the GPU (decoding: a few query rows against a long key
 * sequence). The Nk keys are cut into n_splits consecutive ranges of whole
 * 128-key tiles: range s holds key tiles [s*T/n_splits, (s+1)*T/n_splits),
 * T = ceil(Nk/128). Step 1 computes, for every query row and range, the
 * softmax-weighted mean of that range's values, O_s (fp32), and the log of its
 * exp-sum, lse_s (fp32, -inf if the row has no allowed key in the range); step 2
 * merges them: lse = log sum_s exp(lse_s), O = sum_s exp(lse_s - lse) O_s (the
 * online-softmax update of the interview explainer, section 3.2, applied to
 * whole ranges).
 * Arguments as fa_fwd_qk (q, o [B,H,Nq,d]; k, v [B,H,Nk,d]; lse [B,H,Nq];
 * bottom-right causal; optional block_mask [Nq/128][Nk/128]), plus:
 *   n_splits  1 <= n_splits <= ceil(Nk/128) (else FA_ERR_INVALID_ARG);
 *             fa_fwd_splitkv_splits() suggests one.
 *   workspace DEVICE buffer of fa_fwd_splitkv_workspace_size() bytes, 256-byte
 *             aligned, owned by the caller; on return (after the stream
 *             completes) it holds the partials: O_s as fp32
 *             [n_splits][B*H][Nq][d] at offset 0, then lse_s as fp32
 *             [n_splits][B*H][Nq] at the next 256-byte boundary after O_s.
 * Two launches on `stream`; asynchronous, allocates nothing. With Nq <= 4
 * (decoding) step 1 runs on the CUDA cores, which read each range's K and V
 * once; larger Nq use the tensor-core forward. The partials are the same.
 */
size_t fa_fwd_splitkv_workspace_size(int B, int H, int Nq, int d, int n_splits);
int fa_fwd_splitkv_splits(int B, int H, int Nq, int Nk);
fa_status fa_fwd_splitkv(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int Nq, int Nk, int d, float softmax_scale, int causal, const uint8_t* block_mask,
                         int n_splits, void* workspace, cudaStream_t stream);

/*
 * Attention with dropout on the probabilities, fused in the same kernels
 * ("FlashAttention" concept card, 算法要点 "Kernel fusion": QK^T -> softmax
 * (+ mask / dropout) -> PV). O = (P o Z) V, with P the softmax of the scaled,
 * masked scores (lse is that of P) and Z the dropout keep decisions: element
 * (i, j) of head bh = b*H + h is kept iff its draw u >= t, t = floor(256 p + 1/2),
 * and a kept entry is 256 / (256 - t) (so p is used rounded to t/256). The
 * draws come from Philox4x32-10 (Salmon et al., SC'11): one block per 4 x 4
 * block of (query row, key), counter (j >> 2, i >> 2, bh, 0), key (seed low
 * 32 bits, seed high 32 bits); output word (i & 3) holds row i's draws, byte
 * (j & 3) of it, least significant first, is u. The backward draws them again
 * from the same seed (nothing is stored) and computes, through O = (P o Z) V:
 * dV = (P o Z)^T dO, dP = (dO V^T) o Z, dS = P o (dP - D) with
 * D = rowsum(dO o O), dQ = scale dS K, dK = scale dS^T Q.
 * Arguments as fa_fwd_qk / fa_bwd_qk, plus p_drop in [0, 1) (else
 * FA_ERR_INVALID_ARG; p_drop = 0 is exactly fa_fwd_qk / fa_bwd_qk) and the
 * 64-bit seed; fa_bwd_dropout must get the forward's p_drop and seed.
 */
fa_status fa_fwd_dropout(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int Nq, int Nk, int d, float softmax_scale, int causal, const uint8_t* block_mask,
                         float p_drop, unsigned long long seed, cudaStream_t stream);
fa_status fa_bwd_dropout(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dout, void* dq, void* dk, void* dv, void* workspace, int B, int H, int Nq, int Nk,
                         int d, float softmax_scale, int causal, const uint8_t* block_mask, float p_drop,
                         unsigned long long seed, cudaStream_t stream);

/*
 * 8-bit forward (the FP8 variant the "FlashAttention" concept card's lineage
 * table lists for FlashAttention-3). q8 [B,H,Nq,128], k8 and v8 [B,H,Nk,128]
 * are DEVICE arrays of e4m3 values (1 sign, 4 exponent bits with bias 7, 3
 * mantissa bits; one byte each); the tensors attended are q_scale * q8,
 * k_scale * k8, v_scale * v8 (per-tensor scales > 0). Writes O [B,H,Nq,128] as
 * bf16 and lse [B,H,Nq] (fp32) of exact attention on those tensors, with the
 * masks of fa_fwd_qk (bottom-right causal, optional block_mask). S = Q K^T runs
 * on the stored e4m3 values (kind::f8f6f4 MMAs, fp32 accumulation; the scales
 * join the softmax scale); V is widened to bf16 on chip and P V runs in bf16.
 * d must be 128 (else FA_ERR_UNSUPPORTED); scales must be finite and > 0 (else
 * FA_ERR_INVALID_ARG). Otherwise as fa_fwd_qk.
 */
fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* v8, float q_scale, float k_scale, float v_scale,
                     void* o, float* lse, int B, int H, int Nq, int Nk, int d, float softmax_scale, int causal,
                     const uint8_t* block_mask, cudaStream_t stream);

/*
 * ---------------------------------------------------------------- paged cache
 * Serving over a key/value cache kept in pages: fa_cache_plan hands out pages and
 * builds the slot map of a step's new rows, fa_rope_append rotates q and k and
 * writes k and v to their slots, fa_tree_fwd attends over the pages, and
 * fa_cache_commit moves the rows of an accepted draft to the front. The batch is
 * ragged and packed: request b owns rows cu[b] .. cu[b+1]-1 of the [rows][heads][d]
 * tensors. All lengths, tables and maps live on the device, so a step can be
 * captured in a CUDA graph and replayed with other lengths (make the first call of
 * each kind on a device before any capture). Outputs must not overlap inputs, or one
 * another, except where a comment says so. Offsets into caches and tensors are 64-bit.
 */

/*
 * A paged cache. Row r of page p, head h starts at element
 * p*page_stride + h*head_stride + r*row_stride of k and of v (so pages laid out
 * [head][row][d] or [row][head][d], and one layer of a larger pool, are all
 * reachable). k, v: DEVICE, 16-byte aligned; the strides are multiples of 8
 * elements, at least d; page_size is a power of two, 8..1024; d as for the forward
 * entry points; num_pages * page_size <= 2^31 - 1.
 */
typedef struct {
  void* k;
  void* v;
  fa_dtype dtype;
  int num_pages, page_size, H_kv, d;
  long long page_stride, head_stride, row_stride;
} fa_kv_cache;

/*
 * Packed rows [rows][heads][d]: head h of row t starts at element
 * t*row_stride + h*head_stride; its d elements are contiguous. DEVICE, 16-byte
 * aligned, strides multiples of 8 elements (a slice of a fused projection is
 * fine; an input's may be 0 where rows or heads are shared, an output's are at
 * least d where there is more than one).
 */
typedef struct {
  void* data;
  long long row_stride, head_stride;
} fa_rows;

/*
 * Pages, slot map, positions and tree masks of a step, from the requests'
 * lengths. Request b holds ctx_len[b] cached rows and adds n_b = cu_new[b+1] -
 * cu_new[b] new ones; it then needs ceil((ctx_len[b] + n_b) / page_size) pages.
 *   1. Requests that hold more give the rest back: their last pages are pushed on
 *      the free list, in the order of the requests, and the table entries set to -1
 *      (a request with no rows at all gives back everything).
 *   2. Requests that need more take them from the end of the free list, in the order
 *      of the requests. Request b is granted iff it needs none, or the needs of
 *      requests 0..b together do not exceed the free pages. A request whose
 *      ctx_len is negative, whose n_b is negative or over max_new, whose new rows do
 *      not all lie in 0 .. rows-1, or which needs more than max_pages pages, takes no
 *      part and is refused.
 *   3. Granted: n_pages[b] and block_table row b are updated and seq_len[b] =
 *      ctx_len[b] + n_b. Refused: pages and table stay, seq_len[b] = 0.
 *   4. slot[cu_new[b] + i] = row ctx_len[b] + i as page * page_size + row in page, -1
 *      if b was refused; position[cu_new[b] + i] = ctx_len[b] + i, or with `parent`
 *      ctx_len[b] + the token's depth in its tree. Rows of no request (from
 *      cu_new[B] to `rows`) get slot -1 and position 0.
 *   5. With `parent` (request-local index of each new token's parent, -1 for a child
 *      of the cached context; an entry outside [-1, i) counts as -1), tree_mask
 *      [rows][ceil(max_new/64)] gets each token's branch: bit j of the row (word
 *      j / 64, bit j % 64) is set iff new token j of the request is the token
 *      itself or one of its ancestors. Rows of no request keep theirs.
 * block_table int32 [B][max_pages]; n_pages int32 [B] (pages held); free_list int32
 * [num_pages], of which the first *free_count are free; ctx_len, seq_len [B]; cu_new
 * [B+1]; slot, position, parent [rows], all int32 on the DEVICE. block_table,
 * n_pages, free_list and free_count are the cache's state and updated in place:
 * calls on one cache must be ordered. cu_new must not fall: the requests before and
 * behind a negative n_b would claim the same rows, of which each gets one slot. parent
 * and tree_mask are both given or both NULL. 1 <= B <= 4096, 0 <= rows, 1 <= max_new
 * (with parent: <= 512, else FA_ERR_UNSUPPORTED). One launch.
 */
#define FA_TREE_MAX 512
fa_status fa_cache_plan(int B, int rows, int max_new, int page_size, int num_pages, int max_pages,
                        const int32_t* ctx_len, const int32_t* cu_new, const int32_t* parent, int32_t* block_table,
                        int32_t* n_pages, int32_t* free_list, int32_t* free_count, int32_t* seq_len, int32_t* slot,
                        int32_t* position, uint64_t* tree_mask, cudaStream_t stream);

/*
 * Rotary positions over several axes. Of each row x the first rot elements are
 * rotated in pairs and the rest copied: pair i of token (b, n) turns by the angle
 *   positions[axis[i]][b][n] * inv_freq[i]
 * (the caller's tables choose the frequencies and which pairs belong to time,
 * height or width; one axis is ordinary rotary), (x, y) -> (x cos - y sin,
 * x sin + y cos). Pair i is elements (i, i + rot/2), or (2i, 2i+1) with pairs != 0.
 * inverse != 0 turns back: the rotation is orthogonal, so this is also its
 * gradient. Angles are reduced in 64 bits, so far positions lose nothing.
 * x, out [B, H, N, d] with element strides of b, h and n (multiples of 8; the d
 * elements contiguous; 16-byte aligned; those of out at least d where there is more
 * than one); out may be x itself, but must not overlap it in another way. positions
 * int32 [n_axes][B][N] with element strides of axis and b (0: shared by the batch);
 * inv_freq fp32 [rot/2]; axis uint8 [rot/2], an entry >= n_axes leaves its pair
 * unturned. rot a multiple of 16, 16..d; 1 <= n_axes <= 8; d as for the forward entry
 * points.
 */
fa_status fa_rope(fa_dtype dtype, const void* x, void* out, int B, int H, int N, int d, const long long x_strides[3],
                  const long long out_strides[3], const int32_t* positions, long long pos_axis_stride,
                  long long pos_b_stride, int n_axes, const float* inv_freq, const uint8_t* axis, int rot, int inverse,
                  int pairs, cudaStream_t stream);

/*
 * The same rotation of a step's new q and k, with k and v written to the cache:
 * q -> q_out [rows][Hq][d], k and v [rows][H_kv][d] -> row slot[t] of the cache (page
 * slot / page_size, row slot % page_size). A slot outside the cache (-1) writes
 * nothing; two rows with one slot leave pieces of both. positions int32 [n_axes][rows]
 * with an axis stride. q and q_out may both be NULL (k and v only) and q_out may be q.
 * rot = 0 rotates nothing (positions, inv_freq, axis are not read). One launch.
 */
fa_status fa_rope_append(const fa_kv_cache* cache, int rows, int Hq, const fa_rows* q, const fa_rows* k,
                         const fa_rows* v, const fa_rows* q_out, const int32_t* slot, const int32_t* positions,
                         long long pos_axis_stride, int n_axes, const float* inv_freq, const uint8_t* axis, int rot,
                         int pairs, cudaStream_t stream);

/*
 * Attention of a step's new rows over the paged cache, exact as fa_fwd_qk is.
 * Request b's rows are q rows cu_q[b] .. cu_q[b+1]-1 (n_b of them, at most max_q) and
 * its keys the first seq_len[b] rows of its pages; the last n_b keys are its own new
 * tokens, already written. Head h reads cache head h / (Hq / H_kv). Row i sees key j
 * iff j < seq_len[b] and
 *   tree_mask NULL:  j <= i + seq_len[b] - n_b     (a chain: decoding, prompt chunks)
 *   otherwise:       j < seq_len[b] - n_b, or bit j - (seq_len[b] - n_b) of the row's
 *                    tree_mask [rows][ceil(max_q/64)] is set (a drafted tree).
 * Keys on a page index outside [0, num_pages) are not seen. A row that sees no key
 * gets O = 0, lse = -inf. o [rows][Hq][d]; lse fp32 [rows][Hq], natural log as
 * fa_fwd. Rows of no request stay as they were. Where cu_q goes beyond `rows`, the
 * rows there are computed, in their places, and the others are not. What the cache holds behind
 * seq_len[b] is never used, whatever it is; K and V of a request's own keys that some
 * row does not see must be finite in V (P = 0 there multiplies them).
 * block_table int32 [B][max_pages]. Hq a multiple of H_kv; 1 <= B <= 4096; max_q >= 1,
 * with tree_mask <= FA_TREE_MAX. workspace: DEVICE, 256-byte aligned,
 * fa_tree_fwd_workspace_size() bytes, contents irrelevant; calls that may overlap need
 * one each. softmax_scale finite. o must not overlap q. One launch or (units of rows cut
 * among CTAs, see fa_tree.cuh) two. The results do not depend on the order in which CTAs
 * run: equal arguments give equal bits.
 */
size_t fa_tree_fwd_workspace_size(int B, int rows, int max_q, int Hq, int H_kv, int d);
fa_status fa_tree_fwd(const fa_kv_cache* cache, const fa_rows* q, const fa_rows* o, float* lse, int B, int rows,
                      int max_q, int Hq, int max_pages, const int32_t* block_table, const int32_t* cu_q,
                      const int32_t* seq_len, const uint64_t* tree_mask, float softmax_scale, void* workspace,
                      cudaStream_t stream);

/*
 * Keeps the accepted path of each request's draft: row ctx_len[b] + accepted[b][j] of
 * the cache moves to row ctx_len[b] + j, for j < n_accepted[b], and new_len[b] =
 * ctx_len[b] + the rows kept (a request that fa_cache_plan refused accepts none: its
 * n_accepted has to be 0, since nothing was written). accepted int32 [B][max_accept]
 * holds request-local indices of new tokens, strictly increasing (a path from the root
 * is); the path ends before the first entry that is not larger than the one before (or
 * is negative), or whose row has no page in the table. new_len may be ctx_len. DEVICE
 * pointers; ctx_len, n_accepted, new_len int32 [B]. One launch.
 */
fa_status fa_cache_commit(const fa_kv_cache* cache, int B, int max_pages, int max_accept, const int32_t* block_table,
                          const int32_t* ctx_len, const int32_t* accepted, const int32_t* n_accepted,
                          int32_t* new_len, cudaStream_t stream);

/*
 * Debug: the dropout draws u (uint8) of every (head, query row, key) for
 * B*H heads, Nq query rows, Nk keys, written to two DEVICE buffers of
 * B*H*Nq*Nk bytes, [bh][i][j]: row_major through the generator path of the
 * forward and query-stationary backward (a thread per query row), col_major
 * through that of the key-stationary backward (a thread per key). Both equal
 * the layout described at fa_fwd_dropout.
 */
fa_status fa_debug_dropout_draws(int B, int H, int Nq, int Nk, unsigned long long seed, uint8_t* row_major,
                                 uint8_t* col_major, cudaStream_t stream);

/*
 * Debug: the forward / backward with a record of the tiles each CTA loaded.
 * trace: DEVICE int32 buffer of fa_*_trace_size() entries; each record is a
 * count followed by entries (tile index) | (flags << 16).
 * Forward: T_kv = ceil(N/128) key tiles; CTA c covers query tiles 2p and 2p+1
 * (p = c % n_pairs, n_pairs = ceil(T_kv/2)) of head c / n_pairs; its record of
 * T_kv + 1 entries starts at c * (T_kv + 1); flags bit q = the key tile is used
 * by query tile 2p+q.
 * Backward: key-stationary CTA (head h, key tile j) lists the query tiles of
 * fa_bwd_row_tile(d) rows it visits, record of T_q + 1 entries at
 * (h * T_kv + j) * (T_q + 1), T_q = ceil(N / fa_bwd_row_tile(d)); after all of
 * those, query-stationary CTA (head h, 128-row query tile i) lists the key
 * tiles it visits, record of T_kv + 1 entries at
 * B*H*T_kv*(T_q + 1) + (h * T_kv + i) * (T_kv + 1). Backward flags = 1.
 */
size_t fa_fwd_trace_size(int B, int H, int N);
size_t fa_bwd_trace_size(int B, int H, int N, int d);
int fa_bwd_row_tile(int d);
fa_status fa_debug_fwd_trace(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse,
                             int B, int H, int N, int d, float softmax_scale, int causal,
                             const uint8_t* block_mask, int32_t* trace, cudaStream_t stream);
fa_status fa_debug_bwd_trace(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                             int B, int H, int N, int d, float softmax_scale, int causal,
                             const uint8_t* block_mask, int32_t* trace, cudaStream_t stream);

/*
 * Debug: one of the two launches fa_bwd makes, selected by `phase`:
 * 0 = prep (D = rowsum(dO o O) and lse in log2 units, into the workspace),
 * 1 = main (recompute P; dK, dV by key tile and dQ by query tile, all
 * accumulated in TMEM). Running phases 0 and 1 in order on one stream with the
 * same arguments is exactly fa_bwd. Used to time the main kernel on its own.
 */
fa_status fa_debug_bwd_phase(int phase, fa_dtype dtype, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                             void* workspace, int B, int H, int N, int d, float softmax_scale, int causal,
                             const uint8_t* block_mask, cudaStream_t stream);

/*
 * Device status: synchronises `stream`, returns the status word that kernels
 * set when a device-side wait timed out (FA_OK if none), and clears it.
 */
fa_status fa_device_status(cudaStream_t stream);

/*
 * Debug: launches one CTA that waits on a barrier nothing will complete, with
 * a time limit of `timeout_ms`; the wait gives up, records FA_ERR_TIMEOUT in
 * the status word and the CTA exits normally. Used to test the time-out path.
 */
fa_status fa_debug_timeout_probe(int timeout_ms, cudaStream_t stream);

/*
 * Debug: the real forward kernel with its TMA producer issuing no load at all
 * and every device-side wait limited to `timeout_ms` (1..5000). The MMA
 * issuer's first wait (for Q) runs out, records FA_ERR_TIMEOUT in the status
 * word and raises the CTA's abort flag; every role then leaves its loop, and,
 * as nothing was issued, nothing is in flight when the CTAs exit. o and lse
 * are not written. Used to test the abort path of the production kernel
 * without a fault. Arguments otherwise as fa_fwd.
 */
fa_status fa_debug_fwd_withhold(fa_dtype dtype, const void* q, const void* k, const void* v, void* o, float* lse,
                                int B, int H, int N, int d, float softmax_scale, int causal, int timeout_ms,
                                cudaStream_t stream);

/*
 * Debug: fa_bwd with the main kernel's TMA producers issuing no load and every
 * device-side wait limited to `timeout_ms` (1..5000): the MMA issuers' first
 * waits run out (key-stationary CTAs: K/V; query-stationary CTAs: their first
 * K), record FA_ERR_TIMEOUT and raise the CTA's abort flag; every role leaves
 * its loop, the issuers wait for what they issued, and the CTAs exit. The prep
 * launch runs normally. dq, dk, dv are not written. Arguments otherwise as
 * fa_bwd.
 */
fa_status fa_debug_bwd_withhold(fa_dtype dtype, const void* q, const void* k, const void* v, const void* o,
                                const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                int B, int H, int N, int d, float softmax_scale, int causal, int timeout_ms,
                                cudaStream_t stream);

/*
 * Debug: fa_tree_fwd with producers that issue no load and every device-side wait
 * limited to `timeout_ms` (1..5000): the MMA warps' first waits (for K) run out,
 * record FA_ERR_TIMEOUT and raise the CTA's abort flag; the softmax warps then go
 * through their remaining steps without waiting, and the CTAs exit. What o and lse
 * hold for rows with keys is meaningless. Arguments otherwise as fa_tree_fwd.
 */
fa_status fa_debug_tree_withhold(const fa_kv_cache* cache, const fa_rows* q, const fa_rows* o, float* lse, int B,
                                 int rows, int max_q, int Hq, int max_pages, const int32_t* block_table,
                                 const int32_t* cu_q, const int32_t* seq_len, const uint64_t* tree_mask,
                                 float softmax_scale, void* workspace, int timeout_ms, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
