/*
 * packattn_block.h -- C ABI of what stands around and inside the packed attention in a DiT block
 * (same library as packattn.h, whose status codes, conventions and pa_get_error it shares):
 *
 *   pa_block_norm_fwd / _bwd         gated residual join with the norm behind a block and the norm in
 *                                    front of the next
 *   pa_rope_axes / pa_qkv_rope_axes_fwd
 *                                    rotary positions with several axes (time, height, width)
 *   pa_block_select, pa_block_sparse_attn_fwd / _bwd
 *                                    attention over the key blocks that a cheap score selects
 *
 * Unlike packattn.h's entry points these take their scratch memory from the caller, so that two captured
 * graphs, or two streams, that use different buffers never share one; the library itself holds only the
 * status word of the (device, stream) pair.  None of them synchronises or allocates on the device after
 * the first call on a stream, each may be captured into a CUDA graph, and each leaves the calling
 * thread's current device as it was.  Device-side errors go to the status word of the stream that the call
 * was made on (for a captured call: the capturing stream), to be read with pa_get_error.  After
 * pa_release_workspace, graphs captured before must not be replayed (they hold that word's address).
 */
#ifndef PACKATTN_BLOCK_H_
#define PACKATTN_BLOCK_H_

#include "packattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further status codes (see enum pa_status). */
enum pa_block_status {
  PA_ERR_WORKSPACE = -12, /* the workspace is NULL, misaligned or too small */
  PA_ERR_BLOCKS = -13,    /* a list of key blocks is not increasing, leaves its segment, or is too long */
  PA_ERR_MODE = -14       /* a norm kind, or a combination of given and missing buffers, that the call does not have */
};

enum pa_norm_kind {
  PA_NORM_NONE = 0,
  PA_NORM_LAYER = 1, /* (v - mean) / sqrt(mean((v - mean)^2) + eps) over the channels */
  PA_NORM_RMS = 2    /* v / sqrt(mean(v^2) + eps) */
};

/*
 * The join between two blocks of a packed stream x [total_tokens, hidden], with s the segment (image) of a
 * token:
 *     u = N_post(y) * w_post                          (the block's output y behind its norm)
 *     r = residual_scale * x + gate[s] * u            (stored in the residual's type)
 *     z = N_pre(r) * w_pre * (1 + scale[s]) + shift[s]   (the next block's input)
 * N_pre is taken of r as it is stored.  A NULL gate, weight or scale counts as 1 (scale: as 0), a NULL shift
 * as 0.  Statistics, sums and products are fp32; r and z are rounded once each.
 *
 *   total_tokens, batch, cu_seqlens   the pack, as for pa_varlen_attn_fwd; cu_seqlens is read (and may only
 *                     be NULL if it is not) when gate, scale or shift is given.
 *   hidden            channels, a multiple of 8, 8 .. 8192.
 *   residual_fp32     type of x, r, dr, dx: 1 fp32, 0 bf16.  y, z, dy, dz are bf16.
 *   param_fp32        type of gate, scale, shift, w_post, w_pre: 1 fp32, 0 bf16.
 *   post, pre         enum pa_norm_kind of N_post and N_pre.
 *   gate_stride, scale_stride, shift_stride   elements from one segment's row of [batch, hidden] to the next
 *                     (slices of one projection's output; 0: one row for all); rows 16-byte aligned.
 * Every buffer is 16-byte aligned (cu_seqlens 4-byte), on one device, and token rows are contiguous.
 */
typedef struct pa_block_norm_desc {
  int32_t total_tokens, batch, hidden;
  int32_t residual_fp32, param_fp32;
  int32_t post, pre;
  float residual_scale, eps;
  const int32_t* cu_seqlens;
  const void* gate;
  const void* scale;
  const void* shift;
  int64_t gate_stride, scale_stride, shift_stride;
  const void* w_post;
  const void* w_pre;
} pa_block_norm_desc;

/*
 * pa_block_norm_fwd -- enqueue the join on `stream`.
 *   y NULL: no join, z is the norm of x; then r is NULL, residual_scale 1, post NONE, and w_post and gate NULL.
 *   z NULL: no norm in front; then pre is NONE, and w_pre, scale and shift NULL.  pre NONE needs z NULL.
 *   r may be x (in place).  No other buffers overlap.
 * Errors the host sees: PA_ERR_NULL, PA_ERR_SHAPE (sizes), PA_ERR_ALIGN, PA_ERR_SCALE (residual_scale or eps
 * not finite, eps < 0), PA_ERR_MODE, PA_ERR_NOT_DEVICE.  Bad cu_seqlens: PA_ERR_CU_SEQLENS in the status word.
 * Bitwise deterministic.
 */
PA_API int pa_block_norm_fwd(const pa_block_norm_desc* desc, const void* x, const void* y, void* r, void* z,
                             void* stream);

/*
 * pa_block_norm_bwd -- enqueue the gradients of the join: from dr = dL/dr (the later uses of r; NULL counts
 * as 0) and dz = dL/dz, with dr' = dr + the norm's gradient,
 *     dx = residual_scale * dr',  dy = N_post's gradient of gate[s] * w_post * dr',
 *     dgate[s] = sum over s's tokens of dr' u,  dscale[s] = sum of dz N_pre(r) w_pre,  dshift[s] = sum of dz,
 *     dw_post = sum over all tokens of dr' gate N_post(y),  dw_pre = sum of dz (1 + scale) N_pre(r).
 *   r            as the forward stored it (x when y is NULL).
 *   dz           NULL exactly when pre is NONE; with dz NULL, dr and y are given.
 *   dx           may be dr (in place).       dy   NULL exactly when y is.
 *   dgate, dscale, dshift   fp32 [batch, hidden], NULL if not wanted; a segment without tokens gets 0 (its rows of
 *                gate, scale and shift have no effect on anything, whatever they hold).
 *   dw_post, dw_pre         fp32 [hidden], NULL if not wanted.
 *     A gradient of something that was not given (a NULL gate, ...) must be NULL: PA_ERR_MODE.
 *   workspace    pa_block_norm_workspace_bytes(batch, total_tokens, hidden) bytes, 16-byte aligned; only read
 *                (and may only be NULL if it is not) when one of the five sums is wanted.
 * Column sums are added in a fixed order: bitwise deterministic.
 */
PA_API int64_t pa_block_norm_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t hidden);
PA_API int pa_block_norm_bwd(const pa_block_norm_desc* desc, const void* r, const void* y, const void* dr,
                             const void* dz, void* dx, void* dy, float* dgate, float* dscale, float* dshift,
                             float* dw_post, float* dw_pre, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Rotary positions with several axes.  The d/2 rotated pairs of a head are shared out over the axes:
 * axis a has dims[a] channels, that is dims[a]/2 pairs, in order; pair i of axis a turns by the angle
 *     pos[t, a] * theta[a]^(-2 i / dims[a]).
 * Pair p of the head is (x_p, x_{p + d/2}), or (x_{2p}, x_{2p+1}) when interleaved; pairs past the axes' total
 * (sum of dims < head_dim) are left as they are.  Angles are formed and reduced in fp64.
 *
 *   axes        1 .. 4;  dims, theta: host arrays of that length; dims even, >= 2, sum <= head_dim; theta > 0.
 *   pos         device, fp32, [total_tokens, axes], contiguous, 4-byte aligned (any position, fractions too).
 *   interleaved 0 or 1.
 */
typedef struct pa_rope_axes_desc {
  int32_t axes;
  int32_t dims[4];
  double theta[4];
  int32_t interleaved;
} pa_rope_axes_desc;

/*
 * pa_rope_axes -- rotate q and k [total_tokens, heads, head_dim] (bf16, contiguous, 16-byte aligned) on `stream`.
 *   inverse     0: the rotation; 1: its inverse, which is also its gradient (dq, dk in, gradients out).
 *   q_out, k_out may be q and k (in place); each rounded once.  k and k_out may both be NULL (q alone).
 *   heads * head_dim below 2^19.  A position that is not finite makes its own axis' pairs NaN.
 */
PA_API int pa_rope_axes(const void* q, const void* k, const float* pos, int32_t total_tokens, int32_t heads,
                        int32_t head_dim, const pa_rope_axes_desc* rope, int32_t inverse, void* q_out, void* k_out,
                        void* stream);

/*
 * pa_qkv_rope_axes_fwd -- pa_qkv_rope_fwd's projection with these positions: qkv = x W_qkv^T, q and k rotated
 * in the GEMM's epilogue (fp32 accumulators), q, k, v rounded once.  Arguments as there.
 *   workspace   pa_rope_axes_workspace_bytes(total_tokens, head_dim) bytes, 16-byte aligned: the (cos, sin) of
 *               every token and pair.
 */
PA_API int64_t pa_rope_axes_workspace_bytes(int32_t total_tokens, int32_t head_dim);
PA_API int pa_qkv_rope_axes_fwd(const void* x, const void* w_qkv, const float* pos, int32_t total_tokens,
                                int32_t hidden, int32_t heads, int32_t head_dim, const pa_rope_axes_desc* rope,
                                void* q, void* k, void* v, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Block-sparse packed attention (SparseAttn page, sections 3.1-3.4: a softmax restricted to a kept set of
 * keys).  Every segment is cut into blocks of 128 tokens from its first token on (the last one shorter); a
 * block of queries sees the key blocks of its own segment that its list names.
 *
 * pa_block_rows -- rows of the list tables of a pack: total_tokens / 128 + batch (-1 if an argument is
 * negative).  Block b of segment s is row cu_seqlens[s] / 128 + s + b (integer division).
 *
 *   idx   device, int32, [heads, pa_block_rows, width]: key blocks of the row's segment, increasing.
 *   cnt   device, int32, [heads, pa_block_rows]: entries of the row's list, 0 .. width.  Entries past cnt, and
 *         rows that are no block, are not read.
 * heads * head_dim is below 2^23, and a table has at most 2^40 entries.  Keys of a block that no list of a row
 * names, other images' tokens and what lies behind a segment's last token have no influence on the row, whatever
 * they hold (infinities, NaN).
 */
PA_API int64_t pa_block_rows(int32_t batch, int32_t total_tokens);

/*
 * pa_block_select -- write idx and cnt: for each head and query block of a segment of nb blocks, the
 *     min(nb, max(min_blocks, ceil(density * nb)))
 * key blocks whose mean key has the largest inner product with the block's mean query, in increasing order
 * (means and products in fp64, in a fixed order of additions; scores that come out equal: the lower block first; a
 * NaN score ranks last, as -infinity).
 * Unused entries are -1, rows that are no block have cnt 0.
 *   q, k          as for pa_varlen_attn_fwd.     max_seqlen  an upper bound of every segment, <= 262144.
 *   density       0 .. 1 (fp64).                 min_blocks  >= 1.
 *   width         at least the formula's value at nb = ceil(max_seqlen / 128), else PA_ERR_BLOCKS at once.
 *   workspace     pa_block_select_workspace_bytes(...) bytes, 16-byte aligned.
 */
PA_API int64_t pa_block_select_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t heads, int32_t head_dim);
PA_API int pa_block_select(const void* q, const void* k, const int32_t* cu_seqlens, int32_t batch,
                           int32_t total_tokens, int32_t heads, int32_t head_dim, int32_t max_seqlen, double density,
                           int32_t min_blocks, int32_t width, int32_t* idx, int32_t* cnt, void* workspace,
                           int64_t workspace_bytes, void* stream);

/*
 * pa_block_sparse_attn_fwd -- pa_varlen_attn_fwd restricted to the listed blocks (from pa_block_select or the
 * caller's own pattern).  A row with an empty list gets out = 0 and lse = -infinity.  A list that is not
 * increasing, names a block outside its segment, or has cnt outside 0 .. width is recorded as PA_ERR_BLOCKS in
 * the status word, and out and lse are then undefined.
 *   workspace     pa_block_sparse_workspace_bytes(..., backward = 0) bytes, 16-byte aligned.
 * Bitwise deterministic.
 */
PA_API int64_t pa_block_sparse_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t heads, int32_t head_dim,
                                               int32_t max_seqlen, int32_t width, int32_t backward);
PA_API int pa_block_sparse_attn_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                    int32_t batch, int32_t total_tokens, int32_t heads, int32_t head_dim,
                                    int32_t max_seqlen, const int32_t* idx, const int32_t* cnt, int32_t width,
                                    float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                    void* stream);

/*
 * pa_block_sparse_attn_bwd -- its gradients (the lists are constants), arguments as for pa_varlen_attn_bwd and
 * above; workspace with backward = 1.  A key block that no list names gets dk = dv = 0, a query with an empty
 * list dq = 0.  dq sums fp32 partials of different key blocks in whatever order they arrive (its last bits may
 * differ from run to run); dk and dv sum over query blocks in increasing order.
 */
PA_API int pa_block_sparse_attn_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                    const void* dout, const int32_t* cu_seqlens, int32_t batch, int32_t total_tokens,
                                    int32_t heads, int32_t head_dim, int32_t max_seqlen, const int32_t* idx,
                                    const int32_t* cnt, int32_t width, float scale, void* dq, void* dk, void* dv,
                                    void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PACKATTN_BLOCK_H_ */
