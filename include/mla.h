/*
 * mla.h - C ABI of the GB300 (sm_103a) absorbed, NoPE, causal Gated MLA forward.
 *
 * The method is the one on the course-notes page "Gated MLA（矩阵吸收版）"
 * (Gated MLA with matrix absorption): keys and values are never decompressed;
 * each head's query is absorbed into the latent space, q_abs = q . W_UK,
 * scored directly against the shared rank-r latent c, softmax-weighted sums
 * are taken over c itself, and only then are they up-projected by W_UV^T and
 * gated by sigmoid(W_g x) (section "完整计算流（四步）", steps 2-4; shapes from
 * the symbol-table page "符号表", table "MLA 变量").
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    never allocates, frees or retains them past the call.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream).  Nothing is launched when a status other than MLA_OK is returned.
 *  - Layouts are dense row-major (C order) with the shapes given; all float
 *    tensors of one call share one dtype; accumulation is fp32; `out` has the
 *    input dtype.
 *  - Arguments are validated on the host before any launch.  Errors raised on
 *    the device (a bounded wait that gave up) are recorded in a per-device
 *    error word read by mla_get_device_error().
 *  - There is no CPU fallback and no silent slow path: a shape outside the
 *    supported set returns MLA_ERR_UNSUPPORTED.
 */
#ifndef MLA_GB300_H
#define MLA_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(_WIN32)
#define MLA_API
#else
#define MLA_API __attribute__((visibility("default")))
#endif

/* Element types. */
typedef enum {
    MLA_DTYPE_BF16 = 0, /* bfloat16 inputs and output, fp32 accumulation */
    MLA_DTYPE_F32 = 1   /* fp32 inputs and output, fp32 FMA (no TF32)    */
} mla_dtype_t;

/* Status codes (0 = success, negative = error). */
typedef enum {
    MLA_OK = 0,
    MLA_ERR_NULL = -1,           /* a required pointer is NULL                       */
    MLA_ERR_SHAPE = -2,          /* a size is negative, zero where it may not be, or overflows */
    MLA_ERR_DTYPE = -3,          /* unknown dtype                                   */
    MLA_ERR_ALIGN = -4,          /* a pointer or stride is not 16-byte aligned      */
    MLA_ERR_WORKSPACE = -5,      /* workspace missing or smaller than required      */
    MLA_ERR_UNSUPPORTED = -6,    /* valid shape that no kernel of this build serves  */
    MLA_ERR_CUDA = -7,           /* a CUDA runtime/driver call failed               */
    MLA_ERR_DEVICE_TIMEOUT = -8, /* a bounded device-side wait gave up              */
    MLA_ERR_DEVICE_BOUNDS = -9   /* a device-side bounds check rejected an index    */
} mla_status_t;

/*
 * mla_absorbed_attn_fwd - causal prefill of the absorbed Gated MLA.
 * mla_absorbed_attn_fwd_workspace_size - bytes of workspace it needs for these
 * sizes (0 when none; also 0 for invalid or unsupported sizes).
 *
 * Page "Gated MLA（矩阵吸收版）", section "完整计算流（四步）":
 *   step 2  q_abs[b,t,h,:] = q[b,t,h,:] . W_UK[h]                  [B,T,H,r]
 *           score[b,h,t,u] = scale * q_abs[b,t,h,:] . c[b,u,:]     (u <= t)
 *           attn = softmax over u of the causally masked score
 *   step 3  o_lat[b,h,t,:] = sum_u attn[b,h,t,u] * c[b,u,:]        [B,H,T,r]
 *           o[b,h,t,v]     = o_lat[b,h,t,:] . W_UV[h,v,:]
 *   step 4  out[b,t,h*d_v+v] = sigmoid(gate[b,t,h*d_v+v]) * o[b,h,t,v]
 * The output projection W_o of step 4 is not part of this call.
 *
 * Arguments (shapes in elements, dense row-major):
 *   q     [B,T,H,d_q]   queries (the step-1 low-rank query path's output)
 *   c     [B,T,r]       shared latent, used as both key and value
 *   w_uk  [H,d_q,r]     key up-projection W_UK (first block of kv_up.weight)
 *   w_uv  [H,d_v,r]     value up-projection W_UV (second block of kv_up.weight)
 *   gate  [B,T,H*d_v]   pre-sigmoid gate logits W_g x, or NULL for no gate
 *   scale               softmax scale applied to the score (1.0 = the page's listing)
 *   out   [B,T,H*d_v]   result, flat index h*d_v + v; must not alias an input
 *   workspace           device buffer of >= mla_absorbed_attn_fwd_workspace_size(...)
 *                       bytes, 16-byte aligned, not used by any other call in flight;
 *                       may be NULL when that size is 0.  The r = 512 kernel keeps an
 *                       f16 copy of c there (see precision below).
 * Masking: token t attends to tokens 0..t of its own sequence.
 * Precision (BF16): the score operand q_abs * scale is not rounded to bf16.  At
 * r = 512 the score product runs on f16 copies of q_abs and c, each scaled by a
 * power of two (per query row, per sequence) into the f16 range and scaled back
 * exactly in the softmax; at r <= 64 q_abs is split into two bf16 parts.  The
 * softmax weights, o_lat / l and the output are rounded to bf16.
 * Supported: F32 with r, d_q, d_v <= 64 and T <= 1,048,560; BF16 with (r, d_q, d_v) = (512, 128, 128),
 * or r in {32, 64} with d_q, d_v in {16, 32, 48, 64}.  B*T == 0 is a no-op
 * returning MLA_OK.
 * Alignment: every pointer 16-byte aligned.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API size_t mla_absorbed_attn_fwd_workspace_size(int B, int T, int H, int d_q, int d_v, int r, int dtype);
MLA_API int mla_absorbed_attn_fwd(const void *q, const void *c, const void *w_uk, const void *w_uv,
                                  const void *gate, float scale, void *out,
                                  int B, int T, int H, int d_q, int d_v, int r,
                                  int dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * mla_absorbed_attn_fwd_lse - mla_absorbed_attn_fwd that also writes each row's
 * log-sum-exp of the scaled, causally masked scores, for mla_absorbed_attn_bwd_lse:
 *   lse[b,h,t] = ln sum_{u<=t} exp(scale * q_abs[b,t,h,:] . c[b,u,:])   [B,H,T] fp32
 * so that attn[b,h,t,u] = exp(scale * q_abs . c_u - lse[b,h,t]) (page "Gated MLA
 * （矩阵吸收版）", section "完整计算流（四步）", step 2: the softmax's normaliser).
 * Arguments, workspace (mla_absorbed_attn_fwd_workspace_size) and precision as
 * for mla_absorbed_attn_fwd; lse is caller-owned device memory, 16-byte aligned,
 * overwritten.  Supported: BF16 with (r, d_q, d_v) = (512, 128, 128); others
 * return MLA_ERR_UNSUPPORTED.  lse NULL returns MLA_ERR_NULL.
 */
MLA_API int mla_absorbed_attn_fwd_lse(const void *q, const void *c, const void *w_uk, const void *w_uv,
                                      const void *gate, float scale, void *out, float *lse, int B, int T, int H,
                                      int d_q, int d_v, int r, int dtype, void *workspace,
                                      size_t workspace_bytes, void *stream);

/*
 * mla_absorbed_attn_bwd - gradients of the attention (steps 2-4 of section
 * "完整计算流（四步）" of the page "Gated MLA（矩阵吸收版）", which gives the forward
 * only; this takes the chain rule back through it).  For
 * L = sum(dout * out) with out = mla_absorbed_attn_fwd(q, c, w_uk, w_uv, gate,
 * scale) it writes (fp32 whatever the input dtype, caller-owned device memory,
 * overwritten):
 *   dq     [B,T,H,d_q]   dL/dq
 *   dc     [B,T,r]       dL/dc (summed over heads and over the queries that see each key)
 *   dw_uk  [H,d_q,r]     dL/dW_UK (summed over batch and tokens)
 *   dw_uv  [H,d_v,r]     dL/dW_UV
 *   dgate  [B,T,H*d_v]   dL/dgate (the pre-sigmoid logits); NULL exactly when gate is NULL
 * Inputs as for mla_absorbed_attn_fwd, plus dout [B,T,H*d_v], all of dtype
 * `dtype` (MLA_DTYPE_F32 or MLA_DTYPE_BF16; bf16 values are widened to fp32).
 * workspace: >= mla_absorbed_attn_bwd_workspace_size(...) bytes, 16-byte
 * aligned (per-row q_abs, do_lat and softmax statistics between the kernels).
 * Supported:
 *  - r, d_q, d_v <= 64 (the toy sizes), F32 or BF16, T <= 4,194,240: fp32
 *    arithmetic throughout (SIMT).  dc, dw_uk and dw_uv are sums over thread
 *    blocks formed with atomics, so their last bits may differ between calls.
 *  - BF16 with (r, d_q, d_v) = (512, 128, 128): tensor cores.  The call runs the
 *    forward once more (its output before the gate and each row's softmax
 *    statistics), then every product of the chain rule as a batched bf16 GEMM
 *    with fp32 accumulation over per-head matrices kept in the workspace: the
 *    attention matrix and its gradient ([T, T] per head, bf16, causal tiles
 *    only), q_abs, do_lat, o_lat and dq_abs ([T, r] per head, bf16).  The
 *    workspace is therefore O(B H T^2): about 2 B H T^2 + 9 B H T r bytes.
 *    Deterministic (no atomics).
 * Other shapes return MLA_ERR_UNSUPPORTED.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API size_t mla_absorbed_attn_bwd_workspace_size(int B, int T, int H, int d_q, int d_v, int r, int dtype);
MLA_API int mla_absorbed_attn_bwd(const void *q, const void *c, const void *w_uk, const void *w_uv, const void *gate,
                                  float scale, const void *dout, void *dq, void *dc, void *dw_uk, void *dw_uv,
                                  void *dgate, int B, int T, int H, int d_q, int d_v, int r, int dtype,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * mla_absorbed_attn_bwd_lse - mla_absorbed_attn_bwd given what a forward call
 * mla_absorbed_attn_fwd_lse(q, c, w_uk, w_uv, gate, scale) on the same inputs
 * returned: its output `out` [B,T,H*d_v] (after the gate) and `lse` [B,H,T].  The
 * forward is not run again: the attention matrix is rebuilt from lse, and with a
 * gate dgate = dout * out * (1 - sigmoid(gate)).  Outputs, workspace
 * (mla_absorbed_attn_bwd_workspace_size) and determinism as for mla_absorbed_attn_bwd.
 * Supported: BF16 with (r, d_q, d_v) = (512, 128, 128); others return
 * MLA_ERR_UNSUPPORTED.  out or lse NULL returns MLA_ERR_NULL; both 16-byte aligned.
 */
MLA_API int mla_absorbed_attn_bwd_lse(const void *q, const void *c, const void *w_uk, const void *w_uv,
                                      const void *gate, float scale, const void *dout, const void *out,
                                      const float *lse, void *dq, void *dc, void *dw_uk, void *dw_uv, void *dgate,
                                      int B, int T, int H, int d_q, int d_v, int r, int dtype, void *workspace,
                                      size_t workspace_bytes, void *stream);

/*
 * mla_latent_decode_workspace_size - bytes of device workspace mla_latent_decode
 * needs for these sizes on the CURRENT device (it depends on the SM count).
 * Returns 0 for sizes that are invalid or unsupported.
 */
MLA_API size_t mla_latent_decode_workspace_size(int B, int H, int r, int max_len);

/*
 * mla_latent_decode - one decode step over the cached latent.
 *
 * Only the latent c is cached (page "Gated MLA（矩阵吸收版）", sections
 * "标准 MHA 的 KV cache 问题" and "形状与参数对比", KV-cache table: r values
 * per token instead of 2*H*d).  Each sequence b has one new query, already
 * absorbed (q_abs = q . W_UK, step 2), that attends, without a mask, to its
 * cache rows 0 .. lens[b]-1 (the caller has appended the new token's own
 * latent first).  Steps 2-4 then follow as in the prefill.
 *
 * Arguments:
 *   q_abs     [B,H,r]         absorbed queries
 *   c_cache   element (b,u,j) at b*max_len*ld_cache + u*ld_cache + j
 *   ld_cache  row stride of the cache in elements (>= r, multiple of 8)
 *   lens      int32 [B] on the device, 0 <= lens[b] <= max_len;
 *             lens[b] == 0 writes a zero output row.  Rows at or beyond
 *             lens[b] are never used, whatever they hold.
 *   max_len   rows allocated per sequence
 *   w_uv      [H,d_v,r]       value up-projection
 *   gate      [B,H*d_v]       pre-sigmoid gate logits, or NULL
 *   scale     softmax scale
 *   out       [B,H*d_v]
 *   workspace device buffer of >= mla_latent_decode_workspace_size(...) bytes,
 *             16-byte aligned, not used by any other call in flight
 * Supported: BF16 with r = 512, d_v = 128, 1 <= H <= 96.
 * A lens[b] outside [0, max_len] found on the device is clamped to that
 * range and reported as MLA_ERR_DEVICE_BOUNDS by mla_get_device_error().
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_latent_decode(const void *q_abs, const void *c_cache, long long ld_cache, const int *lens,
                              int max_len, const void *w_uv, const void *gate, float scale, void *out,
                              int B, int H, int d_v, int r, int dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * mla_latent_decode_fp8 - mla_latent_decode over a latent cache stored in
 * 8-bit floating point (e4m3: 1 sign, 4 exponent, 3 mantissa bits; largest
 * finite value 448), half the bytes per cached token of the bf16 cache.
 *
 * This carries the cache-size argument of the page "Gated MLA（矩阵吸收版）"
 * (sections "标准 MHA 的 KV cache 问题" and "形状与参数对比": only r values per
 * token are cached) one step further; the page itself caches bf16/fp32 c.
 * The cache holds c / cache_scale: cache row u of sequence b dequantises to
 * cache_scale * e4m3(c8_cache[b, u, :]), and the call computes exactly
 * mla_latent_decode over those dequantised rows.
 *
 * Arguments as for mla_latent_decode, except:
 *   c8_cache     e4m3 bytes; element (b,u,j) at byte b*max_len*ld_cache + u*ld_cache + j
 *   ld_cache     row stride in bytes (>= r, multiple of 16)
 *   cache_scale  positive, finite
 *   q_abs, w_uv, gate, out  bf16 as in mla_latent_decode (there is no dtype argument)
 *   workspace    >= mla_latent_decode_fp8_workspace_size(...) bytes, 16-byte
 *                aligned, not used by any other call in flight
 * Precision: both products run on the 8-bit tensor cores.  The query q_abs is
 * split into two e4m3 parts (after a power-of-two scale per head) and so are
 * the softmax weights, which keeps about 8 significant bits of each, as a
 * bf16 operand would; the cache values themselves are exact.
 * Supported: r = 512, d_v = 128, 1 <= H <= 96.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API size_t mla_latent_decode_fp8_workspace_size(int B, int H, int r, int max_len);
MLA_API int mla_latent_decode_fp8(const void *q_abs, const void *c8_cache, long long ld_cache, const int *lens,
                                  int max_len, float cache_scale, const void *w_uv, const void *gate, float scale,
                                  void *out, int B, int H, int d_v, int r, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * mla_quantize_latent_fp8 - fill an e4m3 latent cache from bf16 latent rows:
 * c8[i, j] = e4m3(c[i, j] * (1 / cache_scale)), the product formed in fp32
 * (1 / cache_scale rounded to fp32 first), rounded to the nearest e4m3 value
 * (ties to even) and clamped to +-448.  Same section as mla_latent_decode_fp8.
 *   c      bf16 [rows, r] with row stride ld_c elements (multiple of 8)
 *   c8     bytes [rows, r] with row stride ld_c8 bytes (multiple of 16)
 * r a multiple of 8; both pointers 16-byte aligned; rows == 0 is a no-op.
 * Latent rows from RMSNorm with unit gain have |c| <= sqrt(r) (22.6 at
 * r = 512), so cache_scale = 1/16 maps them inside e4m3's range.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_quantize_latent_fp8(const void *c, long long ld_c, void *c8, long long ld_c8, long long rows, int r,
                                    float cache_scale, void *stream);

/*
 * The 4-bit latent cache.
 *
 * The cache-size argument of the page "Gated MLA（矩阵吸收版）" (sections "标准 MHA 的 KV cache 问题" and
 * "形状与参数对比": only r values per token are cached) carried one step past the e4m3 cache; the page itself
 * caches bf16/fp32 c.  A row of r latent values (r a multiple of 32) is stored in the OCP MX fp4 format:
 *   r / 2 bytes    e2m1 codes, element 2j in the low half of byte j: a sign bit, then the index of the magnitude
 *                  in {0, 0.5, 1, 1.5, 2, 3, 4, 6}
 *   r / 32 bytes   one scale byte X per 32 consecutive elements: 2^(X - 127), X taken into [87, 167]; 255 is NaN
 *                  (every element of the group is then NaN)
 *   padding        to a multiple of 16 bytes; never read or written
 * Every pointer of the calls below is 16-byte aligned, lens and counts among them.
 * mla_latent_fp4_row_bytes(r) is that row's size: 272 at r = 512 (1024 in bf16).  Returns 0 for an r that is not a
 * positive multiple of 32 up to 65536.
 */
MLA_API size_t mla_latent_fp4_row_bytes(int r);

/*
 * mla_quantize_latent_fp4 - fill rows of an fp4 latent cache from latent rows.
 * Per group of 32: X - 127 = the smallest exponent e in [-40, 40] with max|c| <= 7 * 2^e, and each code is
 * c * 2^-e (exact) rounded to the nearest e2m1 value (ties to the even index, clamped to +-6; a negative value
 * that rounds to zero keeps its sign bit).  A group that holds a NaN or an infinity becomes NaN (X = 255, codes 0).
 *   c      [rows, r] of `dtype` (BF16 or F32), row stride ld_c elements (>= r, rows 16-byte aligned)
 *   c4     [rows] cache rows, row stride ld_c4 bytes (>= mla_latent_fp4_row_bytes(r), a multiple of 16)
 * rows == 0 is a no-op.  Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_quantize_latent_fp4(const void *c, long long ld_c, void *c4, long long ld_c4, long long rows, int r,
                                    int dtype, void *stream);

/*
 * mla_append_latent_fp4 - quantise new latent rows into a cache where each sequence ends: row t of sequence b goes
 * to cache row lens[b] + t, for t < counts[b] (all T when counts is NULL).  T = 1 is a decode step's append, a larger
 * T a chunk of a prompt.  No other cache row is touched.
 *   c         [B, T, r] of `dtype`, dense but for the row stride ld_c (batch stride T * ld_c)
 *   c4_cache  row u of sequence b at byte (b * max_len + u) * ld_cache
 *   lens      int32 [B] on the device, read only: the caller advances it
 *   counts    int32 [B] on the device or NULL; a count below 0 or above T is taken as 0 or T and reported as
 *             MLA_ERR_DEVICE_BOUNDS (mla_get_device_error)
 * A row whose place is outside [0, max_len) is not written and reported as MLA_ERR_DEVICE_BOUNDS.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_append_latent_fp4(const void *c, long long ld_c, void *c4_cache, long long ld_cache, const int *lens,
                                  const int *counts, int max_len, int B, int T, int r, int dtype, void *stream);

/*
 * mla_dequantize_latent_fp4 - read cache rows back as latent rows of `dtype`; every value the format holds is exact
 * in BF16 and F32.
 *   c4        row u of sequence b at byte b * batch_c4 + u * ld_c4 (both multiples of 16, batch_c4 >= 0)
 *   c         [B, rows, r], dense but for the row stride ld_c (elements, >= r, rows 16-byte aligned)
 *   lens      int32 [B] on the device or NULL: only rows u < lens[b] are read and written, the others of c are left
 *             as they were.  A negative length is taken as 0 and reported as MLA_ERR_DEVICE_BOUNDS.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_dequantize_latent_fp4(const void *c4, long long ld_c4, long long batch_c4, const int *lens, void *c,
                                      long long ld_c, int B, int rows, int r, int dtype, void *stream);

/*
 * mla_latent_decode_fp4 - mla_latent_decode over an fp4 latent cache: exactly mla_latent_decode over the rows'
 * values.
 * Arguments as for mla_latent_decode, except:
 *   c4_cache   row u of sequence b at byte (b * max_len + u) * ld_cache; may be NULL when max_len is 0
 *   ld_cache   row stride in bytes (>= 272, a multiple of 16)
 *   q_abs, w_uv, gate, out  bf16 (there is no dtype argument)
 *   workspace  >= mla_latent_decode_fp4_workspace_size(...) bytes, 16-byte aligned, not used by any other call in
 *              flight
 * Precision: the scores take q_abs as two e4m3 parts (exact for a bf16 query but for elements below 2^-9 of their head's
 * largest, which are off by at most 2^-21 of it up to 48 heads, 2^-17 above) and the rows' values exactly.  The softmax
 * weights are two 8-bit parts: a weight is off by at most 2^-8 of itself up to 48 heads and 2^-7 above, and in both cases
 * by 2^-21 of the largest among the 4096 rows around it and 2^-24 of the largest of all (weights times their rows' largest
 * scales); all light rows beside a heavy one together lose at most 1.15 * 2^-9 of its weight.  Sums, maxima and the join
 * are fp32.  Rows that hold a group of values more than 2^14 below their largest scale (and the rows around them) are taken
 * in fp32, one after the other: right, but about fifty times slower.
 * lens[b] outside [0, max_len] is taken into it and reported as MLA_ERR_DEVICE_BOUNDS; lens[b] = 0 gives zeros.
 * B == 0 is a no-op.
 * Supported: r = 512, d_v = 128, 1 <= H <= 96.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API size_t mla_latent_decode_fp4_workspace_size(int B, int H, int r, int max_len);
MLA_API int mla_latent_decode_fp4(const void *q_abs, const void *c4_cache, long long ld_cache, const int *lens,
                                  int max_len, const void *w_uv, const void *gate, float scale, void *out, int B,
                                  int H, int d_v, int r, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The paged latent cache.  Rows live in a pool of `num_blocks` blocks of `block_size` rows (bf16, row stride ld_pool
 * elements, block stride block_size * ld_pool); cache row u of sequence b is row u % block_size of block
 * block_table[b * ld_table + u / block_size].  A serving step of T new tokens per sequence: reserve (blocks for rows
 * lens[b] .. lens[b] + counts[b] - 1 and their slots), append (their latents), attend, then the caller advances lens by
 * the number of tokens it keeps.
 * Kept tokens have to stand one after the other.  Tokens 0, 1, .. of a chunk do.  Of a drafted tree, draft t's latent is
 * row lens[b] + t, but the d-th token of the path that is kept, counted from 0, belongs in row lens[b] + d: unless the path
 * is drafts 0, 1, 2, .., append its latents again, the d-th to slots[b][d] (all sequences' in one call, with -1 where a
 * path is shorter), before lens is advanced.  Otherwise later calls take rows of dropped drafts for the past.  Dropped
 * drafts themselves need nothing: their rows are written again, their blocks go back at the next reserve.
 * num_blocks * block_size and max_blocks * block_size are at most 2^31 - 1024.
 *
 * mla_reserve_latent_blocks - give each sequence the blocks for lens[b] + counts[b] rows and map its new tokens to
 * pool rows.  In place, on the device, in a fixed order (the same inputs give the same blocks):
 *   need_b = ceil((lens[b] + counts[b]) / block_size).  Sequences with held[b] > need_b give up their last blocks;
 *   numbered in order of sequence and index, these go first to the sequences with held[b] < need_b, in the same order;
 *   then the top of the free stack is taken; what nobody takes is put on the stack, the first one given up on top.
 *   A growth followed by the same shrinking leaves the stack as it was.  lens[b] = counts[b] = 0 releases a sequence.
 *   lens, counts  int32 [B] on the device
 *   block_table   int32 [B, max_blocks] (row stride ld_table elements); entries from held[b] on are not read, and those
 *                 past the new held[b] are left as they are
 *   held          int32 [B]: the blocks in each sequence's row of the table; becomes need_b
 *   free_blocks   int32 [capacity]: the free blocks are its first free_count[0] entries, the last one on top
 *   free_count    int32 [1]
 *   slots         int32 [B, T] (16-byte aligned) or NULL when T is 0: block_table[b][u / block_size] * block_size +
 *                 u % block_size with u = lens[b] + t for t < counts[b], -1 for the other t
 * All or nothing: when the free blocks do not suffice, a sequence needs more than max_blocks, a count is above T (with
 * slots), a length, count, held or free_count is out of its range, a block that would be given up or taken is below 0 or
 * 2^31 - 4096 of them or more would be, every sequence and the stack keep their blocks, every slot is -1 and
 * MLA_ERR_DEVICE_BOUNDS is reported (mla_get_device_error); after a block below 0, entries from held[b] on and the stack's
 * from free_count on may hold anything.  Blocks are numbers from 0 on; a new row past pool row 2^31 - 1 is reported the
 * same way and has the slot -1, with more than 8192 slots a sequence whose first one is.
 * A block is in the first held[b] entries of one sequence or on the stack, never in two places: this is not checked, and a
 * block in two places serves two sequences.  That goes for blocks behind a window, too: the attention does not read their
 * entries, but a sequence keeps its blocks until it needs fewer, and gives up its last ones only.
 * Supported: B <= 16384.  Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_reserve_latent_blocks(const int *lens, const int *counts, int *block_table, long long ld_table, int *held,
                                      int *free_blocks, int *free_count, int *slots, int B, int T, int max_blocks,
                                      int capacity, int block_size, void *stream);

/*
 * mla_append_latent_paged - pool row slots[i] becomes row i of c, in bf16 (rounded to nearest even from F32), for every
 * i < rows with a slot; a slot of -1 skips its row, any other outside the pool is skipped and reported as
 * MLA_ERR_DEVICE_BOUNDS.  A slot that occurs twice holds pieces of either row afterwards (mla_reserve_latent_blocks gives
 * each row one of its own).  No other row of the pool is touched.
 *   c      [rows, r] of `dtype`, row stride ld_c elements
 *   pool   pool row i (row i % block_size of block i / block_size) at element i * ld_pool; pool_rows of them
 * Rows 16-byte aligned, r a multiple of 8.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_append_latent_paged(const void *c, long long ld_c, void *pool, long long ld_pool, long long pool_rows,
                                    const int *slots, long long rows, int r, int dtype, void *stream);

/*
 * mla_latent_attend_paged - steps 2-4 for counts[b] new tokens of each sequence over the paged cache, in which the new
 * tokens' own latents are rows lens[b] .. lens[b] + counts[b] - 1 (mla_append_latent_paged); a tree's kept path is appended
 * again afterwards, see above:
 *
 *   out[b,t,h] = sigmoid(gate[b,t,h]) * W_UV[h] . sum_u a_u c_u,   a = softmax over the visible rows u of
 *                scale * q_abs[b,t,h] . c_u
 *
 * Without parents token t is the t-th of a chunk: its position is lens[b] + t and it sees rows u <= lens[b] + t.  With
 * parents it is a draft: parents[b][t] < t is the new token it follows, -1 none; its position is lens[b] + the number of
 * its ancestors among the new tokens, and it sees the rows u < lens[b], its ancestors' and its own.  With window > 0 a row
 * is seen only if its position is above the token's - window or below sinks (window 1: the token itself; 0: no window).
 * A row that a token does not see has no effect on it, whatever it holds.
 *   q_abs        [B, T, H, r] bf16, absorbed queries (unscaled)
 *   block_table  int32 [B, max_blocks] on the device, row stride ld_table; only entries for visible rows are read
 *   lens         int32 [B]: rows cached before the new tokens
 *   counts       int32 [B] or NULL (T each); rows of out for t >= counts[b] are left as they were
 *   parents      int32 [B, T] or NULL; T <= 64 with it
 *   w_uv         [H, d_v, r], gate [B, T, H*d_v] or NULL (pre-sigmoid logits), out [B, T, H*d_v], all bf16
 *   workspace    >= mla_latent_attend_paged_workspace_size(B, T, H, r) bytes (1,040 for each of B * T * H, and 20 to 80 MB),
 *                16-byte aligned, not used by any other call in flight
 * A sequence with a length, count or lens + counts outside [0, T] and [0, max_blocks * block_size] is skipped, rows of a
 * block outside the pool count as zeros, and a parent outside [-1, t) as -1; each is reported as MLA_ERR_DEVICE_BOUNDS.
 * Precision: products of bf16 values in fp32; softmax statistics, sums and the join of split rows in fp32.  Rounded to
 * bf16 are the softmax weights and out.  The weighted latent is kept as f16 with an exponent for each 32 values (2^-11
 * of each part, once more where split rows are joined) and goes to the product with W_UV as two bf16 parts (2^-16).
 * The same call gives the same bits.  Which rows are split depends on all sequences of a call, and so do last bits.
 * Supported: r = 512, d_v = 128, 1 <= H <= 128, block_size a multiple of 64.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API size_t mla_latent_attend_paged_workspace_size(int B, int T, int H, int r);
MLA_API int mla_latent_attend_paged(const void *q_abs, const void *pool, long long ld_pool, const int *block_table,
                                    long long ld_table, const int *lens, const int *counts, const int *parents,
                                    const void *w_uv, const void *gate, float scale, int window, int sinks, void *out,
                                    int B, int T, int H, int d_v, int r, int num_blocks, int block_size, int max_blocks,
                                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * mla_latent_decode_noalloc - mla_latent_decode for callers that cannot
 * allocate device memory.
 *
 * The paper has no counterpart to this entry point; it exists for callers
 * that cannot call cudaMalloc: a host framework that owns all device memory
 * and hands the library only its inputs and outputs, or a service that must
 * not allocate (or pay cudaMalloc's synchronisation) once it is running.  It
 * computes exactly what mla_latent_decode computes, with the same arguments
 * except that there is no workspace: the partial results live in a scratch
 * array that the library reserves in device memory when it is loaded, 48 MiB
 * on every device that loads the library, held until the process exits.
 *
 * - Sizes whose scratch need (mla_latent_decode_workspace_size) exceeds
 *   48 MiB return MLA_ERR_WORKSPACE and launch nothing.  The K3 decode
 *   workload (B = 64, H = 96, r = 512 on a 152-SM GB300) needs 13.9 MB.
 * - The call allocates and frees nothing, on the host or the device.
 * - The first call on a device looks up the scratch array's device address
 *   on that device (cudaGetSymbolAddress); make that first call before any
 *   stream capture.  If that lookup fails (for example inside a capture, or
 *   when the library's device code cannot be loaded on the device) the call
 *   returns MLA_ERR_CUDA, clears the runtime's pending error and launches
 *   nothing; a later call retries the lookup.
 * - Every call uses the same scratch array: calls whose kernels can overlap
 *   on the GPU (different streams, no ordering between them) race on it and
 *   give wrong results.  Calls on one stream, or otherwise ordered, are safe.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_latent_decode_noalloc(const void *q_abs, const void *c_cache, long long ld_cache, const int *lens,
                                      int max_len, const void *w_uv, const void *gate, float scale, void *out,
                                      int B, int H, int d_v, int r, int dtype, void *stream);

/*
 * mla_gated_layer_workspace_size - bytes of device workspace mla_gated_layer_fwd
 * needs for these sizes (0 if the shape or dtype is not supported).
 */
MLA_API size_t mla_gated_layer_workspace_size(int B, int T, int D, int H, int d_q, int d_v, int r, int r_q,
                                              int dtype);

/*
 * mla_gated_layer_fwd - the whole Gated-MLA layer (page "Gated MLA（矩阵吸收版）",
 * section "完整计算流（四步）", steps 1-4, plus the output projection of the
 * listing in section "代码对照"):
 *
 *   c   = RMSNorm(x . w_kv_down^T)                         [B,T,r]
 *   q   = RMSNorm(x . w_q_down^T) . w_q_up^T                 [B,T,H,d_q]
 *   g   = x . w_gate^T                                       [B,T,H*d_v]
 *   o   = mla_absorbed_attn_fwd(q, c, W_UK, W_UV, g, scale)  [B,T,H*d_v]
 *   y   = o . w_o^T                                          [B,T,D]
 *
 * RMSNorm: z / sqrt(mean(z^2) + 1e-6), unit gain.  No biases.  Weights are
 * nn.Linear weights [out_features, in_features], row-major:
 *   w_q_down [r_q, D]   w_q_up [H*d_q, r_q]   w_kv_down [r, D]
 *   w_kv_up  [H*(d_q+d_v), r]: all heads' W_UK rows first (W_UK = w_kv_up as
 *            [H,d_q,r]), then all heads' W_UV rows ([H,d_v,r])
 *   w_gate   [H*d_v, D]   w_o [D, H*d_v]
 * x [B,T,D] and y [B,T,D], row-major.  All tensors share `dtype`.
 *
 * Supported: MLA_DTYPE_F32 with r, d_q, d_v <= 64 and T <= 1,048,560 (SIMT fp32, no TF32);
 * MLA_DTYPE_BF16 with r = 512, d_q = d_v = 128, H even, D and r_q multiples of
 * 256 (tensor-core GEMMs, fp32 accumulation, bf16 intermediate results).
 *
 *   workspace  device buffer of >= mla_gated_layer_workspace_size(...) bytes,
 *              16-byte aligned, caller-owned.  On return (in stream order) it
 *              holds, each part starting on a 256-byte boundary and in the
 *              input dtype: q [B*T, H*d_q], c [B*T, r], g [B*T, H*d_v] and o
 *              [B*T, H*d_v], followed by internal scratch.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_gated_layer_fwd(const void *x, const void *w_q_down, const void *w_q_up, const void *w_kv_down,
                                const void *w_kv_up, const void *w_gate, const void *w_o, float scale, void *y,
                                int B, int T, int D, int H, int d_q, int d_v, int r, int r_q, int dtype,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * mla_gated_layer_decode_workspace_size - bytes of device workspace
 * mla_gated_layer_decode needs on the CURRENT device (0 if unsupported).
 */
MLA_API size_t mla_gated_layer_decode_workspace_size(int B, int D, int H, int d_q, int d_v, int r, int r_q,
                                                     int max_len, int dtype);

/*
 * mla_gated_layer_decode - one decode step of the whole layer with the
 * latent-cache append (page "Gated MLA（矩阵吸收版）": only the latent c is
 * cached, section "低秩压缩"; steps 1-4 of section "完整计算流（四步）"; W_o).
 * For each sequence b, the new token x[b] (position lens[b]):
 *
 *   c_cache[b, lens[b], :] = RMSNorm(x[b] . w_kv_down^T)          (the append)
 *   q_abs = (RMSNorm(x[b] . w_q_down^T) . w_q_up^T) . W_UK          per head
 *   o     = mla_latent_decode(q_abs, c_cache, lens[b] + 1 rows, W_UV, g = x[b] . w_gate^T, scale)
 *   y[b]  = o . w_o^T
 *
 *   x [B, D], y [B, D]; weights as in mla_gated_layer_fwd.
 *   c_cache    [B, max_len, r] with row stride ld_cache (elements, multiple of
 *              8, >= r); row lens[b] of each sequence is written.
 *   lens       int32 [B] on the device: the new token's position, in
 *              [0, max_len).  Read only; the caller advances it after the
 *              step.  A position outside the range is reported as
 *              MLA_ERR_DEVICE_BOUNDS (mla_get_device_error) and that row is
 *              not written.
 *   workspace  >= mla_gated_layer_decode_workspace_size(...) bytes, 16-byte
 *              aligned.
 * Supported: MLA_DTYPE_BF16 with r = 512, d_q = d_v = 128, 1 <= H <= 96 and
 * even, D and r_q multiples of 256.
 * Returns MLA_OK or a negative mla_status_t; nothing is launched on error.
 */
MLA_API int mla_gated_layer_decode(const void *x, const void *w_q_down, const void *w_q_up, const void *w_kv_down,
                                   const void *w_kv_up, const void *w_gate, const void *w_o, float scale, void *y,
                                   void *c_cache, long long ld_cache, const int *lens, int max_len, int B, int D,
                                   int H, int d_q, int d_v, int r, int r_q, int dtype, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * mla_get_device_error - synchronise `stream`, then read and clear the current
 * device's error word.  Returns MLA_OK, MLA_ERR_DEVICE_TIMEOUT,
 * MLA_ERR_DEVICE_BOUNDS, or MLA_ERR_CUDA if the synchronisation itself failed.
 */
MLA_API int mla_get_device_error(void *stream);

/*
 * mla_debug_wait_timeout - exercise the device-side failure path.  The pages
 * have no counterpart: this is a diagnostic of the library's own error
 * handling.  Launches one thread on `stream` that waits, with the same bounded
 * wait every kernel of this library uses, for an mbarrier phase that nothing
 * completes; after `limit_us` microseconds (1 .. 2,000,000) the wait gives up
 * and records MLA_ERR_DEVICE_TIMEOUT in the current device's error word, which
 * mla_get_device_error() then returns.  Nothing faults or traps; the context
 * stays usable.  Returns MLA_OK when launched, MLA_ERR_SHAPE for a limit out
 * of range (nothing launched), MLA_ERR_CUDA if the launch failed.
 */
MLA_API int mla_debug_wait_timeout(unsigned int limit_us, void *stream);

/* mla_status_string - static, NUL-terminated description of a status code. */
MLA_API const char *mla_status_string(int status);

/* mla_version - library version as major*10000 + minor*100 + patch. */
MLA_API int mla_version(void);

/*
 * mla_kernel_launches - kernels this library has launched in this process
 * (every entry point, device and stream; a diagnostic counter, never reset).
 */
MLA_API unsigned long long mla_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_GB300_H */
