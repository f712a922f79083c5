/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention library.
 *
 * The operation is exact scaled-dot-product attention computed tile by tile
 * with an online softmax, forward and backward ("flash-attn-triton" docs page:
 * sections "The argument", "Tiling softmax is exact algebra" with Fig. 3, and
 * "Scope"; FlashAttention note, "Key Mechanisms").  For each (batch b, head h):
 *
 *     S = scale * Q K^T                     (N x N, never stored)
 *     causal: key j is allowed for query i iff j <= i (lower triangle)
 *     P = softmax over the allowed keys of each row
 *     O = P V
 *     L = logsumexp of the allowed scaled scores of each row (natural log)
 *
 * and the backward returns dQ, dK, dV for an upstream gradient dO, rebuilding P
 * from the saved L instead of storing it (docs page, "Scope"; FlashAttention
 * note, "Key Mechanisms", backward recomputation).
 *
 * Conventions shared by every call
 *   Layout     Q, K, V, O, dO, dQ, dK, dV: dense row-major (B, H, N, d) arrays of
 *              16-bit floats (fp16 or bf16, all the same); element (b,h,n,c) at
 *              ((b*H + h)*N + n)*d + c.  L: dense (B, H, N) fp32.
 *   Memory     every pointer is CUDA device memory (or managed memory) of the
 *              current device; the caller owns every buffer; the library keeps
 *              no pointer after a call returns.  Outputs must not overlap inputs.
 *   Alignment  16-bit arrays and the workspace: 16-byte aligned; L: 4-byte aligned.
 *   Streams    `stream` is a cudaStream_t (NULL = the legacy default stream).
 *              Calls only enqueue work: they return before the GPU finishes and
 *              never synchronise, except fa_device_status.  So a sequence of calls
 *              can be captured into a CUDA graph once each call has run eagerly
 *              (the first call of a kind sets kernel attributes) and, for the
 *              backward, with a caller workspace; the replay gives the eager
 *              results bit for bit.
 *   Errors     arguments are validated before anything is launched; a call that
 *              returns an error has enqueued nothing (launch failures excepted:
 *              FA_ERR_CUDA, with the CUDA error code from fa_last_cuda_error()).
 *   Supported  d in {32, 64, 128}; fp16 or bf16; causal 0/1; any N >= 1 (N need
 *              not be a multiple of the 128-row tile); scale finite and > 0.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa_status {
  FA_OK = 0,
  FA_ERR_INVALID_VALUE = 1,  /* NULL pointer, B/H/N < 1, bad scale, short workspace, overlap */
  FA_ERR_UNSUPPORTED = 2,    /* d not in {32,64,128}, unknown dtype, sizes beyond the limits */
  FA_ERR_MISALIGNED = 3,     /* a pointer violates the alignment rule above */
  FA_ERR_CUDA = 4,           /* a CUDA runtime/driver call or a launch failed */
  FA_ERR_TIMEOUT = 5         /* a kernel gave up a bounded wait (see fa_device_status) */
} fa_status;

typedef enum fa_dtype { FA_FP16 = 0, FA_BF16 = 1 } fa_dtype;

/* Forward.  Writes O (B,H,N,d) and L (B,H,N) fp32 = natural-log logsumexp of the
 * allowed scaled scores of each row (docs page Fig. 3: L = m + log l, one float
 * per row, the only state the backward needs).  Q, K, V are read once per
 * 128-query-row tile pair; the N x N score matrix never reaches memory. */
fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* L,
                 int B, int H, int N, int d, int causal, float scale, fa_dtype dtype,
                 void* stream);

/* Bytes of device workspace fa_bwd needs for these sizes: the per-row delta
 * D = rowsum(dO o O) and L * log2(e), both fp32, padded to whole 128-row tiles.
 * Returns 0 for sizes fa_bwd would reject. */
size_t fa_bwd_workspace_size(int B, int H, int N, int d, int causal);

/* Backward.  Given Q, K, V, the forward's O and L, and dO, writes dQ, dK, dV
 * (16-bit, same layout as Q).  P is rebuilt from L (docs page, "Scope"):
 *   dV = P^T dO, dP = dO V^T, D = rowsum(dO o O), dS = P o (dP - D),
 *   dQ = scale dS K, dK = scale dS^T Q.
 * `workspace` is device memory of at least fa_bwd_workspace_size() bytes, used
 * as scratch during the call; pass NULL to let the library take it from the
 * stream-ordered allocator (cudaMallocAsync / cudaFreeAsync on `stream`). */
fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* L, void* dQ, void* dK, void* dV, void* workspace,
                 size_t workspace_bytes, int B, int H, int N, int d, int causal, float scale,
                 fa_dtype dtype, void* stream);

/* Grouped-query and multi-query attention (GQA / MQA).  The docs page lists
 * "MQA/GQA" among the features its kernels do not have yet ("Scope"); the note
 * credits FlashAttention-2 with adding them ("Versions and Evolution").  K and V
 * have Hkv heads instead of H: query head h of batch b attends with K/V head
 * h / (H/Hkv) of batch b (consecutive query heads share one K/V head; Hkv == 1 is
 * MQA, Hkv == H is fa_fwd / fa_bwd).  Each query head computes exactly what
 * fa_fwd computes with that K/V head; in the backward, dK and dV of a shared head
 * are the sums over its H/Hkv query heads.
 *   Layout   Q, O, dO, dQ: (B, H, N, d); K, V, dK, dV: (B, Hkv, N, d); L: (B, H, N).
 *   Errors   as fa_fwd / fa_bwd, plus FA_ERR_INVALID_VALUE when Hkv < 1, Hkv > H
 *            or H is not a multiple of Hkv.
 *   Workspace of fa_bwd_gqa: fa_bwd_workspace_size(B, H, N, d, causal) bytes (it
 *            depends on the query heads only), or NULL as for fa_bwd. */
fa_status fa_fwd_gqa(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H,
                     int Hkv, int N, int d, int causal, float scale, fa_dtype dtype,
                     void* stream);
fa_status fa_bwd_gqa(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                     const float* L, void* dQ, void* dK, void* dV, void* workspace,
                     size_t workspace_bytes, int B, int H, int Hkv, int N, int d, int causal,
                     float scale, fa_dtype dtype, void* stream);

/* Sliding-window (local) attention: causal, each query sees only the `window`
 * most recent keys, itself included: key j is allowed for query i iff
 * i - window < j <= i.  The docs page lists sliding windows among the features its
 * kernels do not have yet ("Scope") and fixes no convention; this causal band is
 * the plain reading.  Hkv as for fa_fwd_gqa (Hkv == H: no sharing).  window >=
 * N is plain causal attention.  Only the KV tiles inside the band are computed.
 *   Errors   as fa_fwd_gqa / fa_bwd_gqa, plus FA_ERR_INVALID_VALUE for window < 1.
 *   Workspace of fa_bwd_swa: fa_bwd_workspace_size(B, H, N, d, 1), or NULL. */
fa_status fa_fwd_swa(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H,
                     int Hkv, int N, int d, int window, float scale, fa_dtype dtype,
                     void* stream);
fa_status fa_bwd_swa(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                     const float* L, void* dQ, void* dK, void* dV, void* workspace,
                     size_t workspace_bytes, int B, int H, int Hkv, int N, int d, int window,
                     float scale, fa_dtype dtype, void* stream);

/* Variable-length batches: B sequences of different lengths packed one after
 * another (the docs page lists "variable-length batches" among the features its
 * kernels do not have yet, "Scope").  Sequence b holds rows cu_seqlens[b] ..
 * cu_seqlens[b+1]-1 of every tensor and attends only to its own keys (causal and
 * window as in fa_fwd / fa_fwd_swa, measured from the sequence's first row; window
 * 0 = none; window > 0 needs causal); K/V heads shared as in fa_fwd_gqa.
 *   Layout   Q, O, dO, dQ: (total, H, d); K, V, dK, dV: (total, Hkv, d), rows
 *            row-major with heads inside a row; L: (H, total) fp32.
 *   cu_seqlens  device int32 [B+1]: 0 = cu[0] <= cu[1] <= ... <= cu[B] = total.
 *            max_seqlen >= every cu[b+1] - cu[b] (it sizes the grid).  The kernels
 *            clamp every sequence to rows [0, total) and to max_seqlen rows, so
 *            offsets that break these rules leave rows uncomputed but never make a
 *            kernel touch memory outside the tensors.
 *   Workspace of fa_bwd_varlen: fa_bwd_varlen_workspace_size(B, max_seqlen, H, d),
 *            or NULL.
 *   Errors   as fa_fwd_gqa / fa_bwd_gqa (max_seqlen in the role of N), plus
 *            FA_ERR_INVALID_VALUE for cu_seqlens NULL, total < 1, window < 0 or a
 *            window without causal; FA_ERR_MISALIGNED if cu_seqlens is not 4-byte
 *            aligned. */
fa_status fa_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* L,
                        const int* cu_seqlens, int B, int total, int max_seqlen, int H, int Hkv,
                        int d, int causal, int window, float scale, fa_dtype dtype, void* stream);
size_t fa_bwd_varlen_workspace_size(int B, int max_seqlen, int H, int d);
fa_status fa_bwd_varlen(const void* Q, const void* K, const void* V, const void* O,
                        const void* dO, const float* L, void* dQ, void* dK, void* dV,
                        void* workspace, size_t workspace_bytes, const int* cu_seqlens, int B,
                        int total, int max_seqlen, int H, int Hkv, int d, int causal, int window,
                        float scale, fa_dtype dtype, void* stream);

/* Forward on 8-bit E4M3 inputs (the FP8 precision that the FlashAttention note
 * credits to FlashAttention-3, "Versions and Evolution"), head dim 128.  The
 * inputs are E4M3 codes with per-tensor descale factors: the result is the
 * attention of q_scale*Q, k_scale*K and v_scale*V, computed as the 16-bit
 * forward does ("flash-attn-triton" docs page, Fig. 3) with both products on the
 * tensor cores in 8 bits: S = Q K^T from the codes (fp32 accumulation), and
 * O += P V with P rounded to E4M3 (p <= 2^8 by the running-max rule); the sum l
 * is taken over the unrounded p.
 *   Q8     (B, H, N, 128) codes, one byte each.
 *   K8     (B, Hkv, N, 128) codes.
 *   Vt8    (B, Hkv, 128, N) codes of V with its last two axes swapped (see
 *          fa_quantize_fp8).
 *   O      (B, H, N, 128) bf16 output.  L (B, H, N) fp32, natural log, of the
 *          scores scale * q_scale * k_scale * (Q8 . K8).
 *   Query head h uses K/V head h / (H / Hkv).  N must be a multiple of 16 (the
 *   rows of Vt8 are N bytes apart and TMA wants 16-byte strides).  Q8, K8, Vt8
 *   and O 16-byte aligned, L 4-byte aligned.
 *   Errors: FA_ERR_UNSUPPORTED for d != 128 or N % 16 != 0; FA_ERR_INVALID_VALUE
 *   for NULL pointers, bad sizes, H not a multiple of Hkv, non-positive or
 *   non-finite scale or descale factors, overlapping buffers; FA_ERR_MISALIGNED
 *   for the alignment rules.  Asynchronous on `stream`. */
fa_status fa_fwd_fp8(const void* Q8, const void* K8, const void* Vt8, void* O, float* L, int B,
                     int H, int Hkv, int N, int d, int causal, float scale, float q_scale,
                     float k_scale, float v_scale, void* stream);

/* E4M3 codes of X * inv_scale, rounded to nearest even and saturated at +-448
 * (the preparation step of fa_fwd_fp8: inv_scale is 1 / descale).  X holds `mats`
 * row-major rows x cols matrices of 16-bit values (dtype FA_FP16 / FA_BF16); X8
 * receives one byte per element, each matrix transposed (cols x rows) when
 * transpose = 1.  Errors: FA_ERR_INVALID_VALUE for NULL pointers, sizes < 1, a
 * non-positive or non-finite inv_scale or overlapping buffers;
 * FA_ERR_UNSUPPORTED for another dtype, or with transpose for more than 65535
 * matrices or 2^21 rows; FA_ERR_MISALIGNED if X is not 2-byte aligned.
 * Asynchronous on `stream`. */
fa_status fa_quantize_fp8(const void* X, void* X8, long long mats, int rows, int cols,
                          float inv_scale, int transpose, fa_dtype dtype, void* stream);

/* Split-KV decoding: one new query row per (batch, head) attends to the first
 * cache_seqlens[b] cached keys of its sequence.  The key range is cut into
 * pieces whose softmax partial states (running max m, sum l, unnormalised
 * output acc) are merged exactly on the GPU: the tutorial page "What is
 * FlashAttention?", "Softmax in pieces" (merging two partial results), applied
 * to a key/value cache (the FlashAttention note lists inference serving with a
 * KV cache among the method's uses: "Applications and Use Cases").
 *   Q            (B, H, d) fp16/bf16, one query row per head.
 *   Kc, Vc       (B, Hkv, Nmax, d) caches; rows at and past cache_seqlens[b]
 *                are never used (their contents may be anything).
 *   cache_seqlens  device int32 [B]; values are clamped to [0, Nmax].  A
 *                sequence with no cached key gets O = 0, L = -inf.
 *   O            (B, H, d) output, same dtype.
 *   L            (B, H) fp32, the natural-log logsumexp of each row's scores.
 *   workspace    fa_decode_workspace_size(B, H, Hkv, Nmax, d) bytes of device
 *                memory (16-byte aligned) for the partial states, or NULL: the
 *                library then allocates and frees it on `stream`.
 *   Query head h uses K/V head h / (H / Hkv).  Q, Kc, Vc and O 16-byte aligned.
 *   Errors: FA_ERR_INVALID_VALUE for NULL pointers, B, H or Nmax < 1, H not a
 *   multiple of Hkv, a non-positive or non-finite scale, a short workspace or
 *   overlapping buffers; FA_ERR_UNSUPPORTED for d not 32/64/128, another dtype,
 *   Nmax above 2^30 or sizes past the index limits; FA_ERR_MISALIGNED for the
 *   alignment rules.
 *   Asynchronous on `stream`; nothing is read back. */
size_t fa_decode_workspace_size(int B, int H, int Hkv, int Nmax, int d);
fa_status fa_decode(const void* Q, const void* Kc, const void* Vc, const int* cache_seqlens,
                    void* O, float* L, void* workspace, size_t workspace_bytes, int B, int H,
                    int Hkv, int Nmax, int d, float scale, fa_dtype dtype, void* stream);

/* Split-KV decoding from 8-bit E4M3 caches with per-tensor descale factors: as
 * fa_decode, with Kc8 and Vc8 (B, Hkv, Nmax, d) holding one E4M3 code per value,
 * standing for k_scale * K and v_scale * V (the FP8 precision of the FlashAttention
 * note's FlashAttention-3 entry, "Versions and Evolution", applied to a decoding
 * cache).  The scores are formed in fp32 from the decoded codes and P stays fp32,
 * so only the cache is in 8 bits.  Q, O in fp16/bf16 (dtype), L fp32 as in
 * fa_decode; the workspace is fa_decode_workspace_size(B, H, Hkv, Nmax, d) bytes or
 * NULL.  d must be 128 (FA_ERR_UNSUPPORTED otherwise); k_scale and v_scale must be
 * positive and finite (FA_ERR_INVALID_VALUE); the other errors are fa_decode's. */
fa_status fa_decode_fp8(const void* Q, const void* Kc8, const void* Vc8, const int* cache_seqlens,
                        void* O, float* L, void* workspace, size_t workspace_bytes, int B, int H,
                        int Hkv, int Nmax, int d, float scale, float k_scale, float v_scale,
                        fa_dtype dtype, void* stream);

/* ---- Norms and rotation of query and key heads before attention.
 * What models do to queries and keys between the projection and fa_fwd (or fa_fwd_varlen), and its
 * gradient between fa_bwd and the projection's: each head x of d columns is divided by its root
 * mean square and weighted (norm), and the pairs of its first rot_dim columns turn by the
 * token's angles (rotary position embedding):
 *     z = x / sqrt(mean x^2 + eps) * w,      (a, b) -> (a cos - b sin, b cos + a sin).
 * Either may be left out.  fp32 arithmetic (a head whose mean of squares overflows fp32 is normed
 * to 0 or NaN), one rounding. */

/* Heads of a (B, heads, N, d) tensor: element (b, h, n, c) at
 * b * batch_stride + h * head_stride + n * row_stride + c (elements; a stride of a dimension of
 * extent 1 is not used).  So dense (B, heads, N, d), (B, N, heads, d), packed (total, heads, d)
 * with B = 1, and slices of one projection's output all fit.
 * zero_rest is of outputs: 1 writes zeros to the rows that the call leaves out (fa_rotation: those of
 * no sequence and those whose position lies outside the table), as a gradient that goes on to the
 * projection's has to have; any other value leaves them as they were. */
typedef struct fa_heads {
  void* data;
  long long batch_stride, head_stride, row_stride;
  int heads;
  int zero_rest;
} fa_heads;

/* Norm of query and key heads: weights w (d), fp32 (weights_fp32 = 1) or of the call's dtype, or NULL:
 * ones.  eps > 0. */
typedef struct fa_head_norm {
  const void* q_weight;
  const void* k_weight;
  int weights_fp32;
  float eps;
} fa_head_norm;

/* Where the angles of tokens come from.
 *   cos_sin      fp32 (max_pos, rot_dim), 16-byte aligned: row p holds cos, then sin, of rot_dim/2
 *                pair angles (scaled for long contexts or not: the table's values are used as they
 *                are).  Pair i is columns (i, i + rot_dim/2), with interleaved = 1 columns
 *                (2i, 2i + 1).  rot_dim a multiple of 16 in [0, d]; 0: no rotation.
 *   cu_seqlens   device int32 [n_seq + 1], or NULL.  With it B is 1 and the rows are packed
 *                sequences: sequence i has rows cu[i] .. cu[i+1]-1.  Rows of no sequence are left
 *                out: an output keeps what it held there (or gets zeros, fa_heads), and they
 *                have no part in the weights' gradients.
 *   positions    device int32, row n of batch entry b at b * positions_stride + n (0: the same
 *                for all entries), or NULL: the row's index in its batch entry or sequence.
 *   A row whose position lies outside the table is left out, too, and fa_device_status then
 *   reports FA_ERR_INVALID_VALUE. */
typedef struct fa_rotation {
  const float* cos_sin;
  int max_pos, rot_dim, interleaved;
  const int* cu_seqlens;
  int n_seq;
  const int* positions;
  long long positions_stride;
} fa_rotation;

/* Forward: q_out and k_out from q and k.  k and k_out may both be NULL.  norm and rot may be NULL.
 * An output may be its own input (same data and strides); otherwise outputs overlap nothing.  Views
 * that interleave without sharing an element do not, where they have a stride in common of which their
 * larger ones are multiples (slices of one projection); others are refused.
 *   Errors: FA_ERR_INVALID_VALUE for NULL pointers, B, N or heads < 1, q and q_out (k and k_out) of
 *   different heads, negative strides, outputs whose elements coincide or that overlap, a norm
 *   whose eps is not positive and finite, weights_fp32 or interleaved not 0/1, rot_dim > 0 without
 *   cos_sin or with max_pos < 1, cu_seqlens with n_seq < 1 or B > 1, a negative positions_stride;
 *   FA_ERR_UNSUPPORTED for d not 32/64/128, another dtype, rot_dim not a multiple of 16 in [0, d],
 *   B * N * heads >= 2^31, strides of 2^40 bytes or more, a view whose (extent - 1) * stride passes 2^46
 *   elements in any dimension, or positions_stride >= 2^40;
 *   FA_ERR_MISALIGNED for data, weights or cos_sin not 16-byte aligned, strides that are not
 *   multiples of 8 elements, or int arrays not 4-byte aligned.
 *   Asynchronous on `stream`; launches are not traced. */
fa_status fa_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* q_out,
                       const fa_heads* k_out, const fa_head_norm* norm, const fa_rotation* rot,
                       int B, int N, int d, fa_dtype dtype, void* stream);

/* Backward: dq and dk (gradients of q and k) from dq_out and dk_out (gradients of the forward's
 * outputs) and, with norm, the forward's inputs q and k, which are not read (and may be NULL)
 * without it.  With norm, dq_weight and dk_weight (fp32 (d), 4-byte aligned; each may be NULL) get
 * the weights' gradients, summed over all rows and heads in an order that depends on sizes alone.
 *   workspace    fa_norm_rope_bwd_workspace_size(d) bytes (16-byte aligned), or NULL: allocated
 *                and freed on `stream` if a weight's gradient is asked for; unused otherwise.  Its
 *                contents do not matter before a call; calls that may overlap need one each.
 *   dq may be dq_out or q itself, dk likewise.  Errors as for the forward, and
 *   FA_ERR_INVALID_VALUE for a short workspace, a weight's gradient without norm or without its heads,
 *   or weights' gradients or a workspace that overlap anything else; FA_ERR_MISALIGNED where they are
 *   not aligned as above. */
size_t fa_norm_rope_bwd_workspace_size(int d);
fa_status fa_norm_rope_bwd(const fa_heads* dq_out, const fa_heads* dk_out, const fa_heads* q,
                           const fa_heads* k, const fa_heads* dq, const fa_heads* dk,
                           const fa_head_norm* norm, const fa_rotation* rot, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes, int B, int N,
                           int d, fa_dtype dtype, void* stream);

/* ---- Paged key/value caches.
 * The caches of many sequences in one pool of equal pages (the FlashAttention note lists
 * inference serving with a KV cache, and paged attention by name, among the method's uses:
 * "Applications and Use Cases").  K and V are pools of `pages` pages, a page holding
 * page_size key rows of each of the Hkv K/V heads; key j of sequence b, head hk, column c is
 *     page p = page_table[b * table_stride + j / page_size], row r = j % page_size,
 *     element p * page_stride + hk * head_stride + r * row_stride + c,
 * the same strides (in elements, columns contiguous) for both pools, so (pages, Hkv,
 * page_size, d), (pages, page_size, Hkv, d) and halves of one common pool all fit.
 *   page_table     device int32 [B][max_pages], rows table_stride entries apart.  Pages may be
 *                  shared by sequences that only read them.
 *   cache_seqlens  device int32 [B]: keys of each sequence; a negative length is 0.  For the
 *                  calls that bring new tokens it counts these in: the new tokens are the
 *                  sequence's last keys.  Of a length beyond max_pages * page_size the keys
 *                  past the table do not exist, and the others keep their positions: new
 *                  tokens, queries and windows stand where the length puts them.
 *   A page id outside [0, pages) stands for an absent page: its keys are not attended (a
 *   sliding window's dropped pages may be marked -1); nothing outside the pools is touched.
 *   Supported: page_size >= 1 (even for d = 32), max_pages * page_size <= 2^30.
 *   Errors of every call that takes one: FA_ERR_INVALID_VALUE for NULL members, pages,
 *   page_size or max_pages < 1, table_stride < max_pages, or strides under which two elements
 *   of the pools would coincide; FA_ERR_MISALIGNED for pools not 16-byte aligned or strides
 *   that are not multiples of 16 bytes (dimensions of extent 1 excepted), or table or lengths
 *   not 4-byte aligned; FA_ERR_UNSUPPORTED beyond the limits above, or for strides of 2^40
 *   bytes or more. */
typedef struct fa_paged_cache {
  void* K;
  void* V;
  const int* page_table;
  const int* cache_seqlens;
  long long page_stride, head_stride, row_stride;
  long long table_stride;
  int pages, page_size, max_pages;
} fa_paged_cache;

/* Append: the keys and values of T new tokens go to their places in the paged cache, the
 * first rot_dim columns of keys turned by the position angles (rotary position embedding) on
 * the way; with Q, the same tokens' queries are turned too and written to Qout.
 *   K, V         (T, Hkv, d), tokens k_stride / v_stride elements apart, heads and columns
 *                contiguous (slices of one projection's output fit).  Q (T, H, d) likewise
 *                with q_stride; Qout dense (T, H, d).  Q and Qout may be NULL, both.
 *   cu_seqlens   device int32 [B+1]: sequence b brings tokens cu[b] .. cu[b+1]-1, its last
 *                keys: token t gets key position cache_seqlens[b] - (cu[b+1] - t).  NULL: one
 *                token per sequence (T = B).  Tokens before cu[0], at or past cu[B], or with a
 *                negative position (a sequence of length 0) are left out: nothing of theirs is
 *                written.
 *   cos_sin      fp32 (max_pos, rot_dim), 16-byte aligned: row p holds cos, then sin, of the
 *                rot_dim/2 pair angles of position p.  Pair i is columns (i, i + rot_dim/2),
 *                with interleaved = 1 columns (2i, 2i + 1); (x, y) becomes (x cos - y sin,
 *                y cos + x sin).  rot_dim = 0: no rotation (cos_sin unused, max_pos 0).
 *   positions    device int32 [T] to look angles up by, or NULL: key positions.
 *   A token whose angle position lies outside the table, or whose page is absent, is left out
 *   (its query too for the former), and fa_device_status then reports FA_ERR_INVALID_VALUE.
 *   Two new tokens must not fall on one cache row: it would hold pieces of both.
 *   Arithmetic in fp32, one rounding.
 *   Errors: as for the cache, FA_ERR_INVALID_VALUE for NULL K or V, one of Q and Qout alone,
 *   B, T or Hkv < 1, H not a multiple of Hkv, T != B without cu_seqlens, strides below a
 *   token's row, cos_sin NULL or max_pos < 1 with rot_dim > 0, interleaved not 0/1 or outputs
 *   that overlap inputs or each other; FA_ERR_UNSUPPORTED for d not 32/64/128, another dtype,
 *   rot_dim not a multiple of 16 in [0, d], or 2^31 or more blocks of work;
 *   FA_ERR_MISALIGNED for K, V, Q, Qout, cos_sin not 16-byte aligned, token strides that are
 *   not multiples of 8 elements, or int arrays not 4-byte aligned.  Asynchronous on `stream`.
 *   Launches of this call are not traced. */
fa_status fa_append_paged(const fa_paged_cache* cache, const void* K, long long k_stride,
                          const void* V, long long v_stride, const void* Q, long long q_stride,
                          void* Qout, const int* cu_seqlens, const int* positions,
                          const float* cos_sin, int max_pos, int rot_dim, int interleaved, int B,
                          int T, int H, int Hkv, int d, fa_dtype dtype, void* stream);

/* The same into pools of E4M3 codes standing for k_scale * K and v_scale * V: each code is
 * x * (1 / scale), the reciprocal in fp32, rounded to nearest even and saturated at +-448.
 * K, V, Q in fp16/bf16 (dtype); d must be 128 (FA_ERR_UNSUPPORTED); scales positive and
 * finite, with finite reciprocals (FA_ERR_INVALID_VALUE).  Pool strides count codes. */
fa_status fa_append_paged_fp8(const fa_paged_cache* cache, const void* K, long long k_stride,
                              const void* V, long long v_stride, const void* Q, long long q_stride,
                              void* Qout, const int* cu_seqlens, const int* positions,
                              const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                              int B, int T, int H, int Hkv, int d, float k_scale, float v_scale,
                              fa_dtype dtype, void* stream);

/* fa_append_paged and fa_append_paged_fp8 with the norm of fa_norm_rope: query and key heads are
 * normed before they turn (and are quantised); values are not.  Errors as there, with T * heads >= 2^31
 * of any of the tensors in the place of the blocks of work (FA_ERR_UNSUPPORTED), and those of a norm as
 * for fa_norm_rope; norm must not be NULL (FA_ERR_INVALID_VALUE). */
fa_status fa_append_paged_norm(const fa_paged_cache* cache, const void* K, long long k_stride,
                               const void* V, long long v_stride, const void* Q, long long q_stride,
                               void* Qout, const int* cu_seqlens, const int* positions,
                               const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                               const fa_head_norm* norm, int B, int T, int H, int Hkv, int d,
                               fa_dtype dtype, void* stream);
fa_status fa_append_paged_norm_fp8(const fa_paged_cache* cache, const void* K, long long k_stride,
                                   const void* V, long long v_stride, const void* Q,
                                   long long q_stride, void* Qout, const int* cu_seqlens,
                                   const int* positions, const float* cos_sin, int max_pos,
                                   int rot_dim, int interleaved, const fa_head_norm* norm, int B,
                                   int T, int H, int Hkv, int d, float k_scale, float v_scale,
                                   fa_dtype dtype, void* stream);

/* Decoding over a paged cache: one query row per (sequence, head) attends to the
 * cache_seqlens[b] keys of its sequence, or with window > 0 to the last `window` of them
 * (the query counts as the last key, as in fa_fwd_swa).  Split over the keys and merged as
 * fa_decode, with the ranges of the split cut from the lengths on the device, so that ragged
 * batches share the GPU evenly.  Results do not depend on timing.
 *   Q (B, H, d), O (B, H, d), L (B, H) as in fa_decode; a row without attended keys gets
 *   O = 0, L = -inf.
 *   workspace    fa_decode_paged_workspace_size(H, Hkv, d) bytes (16-byte aligned), or NULL:
 *                allocated and freed on `stream` if the call cuts rows (it does not where the
 *                table or the window keeps every row short).  Its contents do not matter
 *                before a call.
 *   Errors: as for the cache and fa_decode, FA_ERR_INVALID_VALUE for window < 0 or a scale
 *   that (times k_scale) overflows or vanishes in fp32, and
 *   FA_ERR_UNSUPPORTED for more than 4864 query heads per K/V head or for a table whose rows
 *   have room for about 2^44 bytes of keys together. */
size_t fa_decode_paged_workspace_size(int H, int Hkv, int d);
fa_status fa_decode_paged(const void* Q, const fa_paged_cache* cache, void* O, float* L,
                          void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int d,
                          int window, float scale, fa_dtype dtype, void* stream);

/* The same from pools of E4M3 codes (d = 128) standing for k_scale * K and v_scale * V. */
fa_status fa_decode_paged_fp8(const void* Q, const fa_paged_cache* cache, void* O, float* L,
                              void* workspace, size_t workspace_bytes, int B, int H, int Hkv,
                              int d, int window, float scale, float k_scale, float v_scale,
                              fa_dtype dtype, void* stream);

/* Forward of many new tokens over a paged cache (a prompt, a later part of one, or drafted
 * tokens): sequence b holds query rows cu_seqlens[b] .. cu_seqlens[b+1]-1 of the packed Q, the
 * positions of its last keys (fa_append_paged has put the tokens' keys there): with nq query
 * rows and nk = cache_seqlens[b] keys, causal query i sees keys j <= nk - nq + i, and with
 * window > 0 of those the last `window`; not causal: all nk keys.
 *   Layout   Q, O (total, H, d); L (H, total) as in fa_fwd_varlen; cu_seqlens, total and
 *            max_seqlen too (offsets that break its rules leave rows uncomputed: of a sequence
 *            longer than max_seqlen those past it).  Rows of no
 *            sequence are left as they were.  A row without keys gets O = 0, L = -inf.
 *   workspace  fa_fwd_paged_workspace_size(B, max_seqlen, H, Hkv, d) bytes (16-byte
 *            aligned), or NULL: allocated and freed on `stream`.  0 bytes, and then unused,
 *            where there are query rows enough to fill the GPU without splitting the keys.  Its
 *            contents do not matter before a call.
 *   The softmax weights are rounded to `dtype` before their product with V, as in fa_fwd (the
 *   decoding calls keep twice the bits).
 *   A V element that is not finite reaches the query rows of its 128-key tile that have keys even
 *   where the causal mask or the window hides its key (0 x NaN), as in fa_fwd; what lies in absent
 *   pages and past the last key never does, and rows without keys are 0 whatever the tile holds.
 *   Errors   as for the cache and fa_fwd_varlen, FA_ERR_INVALID_VALUE for a scale that times
 *            log2(e) overflows or vanishes in fp32; FA_ERR_UNSUPPORTED for more than 2^29 rows of
 *            one sequence's heads that share a tile (max_seqlen times the largest power of two
 *            that divides H / Hkv, at most 128) or 2^31 or more query tiles. */
size_t fa_fwd_paged_workspace_size(int B, int max_seqlen, int H, int Hkv, int d);
fa_status fa_fwd_paged(const void* Q, const fa_paged_cache* cache, void* O, float* L,
                       void* workspace, size_t workspace_bytes, const int* cu_seqlens, int B,
                       int total, int max_seqlen, int H, int Hkv, int d, int causal, int window,
                       float scale, fa_dtype dtype, void* stream);

/* The same from pools of E4M3 codes (d = 128) standing for k_scale * K and v_scale * V: prompts and
 * drafts of a model whose cache fa_append_paged_fp8 writes and fa_decode_paged_fp8 reads.  Keys and
 * values are used as their codes stand; queries are not quantised (a bf16 value below 2^-28 of its
 * row's largest loses bits) and the softmax weights are rounded to fp16 for either dtype
 * (fa_decode_paged_fp8 keeps twice the bits: a draft is checked a little more coarsely than its tokens
 * would be decoded one by one; fp16 results are off by 1.4 times their own rounding).  Workspace and
 * errors as for fa_fwd_paged, with fa_decode_paged_fp8's for the scales. */
fa_status fa_fwd_paged_fp8(const void* Q, const fa_paged_cache* cache, void* O, float* L,
                           void* workspace, size_t workspace_bytes, const int* cu_seqlens, int B,
                           int total, int max_seqlen, int H, int Hkv, int d, int causal, int window,
                           float scale, float k_scale, float v_scale, fa_dtype dtype, void* stream);

/* Static description of a status code. */
const char* fa_status_string(fa_status s);

/* CUDA error code (a cudaError_t value) behind the last FA_ERR_CUDA returned on
 * the calling thread; 0 if none. */
int fa_last_cuda_error(void);

/* Synchronises `stream`, then reads and clears the current device's status
 * word: FA_ERR_TIMEOUT if any kernel of this library gave up a bounded wait
 * since the last read; FA_ERR_UNSUPPORTED if a kernel found its dynamic shared
 * memory not aligned to 1024 bytes and skipped its work (not expected on
 * sm_103a); FA_ERR_INVALID_VALUE if an append or a rotation left out a token whose page
 * or angle position lies outside its tensors; FA_OK otherwise (FA_ERR_CUDA if the read failed). */
fa_status fa_device_status(void* stream);

/* Bound, in nanoseconds, on any single wait inside the kernels (default 2 s).
 * ns == 0 restores the default.  Applies to launches made after the call. */
fa_status fa_set_wait_limit_ns(unsigned long long ns);

/* Failure-detection self test: launches one CTA that waits on a barrier nothing
 * will complete, bounded by `limit_ns`; the kernel records a timeout and exits.
 * Synchronises `stream` and returns what fa_device_status then reports
 * (FA_ERR_TIMEOUT when the bound works).  Faults nothing. */
fa_status fa_selftest_timeout(unsigned long long limit_ns, void* stream);

/* Per-kernel timing trace (the method's own benchmark harness measures speed
 * and TFLOP/s: docs page, "Scope" and Table 3).  While enabled, every kernel
 * launch of this library is bracketed by two CUDA events recorded on its
 * stream, from a fixed pool of 4096 launches (later launches are not traced).
 * fa_trace_enable(1) (re)starts recording and clears earlier records (the
 * first call creates the events); fa_trace_enable(0) stops it.  Not
 * thread-safe: trace from one host thread. */
fa_status fa_trace_enable(int on);

/* Name of trace kind `kind` (0: forward kernel, 1: backward pre-pass, 2:
 * backward dK/dV kernel, 3: backward dQ kernel, 4: decode split kernel, 5:
 * decode merge kernel, 6: FP8 forward kernel); NULL when out of range.  The calls on
 * paged caches count under the kinds of their dense counterparts (0, 4, 5); the kernels of
 * fa_append_paged and fa_norm_rope and the join of fa_fwd_paged's key ranges are not traced. */
const char* fa_trace_kind_name(int kind);

/* Waits for the recorded events of kind `kind`, then writes the summed GPU
 * time in milliseconds and the number of traced launches. */
fa_status fa_trace_read(int kind, double* total_ms, long long* launches);

/* Backward that allocates nothing.  The pages have no counterpart: this entry
 * exists for callers, not for the method.  Some callers cannot call cudaMalloc
 * at all -- a plugin inside a host framework that owns every byte of device
 * memory, or a deployment handed a fixed memory budget up front -- and fa_bwd
 * either takes a caller workspace or allocates one.  fa_bwd_noalloc computes
 * what fa_bwd computes, with the same arguments minus the workspace.  Its
 * scratch is a 16 MiB device array inside the library, held by every GPU that
 * loads the library until the process exits; sizes whose scratch need
 * (fa_bwd_workspace_size) exceeds 16 MiB are rejected with FA_ERR_UNSUPPORTED
 * before anything is launched.  The first call in a CUDA context looks up the
 * array's device address there (cudaGetSymbolAddress, with the caller's device and
 * context current; a context destroyed and recreated, e.g. by cudaDeviceReset, is
 * looked up again); make that first call before any stream capture.  The lookup is
 * guarded by a lock, so first calls from several host threads are safe.  All
 * calls share the one array and it keeps the last call's contents: calls that
 * overlap on the GPU (other streams, other host threads) race on it, so
 * serialise them.  Nothing in it
 * needs to start at zero: each call writes every scratch value before reading
 * it.  Capacity: 8 bytes per row, B*H*ceil(N/128)*128 up to 2,097,152 rows. */
fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* L, void* dQ, void* dK, void* dV, int B,
                         int H, int N, int d, int causal, float scale, fa_dtype dtype,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
