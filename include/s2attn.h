/*
 * s2attn.h -- C ABI of the B200 (sm_100a) shifted-short-attention library.
 *
 * The operation (LongLoRA's S^2-Attn, as described on the LongLoRA pages):
 *   - "LongLoRA paper notes" (smallflyingpig blog), section 3.3: a sequence of
 *     length N is cut into groups of G tokens and attention runs only inside each
 *     group, lowering the cost from O(N^2) to O(N^2 / (N/G)); a shifted pattern moves
 *     the groups by half a group so that information crosses group borders
 *     (drawing: groups 1-4, 5-8, 9-12 become 3-6, 7-10, 11-14).
 *   - "LLaMA2 context to 100k" (nearauto.com), section on shift short attention:
 *     two steps, (1) shift the tokens in half of the attention heads, (2) move the
 *     features from the token dimension into the batch dimension.
 *   - python88.com article, mechanism paragraph: the heads are split into two halves
 *     and shifting one half lets neighbouring groups exchange information.
 *   - "LongLoRA paper notes", section 3.1, and the model page (model.aibase.cn),
 *     features list: inference uses ordinary full attention.
 * Precisely, with scale = 1/sqrt(D) and shift s_h = G/2 for heads
 * h >= H - shift_heads (0 otherwise): rolled row r of head h holds original token
 * (r + s_h) mod N; group j owns rolled rows [jG, (j+1)G); query row r attends to the
 * rolled rows r' of its own group with r' <= r (causal, in rolled order); the result
 * of rolled row r is stored back at its original token.  G = N with shift_heads = 0
 * is full causal attention (the inference case).
 *
 * Conventions for every entry point:
 *   - Tensors are dense row-major [B, N, H, D] ("token-major"); lse and delta are
 *     [B, H, N] fp32, indexed by ORIGINAL token.
 *   - Every pointer is a device pointer owned by the caller, 16-byte aligned; the
 *     library never frees or keeps caller memory.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls only
 *     enqueue work and return; nothing synchronizes.
 *   - Return value: S2ATTN_OK or a negative s2attn_status.  Argument errors are
 *     detected on the host before anything is enqueued.  A failure inside a kernel
 *     (a bounded wait that timed out) is recorded in a per-device error word that
 *     s2attn_get_device_error() reads after the caller synchronizes.
 *   - The calls are thread-safe with respect to each other.
 */
#ifndef S2ATTN_H_
#define S2ATTN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  S2ATTN_OK = 0,
  S2ATTN_ERR_INVALID_ARG = -1,    /* bad shape, null or misaligned pointer */
  S2ATTN_ERR_UNSUPPORTED = -2,    /* valid, but not a shape this path handles */
  S2ATTN_ERR_WORKSPACE = -3,      /* workspace missing or too small */
  S2ATTN_ERR_CUDA = -4,           /* a CUDA runtime/driver call failed */
  S2ATTN_ERR_DEVICE_TIMEOUT = -5, /* a kernel gave up on a bounded wait */
  S2ATTN_ERR_DEVICE_INDEX = -6    /* a length, page, row or parent held on the device is out of range */
} s2attn_status;

/* Element types of the calls that take a `dtype`. */
typedef enum { S2ATTN_BF16 = 0, S2ATTN_FP16 = 1, S2ATTN_F32 = 2 } s2attn_dtype;

/* Version of this ABI (major * 100 + minor). */
int s2attn_version(void);

/* Human-readable name of a status code (static string). */
const char* s2attn_status_string(int status);

/*
 * Forward pass, bf16 in / bf16 out, fp32 accumulation (tcgen05 tensor cores).
 *   q, k, v : [B,N,H,D] bf16 inputs
 *   o       : [B,N,H,D] bf16 output (attention output at each original token)
 *   lse     : [B,H,N] fp32 output, natural log of sum over visible keys of exp(scale*q.k)
 * Requirements: D == 128; G >= 1 divides N; 0 <= shift_heads <= H; G % 128 == 0;
 * if shift_heads > 0 then (G/2) % 128 == 0.  Other valid shapes return
 * S2ATTN_ERR_UNSUPPORTED (the fp32 entry points take any valid shape).
 */
int s2attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int N, int H, int D, int G,
               int shift_heads, void* stream);

/* Bytes of device workspace s2attn_bwd needs: an fp32 dQ accumulator [B,N,H,D]
 * followed by delta [B,H,N] fp32 (each start 256-byte aligned).  0 on bad sizes. */
size_t s2attn_bwd_workspace_bytes(int B, int N, int H, int D);

/*
 * Backward pass, bf16, same shape rules as s2attn_fwd.  Inputs: q, k, v, the
 * forward output o and lse, and the output gradient dout.  Outputs dq, dk, dv
 * ([B,N,H,D] bf16).  `workspace` (device, caller-owned, >= the size above,
 * 256-byte aligned) is overwritten.  Runs s2attn_bwd_preprocess, s2attn_bwd_main
 * and s2attn_bwd_dq_convert in that order on `stream`.
 */
int s2attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
               void* dq, void* dk, void* dv, int B, int N, int H, int D, int G, int shift_heads, void* workspace,
               size_t workspace_bytes, void* stream);

/* Backward stage 1: delta[b,h,t] = sum_d dout[b,t,h,d] * o[b,t,h,d] (fp32, delta is
 * [B,H,N]) and dq_acc ([B,N,H,D] fp32) := 0.  D must be 128. */
int s2attn_bwd_preprocess(const void* o, const void* dout, float* delta, float* dq_acc, int B, int N, int H, int D,
                          void* stream);

/* Backward stage 2 (tensor cores): writes dk, dv (bf16) and adds the unscaled
 * dQ = dS K into dq_acc (fp32, zeroed by stage 1).  Same shape rules as s2attn_fwd. */
int s2attn_bwd_main(const void* q, const void* k, const void* v, const void* dout, const float* lse,
                    const float* delta, float* dq_acc, void* dk, void* dv, int B, int N, int H, int D, int G,
                    int shift_heads, void* stream);

/* Backward stage 3: dq = bf16(dq_acc / sqrt(D)), round to nearest even. */
int s2attn_bwd_dq_convert(const float* dq_acc, void* dq, int B, int N, int H, int D, void* stream);

/*
 * Decoding step of full causal attention (inference).  Inference runs ordinary
 * full attention, not S^2-Attn ("LongLoRA paper notes", section 3.1; model.aibase.cn,
 * features list: the shifted attention is only needed in training).  A step appends
 * M new tokens to a sequence of N positions:
 *   q    : [B,M,H,D] bf16, the new queries; query m sits at position N-M+m
 *   k, v : [B,N,H,D] bf16, all N positions (the M new ones included)
 *   o    : [B,M,H,D] bf16 output; query m attends to the keys at positions
 *          0 .. N-M+m with scale 1/sqrt(D)
 *   lse  : [B,H,M] fp32 output, natural log of sum over those keys of exp(scale*q.k)
 * Requirements: 1 <= M <= N; M <= 128 and D == 128 (else S2ATTN_ERR_UNSUPPORTED).
 * One query runs on CUDA cores (HBM-bound matrix-vector work); 2..128 queries run one
 * 128-row query tile on the tensor cores (speculative decoding, chunked prefill).
 * `workspace` (device, caller-owned, 256-byte aligned, at least
 * s2attn_decode_workspace_bytes bytes) receives per-split partial results and is
 * overwritten; its size holds fp32 partials (D outputs, max, sum per query) of at most
 * min(64, ceil(N/64)) splits per (b, h), independent of the device; 0 means invalid sizes.
 * V rows past a query's causal limit are multiplied by a zero weight, so k and v must hold
 * finite values at every position.  Runs two kernels on `stream`; the second (the split
 * combine) is a programmatic dependent launch that waits on the device for the first.
 */
size_t s2attn_decode_workspace_bytes(int B, int M, int N, int H, int D);
int s2attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int M, int N, int H,
                  int D, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Halo rows of sequence-sharded S^2-Attn.  The groups are independent, so a sequence
 * split across ranks in whole groups needs one exchange ("LongLoRA paper notes",
 * section 3.3; nearauto.com article, "shift short attention" steps (1) and (2)).  A
 * rank holding tokens [t0, t0+N) of every head (N a multiple of G) runs the forward and
 * backward above on its own tensors with the shift; their last rolled group of a
 * shifted head reads the rank's tail and then its rows [0, G/2).  Those rows of the
 * shifted heads belong to the previous rank's last group, so the sharded path swaps the
 * next rank's first G/2 rows (the halo) into them for the duration of the calls and
 * swaps them back afterwards; the results written to them belong to the halo's tokens
 * and are returned to their owner.  These two calls are the copies that swap needs:
 *   s2attn_halo_rows: for each of n_tensors bf16 [B,N,H,D] tensors x[i] and contiguous
 *     buffers buf[i] [B, G/2, shift_heads, D]:  to_buf != 0: buf[i][b,r,s,:] =
 *     x[i][b, r, H-shift_heads+s, :] for r < G/2;  to_buf == 0: the reverse copy.
 *   s2attn_halo_lse: the same rows of fp32 [B,H,N] tensors (lse, softmax statistics),
 *     buffers [B, shift_heads, G/2].
 * x and buf are host arrays of n_tensors device pointers (1 <= n_tensors <= 8), bf16
 * pointers 16-byte aligned (lse pointers 4-byte aligned), owned by the caller.
 * Requirements: G divides N, G even, 1 <= shift_heads <= H, D*2 a multiple of 16.
 * One kernel launch per call on `stream`; buffers and tensors must not overlap.
 */
int s2attn_halo_rows(void* const* x, void* const* buf, int n_tensors, int to_buf, int B, int N, int H, int D,
                     int G, int shift_heads, void* stream);
int s2attn_halo_lse(float* const* lse, float* const* buf, int n_tensors, int to_buf, int B, int N, int H, int G,
                    int shift_heads, void* stream);

/*
 * fp32 forward/backward on CUDA cores, any valid shape with 1 <= D <= 128
 * (G >= 1 divides N; G even when shift_heads > 0).  Same tensor layouts, all fp32.
 * s2attn_bwd_f32 uses the delta part of the workspace only
 * (size from s2attn_bwd_workspace_bytes).
 */
int s2attn_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B, int N, int H, int D,
                   int G, int shift_heads, void* stream);
int s2attn_bwd_f32(const float* q, const float* k, const float* v, const float* o, const float* dout,
                   const float* lse, float* dq, float* dk, float* dv, int B, int N, int H, int D, int G,
                   int shift_heads, void* workspace, size_t workspace_bytes, void* stream);

/*
 * RoPE with position interpolation ("LongLoRA paper notes", section 3.4: positions
 * [0, L) are squeezed into [0, L0)), applied in place to bf16 q and k ([B,N,H,D]).
 * Token t is rotated as if at position t * pos_scale (pos_scale = L0 / N).  Element
 * i < D/2 pairs with element i + D/2; the pair turns by angle a = (t*pos_scale) *
 * theta_i with theta_i = base^(-2i/D).  Evaluation order (bit-for-bit contract):
 *   theta_i = (float) pow(base, -2i/D) in double;  a = ((float)t * pos_scale) * theta_i
 *   in float;  c, s = (float) cos/sin((double) a);  y1 = x1*c - x2*s;  y2 = x2*c + x1*s,
 *   every product and sum rounded to fp32, then rounded to bf16 (nearest even).
 * The cos/sin table is computed on the host on first use of each (device, N, D,
 * pos_scale, base) and cached in device memory owned by the library until exit.
 * Either q or k may be NULL.  Requires D % 16 == 0, D <= 256.
 * Backward: with -pos_scale every angle is negated exactly (the products above round
 * symmetrically, cos is even and sin odd), which applies the transposed rotation -- the
 * gradient through RoPE-PI -- to dq and dk in the same operation order.
 */
int rope_pi_apply(void* q, void* k, int B, int N, int H, int D, float pos_scale, float base, void* stream);

/*
 * RoPE-PI as above for tensors whose row t is the token at position pos0 + t: the new
 * tokens of a decoding step (q and the k rows appended to the cache sit at positions
 * N_cache - M .. N_cache - 1).  Identical, bit for bit, to rows pos0 .. pos0+N-1 of
 * rope_pi_apply over the whole sequence (same operation order and table entries).
 * Requires pos0 >= 0 and pos0 + N <= 2^24.  The table is built on the host and cached in
 * device memory for the next power of two >= pos0 + N positions (at least 1024): D*4 bytes
 * per position, 64 MB for 128k positions at D = 128.
 */
int rope_pi_apply_offset(void* q, void* k, int B, int N, int H, int D, int pos0, float pos_scale, float base,
                         void* stream);

/*
 * RMS norm of every q and k head with the rotary embedding, in one pass.  For a head's row x
 * of D elements at position t (norm != 0; without it y = x):
 *   y = w * x / sqrt(mean(x^2) + eps)
 * and the first R elements of y turn in pairs by the angles t * inv_freq[i], i < R/2:
 *   (a, b) -> attn_factor * (a cos - b sin, b cos + a sin)
 * with pairs (i, i + R/2), or (2i, 2i + 1) when interleaved != 0; the other D - R pass.
 *   q, q_out : [B, N, Hq, D]     k, k_out : [B, N, Hk, D]   (q or k with its output may be NULL)
 *   wq, wk   : [D] weights of dtype, NULL for 1
 *   positions: [B, N] int32, any value, or NULL: row t of every sequence is at pos0 + t
 *   inv_freq : [R/2] fp32 frequencies (device), e.g. from rope_inv_freq
 * dtype: S2ATTN_BF16, S2ATTN_FP16 or S2ATTN_F32.  Sums and products are fp32, angles are formed and reduced in
 * 64 bits, the result is rounded once.  q_out == q and k_out == k (in place) are allowed; other overlaps are
 * not.  Requirements: D % 16 == 0, D <= 256; R % 16 == 0, 0 <= R <= D; Hq, Hk <= 16384; B * N < 2^30; pos0 + N
 * < 2^31; eps >= 0; a row's sum of squares within fp32; device pointers 16-byte aligned (positions and inv_freq 4-byte).
 */
int qk_norm_rope_fwd(const void* q, const void* k, const void* wq, const void* wk, const int* positions,
                     const float* inv_freq, void* q_out, void* k_out, int B, int N, int Hq, int Hk, int D, int R,
                     int interleaved, int norm, float eps, float attn_factor, int pos0, int dtype, void* stream);

/*
 * Backward of qk_norm_rope_fwd: dq, dk (of dtype) from the gradients dq_out, dk_out and the
 * forward's inputs q, k (not read, and may be NULL, when norm == 0), and dwq, dwk [D] of dtype
 * (either may be NULL: not wanted; both must be NULL when norm == 0).  dw is the fp32 sum over
 * all tokens and heads, added in an order that depends on the sizes and the device alone.
 * dq == dq_out and dk == dk_out are allowed.  `workspace`: device, 256-byte aligned, at
 * least qk_norm_rope_bwd_workspace_bytes(D) bytes, one per call that may overlap on the GPU; may be NULL
 * when dwq and dwk are.
 */
size_t qk_norm_rope_bwd_workspace_bytes(int D);
int qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, const void* wq,
                     const void* wk, const int* positions, const float* inv_freq, void* dq, void* dk, void* dwq,
                     void* dwk, int B, int N, int Hq, int Hk, int D, int R, int interleaved, int norm, float eps,
                     float attn_factor, int pos0, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotary frequencies for a context stretched by `factor` (host arrays; no GPU is used):
 * inv_freq[0 .. R/2) and *attn_factor.  With f_i = base^(-2i/R):
 *   scaling 0: f_i.   1 (position interpolation): f_i / factor.
 *   2 (a larger base): the base becomes base * factor^(R / (R - 2)).
 *   3 (by wavelength): frequencies that turn more than beta_fast times within original_len
 *     tokens stay, those below beta_slow are divided by factor, with a linear ramp over i
 *     between lo = max(0, floor(i_fast)) and hi = min(R - 1, ceil(i_slow)),
 *     i_n = R ln(original_len / (2 pi n)) / (2 ln base) (hi <= lo: a step behind lo; hi may lie
 *     behind the last frequency); *attn_factor = 0.1 ln(factor) + 1.
 * *attn_factor is 1 otherwise.  Requirements: R even, 2 <= R <= 256 (R >= 4 for scaling 2);
 * base > 1; factor >= 1; for scaling 3 original_len >= 1 and beta_fast > beta_slow > 0.
 */
int rope_inv_freq(float* inv_freq, float* attn_factor, int R, float base, int scaling, float factor,
                  int original_len, float beta_fast, float beta_slow);

/*
 * The paged cache of the calls below.  k_pages and v_pages are pools [n_pages, page_size, Hkv, D];
 * row b of page_table ([B, table_width] int32) lists the pages of sequence b in order, so
 * its token t lies in page page_table[b][t / page_size] at row t % page_size.  cache_len ([B]
 * int32) counts its tokens.  Entries behind the last token's page are never read.
 * page_size is a power of two >= 16; n_pages * page_size <= 2^31 - 256.
 * Lengths, pages, rows and parents are read on the device: one that is out of range is
 * recorded (s2attn_get_device_error returns S2ATTN_ERR_DEVICE_INDEX until cleared) and faults
 * nothing; the outputs of the sequence that holds it are then unspecified, those of others
 * are not affected, and later calls run.
 */

/*
 * Ancestor masks of trees of drafted tokens: parents [B, M] int32, parents[b][m] < m or -1
 * for a node that follows the cache directly.  mask [B, M, ceil(M/64)] 64-bit words: bit j%64
 * of word j/64 of row m is set where j is m or one of its ancestors.  depth ([B, M] int32, may
 * be NULL): the number of m's ancestors, so that m's position is cache_len + depth.
 * 1 <= M <= 128 (else S2ATTN_ERR_UNSUPPORTED).  A parent outside [-1, m) is recorded and
 * read as -1.
 */
int s2attn_tree_mask(const int* parents, unsigned long long* mask, int* depth, int B, int M, void* stream);

/*
 * Attention of M drafted tokens of each sequence over its paged cache and over each other, with
 * scale 1/sqrt(D): a decoding step for one token (M = 1), several in a row (mask NULL), or a tree.
 *   q            : [B, M, H, D]; query heads [g*H/Hkv, (g+1)*H/Hkv) use key head g
 *   k_new, v_new : [B, M, Hkv, D], the drafted tokens' keys and values
 *   tree_mask    : [B, M, ceil(M/64)] words as above, any bits; NULL: token m sees j <= m
 *   new_len      : [B] int32 in 0..M, or NULL for M: sequence b has new_len[b] drafted tokens
 *   o            : [B, M, H, D];  lse: [B, H, M] fp32, natural log of the sum of exp(score)
 * Token m of sequence b attends to the cache's cache_len[b] tokens and to the drafted tokens j < new_len[b]
 * whose bit is set in its mask row.  Rows m >= new_len[b] of o and lse are left as they were.  A token that
 * sees nothing gets o = 0 and lse = -inf.  What is not visible to a token does not reach it, whatever it holds
 * (infinities and NaN included).  A visible key of score -inf has weight 0; a token whose scores are all -inf
 * gets o = 0 and lse = -inf too.
 * dtype: S2ATTN_BF16 or S2ATTN_FP16.  Scores and sums are fp32; P is rounded to dtype for the second product
 * (in fp16 what is below 2^-36 of a row's largest weight is lost there).
 * Requirements: Hkv divides H, H/Hkv <= 128; D 64 or 128, M <= 128, B <= 1024, B * M * H < 2^31 and
 * B * (table_width * page_size / 64 + 16) < 2^30 (else S2ATTN_ERR_UNSUPPORTED).  `workspace` (device, 256-byte
 * aligned, at least s2attn_tree_decode_workspace_bytes bytes) is overwritten: calls that may overlap on the
 * GPU need one each.  Lengths are read on the device only, so a captured call follows them; they must not
 * change while it runs.  o and lse must not overlap the inputs.  Runs up to two kernels on `stream`.  Repeated
 * calls give the same bits; the lengths of a batch decide where a sequence's keys are cut, so its last bits
 * may differ between batches.
 */
size_t s2attn_tree_decode_workspace_bytes(int B, int M, int H, int Hkv, int D);
int s2attn_tree_decode(const void* q, const void* k_new, const void* v_new, const void* k_pages,
                       const void* v_pages, const int* page_table, const int* cache_len, const int* new_len,
                       const unsigned long long* tree_mask, void* o, float* lse, int B, int M, int H, int Hkv, int D,
                       int n_pages, int page_size, int table_width, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Writes rows of k_new and v_new ([B, M, Hkv, D]) into the pages of their sequences: for j < n_rows[b], row
 * rows[b][j] goes to position cache_len[b] + j.  rows [B, A] int32 (any order, repeats allowed); NULL: row j,
 * A = M.  n_rows [B] int32 (values above A count as A, below 0 as 0); NULL: A.  cache_len is not changed.
 * k_new and v_new must not overlap the pools.  elem_size: bytes of an element (2 or 4); Hkv * D * elem_size
 * must be a multiple of 16, at most 2^20, and B * M and B * A below 2^30 (else S2ATTN_ERR_UNSUPPORTED).  No
 * two sequences may own the same page at a position that is written.
 */
int s2attn_cache_append(const void* k_new, const void* v_new, void* k_pages, void* v_pages, const int* page_table,
                        const int* cache_len, const int* rows, const int* n_rows, int B, int M, int A, int Hkv, int D,
                        int n_pages, int page_size, int table_width, int elem_size, void* stream);

/*
 * Copies whole pages inside each of n_pools pools (1 .. 128 device pointers in a host array;
 * e.g. the K and V pools of every layer): page pairs[2i] to page pairs[2i + 1].  Used to fork a
 * sequence (its last, partly filled page gets a copy; full pages are shared by the tables) and
 * to move pages.  pairs is a host array, checked before anything is enqueued: pages in
 * [0, n_pages), no page written twice, none both read and written (S2ATTN_ERR_INVALID_ARG).
 * One page may be read several times.  page_bytes: bytes of a page, a multiple of 16, at most 2^40.
 * n_pairs = 0 does nothing.
 */
int s2attn_cache_copy_pages(void* const* pools, int n_pools, const int* pairs, int n_pairs, int n_pages,
                            size_t page_bytes, void* stream);

/*
 * LoRA-adapted linear projections, the steps on either side of S^2-Attn in a LongLoRA
 * layer ("LongLoRA paper notes", section 3.2: low-rank adapters on the Q, K, V and O
 * projections; nearauto.com article, "long-context LoRA improvement").  For `parts`
 * projections stacked along the output (3 for q, k, v; 1 for o), part p computes
 *   y[p] = x W_p^T + scaling * (x A_p^T) B_p^T
 * and the first `rope_parts` parts are then rotated by RoPE-PI, so q and k come out ready
 * for s2attn_fwd.  All bf16, accumulated in fp32 on the tensor cores:
 *   x      : [T, K], T = B*seq_len tokens (row t is position t mod seq_len)
 *   w      : [parts*n_out, K], the frozen weights (the layout of a linear layer's weight)
 *   lora_a : [parts*r, K], the adapters' down projections (NULL when r == 0)
 *   lora_b : [parts*n_out, r], the adapters' up projections (NULL when r == 0)
 *   y      : [parts, T, n_out] output; y[p] is a contiguous [B, seq_len, H, D] tensor when
 *            n_out = H*D, so q, k and v need no copy before attention
 * Rounding: the rank-r intermediate is held in bf16 after scaling, bf16(scaling * x A_p^T),
 * and y is rounded once (nearest even) from the fp32 accumulator.  With rope_parts > 0,
 * the rotated parts are bit-identical to this call with rope_parts = 0 followed by
 * rope_pi_apply(y[p], ..., B, seq_len, n_out/head_dim, head_dim, pos_scale, base) on
 * each: the same table (cached per device, seq_len, head_dim, pos_scale, base) and the
 * same fp32 operation order, applied to the bf16-rounded projection.  As for rope_pi_apply,
 * the first call with a new table builds it on the host and copies it synchronously; make
 * that call before any stream capture.
 * Requirements: K >= 8 and K % 8 == 0; 0 <= r <= 64; 0 <= rope_parts <= parts;
 * n_out % 256 == 0 and K >= 64 (else S2ATTN_ERR_UNSUPPORTED); x, w, y, lora_a 16-byte aligned; with
 * rope_parts > 0: head_dim in {32, 64, 128, 256}, T % seq_len == 0, base > 0.
 * `workspace` (device, caller-owned, 256-byte aligned, at least
 * lora_proj_workspace_bytes(T, K, n_out, parts, r) bytes; may be NULL when r == 0) holds the
 * zero-padded adapters and the intermediate and is overwritten.  Runs up to three kernels
 * on `stream` (adapter padding, the rank-r down projection, the projection); invalid
 * arguments return before any launch.
 */
size_t lora_proj_workspace_bytes(int T, int K, int n_out, int parts, int r);
int lora_proj_fwd(const void* x, const void* w, const void* lora_a, const void* lora_b, void* y, int T, int K,
                  int n_out, int parts, int r, float scaling, int rope_parts, int head_dim, int seq_len,
                  float pos_scale, float base, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of lora_proj_fwd for training (the frozen W gets no gradient; notes section 3.2):
 *   dx       = sum_p dy_p W_p + s (dy_p B_p) A_p           [T, K]
 *   d_lora_a = per part, s (dy_p B_p)^T x                  [parts*r, K]
 *   d_lora_b = per part, s dy_p^T (x A_p^T)                [parts*n_out, r]
 * dy [parts, T, n_out] is the gradient of y before RoPE: take dq and dk back through the
 * rotation first with rope_pi_apply(dq, dk, ..., -pos_scale, ...).  Same layouts and
 * requirements as lora_proj_fwd (K >= 64, n_out % 256 == 0, r <= 64); d_lora_a / d_lora_b may be
 * NULL when r == 0.  `workspace` (device, caller-owned, 256-byte aligned, at least
 * lora_proj_bwd_workspace_bytes bytes) holds the padded adapters, the recomputed intermediate
 * s x A^T, s dy B, and fp32 accumulators for the adapter gradients.  The adapter gradients add
 * fp32 partial sums over token ranges, so they are not bitwise reproducible run to run.
 */
size_t lora_proj_bwd_workspace_bytes(int T, int K, int n_out, int parts, int r);
int lora_proj_bwd(const void* x, const void* w, const void* lora_a, const void* lora_b, const void* dy, void* dx,
                  void* d_lora_a, void* d_lora_b, int T, int K, int n_out, int parts, int r, float scaling,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass that allocates nothing.  The LongLoRA pages have no counterpart of
 * this entry point; it exists for callers that cannot allocate device memory on
 * the call path (a runtime whose allocator already holds the device's memory, a
 * plugin whose enqueue step must not allocate, or a latency-critical loop that
 * cannot afford cudaMalloc's implicit device synchronisation) and so cannot hand
 * s2attn_bwd a workspace.
 * Same arguments, shape rules and results as s2attn_bwd, minus the workspace: the
 * fp32 dQ accumulator and delta live in a fixed array of
 * S2ATTN_NOALLOC_SCRATCH_BYTES in the library's device memory, held until the
 * process exits.  The array is reserved when the module holding it is loaded on a
 * device; with CUDA's lazy module loading (the default) that happens inside the
 * first call on each device, which looks up the array's device address (with that
 * device current) and caches it.  So the first call on a device does take
 * S2ATTN_NOALLOC_SCRATCH_BYTES of device memory: make it before the caller's own
 * allocator reserves the device (else it fails with S2ATTN_ERR_CUDA) and before any
 * stream capture.  Later calls take no device memory.
 * Problems needing more (B*N*H*D*4 + B*H*N*4 bytes, each part rounded up to 256)
 * return S2ATTN_ERR_WORKSPACE; at D = 128 that is about 130k (token, head) rows.
 * Every call uses the same array and leaves its last contents there (the
 * accumulator is zeroed at the start of each call): calls whose work overlaps on
 * the GPU -- on different streams, or on different host threads -- race on it.
 * Calls no cudaMalloc, cudaFree or other allocating routine.
 */
#define S2ATTN_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
int s2attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                       const float* lse, void* dq, void* dk, void* dv, int B, int N, int H, int D, int G,
                       int shift_heads, void* stream);

/*
 * Reads the current device's error word: S2ATTN_OK if no kernel has failed since
 * the last clear, else S2ATTN_ERR_DEVICE_TIMEOUT with *detail (if non-NULL) set to
 * (kernel << 8) | site (kernel 1 = forward, 2 = backward, 4 = decoding step,
 * 5 = LoRA projection, 6 = tree attention and masks, 7 = cache).  An index out of range
 * (site 0x40) is held in a word of its own, which makes no kernel skip its work: it returns
 * S2ATTN_ERR_DEVICE_INDEX when no other failure is recorded.  In the
 * bounds-checked build (libs2attn_debug.so, compiled with S2ATTN_DEBUG) a site with bit
 * 0x80 set is a global store or reduction whose computed index fell outside its tensor;
 * the access was skipped.  Synchronize the streams
 * that ran library kernels first.
 */
int s2attn_get_device_error(int* detail);

/* Resets the current device's error words to 0 (synchronous). */
int s2attn_clear_device_error(void);

/*
 * Self-test of the device-side failure path used by every kernel above: launches one
 * thread that waits on a barrier nothing ever arrives at, with a wait limit of
 * `timeout_us` microseconds (1 .. 1000000).  After the caller synchronizes `stream`,
 * s2attn_get_device_error() returns S2ATTN_ERR_DEVICE_TIMEOUT with detail
 * (3 << 8) | 1, and the context stays usable (clear the word to continue).  The
 * kernels' own waits give up after 2 s the same way instead of hanging the GPU.
 */
int s2attn_selftest_bounded_wait(unsigned timeout_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S2ATTN_H_ */
