/*
 * saf.h - C ABI of the hybrid causal-attention layer of Selective Attention
 * Freezing (SAF), forward and backward, on one NVIDIA GB300 (sm_103a).
 *
 * Source: "When Can Attention Heads Be Statically Defined?" (arXiv 2609.34650).
 *
 *   Ordinary head (App. A.1, Eqs. 5-7):
 *       S = Q K^T / sqrt(d),  A = softmax_causal(S),  O = A V.
 *   Frozen head (§3.2, Eq. 3; §3.3 "Fused computation"):
 *       W(i, j) = exp(a[j] + r[i - j]) / Z(i) for j <= i, 0 for j > i,
 *       Z(i)    = sum_{k <= i} exp(a[k] + r[i - k]),        O = W V.
 *     The pattern never looks at Q or K. Its backward pass is only
 *     dV = W^T dO (§3.3, App. D.2); a frozen head has no query/key slot, so
 *     its dQ and dK are zero, and a, r and the normalisers take no gradient.
 *   Both kinds of head run in one fused launch per pass and write their
 *   outputs in the original head order (App. D.2).
 *
 * Indexing is 0-based: the paper's alpha(j) (keys 1..T) is a[j-1] and its
 * rho(delta) (offsets 0..T-1) is r[delta].
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors q, k, v, o, dO, dq, dk, dv have layout [B, H, T, d], contiguous,
 *    element type `dt` (bf16 or fp32). lse and the normalisers are fp32.
 *    d = 64, 96 or 128. SAF_BF16 runs on tensor-core kernels, SAF_FP32 on
 *    CUDA-core kernels, for the multi-head and grouped-query layouts, with
 *    per-call or prepared normalisers. Other values return SAF_EUNSUPPORTED.
 *    Every tensor pointer must be 16-byte aligned (SAF_EALIGN otherwise).
 *  - a, r: fp32 [H, ld_prior] device arrays, ld_prior >= T; row h holds the
 *    absolute-key preference a and the relative-distance preference r of
 *    head h. Only a[h, 0..T-1], r[h, 0..T-1] of frozen heads are read, so a
 *    stored prior longer than T may be passed (App. D.2 tests prior length
 *    192 at T = 129). a and r may be NULL when no head is frozen.
 *  - frozen: HOST array of H bytes, nonzero = frozen head. NULL means no
 *    frozen head. H <= SAF_MAX_HEADS.
 *  - q and k of frozen heads are never read (they may hold anything,
 *    including NaN); q and k may be NULL only when every head is frozen.
 *  - workspace: caller-owned DEVICE scratch of at least
 *    saf_attn_workspace_bytes(...) bytes, 256-byte aligned. The library
 *    allocates no memory and keeps no state across calls other than cached
 *    device attributes, CUDA function attributes, a launch counter and the
 *    optional trace hook below. Calls that share a workspace must be
 *    ordered on one stream.
 *  - stream: a cudaStream_t passed as void* (NULL = legacy default stream).
 *    All device work is enqueued on it; no entry point synchronises except
 *    saf_device_status.
 *  - Return value: SAF_OK (0) or a negative saf_status_t. Argument, shape,
 *    alignment and device errors are returned synchronously before any
 *    work is enqueued. An error raised while kernels run (a bounded device
 *    wait that expired) is recorded in the workspace and reported by
 *    saf_device_status.
 *  - T == 0 or B == 0 is a valid empty call: nothing is launched.
 */
#ifndef SAF_H_
#define SAF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SAF_MAX_HEADS 256

#if defined(__GNUC__)
#define SAF_API __attribute__((visibility("default")))
#else
#define SAF_API
#endif

typedef enum { SAF_BF16 = 0, SAF_FP32 = 1 } saf_dtype_t;

typedef enum {
    SAF_OK = 0,
    SAF_EINVAL = -1,        /* null pointer, bad shape, ld_prior < T, H > SAF_MAX_HEADS   */
    SAF_EALIGN = -2,        /* a tensor or the workspace is not aligned                   */
    SAF_EUNSUPPORTED = -3,  /* device is not sm_103, or d / dtype not supported          */
    SAF_ELAUNCH = -4,       /* a kernel launch or an async CUDA call failed               */
    SAF_EWORKSPACE = -5,    /* workspace NULL or smaller than saf_attn_workspace_bytes    */
    SAF_ETIMEOUT = -6,      /* a bounded device wait expired (from saf_device_status)    */
    SAF_ECUDA = -8,         /* a CUDA runtime query failed (no device, driver error)    */
    SAF_ESCRATCH = -9,      /* saf_attn_fwd_noalloc: the problem needs more workspace
                               than its fixed device scratch holds                     */
    SAF_EPAGE = -10         /* a paged call met a page or a token count outside its
                               bounds (from saf_device_status)                         */
} saf_status_t;

/* Bytes of device workspace that saf_attn_fwd (backward = 0) or
 * saf_attn_bwd (backward = 1) needs for these sizes. Returns 0 for an
 * invalid size. */
SAF_API size_t saf_attn_workspace_bytes(int B, int H, int T, int d, saf_dtype_t dt, int backward);

/* Forward pass of the hybrid layer.
 *
 * In:  q, k, v [B,H,T,d] (dt); a, r [H, ld_prior] fp32; frozen [H] host bytes.
 * Out: o [B,H,T,d] (dt): ordinary heads A V (Eqs. 5-7), frozen heads W V
 *      (Eq. 3); lse [B,H,T] fp32: for ordinary rows the natural-log
 *      normaliser of the scaled scores, m_i + log sum_j exp(S_ij - m_i); for
 *      frozen rows log Z(i). saf_attn_bwd consumes lse.
 * The normalisers log Z of the frozen heads are computed here ("precomputed
 * normalisers", §3.3), once per head, independent of the batch.
 * Supported: d in {64, 96, 128}; SAF_BF16 on the tensor cores with fp32
 * accumulation (App. C.5's 1B model has d_h = 96), SAF_FP32 in fp32 arithmetic
 * throughout on CUDA cores. */
SAF_API int saf_attn_fwd(const void* q, const void* k, const void* v,
                 const float* a, const float* r, int ld_prior, const uint8_t* frozen,
                 int B, int H, int T, int d, saf_dtype_t dt,
                 void* o, float* lse,
                 void* workspace, size_t ws_bytes, void* stream);

/* Forward pass for callers that cannot allocate device memory.
 *
 * The paper has no counterpart to this entry point; it exists for callers
 * that cannot hand the library a workspace: code that runs where
 * cudaMalloc is not allowed (for example inside a framework that owns every
 * allocation and passes plugins only their input and output buffers, or in
 * a context where allocating could deadlock or fragment a caching
 * allocator). It computes exactly what saf_attn_fwd computes, with the same
 * kernels, arguments and outputs, but takes its workspace from a fixed
 * array of 8 MiB in device memory that the library declares statically;
 * every GPU that loads the library holds that array until the process
 * exits. It calls no cudaMalloc, cudaFree or other allocating routine.
 *
 *  - Size limit: saf_attn_workspace_bytes(B, H, T, d, dt, 0) must be at most
 *    8 MiB: about H * T <= 340,000 for SAF_BF16 (for example 12 heads of
 *    16,384 tokens) and H * T <= 2,000,000 for SAF_FP32, independent of B;
 *    larger problems return SAF_ESCRATCH and enqueue nothing.
 *  - Set-up: the first call on each device looks up the array's device
 *    address (cudaGetSymbolAddress, with that device current) and caches
 *    it. Make that first call before any stream capture begins. The cached
 *    address belongs to the device's primary context: after
 *    cudaDeviceReset (or anything else that ends that context) it is stale,
 *    so a process that resets a device must not call this entry point on
 *    that device again.
 *  - Sharing: every call on a device uses the same array, which keeps the
 *    contents the last call left. Each call's first kernel clears the parts
 *    that must start at zero before anything reads them. Calls whose work overlaps on the
 *    GPU (two streams, or two host threads) race on the array: order them
 *    on one stream.
 *  - Device-side status words live in that array and are not reported;
 *    callers that need saf_device_status use saf_attn_fwd with a workspace. */
SAF_API int saf_attn_fwd_noalloc(const void* q, const void* k, const void* v,
                                 const float* a, const float* r, int ld_prior, const uint8_t* frozen,
                                 int B, int H, int T, int d, saf_dtype_t dt,
                                 void* o, float* lse, void* stream);

/* Backward pass of the hybrid layer, given dO = dL/dO.
 *
 * In:  q, k, v, o, dO [B,H,T,d] (dt), lse [B,H,T] from saf_attn_fwd with the
 *      same inputs; a, r, frozen as in saf_attn_fwd.
 * Out: dq, dk, dv [B,H,T,d] (dt). Ordinary heads: the gradient of Eqs. 5-7.
 *      Frozen heads: dv = W^T dO; dq and dk are written as exact zeros
 *      (§3.3, App. D.2). dq may be the buffer of q or of dO, here and in every
 *      other backward call: it is then written when nothing reads that any more.
 * Supported: d in {64, 96, 128} for both types. */
SAF_API int saf_attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, const float* a, const float* r, int ld_prior,
                 const uint8_t* frozen, int B, int H, int T, int d, saf_dtype_t dt,
                 void* dq, void* dk, void* dv,
                 void* workspace, size_t ws_bytes, void* stream);

/* Grouped-query forward pass (§3.3: the grouped-query path keeps the shared
 * key and value projections and drops the replaced heads' query projections;
 * App. C.6: Qwen3-4B shares 8 key/value heads among 32 query heads; App. D.2:
 * each ordinary query head is mapped to its retained key/value group).
 *
 * Same as saf_attn_fwd, except that k and v have Hkv heads:
 * In:  q [B,H,T,d], k, v [B,Hkv,T,d] (dt), H a multiple of Hkv; query head h
 *      reads key/value head h / (H / Hkv). a, r, frozen are per query head
 *      ([H, ld_prior], H bytes): a frozen query head applies its own Eq. 3
 *      pattern to the values of its group and reads no q or k.
 * Out: o [B,H,T,d], lse [B,H,T] as for saf_attn_fwd.
 * Workspace: saf_attn_workspace_bytes(B, H, T, d, dt, 0) (query heads).
 * Errors: as saf_attn_fwd; SAF_EINVAL also for Hkv <= 0 or H % Hkv != 0.
 * saf_attn_fwd(...) equals saf_attn_fwd_gqa(..., Hkv = H, ...). */
SAF_API int saf_attn_fwd_gqa(const void* q, const void* k, const void* v,
                     const float* a, const float* r, int ld_prior, const uint8_t* frozen,
                     int B, int H, int Hkv, int T, int d, saf_dtype_t dt,
                     void* o, float* lse,
                     void* workspace, size_t ws_bytes, void* stream);

/* Grouped-query backward pass (§3.3, App. C.6, App. D.2), given dO.
 *
 * In:  q, o, dO [B,H,T,d]; k, v [B,Hkv,T,d]; lse [B,H,T] from
 *      saf_attn_fwd_gqa with the same inputs; a, r, frozen per query head.
 * Out: dq [B,H,T,d]: the gradient of Eqs. 5-7 for ordinary query heads,
 *      exact zeros for frozen ones. dk, dv [B,Hkv,T,d]: the gradient of a
 *      shared head is the sum over the query heads of its group; frozen query
 *      heads add W^T dO to dv only, so a group with no ordinary query head
 *      gets dk = 0 exactly.
 * Workspace: saf_attn_workspace_bytes(B, H, T, d, dt, 1).
 * Errors: as saf_attn_bwd; SAF_EINVAL also for Hkv <= 0 or H % Hkv != 0.
 * saf_attn_bwd(...) equals saf_attn_bwd_gqa(..., Hkv = H, ...). */
SAF_API int saf_attn_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, const float* a, const float* r, int ld_prior,
                     const uint8_t* frozen, int B, int H, int Hkv, int T, int d, saf_dtype_t dt,
                     void* dq, void* dk, void* dv,
                     void* workspace, size_t ws_bytes, void* stream);

/* ---- Prepared frozen-pattern state -------------------------------------------
 * A frozen head's pattern depends on a and r alone (§3.2, Eq. 3), so its
 * normalisers can be computed once and kept: the paper's persistent state per
 * replaced head is alpha, rho, the normalisers and a small relative-distance
 * band (§3.3 "precomputed normalisers"; App. D.2). saf_attn_fwd / saf_attn_bwd
 * recompute them in every call; the calls below take them from a state that
 * saf_frozen_prepare filled once for fixed (a, r).
 *
 * saf_frozen_state_bytes: bytes of DEVICE state for H heads of length T
 * (0 for invalid sizes). It does not depend on B.
 *
 * saf_frozen_prepare: fills `state` (caller-owned, 256-byte aligned) for the
 * frozen heads of `frozen` from a, r [H, ld_prior]. Enqueued on `stream`.
 * Prepare again after a or r change (the trainable variant of App. C.3.2
 * refreshes its normalisers after each update).
 *
 * saf_attn_fwd_prepared / saf_attn_bwd_prepared: saf_attn_fwd_gqa /
 * saf_attn_bwd_gqa (Hkv = H for the multi-head layer) with the frozen-pattern
 * data read from `state`. a, r, ld_prior and frozen must be the ones the state
 * was prepared with (the fp32 path still reads a and r). `workspace` is the
 * per-call workspace of saf_attn_workspace_bytes. Calls may share one state
 * while nothing prepares it again. Results equal those of the unprepared
 * calls up to rounding (the forward's exactly). Errors as the unprepared
 * calls, and SAF_EWORKSPACE for a NULL state. */
SAF_API size_t saf_frozen_state_bytes(int H, int T, saf_dtype_t dt);
SAF_API int saf_frozen_prepare(const float* a, const float* r, int ld_prior, const uint8_t* frozen, int H, int T,
                               saf_dtype_t dt, void* state, size_t state_bytes, void* stream);
SAF_API int saf_attn_fwd_prepared(const void* q, const void* k, const void* v, const float* a, const float* r,
                                  int ld_prior, const uint8_t* frozen, const void* state, int B, int H, int Hkv,
                                  int T, int d, saf_dtype_t dt, void* o, float* lse, void* workspace,
                                  size_t ws_bytes, void* stream);
SAF_API int saf_attn_bwd_prepared(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                  const float* lse, const float* a, const float* r, int ld_prior,
                                  const uint8_t* frozen, const void* state, int B, int H, int Hkv, int T, int d,
                                  saf_dtype_t dt, void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes,
                                  void* stream);

/* ---- Sliding window with sinks -------------------------------------------------
 * The layer (saf_attn_fwd_gqa / saf_attn_bwd_gqa, Hkv = H for the multi-head
 * layer) with ordinary heads that see the last `window` keys and the first
 * `sinks`: query i attends to the keys j <= i with i - j < window or j < sinks,
 *     A(i, j) = exp(S(i, j)) / sum over the keys that i sees,
 * and its own key is always among them. Only key blocks that a block of queries
 * sees are visited, forward and backward. Frozen heads keep their whole pattern
 * (Eq. 3): it is a fixed matrix, cut by its own r.
 *
 * window >= 0, sinks >= 0 (else SAF_EINVAL); window = 0 or window >= T is the layer
 * without a window, the forward with the same bits. The SAF_BF16 backward is nearer to
 * the exact gradients than the layer's: at d = 64 it forms dS from unrounded weights,
 * and where no row sees more than 16 keys, or T <= 32, it sums dO . o over the keys in
 * fp32 (the rounding of o would be the largest error of dq and dk). state: NULL, or the prepared state of
 * saf_frozen_prepare for these a, r and frozen (as for the _prepared calls).
 * Everything else (shapes, workspace, empty calls, errors, outputs) is as for the
 * calls named above.
 *
 * What is hidden must still be finite in most places. A block of rows visits whole blocks of keys:
 * those of the sinks, and those from its first row's first key to its last row (all up to there for a
 * frozen head). A hidden pair of a visited block has weight 0, and 0 * NaN is NaN: a NaN or an
 * infinity in the k or v of a key reaches o and dq of every row whose block visits the key's, and one
 * in the q, o, dO or lse of a row reaches dk and dv of every key whose block the row's visits. What
 * is not visited may be anything. Blocks hold 128 keys and 128 rows, 256 rows in the forward of
 * SAF_BF16 at d = 64, and 64 of each in SAF_FP32.
 *
 * The outputs overlap nothing else, but that dq may be the buffer of q or of dO (dq also holds
 * partial sums until the call ends, of blocks of sinks that are then not split: slower). */
SAF_API int saf_attn_fwd_window(const void* q, const void* k, const void* v, const float* a, const float* r,
                                int ld_prior, const uint8_t* frozen, const void* state, int window, int sinks, int B,
                                int H, int Hkv, int T, int d, saf_dtype_t dt, void* o, float* lse, void* workspace,
                                size_t ws_bytes, void* stream);
SAF_API int saf_attn_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                const float* lse, const float* a, const float* r, int ld_prior,
                                const uint8_t* frozen, const void* state, int window, int sinks, int B, int H,
                                int Hkv, int T, int d, saf_dtype_t dt, void* dq, void* dk, void* dv, void* workspace,
                                size_t ws_bytes, void* stream);

/* ---- Paged cache ---------------------------------------------------------------
 * Serving: keys and values of B sequences live in fixed-size pages of two caches,
 *     k_cache, v_cache [num_pages, Hkv, page_size, d]  (dt, contiguous, 16-byte aligned),
 * and page_table [B, max_pages] (DEVICE int32) names a sequence's pages in order: slot x
 * of sequence b is row x mod page_size of page page_table[b, x / page_size]. page_size is
 * a power of two, 8 to 1024; num_pages * Hkv <= 2^31 - 1.
 *
 * A step brings up to T new tokens per sequence. ctx [B] (DEVICE int32) counts the
 * tokens in the cache before them and n_new [B] (DEVICE int32, NULL: T each) the new
 * ones, 0 <= n_new[b] <= T; rows t >= n_new[b] of a padded batch hold no token. The
 * counts are read on the device, so a captured graph serves every step.
 *
 * What the device finds outside its bounds (a negative ctx, an n_new outside [0, T],
 * tokens past max_pages * page_size or max_len, a page outside [0, num_pages)) never
 * leads to an access: counts are cut to their bounds (a negative ctx: no tokens; what is
 * cut off is no token, its rows of q_out and o are those of none), keys of such a page are not written and not seen, and the call ORs a bit into its status
 * words, which saf_device_status answers with SAF_EPAGE. The status words of these
 * calls stay as they are until the caller clears them; zero them when you make them.
 * Entries of page_table behind a sequence's last token, and behind the window of a call
 * whose heads are all cut by one, are not read as pages and may hold anything.
 *
 * saf_kv_append
 * writes the new tokens' k and v into the caches: token t of sequence b into slot
 * ctx[b] + t, with the rotary position rotation applied to k, and to q for the
 * attention that follows:
 *     pair c of a row:  (y0, y1) = (x0 cos w - x1 sin w, x0 sin w + x1 cos w),
 *     w = (pos_base + ctx[b] + t) inv_freq[c],
 * for the rope_dim / 2 pairs of the first rope_dim elements (a multiple of 16, 0: no
 * rotation): elements (c, c + rope_dim / 2), or (2c, 2c + 1) when interleaved = 1. The
 * rest is copied. The angle modulo a turn is off by at most 2^-64 of a turn per position
 * (frequencies as given, in double), and in fp32 from there on; results are rounded once to dt.
 * In:  q [B,H,T,d] (NULL: no q), k, v [B,Hkv,T,d] with element strides (sequence, head,
 *      token) strides[0..2], [3..5], [6..8] (HOST; NULL: contiguous), rows of d elements
 *      contiguous, every row 16-byte aligned: slices of one projection's output do.
 *      inv_freq: HOST double [rope_dim / 2], finite. frozen: as elsewhere; q rows of
 *      frozen heads are neither read nor written, and keys of key/value heads that no
 *      ordinary head reads are not either (k and k_cache may be NULL if that is all).
 * Out: q_out [B,H,T,d] contiguous (q_out = q only where q is contiguous; else they must
 *      not overlap), the slots of k_cache and v_cache. Rows without a token, and every
 *      other slot, stay as they were. Two tokens of one call must not share a slot.
 * 0 <= pos_base <= 2^40, T <= 2^21 and B T <= 2^30, else SAF_EINVAL.
 * status: DEVICE uint32[2] (see above), for example a paged workspace; NULL: not recorded.
 *
 * saf_attn_paged
 * is the attention of the new tokens over their sequence's cache, after saf_kv_append:
 * token t of sequence b stands at position i = ctx[b] + t and sees the keys j <= i,
 * ordinary heads within (window, sinks) as for saf_attn_fwd_window (window = 0: all),
 * frozen heads with the weights of Eq. 3 at row i (k is not read for them):
 * ld_prior >= max_len. Entries of a and r may be -infinity; a logit a + r below -2.3e38,
 * the type's lowest value among them, counts as -infinity: a key that is not seen.
 * In:  q [B,H,T,d]; max_len: an upper bound of ctx[b] + n_new[b], at most
 *      max_pages * page_size, known on the host: it sets the launch's size.
 * Out: o [B,H,T,d], lse [B,H,T] as for saf_attn_fwd; o = 0, lse = -inf for rows without
 *      a token and rows that see no key.
 * A key or value that one row sees must be finite where another row beside it does not see
 * it, which takes it with weight 0, and so must a value that a pattern of -infinity alone hides; what
 * lies behind the rows' positions or outside their windows, for all of them, may be anything.
 * T is 1 for a decoding step, a few for drafted tokens, and may be any length for a
 * chunk of a prompt. SAF_FP32 is computed in fp32 throughout; sums and softmax statistics
 * are fp32 in both types.
 *
 * saf_attn_paged_shared
 * is the same for sequences that all begin with one prefix of prefix_len tokens (HOST;
 * 0: as saf_attn_paged), held once in prefix_pages [ceil(prefix_len / page_size)] (DEVICE
 * int32): key j < prefix_len is the prefix's slot j, key prefix_len + x slot x of the
 * sequence's own pages (which begin with a page of their own), and token t stands at
 * position prefix_len + ctx[b] + t: ctx, n_new and max_len count own tokens, append them
 * with pos_base = prefix_len. ld_prior >= prefix_len + max_len. The prefix's keys and
 * values are read for all sequences together.
 *
 * workspace: DEVICE, 256-byte aligned, saf_attn_paged_workspace_bytes(...) bytes (enough
 * for every window and choice of frozen heads; 0 for invalid sizes; fewer sequences are
 * split into more items and may need more: ask for every batch size that shares one); it
 * begins with the status words. Calls that share one must be ordered on one stream, replays of captured
 * graphs among them.
 * Errors before any work is enqueued: SAF_EINVAL, SAF_EALIGN, SAF_EWORKSPACE,
 * SAF_EUNSUPPORTED, SAF_ECUDA as elsewhere (prefix_len + max_len <= 2^30 and B H T <= 2^29,
 * else SAF_EINVAL). B = 0 or T = 0 is an empty call. */
SAF_API int saf_kv_append(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* ctx,
                          const int32_t* n_new, const int32_t* page_table, int max_pages, const double* inv_freq,
                          int rope_dim, int interleaved, int64_t pos_base, const uint8_t* frozen, int B, int H,
                          int Hkv, int T, int d, int num_pages, int page_size, saf_dtype_t dt, void* q_out,
                          void* k_cache, void* v_cache, uint32_t* status, void* stream);
SAF_API size_t saf_attn_paged_workspace_bytes(int B, int H, int Hkv, int T, int d, int max_len, int prefix_len,
                                              saf_dtype_t dt);
SAF_API int saf_attn_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                           int max_pages, const int32_t* ctx, const int32_t* n_new, const float* a, const float* r,
                           int ld_prior, const uint8_t* frozen, int window, int sinks, int B, int H, int Hkv, int T,
                           int d, int max_len, int num_pages, int page_size, saf_dtype_t dt, void* o, float* lse,
                           void* workspace, size_t ws_bytes, void* stream);
SAF_API int saf_attn_paged_shared(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* prefix_pages, int prefix_len, const int32_t* page_table,
                                  int max_pages, const int32_t* ctx, const int32_t* n_new, const float* a,
                                  const float* r, int ld_prior, const uint8_t* frozen, int window, int sinks, int B,
                                  int H, int Hkv, int T, int d, int max_len, int num_pages, int page_size,
                                  saf_dtype_t dt, void* o, float* lse, void* workspace, size_t ws_bytes,
                                  void* stream);

/* ---- 8-bit paged cache ---------------------------------------------------------
 * The paged cache in 8 bits: k_cache, v_cache [num_pages, Hkv, page_size, d] hold codes of
 * float8 e4m3 (4 exponent and 3 mantissa bits, largest 448, no infinity), and k_scale, v_scale
 * [num_pages, Hkv, page_size] (fp32, 16-byte aligned) one scale for each row of d codes. A row
 * stands for the values code_c * scale. dt is the type of q, k, v, o and of rows read back.
 *
 * saf_kv_append_quant is saf_kv_append into such caches. A row y (k after its rotation, which is
 * not rounded before) is written as
 *     scale = max(max_c |y_c| / 448, 2^-126),   code_c = y_c / scale, rounded to nearest even,
 * in fp32: a code is off by half a step of e4m3 (2^-4 of the value, or 2^-10 scale near zero, and
 * 2^-22 of the value by the arithmetic before it). A NaN keeps its place; a row with an infinity
 * has an infinite scale and reads back as NaN. q is rotated and rounded to dt as there.
 * k_scale may be NULL where k_cache may. The scales of slots that are not written stay as they were.
 *
 * saf_kv_read_quant reads rows back: row t of sequence b, t < count[b], is its slot first[b] + t,
 * as code_c * scale rounded to dt. first [B] (DEVICE int32; NULL: 0) and count [B] (DEVICE int32;
 * NULL: T each), 0 <= count[b] <= T.
 * Out: k_out, v_out [B, Hkv, T, d] (dt), contiguous, all of them written: rows without a token, and
 * rows of a page outside the cache, as zeros. k_cache, k_scale and k_out may be NULL together
 * (values only). Counts and pages outside their bounds are reported in status as by saf_kv_append.
 * B T <= 2^30 and T <= 2^21, else SAF_EINVAL.
 *
 * saf_attn_paged_quant and saf_attn_paged_shared_quant are saf_attn_paged and saf_attn_paged_shared
 * over such caches: every rule above holds, with code_c * scale for the cache's values. Scales that
 * a row sees must be finite and not negative (an infinite one of a value, which stands for a row of
 * NaN, makes NaN of the outputs that see it); those of slots that no row sees may be anything, as
 * the codes. The workspace is that of saf_attn_paged_quant_workspace_bytes. */
SAF_API int saf_kv_append_quant(const void* q, const void* k, const void* v, const int64_t* strides,
                               const int32_t* ctx, const int32_t* n_new, const int32_t* page_table, int max_pages,
                               const double* inv_freq, int rope_dim, int interleaved, int64_t pos_base,
                               const uint8_t* frozen, int B, int H, int Hkv, int T, int d, int num_pages,
                               int page_size, saf_dtype_t dt, void* q_out, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, uint32_t* status, void* stream);
SAF_API int saf_kv_read_quant(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* page_table, int max_pages, const int32_t* first, const int32_t* count,
                             int B, int Hkv, int T, int d, int num_pages, int page_size, saf_dtype_t dt, void* k_out,
                             void* v_out, uint32_t* status, void* stream);
SAF_API size_t saf_attn_paged_quant_workspace_bytes(int B, int H, int Hkv, int T, int d, int max_len, int prefix_len,
                                                   saf_dtype_t dt);
SAF_API int saf_attn_paged_quant(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const int32_t* page_table, int max_pages, const int32_t* ctx,
                                const int32_t* n_new, const float* a, const float* r, int ld_prior,
                                const uint8_t* frozen, int window, int sinks, int B, int H, int Hkv, int T, int d,
                                int max_len, int num_pages, int page_size, saf_dtype_t dt, void* o, float* lse,
                                void* workspace, size_t ws_bytes, void* stream);
SAF_API int saf_attn_paged_shared_quant(const void* q, const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale, const int32_t* prefix_pages,
                                       int prefix_len, const int32_t* page_table, int max_pages, const int32_t* ctx,
                                       const int32_t* n_new, const float* a, const float* r, int ld_prior,
                                       const uint8_t* frozen, int window, int sinks, int B, int H, int Hkv, int T,
                                       int d, int max_len, int num_pages, int page_size, saf_dtype_t dt, void* o,
                                       float* lse, void* workspace, size_t ws_bytes, void* stream);

/* Diagnostic forward pass for testing failure detection (the paper has no
 * counterpart; it exercises this library's bounded waits).
 *
 * Every wait inside the tensor-core kernels is bounded: when it expires, the
 * kernel records SAF_ETIMEOUT in the workspace's error word, its other warps
 * give up too, it frees its tensor memory and returns, so the CUDA context
 * stays usable. This entry point makes that happen on purpose, without any
 * fault: it is saf_attn_fwd (SAF_BF16 only, else SAF_EUNSUPPORTED) with
 *  - withhold = 1: the forward kernel's producer publishes no work item, so
 *    every other role's first wait expires (o and lse are not written);
 *    withhold = 0 runs the normal pass;
 *  - wait_limit_us: the limit of every bounded wait in the forward kernel,
 *    in microseconds (0: the default of 2 s). A wait ends at most one
 *    suspend interval (about 10 ms) after its limit.
 * The next saf_device_status on `workspace` reports SAF_ETIMEOUT after a
 * withheld call; the next normal call clears the word. */
SAF_API int saf_attn_fwd_diag(const void* q, const void* k, const void* v,
                              const float* a, const float* r, int ld_prior, const uint8_t* frozen,
                              int B, int H, int T, int d, saf_dtype_t dt,
                              void* o, float* lse,
                              void* workspace, size_t ws_bytes, void* stream,
                              int withhold, unsigned wait_limit_us);

/* Waits for `stream`, then reads the error word that the kernels of the last
 * call on `workspace` left there. Returns SAF_OK, SAF_ETIMEOUT, SAF_EPAGE (paged
 * calls), or SAF_ECUDA if the stream reported a CUDA error. */
SAF_API int saf_device_status(const void* workspace, void* stream);

/* Static, human-readable text for a status code. Never NULL. */
SAF_API const char* saf_error_string(int status);

/* ABI version of this library (major * 100 + minor). */
SAF_API int saf_version(void);

/* ---- Compact fitting of a frozen pattern -----------------------------------
 * Fits a, r of Eq. 3 to a target pattern P, given only P's sufficient
 * statistics (§3.2 "Fitting", Eq. 4; App. D.1, Eq. 20):
 *   eta_abs(j)   = sum_{i >= j} P(i, j)          (key-column sums)
 *   eta_rel(d)   = sum_{i - d >= 0} P(i, i - d)  (diagonal sums)
 * It starts from a = 0, r(d) = log max(eta_rel(d) / (T - d), 1e-9) and takes
 * `steps` Adam steps (moment decays 0.9 and 0.999, epsilon 1e-8, bias-corrected)
 * at learning rate `lr` on
 *   L(a, r) = (1/T) [sum_i log Z(i) - sum_j eta_abs(j) a(j) - sum_d eta_rel(d) r(d)],
 * whose gradient is the fitted pattern's marginals minus the target's, over T.
 * The paper's settings are steps = 400, lr = 0.05 (App. C.1).
 *
 * In:  eta_abs, eta_rel: DEVICE fp32 [H, T] (row h: head h); H <= SAF_MAX_HEADS.
 * Out: a, r: DEVICE fp32 [H, T], the fitted parameters (row stride T, ready to
 *      pass to saf_attn_fwd with ld_prior = T); loss: DEVICE fp32 [H], L at the
 *      result. The paper's acceptance statistic kappa (mean KL per row of the
 *      target from the fit) is loss[h] + (1/T) sum P log P of the target
 *      (saf_fit_target_stats computes that term; saf_fit_from_target runs the
 *      whole path); a fit passes when kappa <= 0.2.
 * workspace: DEVICE scratch of saf_fit_workspace_bytes(H, T) bytes, 256-byte
 * aligned. fp32 pointers must be 4-byte aligned. Work is enqueued on `stream`;
 * errors in the arguments return before any work is enqueued. */
SAF_API size_t saf_fit_workspace_bytes(int H, int T);
SAF_API int saf_fit_compact(const float* eta_abs, const float* eta_rel, int H, int T, int steps, float lr,
                            float* a, float* r, float* loss, void* workspace, size_t ws_bytes, void* stream);

/* ---- From a measured target to accept / reject ------------------------------
 * The selection algorithm's target steps (§3.2 "Fitting"; App. A.2; App. C.1):
 * the measured mean attention matrix A of a head has its causal entries
 * floored at 1e-9 and every row normalised, P = floor-and-normalise(A); Eq. 4
 * needs only P's key-column sums eta_abs(j) = sum_{i >= j} P(i, j) and diagonal
 * sums eta_rel(d) = sum_{i >= d} P(i, i - d); a fitted head is accepted when
 * kappa = (1/T) sum_i KL(P(i, .) || W(i, .)) <= 0.2 nats (App. C.1). Since
 * kappa = (1/T) sum_i sum_j P log P + L(a, r) with L the Eq. 4 loss, the
 * target's negative entropy per row, negent = (1/T) sum P log P, completes it.
 *
 * saf_fit_target_stats
 * In:  A: DEVICE fp32 [H, T, T] row-major; entries above the diagonal are not
 *      read. P is never stored.
 * Out: eta_abs, eta_rel: DEVICE fp32 [H, T]; negent: DEVICE fp32 [H].
 * Sums run in a fixed order: results are the same on every run.
 * workspace: DEVICE scratch of saf_fit_stats_workspace_bytes(H, T) bytes,
 * 256-byte aligned. Errors: SAF_EINVAL (sizes, NULL), SAF_EALIGN, SAF_EWORKSPACE,
 * SAF_EUNSUPPORTED (device), all before any work is enqueued.
 *
 * saf_fit_from_target: the whole path on the device: the statistics above,
 * saf_fit_compact's `steps` Adam steps at rate `lr`, then kappa.
 * Out: a, r: DEVICE fp32 [H, T] (the fitted pattern); kappa: DEVICE fp32 [H];
 *      accept: DEVICE uint8 [H], 1 when kappa <= tol (the paper: 0.2).
 * workspace: saf_fit_from_target_workspace_bytes(H, T) bytes, 256-byte aligned.
 * Errors as above, and SAF_EINVAL for steps < 0, lr <= 0 or tol < 0. */
SAF_API size_t saf_fit_stats_workspace_bytes(int H, int T);
SAF_API int saf_fit_target_stats(const float* A, int H, int T, float* eta_abs, float* eta_rel, float* negent,
                                 void* workspace, size_t ws_bytes, void* stream);
SAF_API size_t saf_fit_from_target_workspace_bytes(int H, int T);
SAF_API int saf_fit_from_target(const float* A, int H, int T, int steps, float lr, float tol, float* a, float* r,
                                float* kappa, uint8_t* accept, void* workspace, size_t ws_bytes, void* stream);

/* ---- Gradients of trainable patterns ---------------------------------------
 * For the variant whose patterns keep training (App. C.3.2): the gradients of
 * the loss with respect to a and r of every frozen head, given the forward
 * output and the output gradient. Eq. 3 is a row softmax of the logits
 * a(j) + r(i - j); with G(i, j) = dO_i . V_j and D_i = dO_i . O_i,
 *   dL(i, j) = W(i, j) (G(i, j) - D_i),
 *   da(j) = sum_b sum_{i >= j} dL(i, j),   dr(d) = sum_b sum_{i >= d} dL(i, i - d).
 *
 * In:  v, dO, o [B, H, T, d] (dt, d = 64, 96 or 128), lse [B, H, T] as
 *      saf_attn_fwd wrote it (the frozen rows hold log Z), a, r, ld_prior,
 *      frozen as for saf_attn_fwd.
 * Out: da, dr: DEVICE fp32 [H, T]; rows of ordinary heads are zero. They are
 *      overwritten (cleared on `stream` first).
 * fp32 arithmetic on CUDA cores; the additions into da and dr are atomic, so
 * their last bits vary from run to run. No workspace. */
SAF_API int saf_pattern_grad(const void* v, const void* dO, const void* o, const float* lse, const float* a,
                             const float* r, int ld_prior, const uint8_t* frozen, int B, int H, int T, int d,
                             saf_dtype_t dt, float* da, float* dr, void* stream);

/* The same gradients on the tensor cores (bf16 inputs, d = 64, 96 or 128), with
 * sums in a fixed order: the results have the same bits on every run.
 * G^T = V dO^T is formed per causal 128 x 128 tile with tcgen05 MMAs (fp32 in
 * tensor memory); W is rebuilt from a, r and the log Z rows of lse in the form
 * the layer's backward uses (factorised, or exact when a head's log Z' falls
 * below -64); tiles are visited band by band (band = query block - key block),
 * each thread summing its elements of one distance i - j over the band in
 * registers, and the per-tile key sums and per-band distance sums are written
 * to the workspace and added up by a last kernel.
 * In:  v, dO, o [B, H, T, d] bf16, 16-byte aligned; lse [B, H, T] fp32 as
 *      saf_attn_fwd wrote it; a, r, ld_prior, frozen as for saf_attn_fwd.
 * Out: da, dr: DEVICE fp32 [H, T], overwritten; rows of ordinary heads zero.
 * workspace: DEVICE scratch of saf_pattern_grad_tc_workspace_bytes(B, H, T,
 * n_frozen) bytes (n_frozen = number of nonzero entries of `frozen`), 256-byte
 * aligned; clobbered. Its first 256 bytes are the status words that
 * saf_device_status reads after the call (SAF_ETIMEOUT when a bounded
 * wait of the kernel expired).
 * Errors: SAF_EINVAL (sizes, NULL), SAF_EALIGN, SAF_EWORKSPACE,
 * SAF_EUNSUPPORTED (d not 64, 96 or 128; device), all before any work is
 * enqueued; SAF_ELAUNCH. saf_pattern_grad_tc_workspace_bytes returns 0 for
 * invalid sizes. */
SAF_API size_t saf_pattern_grad_tc_workspace_bytes(int B, int H, int T, int n_frozen);
SAF_API int saf_pattern_grad_tc(const void* v, const void* dO, const void* o, const float* lse, const float* a,
                                const float* r, int ld_prior, const uint8_t* frozen, int B, int H, int T, int d,
                                float* da, float* dr, void* workspace, size_t ws_bytes, void* stream);

/* ---- Profiling hooks (not part of the layer's arithmetic) ----------------
 * Kernel identifiers for saf_set_trace_events. */
typedef enum {
    SAF_KERNEL_NONE = 0,
    SAF_KERNEL_LOGNORM = 1,     /* forward: init kernel, log Z of frozen heads  */
    SAF_KERNEL_FWD = 2,         /* fused forward (both kinds of head)           */
    SAF_KERNEL_BWD_DELTA = 3,   /* D_i = sum_c dO_ic O_ic (bf16: also the row   *
                                 * vectors, dQ accumulator zeroing and 1 / Z')  */
    SAF_KERNEL_BWD_KV = 4,      /* backward key-block pass (dV, dK)            */
    SAF_KERNEL_BWD_Q = 5,       /* backward query-block pass (dQ)              */
    SAF_KERNEL_BWD = 6,         /* fused backward (dQ, dK, dV in one launch)   */
    SAF_KERNEL_DQ_FINISH = 7,   /* dQ accumulator -> dq (scale, dtype, zeros)  */
    SAF_KERNEL_PATTERN_PREP = 8, /* backward: init kernel (clears the status   *
                                  * words; maxima and padded a, r slices)       */
    SAF_KERNEL_PATTERN_GRAD = 9, /* saf_pattern_grad_tc: all of its launches    */
    SAF_KERNEL_KV_APPEND = 10,  /* saf_kv_append(_quant)                        */
    SAF_KERNEL_PAGED = 11,      /* saf_attn_paged(_shared)(_quant): all of its launches */
    SAF_KERNEL_KV_READ = 12     /* saf_kv_read_quant                            */
} saf_kernel_t;

/* From the next call on, record `start` (a cudaEvent_t as void*) on the
 * call's stream right before the launches that `kernel` names, and `stop`
 * right after them. Each kernel id has its own pair; NULL events switch that id
 * off, SAF_KERNEL_NONE switches every id off. The hook is process-wide and
 * not thread-safe; it is meant for benchmarks. Returns SAF_OK or
 * SAF_EINVAL for an unknown id. */
SAF_API int saf_set_trace_events(int kernel, void* start, void* stop);

/* Number of kernels this library has launched since it was loaded
 * (host-side counter, all devices and streams). */
SAF_API unsigned long long saf_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* SAF_H_ */
