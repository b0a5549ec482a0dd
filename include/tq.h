/*
 * tq.h -- C ABI of libtq: TurboQuant KV-cache compression and decode attention
 * over the compressed cache, for NVIDIA B200 (sm_100a).
 *
 * The method (page "Apple Silicon向けSwiftLM、TurboQuant KVキャッシュ圧縮とSSD
 * Expert Streamingを実装", ai-heartland.com):
 *   K cache, section "K-Cache圧縮：3-bit PolarQuant + 1-bit QJL = 4.25 bits/dim":
 *     1. L2-norm extraction and normalisation, x_hat = x / ||x||;
 *     2. a fast Walsh-Hadamard rotation that spreads outliers (applied here
 *        after a fixed random sign diagonal D: y = H D x_hat);
 *     3. a 3-bit non-linear Lloyd-Max codebook per coordinate;
 *     4. the residual of step 3;
 *     5. a Johnson-Lindenstrauss (QJL) projection of the residual, keeping one
 *        sign bit per projection.
 *   V cache, section "V-Cache圧縮：3-bit PolarQuant = 3.125 bits/dim":
 *     steps 1-3 only; V is not used for scoring, so it carries no QJL bit.
 *   Attention, section on the hybrid V2+V3 design: dequantisation is fused
 *     into the attention kernel, which reads the packed cache directly.
 *
 * Conventions.  d = head_dim (64, 128 or 256); m = d JL rows; tokens per cache
 * block = 64.  All data buffers (inputs, caches, outputs, workspace) are
 * device memory owned by the caller; the library owns only the constants
 * created by tq_init.  Hot calls (encode, attend) allocate nothing, do not
 * synchronise and copy nothing to the host; they enqueue kernels on the
 * caller's stream and return.  Errors in the arguments are detected on the
 * host before anything is launched and leave all buffers untouched.
 * Asynchronous device faults surface at the caller's next synchronisation.
 * A handle is read-only after tq_init, so concurrent calls on different
 * streams are safe; calls whose outputs overlap race.
 */
#ifndef TQ_H_
#define TQ_H_

#include <stddef.h>
#include <stdint.h>

#ifndef TQ_API
#define TQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tq_handle tq_handle;

/* Status codes.  TQ_ERR_CUDA: a CUDA runtime call or a launch failed.
 * TQ_ERR_WORKSPACE: the workspace passed is smaller than required.
 * TQ_ERR_DEVICE_CHECK: a kernel recorded a failed device-side check (a bounded
 * wait that ran out); reported by tq_device_status. */
typedef enum {
    TQ_OK = 0,
    TQ_ERR_INVALID_ARG = 1,
    TQ_ERR_UNSUPPORTED = 2,
    TQ_ERR_CUDA = 3,
    TQ_ERR_WORKSPACE = 4,
    TQ_ERR_DEVICE_CHECK = 5
} tq_status;

/* Element type of K/V inputs and of queries. */
typedef enum { TQ_F32 = 0, TQ_BF16 = 1, TQ_F16 = 2 } tq_dtype;

/* A compressed cache: caller-owned device buffer of tq_cache_bytes() bytes,
 * 16-byte aligned, laid out as [B][Hkv][Tcap/64] blocks (Tcap a multiple of 64).
 * Paged form (block_table != NULL): base is a pool of pool_blocks blocks of
 * tq_block_bytes(d, is_k) bytes, and block_table (device int32
 * [B*Hkv][Tcap/64], row b*Hkv + h) gives the pool block that holds tokens
 * [64 lb, 64 lb + 64) of (batch b, kv head h).  Blocks of different sequences
 * may be anywhere in the pool; a block must not be shared by two live
 * (sequence, logical block) pairs that are written.  A table entry outside
 * [0, pool_blocks) is a device-side check failure (reported by
 * tq_device_status): nothing is written through it and reads go to block 0.
 * With block_table == NULL pool_blocks is ignored.
 * K block (64 tokens): codes 64 x 3d/8 B | signs 64 x d/8 B | ||k|| fp16 x 64 |
 *                      gamma = ||residual|| fp16 x 64
 * V block (64 tokens): codes 64 x 3d/8 B | ||v|| fp16 x 64
 * Per token the 3-bit codes are 3d/32 little-endian uint32 words.  Slice s
 * (128 coordinates) and slot t (0..3) own words 12s+3t+{0,1,2} (Wa, Wb, Wc)
 * holding slot codes i = 0..31, where slot code i is coordinate
 *     j = 128 s + 16 (i >> 2) + 2 t + (i & 1) + 8 ((i >> 1) & 1).
 * Nibble k of Wa: bits 0-2 = code(i = k), bit 3 = bit 0 of code(24 + k);
 * Wb: code(8 + k) and bit 1 of code(24 + k); Wc: code(16 + k) and bit 2 of
 * code(24 + k).  Signs are d/32 words per token; word 4s+t holds the sign of
 * JL row i = 2q at bit q and of row 2q+1 at bit 16+q (q = 0..15), rows mapped
 * to indices exactly as coordinates above.  d = 64 is one slice of 16 codes
 * per slot (i = 0..15, s = 0): word t (t = 0..3) holds code(k) in bits 0-2 of
 * nibble k (k = 0..7); halfword t of bytes 16..23 holds code(8 + k) in bits
 * 0-2 of nibble k (k = 0..3); bits 0, 1, 2 of code(12 + k) are bit 3 of
 * nibble k of word t, of nibble 4 + k of word t and of nibble k of halfword t.
 * Its signs are 4 halfwords per token: bit i of halfword t is the sign of the
 * JL row of slot position i.  A sign bit is 1 when the projection is >= 0.  Storage: (3d + m + 32)/d bits/dim for K (4.25 at
 * d = 128) and (3d + 16)/d for V (3.125 at d = 128). */
typedef struct {
    void* base;
    int64_t B;
    int64_t Hkv;
    int64_t Tcap;
    const int32_t* block_table;   /* NULL: contiguous cache */
    int64_t pool_blocks;
} tq_cache;

/* ---- constants -------------------------------------------------------- */

/* Compute the method's constants on the host, with no device involved:
 * D (d signs, +-1), S (m x d fp32, row-major, iid N(0,1)), the 8 codebook
 * centroids (ascending) and the 7 decision boundaries (midpoints).
 * Readings: counter-based SplitMix64 stream `seed`; D_j = -1 iff the top bit of
 * draw j is set; S from Box-Muller on draws d+2p, d+2p+1 (cosine output to
 * element 2p, sine output to 2p+1), rounded to fp32; centroids = the 8-level
 * Lloyd-Max quantiser of N(0,1) (K flow step 3), scaled by 1/sqrt(d), rounded
 * to fp16.  Any output pointer may be NULL.  Errors: INVALID_ARG (d not 64, 128
 * or 256). */
TQ_API tq_status tq_params_host(int head_dim, uint64_t seed, int8_t* D, float* S, float* centroids8,
                         float* bounds7);

/* Create a handle on the current CUDA device: computes the constants as
 * tq_params_host does and uploads them (the only allocating call).
 * Errors: INVALID_ARG (bad d or NULL out), CUDA. */
TQ_API tq_status tq_init(int head_dim, uint64_t seed, tq_handle** out);

/* Free the handle's device constants.  NULL is accepted. */
TQ_API tq_status tq_destroy(tq_handle* h);

/* Copy the handle's constants to host arrays (any may be NULL); synchronous. */
TQ_API tq_status tq_get_params(const tq_handle* h, int8_t* D, float* S, float* centroids8,
                        float* bounds7);

TQ_API int tq_head_dim(const tq_handle* h);

/* ---- sizes ------------------------------------------------------------ */

/* Bytes of one 64-token block; 0 for an unsupported d. */
TQ_API size_t tq_block_bytes(int head_dim, int is_k);

/* Bytes of a cache [B][Hkv][Tcap/64 blocks]; 0 if Tcap is not a positive
 * multiple of 64 or d is unsupported. */
TQ_API size_t tq_cache_bytes(int head_dim, int is_k, int64_t B, int64_t Hkv, int64_t Tcap);

/* ---- encode (K flow steps 1-5 / V steps 1-3) --------------------------- */

/* Encode Tnew new vectors per (batch, kv head) into token positions
 * [t0, t0 + Tnew) of the cache.  x is a device tensor of `dtype` with element
 * strides (sb, sh, st) for (batch, head, token) and a contiguous last
 * dimension of d elements: vector (b, h, t) starts at x + b*sb + h*sh + t*st.
 * Each vector is normalised (n = ||x||, stored as fp16), rotated, quantised
 * to 3-bit codes against the boundaries (a coordinate equal to a boundary
 * takes the upper cell), and for K the residual's norm gamma (fp16) and the
 * sign bits of S * residual are stored.  A zero vector stores code 4, gamma 0,
 * all signs 1.  Tokens outside [t0, t0+Tnew) are not touched.
 * Stream order holds as for any launch.  A bulk encode of 16-bit input (at
 * d = 64 and 128, at least 16384 contiguous vectors) starts its set-up while
 * the previous kernel on the stream finishes, and it waits for that kernel
 * before it reads x or writes the cache.
 * Errors: INVALID_ARG (NULL pointers, B/Hkv mismatch with the cache, Tnew < 0,
 * t0 < 0, t0 + Tnew > Tcap, misaligned x or cache), CUDA. */
TQ_API tq_status tq_encode_k(const tq_handle* h, const void* x, tq_dtype dtype, int64_t B, int64_t Hkv,
                      int64_t Tnew, int64_t sb, int64_t sh, int64_t st, const tq_cache* kc,
                      int64_t t0, void* stream);
TQ_API tq_status tq_encode_v(const tq_handle* h, const void* x, tq_dtype dtype, int64_t B, int64_t Hkv,
                      int64_t Tnew, int64_t sb, int64_t sh, int64_t st, const tq_cache* vc,
                      int64_t t0, void* stream);

/* ---- decode attention --------------------------------------------------- */

/* Workspace bytes tq_attend_decode needs for these sizes on this handle's
 * device (query rotation, per-split softmax partials).  0 on bad arguments. */
TQ_API size_t tq_attend_workspace_bytes(const tq_handle* h, int64_t B, int64_t Hq, int64_t Hkv,
                                 int64_t Tmax);

/* Decode attention over the compressed cache: the page's hybrid V2+V3 section
 * (dequantisation fused into the attention kernel, which reads the packed
 * cache directly), with scores from its K section (3-bit codes plus the 1-bit
 * QJL residual correction) and values from its V section.
 * One decode step of attention for B x Hq queries (q [B][Hq][d] contiguous,
 * `qdtype`) over the compressed caches kc (K) and vc (V).  Query head h uses
 * kv head h / (Hq/Hkv).  Sequence b attends over tokens [0, seq_lens[b]) when
 * seq_lens (device int32[B]) is not NULL, else over [0, T).  Computes, per
 * query head, q' = H D q, u = S q' and
 *   s_t = scale * n_t * (<q', c[idx_t]> + gamma_t * sqrt(pi/2)/m * <u, 2 sigma_t - 1>),
 *   out = D H sum_t softmax(s)_t * nv_t * c[idxv_t],
 * with n_t, gamma_t, nv_t the stored fp16 values, in fp32 with split-K
 * (flash-decoding) partials in `ws` merged by a final kernel.  out is fp32
 * [B][Hq][d]; an empty sequence gives zeros.  Supported: d in {64, 128, 256},
 * any Hq/Hkv (kv heads with more than 8 query heads are served in groups of
 * up to 8), B <= 65535, Hkv * ceil(Hq/Hkv / 8) <= 65535, B * Hq < 2^31.  ws must be 256-byte
 * aligned with at least
 * tq_attend_workspace_bytes(h, B, Hq, Hkv, T or max seq_len) bytes.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
TQ_API tq_status tq_attend_decode(const tq_handle* h, const void* q, tq_dtype qdtype, int64_t B,
                           int64_t Hq, const tq_cache* kc, const tq_cache* vc,
                           const int32_t* seq_lens, int64_t T, float scale, float* out, void* ws,
                           size_t ws_bytes, void* stream);

/* ---- PolarQuant-only K (no QJL bit) --------------------------------------- */

/* Attention over a PolarQuant-only K cache: K stored like V, with 3-bit codes
 * and the fp16 norm but no QJL sign bits and no gamma (3.125 bits/dim at
 * d = 128 instead of 4.25).  Encode such a K cache with tq_encode_v into a
 * V-layout buffer (tq_cache_bytes(d, 0, ...)).  Scores drop the QJL term:
 *   s_t = scale * n_t * <q', c[idx_t]>,
 * the rest as tq_attend_decode (same arguments, workspace and errors).  The
 * page weighs the two K flows against each other: its K section adds the
 * 1-bit QJL residual to correct the inner-product bias of the 3-bit codes,
 * and its hybrid V2+V3 section trades that accuracy against the faster
 * PolarQuant-only path. */
TQ_API tq_status tq_attend_decode_polar(const tq_handle* h, const void* q, tq_dtype qdtype, int64_t B,
                                        int64_t Hq, const tq_cache* kc, const tq_cache* vc,
                                        const int32_t* seq_lens, int64_t T, float scale, float* out, void* ws,
                                        size_t ws_bytes, void* stream);

/* ---- chunked prefill ------------------------------------------------------ */

/* Workspace bytes tq_attend_prefill needs (rotated queries and the softmax
 * partials of B * Lq * Hq query rows; at head_dim 128 a row tile's tokens may
 * be spread over several CTAs, each writing one partial, up to a bound that
 * depends on the row count and the device's SM count).  0 on bad arguments. */
TQ_API size_t tq_prefill_workspace_bytes(const tq_handle* h, int64_t B, int64_t Lq, int64_t Hq);

/* Attention for a chunk of Lq new queries per sequence (q [B][Lq][Hq][d]
 * contiguous, `qdtype`) over the compressed caches, causal: query i of the
 * chunk attends over tokens [0, T0 + i] of its sequence, so the chunk's own K
 * and V must already be encoded at positions T0 .. T0 + Lq - 1.  Scores and
 * output as tq_attend_decode (the same estimator, in the page's K section and
 * hybrid V2+V3 section); out is fp32 [B][Lq][Hq][d].  With many queries per
 * kv head the score and value contractions are dense and run on tensor cores:
 * at d = 128 on tcgen05 with each 64-token block dequantised once per 128
 * query rows (q' and u' as fp16 hi and lo limbs), the row tiles' token ranges
 * spread evenly over one CTA per SM; at d = 64 and 256 on mma.sync tiles with
 * the keys dequantised once per 16 query rows and the QJL term on 16-bit
 * fixed-point u' (at d = 256 two CTAs share each 64 query rows, each
 * accumulating half of the value coordinates).  Supported: d in {64, 128,
 * 256}, any Hq/Hkv, B <= 65535, Lq Hq / Hkv <= 2^27, T0 + Lq <= Tcap;
 * contiguous or paged caches.  Errors: INVALID_ARG, UNSUPPORTED (grid or size
 * limits), WORKSPACE, CUDA. */
TQ_API tq_status tq_attend_prefill(const tq_handle* h, const void* q, tq_dtype qdtype, int64_t B, int64_t Lq,
                                   int64_t Hq, const tq_cache* kc, const tq_cache* vc, int64_t T0, float scale,
                                   float* out, void* ws, size_t ws_bytes, void* stream);

/* ---- fused append-and-attend step ---------------------------------------- */

/* One decode step of a serving loop: encode Tnew new K and V vectors per
 * (batch, kv head) into token positions [t0, t0 + Tnew) of kc and vc, then
 * attend for B x Hq queries over tokens [0, t0 + Tnew) of every sequence.
 * The page's decode loop appends each generated token's K/V to the
 * compressed cache and attends over it (page "Apple Silicon向けSwiftLM ...",
 * K/V sections and the hybrid V2+V3 section); this call does both in one
 * launch chain.  Results (cache bytes and out) are identical to
 * tq_encode_k + tq_encode_v + tq_attend_decode with T = t0 + Tnew.
 * k_new and v_new share `kv_dtype` and the element strides (sb, sh, st) as in
 * tq_encode_k; B and Hkv are the caches'.  q, out, ws and scale as in
 * tq_attend_decode (ws sized by tq_attend_workspace_bytes(h, B, Hq, Hkv,
 * t0 + Tnew)).  The kernels are chained with programmatic dependent launch:
 * the query prologue runs alongside the encodes and the attention kernel
 * sets up while they run, reading the cache only after they complete; every
 * kernel completes only after the one before it, so the next work on the
 * stream sees the finished step.
 * Errors: those of tq_encode_k and tq_attend_decode (checked before any
 * launch). */
TQ_API tq_status tq_append_attend(const tq_handle* h, const void* k_new, const void* v_new, tq_dtype kv_dtype,
                                  int64_t Tnew, int64_t sb, int64_t sh, int64_t st, const tq_cache* kc,
                                  const tq_cache* vc, int64_t t0, const void* q, tq_dtype q_dtype, int64_t Hq,
                                  float scale, float* out, void* ws, size_t ws_bytes, void* stream);

/* ---- decode attention without device allocation ------------------------- */

/* Size of the scratch array inside the library used by tq_attend_decode_static. */
#define TQ_STATIC_SCRATCH_BYTES (8u << 20)

/* The method's pages have no counterpart to this call; it exists for callers.
 * Same computation, arguments and results as tq_attend_decode, but with no
 * workspace argument: the scratch (rotated queries, split-K partials) is a
 * fixed TQ_STATIC_SCRATCH_BYTES (8 MiB) array inside the library, which every
 * GPU that loads the library keeps until the process exits.  It is for callers
 * that cannot allocate device memory when they run a decode step: a plugin or
 * custom operator handed only input and output pointers by a host framework
 * that owns the allocator, a serving loop that fixes its memory budget at
 * start-up and must not grow it or pay an allocation's implicit
 * synchronisation per token, or a deployment that forbids dynamic device
 * allocation after initialisation.  Nothing here calls cudaMalloc or cudaFree.
 * The first call on each device resolves the array's device address
 * (cudaGetSymbolAddress, with that device current) and caches it; make that
 * first call before any stream capture.  Sizes that need more scratch than
 * the array holds (tq_attend_workspace_bytes(...) above 8 MiB) are rejected
 * with TQ_ERR_WORKSPACE before anything is launched.  All calls on a device
 * share the one array and it keeps the last call's contents (every byte a call
 * reads is written by that call first, so nothing needs clearing); calls that
 * overlap on the GPU -- on different streams, or from different threads --
 * race on it and must be serialised by the caller.
 * Errors: those of tq_attend_decode; CUDA if the address cannot be resolved. */
TQ_API tq_status tq_attend_decode_static(const tq_handle* h, const void* q, tq_dtype qdtype, int64_t B,
                                         int64_t Hq, const tq_cache* kc, const tq_cache* vc,
                                         const int32_t* seq_lens, int64_t T, float scale, float* out,
                                         void* stream);

/* ---- 4-bit caches ------------------------------------------------------- */

/* A cache of plain 4-bit codes with group scales, beside the TurboQuant
 * caches: no rotation and no codebook, 4 + 32 / group bits per value (4.5 at
 * group 64).  Each vector of d values is cut into groups of `group`
 * consecutive values (32, 64 or 128, at most d).  A group stores an fp16 zero
 * and an fp16 scale, a value stands for zero + scale * code:
 *   x taken within +-65504;  zero = fp16(min x)
 *   scale = fp16((max x - zero) * fp32(1/15));  r = 1 / scale (0 if scale <= 0)
 *   code = min(15, max(0, rint((x - zero) * r)))     (half to even)
 * each step one correctly rounded fp32 operation.  A group with a NaN stores
 * NaN for both.  K and V have the same format.  The cache is a tq_cache
 * (contiguous or paged, 64 tokens per block) whose blocks are
 * tq_int4_block_bytes(d, group) long: codes 64 x d/2 B | (scale, zero) fp16
 * pairs 64 x d/group x 4 B.  Byte j of token tau's codes (values 2j in the low,
 * 2j + 1 in the high nibble) is stored at j ^ 16 s, s = (tau & 2 if d >= 128,
 * else 0) + (4 (tau & 1) if d = 256, else 0). */

/* Bytes of one 64-token block; 0 for an unsupported d or group. */
TQ_API size_t tq_int4_block_bytes(int head_dim, int group);

/* Bytes of a contiguous cache; 0 as tq_cache_bytes, or for an unsupported group. */
TQ_API size_t tq_int4_cache_bytes(int head_dim, int group, int64_t B, int64_t Hkv, int64_t Tcap);

/* Encode T new vectors per (batch, kv head); x, dtype and strides as
 * tq_encode_k.  Token i of sequence b goes to position pos[b] + i (pos: device
 * int32[B]), or t0 + i when pos is NULL.  Positions from pos outside
 * [0, Tcap), and positions on a bad block-table entry, are skipped and
 * reported by tq_device_status.  Other tokens are not touched.
 * Errors: INVALID_ARG (as tq_encode_k; a bad group), UNSUPPORTED (2^31 words
 * of 8 values or more), CUDA. */
TQ_API tq_status tq_encode_int4(const tq_handle* h, int group, const void* x, tq_dtype dtype, int64_t B, int64_t Hkv,
                                int64_t T, int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos,
                                int64_t t0, void* stream);

/* Read T tokens per (batch, kv head) back as values of `dtype` (fp32 value
 * zero + scale * code rounded once); positions as tq_encode_int4, x is the
 * output with its strides (no two vectors on the same bytes).  Vectors of
 * skipped positions are left as they were.  Errors: as tq_encode_int4. */
TQ_API tq_status tq_expand_int4(const tq_handle* h, int group, void* x, tq_dtype dtype, int64_t B, int64_t Hkv,
                                int64_t T, int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos,
                                int64_t t0, void* stream);

/* Workspace bytes of tq_attend_int4 and tq_append_attend_int4 on this handle's
 * device; it does not depend on the context length.  0 on bad arguments. */
TQ_API size_t tq_attend_int4_workspace_bytes(const tq_handle* h, int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv);

/* Attention of Lq >= 1 new queries per sequence over 4-bit caches (Lq = 1: a
 * decode step; small Lq: speculative tokens; large Lq: a prefill chunk).
 * q and out are [B][Lq][Hq][d] contiguous, both of `qdtype`.  Sequence b has
 * n = seq_lens[b] tokens (device int32[B]; clamped to [0, Tcap]), or n = T when
 * seq_lens is NULL, its Lq newest among them: query i attends over tokens
 * [0, n - Lq + 1 + i), and a query that sees none gives zeros.  Query head h
 * uses kv head h / (Hq/Hkv); scores are scale <q, k>, softmax and sums in fp32.
 * What lies in the caches behind a query's last visible token has no effect on
 * it, whatever it is.  Sequences may have any mixture of lengths: the work is
 * shared out over the SMs on the device.  Precision: sums, maxima and softmax
 * statistics are fp32 (integer products exact); queries, keys, weights and
 * values carry at least 22 bits for fp32 and fp16 calls.  bf16 calls round the
 * weights times the value scales to fp16 (2^-11, against 2^-8 of their output),
 * and with more than 16 query rows per kv head (head_dim 64 and 128) the
 * expanded keys and values too, to 65504 at most (a group whose maximum is
 * clipped there may stand for up to 64 more).
 * Those calls, and fp32 and fp16 ones of more than 32 rows, sum all tokens on
 * the tensor core, which truncates: values with a mean come out low by up to
 * 8e-6 (fp32) or 1.3e-4 (fp16) of it however long the context, in bf16 calls by
 * 3e-4 per 1000 blocks of 64 tokens that one SM walks.
 * Supported: any Hq/Hkv, B < 2^31, Lq * Hq / Hkv < 2^31, Hkv * row groups <
 * 2^31 (row groups: query rows per kv head / 4, rounded up); contiguous or
 * paged caches.  ws: 256-byte aligned, at least
 * tq_attend_int4_workspace_bytes(h, B, Lq, Hq, Hkv) bytes; two calls that may
 * overlap on the GPU need two workspaces.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
TQ_API tq_status tq_attend_int4(const tq_handle* h, int group, const void* q, tq_dtype qdtype, int64_t B, int64_t Lq,
                                int64_t Hq, const tq_cache* kc, const tq_cache* vc, const int32_t* seq_lens, int64_t T,
                                float scale, void* out, void* ws, size_t ws_bytes, void* stream);

/* One serving step: encode Lq new K and V vectors per (batch, kv head) at
 * positions pos[b] + i (t0 + i when pos is NULL) of kc and vc, then attend
 * with their Lq queries over the pos[b] + Lq tokens.  Results are those of
 * tq_encode_int4 on both caches and tq_attend_int4 with seq_lens = pos + Lq.
 * k_new and v_new share kv_dtype and strides.  The encodes are one launch, and
 * the attention's set-up overlaps it.  kc and vc must not share blocks
 * (contiguous caches that overlap, or one pool under one table, are refused).
 * Errors: those of tq_encode_int4 and tq_attend_int4, before any launch. */
TQ_API tq_status tq_append_attend_int4(const tq_handle* h, int group, const void* k_new, const void* v_new,
                                       tq_dtype kv_dtype, int64_t Lq, int64_t sb, int64_t sh, int64_t st,
                                       const tq_cache* kc, const tq_cache* vc, const int32_t* pos, int64_t t0,
                                       const void* q, tq_dtype q_dtype, int64_t Hq, float scale, void* out, void* ws,
                                       size_t ws_bytes, void* stream);

/* ---- pages of paged caches ----------------------------------------------- */

/* The pages that hold paged caches of any format, managed on the device so
 * that a captured serving step needs no host bookkeeping.  block_table (device
 * int32 [B*Hkv][NB], rows as tq_cache's, -1: no page) and refs (device
 * int32[pool_blocks]) are the state: refs[p] is the number of table entries
 * that name page p, and a page with 0 is free.  An empty state is a table of
 * -1 and zero refs.  Page p is block p of each of the n_buffers pools
 * `buffers` (device pointers, 16-byte aligned, in a host array) with
 * block_bytes[i] bytes per page (multiples of 16): the K and the V pool of one
 * layer or of several that share the table.  The same block_table goes into
 * the tq_cache of each.  A cache whose pages are shared (refs > 1) must not be
 * written there: tq_pages_alloc gives the writer its own copy first.
 * Any negative entry counts as -1.  Entries of pool_blocks or more are left
 * alone and reported by tq_device_status, as are indices out of range.  Calls enqueue kernels, do
 * not synchronise, and their outcome does not depend on thread order.  One
 * call at a time may work on a state. */
#define TQ_MAX_PAGE_BUFFERS 128
typedef struct {
    int32_t* block_table;
    int32_t* refs;
    int64_t B, Hkv, NB;
    int64_t pool_blocks;
    int32_t n_buffers;            /* 0 .. TQ_MAX_PAGE_BUFFERS */
    void* const* buffers;         /* host array */
    const int64_t* block_bytes;   /* host array */
} tq_pages;

/* Workspace bytes of tq_pages_alloc and tq_pages_compact; 0 on bad arguments. */
TQ_API size_t tq_pages_workspace_bytes(const tq_pages* p);

/* Make tokens [lo[b], hi[b]) of every sequence writable (device int32[B];
 * lo = hi: nothing asked): a block of them without a page gets a fresh one,
 * and a block whose page has refs > 1 gets a fresh copy of it (copy on write;
 * the page loses one reference).  Fresh pages are the free ones in ascending
 * order, given to the asking blocks in (row, block) order; contents of fresh
 * pages that are no copies are undefined.  When the pool runs out the rest of
 * the blocks stay as they are.  info (device int32[2], may be NULL): pages
 * free afterwards, blocks left without.  Errors: INVALID_ARG, UNSUPPORTED
 * (2^31 table entries or more), WORKSPACE, CUDA. */
TQ_API tq_status tq_pages_alloc(const tq_handle* h, const tq_pages* p, const int32_t* lo, const int32_t* hi,
                                int32_t* info, void* ws, size_t ws_bytes, void* stream);

/* Every sequence b takes the pages of sequence parent[b] as they were before
 * the call (device int32[B]; b itself: unchanged, -1: none): entries are
 * shared, not copied, and refs follow on both sides.  Any mapping is allowed,
 * exchanges and repeated parents included; a parent outside [-1, B) leaves its
 * sequence unchanged and is reported.  Errors: INVALID_ARG, UNSUPPORTED
 * (B > 7168, Hkv > 65535), CUDA. */
TQ_API tq_status tq_pages_fork(const tq_handle* h, const tq_pages* p, const int32_t* parent, void* stream);

/* Release what sequence b holds behind its first keep[b] tokens (device
 * int32[B]; <= 0: everything): blocks from ceil(keep[b] / 64) on lose their
 * page (entry -1, refs - 1).  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
TQ_API tq_status tq_pages_free(const tq_handle* h, const tq_pages* p, const int32_t* keep, void* stream);

/* Move the live pages (refs > 0) into the lowest places of the pools: with L
 * of them, the k-th lowest free page below L takes the contents and references
 * of the k-th highest live page, and the table follows.  Pages from L on are
 * free afterwards (their contents are left).  info (device int32[2], may be
 * NULL): free pages, pages moved.  Errors: as tq_pages_alloc. */
TQ_API tq_status tq_pages_compact(const tq_handle* h, const tq_pages* p, int32_t* info, void* ws, size_t ws_bytes,
                                  void* stream);

/* Copy pages src[i] of `from`'s buffers to pages dst[i] of `to`'s (device
 * int32[n]), buffer by buffer; tables and refs are not used.  `from` and `to`
 * need the same buffer count and block_bytes, and may be the same.  Pairs with
 * a -1 are skipped; indices out of range are skipped and reported.  A page may
 * be read many times, but each written page must appear once and not be read.
 * Errors: INVALID_ARG, CUDA. */
TQ_API tq_status tq_pages_copy(const tq_handle* h, const tq_pages* from, const tq_pages* to, const int32_t* src,
                               const int32_t* dst, int64_t n, void* stream);

/* ---- diagnostics -------------------------------------------------------- */

/* Synchronise `stream`, then report and clear the handle's device check word:
 * TQ_ERR_DEVICE_CHECK if a kernel gave up a bounded wait since the last call. */
TQ_API tq_status tq_device_status(const tq_handle* h, void* stream);

/* Diagnostics: when ev_start/ev_stop (cudaEvent_t, created by the caller) are
 * not NULL, each later tq_attend_decode records ev_start just before its
 * split-K attention kernel and ev_stop just after it, on the call's stream, so
 * the caller can time that kernel alone.  Pass NULLs to stop.  Not thread-safe
 * with concurrent tq_attend_decode calls on the same handle. */
TQ_API tq_status tq_set_decode_events(tq_handle* h, void* ev_start, void* ev_stop);

/* Diagnostics: the number of times each warp of the split-K attention kernel
 * polls the mbarrier of its first staged chunk before giving up (every wait in
 * the kernels is bounded; normally 2^20 polls).  A give-up sets the handle's
 * check word, waits with the full bound for the warp's copies still in flight,
 * and leaves that warp's tokens out of the result (the outputs of such a call
 * are not the attention; tq_device_status reports TQ_ERR_DEVICE_CHECK).  0
 * makes every first wait give up at once, which lets a test exercise this path
 * without a fault; a negative value restores the full bound.  Not thread-safe
 * with concurrent calls on the same handle.  Errors: INVALID_ARG (NULL h). */
TQ_API tq_status tq_set_wait_limit(tq_handle* h, int first_wait);

/* Diagnostics: choose the decode kernel of later tq_attend_decode calls on this
 * handle: 0 = automatic (tensor-core kernel where supported, with the work
 * partition its cost model prefers), 1 = the SIMT kernel, 2 = the tensor-core
 * kernel on the uniform split grid only, 3 = the tensor-core kernel on the
 * stream-K grid wherever that fits (sequences of one length, no more
 * (batch, kv head, head group) units than CTA slots, partial slots within the
 * workspace bound).  Paths 0, 2 and 3 give the same outputs up to the fp32
 * order of the softmax merge.  Changes the workspace size
 * tq_attend_workspace_bytes reports (path 1).  Errors: INVALID_ARG (NULL h,
 * path outside 0..3). */
TQ_API tq_status tq_set_decode_path(tq_handle* h, int path);

/* Diagnostics, host only (no device or handle needed): the work partition the
 * tensor-core decode takes for a call of these sizes (head_dim, B sequences,
 * Hq / Hkv heads, T tokens) on a GPU with num_sms SMs, automatic path.
 * equal_len != 0: every sequence has T tokens (a call without seq_lens; only
 * then is the stream-K grid considered), else T is the cache capacity.
 * Outputs: *nsplit partial slots per query head; *split_tokens tokens per
 * split of the uniform grid; *streamk_ctas the CTAs of the stream-K grid (0:
 * the uniform grid is used) and *streamk_chunks the chunks of one (batch, kv
 * head, query-head group) unit that it divides; *chunk_tokens tokens per chunk.
 * Errors: INVALID_ARG (head_dim not 64/128/256, sizes as tq_attend_decode
 * rejects them, num_sms < 1, a NULL output). */
TQ_API tq_status tq_decode_plan(int num_sms, int head_dim, int64_t B, int64_t Hq, int64_t Hkv, int64_t T,
                                int equal_len, int* nsplit, int64_t* split_tokens, int64_t* streamk_ctas,
                                int64_t* streamk_chunks, int* chunk_tokens);

/* Name of the kernel path tq_attend_decode uses for these sizes on this handle
 * ("mma" or "simt"); static string. */
TQ_API const char* tq_attend_path(const tq_handle* h, int64_t Hq, int64_t Hkv);

TQ_API const char* tq_status_string(tq_status s);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H_ */
