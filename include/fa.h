/*
 * fa.h — C ABI of the GB300 (sm_103a) exact-attention library.
 *
 * The library computes exact scaled-dot-product attention the IO-aware way:
 * the forward pass streams K/V tiles through on-chip memory, keeps a running
 * row maximum and sum (online softmax) and writes only O and the per-row
 * logsumexp; the backward pass recomputes S and P on chip from that
 * logsumexp and produces dQ, dK and dV without writing any N x N matrix to
 * device memory.  (FlashAttention deep-read report, sections 2.4 "tiling and
 * incremental softmax", 2.5 "recomputation", 3.2 "Algorithm 1" and 3.3
 * "backward pass and memory layout"; Attention Kernel page, "FlashAttention's
 * insight: IO-aware" and "why tiling also works for training".)
 *
 * Conventions shared by every entry point
 *   - q, k, v, o, dout, dq, dk, dv: bf16, contiguous, layout [B, H, N, d]
 *     (row-major; element (b,h,i,c) at ((b*H + h)*N + i)*d + c). Device
 *     pointers, 16-byte aligned. A [B, N, H, d] tensor must be transposed
 *     by the caller first.
 *   - lse: fp32 [B, H, N], natural-log logsumexp of the scaled scores of each
 *     query row (this replaces the pair (m, l) that the pages store); a row
 *     with no allowed key gets -inf and O = 0 for that row.
 *   - d (head dimension) must be 64 or 128; N >= 1; B, H >= 1;
 *     B*H*N < 2^31.
 *   - scale > 0 multiplies Q K^T (the usual value is 1/sqrt(d)).
 *   - causal != 0 masks key j for query i when j > i (square, top-left aligned).
 *   - seqlens_k (nullable): device int32 [B]; keys j >= seqlens_k[b] are
 *     masked for every query row of batch b (key padding; query rows are still
 *     computed). Values are clamped to [0, N].
 *   - block_mask (nullable): device uint8 [nb, nb], nb = ceil(N / 128), row
 *     major, shared by all (b, h): a zero byte at (r, c) removes every pair
 *     with query block r and key block c (FlashAttention deep-read report,
 *     sections 2.6 and 3.5, block-sparse attention; blocks are 128 x 128).
 *     The C entry points receive only the two pointers and cannot check the
 *     sizes of these arrays: a shorter seqlens_k or block_mask makes the
 *     kernels read past its end. (The Python binding checks both shapes.)
 *   - dropout_p in [0, 1): dropout on the normalised probabilities, applied
 *     on chip (deep-read report section 3.2). It is quantised to
 *     p8 = round(256 p) and the effective rate is p8/256 (see fa_dropout_p8).
 *     Element (b,h,i,j) is dropped iff byte (j & 15) of
 *       Philox4x32-10(counter = (j >> 4, (b*H + h)*N + i, lo32(offset), hi32(offset)),
 *                     key = (lo32(seed), hi32(seed)))
 *     is below p8 (byte index j&15 = word (j&15)>>2, little-endian byte j&3),
 *     Philox as published by Salmon, Moraes, Dror and Shaw (SC'11). Kept
 *     elements are scaled by 1/(1 - p8/256). fa_fwd and fa_bwd must be given
 *     the same seed and offset. The logsumexp is that of the undropped softmax.
 *   - stream: a cudaStream_t (NULL = legacy default stream). Every call is
 *     asynchronous on that stream; the return value reports argument errors
 *     and launch failures only.
 *   - The library never allocates device memory. The caller owns every buffer.
 *   - Device-side failures (a bounded wait that ran out) are recorded in a
 *     per-device status word; fa_device_status() reads and optionally clears it.
 */
#ifndef FA_GB300_H_
#define FA_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null/unaligned pointer, bad size, bad value */
  FA_ERR_UNSUPPORTED = 2, /* head dimension other than 64/128, not an sm_100-family GPU */
  FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (launch, attribute) */
  FA_ERR_WORKSPACE = 4,   /* workspace missing or smaller than fa_bwd_workspace_size() */
  FA_ERR_TIMEOUT = 5      /* a device-side wait ran out (reported by fa_device_status) */
} fa_status;

/* Forward pass: O = softmax(scale * Q K^T, masked) V, plus lse.
 * Writes o [B,H,N,d] bf16 and lse [B,H,N] fp32 (both device). */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, float dropout_p, uint64_t seed,
                 uint64_t offset, const uint8_t* block_mask, const int32_t* seqlens_k,
                 void* stream);

/* Bytes of device workspace fa_bwd needs (the per-row D = rowsum(dO * O), fp32 [B,H,N],
 * rounded up to 256 bytes). */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/* Backward pass of L = sum(O * dO) for the forward above. o and lse are the
 * forward's outputs for the same inputs and options. Writes dq, dk, dv
 * (bf16 [B,H,N,d], device). workspace: device, >= fa_bwd_workspace_size(),
 * 16-byte aligned; its contents on entry do not matter. Three kernels run in
 * order on `stream`: D = rowsum(dO * O); dK and dV (one pass over key tiles,
 * recomputing S^T and P^T); dQ (one pass over query tiles, recomputing S and P).
 * dQ is accumulated without atomics, so every output is deterministic. */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, float dropout_p, uint64_t seed, uint64_t offset,
                 const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Grouped-query attention (query heads sharing K/V heads, which the page
 * "Attention Kernel: FlashAttention 与它的后继者", section on FlashAttention's
 * IO-aware insight, names as a further cut of K/V reads): H query heads and
 * H_kv K/V heads, H a multiple of H_kv, query head h of batch row b attending
 * with K/V head h / (H / H_kv).
 * q, o, dout, dq: bf16 [B,H,N,d]; k, v, dk, dv: bf16 [B,H_kv,N,d]; lse:
 * fp32 [B,H,N]. dk and dv of a K/V head are the sums over the query heads
 * that share it, formed on chip (the key-tile kernel walks every query head
 * of the group), so they stay atomic-free and deterministic. Dropout keys on
 * the query head, as for H independent heads. H_kv = H is fa_fwd / fa_bwd;
 * H_kv = 1 is multi-query attention. Errors as for fa_fwd / fa_bwd, plus
 * FA_ERR_INVALID_ARG when H_kv < 1 or H % H_kv != 0. The workspace is
 * fa_bwd_workspace_size(B, H, N, d). */
fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int H, int H_kv, int N, int d, float scale, int causal, float dropout_p,
                     uint64_t seed, uint64_t offset, const uint8_t* block_mask,
                     const int32_t* seqlens_k, void* stream);
fa_status fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, int B, int H, int H_kv, int N,
                     int d, float scale, int causal, float dropout_p, uint64_t seed,
                     uint64_t offset, const uint8_t* block_mask, const int32_t* seqlens_k,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Sliding-window (local) attention, with every other option of fa_fwd_gqa /
 * fa_bwd_gqa: key j is visible to query i only if
 * i - window_left <= j <= i + window_right (-1 leaves that side unbounded);
 * it composes with causal (which caps j <= i), key padding and the block mask.
 * The cross-paper synthesis page on FlashAttention lists sliding-window
 * attention among the variants an IO-aware kernel should cover (section 5),
 * and the Attention Kernel page counts sliding windows among the sparse
 * patterns whose blocks are skipped (section on xFormers, cuDNN and sparse
 * attention). The kernels skip every 128 x 128 tile the band misses and mask
 * elements only on tiles an edge crosses, so the work is O(N * window).
 * Arguments, layouts, outputs and errors are those of fa_fwd_gqa /
 * fa_bwd_gqa, plus FA_ERR_INVALID_ARG when a window bound is below -1. */
fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int H, int H_kv, int N, int d, float scale, int causal, int window_left,
                        int window_right, float dropout_p, uint64_t seed, uint64_t offset,
                        const uint8_t* block_mask, const int32_t* seqlens_k, void* stream);
fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int H, int H_kv, int N, int d, float scale, int causal, int window_left,
                        int window_right, float dropout_p, uint64_t seed, uint64_t offset,
                        const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Attention of queries over keys of another length (cross attention to an encoder's states, or to
 * a memory in front of the queries), with or without a learned bias by relative position, and
 * its backward pass. (The cross-paper synthesis page on FlashAttention lists cross attention
 * among the variants an IO-aware kernel should cover, section 5.)
 *   q, o, dout, dq: bf16 [B, H, Nq, d]; k, v, dk, dv: bf16 [B, H_kv, Nk, d]; lse: fp32
 *   [B, H, Nq]; contiguous, 16-byte aligned. Query head h attends with K/V head h / (H / H_kv).
 *   Query i sits at position p = i + q_offset of the key axis (0: at key i; Nk - Nq: at the last
 *   Nq positions). Key j is visible to it if j < seqlens_k[b] (Nk if null; clamped to [0, Nk]),
 *   with causal j <= p, and p - window_left <= j <= p + window_right (-1: unbounded). A row that
 *   sees no key gets O = 0, lse = -inf and no gradient. What K and V hold at and behind
 *   seqlens_k[b], NaN and infinities too, does not matter; dK and dV are 0 there.
 *   Dropout as in fa_fwd, with row index (b*H + h)*Nq + i.
 *   rel_lines: null, or the bias of the scores as fa_rel_bias laid it out for H heads and these
 *   rel_left and rel_right: key j gets the bias of distance j - p.
 *   dtable: null, or fp32 [num_buckets, H], the gradient of the bias table: entry (n, h) is the
 *   sum of dS of head h over the pairs whose distance maps to n (rel_map: as given to
 *   fa_rel_bias; entries outside [0, num_buckets) take part in no sum). Written whole. Its sums
 *   are fp32, the last ones (over distances and over the keys beyond the range) with what each
 *   addition rounds off kept, and are taken with the D of the unrounded O.
 * fa_bwd_cross: o and lse are fa_fwd_cross's outputs for the same inputs and options, over all the
 * keys that they were computed from. (D is formed from the scores where a query tile sees a single key
 * tile, without a look at o, and dtable rests on a row's weights summing to one: with the o and lse of an
 * attention whose keys are divided among several calls these gradients would be wrong.)
 * Every output is deterministic on one device. fa_bwd_cross runs the kernels of fa_bwd; one that
 * takes the D of rows whose tile sees a single key tile from their scores, since few weights leave
 * nothing over which O's rounding would even out (not launched where no row can be one); and
 * for dtable three more: the tiles near the diagonal, the sums by distance and beyond the range,
 * those by bucket. Where there are few key tiles (B*H_kv*ceil(Nk/128) well below the number of SMs)
 * the dK/dV kernel's CTAs share the queries of each and another kernel adds up their parts, which
 * the workspace has room for (at most 304 * d KB). workspace:
 * fa_bwd_cross_workspace_size(...) bytes (rel_grad: whether dtable is wanted), 16-byte aligned;
 * its contents on entry do not matter; calls that may overlap need one each.
 * Errors: FA_ERR_INVALID_ARG (as for fa_fwd and fa_bwd; Nq or Nk above 2^28, |q_offset| above
 * 2^28, B*H_kv*Nk >= 2^31, a window bound below -1, a dtable without lines or map),
 * FA_ERR_UNSUPPORTED (d, more than 65536 distances or buckets or 65535 heads with a bias),
 * FA_ERR_WORKSPACE, FA_ERR_CUDA. Asynchronous on `stream`; nothing is allocated. */
fa_status fa_fwd_cross(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                       int q_offset, int window_left, int window_right, float dropout_p,
                       uint64_t seed, uint64_t offset, const int32_t* seqlens_k,
                       const float* rel_lines, int rel_left, int rel_right, void* stream);
size_t fa_bwd_cross_workspace_size(int B, int H, int Nq, int Nk, int d, int causal, int q_offset,
                                   int rel_grad, int rel_left, int rel_right);
fa_status fa_bwd_cross(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                       int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                       int q_offset, int window_left, int window_right, float dropout_p,
                       uint64_t seed, uint64_t offset, const int32_t* seqlens_k,
                       const float* rel_lines, int rel_left, int rel_right,
                       const int32_t* rel_map, int num_buckets, float* dtable, void* workspace,
                       size_t workspace_bytes, void* stream);

/* A learned bias of the scores by relative position, in buckets of distances: key j gets
 * table[map[clamp(j - p, -left, right) + left], h] from the query at position p in head h.
 * fa_rel_bias lays it out for the attention calls, a line of fa_rel_line_length(left, right)
 * floats per head (0 where left or right is out of range), in log2 units and in an order of its own:
 *   table: [num_buckets, H], fp32 (FA_TABLE_F32) or bf16 (FA_TABLE_BF16), contiguous, device;
 *          an entry of -2^15 or lower, -inf among them, hides the bucket's keys (a row whose keys
 *          are all hidden sees none); one above 2^15 counts as 2^15 and is reported as
 *          FA_ERR_INVALID_ARG by fa_device_status. Between them a weight is off by what fp32 scores of
 *          that size round, a few times 2^-24 of the score.
 *   map:   int32 [left + right + 1], device: the bucket of distances -left .. right. An entry
 *          outside [0, num_buckets) gives a bias of 0 and is reported as FA_ERR_INVALID_ARG by
 *          fa_device_status.
 *   lines: fp32 [H, fa_rel_line_length(left, right)], device, 16-byte aligned
 * A line holds the table's values as they were: lay it out again after the table changes.
 * Errors: FA_ERR_INVALID_ARG (null or unaligned pointers, sizes below 1, left or right below 0),
 * FA_ERR_UNSUPPORTED (left + right + 1 or num_buckets above 65536, H above 65535, type),
 * FA_ERR_CUDA. Asynchronous on `stream`; nothing is allocated. */
typedef enum { FA_TABLE_F32 = 0, FA_TABLE_BF16 = 1 } fa_table_type;
int fa_rel_line_length(int left, int right);
fa_status fa_rel_bias(const void* table, int table_type, const int32_t* map, int left, int right,
                      int num_buckets, int H, float* lines, void* stream);

/* fa_rel_bias with its arguments in a block (see fa_paged_attn_block). */
fa_status fa_rel_bias_block(const int64_t* args, void* stream);

/* Host helper: the usual map of distances to num_buckets buckets. Of half = num_buckets buckets
 * (num_buckets / 2 if bidirectional: keys behind the query's position take the second half), the
 * first half / 2 hold one distance each, the others share the distances up to max_distance by
 * their logarithm: n >= e = half / 2 falls into min(half - 1, e + floor(log(n / e) /
 * log(max_distance / e) * (half - e))), with the borders computed in whole numbers. Without
 * bidirectional, keys behind the position count as distance 0. Writes the map of distances -left ..
 * right to host memory (nothing if map_host is null) and left, and returns left + right + 1; 0
 * if an argument is out of range (num_buckets odd with bidirectional or above 1024, half < 2,
 * max_distance <= half / 2 or above 32767) or the map does not fit in `capacity` entries. */
int fa_rel_buckets(int32_t* map_host, int capacity, int num_buckets, int max_distance,
                   int bidirectional, int* left);

/* The three stages fa_bwd runs, for callers that schedule or time them
 * separately. They must run in this order on one stream with the same
 * workspace (it carries D from the first stage to the other two); dK/dV and
 * dQ are independent of each other once D exists.
 *   fa_bwd_preprocess: D = rowsum(dO * O) into the workspace.
 *   fa_bwd_dkdv:       dK, dV (one CTA owns each 128-row key tile).
 *   fa_bwd_dq:         dQ (one CTA owns each 128-row query tile). */
fa_status fa_bwd_preprocess(const void* o, const void* dout, int B, int H, int N, int d,
                            void* workspace, size_t workspace_bytes, void* stream);
fa_status fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dout,
                      const float* lse, void* dk, void* dv, int B, int H, int N, int d,
                      float scale, int causal, float dropout_p, uint64_t seed, uint64_t offset,
                      const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                      size_t workspace_bytes, void* stream);
fa_status fa_bwd_dq(const void* q, const void* k, const void* v, const void* dout,
                    const float* lse, void* dq, int B, int H, int N, int d, float scale,
                    int causal, float dropout_p, uint64_t seed, uint64_t offset,
                    const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                    size_t workspace_bytes, void* stream);

/* fa_bwd without a caller-provided workspace: for callers that cannot allocate
 * device memory themselves, such as plugins inside a host framework that owns
 * all device memory and offers them no workspace, or code that must not call
 * cudaMalloc / cudaFree because those can synchronise the device or fail under
 * a fixed memory budget. This entry point allocates nothing: D = rowsum(dO * O)
 * goes to a static device array of 2^22 floats (16 MiB) that every GPU loading
 * the library holds until the process exits. The pages have no counterpart of
 * this call; it exists only for such callers.
 *   - Arguments and outputs are exactly those of fa_bwd minus the workspace.
 *   - B*H*N above 2^22 (4,194,304 query rows) is rejected with FA_ERR_WORKSPACE
 *     before any device work.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that first call before any stream capture.
 *   - All calls on a device share the one array. Its contents left by an earlier
 *     call do not matter (D is fully rewritten before it is read), but two calls
 *     whose kernels overlap on the GPU (different streams, or one device used
 *     from several threads without ordering) race on it: order them. */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, float dropout_p,
                         uint64_t seed, uint64_t offset, const uint8_t* block_mask,
                         const int32_t* seqlens_k, void* stream);

/* Short-query attention over a key/value cache (decode): Nq new query rows
 * per head attend over a cache of Nk keys, forward only. The page
 * "FlashAttention — L3 Cross-Paper Synthesis" (section 3) names this case,
 * bound by reading the K/V cache from HBM, as one the FlashAttention kernels
 * leave unoptimised. Query rows are the last Nq positions of each sequence:
 * row i of batch b sits at position L_b - Nq + i, where L_b = seqlens_k[b]
 * (clamped to [0, Nk]; Nk when seqlens_k is null). Without causal it sees
 * cache keys j < L_b; with causal, j <= L_b - Nq + i as well. A row that
 * sees no key gets O = 0 and lse = -inf. window_left >= 0 adds a sliding window:
 * row i sees only keys j >= L_b - Nq + i - window_left (cache tiles below every
 * row's window are not read); -1 for none.
 *   q, o:          bf16 [B, H, Nq, d], contiguous, 16-byte aligned (device)
 *   k_cache, v_cache: bf16 [B, H_kv, Nk, d], contiguous, 16-byte aligned
 *   lse:           fp32 [B, H, Nq], natural log (device)
 *   seqlens_k:     int32 [B] (device) or NULL
 *   H a multiple of H_kv (query head h reads K/V head h / (H / H_kv)), with
 *   (H / H_kv) * Nq <= 128: the query rows of a K/V group form one tile, so
 *   every K/V tile is read from HBM once per group. d = 64 or 128.
 *   num_ctas: number of CTAs the (K/V head, key tile) pairs are divided
 *   among in equal runs; 0 = automatic: whole K/V heads per CTA when that
 *   keeps at least 4/5 of the SMs busy, else one CTA per SM with heads cut
 *   between them. A K/V head cut between two CTAs is finished by a
 *   second, small kernel that merges the pieces' normalised outputs with the
 *   online softmax's merge rule; it needs the caller's workspace of
 *   fa_decode_workspace_size(...) bytes (16-byte aligned, device; 0 when no
 *   head is cut, and then workspace may be NULL). The result does not depend
 *   on num_ctas beyond fp32 rounding of the merge.
 * Errors: FA_ERR_INVALID_ARG (null or unaligned pointers, sizes < 1, H not a
 * multiple of H_kv, scale not positive and finite, num_ctas < 0,
 * window_left < -1),
 * FA_ERR_UNSUPPORTED (d not 64/128, (H / H_kv) * Nq > 128, not an sm_100-family
 * GPU), FA_ERR_WORKSPACE, FA_ERR_CUDA. Asynchronous on `stream`; nothing is
 * allocated. */
size_t fa_decode_workspace_size(int B, int H, int H_kv, int Nq, int Nk, int d, int num_ctas);
fa_status fa_decode(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                    int B, int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                    int window_left, const int32_t* seqlens_k, int num_ctas, void* workspace,
                    size_t workspace_bytes, void* stream);

/* fa_decode with a bias by relative position: rel_lines as for fa_fwd_cross, row i of batch b at
 * position L_b - Nq + i. What the caches hold at and behind L_b, NaN and infinities too, does not
 * matter. The key tiles within the lengths are divided among num_ctas CTAs (0: one per SM, and
 * whole heads where Nk is at most 512) by the lengths found on the device, so a captured call may be
 * replayed with other lengths. workspace: fa_decode_rel_workspace_size(...) bytes. Errors as
 * fa_decode, plus FA_ERR_INVALID_ARG when rel_lines is null or Nk is above 2^28. */
size_t fa_decode_rel_workspace_size(int B, int H, int H_kv, int Nq, int Nk, int d, int num_ctas);
fa_status fa_decode_rel(const void* q, const void* k_cache, const void* v_cache, void* o,
                        float* lse, int B, int H, int H_kv, int Nq, int Nk, int d, float scale,
                        int causal, int window_left, const int32_t* seqlens_k,
                        const float* rel_lines, int rel_left, int rel_right, int num_ctas,
                        void* workspace, size_t workspace_bytes, void* stream);

/* These calls with their arguments in a block, 8 bytes each in the order above but for the
 * stream: pointers and integers as int64_t, scale and dropout_p as doubles (see
 * fa_paged_attn_block). */
fa_status fa_fwd_cross_block(const int64_t* args, void* stream);
fa_status fa_bwd_cross_block(const int64_t* args, void* stream);
fa_status fa_decode_rel_block(const int64_t* args, void* stream);

/* Attention over a paged key/value cache. The page "FlashAttention — L3
 * Cross-Paper Synthesis" (section 3) names short-query attention over a cache,
 * bound by reading K and V from HBM, as left unoptimised; a server keeps that
 * cache in pages, so that sequences of any length share one pool, and quantises
 * it, which halves the bytes to read. Three calls work on it: fa_paged_write
 * (new rows enter the cache), fa_paged_read (rows come back out of it) and
 * fa_paged_attn (attention of the new tokens, one per sequence or a chunk).
 *
 * The cache, a pool of pages shared by all sequences:
 *   k_pages, v_pages: row r of page p and K/V head h is the d values from element
 *     p * stride_page + h * stride_head + r * stride_row on (the strides count
 *     elements and are the same for both), so [num_pages, H_kv, page_size, d],
 *     [num_pages, page_size, H_kv, d] and views into larger tensors all do. Base
 *     pointers are 16-byte aligned, and the strides are positive multiples of
 *     16 bytes, below 2^40 bytes.
 *   type: FA_CACHE_BF16 (bf16 values) or FA_CACHE_E4M3 (one e4m3 code per value and
 *     one scale byte per row, k_scale and v_scale: uint8 [num_pages, H_kv,
 *     page_size], contiguous, 16-byte aligned; not used for bf16). A quantised value is
 *     code * 2^E with scale byte E + 127, E the smallest exponent in [-117, 7] that
 *     keeps the row's largest magnitude within 448 * 2^E (0 for a row of zeros); codes
 *     are rounded to nearest even and saturate (magnitudes above 57344 = 448 * 2^7). A
 *     row that holds a NaN or an infinity gets scale byte 255 and code 0x7F throughout
 *     and counts as NaN. code * 2^E is exact in bf16, and read-back gives it so. Scale
 *     bytes 135 to 254 are never written; they count as 134.
 *   page_size: a multiple of 16; d: 64 or 128.
 * The batch, B sequences (device pointers):
 *   page_table: int32, row b at b * table_stride (at least max_pages); its entry i <
 *     max_pages names the page of positions i * page_size .. of sequence b. Entries past a
 *     sequence's length are not read. max_pages * page_size < 2^31 - 256.
 *   kv_lens: int32 [B], the length of each sequence, its new tokens included.
 *   cu_seqlens_q: int32 [B + 1], new tokens of sequence b are rows cu[b] .. cu[b+1]
 *     of the T packed token rows (none is possible), the last positions of the
 *     sequence: token i of n sits at position kv_lens[b] - n + i. Rows from cu[B] on
 *     are neither read nor written. NULL: max_q rows each, T = B * max_q.
 * What lies on the device is checked there, before any access: offsets out of order
 * or beyond T, a length outside [0, max_pages * page_size], the number of a page that
 * the call reads or writes outside [0, num_pages) and, for fa_paged_attn, a sequence
 * with more than max_q new tokens. Each is reported as FA_ERR_INVALID_ARG by
 * fa_device_status (a call with T = 0 looks at nothing); such a page reads as zeros and
 * is not written, such a length counts as 0 and such a sequence has no new tokens. Where
 * offsets out of order give a token to several sequences, it may be taken for any of
 * them or for none. Pages that two sequences share are fine to read. Where a
 * write's positions lead to the same row of a page several times, the row ends up as a
 * mixture: each 16 bytes of a bf16 row, each 8 codes and the scale byte of a quantised one,
 * come from any of the tokens. */
typedef enum { FA_CACHE_BF16 = 0, FA_CACHE_E4M3 = 1 } fa_cache_type;

/* Stores k_new and v_new into the pages at their positions. k_new, v_new: bf16 [T,
 * H_kv, d], token t at t * k_stride and t * v_stride (elements, multiples of 8), heads
 * and d contiguous, 16-byte aligned. Tokens at negative positions (a length below the
 * number of new tokens) are not stored. Deterministic, but for rows written several times.
 * Errors: FA_ERR_INVALID_ARG (null or unaligned pointers, sizes, strides),
 * FA_ERR_UNSUPPORTED (d, type, page_size not a multiple of 16), FA_ERR_CUDA.
 * Asynchronous on `stream`; nothing is allocated. T = 0 is allowed and does nothing. */
fa_status fa_paged_write(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                         uint8_t* k_scale, uint8_t* v_scale, int type, int num_pages,
                         int page_size, int H_kv, int d, int64_t stride_page, int64_t stride_head,
                         int64_t stride_row, const int32_t* page_table, int64_t table_stride,
                         int max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens_q, int B,
                         int T, int max_q, int64_t k_stride, int64_t v_stride, void* stream);

/* Copies positions 0 .. N - 1 of every sequence out of the pages, dequantised, into
 * k_out and v_out: bf16 [B, H_kv, N, d], contiguous, 16-byte aligned, the layout that
 * fa_fwd, fa_decode (with seqlens_k = kv_lens) and fa_fp8_quantize take. Positions at or
 * behind a sequence's length are written as zeros. Errors and conventions as above. */
fa_status fa_paged_read(const void* k_pages, const void* v_pages, const uint8_t* k_scale,
                        const uint8_t* v_scale, int type, int num_pages, int page_size, int H_kv,
                        int d, int64_t stride_page, int64_t stride_head, int64_t stride_row,
                        const int32_t* page_table, int64_t table_stride, int max_pages,
                        const int32_t* kv_lens, int B, int N, void* k_out, void* v_out,
                        void* stream);

/* Attention of the new tokens over the cache, which holds their own keys and values
 * already. q: bf16 [T, H, d], token t at t * q_stride (elements, a multiple of 8), 16-byte
 * aligned; query head h reads K/V head h / (H / H_kv), H / H_kv <= 128. The token at
 * position p of a sequence of length L sees keys j < L, with causal j <= p, and with
 * window_left >= 0 only j >= p - window_left. Writes o (bf16 [T, H, d], contiguous,
 * 16-byte aligned; not overlapping q) and lse (fp32 [T, H], natural log); a row that sees no
 * key gets O = 0 and lse = -inf; a NaN in a row of q makes that row's O and lse NaN. Cached rows
 * of positions below a sequence's length are expected to be finite (a NaN or an infinity there may
 * reach every new token of the sequence; a NaN in a key makes O and lse NaN for the rows that see
 * it); what lies behind the length, in the same page too, does not matter.
 *   max_q: the largest number of new tokens of one sequence (a bound on it is enough).
 *   workspace: fa_paged_workspace_size(H, H_kv, d, max_q, max_pages * page_size) bytes,
 *   16-byte aligned (NULL where that is 0); its contents on entry do not matter. Calls that
 *   may overlap need one each.
 * The work of a call is divided among the SMs by the lengths found on the device, so a
 * captured call may be replayed with other lengths. Results do not depend on atomics.
 * Accuracy, against exact attention of the cached values: scores, sums and O's accumulators
 * are fp32; the weights P are rounded to bf16 (by at most 2^-8 of each), from a quantised
 * cache to f16 (2^-11 of each, or 2^-32 of the row's largest weight times value scale where
 * that is more); O is rounded to bf16. From a quantised cache q enters the product in f16,
 * each row times the power of two that brings its largest magnitude into [2^14, 2^15), 2^60 at
 * most: an element below 2^-29 of that magnitude is off by at most 2^-40 of it. With more than
 * 24 query rows per K/V head ((H / H_kv) * max_q) the keys and values are f16 too, relative to
 * the largest scale 2^E among the 128 keys around them: exact where their own is at least 2^-15
 * of it, off by at most 2^-25 of it otherwise; that largest scale counts as at least 2^-40 for
 * keys and 2^-60 for values.
 * Errors: FA_ERR_INVALID_ARG (as above, H not a multiple of H_kv, scale not positive and
 * finite, window_left < -1, max_q < 1, T * H >= 2^31, max_pages * page_size + max_q >=
 * 2^31 - 256), FA_ERR_UNSUPPORTED (H / H_kv > 128, and as above), FA_ERR_WORKSPACE,
 * FA_ERR_CUDA. */
size_t fa_paged_workspace_size(int H, int H_kv, int d, int max_q, int max_keys);
fa_status fa_paged_attn(const void* q, const void* k_pages, const void* v_pages,
                        const uint8_t* k_scale, const uint8_t* v_scale, void* o, float* lse,
                        int type, int num_pages, int page_size, int H, int H_kv, int d,
                        int64_t stride_page, int64_t stride_head, int64_t stride_row,
                        const int32_t* page_table, int64_t table_stride, int max_pages,
                        const int32_t* kv_lens, const int32_t* cu_seqlens_q, int B, int T,
                        int max_q, int64_t q_stride, float scale, int causal, int window_left,
                        void* workspace, size_t workspace_bytes, void* stream);

/* The three calls with their arguments in a block, 8 bytes each in the order above but for the
 * stream: pointers and integers as int64_t, scale as a double. For bindings that spend time on
 * every argument of a call (through Python's ctypes the 30 of fa_paged_attn cost as much as its
 * launch). An integer outside its parameter's range is refused with FA_ERR_INVALID_ARG. */
fa_status fa_paged_write_block(const int64_t* args, void* stream);
fa_status fa_paged_read_block(const int64_t* args, void* stream);
fa_status fa_paged_attn_block(const int64_t* args, void* stream);

/* FP8 forward with incoherent processing (FA-3's FP8 path, which the
 * cross-paper synthesis page on FlashAttention names in its section 2), head
 * dimension 128, forward only.
 * fa_fp8_quantize: Q' = Q M and K' = K M with M = diag(signs) H / sqrt(128),
 *   H the Sylvester Hadamard matrix (signs: fp32 [128] of +-1, device; NULL
 *   means no rotation), each stored as e4m3 codes with one scale per head,
 *   s = amax / 448 (1 for an all-zero head); V as e4m3 with one scale per
 *   (head, column), written transposed.
 *     q, k, v:  bf16 [B, H, N, 128] (device, 16-byte aligned)
 *     q8, k8:   uint8 [B, H, N, 128] (e4m3 codes, rounded to nearest even,
 *               saturating at 448)
 *     vt8:      uint8 [B, H, 128, Np], Np = fa_fp8_vt_stride(N) (N rounded up
 *               to 16; keys N .. Np-1 are written as zero)
 *     s_q, s_k: fp32 [B, H]; s_v: fp32 [B, H, 128]
 *     workspace: fa_fp8_workspace_size(B, H, 128) bytes (device, 16-byte aligned)
 * fa_fwd_fp8: attention of Q^ = dec(q8) s_q, K^ = dec(k8) s_k, V^ = dec(vt8)^T s_v
 *   (rotated Q and K give the same scores), both products on the tensor core
 *   in FP8 with fp32 accumulation; P is rounded to e4m3 for the PV product
 *   (kept between 2^5 and 2^8 at each row's maximum, so weights down to 2^-14
 *   of it are represented). Causal and key padding as fa_fwd. o: bf16
 *   [B, H, N, 128]; lse: fp32 [B, H, N] (natural log).
 * Accuracy contract (the exactness of fa_fwd does not carry over): against
 * exact attention of the dequantised inputs, |O - O^| <= 2^-4 sum_j P_ij |v^_j|
 * + 2^-15 sum_j |v^_j| (the e4m3 rounding of P, with underflow below 2^-9)
 * + 1.5 bf16 half-ulps of O; lse within 1e-3. Against the bf16 inputs the
 * error adds the quantisation of Q, K, V, which the rotation reduces when
 * channels carry outliers.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (d != 128), FA_ERR_WORKSPACE,
 * FA_ERR_CUDA. Asynchronous on `stream`; nothing is allocated. */
size_t fa_fp8_workspace_size(int B, int H, int d);
int fa_fp8_vt_stride(int N);
fa_status fa_fp8_quantize(const void* q, const void* k, const void* v, const float* signs, int B,
                          int H, int N, int d, void* q8, void* k8, void* vt8, float* s_q,
                          float* s_k, float* s_v, void* workspace, size_t workspace_bytes,
                          void* stream);
fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, const float* s_q,
                     const float* s_k, const float* s_v, void* o, float* lse, int B, int H, int N,
                     int d, float scale, int causal, const int32_t* seqlens_k, void* stream);

/* Grouped K/V heads (H_kv dividing H; query head h of batch b uses K/V head
 * b H_kv + h / (H / H_kv), as fa_fwd_gqa): the same two calls with k, v, k8
 * shaped [B, H_kv, N, 128], vt8 [B, H_kv, 128, Np], s_k [B, H_kv] and s_v
 * [B, H_kv, 128]; q, q8, s_q, o and lse keep H. The workspace of
 * fa_fp8_workspace_size(B, H, 128) bytes also covers this case. fa_fp8_quantize
 * and fa_fwd_fp8 are these with H_kv = H. FA_ERR_INVALID_ARG also when H_kv < 1
 * or H is not a multiple of H_kv. */
fa_status fa_fp8_quantize_gqa(const void* q, const void* k, const void* v, const float* signs,
                              int B, int H, int H_kv, int N, int d, void* q8, void* k8, void* vt8,
                              float* s_q, float* s_k, float* s_v, void* workspace,
                              size_t workspace_bytes, void* stream);
fa_status fa_fwd_fp8_gqa(const void* q8, const void* k8, const void* vt8, const float* s_q,
                         const float* s_k, const float* s_v, void* o, float* lse, int B, int H,
                         int H_kv, int N, int d, float scale, int causal,
                         const int32_t* seqlens_k, void* stream);

/* Quantised dropout threshold round(256 p) used by fa_fwd / fa_bwd (-1 if p is
 * outside [0, 1)). The effective dropout rate is fa_dropout_p8(p) / 256. */
int fa_dropout_p8(float dropout_p);

/* Test hook: writes keep[b][h][i][j] (uint8 0/1, device, [B,H,N,N]) for the
 * dropout mask that fa_fwd / fa_bwd use with these arguments, computed by the
 * same device Philox code. */
fa_status fa_debug_dropout_keep(uint8_t* keep, int B, int H, int N, float dropout_p,
                                uint64_t seed, uint64_t offset, void* stream);

/* Test hook: raw Philox4x32-10 blocks from the device generator the kernels
 * use: out[4*t .. 4*t+3] = Philox(counter[4*t .. 4*t+3], key) for t < n.
 * counters and out are device uint32 arrays. */
fa_status fa_debug_philox(const uint32_t* counters, uint32_t* out, int n, uint32_t key0,
                          uint32_t key1, void* stream);

/* Host helper: the butterfly block mask (FlashAttention deep-read report,
 * sections 2.6 and 3.5, "fixed butterfly sparsity pattern"): with nb blocks per
 * side, mask[r*nb + c] = 1 iff r XOR c is 0 or a power of two below nb.
 * Writes nb*nb bytes to host memory. */
fa_status fa_butterfly_mask(uint8_t* mask_host, int nb);

/* Reads the status word of the current device after synchronising `stream`;
 * returns FA_OK or the first device-side error recorded since the last clear:
 * FA_ERR_TIMEOUT (a bounded wait ran out), FA_ERR_INVALID_ARG when a paged call
 * met a length, offset or page number out of range (see there), or FA_ERR_CUDA
 * when a kernel found its launch unusable and returned without work (the d = 128 forward and the
 * d = 128 key-tile backward kernel use nearly all 227 KB of shared memory with
 * no alignment slack and check that their dynamic shared memory starts on a
 * 1024-byte boundary).
 * clear != 0 resets it to FA_OK.
 * The word is one per device, shared by every call on that device: the
 * forward entry points take no workspace to hold a per-call word. An error
 * recorded by a kernel on one stream is therefore seen by whichever caller
 * reads the word next, also from another stream or thread; callers that need
 * to attribute errors to one call must order their calls and read the word
 * between them. */
fa_status fa_device_status(void* stream, int clear);

/* Upper bound on every device-side wait, in nanoseconds (default 4e9). A wait
 * that runs out records FA_ERR_TIMEOUT and the kernel exits early. */
void fa_set_wait_timeout_ns(uint64_t ns);

/* Test hook for failure detection (host-side injection; nothing faults or
 * traps on the GPU). The armed launch waits on a barrier that nothing
 * completes, so its bounded wait runs out and the kernel returns with
 * FA_ERR_TIMEOUT recorded; the hook is consumed by that launch and later
 * launches run normally. mode selects the launch:
 *   1: the next forward-type kernel (fa_fwd and its _gqa / _window forms,
 *      fa_fwd_cross, fa_decode, fa_fwd_fp8, fa_fwd_fp8_gqa, and, with enough
 *      query rows per K/V head, fa_paged_attn (more than 24) and fa_decode_rel
 *      (more than 16 at d = 64, 8 at d = 128): with fewer their kernel waits for
 *      nothing);
 *   2: the next dK/dV kernel (fa_bwd and its _gqa / _window / _noalloc forms,
 *      fa_bwd_cross, fa_bwd_dkdv);
 *   3: the next dQ kernel (the same backward calls, fa_bwd_dq).
 * mode 0 (or any other value) clears it. */
void fa_test_inject_stall(int mode);

/* Static description of an error code. */
const char* fa_status_string(fa_status s);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H_ */
