/*
 * kvq.h -- C ABI of libkvq: attention over a block-quantized KV cache on one
 * GB300 (sm_103a).
 *
 * Operations (all asynchronous on the caller's CUDA stream):
 *   kv_append_quantize   quantize new K/V rows into the cache (f16 / q8_0 / q4_0)
 *   attn_decode          split-K decode attention over every cached key
 *   attn_prefill_chunk   causal attention of one prefill chunk (ubatch)
 *   kv_requantize        degrade one (layer, side) tensor to another codec
 *   kvq_aggregate_bpv    aggregate bits per value of a set of tensors
 *   kvq_ladder_next      the next step of the banded classic degrade ladder
 *   kvq_rope_table       the angles of every position (rotary position embedding)
 *   kvq_rope_apply       rotate query rows, or the transpose (their gradient)
 *   kv_append_rope       rotate new keys and append them, with the values
 *   kv_rope_shift        rotate cached keys again after their positions moved
 *   attn_decode_append_rope   one decode step with the rotation in it
 *   attn_cross           query rows against every key of their sequence
 *   attn_decode_prefix   decode attention of sequences that share a prefix
 *   kv_append_rows       packed or padded rows appended as they are
 *   kv_read_rows         cached rows read back as values
 *
 * Sources.  The codecs and their sizes follow the "Codecs" table of the
 * buun-llama-cpp listing (f16 16.0, q8_0 8.5, q4_0 4.5 bits per value); the
 * per-(layer, side) codec choice follows its "VBR -- Variable Bit-Rate KV
 * Cache" section (the classic F16 -> Q8_0 -> Q4_0 ladder, K and V typed
 * independently, flash attention mandatory); the asymmetric K=f16 / V=q8_0
 * contract, the ubatch-sized prefill chunks and the 256-aligned per-slot
 * pools follow the serverAppConfigs commit log (frank_small_unit.bats
 * commit).  Softmax attention is the plain definition: o = softmax(scale *
 * q K^T) V over the attended keys, K and V dequantized.
 *
 * Ownership.  The caller allocates every buffer (cache, lengths, inputs,
 * outputs, workspace) in device memory and keeps it alive until the work on
 * the stream has finished.  The library never allocates, frees or
 * synchronizes; it keeps no state between calls besides cached device
 * attributes.
 *
 * Errors.  Every entry point validates its arguments on the host before any
 * launch and returns a kvq_status; it never aborts.  Conditions that only the
 * device can see (a length that passes capacity, a wait that timed out) set
 * bits in the optional device word kvq_layer.err (KVQ_DEVERR_*) and the
 * affected rows are skipped.
 *
 * ------------------------------------------------------------------------
 * Block codecs (head_dim 128 = four 32-value blocks per row):
 *   f16  : 128 fp16 values.                              256 bytes / row
 *   q8_0 : per block fp16 d16 + 32 int8 q.               136 bytes / row
 *          amax = max|x| (fp32); d = amax / 127 (fp32, IEEE RN division);
 *          q = round-half-away-from-zero(x / d) (IEEE RN division), or 0 when
 *          d == 0; d16 = fp16_RN(d).  x^ = d16 * q.
 *   q4_0 : per block fp16 d16 + 16 bytes of nibbles.      72 bytes / row
 *          m = the signed x with the largest |x| (lowest index wins ties);
 *          d = m / -8 (fp32 RN); t = x / d (fp32 RN; 0 when d == 0);
 *          u = t + 8.5 (fp32 RN); q = min(15, trunc(u)), its lowest 4 bits;
 *          canonical byte j = q[j] | q[j+16] << 4; d16 = fp16_RN(d).
 *          x^ = d16 * (q - 8).
 *   turbo4: a Walsh-Hadamard-rotated 4-bit row (the turbo4 row of the
 *          "Codecs" table of the buun-llama-cpp listing, 4.125 bits per value;
 *          the FWHT with random sign flips of its TCQ "How it works" list;
 *          the scale and levels are this library's reading).   66 bytes / row
 *          signs s_j = -1 where bit 63 of output j (j = 0..127) of SplitMix64
 *          (Steele, Lea, Flood 2014) seeded with 0x4B5651 is set, else +1;
 *          t = s * x; unnormalised FWHT of t in Sylvester order, stages
 *          h = 1, 2, ..., 64 turning each pair (j, j + h), j & h == 0, into
 *          (a + b, a - b) with fp32 RN additions; y = t / 8; then the q4_0
 *          rule over all 128 values of y (one d16 per row); canonical byte
 *          16 g + j (group g < 4, j < 16) = q[32g + j] | q[32g + j + 16] << 4.
 *          Decoded: y^ = d16 * (q - 8) and x^ = s * H y^ / 16, exact in fp32.
 *          Attention never forms x^: q . x^ = (H (s * q) / 16) . y^, so the
 *          kernels rotate the query once, accumulate V in the rotated space
 *          and rotate the output back once.
 *   Values that are not finite: f16 keeps them (a NaN's payload may change).
 *   In the other codecs a NaN is left out of the maximum (amax, m; 0 where a
 *   block is all NaN) and takes the code of 0 (q = 0, level 8): it reads back
 *   as 0, and a turbo4 row whose sums are all NaN, as one NaN makes them, as
 *   zeros.  An infinity makes d16 infinite and every code that of 0: its block
 *   (turbo4: its row) reads back as NaN.  The bytes are the same on every path.
 *   The canonical row is the row's four blocks end to end (d16 little-endian
 *   before each block's quants); for turbo4 the row's d16 then its 64 bytes.
 *
 * Cache layout (one layer, one side):
 *   [n_seqs][n_kv_heads][capacity / 16 units][unit_bytes]
 *   A unit holds 16 consecutive tokens (unit_bytes = 16 * row bytes: 4096,
 *   2176, 1152, 1056).  Inside a unit, canonical byte cb of token row r (0..15) is
 *   placed as follows (all integer arithmetic; g = r & 7, rh = r >> 3,
 *   tig = (r & 7) >> 1, par = r & 1):
 *   K side
 *     f16  value d, byte k:  b=d>>5, h=(d>>4)&1, w=(d>>2)&3, i=d&3
 *          -> (2b+rh)*512 + (4g+w)*16 + h*8 + i*2 + k
 *     q8_0 quant of dim 32b+e: h=e>>4, w=(e>>2)&3, i=e&3
 *          -> b*512 + (4g+w)*16 + (2rh+h)*4 + i
 *          scale byte k of block b -> 2048 + g*16 + rh*8 + b*2 + k
 *     q4_0 canonical byte jc (0..15) of block b: w=jc>>2, i=jc&3
 *          -> (b>>1)*512 + (4g+w)*16 + ((b&1)*2+rh)*4 + i
 *          scale byte k of block b -> 1024 + g*16 + rh*8 + b*2 + k
 *     turbo4 canonical byte jc of group b: as q4_0's byte jc of block b;
 *          scale byte k -> 1024 + g*4 + rh*2 + k
 *   V side
 *     f16  value d, byte k:  mt=d>>4, gq=(d&15)>>1, s=d&1
 *          -> mt*512 + (4gq+tig)*16 + (rh*4+s*2+par)*2 + k
 *     q8_0 quant of dim d: mt=d>>4, gq=(d&15)>>1, s=d&1
 *          -> (mt>>1)*512 + (4gq+tig)*16 + ((mt&1)*2+rh)*4 + par*2 + s
 *          scale byte k of block b -> 2048 + tig*32 + b*8 + rh*4 + par*2 + k
 *     q4_0 canonical byte jc of block b: mt=2b+(jc>>3), gq=jc&7
 *          -> (mt>>2)*512 + (4gq+tig)*16 + (mt&3)*4 + par*2 + rh
 *          scale byte k of block b -> 1024 + tig*32 + b*8 + rh*4 + par*2 + k
 *     turbo4 canonical byte jc of group b: as q4_0's byte jc of block b;
 *          scale byte k -> 1024 + tig*8 + rh*4 + par*2 + k
 *   The layout stores exactly the canonical bytes (8.5 / 4.5 / 16 / 4.125
 *   bits per value); it only orders them so that each thread of the decode kernel
 *   reads its tensor-core operand fragments with aligned 16-byte loads.
 *
 * Paged layout (kvq_layer.pages_per_seq > 0; block-level KV management as in
 * the vLLM PagedAttention entry of the buun-llama-cpp references, with the
 * pool shared by the sequences and 256-aligned as in the serverAppConfigs
 * commit log):
 *   a page is 256 tokens (16 units) of every kv head of one sequence; each
 *   side's pool is [n_pages][n_kv_heads][16 units][unit_bytes]
 *   (kvq_pool_bytes()); block_table[s][p] is the pool page that holds
 *   tokens 256p .. 256p + 255 of sequence s (-1: not mapped).  Unit j of
 *   (sequence s, kv head h) is pool unit
 *   (block_table[s][j / 16] * n_kv_heads + h) * 16 + j % 16.  capacity is
 *   then pages_per_seq * 256.  Every page a call touches (tokens below the
 *   length, or being appended) must be mapped to a page in [0, n_pages);
 *   otherwise the device sets KVQ_DEVERR_PAGE and skips the row (append,
 *   re-encode) or reads pool page 0 in its place (attention).
 * ------------------------------------------------------------------------
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Codec of one (layer, side) cache tensor. */
typedef enum { KVQ_F16 = 0, KVQ_Q8_0 = 1, KVQ_Q4_0 = 2, KVQ_TURBO4 = 3 } kvq_codec;

/* Host-side status returned by every entry point. */
typedef enum {
    KVQ_OK = 0,
    KVQ_EINVAL = 1,       /* null pointer, non-positive size, bad index, n_q % n_kv != 0 */
    KVQ_EUNSUPPORTED = 2, /* head_dim != 128 or unknown codec */
    KVQ_ECAPACITY = 3,    /* a host-known position passes capacity */
    KVQ_EALIGN = 4,       /* capacity not a multiple of 256, or a misaligned pointer */
    KVQ_EWORKSPACE = 5,   /* workspace null or smaller than the *_workspace query says */
    KVQ_ECUDA = 6         /* a CUDA runtime call or a launch failed */
} kvq_status;

/* Bits OR-ed into *kvq_layer.err by the device (the word is never cleared). */
#define KVQ_DEVERR_CAPACITY 1 /* append: seq_lens[s] + n_new[s] > capacity; rows skipped */
#define KVQ_DEVERR_MAXLEN 2   /* decode, cross: seq_lens[s] > max_len; keys past max_len ignored */
#define KVQ_DEVERR_TIMEOUT 4  /* a bounded wait on an async copy gave up */
#define KVQ_DEVERR_SEQLEN 8   /* prefill: seq_lens[seq] < q_start + n_q_tok; read: a token outside
                               * the sequence */
#define KVQ_DEVERR_PAGE 16    /* paged: a block-table entry outside [0, n_pages) */
#define KVQ_DEVERR_EVICT 32   /* kv_compact: an eviction list not increasing below the length */
#define KVQ_DEVERR_POS 64     /* rotary: a position (or shift) outside the angle table, clamped to it */
#define KVQ_DEVERR_ROWS 128   /* packed or padded rows: a count or row_start entry out of range */

/* One layer's cache.  All pointers are device pointers owned by the caller.
 * k_cache / v_cache: kvq_cache_bytes() bytes each (kvq_pool_bytes() when
 * paged), 16-byte aligned, in the layouts above.  seq_lens: int32[n_seqs],
 * the number of valid tokens of each sequence.  err: optional int32 error
 * word (NULL to skip). */
typedef struct kvq_layer {
    int32_t n_seqs;
    int32_t n_kv_heads;
    int32_t n_q_heads;  /* multiple of n_kv_heads; head h reads kv head h / (n_q/n_kv) */
    int32_t head_dim;   /* must be 128 */
    int32_t capacity;   /* tokens per (seq, kv head) stream; multiple of 256 */
    int32_t codec_k;    /* kvq_codec of the K side */
    int32_t codec_v;    /* kvq_codec of the V side */
    int32_t pages_per_seq; /* 0: contiguous caches; > 0: paged (capacity = 256 * this) */
    void *k_cache;
    void *v_cache;
    int32_t *seq_lens;
    int32_t *err;
    const int32_t *block_table; /* paged: int32 [n_seqs][pages_per_seq], device; else NULL */
    int32_t n_pages;            /* paged: pages in each side's pool; else 0 */
    int32_t reserved;           /* must be 0 */
} kvq_layer;

/* Human-readable name of a status code (static string). */
KVQ_API const char *kvq_status_str(int status);

/* Bytes of one canonical row (256 / 136 / 72 for head_dim 128), or -1. */
KVQ_API int64_t kvq_row_bytes(int codec, int32_t head_dim);

/* Bytes of one side's page pool: n_pages * n_kv_heads * 256 * row bytes, or
 * -1 on bad arguments. */
KVQ_API int64_t kvq_pool_bytes(int codec, int32_t n_pages, int32_t n_kv_heads, int32_t head_dim);

/* Bytes of one side's cache for the given geometry, or -1 on bad arguments. */
KVQ_API int64_t kvq_cache_bytes(int codec, int32_t n_seqs, int32_t n_kv_heads, int32_t capacity,
                        int32_t head_dim);

/* Quantize-on-append (block codecs above).
 * k_new, v_new: fp16 [n_seqs][max_new][n_kv_heads][128], 8-byte aligned.
 * n_new: device int32[n_seqs], rows to append per sequence (0..max_new).
 * Row i < n_new[s] of sequence s is encoded with the side's codec and written
 * at token position seq_lens[s] + i.  When update_lens != 0, seq_lens[s] +=
 * n_new[s] afterwards (stream-ordered).  Positions past capacity set
 * KVQ_DEVERR_CAPACITY and are skipped. */
KVQ_API int kv_append_quantize(const kvq_layer *layer, const void *k_new, const void *v_new,
                       const int32_t *n_new, int32_t max_new, int32_t update_lens,
                       void *stream);

/* Workspace bytes that attn_decode needs for this layer and max_len. */
KVQ_API int attn_decode_workspace(const kvq_layer *layer, int32_t max_len, size_t *bytes);

/* Decode attention: every query head of every sequence attends all
 * seq_lens[s] cached keys (split-K over the token axis; two launches: the
 * split kernel writes partials, the merge kernel combines them by
 * log-sum-exp).  The first 64 KiB of the workspace are a counter region that
 * must be zero before the first call (zero-fill the workspace once after
 * allocating it); every call that completes without KVQ_DEVERR_TIMEOUT
 * leaves it zero again, so one workspace serves any number of calls and
 * layers without clearing.  Calls that may run concurrently need separate
 * workspaces.  Limits: 1024 sequences and 16383 streams (sequence x kv head
 * x group of 8 query heads) per call, else KVQ_EINVAL.
 * q: fp16 [n_seqs][n_q_heads][128] (8-byte aligned); out: fp16
 * [n_seqs][n_q_heads][128]; lse: optional fp32 [n_seqs][n_q_heads] natural-log
 * sum-exp of the scaled scores (NULL to skip).  max_len bounds every
 * seq_lens[s] (1..capacity).  workspace: device, 16-byte aligned, at least
 * attn_decode_workspace() bytes.  A sequence of length 0 gives out = 0 and
 * lse = -inf.
 * Accuracy: softmax weights p, and their products with a quantized value's
 * scale d, are fp16 operands.  Before its own rounding an output is within
 * (2^-11 sum p (|v| + |d c|) + 2^-25 sum (|v| + |c|)) / sum p of softmax
 * attention over the decoded rows, c being the code (q8_0's, q4_0's level - 8,
 * 0 for f16) and p relative to the largest; in turbo4's rotated space within
 * (2^-11 sum p |v| + 2^-25 sum |c|) / sum p.  The other sums are fp32. */
KVQ_API int attn_decode(const kvq_layer *layer, const void *q, float scale, void *out, float *lse,
                int32_t max_len, void *workspace, size_t ws_bytes, void *stream);

/* One decode step of a layer with no launch for the append: quantize-on-append
 * of one new token per sequence (the kv_append_quantize row encoding, at position
 * seq_lens[s]), then attn_decode over seq_lens[s] + 1 keys, then
 * seq_lens[s] += 1.  The result (cache bytes, lengths, out, lse) is that of
 * kv_append_quantize(n_new = 1 for every sequence, update_lens = 1)
 * followed by attn_decode on the same stream (a new token's keys enter the
 * typed cache before it is attended, as in the serverAppConfigs commit log,
 * frank_small_unit.bats commit), fused so that the append costs no launch
 * of its own.
 * k_new, v_new: fp16 [n_seqs][n_kv_heads][128], 8-byte aligned.  A sequence
 * whose length is already capacity (or negative) gets no new token (sets
 * KVQ_DEVERR_CAPACITY) and attends its existing keys.  max_len must bound
 * every new length.  The workspace is attn_decode_workspace(layer, max_len)
 * bytes, with the same zero-between-calls contract as attn_decode; its
 * 64 KiB counter region also counts the CTAs that have read the lengths.
 * Other arguments and limits are those of attn_decode. */
KVQ_API int attn_decode_append(const kvq_layer *layer, const void *k_new, const void *v_new,
                               const void *q, float scale, void *out, float *lse,
                               int32_t max_len, void *workspace, size_t ws_bytes, void *stream);

/* attn_decode without a workspace argument, for callers that cannot allocate
 * device memory where they run attention (an interface that hands them only
 * the input and output buffers, a loop where a device allocation is not
 * allowed, a fully committed memory budget).  There is no counterpart in the
 * source material; it is a convenience of this library.  The scratch that
 * attn_decode keeps in the caller's workspace lives instead in one 8 MiB
 * device array inside the library (reserved on every GPU that loads it, until
 * the process exits); nothing is allocated.  The first call on a device looks
 * the array up (cudaGetSymbolAddress) and must come before any stream capture.
 * The array is shared by all calls and keeps the previous call's contents:
 * its counter region is cleared on `stream` before each launch, and calls
 * that can overlap on the GPU race on it, so issue them in order on one
 * stream.  A layer whose attn_decode_workspace() exceeds 8 MiB is refused
 * with KVQ_EWORKSPACE.  Arguments and results are those of attn_decode. */
KVQ_API int attn_decode_noalloc(const kvq_layer *layer, const void *q, float scale, void *out,
                                float *lse, int32_t max_len, void *stream);

/* Workspace bytes that attn_prefill_chunk needs for a chunk ending at
 * q_start + n_q_tok. */
KVQ_API int attn_prefill_workspace(const kvq_layer *layer, int32_t q_start, int32_t n_q_tok,
                           size_t *bytes);

/* Causal attention of one prefill chunk of sequence `seq`: query i (absolute
 * position q_start + i) of head h attends keys 0 .. q_start + i of kv head
 * h / (n_q/n_kv).  The chunk's own keys must already be appended.
 * q: fp16 [n_q_tok][n_q_heads][128] (16-byte aligned); out: fp16
 * [n_q_tok][n_q_heads][128] (16-byte aligned); lse: optional fp32
 * [n_q_tok][n_q_heads]; scale > 0.  The keys and values are dequantized once
 * into the workspace as fp16 (each value rounded once to fp16, the tensor-core
 * operand type).  workspace: device, 16-byte aligned, at least
 * attn_prefill_workspace() bytes. */
KVQ_API int attn_prefill_chunk(const kvq_layer *layer, int32_t seq, int32_t q_start, int32_t n_q_tok,
                       const void *q, float scale, void *out, float *lse, void *workspace,
                       size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Degrade ladder ("VBR -- Variable Bit-Rate KV Cache" section of the
 * buun-llama-cpp listing: the cache degrades one (layer, side) tensor at a
 * time down the classic f16 -> q8_0 -> q4_0 ladder; the classic order is
 * strictly banded, every movable tensor reaching q8_0 before any reaches
 * q4_0; degrades stop at the last step whose aggregate bits per value stays
 * at or above the floor).
 * ------------------------------------------------------------------------ */

/* Re-encode side `side` (0 = K, 1 = V) of the layer with codec dst_codec into
 * dst_cache: for every sequence s and kv head, tokens [0, seq_lens[s]) are
 * decoded (exactly, as fp32: d16 * q, d16 * (n - 8), or the fp16 value) and
 * encoded again with the append encoder of dst_codec (an f16 target rounds to
 * fp16); tokens past the length are not written.  From f16 the result equals
 * appending the original rows with dst_codec.
 * dst_cache: device, kvq_cache_bytes(dst_codec, ...) bytes, 16-byte aligned,
 * not overlapping the source (the degrade is done out of place; the caller
 * then points the layer's side at dst_cache and sets its codec).  Any pair of
 * codecs is accepted. */
KVQ_API int kv_requantize(const kvq_layer *layer, int32_t side, int32_t dst_codec, void *dst_cache,
                          void *stream);

/* Aggregate bits per value of n tensors holding equally many values: the mean
 * of the codecs' bits per value (16, 8.5, 4.5).  -1 on bad arguments.  Host
 * only. */
KVQ_API double kvq_aggregate_bpv(const int32_t *codecs, int32_t n);

/* The next degrade step of the banded classic ladder for n tensors with the
 * given codecs.  order: the n_order movable tensor indices in price order
 * (tensors missing from it are pinned and never move); NULL with n_order = 0
 * means every tensor in index order.  The first tensor in order still above
 * q8_0 goes to q8_0; once none is, the first one still above q4_0 goes to
 * q4_0; the step is taken only if the aggregate bits per value afterwards is
 * >= floor_bpv.  On KVQ_OK, *tensor and *codec hold the step, or *tensor = -1
 * when no step remains.  Host only. */
KVQ_API int kvq_ladder_next(const int32_t *codecs, int32_t n, const int32_t *order,
                            int32_t n_order, double floor_bpv, int32_t *tensor, int32_t *codec);

/* ------------------------------------------------------------------------
 * Probe-scored eviction (the "Sparse KV eviction" item of the "How It Works"
 * section of the GitHot listing of VITRIOL: an attention probe, a q.K softmax
 * with exponential decay, scores the cells; the lowest-scored middle cells
 * are evicted first; the sink cells at the start and the recent cells at the
 * end are protected).
 * Scores are fp32 [n_seqs][capacity] by logical position, for contiguous and
 * paged layers alike.
 * ------------------------------------------------------------------------ */

/* Fold one probe into the scores: for every sequence s and token
 * t < seq_lens[s],
 *   mass_t = sum over the query heads h of exp(scale * q_h . k^_t - lse[s][h])
 * (the softmax weight head h puts on t; k^ the decoded key of h's kv head) and
 *   scores[s][t] = decay * scores[s][t] + mass_t.
 * Entries at t >= seq_lens[s] are not touched.  q: fp16 [n_seqs][n_q][128]
 * (8-byte aligned), the query of the decode step; lse: fp32 [n_seqs][n_q],
 * the natural-log log-sum-exp that attn_decode wrote for the same q, scale
 * and cache (the probe reads K once more and never recomputes it); scores:
 * device, 4-byte aligned.  Results are deterministic (a fixed summation
 * order). */
KVQ_API int kv_probe_scores(const kvq_layer *layer, const void *q, float scale, const float *lse,
                            float decay, float *scores, void *stream);

/* For every sequence s, the min(n_evict, len - n_recent - n_sink) positions t
 * in [n_sink, len - n_recent) with the smallest (scores[s][t], t) pairs
 * (equal scores: the lower position first; -0 equals +0; NaN scores are
 * outside the contract and order after every number), written in increasing
 * order to evict[s][0 ..); n_evicted[s] = their count (0 when the middle
 * range is empty).  evict: device int32 [n_seqs][n_evict]; n_evicted: device
 * int32 [n_seqs]; n_sink, n_recent >= 0, n_evict >= 0. */
KVQ_API int kv_evict_select(const kvq_layer *layer, const float *scores, int32_t n_sink,
                            int32_t n_recent, int32_t n_evict, int32_t *evict,
                            int32_t *n_evicted, void *stream);

/* Remove the listed tokens from both sides of every sequence: the kept tokens
 * t < seq_lens[s] move down in order into k_dst / v_dst, bytes unchanged
 * (same codecs and layout as the layer's caches, same block table for a paged
 * layer).  evict: device int32 [n_seqs][max_evict], the n_evicted[s] first
 * entries of row s increasing and below seq_lens[s] (as kv_evict_select
 * writes them; otherwise the device sets KVQ_DEVERR_EVICT and the result is
 * unspecified but in bounds).  Inside the last unit written, rows past the new
 * length are zero; units past it are not written.  Optional (null to skip):
 * scores_dst[s][w] = scores[s][source of w] for w below the new length, and
 * lens_dst[s] = seq_lens[s] - n_evicted[s].  Every destination is out of
 * place (it must not overlap the layer's caches or the scores); the caller
 * then points the layer at k_dst, v_dst and lens_dst.  k_dst, v_dst: 16-byte
 * aligned, kvq_cache_bytes (kvq_pool_bytes for a paged layer) of the codecs. */
KVQ_API int kv_compact(const kvq_layer *layer, const int32_t *evict, const int32_t *n_evicted,
                       int32_t max_evict, void *k_dst, void *v_dst, const float *scores,
                       float *scores_dst, int32_t *lens_dst, void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions (rotary position embedding, Su et al. 2021).  The pages
 * name no position encoding; the definitions below are this library's.
 *
 * A row x of 128 values at position p has its first rot_dim values turned in
 * rot_dim / 2 planes.  Plane i holds the elements (a, b) = (2i, 2i + 1) in
 * the interleaved layout and (i, i + rot_dim / 2) in the half layout; the
 * values from rot_dim on are unchanged.  With (cos, sin) = table[p][i],
 * c = RN(cos * magnitude) and s = RN(sin * magnitude), all in fp32:
 *     y_a = RN(RN(x_a c) - RN(x_b s))      y_b = RN(RN(x_a s) + RN(x_b c))
 * and one more rounding to the output's type; nothing is contracted, so the
 * rotated keys' codec bytes are reproducible bit for bit.  A position outside
 * [0, n_pos) sets KVQ_DEVERR_POS and takes the nearest row of the table.
 * ------------------------------------------------------------------------ */

typedef enum { KVQ_ROPE_INTERLEAVED = 0, KVQ_ROPE_HALF = 1 } kvq_rope_layout;

/* How the frequencies f_i = base^(-2i / rot_dim) are scaled for a context
 * `factor` times the original one of orig_len positions:
 *   PLAIN   f_i
 *   LINEAR  f_i / factor (position interpolation)
 *   NTK     base * factor^(rot_dim / (rot_dim - 2)) in the place of base
 *           (one plane: unchanged)
 *   PARTS   by the turns r = orig_len f_i / 2 pi that a plane makes over the
 *           original context: keep = clamp((r - low) / (high - low), 0, 1),
 *           f_i keep + f_i / factor (1 - keep)   (the interpolation by parts
 *           of Peng et al. 2023, who take low = 1 and high = 32)
 *   YARN    the same blend with keep = 1 - clamp((i - l) / max(h - l, 0.001),
 *           0, 1) (Peng et al. 2023, as published checkpoints are run), where
 *           l = max(floor(at(high)), 0) and h = min(ceil(at(low)), rot_dim - 1)
 *           are the plane indexes that make `high` and `low` turns: at(r) =
 *           rot_dim ln(orig_len / (2 pi r)) / (2 ln base).  h may lie past the
 *           last plane, rot_dim / 2 - 1, where even that one makes `low` turns */
typedef enum {
    KVQ_ROPE_PLAIN = 0,
    KVQ_ROPE_LINEAR = 1,
    KVQ_ROPE_NTK = 2,
    KVQ_ROPE_PARTS = 3,
    KVQ_ROPE_YARN = 4
} kvq_rope_scaling;

/* Type of rows handed to the rotary calls. */
typedef enum { KVQ_T_F16 = 0, KVQ_T_BF16 = 1, KVQ_T_F32 = 2 } kvq_type;

/* Angles and how to use them. */
typedef struct kvq_rope {
    const float *table; /* device, fp32 [n_pos][rot_dim / 2][2] (cos, sin), 16-byte aligned */
    int32_t n_pos;      /* > 0 */
    int32_t rot_dim;    /* even, 2..128 */
    int32_t layout;     /* kvq_rope_layout */
    float magnitude;    /* finite; multiplies cos and sin (1 for none) */
} kvq_rope;

/* Rows of 128 contiguous values: [rows][heads][128] with strides in elements.
 * data 16-byte aligned, both strides multiples of 16 bytes. */
typedef struct kvq_rows {
    void *data;
    int64_t row_stride;
    int64_t head_stride;
    int32_t type; /* kvq_type */
    int32_t reserved; /* must be 0 */
} kvq_rows;

/* The rot_dim / 2 frequencies in radians per position into freqs (host), by
 * the formulas above in double.  base > 1; factor >= 1 and finite; PARTS and
 * YARN: orig_len > 0 and 0 < low < high.  Host only. */
KVQ_API int kvq_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                           double orig_len, double low, double high, double *freqs);

/* table[p][i] = (cos, sin)(p * freqs[i]) for p < n_pos, i < rot_dim / 2, in
 * fp32, each within 2^-23 of the exact value.  freqs: host, each in [0, 2 pi).
 * The product is reduced as a 64-bit fixed-point number of turns, so far
 * positions lose nothing.
 * table: device, fp32 [n_pos][rot_dim / 2][2], 16-byte aligned. */
KVQ_API int kvq_rope_table(const double *freqs, int32_t rot_dim, int32_t n_pos, float *table,
                           void *stream);

/* Rotate n_rows x n_heads rows of x into y.  positions: device int32 [n_rows],
 * or NULL for position pos0 + row.  transpose != 0 applies the transposed
 * rotation (s taken as -s): the gradient with respect to x of a rotation,
 * given the gradient with respect to y.  y has x's type or fp16; y may be x
 * itself (same data, strides and type); otherwise the ranges from the first to
 * the last byte of x and of y must not meet.  x may repeat rows or heads (a
 * stride of 0), y may not.  err: optional device word for KVQ_DEVERR_POS.
 * n_rows = 0 launches nothing. */
KVQ_API int kvq_rope_apply(const kvq_rope *rope, const kvq_rows *x, const kvq_rows *y,
                           int64_t n_rows, int32_t n_heads, const int32_t *positions,
                           int32_t pos0, int32_t transpose, int32_t *err, void *stream);

/* Quantize-on-append with the rotation applied on the way: k rows are rotated
 * in fp32 and encoded from there with codec_k (an f16 cache rounds to fp16),
 * v rows are encoded as they are (bf16 and fp32 rows: from fp32).
 * Rows: k, v [n_rows][n_kv_heads][128], and optionally q
 * [n_rows][n_q_heads][128] (NULL: none), whose rotated rows go to q_out, fp16
 * [n_rows][n_q_heads][128] contiguous and 16-byte aligned: the query of
 * attn_decode or attn_prefill_chunk.  q, k and v have one type.
 * Which rows belong to which sequence, one of:
 *   row_start (device int32 [n_seqs + 1], non-decreasing, packed rows):
 *     sequence s has rows row_start[s] .. row_start[s + 1] - 1; rows from
 *     row_start[n_seqs] on are padding: nothing is written for them;
 *   n_new (device int32 [n_seqs], padded rows): sequence s has rows
 *     s * (n_rows / n_seqs) .. + n_new[s] - 1 (n_rows a multiple of n_seqs,
 *     n_new[s] up to n_rows / n_seqs).
 * Row i of sequence s goes to token seq_lens[s] + i and is rotated by
 * positions[row] (device int32 [n_rows]), or with NULL by that token index.
 * When update_lens != 0, the lengths advance afterwards (stream-ordered).
 * n_rows = 0 launches nothing.
 * Device conditions: KVQ_DEVERR_CAPACITY, KVQ_DEVERR_PAGE (the row's k and v
 * are skipped), KVQ_DEVERR_POS, KVQ_DEVERR_ROWS (a row_start or n_new entry out
 * of its range: that sequence's rows are unspecified, in bounds, and its
 * length stays).  q_out may be q itself when q is fp16 and contiguous;
 * otherwise it must not meet the ranges of q, k and v. */
KVQ_API int kv_append_rope(const kvq_layer *layer, const kvq_rope *rope, const kvq_rows *q,
                           const kvq_rows *k, const kvq_rows *v, int64_t n_rows,
                           const int32_t *n_new, const int32_t *row_start,
                           const int32_t *positions, void *q_out, int32_t update_lens,
                           void *stream);

/* How far kv_compact moves each kept token: for w < seq_lens[s] - n_evicted[s],
 * delta[s][w] = w - (the position that token w had).  Call it with the lengths
 * from before the eviction; arguments as kv_compact's (evict increasing and
 * below the length, otherwise the values are unspecified).  delta: device
 * int32 [n_seqs][capacity]; entries behind the new length are not written.
 * At most 65535 sequences, as kv_rope_shift. */
KVQ_API int kv_evict_delta(const kvq_layer *layer, const int32_t *evict,
                           const int32_t *n_evicted, int32_t max_evict, int32_t *delta,
                           void *stream);

/* Move cached keys to other positions: for every token t < seq_lens[s] with
 * delta[s][t] != 0, its K rows are decoded exactly, rotated by delta[s][t]
 * (sin negated for a negative one; magnitude is not applied: the rows carry
 * it already) and encoded again in place with codec_k (f16: rounded to
 * fp16).  Tokens with delta 0 keep their bytes.  delta: device int32
 * [n_seqs][capacity], |delta| < n_pos (otherwise KVQ_DEVERR_POS, clamped).
 * A page shared by two sequences is outside the contract, as for an append. */
KVQ_API int kv_rope_shift(const kvq_layer *layer, const kvq_rope *rope, const int32_t *delta,
                          void *stream);

/* attn_decode_append with the rotation in it: the new key is rotated before
 * it is encoded and q is rotated before it attends, both by positions[s]
 * (device int32 [n_seqs]), or with NULL by the length before the step.  The
 * result is that of kv_append_rope (one row per sequence, update_lens = 1, q_out)
 * followed by attn_decode of q_out, bit for bit.  q, k_new, v_new: fp16 as
 * attn_decode_append takes them; positions NULL needs n_pos >= max_len
 * (KVQ_ECAPACITY).  A sequence already at capacity gets no new token
 * and attends its keys.  From 8 sequences on the append is a launch of its
 * own and `out` holds the rotated queries until the results replace them.
 * Everything else as attn_decode_append. */
KVQ_API int attn_decode_append_rope(const kvq_layer *layer, const kvq_rope *rope,
                                    const int32_t *positions, const void *k_new,
                                    const void *v_new, const void *q, float scale, void *out,
                                    float *lse, int32_t max_len, void *workspace,
                                    size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Rows of several sequences against their caches, without a rotation and
 * without a causal mask.  The pages name none of these; the definitions below
 * are this library's.  Which rows belong to which sequence is said as for
 * kv_append_rope, by row_start (packed) or n_new (padded); an entry out of
 * range sets KVQ_DEVERR_ROWS and that sequence's rows are unspecified (where
 * row_start decreases, kv_append_rows and kv_read_rows may leave out rows of other
 * sequences too).  A call has at most 2^31 - 1 rows times query heads.
 * ------------------------------------------------------------------------ */

/* kv_append_rope without the rotation: k and v rows (one type; strided) are
 * encoded as they are, for keys that carry no position or carry it already, an
 * encoder's states among them.  The bytes are those of kv_append_quantize (bf16
 * and fp32 rows: encoded from fp32). */
KVQ_API int kv_append_rows(const kvq_layer *layer, const kvq_rows *k, const kvq_rows *v,
                           int64_t n_rows, const int32_t *n_new, const int32_t *row_start,
                           int32_t update_lens, void *stream);

/* Cached rows as values: row i of sequence s is token first[s] + i (first:
 * device int32 [n_seqs], or NULL for 0), decoded exactly in fp32 and rounded
 * once to the output's type.  k, v: rows [n_rows][n_kv_heads][128] to be
 * written, either of them NULL for a side that is not read; their types and
 * strides may differ, their places may not meet (their ranges only as views of one
 * tensor with the same strides).  n_read, row_start: as n_new
 * and row_start of kv_append_rope.  A token outside [0, seq_lens[s]) sets
 * KVQ_DEVERR_SEQLEN, an unmapped page KVQ_DEVERR_PAGE; such rows, and rows that
 * belong to no sequence, are left as they were. */
KVQ_API int kv_read_rows(const kvq_layer *layer, const kvq_rows *k, const kvq_rows *v,
                         int64_t n_rows, const int32_t *n_read, const int32_t *row_start,
                         const int32_t *first, void *stream);

/* Workspace bytes that attn_cross needs for n_rows rows and max_len: no more for
 * fewer of either, and at most 266 KB an SM (40 MB on 152). */
KVQ_API int attn_cross_workspace(const kvq_layer *layer, int64_t n_rows, int32_t max_len,
                                 size_t *bytes);

/* Attention of query rows to every key of their sequence: row r of sequence s,
 * head h: softmax(scale q k^T) v over the tokens t < seq_lens[s] of kv head
 * h / (n_q/n_kv); cross attention to an encoder's states, whose lengths have
 * nothing to do with the rows'.
 * q: rows [n_rows][n_q_heads][128], fp16 or bf16 (rounded to fp16 first, within
 * its range); out: rows of the same type, not meeting q (views of one tensor may
 * lie beside each other with the same strides); lse:
 * optional fp32 [n_rows][n_q_heads], natural log.  Rows belong to sequences by
 * n_new or row_start; both NULL: row s to sequence s (n_rows = n_seqs).  Rows
 * that belong to no sequence are left as they were; a sequence of length 0 gives
 * out = 0 and lse = -inf, a NaN in a row's query or in one of its keys NaN in
 * both.  scale > 0.  max_len bounds every seq_lens[s].
 * workspace: device, 16-byte aligned, of any contents; calls that may run
 * concurrently need separate ones.  At most 1024 sequences.
 * Keys and values go through the products as fp16 (quantized ones as a pair of
 * fp16 numbers that add up to them exactly), softmax weights as fp16, sums as
 * fp32.  Rows for which that does not do - a cached value (turbo4: a rotated
 * one) or a query past 65504, scores past 2^22 - are computed in fp32 instead,
 * key by key: many times slower.  turbo4 keys cost a third more than the other
 * codecs' where rows are many; for one fp16 row per sequence attn_decode is faster
 * (16 sequences of 1500 keys 14.5 and 17.8 us, 64 of 4096 110 and 197). */
KVQ_API int attn_cross(const kvq_layer *layer, const kvq_rows *q, int64_t n_rows,
                       const int32_t *n_new, const int32_t *row_start, float scale,
                       const kvq_rows *out, float *lse, int32_t max_len, void *workspace,
                       size_t ws_bytes, void *stream);

/* Workspace bytes that attn_decode_prefix needs. */
KVQ_API int attn_decode_prefix_workspace(const kvq_layer *layer, const kvq_layer *prefix,
                                         int32_t max_len, int32_t max_prefix, size_t *bytes);

/* attn_decode of sequences that share long prefixes, each prefix held and read
 * once: sequence s of `layer` attends every key of its group's sequence of
 * `prefix` and every key of its own, one softmax over both.  prefix: a layer of
 * the same heads whose sequence g is the prefix of the sequences group_start[g]
 * .. group_start[g + 1] - 1 of `layer` (device int32 [prefix n_seqs + 1],
 * non-decreasing; NULL: the one prefix of all); sequences outside the groups, and
 * those of a group whose entries are out of range, attend their own keys alone.  Its codecs, capacity and pages are its own: two
 * paged layers may be views of one pool, the prefix's block table over the shared
 * pages, the layer's over the rest (their lengths then count those alone).
 * q, out, lse, max_len: as attn_decode (q 16-byte aligned and not meeting out;
 * scale > 0) but for a NaN in a query or a key, which makes lse NaN with the row;
 * the prefix's keys and values are taken as attn_cross takes them;
 * max_prefix bounds the prefix's lengths.  max_len also chooses how the own keys
 * are read (whole sequences up to 1024 keys and 20 more for each sequence and kv
 * head, at most 8192; split over the GPU beyond): a bound far above the lengths
 * makes short ones slower.  workspace: as attn_cross.
 * Conditions of the prefix (and of group_start) are set in its own err word. */
KVQ_API int attn_decode_prefix(const kvq_layer *layer, const kvq_layer *prefix,
                               const int32_t *group_start, const void *q, float scale,
                               void *out, float *lse, int32_t max_len, int32_t max_prefix,
                               void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
