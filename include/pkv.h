/*
 * pkv.h -- C ABI of libpkv, paged-KV attention for a GB300 (sm_103a).
 *
 * The library implements the data-parallel hot path of LLM decoding in an
 * audio-LLM ASR server: appending new key/value rows to a paged KV cache,
 * batched decode attention over that cache, and chunked-prefill attention.
 *
 * Sources of the operations (titles of the pages they come from):
 *  - "FunASR vLLM Inference Engine Guide", section 2 "vLLM Engine Architecture"
 *    and the table "Why vLLM?": the LLM engine runs PagedAttention over a KV
 *    cache that is allocated on demand, with continuous batching and CUDA
 *    graphs.
 *  - "Fun-ASR-Nano Native Runtime Design", section "Decoder And Prompt": the
 *    decoder is a Qwen3-0.6B with 28 layers and 16 query / 8 KV heads.
 *  - "Optimizing ASR for 90-minute multi-speaker audio" (MOSS-TD in
 *    SGLang-Omni): section "Time spent: profiling" (decode takes over 94% of
 *    the time on long audio), section "Chunked prefill for long audio"
 *    (4096-token prefill chunks interleaved with decode steps) and section
 *    "Autoregressive decoding" (decode replayed as CUDA graphs over batches
 *    padded to buckets 1, 2, 4, 8, ...).
 *
 * Data layout (a reading; no page gives one):
 *  - k_pages, v_pages: bf16 [num_pages][num_kv_heads][page_size][head_dim],
 *    K and V in separate pools. One (page, KV head) tile is contiguous.
 *  - Logical position j of request b is page block_table[b][j / page_size],
 *    slot j % page_size. A slot index s names page s / page_size, slot
 *    s % page_size.
 *  - Query head h reads KV head h / (num_q_heads / num_kv_heads).
 *  - q and out: bf16, row-major [rows][num_q_heads][head_dim].
 *  - block_table: int32 [rows][max_pages_per_seq]; entries past a request's
 *    last page are never read.
 *
 * Supported geometry:
 *  - Every call: num_q_heads = 16, num_kv_heads = 8, head_dim = 128,
 *    page_size = 16 (the Qwen3 decoder; the tuned kernels).
 *  - pkv_append, pkv_decode_attn, pkv_decode_append_attn,
 *    pkv_decode_append_rope_attn, pkv_append_rope, pkv_prefill_chunk_attn,
 *    pkv_tree_attn, pkv_keep_nodes, pkv_copy_pages and the calls of the 8-bit
 *    cache also take page_size = 16, head_dim 64 or 128,
 *    any num_kv_heads and num_q_heads = G * num_kv_heads with G from 1 to 8
 *    (other decoder backbones; decode runs the same persistent split-KV
 *    kernel with the head counts read at run time, early prefetch included;
 *    prefill runs its tensor-core kernel on pairs of query heads).
 *  - Anything else returns PKV_ERR_UNSUPPORTED.
 *
 * Conventions for every entry point:
 *  - Every pointer argument except `desc` (and the arrays of pools of
 *    pkv_keep_nodes and pkv_copy_pages) is DEVICE memory owned by the
 *    caller; `desc` is a host pointer read during the call only. The library
 *    never allocates, frees or synchronises, and keeps no state between calls
 *    apart from a per-device cache of the SM count. The one exception is
 *    pkv_decode_attn_noalloc, which owns a fixed device array per GPU and has
 *    no status word the caller can read (see its own block).
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and is
 *    ordered with the caller's other work on that stream. No call reads
 *    device memory from the host, so the calls can be captured in a CUDA graph.
 *  - Return value: PKV_OK, or a negative PKV_ERR_* code when the arguments are
 *    rejected on the host (nothing is launched) or the launch fails.
 *  - Errors found on the device (a page id outside the pool, a length beyond
 *    the block table, a wait that ran out of time) are written to the status
 *    word at the start of the workspace; the first error wins. The kernel
 *    skips the offending access and stays within the caller's buffers.
 *    Read the word with pkv_read_status().
 *  - A workspace must be zero-filled once before its first use
 *    (pkv_workspace_init); the kernels leave it ready for the next call. Calls
 *    that may run concurrently (different streams) need separate workspaces.
 *  - After any call whose status word is not PKV_OK, run pkv_workspace_init on
 *    the workspace again before its next use. A call that stopped early (a
 *    bounded wait that ran out, a skipped access) may leave split counters
 *    above zero or tagged partial records behind, and the next call would
 *    take them for its own.
 *  - Split merge of decode batches: the CTA that merges a (request, KV head)
 *    waits, with a bound, for the partial records of CTAs with lower block
 *    indices. This relies on the hardware starting a grid's CTAs in
 *    block-index order, which NVIDIA GPUs do but CUDA does not promise. Were
 *    it not so, the wait would run out after about one second and report
 *    PKV_ERR_DEVICE_TIMEOUT; it never hangs.
 *  - A workspace serves one kind of attention call: decode calls
 *    (pkv_decode_attn, pkv_decode_append_attn, and the 8-bit cache's) or prefill calls
 *    (pkv_prefill_chunk_attn), not both: each kind relies on its own split
 *    scratch (counters, and for decode tagged records) having been left
 *    cleared by the previous call of that kind. Decode calls of any geometry,
 *    batch and cache type may share a workspace that is large enough for each
 *    of them. The tree attention calls are a third kind. The appends,
 *    pkv_expand_fp8, pkv_keep_nodes and pkv_copy_pages use only the status word
 *    and may share any kind's.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
struct CUstream_st;
typedef struct CUstream_st* pkv_stream_t;

typedef struct pkv_cache_desc {
  int32_t num_q_heads;  /* query heads (16; see "Supported geometry") */
  int32_t num_kv_heads; /* KV heads (8) */
  int32_t head_dim;     /* 128 (or 64) */
  int32_t page_size;    /* tokens per page (16) */
  int32_t num_pages;    /* pages in each of k_pages / v_pages */
} pkv_cache_desc;

enum {
  PKV_OK = 0,
  PKV_ERR_NULL_ARG = -1,            /* a required pointer is NULL */
  PKV_ERR_BAD_SHAPE = -2,           /* a size is negative, zero where it may not be, or inconsistent */
  PKV_ERR_UNSUPPORTED = -3,         /* geometry the call does not serve, or no sm_103 device */
  PKV_ERR_WORKSPACE_TOO_SMALL = -4, /* workspace_bytes below the matching *_workspace_bytes() */
  PKV_ERR_CUDA = -5,                /* a CUDA runtime call or the launch failed */
  PKV_ERR_DEVICE_TIMEOUT = -6,      /* device: a bounded wait for a copy ran out (status word only) */
  PKV_ERR_OUT_OF_BOUNDS = -7,       /* device: page id, slot or length outside the pool/table (status word only) */
  PKV_ERR_MISALIGNED = -8           /* a buffer is not 16-byte aligned */
};

/* Bytes of the status header at the start of every workspace. */
#define PKV_STATUS_BYTES 256

/* Zero a workspace (cudaMemsetAsync on `stream`). Call once after allocating it. */
int pkv_workspace_init(void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/*
 * Read the status word of a workspace: waits for `stream`, then copies the
 * word to the host. For tests and debugging only (it synchronises).
 * Returns the device status (PKV_OK or a PKV_ERR_* code), or PKV_ERR_CUDA.
 */
int pkv_read_status(const void* workspace, pkv_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* pkv_status_string(int status);

/*
 * pkv_append -- write the key and value rows of new tokens into their slots.
 *
 * Source: the KV cache grows by one row per generated token and by a chunk of
 * rows per prefill chunk ("FunASR vLLM Inference Engine Guide", section 2:
 * PagedAttention with on-demand allocation; "Optimizing ASR for 90-minute
 * multi-speaker audio", section "LLM prefill").
 *
 *  k_new, v_new:  bf16 [n_tokens][num_kv_heads][head_dim], 16-byte aligned.
 *  slot_mapping:  int32 [n_tokens]; token t goes to slot slot_mapping[t];
 *                 a negative slot skips the token; a slot >= num_pages *
 *                 page_size sets PKV_ERR_OUT_OF_BOUNDS and is skipped.
 *  n_tokens:      >= 0 (0 launches nothing).
 *  k_pages, v_pages: the pools, updated in place. Bit-exact copy.
 *  workspace:     may be NULL (device errors then go unreported); otherwise
 *                 at least PKV_STATUS_BYTES, 4-byte aligned.
 */
int pkv_append(const void* k_new, const void* v_new, const int32_t* slot_mapping, int32_t n_tokens,
               void* k_pages, void* v_pages, const pkv_cache_desc* desc, pkv_stream_t stream,
               void* workspace, size_t workspace_bytes);

/*
 * Workspace bytes pkv_decode_attn needs for `batch` requests on the current
 * device: the status header, one counter per (request, KV head), and the
 * split-KV partial records (two areas of two 1056-byte records per CTA of the
 * launch grid, one per merge scheme). Returns 0 for unsupported arguments.
 */
size_t pkv_decode_workspace_bytes(const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq);

/*
 * pkv_decode_attn -- decode attention over the paged KV cache.
 *
 * Source: PagedAttention decoding ("FunASR vLLM Inference Engine Guide",
 * section 2); decode dominates long-audio serving ("Optimizing ASR for
 * 90-minute multi-speaker audio", section "Time spent: profiling").
 *
 * For every request b and query head h:
 *   out[b][h] = sum_j softmax_j(scale * <q[b][h], k_j>) v_j,  j < seq_lens[b],
 * with k_j, v_j the rows of KV head h / (num_q_heads / num_kv_heads) at
 * logical position j. seq_lens counts the token appended this step (append
 * first). A request with seq_lens[b] == 0 (a padding row of a graph bucket)
 * gets an all-zero output row. Inputs bf16, fp32 accumulation, bf16 output.
 * The split of long contexts over CTAs and the merge of the partial results
 * happen inside the call; the result does not depend on page placement.
 *
 *  q:            bf16 [batch][num_q_heads][head_dim]
 *  k_pages, v_pages: bf16 pools (see layout above), 16-byte aligned
 *  block_table:  int32 [batch][max_pages_per_seq]
 *  seq_lens:     int32 [batch], 0 <= seq_lens[b] <= max_pages_per_seq * page_size
 *                (larger values are clamped and set PKV_ERR_OUT_OF_BOUNDS)
 *  out:          bf16 [batch][num_q_heads][head_dim]
 *  scale:        softmax scale (1/sqrt(head_dim) for the Qwen3 decoder)
 *  batch:        >= 0 (0 launches nothing), max_pages_per_seq >= 1;
 *                batch * max_pages_per_seq * max(num_kv_heads, 8) < 2^31
 *                (PKV_ERR_BAD_SHAPE beyond; the same for the fused calls)
 *  workspace:    >= pkv_decode_workspace_bytes(desc, batch, max_pages_per_seq)
 */
int pkv_decode_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                    const int32_t* seq_lens, void* out, float scale, pkv_stream_t stream,
                    const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq, void* workspace,
                    size_t workspace_bytes);

/*
 * pkv_decode_append_attn -- one decode step of one layer: KV append fused into
 * decode attention (one launch instead of pkv_append + pkv_decode_attn).
 *
 * Source: each generated token adds one K/V row per layer to the paged cache
 * and then attends over the whole cache ("FunASR vLLM Inference Engine Guide",
 * section 2; "Optimizing ASR for 90-minute multi-speaker audio", section
 * "Autoregressive decoding").
 *
 * For every request b with seq_lens[b] > 0, the rows k_new[b][g][:] and
 * v_new[b][g][:] of every KV head g are written at logical position
 * seq_lens[b] - 1 (page block_table[b][(seq_lens[b]-1) / page_size], slot
 * (seq_lens[b]-1) % page_size), bit-exactly; then out is computed exactly as
 * by pkv_decode_attn over seq_lens[b] positions, the new one included. The
 * result equals pkv_append with slot_mapping[b] = that slot followed by
 * pkv_decode_attn.
 *
 *  k_new, v_new: bf16 [batch][num_kv_heads][head_dim], 16-byte aligned
 *  k_pages, v_pages: the pools, updated in place at the new slots only
 *  flags:        0 or PKV_DECODE_EARLY_PREFETCH (see below); other bits are
 *                rejected with PKV_ERR_UNSUPPORTED
 *  other arguments and the workspace: as for pkv_decode_attn
 */
int pkv_decode_append_attn(const void* q, const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                           const int32_t* block_table, const int32_t* seq_lens, void* out, float scale,
                           pkv_stream_t stream, const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq,
                           void* workspace, size_t workspace_bytes, uint32_t flags);

/*
 * Flag for pkv_decode_append_attn (pkv_decode_attn_fp8 has a wider promise, see
 * there). Every kernel of the library is launched
 * with programmatic stream serialisation and normally waits for the previous
 * kernel in the stream before it reads any argument. With this flag the
 * caller promises that the previous kernel writes neither k_pages / v_pages
 * nor block_table nor seq_lens (the usual case in a decode step, where the
 * previous kernel produces q, k_new and v_new): the call then reads those
 * while that kernel is still finishing and starts copying pages into shared
 * memory, and waits for it only before it reads q / k_new / v_new or writes
 * anything. Pass 0 when the promise does not hold (for example right after
 * pkv_append or a prefill chunk that wrote the same pool).
 */
#define PKV_DECODE_EARLY_PREFETCH 1u

/*
 * pkv_decode_append_rope_attn -- pkv_decode_append_attn with the rotary
 * position embedding of the new token applied on the way: one launch for the
 * step that precedes decode attention in a RoPE decoder and the attention.
 *
 * Source: the decoder is a Qwen3-style causal LM with RoPE theta 1e6
 * ("Fun-ASR-Nano Native Runtime Design", section "Decoder And Prompt"). The
 * pages name RoPE and theta only; the rotate-half form of Qwen3 decoders is
 * taken: dims i and i + head_dim/2 form a pair rotated by the angle of
 * (position, i).
 *
 * For every request b with seq_lens[b] > 0, at position p = seq_lens[b] - 1,
 * with c = rope_cos_sin[p][i] and s = rope_cos_sin[p][head_dim/2 + i]:
 *  - the key row written is k_new[b][g] rotated and rounded to bf16 (ties to
 *    even), each pair (x1, x2) = (k[i], k[i + head_dim/2]) evaluated in fp32
 *    as y1 = fmaf(x1, c, -(x2 * s)), y2 = fmaf(x2, c, x1 * s), each product
 *    rounded to fp32 first (so the written bits are defined exactly);
 *  - every query row q[b][h] is rotated the same way in fp32, then rounded to
 *    bf16 (ties to even), the operand precision of the score product;
 *  - v_new is written unchanged; everything else is as pkv_decode_append_attn.
 *
 *  rope_cos_sin: fp32 [rope_max_pos][head_dim], row p = cos(p w_i) for
 *                i < head_dim/2, then sin(p w_i) (w_i = theta^(-2i/head_dim));
 *                caller-owned device memory, 16-byte aligned, read only
 *                (pkv_rope_table builds it).
 *                A position >= rope_max_pos is reported as
 *                PKV_ERR_OUT_OF_BOUNDS in the status word and clamped to the
 *                last row.
 *  rope_max_pos: rows of the table (>= 1)
 *  other arguments, flags and the workspace: as for pkv_decode_append_attn
 */
int pkv_decode_append_rope_attn(const void* q, const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                                const int32_t* block_table, const int32_t* seq_lens, const float* rope_cos_sin,
                                int32_t rope_max_pos, void* out, float scale, pkv_stream_t stream,
                                const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq, void* workspace,
                                size_t workspace_bytes, uint32_t flags);

/*
 * pkv_rope_table -- build the cos/sin table the RoPE decode call reads.
 *
 * Source: the decoder's rotary position embedding with theta 1e6
 * ("Fun-ASR-Nano Native Runtime Design", section "Decoder And Prompt"), in the
 * rotate-half form of Qwen3 decoders (the pages name RoPE and theta only).
 *
 * Writes table[p][i] = cos(p w_i) and table[p][head_dim/2 + i] = sin(p w_i)
 * for p < max_pos, i < head_dim/2, w_i = theta^(-2i / head_dim); each angle
 * and its cosine and sine are evaluated in double and rounded to float once.
 *
 *  table:     fp32 [max_pos][head_dim], caller-owned device memory, 16-byte
 *             aligned, written on `stream`
 *  max_pos:   >= 1 rows (positions 0 .. max_pos - 1)
 *  head_dim:  even, 2 .. 1024 (the decode calls use 64 or 128)
 *  theta:     > 0 (1e6 for the Qwen3 decoder)
 * Returns PKV_ERR_BAD_SHAPE for other sizes, PKV_ERR_MISALIGNED for an
 * unaligned table; nothing is written then.
 */
int pkv_rope_table(float* table, int32_t max_pos, int32_t head_dim, double theta, pkv_stream_t stream);

/*
 * pkv_append_rope -- write the key and value rows of new tokens into their
 * slots with the rotary position embedding (and the per-head RMS norm of
 * Qwen3-style decoders) applied on the way, and rotate the tokens' query rows.
 *
 * Source: as for pkv_append; the decoder is a Qwen3-style causal LM with RoPE
 * theta 1e6 ("Fun-ASR-Nano Native Runtime Design", section "Decoder And
 * Prompt"). The pages name RoPE and theta only; rotate-half pairs and the
 * norms of the q and k rows before the rotation are those of Qwen3 decoders.
 * It is the step before pkv_prefill_chunk_attn (whose queries and cached keys
 * are already rotated) and before pkv_decode_attn.
 *
 * For token t, position p = positions[t], every row x of head_dim values, fp32:
 *   u = x * w,  w = q_weight or k_weight     (u = x where the weight is NULL)
 *   y1 = fmaf(u1, c, -(u2 * s)),  y2 = fmaf(u2, c, u1 * s)   for the pairs
 *     (u1, u2) = (u[i], u[i + head_dim/2]), c = table[p][i],
 *     s = table[p][head_dim/2 + i]           (y = u where the table is NULL)
 *   y *= 1 / sqrt(mean(x^2) + eps)           (only where a weight is given)
 * and y is rounded to bf16 (ties to even) once. Without weights the key rows
 * written are those of pkv_decode_append_rope_attn, bit for bit; without
 * weights and table they are pkv_append's. Value rows are copied bit for bit.
 *
 *  q:            bf16, token t's [num_q_heads][head_dim] at q + t * q_stride,
 *                or NULL (with q_out NULL): no query rows
 *  k_new, v_new: bf16, token t's [num_kv_heads][head_dim] at k_new + t *
 *                k_stride, v_new + t * v_stride
 *  *_stride:     elements between tokens, at least one token's row count *
 *                head_dim and a multiple of 8 (rows of a fused q/k/v
 *                projection need no copy); not used for n_tokens = 1
 *  positions:    int32 [n_tokens]; needed with a table only. A position
 *                outside [0, rope_max_pos) is clamped and, unless the token has
 *                neither a query row nor a slot, sets PKV_ERR_OUT_OF_BOUNDS
 *  slot_mapping: int32 [n_tokens]; as for pkv_append: a negative slot skips
 *                the token's k and v (its query rows are still written), one
 *                past the pool sets PKV_ERR_OUT_OF_BOUNDS and is skipped. The
 *                slots that are not negative must differ from each other (of
 *                two equal ones either row's values may end up in the slot)
 *  n_tokens:     >= 0 (0 launches nothing); n_tokens * (num_q_heads + 2 *
 *                num_kv_heads) < 2^31
 *  rope_cos_sin: fp32 [rope_max_pos][head_dim] (pkv_rope_table), or NULL
 *  q_weight, k_weight: bf16 [head_dim], each may be NULL
 *  eps:          >= 0, read where a weight is given
 *  q_out:        bf16 [n_tokens][num_q_heads][head_dim]; may be q itself where
 *                q's tokens are contiguous
 *  k_pages, v_pages: the bf16 pools, updated in place
 *  workspace:    as for pkv_append (may be NULL)
 * Every buffer but positions and slot_mapping is 16-byte aligned.
 */
int pkv_append_rope(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                    int64_t v_stride, const int32_t* positions, const int32_t* slot_mapping, int32_t n_tokens,
                    const float* rope_cos_sin, int32_t rope_max_pos, const void* q_weight, const void* k_weight,
                    float eps, void* q_out, void* k_pages, void* v_pages, const pkv_cache_desc* desc,
                    pkv_stream_t stream, void* workspace, size_t workspace_bytes);

/*
 * The 8-bit paged KV cache. The source pages have no counterpart: decode is
 * bound by the bytes of the cache, and this cache has half of them.
 *
 *  - k_pages, v_pages: e4m3 [num_pages][num_kv_heads][page_size][head_dim]
 *    (4 exponent bits, 3 mantissa bits, largest value 448, no infinities).
 *  - kv_scales: one byte per row, [num_pages][num_kv_heads][2][page_size]: the
 *    K rows' scales, then the V rows'. Byte b stands for 2^(b - 127) (e8m0).
 *    The appends write 47 .. 227. Of the other bytes, which only a caller can
 *    put there, pkv_expand_fp8 and pkv_tree_attn_fp8 take 255 (NaN in e8m0) as
 *    infinity and 0 as zero; a product past bf16's range is infinite.
 *  - A row x stands for 2^e v: e is the least integer with max |x_i| <= 448 *
 *    2^e over the finite x_i, clamped to [-80, 100] (-80 for a row of zeros),
 *    and v_i = x_i * 2^-e rounded to e4m3, ties to even, saturating at 448
 *    (infinities saturate too; NaN stays NaN). 2^e v is exact in bf16.
 *  - Layout, block tables, slots and geometry as for the bf16 pools: page_size
 *    16, head_dim 64 or 128, 1 to 8 query heads per KV head.
 *  - max_pages_per_seq <= 2^27 - 2 in the calls that take it.
 */

/*
 * pkv_append_rope_fp8 -- pkv_append_rope into the 8-bit cache: key rows are
 * quantised from the fp32 y above (no bf16 rounding in between), value rows
 * from their bf16 values. The query rows are as for pkv_append_rope. Without
 * table and weights it is the plain append of the 8-bit cache.
 */
int pkv_append_rope_fp8(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                        int64_t v_stride, const int32_t* positions, const int32_t* slot_mapping, int32_t n_tokens,
                        const float* rope_cos_sin, int32_t rope_max_pos, const void* q_weight, const void* k_weight,
                        float eps, void* q_out, void* k_pages, void* v_pages, void* kv_scales,
                        const pkv_cache_desc* desc, pkv_stream_t stream, void* workspace, size_t workspace_bytes);

/*
 * pkv_decode_attn_fp8 -- pkv_decode_attn over the 8-bit cache: the same sums
 * over the rows that the cache stands for, in fp32, with the keys and values
 * unrounded and the softmax weights p_j rounded to fp16, with the scale 2^(e_j)
 * of their value row, before they multiply V: p_j 2^(e_j) is off by at most
 * 2^-11 of itself, or by 2^-39 of the largest of them where that is more.
 * Weights below 2^-126 count as 0. Query values are exact down to 2^-31 of
 * their row's largest and held to 2^-39 of it below. Arguments, lengths of
 * zero, errors and the workspace (pkv_decode_workspace_bytes) are
 * pkv_decode_attn's; a workspace may serve both in turn.
 *
 *  flags: 0 or PKV_DECODE_EARLY_PREFETCH. Here the caller promises that the
 *         previous kernel on the stream writes neither block_table nor
 *         seq_lens, and of the cache at most the rows at position
 *         seq_lens[b] - 1 of the requests (so pkv_append_rope_fp8 of the
 *         step's tokens qualifies): the call then copies every request's pages
 *         but the last two while that kernel is still finishing, and waits for
 *         it before it reads those, q or anything else. Other bits are
 *         rejected with PKV_ERR_UNSUPPORTED.
 */
int pkv_decode_attn_fp8(const void* q, const void* k_pages, const void* v_pages, const void* kv_scales,
                        const int32_t* block_table, const int32_t* seq_lens, void* out, float scale,
                        pkv_stream_t stream, const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq,
                        void* workspace, size_t workspace_bytes, uint32_t flags);

/*
 * pkv_decode_append_attn_fp8 -- one decode step of one layer over the 8-bit
 * cache in one launch: pkv_append_rope_fp8 of each request's new token at
 * position seq_lens[b] - 1, then pkv_decode_attn_fp8 over seq_lens[b]
 * positions with the query rows normalised, rotated and rounded to bf16 as that
 * append would (nothing is written to q). The rows written and the outputs are
 * those of the two calls, bit for bit.
 *
 *  q, k_new, v_new: bf16 [batch][num_q_heads][head_dim] and
 *                [batch][num_kv_heads][head_dim], contiguous; requests of
 *                length 0 write nothing
 *  rope_cos_sin, q_weight, k_weight: each may be NULL, as for
 *                pkv_append_rope. A position >= rope_max_pos is clamped to the
 *                table's last row and sets PKV_ERR_OUT_OF_BOUNDS
 *  flags:        0 or PKV_DECODE_EARLY_PREFETCH, with the promise that the
 *                previous kernel writes neither the cache (scales included)
 *                nor block_table, seq_lens, rope_cos_sin or the weights
 *  other arguments and the workspace: as for pkv_decode_attn_fp8
 */
int pkv_decode_append_attn_fp8(const void* q, const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                               void* kv_scales, const int32_t* block_table, const int32_t* seq_lens,
                               const float* rope_cos_sin, int32_t rope_max_pos, const void* q_weight,
                               const void* k_weight, float eps, void* out, float scale, pkv_stream_t stream,
                               const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq, void* workspace,
                               size_t workspace_bytes, uint32_t flags);

/*
 * pkv_expand_fp8 -- pages of the 8-bit cache as bf16 pages, exactly: the
 * prefix that pkv_prefill_chunk_attn reads when a prompt is cached in 8 bits.
 *
 * For every request s and page p < ceil(seq_lens[s] / page_size), the rows of
 * page block_table[s][p] of the 8-bit cache that lie before seq_lens[s] are
 * written to the same rows of page out_block_table[s][p] of k_out and v_out
 * (bf16 [out_num_pages][num_kv_heads][page_size][head_dim]). Rows at or past
 * seq_lens[s] and other pages are left as they were.
 *
 *  block_table, out_block_table: int32 [num_seqs][max_pages_per_seq]; entries
 *                past a request's last page are never read. A page id outside
 *                its pool sets PKV_ERR_OUT_OF_BOUNDS and the page is skipped.
 *                No two pages of a call may have the same output page
 *  seq_lens:     int32 [num_seqs]; clamped to [0, max_pages_per_seq *
 *                page_size] with PKV_ERR_OUT_OF_BOUNDS
 *  num_seqs:     >= 0 (0 launches nothing); num_seqs * max_pages_per_seq *
 *                max(num_kv_heads, 8) < 2^31
 *  desc:         the 8-bit cache's geometry (num_pages its pages)
 *  workspace:    as for pkv_append (may be NULL)
 */
int pkv_expand_fp8(const void* k_pages, const void* v_pages, const void* kv_scales, const int32_t* block_table,
                   const int32_t* seq_lens, int32_t num_seqs, int32_t max_pages_per_seq, void* k_out, void* v_out,
                   const int32_t* out_block_table, int32_t out_num_pages, const pkv_cache_desc* desc,
                   pkv_stream_t stream, void* workspace, size_t workspace_bytes);

/*
 * Workspace bytes pkv_prefill_chunk_attn needs: the status header, two partial
 * records per SM of the current device (for each of the 2 query heads of a
 * pair: 128 rows x head_dim dims of fp16 O / l, then fp32 max and sum per row:
 * 67,584 bytes at head_dim 128, and as much room at 64), for query tiles whose
 * key range is cut between CTAs, and split counters (num_seqs x head pairs x
 * ceil(max_q_len / 128) x 2 ints, with num_kv_heads x ceil(G / 2) head pairs).
 * Calls of any geometry, num_seqs and max_q_len may share a workspace that is
 * large enough for each of them.
 */
size_t pkv_prefill_workspace_bytes(const pkv_cache_desc* desc, int32_t num_seqs, int32_t max_q_len);

/*
 * pkv_prefill_chunk_attn -- causal attention of prefill chunks over the cache.
 *
 * Source: "Optimizing ASR for 90-minute multi-speaker audio", section
 * "Chunked prefill for long audio": a long prompt is prefilled in 4096-token
 * chunks, one per scheduler step, between other requests' decode steps.
 *
 * Request n owns query rows cu_q_lens[n] .. cu_q_lens[n+1]-1 of q; its chunk
 * follows prefix_lens[n] cached tokens, and row i of the chunk (absolute
 * position prefix_lens[n] + i) attends keys 0 .. prefix_lens[n] + i of the
 * request (bottom-right causal alignment). The chunk's own K/V rows must
 * already be in the pool (pkv_append first). bf16 inputs, fp32 accumulation on
 * the tensor cores, the softmax weights rounded to bf16 before they multiply
 * V, bf16 output.
 *
 *  q, out:       bf16 [total_q][num_q_heads][head_dim]
 *  block_table:  int32 [num_seqs][max_pages_per_seq]
 *  prefix_lens:  int32 [num_seqs]
 *  cu_q_lens:    int32 [num_seqs + 1], cu_q_lens[0] = 0, non-decreasing,
 *                cu_q_lens[num_seqs] <= total_q
 *  total_q:      rows of q and out (host value; bounds every access)
 *  max_q_len:    host-side upper bound on any chunk length (sizes the grid
 *                and the workspace). A chunk longer than
 *                128 * ceil(max_q_len / 128) rows sets PKV_ERR_OUT_OF_BOUNDS
 *                in the status word; its rows past that bound are not
 *                computed.
 *  workspace:    >= pkv_prefill_workspace_bytes(...), zeroed once by
 *                pkv_workspace_init (the call leaves its counters at zero)
 * Limits: num_pages * num_kv_heads * page_size < 2^31 rows per pool;
 * num_seqs <= 1024 (PKV_ERR_UNSUPPORTED beyond).
 */
int pkv_prefill_chunk_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                           const int32_t* prefix_lens, const int32_t* cu_q_lens, int32_t num_seqs, int32_t total_q,
                           void* out, float scale, pkv_stream_t stream, const pkv_cache_desc* desc,
                           int32_t max_pages_per_seq, int32_t max_q_len, void* workspace, size_t workspace_bytes);

/*
 * Workspace bytes pkv_mixed_step_attn needs: the prefill workspace of the
 * chunk part (see pkv_prefill_workspace_bytes), then one counter per (decode
 * request, KV head) and, where a decode context spans more than 64 pages,
 * partial records of its 64-page chunks (1056 bytes each). Returns 0 for
 * unsupported arguments.
 */
size_t pkv_mixed_workspace_bytes(const pkv_cache_desc* desc, int32_t num_seqs, int32_t max_q_len, int32_t dec_batch,
                                 int32_t dec_max_pages_per_seq);

/*
 * pkv_mixed_step_attn -- one scheduler step that interleaves chunked prefill
 * with decode: the attention of prefill chunks and of decode requests over
 * the same paged cache, in one launch.
 *
 * Source: a long prompt is prefilled in 4096-token chunks, one per scheduler
 * step, between other requests' decode steps ("Optimizing ASR for 90-minute
 * multi-speaker audio", section "Chunked prefill for long audio"); running
 * the chunk and the decode batch as one kernel is the step the same page's
 * section "后续计划" (future work) leaves open with CUDA-graph capture of
 * chunked prefill.
 *
 * Computes exactly what pkv_prefill_chunk_attn computes for the chunk
 * arguments (q .. max_q_len) and what pkv_decode_attn computes for the decode
 * arguments (dec_*), both over k_pages / v_pages; results are within the same
 * tolerance as those calls but not bit-identical to them (the work is split
 * differently). All K/V rows, the chunks' and the decode tokens', must already
 * be in the pools (pkv_append first). The decode requests run in CTAs of their
 * own, one per chunk of up to 64 pages of a (request, KV head), that the
 * hardware starts on the SMs the chunk leaves free (the tail of a short chunk;
 * for a long cached prefix the chunk's persistent schedule keeps a few SMs for
 * them, in proportion to their pages); chunks of one context are merged by
 * log-sum-exp.
 *
 *  chunk arguments: as for pkv_prefill_chunk_attn; num_seqs = 0 (or total_q =
 *                   0, max_q_len = 0) means no chunk, and q, out, block_table,
 *                   prefix_lens and cu_q_lens may then be NULL
 *  dec_q, dec_out:  bf16 [dec_batch][16][128], 16-byte aligned
 *  dec_block_table: int32 [dec_batch][dec_max_pages_per_seq]
 *  dec_seq_lens:    int32 [dec_batch]; 0 gives an all-zero output row; larger
 *                   than dec_max_pages_per_seq * 16 is clamped and set
 *                   PKV_ERR_OUT_OF_BOUNDS
 *  dec_batch:       0 .. 1024 (0: the call is pkv_prefill_chunk_attn)
 *  workspace:       >= pkv_mixed_workspace_bytes(desc, num_seqs, max_q_len,
 *                   dec_batch, dec_max_pages_per_seq), zeroed once by
 *                   pkv_workspace_init (the call leaves its counters at zero);
 *                   serves mixed-step calls only, of any sizes it is large
 *                   enough for
 * Geometry: 16 query / 8 KV heads, head_dim 128, page 16 (PKV_ERR_UNSUPPORTED
 * otherwise).
 */
int pkv_mixed_step_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                        const int32_t* prefix_lens, const int32_t* cu_q_lens, int32_t num_seqs, int32_t total_q,
                        void* out, int32_t max_pages_per_seq, int32_t max_q_len, const void* dec_q,
                        const int32_t* dec_block_table, const int32_t* dec_seq_lens, void* dec_out, int32_t dec_batch,
                        int32_t dec_max_pages_per_seq, float scale, pkv_stream_t stream, const pkv_cache_desc* desc,
                        void* workspace, size_t workspace_bytes);

/*
 * Workspace bytes the tree attention calls need: the status header, a 16-byte
 * descriptor per SM of the current device and two partial records per SM (67,584
 * bytes each), for items whose keys are cut between CTAs. One size for all calls
 * on a device: tree attention calls of any geometry, sizes and cache type may
 * share a workspace (in stream order). Returns 0 for unsupported arguments.
 */
size_t pkv_tree_workspace_bytes(const pkv_cache_desc* desc, int32_t num_seqs, int32_t max_nodes);

/*
 * pkv_tree_attn -- attention of drafted tokens over the paged cache: the
 * verification step of speculative decoding.
 *
 * Source: the pages have no counterpart. Decode takes over 94% of the time on
 * long audio ("Optimizing ASR for 90-minute multi-speaker audio", section "Time
 * spent: profiling") and reads a request's whole cache for each new token; this
 * call reads it once for all tokens that a draft proposes.
 *
 * Request n owns the nodes (rows of q) cu_nodes[n] .. cu_nodes[n+1]-1, T of
 * them, in any order that the caller numbers them in (for pkv_keep_nodes:
 * parents before children). Their key and value rows lie in the cache behind the
 * request's P = prefix_lens[n] tokens, node i's at position P + i (append them
 * first: pkv_append_rope with slots of positions P + i and rotary positions of
 * the nodes' depths). Node i sees positions 0 .. P - 1 and the nodes j < T whose
 * bit j of tree_mask[cu_nodes[n] + i] is set (its ancestors and, usually,
 * itself). Without masks the nodes are a chain: node i sees nodes 0 .. i.
 *   out[i][h] = sum_j softmax_j(scale * <q[i][h], k_j>) v_j over what it sees,
 * zeros for a node that sees nothing. bf16 inputs, fp32 sums and statistics, the
 * softmax weights rounded to bf16 before they multiply V, bf16 output. Rows that a
 * node does not see have no influence, whatever they hold.
 *
 *  q, out:       bf16 [total_nodes][num_q_heads][head_dim]; rows past
 *                cu_nodes[num_seqs] of out are left as they were
 *  block_table:  int32 [num_seqs][max_pages_per_seq]; it covers the nodes too
 *  prefix_lens:  int32 [num_seqs], >= 0; P + T <= max_pages_per_seq * page_size
 *  cu_nodes:     int32 [num_seqs + 1], non-decreasing, cu_nodes[num_seqs] <=
 *                total_nodes. A request without nodes (padding) costs nothing
 *  tree_mask:    int64 [total_nodes], 8-byte aligned, or NULL. Bits at and
 *                past T are ignored
 *  max_nodes:    host-side upper bound on any request's nodes, 0 .. 64
 *                (PKV_ERR_UNSUPPORTED beyond; 0 launches nothing)
 *  num_seqs:     0 .. 1024 (PKV_ERR_UNSUPPORTED beyond); num_seqs *
 *                max_pages_per_seq * max(num_kv_heads, 8) < 2^31;
 *                max_pages_per_seq <= 2^27 - 8
 *  workspace:    >= pkv_tree_workspace_bytes(...), its status header zeroed once
 *                by pkv_workspace_init; a call writes what it reads of the rest.
 *                It serves tree attention calls only
 * Two kernels where a request's keys may be cut between CTAs (tables of more than
 * 32 pages), else one. A request whose lengths are out of bounds, or that has more
 * than max_nodes nodes, sets PKV_ERR_OUT_OF_BOUNDS and its rows are not written. A
 * page id outside the pool sets it too; the rows of that request are then
 * undefined.
 * Geometry: head_dim 64 or 128, 1 to 8 query heads per KV head, page_size 16.
 */
int pkv_tree_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                  const int32_t* prefix_lens, const int32_t* cu_nodes, const int64_t* tree_mask, int32_t num_seqs,
                  int32_t total_nodes, int32_t max_nodes, void* out, float scale, pkv_stream_t stream,
                  const pkv_cache_desc* desc, int32_t max_pages_per_seq, void* workspace, size_t workspace_bytes);

/*
 * pkv_tree_attn_fp8 -- pkv_tree_attn over the 8-bit cache. The rows that it
 * stands for are exact in bf16: the outputs are those of pkv_expand_fp8 followed
 * by pkv_tree_attn, bit for bit, the softmax weights in bf16 (pkv_decode_attn_fp8
 * holds them in fp16). It halves the cache's memory, not the time: the expansion
 * takes what the bytes save.
 */
int pkv_tree_attn_fp8(const void* q, const void* k_pages, const void* v_pages, const void* kv_scales,
                      const int32_t* block_table, const int32_t* prefix_lens, const int32_t* cu_nodes,
                      const int64_t* tree_mask, int32_t num_seqs, int32_t total_nodes, int32_t max_nodes, void* out,
                      float scale, pkv_stream_t stream, const pkv_cache_desc* desc, int32_t max_pages_per_seq,
                      void* workspace, size_t workspace_bytes);

/*
 * pkv_keep_nodes -- after verification: the rows of the accepted nodes move up
 * to consecutive positions behind the prefix, in all layers at once.
 *
 * Source: the pages have no counterpart (see pkv_tree_attn).
 *
 * For every request s, layer and i < path_lens[s], the K and V rows (and, of an
 * 8-bit cache, their scale bytes) at position prefix_lens[s] + path[s][i] are
 * written to position prefix_lens[s] + i, bit-exactly and as if all rows were
 * read before any is written. The request's length is then prefix_lens[s] +
 * path_lens[s]. Other rows are left as they were.
 *
 *  path:         int32 [num_seqs][max_path], the accepted nodes' numbers,
 *                rising (0 <= path[s][0] < path[s][1] < ...); entries at and
 *                past path_lens[s] are not read. An entry that does not rise, or
 *                whose position or page lies outside the table or the pool, sets
 *                PKV_ERR_OUT_OF_BOUNDS and its row is not moved
 *  path_lens:    int32 [num_seqs], 0 .. max_path (clamped, with
 *                PKV_ERR_OUT_OF_BOUNDS)
 *  prefix_lens, block_table: as for pkv_tree_attn; no two requests may have
 *                the same page among those that hold their nodes
 *  num_seqs:     >= 0 (0 launches nothing); num_seqs * max_pages_per_seq *
 *                max(num_kv_heads, 8) < 2^31; max_pages_per_seq <= 2^27 - 2
 *  max_path:     0 .. 64 (PKV_ERR_UNSUPPORTED beyond; 0 launches nothing)
 *  k_pages, v_pages, kv_scales: HOST arrays of n_layers device pointers, one
 *                pool per layer, no pool twice, read during the call only; all
 *                pools of the geometry of `desc`. kv_scales NULL: bf16 pools; else 8-bit ones
 *  n_layers:     >= 0 (0 launches nothing); one launch per 64 layers
 *  workspace:    as for pkv_append (may be NULL)
 */
int pkv_keep_nodes(const int32_t* path, const int32_t* path_lens, const int32_t* prefix_lens,
                   const int32_t* block_table, int32_t num_seqs, int32_t max_path, int32_t max_pages_per_seq,
                   void* const* k_pages, void* const* v_pages, void* const* kv_scales, int32_t n_layers,
                   const pkv_cache_desc* desc, pkv_stream_t stream, void* workspace, size_t workspace_bytes);

/*
 * pkv_copy_pages -- whole pages to other pages, in all layers at once: what a
 * forked request (a companion prompt, another hypothesis) cannot share with its
 * origin, usually the last page that both would append to.
 *
 * Source: the cache is allocated on demand, page by page ("FunASR vLLM Inference
 * Engine Guide", section 2); the pages do not say how requests part.
 *
 *  src, dst:     int32 [n_pairs]; page dst[i] of every pool becomes page src[i]
 *                of it (and, of an 8-bit cache, its scale bytes). A pair with a
 *                negative page is skipped; one with a page >= num_pages sets
 *                PKV_ERR_OUT_OF_BOUNDS and is skipped. No dst may be another
 *                pair's src or dst (either row's bytes may end up there)
 *  n_pairs:      >= 0 (0 launches nothing)
 *  k_pages, v_pages, kv_scales, n_layers, workspace: as for pkv_keep_nodes
 */
int pkv_copy_pages(const int32_t* src, const int32_t* dst, int32_t n_pairs, void* const* k_pages, void* const* v_pages,
                   void* const* kv_scales, int32_t n_layers, const pkv_cache_desc* desc, pkv_stream_t stream,
                   void* workspace, size_t workspace_bytes);

/*
 * pkv_decode_attn_noalloc -- pkv_decode_attn without a caller-provided workspace.
 *
 * The source pages have no counterpart to this call: it exists for callers
 * that may not allocate device memory where they run decode attention (for
 * example a plug-in inside a host runtime that owns all device memory through
 * its own pool, or a serving loop that reserves memory once at start-up and
 * must not allocate, or implicitly synchronise, afterwards). The caller still
 * passes q, the pools, the block table, the lengths and out, with the same
 * meaning and layout as for pkv_decode_attn; the split-KV scratch comes from a
 * fixed array inside the library instead of a workspace.
 *
 *  - The scratch is one device array of PKV_NOALLOC_SCRATCH_BYTES (2 MiB).
 *    Every GPU that loads the library holds it until the process exits. The
 *    call itself allocates and frees nothing.
 *  - Geometry: 16 query / 8 KV heads, head_dim 128, page size 16 only (the
 *    tuned decode kernel); other geometries return PKV_ERR_UNSUPPORTED.
 *  - Limit: batch <= PKV_NOALLOC_MAX_BATCH (256), and the scratch must cover
 *    the device's split partials (it does for up to ~240 SMs; a GB300 has 152).
 *    Larger requests return PKV_ERR_WORKSPACE_TOO_SMALL without launching.
 *  - The first call on a device, and the first call in each other context
 *    on it, looks up the array's device address (each context loads its own
 *    copy of the array): a one-time set-up; make that first call before any
 *    CUDA-graph capture. The call is not supported after cudaDeviceReset in
 *    the same process: the device's primary context may come back under the
 *    same handle while the array has moved.
 *  - Every call uses the same array and it keeps the previous call's
 *    contents; each call zeroes the status word, the split counters and records on
 *    `stream` before its kernel. Calls whose kernels overlap on the GPU (on
 *    different streams, or in parallel graph branches) race on the array:
 *    issue them in order on one stream.
 *  - Device-side errors are not reported: the status word lives in the
 *    library's array and no call reads it back. A page id outside the pool or
 *    a length beyond the block table is skipped as in pkv_decode_attn. A
 *    bounded wait of the split merge that runs out (see the convention on the
 *    split merge above) leaves the output rows of the affected (request, KV
 *    head) unwritten: `out` keeps whatever it held there, with no signal.
 *    Callers that need to see such errors use pkv_decode_attn.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (2u << 20)
#define PKV_NOALLOC_MAX_BATCH 256

int pkv_decode_attn_noalloc(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                            const int32_t* seq_lens, void* out, float scale, pkv_stream_t stream,
                            const pkv_cache_desc* desc, int32_t batch, int32_t max_pages_per_seq);

/*
 * pkv_selftest_wait_timeout -- diagnostic of the bounded device waits.
 *
 * Not a step of the attention path (the pages have no counterpart): it runs
 * one CTA that waits, through the same bounded-wait helper the kernels use,
 * on a shared-memory barrier that nothing ever completes, for at most
 * limit_cycles SM clock cycles (<= 2^32), and then writes
 * PKV_ERR_DEVICE_TIMEOUT into the workspace status word. Shows that a wait
 * which runs out ends the kernel with an error the host can read
 * (pkv_read_status) and leaves the context usable.
 */
int pkv_selftest_wait_timeout(void* workspace, size_t workspace_bytes, int64_t limit_cycles, pkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
