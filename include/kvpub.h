/*
 * kvpub.h -- replicated FP8 KV cache-store and device-epoch fence (MI355X, gfx950).
 *
 * C ABI of libkvpub.so.  Plain pointers and sizes only: device pointers are
 * HIP device addresses (for example torch tensors' data_ptr()), streams are
 * hipStream_t values passed as void*.
 *
 * What the library does, and where the pages define it:
 *   - kvpub_store: quantize each new token's final Main-KV row (bf16 latent
 *     [512] + bf16 RoPE [64]) and Indexer-K row (bf16 [128]) to FP8 once and
 *     write the bytes straight into every replica of a paged KV cache, with
 *     no gather and no receive-side insert (vLLM PR #52863 "[Kernel][PCP]
 *     Publish replicated KV updates through PyTorch symmetric memory",
 *     Summary, the "THIS PR: publish final rows directly" diagram, and the
 *     Design bullet on fused cache-store kernels writing to every peer).
 *     The replicas must end byte-identical to what gather-then-insert would
 *     give, padded and invalid slots and guard bytes included (same page,
 *     "Correctness and current-head validation").
 *   - kvpub_fence: one launch that advances a device-resident epoch with a
 *     system-scope release and then acquire-waits for every participant, so
 *     that a captured graph advances the epoch on every replay (vLLM PR
 *     #54030 "[Perf][PCP] Fuse direct-KV publication fence", its commit list
 *     and Motivation; PR #52863 Design bullet on the device-epoch barrier and
 *     separate DBO lanes).
 *   - kvpub_graph_create / kvpub_graph_replay: the store + fence sequence of
 *     several layers captured once in a hipGraph and replayed (PR #54030
 *     commit list: a two-GPU replay test checks that every replay advances the
 *     epoch; PR #52863 Design: graph replay is supported).
 *   - kvpub_gather: the reader side -- the rows of given slots read back from
 *     one replica and dequantized to bf16, which is what the attention kernels
 *     that keep reading the local replica consume (PR #52863 Summary and
 *     Design: the existing attention kernels read the local replica in the
 *     fp8_ds_mla layout this path writes).
 *   - kvpub_vmm_*: replica storage at stable virtual addresses that can grow
 *     without moving (PR #52863 Relationship to existing work: the path builds
 *     on a KV cache kept at a stable VA with its own rendezvous, so that the
 *     cache can expand without re-exchanging views).
 *   - all-or-nothing creation and fail-closed fences (PR #54030 commit list:
 *     opt-in allocation is all-or-nothing at startup; a fence timeout must not
 *     let work continue).
 *
 * Byte layout (the pages name the FP8 Main-KV format, fp8_ds_mla, without
 * printing its bytes; this is the library's reading):
 *   Main-KV row, 656 B, at replica + layer*main_layer_stride
 *                          + page*main_page_stride + offset*656:
 *     [0,512)   e4m3fn codes of latent[0..511]
 *     [512,528) fp32 scales of latent tiles [0,128) [128,256) [256,384) [384,512)
 *     [528,656) RoPE bf16 bit patterns, copied unchanged
 *   Indexer-K, at replica + layer*idx_layer_stride + page*idx_page_stride:
 *     [offset*128, +128)     e4m3fn codes of indexer[0..127]
 *     [8192 + offset*4, +4)  fp32 scale of the indexer row
 *   Scaling: per 128-element tile, scale = amax / 448 (binary32), code =
 *   e4m3fn(x / scale) with x / scale rounded to binary32, then rounded to
 *   nearest-even e4m3fn saturating at +-448; an all-zero tile stores scale
 *   +0 and codes 0x00.  All multi-byte fields are little-endian.
 *   Slots: slot s lives in page s / 64 at offset s % 64.  s == -1 marks a
 *   padded token: it is neither read nor written.  Any other slot outside
 *   [0, num_pages*64) is skipped and counted (kvpub_error_read).
 *
 * Errors: functions never abort and no C++ exception crosses this ABI.
 * Argument problems are reported before anything is launched, so nothing is
 * written.  Device-side problems (invalid slots, a fence that timed out) are
 * recorded in the context's device words and reported by kvpub_error_read.
 *
 * Logging: with the environment variable KVPUB_LOG=1 (read once), every
 * kvpub_create, kvpub_create_static and kvpub_destroy of a context prints one
 * line to stderr with its configuration and status; no other call logs.
 */
#ifndef KVPUB_H
#define KVPUB_H

#include <stdint.h>

#if defined(KVPUB_BUILD_SHARED)
#define KVPUB_API __attribute__((visibility("default")))
#else
#define KVPUB_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define KVPUB_ABI_VERSION 1u

#define KVPUB_SLOTS_PER_PAGE 64u
#define KVPUB_LATENT_DIM 512u
#define KVPUB_ROPE_DIM 64u
#define KVPUB_INDEXER_DIM 128u
#define KVPUB_MAIN_ROW_BYTES 656u
#define KVPUB_MAIN_PAGE_BYTES (64u * 656u)            /* 41984 */
#define KVPUB_IDX_PAGE_BYTES (64u * 128u + 64u * 4u)  /* 8448 */
#define KVPUB_IDX_SCALES_OFFSET (64u * 128u)          /* 8192 */
#define KVPUB_MAX_REPLICAS 8u
#define KVPUB_MAX_LANES 64u
#define KVPUB_MAX_PARTICIPANTS 8u
#define KVPUB_MAX_TOKENS (1ll << 30)

typedef struct kvpub_ctx kvpub_ctx;
typedef struct kvpub_graph kvpub_graph;
typedef struct kvpub_vmm kvpub_vmm;
typedef void *kvpub_stream_t; /* hipStream_t; NULL = the null stream */

typedef enum {
    KVPUB_OK = 0,
    KVPUB_ERR_INVALID_ARG = 1,   /* bad argument; nothing was launched */
    KVPUB_ERR_OUT_OF_MEMORY = 2, /* an allocation failed; nothing is left allocated */
    KVPUB_ERR_UNSUPPORTED = 3,   /* device is not gfx950, or the call does not support this
                                    configuration (documented per call) */
    KVPUB_ERR_HIP = 4,           /* a HIP runtime call failed */
    KVPUB_ERR_CAPTURING = 5,     /* a synchronizing call while a stream capture is active */
    KVPUB_ERR_FENCE_TIMEOUT = 6, /* a fence timed out: the context is poisoned */
    KVPUB_ERR_IN_USE = 7,        /* the device's static context (kvpub_create_static) is in use */
    KVPUB_STATUS_MAX_ENUM = 0x7FFFFFFF /* not a status: makes every non-negative int32 a valid
                                          kvpub_status value, so a C caller may pass any code */
} kvpub_status;

/* Sticky device flags reported by kvpub_error_read. */
#define KVPUB_FLAG_FENCE_TIMEOUT 0x1u /* a fence gave up waiting */
#define KVPUB_FLAG_POISONED 0x2u      /* later stores and fences do nothing */

typedef struct {
    uint32_t struct_size;       /* sizeof(kvpub_config) */
    uint32_t num_replicas;      /* R, 1..8 */
    uint32_t num_layers;        /* L >= 1 */
    uint32_t block_size;        /* slots per page; must be 64 */
    uint64_t num_pages;         /* pages per replica per layer, >= 1 */
    uint64_t main_page_stride;  /* bytes, >= 41984, multiple of 16 */
    uint64_t main_layer_stride; /* bytes, >= num_pages*main_page_stride, multiple of 16 (L == 1: see below) */
    uint64_t idx_page_stride;   /* bytes, >= 8448, multiple of 16 */
    uint64_t idx_layer_stride;  /* bytes, >= num_pages*idx_page_stride, multiple of 16 (L == 1: see below) */
    uint32_t num_lanes;         /* fence lanes (one per overlapped micro-batch), 1..64 */
    uint32_t num_participants;  /* fence participants, 1..8; > 1 only with host-driven peers (tests) */
    uint64_t fence_timeout_ns;  /* 0 = 5 s */
    int32_t device;             /* HIP device ordinal */
    uint32_t flags;             /* 0 or KVPUB_CONFIG_FENCE_RELEASE_ONLY; other bits must be 0 */
} kvpub_config;

/* With L == 1 the layer strides address nothing and are not checked; a value
 * above num_pages * page stride states the span the layer may grow into
 * (kvpub_vmm_create sets it to the reserved range), which large stores use as
 * the bound of their write-through buffer range.  Any value is safe: no store
 * goes beyond the context's capacity. */

/* kvpub_config.flags: with one participant, kvpub_fence is by default the
 * system-scope release RMW of the lane's epoch followed by acquire loads of the
 * epoch until it holds the value the RMW produced (with one participant the
 * epoch is the only signal) -- the release/acquire pair of vLLM PR #52863,
 * Design (device-epoch barrier).  With this flag it is the release RMW alone:
 * no other agent publishes into this GPU's memory, and work after the fence
 * runs in later kernels, which the queue orders with its own acquire at
 * dispatch, so the acquire half has nothing to act on; it saves the system-
 * scope cache invalidation of the acquire.  No effect with peers: their fence
 * always acquire-waits. */
#define KVPUB_CONFIG_FENCE_RELEASE_ONLY 0x1u

/* Fill *cfg with defaults for R replicas of L layers of num_pages dense pages:
 * page strides 41984 / 8448, layer strides num_pages * page stride, one lane,
 * one participant, device 0. */
KVPUB_API void kvpub_config_init(kvpub_config *cfg, uint32_t num_replicas, uint32_t num_layers,
                       uint64_t num_pages);

/* Create a context over R caller-owned replica buffers.
 * main_bases[r] / idx_bases[r]: device pointers, 16-byte aligned, each at least
 * (L-1)*layer_stride + num_pages*page_stride bytes.  The caller keeps ownership
 * and must keep them alive until kvpub_destroy.  The context owns only its
 * device words (status flags and slot capacity, invalid-slot counter, epochs,
 * participant signals) on `device`.
 * All-or-nothing: on any failure every resource it made is released and *out
 * is set to NULL.  Returns KVPUB_ERR_UNSUPPORTED unless the device is gfx950. */
KVPUB_API kvpub_status kvpub_create(const kvpub_config *cfg, void *const *main_bases,
                          void *const *idx_bases, kvpub_ctx **out);

/* kvpub_create for callers that cannot allocate: code that must not call
 * hipMalloc or any other allocator (tight serving loops, harnesses that forbid
 * allocation).  Same configuration rules, bases and behaviour as kvpub_create,
 * and the context is used and destroyed the same way (kvpub_destroy), but this
 * call allocates nothing, host or device: the context's device words (status
 * and capacity, invalid-slot counter, one epoch per lane) live in a fixed
 * 8448-byte array of the library's, one per GPU, held until the process ends,
 * and its host part in static storage.  The words are cleared and the capacity
 * written by a kernel enqueued on `stream` (a hipStream_t; NULL = the null
 * stream): work on the context must follow it on that stream or after it.
 * Limits: one participant (peers' signals need host memory:
 * KVPUB_ERR_UNSUPPORTED), device ordinal < 64, and one static context per GPU
 * at a time -- a second call while one is alive returns KVPUB_ERR_IN_USE.
 * Every static context on a GPU uses that GPU's one array, so calls on it that
 * overlap (another thread creating a static context the moment this one is
 * destroyed, while kernels of the old one still run on another stream) race;
 * kvpub_destroy synchronizes the device first.  Not during stream capture of
 * `stream` (KVPUB_ERR_CAPTURING).  kvpub_graph_create on such a context
 * captures on a temporary stream (creating the graph allocates, as always). */
KVPUB_API kvpub_status kvpub_create_static(const kvpub_config *cfg, void *const *main_bases,
                                           void *const *idx_bases, kvpub_stream_t stream, kvpub_ctx **out);

/* Quantize num_tokens tokens' final rows and write them into every replica's
 * layer `layer`, asynchronously on `stream`.
 *   latent:  bf16 [T, 512], row stride latent_row_stride elements
 *   rope:    bf16 [T, 64],  row stride rope_row_stride elements
 *   indexer: bf16 [T, 128], row stride indexer_row_stride elements
 *   slot_mapping: int64 [T] device array (-1 = padded token)
 * Inputs are device pointers, 16-byte aligned, with row strides that are
 * multiples of 8 elements, at least the row width and at most 2^31 - 1
 * elements; slot_mapping is 8-byte aligned.  Valid slots within one call must be distinct and inputs finite.
 * num_tokens == 0 returns KVPUB_OK and launches nothing.  No allocation and no
 * synchronization: safe under stream capture.  Inputs must stay alive until
 * the stream work completes. */
KVPUB_API kvpub_status kvpub_store(kvpub_ctx *ctx, uint32_t layer, int64_t num_tokens,
                         const void *latent, int64_t latent_row_stride,
                         const void *rope, int64_t rope_row_stride,
                         const void *indexer, int64_t indexer_row_stride,
                         const int64_t *slot_mapping, kvpub_stream_t stream);

/* Dequantizing gather from replica `replica`, layer `layer`, asynchronously on
 * `stream` (the reader side of the cache this library writes).  For token t
 * with slot s = slot_mapping[t]:
 *   latent_out[t][k]  = bf16(RN32(value(code_k) * scale_(k/128))) for k < 512,
 *   rope_out[t][k]    = the stored RoPE bits, k < 64,
 *   indexer_out[t][k] = bf16(RN32(value(icode_k) * iscale)), k < 128,
 * where value() is the OCP E4M3 value of a stored code, the product is rounded
 * once to binary32 and then to bf16 (nearest, ties to even).  s == -1 or s
 * outside [0, num_pages*64) gives all-zero output rows; the out-of-range ones
 * are added to the context's invalid-slot counter (kvpub_error_read).
 *   latent_out:  bf16 [T, 512], row stride latent_row_stride elements
 *   rope_out:    bf16 [T, 64],  row stride rope_row_stride elements
 *   indexer_out: bf16 [T, 128], row stride indexer_row_stride elements
 *   slot_mapping: int64 [T] device array
 * Outputs are caller-owned device buffers, 16-byte aligned, row strides
 * multiples of 8 elements, at least the row width and at most 2^31 - 1
 * elements; slot_mapping is 8-byte aligned.  Only the output rows are written; the cache is only read.  A
 * context poisoned by a fence timeout still gathers (reading publishes
 * nothing).  num_tokens == 0 returns KVPUB_OK and launches nothing.  No
 * allocation and no synchronization: safe under stream capture.  Argument
 * problems (replica >= R, layer >= L, bad pointers or strides, or a context
 * with no backed pages -- see kvpub_vmm_grow) return KVPUB_ERR_INVALID_ARG
 * before anything is launched. */
KVPUB_API kvpub_status kvpub_gather(kvpub_ctx *ctx, uint32_t replica, uint32_t layer, int64_t num_tokens,
                                    const int64_t *slot_mapping, void *latent_out, int64_t latent_row_stride,
                                    void *rope_out, int64_t rope_row_stride, void *indexer_out,
                                    int64_t indexer_row_stride, kvpub_stream_t stream);

/* ---- Attention over the published cache ------------------------------------
 *
 * The rows of one replica's layer are the keys and the values of latent
 * attention in its absorbed form: for the row at position p of a sequence,
 *   c_p[k] = value(code_k) * scale_(k/128), k < 512, and r_p = its 64 RoPE values,
 * and for query token t and head h
 *   s(t,h,p) = scale * (q_latent[t,h] . c_p + q_rope[t,h] . r_p),
 *   lse[t,h] = ln sum_p exp(s(t,h,p)),  out[t,h] = sum_p exp(s(t,h,p) - lse[t,h]) c_p
 * over the positions that t sees; every head shares the position's one vector.
 * A query that sees nothing gives out = 0 and lse = -inf.  What a query does
 * not see has no effect on it, whatever its bytes hold (NaN codes, infinite
 * scales); a NaN or an infinity in a row that it does see leaves its output
 * row unspecified, NaN as a rule.  Scores, maxima, sums and outputs are held in binary32; the
 * weights are rounded to bf16 (times the row's tile scale) for the product
 * with the codes, and out once at the end.  Results do not depend on timing:
 * the same call on the same GPU gives the same bits.
 *
 * All pointers below are device pointers; descriptors are host structures that
 * are read during the call only.  No call here allocates or synchronizes: all
 * are safe under stream capture.  A context poisoned by a fence timeout still
 * attends (reading publishes nothing) but does not evict. */

/* Query tokens, bf16.  Element (t, h, k) is at t*token_stride + h*head_stride + k.
 * Pointers 16-byte aligned, strides multiples of 8 elements, at most 2^31 - 1;
 * head strides at least the row width (any value if num_heads is 1). */
typedef struct {
    const void *q_latent;             /* [T, H, 512] */
    const void *q_rope;               /* [T, H, 64] */
    int64_t q_latent_token_stride;
    int64_t q_latent_head_stride;
    int64_t q_rope_token_stride;
    int64_t q_rope_head_stride;
    int64_t num_tokens;               /* T, 0..2^24 */
    uint32_t num_heads;               /* H, 1..128 */
    float scale;                      /* finite; the softmax scale (not implied by any dimension) */
} kvpub_queries;

/* The cached positions of num_seqs sequences.  Position p of sequence b is row
 * p % 64 of page page_table[b*page_table_stride + p/64].  Sequence b's query
 * tokens are q_start[b] .. q_start[b+1]-1 (n of them); they are the newest
 * positions of the sequence, stored before the call: token i of n is position
 * kv_len[b] - n + i.
 *   tree_mask == NULL: token i sees positions 0 .. kv_len[b] - n + i.
 *   otherwise the n tokens are nodes of a drafted tree: token i sees every
 *   position below kv_len[b] - n, and of the drafted ones those node j with bit
 *   j % 64 of tree_mask[t*tree_words + j/64] set, t = q_start[b] + i (nodes
 *   beyond 64*tree_words are not seen).  A node sees itself only if its bit says so.
 * If kv_len[b] < n the first positions are negative and not there.
 * kv_len values are taken as at least 0 and at most max_kv_len; tokens
 * beyond the first max_q_len of a sequence, and tokens that belong to no
 * sequence, keep their output as it was.  A page number outside the context's
 * pages hides its 64 positions, and is counted once a call if some token would
 * have seen one of its tile's positions (kvpub_error_read's invalid count). */
typedef struct {
    const int32_t *kv_len;            /* [num_seqs] */
    const int32_t *q_start;           /* [num_seqs + 1], ascending; NULL: one token a sequence */
    const int32_t *page_table;        /* [num_seqs, >= ceil(max_kv_len / 64)] */
    int64_t page_table_stride;        /* elements, >= ceil(max_kv_len / 64) */
    const uint64_t *tree_mask;        /* [T, tree_words] or NULL */
    uint32_t tree_words;              /* 0 without a tree_mask, else 1..64 */
    uint32_t num_seqs;                /* 0..65536 */
    uint32_t max_q_len;               /* >= 1; most query tokens of one sequence */
    uint32_t max_kv_len;              /* most cached positions of one sequence, at most 2^30 */
} kvpub_pages;

/* Bytes of workspace that kvpub_attend / kvpub_attend_slots takes for such a
 * call (0 if the descriptor is not valid).  It depends on num_heads,
 * num_tokens, num_seqs, max_q_len, max_kv_len (num_slots) alone and grows with
 * each, so a program sizes it once for its largest call.  The workspace holds
 * the partial results of one call while that call runs, needs no
 * initialization and keeps nothing between calls; calls that may run at the
 * same time (other streams, captured graphs replayed side by side) each need
 * one of their own. */
KVPUB_API uint64_t kvpub_attend_workspace(const kvpub_queries *q, const kvpub_pages *pages);
KVPUB_API uint64_t kvpub_attend_slots_workspace(const kvpub_queries *q, uint32_t num_slots);

/* Latent attention of q over the sequences' cached positions in replica
 * `replica`, layer `layer`, asynchronously on `stream`.
 *   out: bf16, element (t,h,k) at t*out_token_stride + h*out_head_stride + k,
 *        512 values a row; alignment and stride rules as for the queries
 *   lse: binary32 (t,h) at t*lse_token_stride + h, or NULL; 4-byte aligned
 *   workspace: 16-byte aligned, workspace_bytes >= kvpub_attend_workspace(q, pages)
 * out, lse and the workspace overlap neither each other nor what the call reads.
 * num_seqs * ceil(max_q_len*num_heads / 64) * ceil(max_kv_len / 64) stays below
 * 2^31 (KVPUB_ERR_INVALID_ARG, as for every argument out of its range).
 * T == 0 or num_seqs == 0 launches nothing. */
KVPUB_API kvpub_status kvpub_attend(kvpub_ctx *ctx, uint32_t replica, uint32_t layer, const kvpub_queries *q,
                                    const kvpub_pages *pages, void *out, int64_t out_token_stride,
                                    int64_t out_head_stride, float *lse, int64_t lse_token_stride,
                                    void *workspace, uint64_t workspace_bytes, kvpub_stream_t stream);

/* kvpub_attend over a list of slots for each token, as a selection gives it:
 * token t sees the slots slots[t*slots_stride + i], i < num_slots.  -1 is
 * padding; any other slot outside [0, num_pages*64) is skipped and counted.  A
 * slot listed twice counts twice.  slots: int64, 8-byte aligned, num_slots
 * at most 2^24 (0: every out is 0), slots_stride >= num_slots. */
KVPUB_API kvpub_status kvpub_attend_slots(kvpub_ctx *ctx, uint32_t replica, uint32_t layer, const kvpub_queries *q,
                                          const int64_t *slots, int64_t slots_stride, uint32_t num_slots, void *out,
                                          int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                          int64_t lse_token_stride, void *workspace, uint64_t workspace_bytes,
                                          kvpub_stream_t stream);

/* The softmax weight that each cached position received from q, summed over
 * the sequence's tokens and heads, on top of what it had:
 *   weights_out[b][p] = weights_in[b][p] + sum_{t,h} exp(s(t,h,p) - lse[t,h])
 * for p < max_kv_len, the sum over the tokens that see p (0 for positions at
 * or beyond kv_len[b] and on bad pages).  weights_in NULL: zeros; weights_in ==
 * weights_out adds in place; otherwise the two do not overlap.  lse is what
 * kvpub_attend gave for the same queries and pages; a row of -inf adds nothing.
 *   weights: binary32 [num_seqs], row stride weights_stride >= max_kv_len elements;
 *            num_seqs * ceil(max_kv_len / 64) below 2^31
 * Without query tokens (T == 0) nothing but the weights is read.  The sums run in one fixed order (no atomics). */
KVPUB_API kvpub_status kvpub_attend_weights(kvpub_ctx *ctx, uint32_t replica, uint32_t layer, const kvpub_queries *q,
                                            const kvpub_pages *pages, const float *lse, int64_t lse_token_stride,
                                            const float *weights_in, float *weights_out, int64_t weights_stride,
                                            kvpub_stream_t stream);

/* One eviction: sequence b, of len = kv_len[b] positions (taken as 0 ..
 * max_kv_len), keeps min(len, budget) of them.  If len > budget those are the
 * first `first`, the last `last`, and of the rest the budget - first - last of
 * the largest accumulated weight; equal weights keep the lower position, a NaN
 * counts below every number.  In ascending order they become positions 0, 1, ..
 * of the destination table: the Main-KV row (656 bytes) and the Indexer-K row
 * (128 codes and their scale) of layer `layer` are read once, from replica 0,
 * and written to every replica.  The destination is the source table itself (in
 * place: dst_table == page_table with equal strides, and no page twice in it)
 * or pages that no source sequence of the call uses (a shared prefix stays
 * whole).
 *   kept[b][i]        = position that moved to i, -1 for new_len <= i < budget
 *   new_len[b]        = min(len, budget)
 *   weights_out[b][i] = weights_in[b][kept[b][i]] for i < new_len, 0 up to max_kv_len
 * weights_out may be weights_in itself, otherwise the two do not overlap;
 * new_len is not kv_len, and no other array of the call overlaps another.
 * A kept position whose source or destination page is outside the context's
 * pages is not copied, and counted.  The rows behind new_len keep their bytes. */
typedef struct {
    const float *weights_in;          /* [num_seqs], row stride weights_stride >= max_kv_len */
    float *weights_out;               /* the same shape and stride */
    int64_t weights_stride;
    const int32_t *kv_len;            /* [num_seqs] */
    const int32_t *page_table;        /* as in kvpub_pages */
    int64_t page_table_stride;
    const int32_t *dst_table;         /* [num_seqs, >= ceil(min(budget, max_kv_len) / 64)] */
    int64_t dst_table_stride;
    int32_t *kept;                    /* [num_seqs, budget], row stride kept_stride >= budget */
    int64_t kept_stride;
    int32_t *new_len;                 /* [num_seqs] */
    uint32_t num_seqs;                /* 0..65536 */
    uint32_t max_kv_len;              /* 1..2^30 */
    uint32_t budget;                  /* 1..2^30 */
    uint32_t first;                   /* first + last <= budget */
    uint32_t last;
    uint32_t reserved;                /* must be 0 */
} kvpub_evict_io;

/* Bytes of workspace of an eviction; rules as for kvpub_attend_workspace. */
KVPUB_API uint64_t kvpub_evict_workspace(const kvpub_evict_io *io);

/* Evict asynchronously on `stream`.  weights, tables, kept and lengths are
 * 4-byte aligned, the workspace 16-byte.  A poisoned context changes nothing;
 * if it is poisoned while the call runs, each sequence is evicted whole (rows,
 * weights, kept and new_len) or left as it was. */
KVPUB_API kvpub_status kvpub_evict(kvpub_ctx *ctx, uint32_t layer, const kvpub_evict_io *io, void *workspace,
                                   uint64_t workspace_bytes, kvpub_stream_t stream);

/* Latent attention in its expanded form, for prefill: the latent vectors of the
 * keys (kvpub_gather) have been projected up to a key part and a value for each
 * head, and the 64 RoPE values stay shared:
 *   s(t,h,u) = scale * (q_nope[t,h] . k_nope[u,h] + q_rope[t,h] . k_rope[u]),
 *   out[t,h] = sum_u softmax_u(s(t,h,u)) v[u,h]
 * Sequence b's tokens are q_start[b] .. q_start[b+1]-1 (n) and its keys
 * k_start[b] .. k_start[b+1]-1 (m).  causal: token i sees keys 0 .. m - n + i,
 * else all m.  No key seen: out 0, lse -inf.  All bf16, accumulated in
 * binary32; the weights are rounded to bf16 for the product with v.  Keys and
 * values that a token does not see have no effect on it; one that is not finite
 * leaves the rows that see it unspecified.  16-byte
 * aligned, strides multiples of 8 elements and at most 2^31 - 1, as for
 * kvpub_queries.  Values and key parts may be interleaved (strides of 256 a head).
 * The context gives the device only. */
typedef struct {
    const void *q_nope;               /* [T, H, 128] */
    const void *q_rope;               /* [T, H, 64] */
    const void *k_nope;               /* [U, H, 128] */
    const void *k_rope;               /* [U, 64] */
    const void *v;                    /* [U, H, 128] */
    void *out;                        /* [T, H, 128] */
    float *lse;                       /* [T, H] at t*lse_token_stride + h, or NULL */
    int64_t q_nope_token_stride, q_nope_head_stride;
    int64_t q_rope_token_stride, q_rope_head_stride;
    int64_t k_nope_token_stride, k_nope_head_stride;
    int64_t k_rope_token_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t lse_token_stride;
    const int32_t *q_start;           /* [num_seqs + 1], ascending */
    const int32_t *k_start;           /* [num_seqs + 1], ascending */
    int64_t num_tokens;               /* T, 0..2^24 */
    int64_t num_keys;                 /* U, 0..2^24 */
    uint32_t num_seqs;                /* 0..65535 */
    uint32_t num_heads;               /* 1..128 */
    uint32_t max_q_len;               /* >= 1; tokens beyond the first max_q_len of a sequence keep their output */
    uint32_t causal;                  /* 0 or 1 */
    float scale;
    uint32_t reserved;                /* must be 0 */
} kvpub_expanded_io;

KVPUB_API kvpub_status kvpub_attend_expanded(kvpub_ctx *ctx, const kvpub_expanded_io *io, kvpub_stream_t stream);

/* ---- Rotary positions --------------------------------------------------------
 *
 * A rotation turns pairs of a row's values by angles that go by the token's
 * position: pair i by a = 2 pi frac(position * turns[i] / 2^64),
 *   y1 = magnitude * (x1 cos a - x2 sin a),  y2 = magnitude * (x1 sin a + x2 cos a).
 * The frequencies are a table of turns a position in units of 2^-64, so that an
 * angle is one 64-bit product whatever the position: far ones lose nothing.
 * Angles are rounded to 2^-32 of a turn, sines, cosines and products are binary32.
 * Positions are int32 and may be negative (they turn back). */
#define KVPUB_ROTATE_PAIRS 0u   /* pair i: values start + 2i and start + 2i + 1 */
#define KVPUB_ROTATE_HALVES 1u  /* pair i: values start + i and start + dim/2 + i */

typedef struct {
    const uint64_t *turns;            /* device, [dim / 2], 8-byte aligned */
    uint32_t dim;                     /* rotated values of a row: a multiple of 8, at least 8 */
    uint32_t start;                   /* the first of them: a multiple of 8; start + dim at most the row's width */
    uint32_t layout;                  /* KVPUB_ROTATE_* */
    float magnitude;                  /* of the rotated values; finite, 1 where a scaling asks for nothing else */
} kvpub_rotation;

/* How a model's frequencies f_i = base^(-2i/dim) (radians a position) are
 * stretched for contexts longer than those it was trained on:
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   GROWN   f_i of the base grown to base * factor^(dim / (dim - 2))
 *   RAMP    f_i k_i + f_i / factor * (1 - k_i), k_i = 1 - clamp((i - lo) / (hi - lo), 0, 1)
 *           with lo = max(0, floor(d(high))), hi = min(dim - 1, ceil(d(low))) (hi - lo at least 0.001),
 *           d(t) = dim * ln(original / (2 pi t)) / (2 ln base): by the pair's index between those
 *           that turn `high` and `low` times over the original length
 *   BLEND   the same with k_i = clamp((original * f_i / (2 pi) - low) / (high - low), 0, 1): by the turns */
#define KVPUB_SCALING_NONE 0u
#define KVPUB_SCALING_LINEAR 1u
#define KVPUB_SCALING_GROWN 2u
#define KVPUB_SCALING_RAMP 3u
#define KVPUB_SCALING_BLEND 4u

typedef struct {
    uint32_t dim;                     /* a multiple of 8, 8..1024 */
    uint32_t scaling;                 /* KVPUB_SCALING_* */
    double base;                      /* finite, > 1 */
    double factor;                    /* finite, >= 1 (not read by NONE) */
    double original;                  /* positions of the original context, >= 1 (RAMP, BLEND) */
    double low;                       /* turns over it, 0 < low < high, finite (RAMP, BLEND) */
    double high;
} kvpub_rotation_config;

/* Fill turns[0 .. dim/2 - 1], a host array, for the caller to copy to the
 * device once.  Host arithmetic only: needs no device. */
KVPUB_API kvpub_status kvpub_rotation_turns(const kvpub_rotation_config *config, uint64_t *turns);

/* Element types of the calls below. */
#define KVPUB_BF16 0u
#define KVPUB_FP16 1u
#define KVPUB_FP32 2u

/* Rows of heads rotated by their tokens' positions: y = the rotation of x, the
 * values outside [start, start + dim) copied.  y == x with equal strides rotates in
 * place (only the rotated values are touched); otherwise the two do not overlap.
 * transpose: by the negative angles (times the same magnitude), which takes the
 * gradient of y to the gradient of x.  Rounded once, to the element type.
 * Element (t, h, k) is at t*token_stride + h*head_stride + k; pointers 16-byte
 * aligned, strides multiples of 8 elements, at most 2^31 - 1, head strides at
 * least head_dim (any value if num_heads is 1); x's token stride may be 0.
 * A value that is not finite reaches its own pair only. */
typedef struct {
    const void *x;                    /* [T, H, head_dim] */
    void *y;                          /* [T, H, head_dim] */
    int64_t x_token_stride, x_head_stride;
    int64_t y_token_stride, y_head_stride;
    const int32_t *positions;         /* [T], 4-byte aligned */
    kvpub_rotation rotation;
    int64_t num_tokens;               /* 0..2^24 */
    uint32_t num_heads;               /* 1..1024 */
    uint32_t head_dim;                /* a multiple of 8, 8..1024 */
    uint32_t type;                    /* KVPUB_BF16, KVPUB_FP16 or KVPUB_FP32 */
    uint32_t transpose;               /* 0 or 1 */
} kvpub_rotate_io;

/* Asynchronously on `stream`; no allocation, no synchronization, safe under
 * stream capture.  The context gives the device only. */
KVPUB_API kvpub_status kvpub_rotate(kvpub_ctx *ctx, const kvpub_rotate_io *io, kvpub_stream_t stream);

/* kvpub_store with the rotation applied on the way: token t's RoPE row and its
 * Indexer-K row are rotated by positions[t] before they are stored (a NULL
 * rotation leaves that row as it is; both NULL is kvpub_store, and `positions`
 * is not read).  The RoPE values are rounded to bf16 once; the Indexer-K values are
 * not rounded before their scale and codes: scale = RN32(amax / 448), code =
 * e4m3fn(RN32(x / scale)) of the rotated binary32 values.  If the context is
 * poisoned while the call runs, each token's two rows are stored whole, in every
 * replica, or left as they were.  Everything else, arguments and slots included, is
 * as for kvpub_store. */
KVPUB_API kvpub_status kvpub_store_rotated(kvpub_ctx *ctx, uint32_t layer, int64_t num_tokens,
                                           const void *latent, int64_t latent_row_stride,
                                           const void *rope, int64_t rope_row_stride,
                                           const void *indexer, int64_t indexer_row_stride,
                                           const int64_t *slot_mapping, const int32_t *positions,
                                           const kvpub_rotation *rope_rotation,
                                           const kvpub_rotation *indexer_rotation, kvpub_stream_t stream);

/* ---- A cache of key and value heads ------------------------------------------
 *
 * For attention that keeps keys and values of several heads instead of one
 * latent vector: a replicated paged cache of e4m3 codes with one scale for each
 * block of 64 tokens (a page) and head, keys and values apart.
 * A page of one layer, G heads of D values, at
 * replica + layer*layer_stride + page*page_stride:
 *   head g at g*128*D:  [64][D] codes of the keys, then [64][D] codes of the values
 *   behind all heads, at G*128*D + 2*g: the scale byte of the keys, then of the values
 * A byte b stands for 2^(b - 127), b taken as 1..245.  A stored value is code * scale.
 * A power of two costs a floating code no precision, and lets a block that is
 * partly filled take a larger scale later without rounding its codes again
 * (but for those that become subnormal).
 *
 * The context gives the device, the fail-closed state of its fences and the
 * counter of bad pages; the descriptor names the memory, which is the caller's.
 * A program without a latent cache makes its context over one page of that, which
 * the calls below do not touch: kvpub_config_init(&cfg, 1, 1, 1) and device
 * allocations of KVPUB_MAIN_PAGE_BYTES and KVPUB_IDX_PAGE_BYTES as its two bases. */
#define KVPUB_HEADS_PAGE_BYTES(num_kv_heads, head_dim) \
    (((uint64_t)(num_kv_heads) * (128u * (uint64_t)(head_dim) + 2u) + 15u) / 16u * 16u)

typedef struct {
    void *bases[KVPUB_MAX_REPLICAS];  /* device, 16-byte aligned; num_replicas of them are read */
    uint64_t num_pages;               /* pages of a layer, 1..2^31 - 1 */
    uint64_t page_stride;             /* bytes, >= KVPUB_HEADS_PAGE_BYTES, multiple of 16 */
    uint64_t layer_stride;            /* bytes, >= num_pages*page_stride, multiple of 16 (one layer: not read) */
    uint32_t num_replicas;            /* 1..8 */
    uint32_t num_layers;              /* >= 1 */
    uint32_t num_kv_heads;            /* G, 1..128 */
    uint32_t head_dim;                /* D: 64, 128 or 256 */
} kvpub_heads;

/* New keys and values.  Element (t, g, k) is at t*token_stride + g*head_stride + k;
 * alignment and strides as for kvpub_rotate_io's x. */
typedef struct {
    const void *k;                    /* [T, G, D] */
    const void *v;                    /* [T, G, D] */
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t num_tokens;               /* T, 0..2^24 */
    uint32_t type;                    /* KVPUB_BF16 or KVPUB_FP16 */
    uint32_t reserved;                /* must be 0 */
} kvpub_heads_rows;

/* Append: token i of sequence b's n (q_start as in kvpub_pages) becomes its
 * position p = kv_len[b] - n + i, in every replica; kv_len counts the new tokens.
 * The key is rotated first, by positions[t], or by p if positions is NULL; a NULL
 * rotation leaves keys as they are (positions is not read).  Rotated values are
 * not rounded before their codes.
 * A block's scale is the least 2^e, -126 <= e <= 118, with every finite |x| of its
 * new tokens at most 448 * 2^e, and, if it holds older positions of the sequence,
 * at least the scale it had (replica 0's): those are brought to the new scale,
 * code = e4m3fn(old value / scale).  Magnitudes beyond 448 scales (infinities
 * among them) become +-448, a NaN becomes a NaN code.
 * Rows of the pages that hold neither older positions nor new ones keep their
 * bytes, and so do the older ones if the scale stays.  A page that gets rows belongs
 * to one sequence of the call (a shared prefix ends on a page's end).  tree_mask
 * is not read; tokens beyond the first max_q_len of a sequence, negative
 * positions, and tokens that belong to no sequence are not stored.  A page
 * number outside the cache's pages drops its rows, and is counted once a call.
 * A context poisoned by a fence timeout stores nothing; if it is poisoned while
 * the call runs, each block of 64 positions and head is stored whole, in every
 * replica, or left as it was.  Asynchronous on `stream`; no allocation, no
 * synchronization, safe under stream capture. */
KVPUB_API kvpub_status kvpub_heads_append(kvpub_ctx *ctx, const kvpub_heads *cache, uint32_t layer,
                                          const kvpub_heads_rows *rows, const kvpub_pages *pages,
                                          const kvpub_rotation *rotation, const int32_t *positions,
                                          kvpub_stream_t stream);

/* Queries of H heads over the cache's G: head h reads key-value head h / (H/G). */
typedef struct {
    const void *q;                    /* [T, H, D] */
    void *out;                        /* [T, H, D], of q's type */
    float *lse;                       /* [T, H] at t*lse_token_stride + h, or NULL; 4-byte aligned */
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t lse_token_stride;
    int64_t num_tokens;               /* T, 0..2^24 */
    uint32_t num_heads;               /* H: a multiple of G, at most 128 * G and 1024 */
    uint32_t type;                    /* KVPUB_BF16 or KVPUB_FP16 */
    float scale;                      /* finite; the softmax scale */
    uint32_t reserved;                /* must be 0 */
} kvpub_heads_queries;

/* Bytes of workspace that kvpub_heads_attend takes for such a call (0 if a
 * descriptor is not valid).  It depends on num_kv_heads, head_dim, num_heads,
 * num_tokens, num_seqs, max_q_len and max_kv_len alone and grows with each; rules as
 * for kvpub_attend_workspace. */
KVPUB_API uint64_t kvpub_heads_attend_workspace(const kvpub_heads *cache, const kvpub_heads_queries *q,
                                                const kvpub_pages *pages);

/* Attention over the sequences' cached positions in replica `replica`, layer `layer`:
 *   s(t,h,p) = scale * (q[t,h] . k[p,g]),  lse[t,h] = ln sum_p exp(s(t,h,p)),
 *   out[t,h] = sum_p exp(s(t,h,p) - lse[t,h]) v[p,g],  g = h / (H/G)
 * over the positions that t sees (kvpub_pages: causal, or a drafted tree).
 * What is said of kvpub_attend holds here: a query that sees nothing gives 0
 * and -inf, what it does not see has no effect whatever its bytes hold, bad pages
 * hide their positions and are counted, tokens of no sequence keep their output,
 * the same call gives the same bits.  Scores, maxima and sums are binary32;
 * weights are rounded to bf16 for the second product (FP16, and calls of at most 16
 * (token, query head) rows a sequence and key-value head: to the sum of two bf16), out once
 * to its type.  A query or a seen row that is not finite, a score whose
 * magnitude passes 2^30, or a value whose magnitude passes 2^88 (the sums are of weights up to 2^8 before they are
 * divided) leaves the rows it reaches unspecified, NaN as a rule.
 * T == 0 or num_seqs == 0 launches nothing. */
KVPUB_API kvpub_status kvpub_heads_attend(kvpub_ctx *ctx, const kvpub_heads *cache, uint32_t replica, uint32_t layer,
                                          const kvpub_heads_queries *q, const kvpub_pages *pages, void *workspace,
                                          uint64_t workspace_bytes, kvpub_stream_t stream);

/* Replica storage at stable virtual addresses, on cfg->device (vLLM PR
 * #52863, Relationship to existing work: the replicated cache builds on a
 * cache kept at a stable virtual address so that it can grow in place).
 * Reserves address space for cfg->num_replicas replicas of cfg->num_layers
 * layers of up to max_pages pages each (one Main-KV and one Indexer-K range
 * per replica) and backs the first cfg->num_pages pages of every layer with
 * device memory (contents undefined until written).  On success the layer
 * strides in *cfg are set to the reserved per-layer spans (max_pages * page
 * stride rounded up to the allocation granularity, plus one granule; every
 * layer is a reservation of its own), main_bases[r] /
 * idx_bases[r] receive the replicas' base addresses, and *cfg is ready for
 * kvpub_create.  The bases never change for the object's lifetime.
 * All-or-nothing: on failure nothing stays reserved or mapped and *out is
 * NULL.  Only backed pages may be accessed: a context over this storage must
 * not claim more pages than are backed (kvpub_vmm_grow keeps them equal). */
KVPUB_API kvpub_status kvpub_vmm_create(kvpub_config *cfg, uint64_t max_pages, void **main_bases,
                                        void **idx_bases, kvpub_vmm **out);

/* Back every layer of every replica up to num_pages pages (num_pages <=
 * max_pages; never shrinks).  Bytes already written and all addresses are
 * unchanged.  If ctx is not NULL it must be a context over exactly this
 * storage (same bases and strides, else KVPUB_ERR_INVALID_ARG); its capacity
 * becomes the backed page count, for launches made after the call and for
 * graphs captured before it alike (the kernels read the capacity from the
 * context's device words when they run).  Host-side, not
 * for use during stream capture or concurrently with launches on ctx from
 * another thread.  On failure the page count stays as it was, except in the
 * unlikely case that a layer's old backing could not be restored either:
 * then the storage reports 0 pages, ctx (if given) accepts no slot any more
 * (stores count every slot as invalid, new gathers are refused and gathers
 * captured earlier write zero rows), and
 * KVPUB_ERR_HIP is returned.  Growing copies each layer's backed bytes
 * once (the addresses stay, the physical memory behind them is replaced). */
KVPUB_API kvpub_status kvpub_vmm_grow(kvpub_vmm *vmm, uint64_t num_pages, kvpub_ctx *ctx);

/* Pages per layer currently backed. */
KVPUB_API kvpub_status kvpub_vmm_pages(kvpub_vmm *vmm, uint64_t *num_pages);

/* Synchronize the device, then unmap and release everything.  Contexts over
 * this storage must be destroyed first. */
KVPUB_API kvpub_status kvpub_vmm_destroy(kvpub_vmm *vmm);

/* One fence on `lane`, asynchronously on `stream`: a single one-wavefront
 * kernel that adds 1 to the lane's device epoch with a system-scope
 * read-modify-write that releases every write made on this GPU before the
 * fence.  With one participant it then acquire-loads the epoch until it holds
 * the new value (KVPUB_CONFIG_FENCE_RELEASE_ONLY: the release RMW alone).
 * With peers the RMW also acquires, then the kernel publishes the new value as
 * this participant's signal and acquire-waits until every other participant's
 * signal has reached it.  The expected value is never a kernel argument, so a captured
 * fence advances the epoch on every replay.  If the wait exceeds
 * fence_timeout_ns the kernel records KVPUB_FLAG_FENCE_TIMEOUT |
 * KVPUB_FLAG_POISONED and returns; from then on stores and fences of this
 * context write nothing (fail-closed; with one participant the wait can only
 * time out if the epoch was moved back, by kvpub_fence_host_epoch on the same
 * lane).
 * No allocation and no synchronization: safe under stream capture. */
KVPUB_API kvpub_status kvpub_fence(kvpub_ctx *ctx, uint32_t lane, kvpub_stream_t stream);

/* The pages' earlier fence, kept for comparison: two launches per fence and an
 * epoch held on the host (vLLM PR #54030 "[Perf][PCP] Fuse direct-KV
 * publication fence", Motivation and commit list: the fence used to be a
 * signal launch and a wait launch, and because the epoch lived on the host a
 * captured graph could not advance it on replay).  The context keeps a host
 * counter per lane; each call takes e = counter + 1 and enqueues on `stream` a
 * kernel that release-stores e into the lane's device epoch at system scope,
 * then a kernel that acquire-loads it until it is >= e (bounded by
 * fence_timeout_ns; a timeout sets KVPUB_FLAG_FENCE_TIMEOUT |
 * KVPUB_FLAG_POISONED), and the counter becomes e.  Under stream capture the
 * counter moves once, at capture: every replay publishes the captured values
 * again, so the device epoch stops advancing -- the failure the single-launch
 * kvpub_fence removes.  kvpub_epoch_read shows the published value.  Do not
 * mix it with kvpub_fence on one lane (the two count independently).  One
 * participant only (KVPUB_ERR_UNSUPPORTED otherwise).  No allocation and no
 * synchronization; the counter is not thread-safe. */
KVPUB_API kvpub_status kvpub_fence_host_epoch(kvpub_ctx *ctx, uint32_t lane, kvpub_stream_t stream);

/* One layer of a captured sequence. */
typedef struct {
    const void *latent;
    const void *rope;
    const void *indexer;
    int64_t latent_row_stride;
    int64_t rope_row_stride;
    int64_t indexer_row_stride;
    const int64_t *slot_mapping;
    int64_t num_tokens;
    uint32_t layer;
    uint32_t reserved; /* must be 0 */
} kvpub_layer_io;

/* Capture n x (kvpub_store(io[i]), kvpub_fence(lane)) once into a hipGraph
 * (on a private stream) and instantiate it.  The graph binds the pointers in
 * io: to publish new data, rewrite those buffers before a replay.  They must
 * outlive the graph.  Argument checks as for kvpub_store, done for every layer
 * before capture begins.  Captures on the context's private stream: create
 * graphs of one context from one thread at a time. */
KVPUB_API kvpub_status kvpub_graph_create(kvpub_ctx *ctx, const kvpub_layer_io *io, uint32_t n,
                                uint32_t lane, kvpub_graph **out);

/* Launch the instantiated graph once on `stream` (asynchronous). */
KVPUB_API kvpub_status kvpub_graph_replay(kvpub_graph *graph, kvpub_stream_t stream);

/* Release a graph (waits for nothing; do not destroy while a replay may run). */
KVPUB_API kvpub_status kvpub_graph_destroy(kvpub_graph *graph);

/* Synchronize the device, then read the lane's epoch (number of fences that
 * ran on it).  KVPUB_ERR_CAPTURING if a capture is active on the calling thread. */
KVPUB_API kvpub_status kvpub_epoch_read(kvpub_ctx *ctx, uint32_t lane, uint64_t *out);

/* Synchronize the device, then read the invalid-slot count and the sticky
 * flags (either output may be NULL).  clear != 0 resets the invalid-slot
 * count; the flags stay set for the context's lifetime.  Returns
 * KVPUB_ERR_FENCE_TIMEOUT if KVPUB_FLAG_FENCE_TIMEOUT is set, else KVPUB_OK. */
KVPUB_API kvpub_status kvpub_error_read(kvpub_ctx *ctx, uint64_t *invalid_slots, uint32_t *flags,
                              int clear);

/* Host address of participant p's signal word on `lane` (1 <= p <
 * num_participants).  It lives in host-coherent memory that the fence kernel
 * reads with system-scope acquire loads; a host thread stands in for peer p by
 * storing the epoch values it publishes.  Only meaningful with
 * num_participants > 1 (one GPU has no real peers). */
KVPUB_API kvpub_status kvpub_participant_signal(kvpub_ctx *ctx, uint32_t lane, uint32_t p,
                                      volatile uint64_t **out);

/* Synchronize the device and release the context's resources.  NULL is OK.
 * The replica buffers are the caller's and are left untouched. */
KVPUB_API kvpub_status kvpub_destroy(kvpub_ctx *ctx);

/* Static description of a status code. */
KVPUB_API const char *kvpub_strerror(kvpub_status status);

/* KVPUB_ABI_VERSION of the loaded library. */
KVPUB_API uint32_t kvpub_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVPUB_H */
