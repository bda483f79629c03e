// Internal interface between the C-ABI host code and the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct kvpub_ctx;

namespace kvpub {

constexpr int kMaxReplicas = 8;
constexpr int kTokensPerWave = 4;     // 4 tokens x 5 tiles = 5 rounds of 4 tiles per wave
constexpr int kWavesPerBlock = 4;     // 256 threads, 16 tokens per block (1, 2 and 8 measured: no better)
constexpr int kTokensPerBlock = kTokensPerWave * kWavesPerBlock;
constexpr int64_t kMaxTokensPerLaunch = int64_t(1) << 24;   // larger batches take several launches

constexpr uint32_t kStatusFenceTimeout = 0x1u;
constexpr uint32_t kStatusPoisoned = 0x2u;

// Words of a context that live in device memory, each on its own 128-byte line.
constexpr size_t kLine = 128;
constexpr size_t kStatusOffset = 0;          // the CtxHead line
constexpr size_t kInvalidOffset = kLine;
constexpr size_t kEpochOffset = 2 * kLine;          // + lane * kLine
constexpr size_t kSignalStride = kLine / 8;         // uint64 words between participant signals

// The first line of a context's device words: the status flags (set by a
// fence that timed out) and the number of slots per layer that may be written
// (set by the host at creation and when a VMM storage grows).  Kernels read
// both with one scalar load at launch time, so a captured graph sees a
// capacity raised after its capture.
struct CtxHead {
    uint32_t status;
    uint32_t reserved;
    int64_t capacity;            // num_pages * 64
};
static_assert(sizeof(CtxHead) == 16, "one 16-byte scalar load");

struct StoreParams {
    const uint16_t* latent;      // bf16 bit patterns
    const uint16_t* rope;
    const uint16_t* indexer;
    int64_t latent_stride;       // elements
    int64_t rope_stride;
    int64_t indexer_stride;
    const int64_t* slots;
    int64_t num_tokens;
    uint64_t main_page_stride;   // bytes
    uint64_t idx_page_stride;
    uint8_t* main_base[kMaxReplicas];  // replica r, already offset to the layer
    uint8_t* idx_base[kMaxReplicas];
    unsigned long long* invalid_count;
    const CtxHead* head;         // status and capacity
    uint32_t main_region;        // bytes of one replica's layer span (all the pages it may ever hold)
    uint32_t idx_region;         // if below 2^32, else 0: the write-through path needs 32-bit offsets
};

struct FenceParams {
    uint64_t* epoch;             // this lane's epoch word
    uint64_t* signals;           // this lane's participant signals, kSignalStride apart (null alone)
    uint32_t num_participants;
    uint32_t self;               // this GPU's participant index (0)
    uint32_t* status;
    uint64_t timeout_ticks;      // in wall-clock (s_memrealtime) ticks
    uint32_t acquire_wait;       // alone: acquire-wait on the epoch after the release RMW (else release only)
};

// Enqueue one store kernel on `stream`; returns the launch status.
hipError_t launch_store(const StoreParams& p, uint32_t num_replicas, hipStream_t stream);
struct GatherParams {
    const uint8_t* main_base;    // the replica, already offset to the layer
    const uint8_t* idx_base;
    uint64_t main_page_stride;   // bytes
    uint64_t idx_page_stride;
    const CtxHead* head;         // capacity (num_pages * 64)
    const int64_t* slots;
    int64_t num_tokens;
    uint16_t* latent;            // bf16 outputs
    uint16_t* rope;
    uint16_t* indexer;
    int64_t latent_stride;       // elements
    int64_t rope_stride;
    int64_t indexer_stride;
    unsigned long long* invalid_count;
    uint32_t offsets32;          // every offset within a layer fits in 32 bits (layer span < 2^32)
};

// The unit that a block began and later ones end: their parts are joined.
struct AttendCut {
    uint32_t slot;               // of this block's part; the others' are their first
    uint32_t q0;                 // first token of the unit's sequence
    uint32_t row0;               // the unit's first (token, head) row of the sequence
    uint32_t rows;               // of the sequence
};

// Latent attention (attend_kernel.hip).  Strides in elements.
struct AttendParams {
    const uint8_t* main_base;    // the replica, already offset to the layer
    uint64_t main_page_stride;   // bytes
    const CtxHead* head;         // capacity (num_pages * 64)
    unsigned long long* invalid_count;
    const uint16_t* q_latent;    // bf16
    const uint16_t* q_rope;
    int64_t q_latent_token, q_latent_head, q_rope_token, q_rope_head;
    uint32_t num_tokens;
    uint32_t heads;
    uint32_t num_seqs;           // slot lists: one for each token
    uint32_t max_q;              // slot lists: 1
    uint32_t max_kv;
    uint32_t num_slots;
    const int32_t* kv_len;
    const int32_t* q_start;      // null: one token a sequence
    const int32_t* pages;
    int64_t pages_stride;
    const uint64_t* tree;        // null: causal
    uint32_t tree_words;
    float scale_log2;            // scale * log2(e)
    uint32_t by_slots;           // 1: slot lists, else pages
    const int64_t* slots;
    int64_t slots_stride;
    uint16_t* out;               // bf16
    int64_t out_token, out_head;
    float* lse;                  // null: not written (attend); the given sums (weights)
    int64_t lse_token;
    const float* weights_in;     // weights only
    float* weights_out;
    int64_t weights_stride;
    uint32_t* cut_last;          // workspace: [blocks] last block of the unit that this one began; 0: none was cut
    AttendCut* cuts;             // workspace: [blocks] that unit, if it was cut
    float* part_lse;             // workspace: [blocks * 2][rows]
    float* part;                 // workspace: [blocks * 2][rows][512]
};

// How a call is cut: query rows of a unit, blocks, and the workspace's parts.
struct AttendPlan {
    uint32_t rows;
    uint32_t blocks;
    uint32_t joins;              // blocks of the join
    bool fits;                   // fewer than 2^31 tiles in all
    uint64_t lse_bytes;
    uint64_t bytes;
};
// rows: the most (token, head) rows of one sequence.
AttendPlan plan_attend(uint64_t rows, uint64_t num_seqs, uint64_t num_tokens, uint64_t heads, uint64_t max_kv);
// Enqueue latent attention on `stream`; returns the launch status.
hipError_t launch_attend(const AttendParams& p, void* workspace, hipStream_t stream);
hipError_t launch_attend_weights(const AttendParams& p, hipStream_t stream);

// Eviction (evict_kernel.hip).
struct EvictParams {
    uint8_t* main_base[kMaxReplicas];   // replica r, already offset to the layer
    uint8_t* idx_base[kMaxReplicas];
    uint64_t main_page_stride;   // bytes
    uint64_t idx_page_stride;
    uint32_t replicas;
    const CtxHead* head;         // status and capacity
    unsigned long long* invalid_count;
    const float* weights_in;
    float* weights_out;
    int64_t weights_stride;
    const int32_t* kv_len;
    const int32_t* pages;
    int64_t pages_stride;
    const int32_t* dst;
    int64_t dst_stride;
    int32_t* kept;
    int64_t kept_stride;
    int32_t* new_len;
    uint32_t num_seqs;
    uint32_t max_kv;
    uint32_t budget;
    uint32_t first;
    uint32_t last;
    uint32_t same_pages;         // dst is pages: rows are moved within the table
    uint32_t chunks;             // set by launch_evict: ceil(max_kv / 64)
    uint32_t* state;             // workspace: each sequence's ticket, flags[chunks], ranks[chunks + 1]
};
hipError_t launch_evict(const EvictParams& p, hipStream_t stream);

// Latent attention in its expanded form (expanded_kernel.hip).  Strides in elements.
struct ExpandedParams {
    const uint16_t* q_nope;
    const uint16_t* q_rope;
    const uint16_t* k_nope;
    const uint16_t* k_rope;
    const uint16_t* v;
    uint16_t* out;
    float* lse;                  // null: not written
    int64_t q_nope_token, q_nope_head, q_rope_token, q_rope_head;
    int64_t k_nope_token, k_nope_head, k_rope_token, v_token, v_head;
    int64_t out_token, out_head, lse_token;
    const int32_t* q_start;
    const int32_t* k_start;
    uint32_t num_tokens;
    uint32_t num_keys;
    uint32_t num_seqs;
    uint32_t heads;
    uint32_t max_q;
    uint32_t causal;
    float scale_log2;
    uint32_t first_seq;          // set by launch_expanded
    uint32_t first_tile;
};
hipError_t launch_expanded(const ExpandedParams& p, hipStream_t stream);

// A rotation by positions (rotation.h); dim == 0: none.
struct RotationParams {
    const uint64_t* turns;
    uint32_t dim;
    uint32_t start;
    uint32_t halves;
    float magnitude;
};

// Rows of heads rotated (rotate_kernel.hip).  Strides in elements.
struct RotateParams {
    const void* x;
    void* y;
    int64_t x_token, x_head, y_token, y_head;
    const int32_t* positions;
    RotationParams rotation;
    uint32_t num_tokens;
    uint32_t heads;
    uint32_t units;              // groups of 8 values of a row that the call touches: the rotated ones, then the copied ones
    uint32_t type;               // KVPUB_BF16, KVPUB_FP16, KVPUB_FP32
    uint32_t across;             // set by launch_rotate: heads that a block takes beside each other
    uint32_t tokens;             // and tokens
    float sign;                  // the magnitude, negative for the transpose
};
hipError_t launch_rotate(const RotateParams& p, hipStream_t stream);

// The latent cache's store with rotations (store_rotated_kernel.hip).
struct StoreRotatedParams {
    StoreParams s;
    const int32_t* positions;
    RotationParams rope;
    RotationParams indexer;
    uint32_t replicas;
};
hipError_t launch_store_rotated(const StoreRotatedParams& p, hipStream_t stream);

// The cache of key and value heads: one replica's layer.
struct HeadsParams {
    uint64_t page_stride;        // bytes
    int64_t num_pages;
    uint32_t groups;             // key-value heads
    uint32_t dim;                // values of a head
};

// The sequences of a call on it (kvpub_pages).
struct SeqParams {
    const int32_t* kv_len;
    const int32_t* q_start;      // null: one token a sequence
    const int32_t* pages;
    int64_t pages_stride;
    uint32_t num_seqs;
    uint32_t num_tokens;
    uint32_t max_q;
    uint32_t max_kv;
};

// Appending to it (heads_append_kernel.hip).
struct HeadsAppendParams {
    HeadsParams heads;
    SeqParams seqs;
    uint8_t* base[kMaxReplicas]; // replica r, already offset to the layer
    uint32_t replicas;
    uint32_t type;               // KVPUB_BF16 or KVPUB_FP16
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_token, k_head, v_token, v_head;
    const int32_t* positions;    // null: the positions in the sequence
    RotationParams rotation;
    const CtxHead* head;         // status
    unsigned long long* invalid_count;
    uint32_t first;              // set by launch_heads_append: the launch's first place
    uint32_t stream;             // and whether codes are stored past the L2s
};
hipError_t launch_heads_append(const HeadsAppendParams& p, hipStream_t stream);

// Attention over it (heads_attend_kernel.hip).
struct HeadsAttendParams {
    HeadsParams heads;
    SeqParams seqs;
    const uint8_t* base;         // the replica, already offset to the layer
    uint32_t type;
    uint32_t group;              // query heads of a key-value head
    uint32_t group_magic;        // row / group = row * group_magic / 2^group_shift below 2^31 rows
    uint32_t group_shift;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_token, q_head, out_token, out_head, lse_token;
    float* lse;                  // null: not written
    float scale_log2;            // scale * log2(e)
    uint32_t tree_words;
    const uint64_t* tree;        // null: causal
    unsigned long long* invalid_count;
    uint32_t chunk;              // positions of a cut
    uint32_t chunks;             // cuts of max_kv
    uint32_t first;              // the launch's first unit
    uint32_t units;              // places for (sequence, rows) units
    float* part;                 // workspace: [units][groups][chunks][rows][dim]
    float* part_ml;              // workspace: [units][groups][chunks][rows][2], maximum and sum
};

// How a call is cut: query rows of a unit, positions of a cut, workspace.
struct HeadsAttendPlan {
    uint32_t rows;
    uint32_t chunk;
    uint32_t chunks;
    uint64_t units;
    uint64_t bytes;
};
HeadsAttendPlan plan_heads_attend(const HeadsParams& h, uint32_t group, uint64_t num_seqs, uint64_t num_tokens, uint64_t max_q,
                                  uint64_t max_kv);
hipError_t launch_heads_attend(const HeadsAttendParams& p, void* workspace, hipStream_t stream);

// Enqueue the dequantizing gather on `stream`; returns the launch status.
hipError_t launch_gather(const GatherParams& p, hipStream_t stream);
// True if ctx's replicas are exactly these bases with these layer and page strides.
bool ctx_uses_storage(const kvpub_ctx* ctx, uint32_t replicas, uint8_t* const* main_bases,
                      uint8_t* const* idx_bases, uint64_t main_layer_stride, uint64_t idx_layer_stride,
                      uint64_t main_page_stride, uint64_t idx_page_stride);
// Set the number of pages per layer that ctx's launches may write, on the host
// and in the device capacity word (synchronous copy; no launch on ctx may run).
hipError_t ctx_set_pages(kvpub_ctx* ctx, uint64_t num_pages);
// Enqueue one fence kernel on `stream`.
hipError_t launch_fence(const FenceParams& p, hipStream_t stream);
// Enqueue the two-launch host-epoch fence (publish e, then wait for e) on `stream`.
hipError_t launch_host_epoch_fence(const FenceParams& p, uint64_t e, hipStream_t stream);

}  // namespace kvpub
