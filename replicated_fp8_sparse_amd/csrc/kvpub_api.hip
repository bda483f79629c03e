// C-ABI host side of libkvpub: argument checks, context lifetime, launches,
// graph capture.  Nothing here allocates or synchronizes on the store / fence
// path; creation is all-or-nothing (vLLM PR #54030 "[Perf][PCP] Fuse
// direct-KV publication fence", commit list: opt-in allocation either fully
// succeeds at startup or leaves nothing behind; teardown drops every view).
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include "kvpub.h"
#include "kvpub_internal.h"

using kvpub::FenceParams;
using kvpub::StoreParams;

struct kvpub_ctx {
    kvpub_config cfg;
    uint8_t* main_base[KVPUB_MAX_REPLICAS];
    uint8_t* idx_base[KVPUB_MAX_REPLICAS];
    uint8_t* words;            // device: status, invalid count, epochs
    uint64_t* host_signals;    // P > 1: host-coherent signals [lanes][P] (kSignalStride apart)
    uint64_t* host_signals_dev;
    uint64_t timeout_ticks;
    hipStream_t capture_stream;
    uint64_t host_epoch[KVPUB_MAX_LANES];   // kvpub_fence_host_epoch: the epoch each lane last published
    bool is_static;            // kvpub_create_static: words in the static array, this struct in static storage
};

struct kvpub_graph {
    kvpub_ctx* ctx;
    hipGraph_t graph;
    hipGraphExec_t exec;
};

namespace {

constexpr uint64_t kDefaultTimeoutNs = 5000000000ull;

size_t words_bytes(const kvpub_config& c) {
    return kvpub::kEpochOffset + (size_t)c.num_lanes * kvpub::kLine;
}

uint64_t* epoch_ptr(kvpub_ctx* c, uint32_t lane) {
    return reinterpret_cast<uint64_t*>(c->words + kvpub::kEpochOffset + (size_t)lane * kvpub::kLine);
}

// Participant signals exist only with peers; alone, the epoch is the barrier.
uint64_t* signals_dev_ptr(kvpub_ctx* c, uint32_t lane) {
    const uint32_t P = c->cfg.num_participants;
    if (P == 1) return nullptr;
    return c->host_signals_dev + (size_t)lane * P * kvpub::kSignalStride;
}

// Sets the context's device current for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) { ok = false; prev = -1; return; }
        if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

// Test hook: KVPUB_TEST_FAIL_ALLOC_AT=k makes the k-th allocation of a
// kvpub_create call fail (k >= 1), to exercise the all-or-nothing cleanup.
struct AllocCounter {
    int fail_at = 0;
    int n = 0;
    AllocCounter() {
        const char* s = std::getenv("KVPUB_TEST_FAIL_ALLOC_AT");
        fail_at = s ? std::atoi(s) : 0;
    }
    bool next_fails() { return ++n == fail_at; }
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kvpub_status map_hip(hipError_t e) {
    switch (e) {
        case hipSuccess: return KVPUB_OK;
        case hipErrorOutOfMemory: return KVPUB_ERR_OUT_OF_MEMORY;
        case hipErrorStreamCaptureUnsupported:
        case hipErrorStreamCaptureInvalidated:
        case hipErrorStreamCaptureImplicit:
        case hipErrorCapturedEvent:
        case hipErrorStreamCaptureWrongThread:
            return KVPUB_ERR_CAPTURING;
        default: return KVPUB_ERR_HIP;
    }
}

kvpub_status check_config(const kvpub_config* c) {
    if (!c || c->struct_size != sizeof(kvpub_config)) return KVPUB_ERR_INVALID_ARG;
    if (c->num_replicas < 1 || c->num_replicas > KVPUB_MAX_REPLICAS) return KVPUB_ERR_INVALID_ARG;
    if (c->num_layers < 1 || c->block_size != KVPUB_SLOTS_PER_PAGE) return KVPUB_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->num_pages > (1ull << 40)) return KVPUB_ERR_INVALID_ARG;
    if (c->main_page_stride < KVPUB_MAIN_PAGE_BYTES || c->main_page_stride % 16) return KVPUB_ERR_INVALID_ARG;
    if (c->idx_page_stride < KVPUB_IDX_PAGE_BYTES || c->idx_page_stride % 16) return KVPUB_ERR_INVALID_ARG;
    if (c->num_layers > 1) {
        if (c->main_layer_stride % 16 || c->idx_layer_stride % 16) return KVPUB_ERR_INVALID_ARG;
        if (c->main_layer_stride / c->main_page_stride < c->num_pages) return KVPUB_ERR_INVALID_ARG;
        if (c->idx_layer_stride / c->idx_page_stride < c->num_pages) return KVPUB_ERR_INVALID_ARG;
    }
    if (c->num_lanes < 1 || c->num_lanes > KVPUB_MAX_LANES) return KVPUB_ERR_INVALID_ARG;
    if (c->num_participants < 1 || c->num_participants > KVPUB_MAX_PARTICIPANTS) return KVPUB_ERR_INVALID_ARG;
    if (c->device < 0 || (c->flags & ~KVPUB_CONFIG_FENCE_RELEASE_ONLY) != 0) return KVPUB_ERR_INVALID_ARG;
    return KVPUB_OK;
}

kvpub_status check_store(const kvpub_ctx* ctx, uint32_t layer, int64_t T, const void* latent,
                         int64_t ls, const void* rope, int64_t rs, const void* indexer,
                         int64_t is, const int64_t* slots) {
    if (!ctx) return KVPUB_ERR_INVALID_ARG;
    if (layer >= ctx->cfg.num_layers) return KVPUB_ERR_INVALID_ARG;
    if (T < 0 || T > KVPUB_MAX_TOKENS) return KVPUB_ERR_INVALID_ARG;
    if (T == 0) return KVPUB_OK;
    if (!latent || !rope || !indexer || !slots) return KVPUB_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(indexer, 16) || !aligned(slots, 8))
        return KVPUB_ERR_INVALID_ARG;
    if (ls < (int64_t)KVPUB_LATENT_DIM || ls % 8 || ls > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (rs < (int64_t)KVPUB_ROPE_DIM || rs % 8 || rs > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (is < (int64_t)KVPUB_INDEXER_DIM || is % 8 || is > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    return KVPUB_OK;
}

StoreParams store_params(kvpub_ctx* ctx, uint32_t layer, int64_t T, const void* latent, int64_t ls,
                         const void* rope, int64_t rs, const void* indexer, int64_t is,
                         const int64_t* slots) {
    StoreParams p;
    std::memset(&p, 0, sizeof p);
    p.latent = static_cast<const uint16_t*>(latent);
    p.rope = static_cast<const uint16_t*>(rope);
    p.indexer = static_cast<const uint16_t*>(indexer);
    p.latent_stride = ls;
    p.rope_stride = rs;
    p.indexer_stride = is;
    p.slots = slots;
    p.num_tokens = T;
    p.main_page_stride = ctx->cfg.main_page_stride;
    p.idx_page_stride = ctx->cfg.idx_page_stride;
    for (uint32_t r = 0; r < ctx->cfg.num_replicas; ++r) {
        p.main_base[r] = ctx->main_base[r] + (uint64_t)layer * ctx->cfg.main_layer_stride;
        p.idx_base[r] = ctx->idx_base[r] + (uint64_t)layer * ctx->cfg.idx_layer_stride;
    }
    p.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    p.head = reinterpret_cast<const kvpub::CtxHead*>(ctx->words + kvpub::kStatusOffset);
    // The write-through store path takes 32-bit offsets within a replica's
    // layer span: every page the layer may ever hold (a VMM storage's capacity
    // can grow under a captured graph, so the span, not the current page count).
    // The layer stride is that span for one layer too: kvpub_vmm_create sets it
    // to the reserved range whatever the layer count.  Stores never go beyond
    // the capacity in the context's device words, so a span larger than the
    // caller's buffer only loosens this second range check.
    const uint64_t main_region = std::max(ctx->cfg.num_pages * ctx->cfg.main_page_stride, ctx->cfg.main_layer_stride);
    const uint64_t idx_region = std::max(ctx->cfg.num_pages * ctx->cfg.idx_page_stride, ctx->cfg.idx_layer_stride);
    if (main_region <= UINT32_MAX && idx_region <= UINT32_MAX) {
        p.main_region = (uint32_t)main_region;
        p.idx_region = (uint32_t)idx_region;
    }
    return p;
}

FenceParams fence_params(kvpub_ctx* ctx, uint32_t lane) {
    FenceParams f;
    f.epoch = epoch_ptr(ctx, lane);
    f.signals = signals_dev_ptr(ctx, lane);
    f.num_participants = ctx->cfg.num_participants;
    f.self = 0;
    f.status = reinterpret_cast<uint32_t*>(ctx->words + kvpub::kStatusOffset);
    f.timeout_ticks = ctx->timeout_ticks;
    f.acquire_wait = (ctx->cfg.flags & KVPUB_CONFIG_FENCE_RELEASE_ONLY) ? 0u : 1u;
    return f;
}

void release_static(kvpub_ctx* c);

void release(kvpub_ctx* c) {
    if (!c) return;
    if (c->is_static) { release_static(c); return; }
    if (c->capture_stream) (void)hipStreamDestroy(c->capture_stream);
    if (c->host_signals) (void)hipHostFree(c->host_signals);
    if (c->words) (void)hipFree(c->words);
    delete c;
}

// KVPUB_LOG=1: one line on stderr for each context created or destroyed (never
// on the store / fence / gather path).
bool log_enabled() {
    static const bool on = [] {
        const char* s = std::getenv("KVPUB_LOG");
        return s != nullptr && s[0] == '1';
    }();
    return on;
}

void log_create(const char* what, const kvpub_config* cfg, kvpub_status st, const kvpub_ctx* c) {
    if (!log_enabled()) return;
    if (cfg && cfg->struct_size == sizeof(kvpub_config))
        std::fprintf(stderr, "kvpub: %s R=%u L=%u pages=%llu lanes=%u participants=%u device=%d flags=%u -> %s (ctx %p)\n",
                     what, cfg->num_replicas, cfg->num_layers, (unsigned long long)cfg->num_pages, cfg->num_lanes,
                     cfg->num_participants, cfg->device, cfg->flags, kvpub_strerror(st), (const void*)c);
    else
        std::fprintf(stderr, "kvpub: %s (no valid config) -> %s\n", what, kvpub_strerror(st));
}

kvpub_status sync_device() {
    return map_hip(hipDeviceSynchronize());
}

// Timeout in wall-clock (s_memrealtime) ticks for a context on `device`.
hipError_t timeout_ticks_for(const kvpub_config* cfg, uint64_t* out) {
    int khz = 0;
    const hipError_t e = hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, cfg->device);
    if (e != hipSuccess) return e;
    if (khz <= 0) return hipErrorInvalidValue;
    const uint64_t ns = cfg->fence_timeout_ns ? cfg->fence_timeout_ns : kDefaultTimeoutNs;
    *out = (uint64_t)((double)ns * (double)khz / 1.0e6);
    if (*out == 0) *out = 1;
    return hipSuccess;
}

// ---- contexts that allocate nothing (kvpub_create_static) -------------------
//
// Their device words live in `scratch`, a file-scope device array of fixed
// size: the status line, the invalid-slot counter and the epochs of the
// largest lane count.  Each GPU holds its own copy for the life of the
// process.  In host code `scratch` names a host-side stand-in, not the device
// memory: the device address comes from hipGetSymbolAddress, resolved once per
// device with that device current, and only that address is used.  The host
// part of the context is one static struct per device.  One static context
// per device at a time: its words are that device's array.
constexpr size_t kStaticWordsBytes = kvpub::kEpochOffset + (size_t)KVPUB_MAX_LANES * kvpub::kLine;  // 8448
constexpr int kMaxStaticDevices = 64;

struct StaticSlot {
    uint8_t* words;   // device address of this device's `scratch`
    bool in_use;
    kvpub_ctx ctx;
};
StaticSlot g_static[kMaxStaticDevices];
std::mutex g_static_mu;

void release_static(kvpub_ctx* c) {
    std::lock_guard<std::mutex> lock(g_static_mu);
    g_static[c->cfg.device].in_use = false;
}

// ---- attention: argument checks and parameter blocks ------------------------

constexpr int64_t kMaxQueryTokens = int64_t(1) << 24;
constexpr uint32_t kMaxPositions = 1u << 30;
constexpr uint32_t kMaxSeqs = 65536;

bool good_stride(int64_t s, int64_t least) { return s >= least && s % 8 == 0 && s <= INT32_MAX; }

// A [T, H, width] bf16 array: token stride any multiple of 8 from 0 on (0 repeats a row).
bool good_rows(const void* base, int64_t token, int64_t head, int64_t width, uint32_t heads) {
    return base && aligned(base, 16) && good_stride(token, 0) && good_stride(head, heads > 1 ? width : 0);
}

bool good_queries(const kvpub_queries* q) {
    return q && q->num_tokens >= 0 && q->num_tokens <= kMaxQueryTokens && q->num_heads >= 1 && q->num_heads <= 128 &&
           std::isfinite(q->scale) && std::isfinite(q->scale * 1.44269504f);
}

bool good_pages(const kvpub_pages* g) {
    if (!g || g->num_seqs > kMaxSeqs || g->max_q_len < 1 || g->max_kv_len > kMaxPositions) return false;
    return g->tree_mask ? g->tree_words >= 1 && g->tree_words <= 64 : g->tree_words == 0;
}

// Rows that a written array must keep apart: heads by head, tokens by token.
bool good_output(const void* out, int64_t token, int64_t head, int64_t width, uint32_t heads, int64_t tokens) {
    if (!good_rows(out, token, head, width, heads)) return false;
    return tokens <= 1 || token >= width;
}

bool good_lse(const float* lse, int64_t stride, uint32_t heads, int64_t tokens) {
    return !lse || (aligned(lse, 4) && stride >= 0 && stride <= INT32_MAX && (tokens <= 1 || stride >= (int64_t)heads));
}

kvpub_status check_reader(const kvpub_ctx* ctx, uint32_t replica, uint32_t layer) {
    if (!ctx || replica >= ctx->cfg.num_replicas || layer >= ctx->cfg.num_layers) return KVPUB_ERR_INVALID_ARG;
    // a page that cannot be read is replaced by page 0 in the address, so one has to be backed
    if (ctx->cfg.num_pages == 0) return KVPUB_ERR_INVALID_ARG;
    return KVPUB_OK;
}

kvpub_status check_queries(const kvpub_queries* q) {
    if (!good_queries(q)) return KVPUB_ERR_INVALID_ARG;
    if (q->num_tokens == 0) return KVPUB_OK;
    if (!good_rows(q->q_latent, q->q_latent_token_stride, q->q_latent_head_stride, KVPUB_LATENT_DIM, q->num_heads) ||
        !good_rows(q->q_rope, q->q_rope_token_stride, q->q_rope_head_stride, KVPUB_ROPE_DIM, q->num_heads))
        return KVPUB_ERR_INVALID_ARG;
    return KVPUB_OK;
}

kvpub_status check_pages(const kvpub_queries* q, const kvpub_pages* g) {
    if (!good_pages(g)) return KVPUB_ERR_INVALID_ARG;
    if (g->num_seqs == 0 || q->num_tokens == 0) return KVPUB_OK;
    const int64_t tiles = ((int64_t)g->max_kv_len + 63) / 64;
    if (!g->kv_len || !aligned(g->kv_len, 4) || !g->page_table || !aligned(g->page_table, 4)) return KVPUB_ERR_INVALID_ARG;
    if (!aligned(g->q_start, 4) || !aligned(g->tree_mask, 8)) return KVPUB_ERR_INVALID_ARG;
    if (g->page_table_stride < tiles || g->page_table_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    // one token a sequence: every sequence needs its token
    if (!g->q_start && (int64_t)g->num_seqs > q->num_tokens) return KVPUB_ERR_INVALID_ARG;
    return KVPUB_OK;
}

kvpub::AttendParams attend_params(kvpub_ctx* ctx, uint32_t replica, uint32_t layer, const kvpub_queries* q) {
    kvpub::AttendParams a;
    std::memset(&a, 0, sizeof a);
    a.main_base = ctx->main_base[replica] + (uint64_t)layer * ctx->cfg.main_layer_stride;
    a.main_page_stride = ctx->cfg.main_page_stride;
    a.head = reinterpret_cast<const kvpub::CtxHead*>(ctx->words + kvpub::kStatusOffset);
    a.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    a.q_latent = static_cast<const uint16_t*>(q->q_latent);
    a.q_rope = static_cast<const uint16_t*>(q->q_rope);
    a.q_latent_token = q->q_latent_token_stride;
    a.q_latent_head = q->q_latent_head_stride;
    a.q_rope_token = q->q_rope_token_stride;
    a.q_rope_head = q->q_rope_head_stride;
    a.num_tokens = (uint32_t)q->num_tokens;
    a.heads = q->num_heads;
    a.scale_log2 = (float)((double)q->scale * 1.4426950408889634074);
    return a;
}

void set_pages(kvpub::AttendParams& a, const kvpub_pages* g) {
    a.num_seqs = g->num_seqs;
    a.max_q = (uint32_t)std::min<int64_t>(g->q_start ? g->max_q_len : 1, a.num_tokens);
    a.max_kv = g->max_kv_len;
    a.kv_len = g->kv_len;
    a.q_start = g->q_start;
    a.pages = g->page_table;
    a.pages_stride = g->page_table_stride;
    a.tree = g->tree_mask;
    a.tree_words = g->tree_words;
}

kvpub::AttendPlan page_plan(const kvpub_queries* q, const kvpub_pages* g) {
    const uint64_t tokens = (uint64_t)std::min<int64_t>(g->q_start ? g->max_q_len : 1, q->num_tokens);
    return kvpub::plan_attend(tokens * q->num_heads, g->num_seqs, q->num_tokens, q->num_heads, g->max_kv_len);
}

kvpub::AttendPlan slot_plan(const kvpub_queries* q, uint32_t num_slots) {
    return kvpub::plan_attend(q->num_heads, q->num_tokens, q->num_tokens, q->num_heads, num_slots);
}

// ---- rotations and the cache of heads: argument checks ------------------------

bool good_rotation(const kvpub_rotation* r, uint32_t width) {
    return r->turns && aligned(r->turns, 8) && r->dim >= 8 && r->dim % 8 == 0 && r->start % 8 == 0 &&
           (uint64_t)r->start + r->dim <= width && r->layout <= KVPUB_ROTATE_HALVES && std::isfinite(r->magnitude);
}

kvpub::RotationParams rotation_params(const kvpub_rotation* r) {
    if (!r) return kvpub::RotationParams{nullptr, 0, 0, 0, 0.f};
    return kvpub::RotationParams{r->turns, r->dim, r->start, r->layout == KVPUB_ROTATE_HALVES ? 1u : 0u, r->magnitude};
}

bool good_heads(const kvpub_heads* c) {
    if (!c || c->num_replicas < 1 || c->num_replicas > KVPUB_MAX_REPLICAS || c->num_layers < 1) return false;
    if (c->num_kv_heads < 1 || c->num_kv_heads > 128) return false;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX) return false;
    if (c->page_stride < KVPUB_HEADS_PAGE_BYTES(c->num_kv_heads, c->head_dim) || c->page_stride % 16) return false;
    if (c->num_layers > 1 && (c->layer_stride % 16 || c->layer_stride / c->page_stride < c->num_pages)) return false;
    for (uint32_t r = 0; r < c->num_replicas; ++r)
        if (!c->bases[r] || !aligned(c->bases[r], 16)) return false;
    return true;
}

uint8_t* heads_layer(const kvpub_heads* c, uint32_t replica, uint32_t layer) {
    return static_cast<uint8_t*>(c->bases[replica]) + (layer ? (uint64_t)layer * c->layer_stride : 0);
}

kvpub::HeadsParams heads_params(const kvpub_heads* c) {
    return kvpub::HeadsParams{c->page_stride, (int64_t)c->num_pages, c->num_kv_heads, c->head_dim};
}

// The sequences of a call with these tokens.
kvpub_status check_seqs(const kvpub_pages* g, int64_t tokens) {
    kvpub_queries q;
    std::memset(&q, 0, sizeof q);
    q.num_tokens = tokens;
    return check_pages(&q, g);
}

kvpub::SeqParams seq_params(const kvpub_pages* g, int64_t tokens) {
    kvpub::SeqParams s;
    s.kv_len = g->kv_len;
    s.q_start = g->q_start;
    s.pages = g->page_table;
    s.pages_stride = g->page_table_stride;
    s.num_seqs = g->num_seqs;
    s.num_tokens = (uint32_t)tokens;
    s.max_q = (uint32_t)std::min<int64_t>(g->q_start ? g->max_q_len : 1, tokens);
    s.max_kv = g->max_kv_len;
    return s;
}

bool good_heads_queries(const kvpub_heads* c, const kvpub_heads_queries* q) {
    return q && q->num_tokens >= 0 && q->num_tokens <= kMaxQueryTokens && q->num_heads >= 1 && q->num_heads <= 1024 &&
           q->num_heads % c->num_kv_heads == 0 && q->num_heads / c->num_kv_heads <= 128 && q->type <= KVPUB_FP16 && q->reserved == 0 &&
           std::isfinite(q->scale) && std::isfinite(q->scale * 1.44269504f);
}

kvpub::HeadsAttendPlan heads_plan(const kvpub_heads* c, const kvpub_heads_queries* q, const kvpub_pages* g) {
    const kvpub::SeqParams s = seq_params(g, q->num_tokens);
    return kvpub::plan_heads_attend(heads_params(c), q->num_heads / c->num_kv_heads, s.num_seqs, s.num_tokens, s.max_q, s.max_kv);
}

}  // namespace

static __device__ __align__(256) uint8_t scratch[kStaticWordsBytes];

namespace {

// Clears a static context's words (status, counter, every lane's epoch) and
// writes the capacity: one block, 16-byte vector stores.
__global__ __launch_bounds__(256) void init_words_kernel(uint8_t* words, uint32_t bytes, int64_t capacity) {
    for (uint32_t i = threadIdx.x * 16u; i < bytes; i += blockDim.x * 16u) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i == 0) {   // the CtxHead line starts with {status, reserved, capacity}
            v.z = (uint32_t)((uint64_t)capacity & 0xFFFFFFFFu);
            v.w = (uint32_t)((uint64_t)capacity >> 32);
        }
        *reinterpret_cast<uint4*>(words + i) = v;
    }
}

// The device address of this device's `scratch` (the device must be current).
hipError_t static_words(int device, uint8_t** out) {
    StaticSlot& slot = g_static[device];
    if (!slot.words) {
        void* ptr = nullptr;
        const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return e;
        if (!ptr) return hipErrorInvalidSymbol;
        slot.words = static_cast<uint8_t*>(ptr);
    }
    *out = slot.words;
    return hipSuccess;
}

}  // namespace

namespace kvpub {

bool ctx_uses_storage(const kvpub_ctx* ctx, uint32_t replicas, uint8_t* const* main_bases,
                      uint8_t* const* idx_bases, uint64_t main_layer_stride, uint64_t idx_layer_stride,
                      uint64_t main_page_stride, uint64_t idx_page_stride) {
    if (ctx->cfg.num_replicas != replicas) return false;
    if (ctx->cfg.main_layer_stride != main_layer_stride || ctx->cfg.idx_layer_stride != idx_layer_stride)
        return false;
    if (ctx->cfg.main_page_stride != main_page_stride || ctx->cfg.idx_page_stride != idx_page_stride)
        return false;
    for (uint32_t r = 0; r < replicas; ++r)
        if (ctx->main_base[r] != main_bases[r] || ctx->idx_base[r] != idx_bases[r]) return false;
    return true;
}

hipError_t ctx_set_pages(kvpub_ctx* ctx, uint64_t num_pages) {
    ctx->cfg.num_pages = num_pages;
    const int64_t capacity = (int64_t)(num_pages * KVPUB_SLOTS_PER_PAGE);
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return hipErrorInvalidDevice;
    return hipMemcpy(ctx->words + kvpub::kStatusOffset + offsetof(CtxHead, capacity), &capacity, sizeof capacity,
                     hipMemcpyHostToDevice);
}

}  // namespace kvpub

extern "C" {

KVPUB_API void kvpub_config_init(kvpub_config* cfg, uint32_t num_replicas, uint32_t num_layers,
                                 uint64_t num_pages) {
    if (!cfg) return;
    std::memset(cfg, 0, sizeof *cfg);
    cfg->struct_size = sizeof(kvpub_config);
    cfg->num_replicas = num_replicas;
    cfg->num_layers = num_layers;
    cfg->block_size = KVPUB_SLOTS_PER_PAGE;
    cfg->num_pages = num_pages;
    cfg->main_page_stride = KVPUB_MAIN_PAGE_BYTES;
    cfg->main_layer_stride = num_pages * KVPUB_MAIN_PAGE_BYTES;
    cfg->idx_page_stride = KVPUB_IDX_PAGE_BYTES;
    cfg->idx_layer_stride = num_pages * KVPUB_IDX_PAGE_BYTES;
    cfg->num_lanes = 1;
    cfg->num_participants = 1;
    cfg->fence_timeout_ns = 0;
    cfg->device = 0;
    cfg->flags = 0;
}

static kvpub_status create_ctx(const kvpub_config* cfg, void* const* main_bases, void* const* idx_bases,
                               kvpub_ctx** out) {
    if (!out) return KVPUB_ERR_INVALID_ARG;
    *out = nullptr;
    kvpub_status st = check_config(cfg);
    if (st != KVPUB_OK) return st;
    if (!main_bases || !idx_bases) return KVPUB_ERR_INVALID_ARG;
    for (uint32_t r = 0; r < cfg->num_replicas; ++r) {
        if (!main_bases[r] || !idx_bases[r]) return KVPUB_ERR_INVALID_ARG;
        if (!aligned(main_bases[r], 16) || !aligned(idx_bases[r], 16)) return KVPUB_ERR_INVALID_ARG;
    }

    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || ndev <= 0) return KVPUB_ERR_HIP;
    if (cfg->device >= ndev) return KVPUB_ERR_INVALID_ARG;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, cfg->device) != hipSuccess) return KVPUB_ERR_HIP;
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return KVPUB_ERR_UNSUPPORTED;

    DeviceGuard guard(cfg->device);
    if (!guard.ok) return KVPUB_ERR_HIP;

    kvpub_ctx* c = new (std::nothrow) kvpub_ctx;
    if (!c) return KVPUB_ERR_OUT_OF_MEMORY;
    std::memset(c, 0, sizeof *c);
    c->cfg = *cfg;
    for (uint32_t r = 0; r < cfg->num_replicas; ++r) {
        c->main_base[r] = static_cast<uint8_t*>(main_bases[r]);
        c->idx_base[r] = static_cast<uint8_t*>(idx_bases[r]);
    }

    AllocCounter alloc;
    const size_t wb = words_bytes(*cfg);
    hipError_t e = alloc.next_fails() ? hipErrorOutOfMemory : hipMalloc(&c->words, wb);
    if (e != hipSuccess) { c->words = nullptr; release(c); return map_hip(e); }
    e = hipMemset(c->words, 0, wb);
    if (e != hipSuccess) { release(c); return map_hip(e); }
    const int64_t capacity = (int64_t)(cfg->num_pages * KVPUB_SLOTS_PER_PAGE);
    e = hipMemcpy(c->words + kvpub::kStatusOffset + offsetof(kvpub::CtxHead, capacity), &capacity,
                  sizeof capacity, hipMemcpyHostToDevice);
    if (e != hipSuccess) { release(c); return map_hip(e); }

    if (cfg->num_participants > 1) {
        const size_t hb = (size_t)cfg->num_lanes * cfg->num_participants * kvpub::kLine;
        e = alloc.next_fails() ? hipErrorOutOfMemory
                               : hipHostMalloc(reinterpret_cast<void**>(&c->host_signals), hb,
                                               hipHostMallocCoherent | hipHostMallocMapped);
        if (e != hipSuccess) { c->host_signals = nullptr; release(c); return map_hip(e); }
        std::memset(c->host_signals, 0, hb);
        e = hipHostGetDevicePointer(reinterpret_cast<void**>(&c->host_signals_dev), c->host_signals, 0);
        if (e != hipSuccess) { release(c); return map_hip(e); }
    }

    e = alloc.next_fails() ? hipErrorOutOfMemory
                           : hipStreamCreateWithFlags(&c->capture_stream, hipStreamNonBlocking);
    if (e != hipSuccess) { c->capture_stream = nullptr; release(c); return map_hip(e); }

    if (timeout_ticks_for(cfg, &c->timeout_ticks) != hipSuccess) { release(c); return KVPUB_ERR_HIP; }

    *out = c;
    return KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_create(const kvpub_config* cfg, void* const* main_bases,
                                   void* const* idx_bases, kvpub_ctx** out) {
    const kvpub_status st = create_ctx(cfg, main_bases, idx_bases, out);
    log_create("create", cfg, st, out ? *out : nullptr);
    return st;
}

static kvpub_status create_static_ctx(const kvpub_config* cfg, void* const* main_bases, void* const* idx_bases,
                                      kvpub_stream_t stream, kvpub_ctx** out) {
    if (!out) return KVPUB_ERR_INVALID_ARG;
    *out = nullptr;
    kvpub_status st = check_config(cfg);
    if (st != KVPUB_OK) return st;
    if (!main_bases || !idx_bases) return KVPUB_ERR_INVALID_ARG;
    for (uint32_t r = 0; r < cfg->num_replicas; ++r) {
        if (!main_bases[r] || !idx_bases[r]) return KVPUB_ERR_INVALID_ARG;
        if (!aligned(main_bases[r], 16) || !aligned(idx_bases[r], 16)) return KVPUB_ERR_INVALID_ARG;
    }
    // host-driven peers' signals would need host memory of their own
    if (cfg->num_participants != 1) return KVPUB_ERR_UNSUPPORTED;
    if (kvpub::kEpochOffset + (size_t)cfg->num_lanes * kvpub::kLine > kStaticWordsBytes) return KVPUB_ERR_INVALID_ARG;
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || ndev <= 0) return KVPUB_ERR_HIP;
    if (cfg->device >= ndev) return KVPUB_ERR_INVALID_ARG;
    if (cfg->device >= kMaxStaticDevices) return KVPUB_ERR_UNSUPPORTED;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, cfg->device) != hipSuccess) return KVPUB_ERR_HIP;
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return KVPUB_ERR_UNSUPPORTED;

    DeviceGuard guard(cfg->device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(static_cast<hipStream_t>(stream), &cap) != hipSuccess) return KVPUB_ERR_HIP;
    if (cap != hipStreamCaptureStatusNone) return KVPUB_ERR_CAPTURING;
    uint64_t ticks = 0;
    if (timeout_ticks_for(cfg, &ticks) != hipSuccess) return KVPUB_ERR_HIP;

    std::lock_guard<std::mutex> lock(g_static_mu);
    StaticSlot& slot = g_static[cfg->device];
    if (slot.in_use) return KVPUB_ERR_IN_USE;
    uint8_t* words = nullptr;
    hipError_t e = static_words(cfg->device, &words);
    if (e != hipSuccess) return map_hip(e);

    (void)hipGetLastError();
    init_words_kernel<<<dim3(1), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
        words, (uint32_t)kStaticWordsBytes, (int64_t)(cfg->num_pages * KVPUB_SLOTS_PER_PAGE));
    e = hipGetLastError();
    if (e != hipSuccess) return map_hip(e);

    kvpub_ctx* c = &slot.ctx;
    std::memset(c, 0, sizeof *c);
    c->cfg = *cfg;
    for (uint32_t r = 0; r < cfg->num_replicas; ++r) {
        c->main_base[r] = static_cast<uint8_t*>(main_bases[r]);
        c->idx_base[r] = static_cast<uint8_t*>(idx_bases[r]);
    }
    c->words = words;
    c->timeout_ticks = ticks;
    c->is_static = true;
    slot.in_use = true;
    *out = c;
    return KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_create_static(const kvpub_config* cfg, void* const* main_bases,
                                          void* const* idx_bases, kvpub_stream_t stream, kvpub_ctx** out) {
    const kvpub_status st = create_static_ctx(cfg, main_bases, idx_bases, stream, out);
    log_create("create_static", cfg, st, out ? *out : nullptr);
    return st;
}

KVPUB_API kvpub_status kvpub_store(kvpub_ctx* ctx, uint32_t layer, int64_t num_tokens,
                                  const void* latent, int64_t latent_row_stride, const void* rope,
                                  int64_t rope_row_stride, const void* indexer,
                                  int64_t indexer_row_stride, const int64_t* slot_mapping,
                                  kvpub_stream_t stream) {
    kvpub_status st = check_store(ctx, layer, num_tokens, latent, latent_row_stride, rope,
                                  rope_row_stride, indexer, indexer_row_stride, slot_mapping);
    if (st != KVPUB_OK || num_tokens == 0) return st;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    const StoreParams p = store_params(ctx, layer, num_tokens, latent, latent_row_stride, rope,
                                       rope_row_stride, indexer, indexer_row_stride, slot_mapping);
    return map_hip(kvpub::launch_store(p, ctx->cfg.num_replicas, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_gather(kvpub_ctx* ctx, uint32_t replica, uint32_t layer, int64_t num_tokens,
                                    const int64_t* slot_mapping, void* latent_out, int64_t latent_row_stride,
                                    void* rope_out, int64_t rope_row_stride, void* indexer_out,
                                    int64_t indexer_row_stride, kvpub_stream_t stream) {
    if (!ctx || replica >= ctx->cfg.num_replicas) return KVPUB_ERR_INVALID_ARG;
    // the kernel reads slot 0's bytes for every padded or out-of-range slot, so
    // at least one page must be backed (a VMM storage that lost a layer has none)
    if (ctx->cfg.num_pages == 0) return KVPUB_ERR_INVALID_ARG;
    // the outputs obey the same pointer, alignment and stride rules as the store's inputs
    kvpub_status st = check_store(ctx, layer, num_tokens, latent_out, latent_row_stride, rope_out,
                                  rope_row_stride, indexer_out, indexer_row_stride, slot_mapping);
    if (st != KVPUB_OK || num_tokens == 0) return st;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::GatherParams g;
    std::memset(&g, 0, sizeof g);
    g.main_base = ctx->main_base[replica] + (uint64_t)layer * ctx->cfg.main_layer_stride;
    g.idx_base = ctx->idx_base[replica] + (uint64_t)layer * ctx->cfg.idx_layer_stride;
    g.main_page_stride = ctx->cfg.main_page_stride;
    g.idx_page_stride = ctx->cfg.idx_page_stride;
    g.head = reinterpret_cast<const kvpub::CtxHead*>(ctx->words + kvpub::kStatusOffset);
    g.slots = slot_mapping;
    g.num_tokens = num_tokens;
    g.latent = static_cast<uint16_t*>(latent_out);
    g.rope = static_cast<uint16_t*>(rope_out);
    g.indexer = static_cast<uint16_t*>(indexer_out);
    g.latent_stride = latent_row_stride;
    g.rope_stride = rope_row_stride;
    g.indexer_stride = indexer_row_stride;
    g.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    // every page the layer may ever hold (as for the store's buffer range):
    // 32-bit offsets if that span stays below 2^32 bytes
    const uint64_t main_span = std::max(ctx->cfg.num_pages * ctx->cfg.main_page_stride, ctx->cfg.main_layer_stride);
    const uint64_t idx_span = std::max(ctx->cfg.num_pages * ctx->cfg.idx_page_stride, ctx->cfg.idx_layer_stride);
    g.offsets32 = main_span <= UINT32_MAX && idx_span <= UINT32_MAX ? 1u : 0u;
    return map_hip(kvpub::launch_gather(g, static_cast<hipStream_t>(stream)));
}

KVPUB_API uint64_t kvpub_attend_workspace(const kvpub_queries* q, const kvpub_pages* pages) {
    if (!good_queries(q) || !good_pages(pages) || q->num_tokens == 0 || pages->num_seqs == 0) return 0;
    return page_plan(q, pages).bytes;
}

KVPUB_API uint64_t kvpub_attend_slots_workspace(const kvpub_queries* q, uint32_t num_slots) {
    if (!good_queries(q) || num_slots > (1u << 24) || q->num_tokens == 0) return 0;
    return slot_plan(q, num_slots).bytes;
}

KVPUB_API kvpub_status kvpub_attend(kvpub_ctx* ctx, uint32_t replica, uint32_t layer, const kvpub_queries* q,
                                    const kvpub_pages* pages, void* out, int64_t out_token_stride,
                                    int64_t out_head_stride, float* lse, int64_t lse_token_stride,
                                    void* workspace, uint64_t workspace_bytes, kvpub_stream_t stream) {
    kvpub_status st = check_reader(ctx, replica, layer);
    if (st == KVPUB_OK) st = check_queries(q);
    if (st == KVPUB_OK) st = check_pages(q, pages);
    if (st != KVPUB_OK || q->num_tokens == 0 || pages->num_seqs == 0) return st;
    if (!good_output(out, out_token_stride, out_head_stride, KVPUB_LATENT_DIM, q->num_heads, q->num_tokens) ||
        !good_lse(lse, lse_token_stride, q->num_heads, q->num_tokens))
        return KVPUB_ERR_INVALID_ARG;
    if (!page_plan(q, pages).fits) return KVPUB_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < kvpub_attend_workspace(q, pages))
        return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::AttendParams a = attend_params(ctx, replica, layer, q);
    set_pages(a, pages);
    a.out = static_cast<uint16_t*>(out);
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.lse_token = lse_token_stride;
    return map_hip(kvpub::launch_attend(a, workspace, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_attend_slots(kvpub_ctx* ctx, uint32_t replica, uint32_t layer, const kvpub_queries* q,
                                          const int64_t* slots, int64_t slots_stride, uint32_t num_slots, void* out,
                                          int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                          int64_t lse_token_stride, void* workspace, uint64_t workspace_bytes,
                                          kvpub_stream_t stream) {
    kvpub_status st = check_reader(ctx, replica, layer);
    if (st == KVPUB_OK) st = check_queries(q);
    if (st != KVPUB_OK) return st;
    if (num_slots > (1u << 24)) return KVPUB_ERR_INVALID_ARG;
    if (q->num_tokens == 0) return KVPUB_OK;
    if (num_slots > 0 && !slots) return KVPUB_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || slots_stride < (int64_t)num_slots || slots_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (!good_output(out, out_token_stride, out_head_stride, KVPUB_LATENT_DIM, q->num_heads, q->num_tokens) ||
        !good_lse(lse, lse_token_stride, q->num_heads, q->num_tokens))
        return KVPUB_ERR_INVALID_ARG;
    if (!slot_plan(q, num_slots).fits) return KVPUB_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < kvpub_attend_slots_workspace(q, num_slots))
        return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::AttendParams a = attend_params(ctx, replica, layer, q);
    a.num_seqs = a.num_tokens;
    a.max_q = 1;
    a.by_slots = 1;
    a.num_slots = num_slots;
    a.slots = slots;
    a.slots_stride = slots_stride;
    a.out = static_cast<uint16_t*>(out);
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.lse_token = lse_token_stride;
    return map_hip(kvpub::launch_attend(a, workspace, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_attend_weights(kvpub_ctx* ctx, uint32_t replica, uint32_t layer, const kvpub_queries* q,
                                            const kvpub_pages* pages, const float* lse, int64_t lse_token_stride,
                                            const float* weights_in, float* weights_out, int64_t weights_stride,
                                            kvpub_stream_t stream) {
    kvpub_status st = check_reader(ctx, replica, layer);
    if (st == KVPUB_OK) st = check_queries(q);
    if (st == KVPUB_OK) st = check_pages(q, pages);
    if (st != KVPUB_OK || pages->num_seqs == 0 || pages->max_kv_len == 0) return st;
    if (q->num_tokens && (!lse || !good_lse(lse, lse_token_stride, q->num_heads, q->num_tokens))) return KVPUB_ERR_INVALID_ARG;
    if (!weights_out || !aligned(weights_out, 4) || !aligned(weights_in, 4)) return KVPUB_ERR_INVALID_ARG;
    if (weights_stride < (int64_t)pages->max_kv_len || weights_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if ((((uint64_t)pages->max_kv_len + 63) / 64) * pages->num_seqs >= (1ull << 31)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::AttendParams a = attend_params(ctx, replica, layer, q);
    set_pages(a, pages);
    a.lse = const_cast<float*>(lse);
    a.lse_token = lse_token_stride;
    a.weights_in = weights_in;
    a.weights_out = weights_out;
    a.weights_stride = weights_stride;
    return map_hip(kvpub::launch_attend_weights(a, static_cast<hipStream_t>(stream)));
}

static bool good_evict(const kvpub_evict_io* io) {
    return io && io->reserved == 0 && io->num_seqs <= kMaxSeqs && io->max_kv_len >= 1 && io->max_kv_len <= kMaxPositions &&
           io->budget >= 1 && io->budget <= kMaxPositions && (uint64_t)io->first + io->last <= io->budget;
}

KVPUB_API uint64_t kvpub_evict_workspace(const kvpub_evict_io* io) {
    if (!good_evict(io)) return 0;
    const uint64_t chunks = (io->max_kv_len + 63) / 64;
    return (uint64_t)io->num_seqs * (2 * chunks + 2) * 4;
}

KVPUB_API kvpub_status kvpub_evict(kvpub_ctx* ctx, uint32_t layer, const kvpub_evict_io* io, void* workspace,
                                   uint64_t workspace_bytes, kvpub_stream_t stream) {
    kvpub_status st = check_reader(ctx, 0, layer);
    if (st != KVPUB_OK) return st;
    if (!good_evict(io)) return KVPUB_ERR_INVALID_ARG;
    if (io->num_seqs == 0) return KVPUB_OK;
    const void* arrays[] = {io->weights_in, io->weights_out, io->kv_len, io->page_table, io->dst_table, io->kept, io->new_len};
    for (const void* p : arrays)
        if (!p || !aligned(p, 4)) return KVPUB_ERR_INVALID_ARG;
    const uint32_t most = std::min(io->budget, io->max_kv_len);
    if (io->weights_stride < (int64_t)io->max_kv_len || io->weights_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (io->kept_stride < (int64_t)io->budget || io->kept_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (io->page_table_stride < ((int64_t)io->max_kv_len + 63) / 64 || io->page_table_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    if (io->dst_table_stride < ((int64_t)most + 63) / 64 || io->dst_table_stride > INT32_MAX) return KVPUB_ERR_INVALID_ARG;
    const bool in_place = io->dst_table == io->page_table;
    if (in_place && io->dst_table_stride != io->page_table_stride) return KVPUB_ERR_INVALID_ARG;
    if (io->new_len == io->kv_len) return KVPUB_ERR_INVALID_ARG;      // one thread writes new_len while others may still read kv_len
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < kvpub_evict_workspace(io)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::EvictParams e;
    std::memset(&e, 0, sizeof e);
    for (uint32_t r = 0; r < ctx->cfg.num_replicas; ++r) {
        e.main_base[r] = ctx->main_base[r] + (uint64_t)layer * ctx->cfg.main_layer_stride;
        e.idx_base[r] = ctx->idx_base[r] + (uint64_t)layer * ctx->cfg.idx_layer_stride;
    }
    e.main_page_stride = ctx->cfg.main_page_stride;
    e.idx_page_stride = ctx->cfg.idx_page_stride;
    e.replicas = ctx->cfg.num_replicas;
    e.head = reinterpret_cast<const kvpub::CtxHead*>(ctx->words + kvpub::kStatusOffset);
    e.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    e.weights_in = io->weights_in;
    e.weights_out = io->weights_out;
    e.weights_stride = io->weights_stride;
    e.kv_len = io->kv_len;
    e.pages = io->page_table;
    e.pages_stride = io->page_table_stride;
    e.dst = io->dst_table;
    e.dst_stride = io->dst_table_stride;
    e.kept = io->kept;
    e.kept_stride = io->kept_stride;
    e.new_len = io->new_len;
    e.num_seqs = io->num_seqs;
    e.max_kv = io->max_kv_len;
    e.budget = io->budget;
    e.first = io->first;
    e.last = io->last;
    e.same_pages = in_place ? 1u : 0u;
    e.state = static_cast<uint32_t*>(workspace);
    return map_hip(kvpub::launch_evict(e, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_attend_expanded(kvpub_ctx* ctx, const kvpub_expanded_io* io, kvpub_stream_t stream) {
    if (!ctx || !io) return KVPUB_ERR_INVALID_ARG;
    if (io->reserved != 0 || io->causal > 1 || io->num_heads < 1 || io->num_heads > 128 || io->num_seqs > 65535 ||
        io->max_q_len < 1 || io->num_tokens < 0 || io->num_tokens > kMaxQueryTokens || io->num_keys < 0 ||
        io->num_keys > kMaxQueryTokens || !std::isfinite(io->scale) || !std::isfinite(io->scale * 1.44269504f))
        return KVPUB_ERR_INVALID_ARG;
    if (io->num_tokens == 0 || io->num_seqs == 0) return KVPUB_OK;
    const uint32_t H = io->num_heads;
    if (!good_rows(io->q_nope, io->q_nope_token_stride, io->q_nope_head_stride, 128, H) ||
        !good_rows(io->q_rope, io->q_rope_token_stride, io->q_rope_head_stride, 64, H) ||
        !good_output(io->out, io->out_token_stride, io->out_head_stride, 128, H, io->num_tokens) ||
        !good_lse(io->lse, io->lse_token_stride, H, io->num_tokens))
        return KVPUB_ERR_INVALID_ARG;
    if (io->num_keys > 0 &&
        (!good_rows(io->k_nope, io->k_nope_token_stride, io->k_nope_head_stride, 128, H) ||
         !good_rows(io->k_rope, io->k_rope_token_stride, 64, 64, 1) ||
         !good_rows(io->v, io->v_token_stride, io->v_head_stride, 128, H)))
        return KVPUB_ERR_INVALID_ARG;
    if (!io->q_start || !io->k_start || !aligned(io->q_start, 4) || !aligned(io->k_start, 4)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::ExpandedParams e;
    std::memset(&e, 0, sizeof e);
    e.q_nope = static_cast<const uint16_t*>(io->q_nope);
    e.q_rope = static_cast<const uint16_t*>(io->q_rope);
    e.k_nope = static_cast<const uint16_t*>(io->k_nope);
    e.k_rope = static_cast<const uint16_t*>(io->k_rope);
    e.v = static_cast<const uint16_t*>(io->v);
    e.out = static_cast<uint16_t*>(io->out);
    e.lse = io->lse;
    e.q_nope_token = io->q_nope_token_stride;
    e.q_nope_head = io->q_nope_head_stride;
    e.q_rope_token = io->q_rope_token_stride;
    e.q_rope_head = io->q_rope_head_stride;
    e.k_nope_token = io->k_nope_token_stride;
    e.k_nope_head = io->k_nope_head_stride;
    e.k_rope_token = io->k_rope_token_stride;
    e.v_token = io->v_token_stride;
    e.v_head = io->v_head_stride;
    e.out_token = io->out_token_stride;
    e.out_head = io->out_head_stride;
    e.lse_token = io->lse_token_stride;
    e.q_start = io->q_start;
    e.k_start = io->k_start;
    e.num_tokens = (uint32_t)io->num_tokens;
    e.num_keys = (uint32_t)io->num_keys;
    e.num_seqs = io->num_seqs;
    e.heads = H;
    e.max_q = (uint32_t)std::min<int64_t>(io->max_q_len, io->num_tokens);
    e.causal = io->causal;
    e.scale_log2 = (float)((double)io->scale * 1.4426950408889634074);
    return map_hip(kvpub::launch_expanded(e, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_rotation_turns(const kvpub_rotation_config* c, uint64_t* turns) {
    if (!c || !turns || c->dim < 8 || c->dim > 1024 || c->dim % 8 || c->scaling > KVPUB_SCALING_BLEND) return KVPUB_ERR_INVALID_ARG;
    if (!std::isfinite(c->base) || c->base <= 1.0) return KVPUB_ERR_INVALID_ARG;
    if (c->scaling != KVPUB_SCALING_NONE && (!std::isfinite(c->factor) || c->factor < 1.0)) return KVPUB_ERR_INVALID_ARG;
    if (c->scaling >= KVPUB_SCALING_RAMP &&
        (!std::isfinite(c->original) || c->original < 1.0 || !(c->low > 0.0) || !(c->low < c->high) || !std::isfinite(c->high)))
        return KVPUB_ERR_INVALID_ARG;
    // in the 64 bits of a long double's significand
    const long double tau = 6.283185307179586476925286766559005768L, dim = c->dim, factor = c->factor;
    long double base = c->base, lo = 0, hi = 0;
    if (c->scaling == KVPUB_SCALING_GROWN) base *= std::pow(factor, dim / (dim - 2));
    if (c->scaling == KVPUB_SCALING_RAMP) {
        lo = std::max(0.0L, std::floor(dim * std::log(c->original / (tau * c->high)) / (2 * std::log(base))));
        hi = std::min(dim - 1, std::ceil(dim * std::log(c->original / (tau * c->low)) / (2 * std::log(base))));
    }
    for (uint32_t i = 0; i < c->dim / 2; ++i) {
        long double f = std::pow(base, -2.0L * i / dim), keep = 1;
        if (c->scaling == KVPUB_SCALING_LINEAR) keep = 0;
        if (c->scaling == KVPUB_SCALING_RAMP) keep = 1 - std::min(1.0L, std::max(0.0L, (i - lo) / std::max(hi - lo, 0.001L)));
        if (c->scaling == KVPUB_SCALING_BLEND) keep = std::min(1.0L, std::max(0.0L, (c->original * f / tau - c->low) / ((long double)c->high - c->low)));
        if (keep < 1) f = f * keep + f / factor * (1 - keep);
        turns[i] = (uint64_t)std::floor(f / tau * 18446744073709551616.0L + 0.5L);      // f <= 1: below 2^62
    }
    return KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_rotate(kvpub_ctx* ctx, const kvpub_rotate_io* io, kvpub_stream_t stream) {
    if (!ctx || !io) return KVPUB_ERR_INVALID_ARG;
    if (io->num_tokens < 0 || io->num_tokens > kMaxQueryTokens || io->num_heads < 1 || io->num_heads > 1024 || io->head_dim < 8 ||
        io->head_dim > 1024 || io->head_dim % 8 || io->type > KVPUB_FP32 || io->transpose > 1 || !good_rotation(&io->rotation, io->head_dim))
        return KVPUB_ERR_INVALID_ARG;
    if (io->num_tokens == 0) return KVPUB_OK;
    if (!good_rows(io->x, io->x_token_stride, io->x_head_stride, io->head_dim, io->num_heads) ||
        !good_output(io->y, io->y_token_stride, io->y_head_stride, io->head_dim, io->num_heads, io->num_tokens) || !io->positions ||
        !aligned(io->positions, 4))
        return KVPUB_ERR_INVALID_ARG;
    const bool in_place = io->x == io->y;
    if (in_place && (io->x_token_stride != io->y_token_stride || io->x_head_stride != io->y_head_stride)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::RotateParams p;
    std::memset(&p, 0, sizeof p);
    p.x = io->x;
    p.y = io->y;
    p.x_token = io->x_token_stride;
    p.x_head = io->x_head_stride;
    p.y_token = io->y_token_stride;
    p.y_head = io->y_head_stride;
    p.positions = io->positions;
    p.rotation = rotation_params(&io->rotation);
    p.num_tokens = (uint32_t)io->num_tokens;
    p.heads = io->num_heads;
    p.units = (in_place ? io->rotation.dim : io->head_dim) / 8;
    p.type = io->type;
    p.sign = io->transpose ? -io->rotation.magnitude : io->rotation.magnitude;
    return map_hip(kvpub::launch_rotate(p, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_store_rotated(kvpub_ctx* ctx, uint32_t layer, int64_t num_tokens, const void* latent, int64_t latent_row_stride,
                                           const void* rope, int64_t rope_row_stride, const void* indexer, int64_t indexer_row_stride,
                                           const int64_t* slot_mapping, const int32_t* positions, const kvpub_rotation* rope_rotation,
                                           const kvpub_rotation* indexer_rotation, kvpub_stream_t stream) {
    if (!rope_rotation && !indexer_rotation)
        return kvpub_store(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride, indexer, indexer_row_stride,
                           slot_mapping, stream);
    kvpub_status st = check_store(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride, indexer, indexer_row_stride,
                                  slot_mapping);
    if (st != KVPUB_OK) return st;
    if ((rope_rotation && !good_rotation(rope_rotation, KVPUB_ROPE_DIM)) ||
        (indexer_rotation && !good_rotation(indexer_rotation, KVPUB_INDEXER_DIM)))
        return KVPUB_ERR_INVALID_ARG;
    if (num_tokens == 0) return KVPUB_OK;
    if (!positions || !aligned(positions, 4)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::StoreRotatedParams p;
    std::memset(&p, 0, sizeof p);
    p.s = store_params(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride, indexer, indexer_row_stride, slot_mapping);
    p.positions = positions;
    p.rope = rotation_params(rope_rotation);
    p.indexer = rotation_params(indexer_rotation);
    p.replicas = ctx->cfg.num_replicas;
    return map_hip(kvpub::launch_store_rotated(p, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_heads_append(kvpub_ctx* ctx, const kvpub_heads* cache, uint32_t layer, const kvpub_heads_rows* rows,
                                          const kvpub_pages* pages, const kvpub_rotation* rotation, const int32_t* positions,
                                          kvpub_stream_t stream) {
    if (!ctx || !good_heads(cache) || layer >= cache->num_layers || !rows) return KVPUB_ERR_INVALID_ARG;
    if (rows->num_tokens < 0 || rows->num_tokens > kMaxQueryTokens || rows->type > KVPUB_FP16 || rows->reserved != 0)
        return KVPUB_ERR_INVALID_ARG;
    if (rotation && !good_rotation(rotation, cache->head_dim)) return KVPUB_ERR_INVALID_ARG;
    kvpub_status st = check_seqs(pages, rows->num_tokens);
    if (st != KVPUB_OK || rows->num_tokens == 0 || pages->num_seqs == 0) return st;
    const uint32_t G = cache->num_kv_heads, D = cache->head_dim;
    if (!good_rows(rows->k, rows->k_token_stride, rows->k_head_stride, D, G) || !good_rows(rows->v, rows->v_token_stride, rows->v_head_stride, D, G))
        return KVPUB_ERR_INVALID_ARG;
    if (rotation && !aligned(positions, 4)) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::HeadsAppendParams p;
    std::memset(&p, 0, sizeof p);
    p.heads = heads_params(cache);
    p.seqs = seq_params(pages, rows->num_tokens);
    for (uint32_t r = 0; r < cache->num_replicas; ++r) p.base[r] = heads_layer(cache, r, layer);
    p.replicas = cache->num_replicas;
    p.type = rows->type;
    p.k = static_cast<const uint16_t*>(rows->k);
    p.v = static_cast<const uint16_t*>(rows->v);
    p.k_token = rows->k_token_stride;
    p.k_head = rows->k_head_stride;
    p.v_token = rows->v_token_stride;
    p.v_head = rows->v_head_stride;
    p.positions = positions;
    p.rotation = rotation_params(rotation);
    p.head = reinterpret_cast<const kvpub::CtxHead*>(ctx->words + kvpub::kStatusOffset);
    p.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    return map_hip(kvpub::launch_heads_append(p, static_cast<hipStream_t>(stream)));
}

KVPUB_API uint64_t kvpub_heads_attend_workspace(const kvpub_heads* cache, const kvpub_heads_queries* q, const kvpub_pages* pages) {
    if (!good_heads(cache) || !good_heads_queries(cache, q) || !good_pages(pages) || q->num_tokens == 0 || pages->num_seqs == 0) return 0;
    return heads_plan(cache, q, pages).bytes;
}

KVPUB_API kvpub_status kvpub_heads_attend(kvpub_ctx* ctx, const kvpub_heads* cache, uint32_t replica, uint32_t layer,
                                          const kvpub_heads_queries* q, const kvpub_pages* pages, void* workspace,
                                          uint64_t workspace_bytes, kvpub_stream_t stream) {
    if (!ctx || !good_heads(cache) || replica >= cache->num_replicas || layer >= cache->num_layers || !good_heads_queries(cache, q))
        return KVPUB_ERR_INVALID_ARG;
    kvpub_status st = check_seqs(pages, q->num_tokens);
    if (st != KVPUB_OK || q->num_tokens == 0 || pages->num_seqs == 0) return st;
    const uint32_t D = cache->head_dim;
    if (!good_rows(q->q, q->q_token_stride, q->q_head_stride, D, q->num_heads) ||
        !good_output(q->out, q->out_token_stride, q->out_head_stride, D, q->num_heads, q->num_tokens) ||
        !good_lse(q->lse, q->lse_token_stride, q->num_heads, q->num_tokens))
        return KVPUB_ERR_INVALID_ARG;
    const kvpub::HeadsAttendPlan plan = heads_plan(cache, q, pages);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < plan.bytes) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub::HeadsAttendParams p;
    std::memset(&p, 0, sizeof p);
    p.heads = heads_params(cache);
    p.seqs = seq_params(pages, q->num_tokens);
    p.base = heads_layer(cache, replica, layer);
    p.type = q->type;
    p.group = q->num_heads / cache->num_kv_heads;
    p.q = static_cast<const uint16_t*>(q->q);
    p.out = static_cast<uint16_t*>(q->out);
    p.q_token = q->q_token_stride;
    p.q_head = q->q_head_stride;
    p.out_token = q->out_token_stride;
    p.out_head = q->out_head_stride;
    p.lse = q->lse;
    p.lse_token = q->lse_token_stride;
    p.scale_log2 = (float)((double)q->scale * 1.4426950408889634074);
    p.tree = pages->tree_mask;
    p.tree_words = pages->tree_words;
    p.invalid_count = reinterpret_cast<unsigned long long*>(ctx->words + kvpub::kInvalidOffset);
    return map_hip(kvpub::launch_heads_attend(p, workspace, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_fence(kvpub_ctx* ctx, uint32_t lane, kvpub_stream_t stream) {
    if (!ctx || lane >= ctx->cfg.num_lanes) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    return map_hip(kvpub::launch_fence(fence_params(ctx, lane), static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_fence_host_epoch(kvpub_ctx* ctx, uint32_t lane, kvpub_stream_t stream) {
    if (!ctx || lane >= ctx->cfg.num_lanes) return KVPUB_ERR_INVALID_ARG;
    if (ctx->cfg.num_participants != 1) return KVPUB_ERR_UNSUPPORTED;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    const uint64_t e = ctx->host_epoch[lane] + 1;
    const hipError_t err = kvpub::launch_host_epoch_fence(fence_params(ctx, lane), e,
                                                          static_cast<hipStream_t>(stream));
    if (err == hipSuccess) ctx->host_epoch[lane] = e;
    return map_hip(err);
}

KVPUB_API kvpub_status kvpub_graph_create(kvpub_ctx* ctx, const kvpub_layer_io* io, uint32_t n,
                                         uint32_t lane, kvpub_graph** out) {
    if (!out) return KVPUB_ERR_INVALID_ARG;
    *out = nullptr;
    if (!ctx || !io || n == 0 || lane >= ctx->cfg.num_lanes) return KVPUB_ERR_INVALID_ARG;
    for (uint32_t i = 0; i < n; ++i) {
        if (io[i].reserved != 0) return KVPUB_ERR_INVALID_ARG;
        kvpub_status st = check_store(ctx, io[i].layer, io[i].num_tokens, io[i].latent,
                                      io[i].latent_row_stride, io[i].rope, io[i].rope_row_stride,
                                      io[i].indexer, io[i].indexer_row_stride, io[i].slot_mapping);
        if (st != KVPUB_OK) return st;
    }
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;

    kvpub_graph* g = new (std::nothrow) kvpub_graph;
    if (!g) return KVPUB_ERR_OUT_OF_MEMORY;
    g->ctx = ctx;
    g->graph = nullptr;
    g->exec = nullptr;

    // A context from kvpub_create_static has no stream of its own: capture on
    // a temporary one.
    hipStream_t s = ctx->capture_stream;
    hipStream_t temp = nullptr;
    if (!s) {
        const hipError_t ce = hipStreamCreateWithFlags(&temp, hipStreamNonBlocking);
        if (ce != hipSuccess) { delete g; return map_hip(ce); }
        s = temp;
    }
    struct TempStream {
        hipStream_t s;
        ~TempStream() { if (s) (void)hipStreamDestroy(s); }
    } temp_guard{temp};
    hipError_t e = hipStreamBeginCapture(s, hipStreamCaptureModeThreadLocal);
    if (e != hipSuccess) { delete g; return map_hip(e); }
    hipError_t launch_err = hipSuccess;
    for (uint32_t i = 0; i < n && launch_err == hipSuccess; ++i) {
        if (io[i].num_tokens > 0) {
            const StoreParams p = store_params(ctx, io[i].layer, io[i].num_tokens, io[i].latent,
                                               io[i].latent_row_stride, io[i].rope,
                                               io[i].rope_row_stride, io[i].indexer,
                                               io[i].indexer_row_stride, io[i].slot_mapping);
            launch_err = kvpub::launch_store(p, ctx->cfg.num_replicas, s);
        }
        if (launch_err == hipSuccess) launch_err = kvpub::launch_fence(fence_params(ctx, lane), s);
    }
    e = hipStreamEndCapture(s, &g->graph);
    if (launch_err != hipSuccess || e != hipSuccess) {
        if (g->graph) (void)hipGraphDestroy(g->graph);
        delete g;
        return map_hip(launch_err != hipSuccess ? launch_err : e);
    }
    e = hipGraphInstantiate(&g->exec, g->graph, nullptr, nullptr, 0);
    if (e != hipSuccess) {
        (void)hipGraphDestroy(g->graph);
        delete g;
        return map_hip(e);
    }
    *out = g;
    return KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_graph_replay(kvpub_graph* g, kvpub_stream_t stream) {
    if (!g || !g->exec) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(g->ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    return map_hip(hipGraphLaunch(g->exec, static_cast<hipStream_t>(stream)));
}

KVPUB_API kvpub_status kvpub_graph_destroy(kvpub_graph* g) {
    if (!g) return KVPUB_OK;
    kvpub_status st = KVPUB_OK;
    {
        DeviceGuard guard(g->ctx->cfg.device);
        if (g->exec && hipGraphExecDestroy(g->exec) != hipSuccess) st = KVPUB_ERR_HIP;
        if (g->graph && hipGraphDestroy(g->graph) != hipSuccess) st = KVPUB_ERR_HIP;
    }
    delete g;
    return st;
}

KVPUB_API kvpub_status kvpub_epoch_read(kvpub_ctx* ctx, uint32_t lane, uint64_t* out) {
    if (!ctx || !out || lane >= ctx->cfg.num_lanes) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub_status st = sync_device();
    if (st != KVPUB_OK) return st;
    return map_hip(hipMemcpy(out, epoch_ptr(ctx, lane), sizeof(uint64_t), hipMemcpyDeviceToHost));
}

KVPUB_API kvpub_status kvpub_error_read(kvpub_ctx* ctx, uint64_t* invalid_slots, uint32_t* flags,
                                       int clear) {
    if (!ctx) return KVPUB_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->cfg.device);
    if (!guard.ok) return KVPUB_ERR_HIP;
    kvpub_status st = sync_device();
    if (st != KVPUB_OK) return st;
    uint32_t status = 0;
    uint64_t invalid = 0;
    hipError_t e = hipMemcpy(&status, ctx->words + kvpub::kStatusOffset, sizeof status,
                             hipMemcpyDeviceToHost);
    if (e == hipSuccess)
        e = hipMemcpy(&invalid, ctx->words + kvpub::kInvalidOffset, sizeof invalid,
                      hipMemcpyDeviceToHost);
    if (e == hipSuccess && clear) e = hipMemset(ctx->words + kvpub::kInvalidOffset, 0, sizeof invalid);
    if (e == hipSuccess && clear) e = hipDeviceSynchronize();
    if (e != hipSuccess) return map_hip(e);
    if (invalid_slots) *invalid_slots = invalid;
    if (flags) *flags = status;
    return (status & kvpub::kStatusFenceTimeout) ? KVPUB_ERR_FENCE_TIMEOUT : KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_participant_signal(kvpub_ctx* ctx, uint32_t lane, uint32_t p,
                                               volatile uint64_t** out) {
    if (!ctx || !out || lane >= ctx->cfg.num_lanes) return KVPUB_ERR_INVALID_ARG;
    if (ctx->cfg.num_participants < 2 || p < 1 || p >= ctx->cfg.num_participants)
        return KVPUB_ERR_INVALID_ARG;
    *out = ctx->host_signals + ((size_t)lane * ctx->cfg.num_participants + p) * kvpub::kSignalStride;
    return KVPUB_OK;
}

KVPUB_API kvpub_status kvpub_destroy(kvpub_ctx* ctx) {
    if (!ctx) return KVPUB_OK;
    const void* id = ctx;
    kvpub_status st;
    {
        DeviceGuard guard(ctx->cfg.device);
        st = sync_device();
        release(ctx);
    }
    if (log_enabled()) std::fprintf(stderr, "kvpub: destroy ctx %p -> %s\n", id, kvpub_strerror(st));
    return st;
}

KVPUB_API const char* kvpub_strerror(kvpub_status s) {
    switch (s) {
        case KVPUB_OK: return "ok";
        case KVPUB_ERR_INVALID_ARG: return "invalid argument";
        case KVPUB_ERR_OUT_OF_MEMORY: return "out of memory";
        case KVPUB_ERR_UNSUPPORTED: return "not supported (device not gfx950, or a configuration this call does not take)";
        case KVPUB_ERR_HIP: return "HIP runtime error";
        case KVPUB_ERR_CAPTURING: return "synchronizing call during stream capture";
        case KVPUB_ERR_FENCE_TIMEOUT: return "fence timed out; context poisoned";
        case KVPUB_ERR_IN_USE: return "the device's static context is in use";
        case KVPUB_STATUS_MAX_ENUM: break;
    }
    return "unknown status";
}

KVPUB_API uint32_t kvpub_abi_version(void) { return KVPUB_ABI_VERSION; }

}  // extern "C"
