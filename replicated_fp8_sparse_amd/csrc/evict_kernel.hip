// Eviction from the published cache by accumulated attention weight, for gfx950
// (vLLM PR #52863 "[Kernel][PCP] Publish replicated KV updates through PyTorch
// symmetric memory", Design: every replica holds the same bytes, so a row is
// read once and written to all of them, as the store writes new ones).
//
// select_kernel, one block of 16 waves a sequence: the k largest of the
// unprotected weights by radix selection, 8 bits a pass from the top, on an
// order-preserving image of the binary32 values (kept in LDS for up to 32768
// positions, read again from memory beyond that).  The k-th largest value and
// the number of its equals that still fit give each position's fate; ranks come
// from ballots and one scan over the waves, so the kept positions come out in
// ascending order.
//
// move_kernel, one block for 64 destination positions: their rows are loaded
// into registers, then written to all replicas.  In place (rows or weights), a row
// may be another block's source.  Positions only move down (kept[i] >= i), so the rows of
// destination chunk c are sources of chunks <= c alone, and as ranks are
// consecutive of at most two of them, which select_kernel's ranks name.  A block
// takes its chunk by a ticket of its sequence's counter, loads, raises its
// chunk's flag and waits for those two flags: they belong to earlier tickets,
// whose blocks already run and raise theirs before waiting for anything, so
// every wait ends.
//
// A fence on another lane may poison the context at any time.  One thread of
// select_kernel reads the status, once for its sequence, and leaves the decision
// in the workspace; all waves of its block and of move_kernel's go by that word,
// so a sequence is evicted whole or left as it was, and no wave leaves a block
// that others wait in.
//
// Measured: 32 sequences of up to 16384 positions to 8192, two replicas, 624 MB:
// select 27 us, move 94 us, 124 us in all, what a copy of the bytes takes (5 TB/s);
// in place 468 us, as blocks wait for those whose rows they overwrite.
// 4 of 1000 to 256: 8 and 5 us, 12.3 us in all, the passes' barriers; in place 14.7.
// 16 waves a sequence and keys in LDS since a pass over memory costs more than its
// arithmetic; 64 rows a block keep 50 KB on the way in registers.
#include "kvpub_internal.h"

namespace kvpub {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class T> using gptr = __attribute__((address_space(1))) T*;
template <class T> using cgptr = const __attribute__((address_space(1))) T*;

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr uint32_t kLdsKeys = 32768;
constexpr int kMoveThreads = 256;
constexpr uint32_t kMoveBlocks = 1u << 22;         // chunks of a launch
constexpr uint32_t kSkipped = ~0u;                 // ranks[0] of a sequence that is left as it was (else 0)

// Larger for larger weights; -0 as +0, a NaN below everything.
__device__ __forceinline__ uint32_t order(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct SelectShared {
    uint32_t key[kLdsKeys];
    uint32_t hist[kSelWaves][256];
    uint32_t above[kSelWaves], equal[kSelWaves];
    uint32_t prefix, need;
    uint32_t status;
};

__global__ __launch_bounds__(kSelThreads) void select_kernel(const EvictParams p) {
    __shared__ SelectShared sh;
    const uint32_t b = blockIdx.x, tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t given = p.kv_len[b];
    const uint32_t len = given < 0 ? 0u : ((uint32_t)given > p.max_kv ? p.max_kv : (uint32_t)given);
    const uint32_t keep = len < p.budget ? len : p.budget;
    int32_t* kept = p.kept + (uint64_t)b * p.kept_stride;
    uint32_t* mine = p.state + (uint64_t)b * (2 * p.chunks + 2);
    uint32_t* flags = mine + 1;
    uint32_t* ranks = mine + 1 + p.chunks;             // kept positions below 64 * c, c = 0..chunks
    const float* w = p.weights_in + (uint64_t)b * p.weights_stride;
    const bool cached = len <= kLdsKeys;
    if (tid == 0) sh.status = __hip_atomic_load(&p.head->status, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (cached && len > p.budget)
        for (uint32_t i = tid; i < len; i += kSelThreads) sh.key[i] = order(w[i]);
    __syncthreads();
    if (sh.status & kStatusPoisoned) {
        if (tid == 0) ranks[0] = kSkipped;
        return;
    }
    if (tid == 0) {
        mine[0] = 0;
        p.new_len[b] = (int32_t)keep;
    }
    for (uint32_t c = tid; c < p.chunks; c += kSelThreads) flags[c] = 0;
    for (uint32_t i = keep + tid; i < p.budget; i += kSelThreads) kept[i] = -1;

    if (len <= p.budget) {
        for (uint32_t i = tid; i < len; i += kSelThreads) kept[i] = (int32_t)i;
        for (uint32_t c = tid; c <= p.chunks; c += kSelThreads) ranks[c] = c * 64u < len ? c * 64u : len;
        return;
    }
    const uint32_t a = p.first, z = len - p.last;     // the unprotected positions; budget < len, so a < z
    const uint32_t k = p.budget - p.first - p.last;
    auto key = [&](uint32_t i) { return cached ? sh.key[i] : order(w[i]); };

    // the k-th largest key, bits from the top: prefix is what is known of it
    uint32_t prefix = 0, need = k;
    if (k > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (uint32_t i = tid; i < kSelWaves * 256; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (uint32_t i = a + tid; i < z; i += kSelThreads) {
                const uint32_t v = key(i);
                if ((v & mask) == prefix) atomicAdd(&sh.hist[wave][(v >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t n = 0;
                for (int v = 0; v < kSelWaves; ++v) n += sh.hist[v][tid];
                sh.hist[0][tid] = n;
            }
            __syncthreads();
            if (wave == 0) {      // 4 digits a lane, the largest in lane 0
                uint32_t n[4], own = 0;
                for (int d = 0; d < 4; ++d) {
                    n[d] = sh.hist[0][255 - (lane * 4 + d)];
                    own += n[d];
                }
                uint32_t upto = own;
                for (int d = 1; d < 64; d <<= 1) {
                    const uint32_t y = __shfl_up(upto, d);
                    if (lane >= (uint32_t)d) upto += y;
                }
                uint32_t before = upto - own;
                if (before < need && need <= upto) {
                    int d = 0;
                    while (before + n[d] < need) before += n[d++];
                    sh.prefix = prefix | ((255 - (lane * 4 + d)) << shift);
                    sh.need = need - before;
                }
            }
            __syncthreads();
            prefix = sh.prefix;
            need = sh.need;
        }
    }
    // keys above `prefix` stay, and the first `need` equal to it (none with k == 0)
    const uint32_t chunks = (len + 63) / 64, per = (chunks + kSelWaves - 1) / kSelWaves;
    const uint32_t c0 = wave * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    auto fate = [&](uint32_t i, bool& above, bool& equal) {
        above = equal = false;
        if (i >= len) return;
        if (i < a || i >= z) { above = true; return; }
        if (k == 0) return;
        const uint32_t v = key(i);
        above = v > prefix;
        equal = v == prefix;
    };
    uint32_t n_above = 0, n_equal = 0;
    for (uint32_t c = c0; c < c1; ++c) {
        bool x, y;
        fate(c * 64u + lane, x, y);
        n_above += __popcll(__ballot(x));
        n_equal += __popcll(__ballot(y));
    }
    if (lane == 0) {
        sh.above[wave] = n_above;
        sh.equal[wave] = n_equal;
    }
    __syncthreads();
    uint32_t above = 0, equal = 0;
    for (uint32_t v = 0; v < wave; ++v) {
        above += sh.above[v];
        equal += sh.equal[v];
    }
    const uint64_t below = (1ull << lane) - 1;
    for (uint32_t c = c0; c < c1; ++c) {
        bool x, y;
        fate(c * 64u + lane, x, y);
        const uint64_t bx = __ballot(x), by = __ballot(y);
        const uint32_t rank_eq = equal + __popcll(by & below);
        const bool stays = x || (y && rank_eq < need);
        const uint64_t bs = __ballot(stays);
        const uint32_t taken = above + (equal < need ? equal : need);
        if (lane == 0) ranks[c] = taken;
        if (stays) kept[taken + __popcll(bs & below)] = (int32_t)(c * 64u + lane);
        above += __popcll(bx);
        equal += __popcll(by);
    }
    for (uint32_t c = chunks + tid; c <= p.chunks; c += kSelThreads) ranks[c] = keep;
}

// Ordered: rows or weights are written over others' sources.
template <bool Ordered>
__global__ __launch_bounds__(kMoveThreads) void move_kernel(const EvictParams p, uint32_t seq0, uint32_t chunk0) {
    __shared__ uint64_t src[64], dst[64], isrc[64], idst[64];    // ~0: not copied
    __shared__ uint32_t ticket;
    const uint32_t b = seq0 + blockIdx.y, tid = threadIdx.x;
    uint32_t* mine = p.state + (uint64_t)b * (2 * p.chunks + 2);
    uint32_t* flags = mine + 1;
    const uint32_t* ranks = mine + 1 + p.chunks;
    const uint32_t decision = ranks[0], keep = (uint32_t)p.new_len[b];
    const int64_t pages = p.head->capacity / 64;
    if (decision == kSkipped) return;                  // the same for all waves: nothing writes it meanwhile
    uint32_t c = chunk0 + blockIdx.x;
    if (Ordered) {
        if (tid == 0) ticket = atomicAdd(mine, 1u);
        __syncthreads();
        c = ticket;
    }
    const uint32_t i0 = c * 64u;
    float weight = 0.f;
    uint64_t my_isrc = ~0ull, my_idst = ~0ull;
    if (tid < 64) {
        uint64_t s = ~0ull, d = ~0ull;
        const uint32_t i = i0 + tid;
        if (i < keep) {
            const uint32_t at = (uint32_t)p.kept[(uint64_t)b * p.kept_stride + i];
            weight = p.weights_in[(uint64_t)b * p.weights_stride + at];
            const int64_t ps = p.pages[(uint64_t)b * p.pages_stride + (at >> 6)];
            const int64_t pd = p.dst[(uint64_t)b * p.dst_stride + (i >> 6)];
            if (ps < 0 || ps >= pages || pd < 0 || pd >= pages) {
                atomicAdd(p.invalid_count, 1ull);
            } else if (!p.same_pages || at != i) {   // in place, a row may stay where it is
                s = (uint64_t)ps * p.main_page_stride + (at & 63u) * 656u;
                d = (uint64_t)pd * p.main_page_stride + (i & 63u) * 656u;
                my_isrc = (uint64_t)ps * p.idx_page_stride + (at & 63u) * 128u;
                my_idst = (uint64_t)pd * p.idx_page_stride + (i & 63u) * 128u;
            }
        }
        src[tid] = s;
        dst[tid] = d;
        isrc[tid] = my_isrc;
        idst[tid] = my_idst;
    }
    __syncthreads();
    // 64 rows x 41 pieces of 16 bytes, 64 x 8 of Indexer-K codes, 64 scales
    u32x4 row[11], code[2];
    uint32_t scale = 0;
#pragma unroll
    for (int k = 0; k < 11; ++k) {
        const uint32_t x = tid + k * kMoveThreads, r = x / 41u;
        if (r < 64 && src[r] != ~0ull)
            row[k] = __builtin_nontemporal_load((cgptr<u32x4>)(p.main_base[0] + src[r] + (x - r * 41u) * 16u));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t x = tid + k * kMoveThreads, r = x >> 3;
        if (isrc[r] != ~0ull) code[k] = __builtin_nontemporal_load((cgptr<u32x4>)(p.idx_base[0] + isrc[r] + (x & 7u) * 16u));
    }
    // the scale of slot s: behind the page's codes, 4 bytes for each 128
    auto scale_at = [&](uint64_t codes) {
        const uint64_t page = codes / p.idx_page_stride, in = codes - page * p.idx_page_stride;
        return page * p.idx_page_stride + 8192u + in / 32u;
    };
    if (my_isrc != ~0ull) scale = *(const uint32_t*)(p.idx_base[0] + scale_at(my_isrc));
    if (Ordered) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // this thread's rows are in its registers
        __syncthreads();
        if (tid == 0) {
            __hip_atomic_store(flags + c, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
            const uint32_t lo = ranks[c], hi = ranks[c + 1];          // who reads the rows written here
            for (uint32_t f = lo / 64u; lo < hi && f <= (hi - 1) / 64u; ++f)
                while (__hip_atomic_load(flags + f, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_AGENT) == 0)
                    __builtin_amdgcn_s_sleep(1);
        }
        __syncthreads();
    }
    if (tid < 64 && i0 + tid < p.max_kv) p.weights_out[(uint64_t)b * p.weights_stride + i0 + tid] = weight;
    for (uint32_t r8 = 0; r8 < p.replicas; ++r8) {
#pragma unroll
        for (int k = 0; k < 11; ++k) {
            const uint32_t x = tid + k * kMoveThreads, r = x / 41u;
            if (r < 64 && dst[r] != ~0ull)
                __builtin_nontemporal_store(row[k], (gptr<u32x4>)(p.main_base[r8] + dst[r] + (x - r * 41u) * 16u));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t x = tid + k * kMoveThreads, r = x >> 3;
            if (idst[r] != ~0ull) __builtin_nontemporal_store(code[k], (gptr<u32x4>)(p.idx_base[r8] + idst[r] + (x & 7u) * 16u));
        }
        if (my_idst != ~0ull) *(uint32_t*)(p.idx_base[r8] + scale_at(my_idst)) = scale;
    }
}

}  // namespace

hipError_t launch_evict(const EvictParams& given, hipStream_t stream) {
    EvictParams p = given;
    p.chunks = (p.max_kv + 63) / 64;
    (void)hipGetLastError();
    select_kernel<<<dim3(p.num_seqs), dim3(kSelThreads), 0, stream>>>(p);
    for (uint32_t b = 0; b < p.num_seqs; b += 32768) {       // the grid's second dimension
        const uint32_t seqs = p.num_seqs - b < 32768 ? p.num_seqs - b : 32768;
        for (uint32_t c = 0; c < p.chunks; c += kMoveBlocks) {       // a dimension's threads stay below 2^32
            const dim3 grid(p.chunks - c < kMoveBlocks ? p.chunks - c : kMoveBlocks, seqs);
            if (p.same_pages || p.weights_out == p.weights_in) move_kernel<true><<<grid, dim3(kMoveThreads), 0, stream>>>(p, b, c);
            else move_kernel<false><<<grid, dim3(kMoveThreads), 0, stream>>>(p, b, c);
        }
    }
    return hipGetLastError();
}

}  // namespace kvpub
