// Latent attention in its expanded form for gfx950: after the latent vectors
// have been projected up, each head has a key part (128) and a value (128) of
// its own and shares the 64 RoPE values of a key.  (The prefill side of the
// cache that vLLM PR #52863 "[Kernel][PCP] Publish replicated KV updates
// through PyTorch symmetric memory" publishes; Design: prefill attention keeps
// consuming local, normalized and rotated K.)
//
// Mathematics: out = softmax(scale * (q_n . k_n + q_r . k_r)) v in one pass with
// a running maximum and sum; 640 operations a (query, key) pair and head against
// 2176 in the absorbed form, which is what the expansion buys for many queries.
//
// Mapping: a block of 4 waves takes 128 queries of one head, 32 a wave with the
// operands (192 values each) in registers, over tiles of 64 keys in LDS (24 KB
// of keys, 16 KB of values, two buffers: two blocks a CU).  Tiles are copied
// straight to LDS; each lane picks its source so that the 16-byte pieces of a
// row land permuted by the row number, which frees both the b128 reads of keys
// and the transposing reads of values of bank conflicts.  Scores come out
// transposed (keys down, queries across), so the weights are already an operand
// of the second product with its keys in that order.  The causal limit cuts a
// block's tiles; blocks with the most tiles start first, and blocks of one head
// go to one XCD (its L2 holds the head's keys).  Bound by the matrix units: 2 x 4096
// queries over 8192 keys, 16 heads, 427-431 us, 830 TFLOP/s, 69 % of a large bf16 matrix
// product, with the exponentials and sums between the products; 100 queries 10 us.
// The weights are rounded to bf16 as an operand of the second product: a second operand
// for their low part would double it, for less than the output's rounding takes away.
#include "kvpub_internal.h"

namespace kvpub {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
template <class T> using lptr = __attribute__((address_space(3))) T*;

constexpr int kThreads = 256;
constexpr int kQueries = 128;                    // of a block
constexpr int kKeys = 64;                        // of a tile
constexpr int kNope = 0;                         // tile parts, bytes
constexpr int kRope = kKeys * 256;
constexpr int kValue = kRope + kKeys * 128;
constexpr int kTile = kValue + kKeys * 256;      // 40960
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLazy = 8.0f;

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(lptr<const uint8_t>)(const uint8_t*)p;
}
// (m0 is a reserved register, which the compiler warns of: it holds no value of its own
// there, but may set it once for several uses.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop

// First token of sequence b (its end is the next one's), kept within the call's.
__device__ __forceinline__ uint32_t token_of(const ExpandedParams& p, uint32_t b) {
    const int32_t t = p.q_start[b];
    return t < 0 ? 0u : ((uint32_t)t > p.num_tokens ? p.num_tokens : (uint32_t)t);
}

// The places of query tiles by tokens: sequence b's begin at place token_of(b) / 128 + b.
// n tokens from there on are at most as many tiles as lie between that and the next
// sequence's places, so num_tokens / 128 + num_seqs places hold all tiles, whatever
// max_q_len allows.  The sequence of place v: 64 candidates at a time.
__device__ __forceinline__ uint32_t sequence_at(const ExpandedParams& p, uint32_t v, uint32_t lane) {
    uint32_t lo = 0, left = p.num_seqs;              // it is one of lo .. lo + left - 1
    while (left > 1) {
        const uint32_t step = (left + 63) / 64, b = lo + lane * step;
        const bool before = lane * step < left && token_of(p, b) / kQueries + b <= v;
        const uint32_t n = (uint32_t)__popcll(__ballot(before)), skip = (n ? n - 1 : 0u) * step;
        lo += skip;
        left = left - skip < step ? left - skip : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// 128 queries of sequence b, head h from tile tile_q on.
__device__ __forceinline__ void attend_tile(const ExpandedParams& p, uint32_t b, uint32_t h, uint32_t tile_q, uint8_t* ring) {
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t q0 = p.q_start[b], q1 = p.q_start[b + 1], k0 = p.k_start[b], k1 = p.k_start[b + 1];
    q0 = q0 < 0 ? 0 : q0;
    q1 = q1 > (int64_t)p.num_tokens ? (int64_t)p.num_tokens : q1;
    k0 = k0 < 0 ? 0 : k0;
    k1 = k1 > (int64_t)p.num_keys ? (int64_t)p.num_keys : k1;
    const int32_t n = q1 > q0 ? (int32_t)(q1 - q0) : 0, m = k1 > k0 ? (int32_t)(k1 - k0) : 0;
    const int32_t live = n < (int32_t)p.max_q ? n : (int32_t)p.max_q;
    const int32_t first = (int32_t)tile_q * kQueries;
    if (first >= live) return;

    // this wave's 32 queries (those behind the last repeat it and are not written)
    bf16x8 q[2][6];
    int32_t lim[2];                              // keys below lim are seen
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        int32_t i = first + (int32_t)wave * 32 + r * 16 + (int32_t)l16;
        i = i < live ? i : live - 1;
        const uint64_t t = (uint64_t)q0 + i;
        const uint16_t* a = p.q_nope + t * p.q_nope_token + h * p.q_nope_head + g * 8;
        const uint16_t* c = p.q_rope + t * p.q_rope_token + h * p.q_rope_head + g * 8;
#pragma unroll
        for (int s = 0; s < 4; ++s) q[r][s] = *(const bf16x8*)(a + s * 32);
#pragma unroll
        for (int s = 0; s < 2; ++s) q[r][4 + s] = *(const bf16x8*)(c + s * 32);
        lim[r] = p.causal ? m - n + i + 1 : m;
        lim[r] = lim[r] < 0 ? 0 : lim[r];
    }
    const int32_t last_i = first + kQueries < live ? first + kQueries - 1 : live - 1;
    const int32_t last = p.causal ? (m - n + last_i + 1 < 0 ? 0 : m - n + last_i + 1) : m;    // keys any query sees
    const int32_t clear = p.causal ? m - n + first + 1 : m;                                 // keys every query sees
    const int32_t tiles = (last + kKeys - 1) / kKeys;

    const uint32_t base = lds_offset(ring);
    // 40 copies of 1024 bytes a tile, 10 a wave: 4 of key parts (4 rows of 16
    // pieces each), 2 of RoPE (8 rows of 8 pieces), 4 of values
    auto fetch = [&](int32_t t, uint32_t to) {
        const int32_t top = m - 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t row = (wave * 4 + c) * 4 + (lane >> 4), piece = (lane & 15u) ^ (row & 15u);
            const int32_t u = t * kKeys + (int32_t)row;
            const uint64_t at = (uint64_t)k0 + (u < top ? u : top);
            copy16_to_lds(p.k_nope + at * p.k_nope_token + h * p.k_nope_head + piece * 8, to + kNope + (wave * 4 + c) * 1024);
            copy16_to_lds(p.v + at * p.v_token + h * p.v_head + piece * 8, to + kValue + (wave * 4 + c) * 1024);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t row = (wave * 2 + c) * 8 + (lane >> 3), piece = (lane & 7u) ^ ((row >> 1) & 7u);
            const int32_t u = t * kKeys + (int32_t)row;
            const uint64_t at = (uint64_t)k0 + (u < top ? u : top);
            copy16_to_lds(p.k_rope + at * p.k_rope_token + piece * 8, to + kRope + (wave * 2 + c) * 1024);
        }
    };

    f32x4 o[2][8];
    float mx[2], sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) o[r][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    if (tiles > 0) fetch(0, base);
    for (int32_t t = 0; t < tiles; ++t) {
        uint8_t* tile = ring + (t & 1) * kTile;
        if (t + 1 < tiles) {
            // the other buffer was read until the last barrier
            fetch(t + 1, base + ((t + 1) & 1) * kTile);
            asm volatile("s_waitcnt vmcnt(10)" ::: "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        asm volatile("s_barrier" ::: "memory");

        const bool masked = t * kKeys + kKeys > clear;
        if (masked) {
            // values that are not finite and may be hidden from some query become
            // zeros, and a NaN in the key gives it to those that see it
            const uint32_t key = threadIdx.x >> 2, j = threadIdx.x & 3u;
            uint8_t* row = tile + kValue + key * 256 + j * 64;
            bool odd = false;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const i32x4 v = *(const i32x4*)(row + c * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    odd |= (v[i] & 0x7F800000) == 0x7F800000 || (v[i] & 0x7F80) == 0x7F80;
            }
            const uint64_t who = __ballot(odd);
            const bool any = ((who >> (lane & ~3u)) & 15u) != 0;
            if (any) {
                const i32x4 z = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) *(i32x4*)(row + c * 16) = z;
            }
            if (any && j == 0) *(uint16_t*)(tile + kNope + key * 256) = 0x7FC0;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }

        f32x4 x[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t row = u * 16 + l16;
            const uint8_t* kn = tile + kNope + row * 256;
            const uint8_t* kr = tile + kRope + row * 128;
#pragma unroll
            for (int r = 0; r < 2; ++r) x[u][r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bf16x8 k = *(const bf16x8*)(kn + ((s * 4 + g) ^ l16) * 16);
#pragma unroll
                for (int r = 0; r < 2; ++r) x[u][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[r][s], x[u][r], 0, 0, 0);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 k = *(const bf16x8*)(kr + ((s * 4 + g) ^ ((row >> 1) & 7u)) * 16);
#pragma unroll
                for (int r = 0; r < 2; ++r) x[u][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[r][4 + s], x[u][r], 0, 0, 0);
            }
        }
        bf16x8 w[2][2];                          // [32 keys][queries]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u][r] *= p.scale_log2;
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t key = u * 16 + 4 * g + i;
                        x[u][r][i] = t * kKeys + (int32_t)key < lim[r] ? x[u][r][i] : -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, x[u][r][i]);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (__any(top > mx[r] + kLazy || (mx[r] == -INFINITY && top > mx[r]))) {
                const float next = fmaxf(mx[r], top);
                const float keep = mx[r] == -INFINITY ? 0.f : exp2f(mx[r] - next);
                mx[r] = next;
                sum[r] *= keep;
#pragma unroll
                for (int d = 0; d < 8; ++d) o[r][d] *= keep;
            }
            const float ref = mx[r] == -INFINITY ? 0.f : mx[r];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(x[u][r][i] - ref);
                    sum[r] += e;
                    w[r][u >> 1][(u & 1) * 4 + i] = (__bf16)e;
                }
        }
        // values: 4 keys of each 16 for this lane group, 16 columns
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                bf16x8 v;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t row = (half * 2 + u) * 16 + 4 * g + (l16 >> 2);
                    const uint8_t* at = tile + kValue + row * 256 + ((d * 2 + ((l16 >> 1) & 1u)) ^ (row & 15u)) * 16 + (l16 & 1u) * 8;
                    const i16x4 c = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr<i16x4>)at);
                    const bf16x4 c4 = __builtin_bit_cast(bf16x4, c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[u * 4 + i] = c4[i];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[r][half], o[r][d], 0, 0, 0);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }

#pragma unroll
    for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor(sum[r], 16);
        sum[r] += __shfl_xor(sum[r], 32);
        const int32_t i = first + (int32_t)wave * 32 + r * 16 + (int32_t)l16;
        if (i >= live) continue;
        const uint64_t t = (uint64_t)q0 + i;
        const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
        uint16_t* out = p.out + t * p.out_token + h * p.out_head + g * 4;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const f32x4 v = o[r][d] * inv;
            *(bf16x4*)(out + d * 16) = __builtin_convertvector(v, bf16x4);
        }
        if (p.lse && g == 0)
            p.lse[t * p.lse_token + h] = sum[r] == 0.f ? -INFINITY : ((mx[r] == -INFINITY ? 0.f : mx[r]) + log2f(sum[r])) * kLn2;
    }
}

// q_tiles tiles of each sequence and head: (sequence, head) by XCD, query tiles in falling order.
__global__ __launch_bounds__(kThreads, 2) void expanded_kernel(const ExpandedParams p, uint32_t q_tiles) {
    __shared__ __align__(16) uint8_t ring[2 * kTile];
    const uint32_t pairs = p.num_seqs * p.heads;
    const uint32_t id = blockIdx.x, xcd = id % 8u, in = id / 8u;
    const uint32_t pair = (in / q_tiles) * 8u + xcd;
    if (pair >= pairs) return;
    attend_tile(p, p.first_seq + pair / p.heads, pair % p.heads, p.first_tile + q_tiles - 1u - in % q_tiles, ring);
}

// The places from first_tile on in falling order, heads across.
__global__ __launch_bounds__(kThreads, 2) void expanded_places_kernel(const ExpandedParams p, uint32_t places) {
    __shared__ __align__(16) uint8_t ring[2 * kTile];
    const uint32_t v = p.first_tile + places - 1u - blockIdx.x / p.heads;
    const uint32_t b = sequence_at(p, v, threadIdx.x & 63u), place = token_of(p, b) / kQueries + b;
    if (v < place) return;                           // before the first sequence's
    attend_tile(p, b, blockIdx.x % p.heads, v - place, ring);
}

}  // namespace

hipError_t launch_expanded(const ExpandedParams& given, hipStream_t stream) {
    // a grid's threads stay below 2^32: at most 2^23 blocks a launch
    const uint32_t all = (given.max_q + kQueries - 1) / kQueries, most = (1u << 23) / 128;
    (void)hipGetLastError();
    // Blocks by tokens where max_q_len pads the sequences' tiles to more than twice the
    // places that the tokens need: one prompt of 8192 tokens among 255 single ones, 16
    // heads, 460 us, against 757 with blocks for every padded tile; one of 2048 among 63,
    // 94 against 91 (the search); 65535 single tokens with no bound 12 ms, against 5e8
    // padded blocks.
    const uint32_t places = given.num_tokens / kQueries + given.num_seqs;
    if ((uint64_t)given.num_seqs * all > 2ull * places) {
        const uint32_t step = (1u << 23) / given.heads;
        for (uint32_t v = 0; v < places; v += step) {
            ExpandedParams p = given;
            p.first_tile = v;
            const uint32_t n = places - v < step ? places - v : step;
            expanded_places_kernel<<<dim3(n * p.heads), dim3(kThreads), 0, stream>>>(p, n);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const uint32_t q_tiles = all < most ? all : most;
    const uint32_t seqs = (1u << 23) / (q_tiles * given.heads);          // 1 and more: 128 heads at most
    for (uint32_t q = 0; q < all; q += q_tiles) {
        for (uint32_t b = 0; b < given.num_seqs; b += seqs) {
            ExpandedParams p = given;
            p.first_seq = b;
            p.first_tile = q;
            p.num_seqs = given.num_seqs - b < seqs ? given.num_seqs - b : seqs;
            const uint32_t groups = (p.num_seqs * p.heads + 7) / 8;
            expanded_kernel<<<dim3(groups * 8 * q_tiles), dim3(kThreads), 0, stream>>>(p, q_tiles);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace kvpub
