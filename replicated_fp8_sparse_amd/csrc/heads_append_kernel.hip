// New keys and values written into the replicated cache of heads: keys rotated on the
// way, a block of 64 positions and head scaled by a power of two, coded in e4m3.
//
// Mathematics.  The scale is the least 2^e with amax <= 448 * 2^e, read off the bits of
// amax = m 2^k, 1 <= m < 2: 448 = 1.75 * 2^8, so e = k - 8, one more where m > 1.75.
// Dividing by it is exact, so a code is the value's own rounding to e4m3, and a block
// that later needs a larger scale shifts its codes' exponents: they round again
// only where they become subnormal.
//
// Mapping.  A block of threads owns one (sequence, block of 64 positions, head):
// nobody else writes that block's rows or scales, so nothing is ordered between
// blocks.  Half of its waves take the keys, half the values.  A row takes D/8 lanes of
// 8 values (4 pairs of the rotation: an angle is computed once), the rows of the block
// pass by in D/32 rounds that stay in registers between the maximum and the codes.
//
// Bound.  Few tokens: a launch and a chain of four reads (lengths, page, context, older scales): 64 sequences x
// one token, 8 heads of 128, 2 replicas 5.2 us, 256 x 1 6.7.  One round of blocks (4 x up to 2048
// tokens, 25 MB): that chain, then its bytes, 11.3-11.9 us.  Long: the angles, once for each head: 8 x up to
// 4096 tokens into 1 replica 33-34 us, where the bytes alone would leave 19.
#include "kvpub.h"
#include "rotation.h"
#include "sequences.h"

namespace kvpub {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));


// Largest finite magnitude of x and m.
__device__ __forceinline__ float amax8(const float (&x)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        m = fmaxf(m, a < INFINITY ? a : 0.f);            // a NaN is not below infinity
    }
    return m;
}

// Scale byte of a largest magnitude (0 or normal, or so small that the least byte serves).
__device__ __forceinline__ int byte_of(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b < 1 ? 1 : (b > 245 ? 245 : b);
}

__device__ __forceinline__ float clamp448(float q) { return q > 448.f ? 448.f : (q < -448.f ? -448.f : q); }   // NaN stays

__device__ __forceinline__ uint32_t codes4(const float* x, float inverse) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(x[0] * inverse), clamp448(x[1] * inverse), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(x[2] * inverse), clamp448(x[3] * inverse), w, true);
}

__device__ __forceinline__ uint32_t recode4(uint32_t old, float factor) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)old, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)old, true);
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * factor, a[1] * factor, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(b[0] * factor, b[1] * factor, w, true);
}

template <uint32_t D> constexpr uint32_t kMany = D == 256 ? 1024 : 512;         // threads of a block, at most 1024

// N threads, half of them for the keys, half for the values; Rounds: of rows that they pass,
// enough for the new ones.
template <class T, uint32_t D, uint32_t N, uint32_t Rounds>
__global__ __launch_bounds__(N) void heads_append_kernel(const HeadsAppendParams p, const Places places) {
    constexpr uint32_t kLanes = D / 8, kRows = N / 2 / kLanes, kHalfWaves = N / 128;
    constexpr bool Many = N > 128;
    __shared__ __attribute__((aligned(16))) uint8_t image[2][Many ? 64 * D : 16];
    __shared__ float top[2][kHalfWaves];
    __shared__ int had[2];
    __shared__ uint32_t stop;
    const uint32_t G = p.heads.groups, tid = threadIdx.x & (N / 2 - 1);
    const uint32_t value = __builtin_amdgcn_readfirstlane(threadIdx.x / (N / 2));       // 0: keys, 1: values
    const uint32_t turn = blockIdx.x / G, g = blockIdx.x - turn * G;
    const SeqOf s = find_sequence(p.seqs, p.first + turn, places);
    // positions [begin, end) are stored; base may be negative
    const int64_t base = (int64_t)s.kv - s.n;
    const int64_t begin = base < 0 ? 0 : base, end = base + s.m;
    const int64_t block = begin / 64 + s.place, low = block * 64;
    if (!s.found || end <= begin || low >= end) return;
    const int32_t page = uniform_load(p.seqs.pages, (int64_t)s.b * p.seqs.pages_stride + block);
    const uint32_t r0 = begin > low ? (uint32_t)(begin - low) : 0u, r1 = end < low + 64 ? (uint32_t)(end - low) : 64u;

    const uint32_t lane = tid % kLanes, row = tid / kLanes, dim = value ? 0u : p.rotation.dim;
    const RowUnit u = row_unit(lane, dim, p.rotation.start, p.rotation.halves);
    const T* src = (const T*)(value ? p.v : p.k) + (int64_t)g * (value ? p.v_head : p.k_head);
    const int64_t token = value ? p.v_token : p.k_token;
    Turns4 turns;
    turns.load(p.rotation.turns, lane, u.turned);
    float x[Rounds][8], m = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < Rounds; ++i) {
        const uint32_t r = r0 + i * kRows + row;
        if (r < r1) {
            const T* from = src + (s.q0 + (low + r - base)) * token;
            const Row4<T> a = *(const Row4<T>*)(from + u.at0), b = *(const Row4<T>*)(from + u.at1);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = (float)a.v[e], x[i][4 + e] = (float)b.v[e];
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < Rounds; ++i) {
        const uint32_t r = r0 + i * kRows + row;
        if (r < r1) {
            if (u.turned) {
                Angles4 angles;
                angles.set(p.positions ? p.positions[s.q0 + (low + r - base)] : (int32_t)(low + r), turns, p.rotation.magnitude, p.rotation.magnitude);
                angles.turn(x[i], p.rotation.halves);
            }
            m = amax8(x[i], m);
        }
    }
    if ((uint32_t)page >= p.heads.num_pages) {
        if (g == 0 && threadIdx.x == 0 && !(p.head->status & kStatusPoisoned)) atomicAdd(p.invalid_count, 1ull);
        return;
    }
    const uint64_t at = (uint64_t)page * p.heads.page_stride, codes = at + (uint64_t)(2 * g + value) * 64 * D, scales = at + (uint64_t)G * 128 * D + 2 * g;
    // the scales that older rows of the block have, read by the thread that later writes them; it also decides
    // for the whole block whether the context is poisoned (a fence that times out on another stream may set the flag
    // at any moment)
    if (threadIdx.x == 0) {
        stop = p.head->status & kStatusPoisoned;
        const uint8_t* o = p.base[0] + scales;
#pragma unroll
        for (int j = 0; j < 2; ++j) had[j] = r0 ? (o[j] < 1 ? 1 : (o[j] > 245 ? 245 : o[j])) : 0;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((tid & 63u) == 0) top[value][tid >> 6] = m;
    __syncthreads();
    if (stop) return;
    int byte[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float a = top[j][0];
#pragma unroll
        for (uint32_t w = 1; w < kHalfWaves; ++w) a = fmaxf(a, top[j][w]);
        const int b = byte_of(a);
        byte[j] = b > had[j] ? b : had[j];
    }
    const int mine = value ? byte[1] : byte[0], grown = mine - (value ? had[1] : had[0]);
    const float inverse = __uint_as_float((uint32_t)(254 - mine) << 23);               // 2^(127 - byte)
#pragma unroll
    for (uint32_t i = 0; i < Rounds; ++i) {
        const uint32_t r = r0 + i * kRows + row;
        if (r >= r1) break;
        const uint32_t w0 = codes4(x[i], inverse), w1 = codes4(x[i] + 4, inverse);
        if constexpr (Many) {
            *(uint32_t*)(image[value] + r * D + u.at0) = w0;
            *(uint32_t*)(image[value] + r * D + u.at1) = w1;
        } else {
            for (uint32_t b = 0; b < p.replicas; ++b) {
                *(uint32_t*)(p.base[b] + codes + r * D + u.at0) = w0;
                *(uint32_t*)(p.base[b] + codes + r * D + u.at1) = w1;
            }
        }
    }
    if constexpr (Many) {
        // the rows put together, and stored in pieces of 16 bytes
        __syncthreads();
        for (uint32_t at = r0 * D + tid * 16; at < r1 * D; at += N / 2 * 16) {
            const u32x4 w = *(const u32x4*)(image[value] + at);
            for (uint32_t b = 0; b < p.replicas; ++b) {
                u32x4* to = (u32x4*)(p.base[b] + codes + at);
                if (p.stream) __builtin_nontemporal_store(w, to);
                else *to = w;
            }
        }
    }
    if (r0 && grown > 0) {
        // older rows take the new scale; below 2^-100 all of them vanish alike
        const float factor = __uint_as_float((uint32_t)(127 - (grown < 100 ? grown : 100)) << 23);
        for (uint32_t r = row; r < r0; r += kRows) {
            const uint64_t c = codes + (uint64_t)r * D + lane * 8;
            const u32x2 old = *(const u32x2*)(p.base[0] + c), w = {recode4(old.x, factor), recode4(old.y, factor)};
            for (uint32_t b = 0; b < p.replicas; ++b) *(u32x2*)(p.base[b] + c) = w;
        }
    }
    if (threadIdx.x == 0)
        for (uint32_t b = 0; b < p.replicas; ++b) *(uint16_t*)(p.base[b] + scales) = (uint16_t)(byte[0] | (byte[1] << 8));
}

// Few new tokens a sequence: two waves a block, for as many rows as they pass in two rounds.
template <class T, uint32_t D>
void launch(const HeadsAppendParams& p, const Places& w, uint32_t blocks, hipStream_t stream) {
    constexpr uint32_t kFew = 2 * 64 / (D / 8);
    if (p.seqs.max_q <= kFew) heads_append_kernel<T, D, 128, 2><<<blocks, 128, 0, stream>>>(p, w);
    else heads_append_kernel<T, D, kMany<D>, 16 * D / kMany<D>><<<blocks, kMany<D>, 0, stream>>>(p, w);
}

}  // namespace

hipError_t launch_heads_append(const HeadsAppendParams& p, hipStream_t stream) {
    (void)hipGetLastError();
    uint64_t total;
    // n tokens lie in at most floor((n + 62) / 64) + 1 blocks
    const Places w = places(1, 6, 2, ((uint64_t)p.seqs.max_q + 62) / 64 + 1, p.seqs.num_seqs, p.seqs.num_tokens, &total);
    const uint32_t G = p.heads.groups;
    // what fills half of the L2s or more is stored past them (8 prompts of up to 4096 tokens, 38 MB: 28.2 us
    // for 32.8; 4 of 2048, 64 values a head, 10 MB: 7.4 for 7.1)
    const bool past = (uint64_t)p.seqs.num_tokens * G * p.heads.dim * 2 * p.replicas > (16u << 20);
    // a launch holds fewer than 2^32 threads, 1024 a block at most: a larger grid is cut modulo 2^32, with no error
    const uint64_t most = ((1u << 22) - 1) / G;
    for (uint64_t first = 0; first < total; first += most) {
        HeadsAppendParams q = p;
        q.first = (uint32_t)first;
        q.stream = past ? 1u : 0u;
        const uint32_t blocks = (uint32_t)std::min(most, total - first) * G;
        const bool half = p.type == KVPUB_FP16;
        if (p.heads.dim == 64) half ? launch<_Float16, 64>(q, w, blocks, stream) : launch<__bf16, 64>(q, w, blocks, stream);
        else if (p.heads.dim == 128) half ? launch<_Float16, 128>(q, w, blocks, stream) : launch<__bf16, 128>(q, w, blocks, stream);
        else half ? launch<_Float16, 256>(q, w, blocks, stream) : launch<__bf16, 256>(q, w, blocks, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kvpub
