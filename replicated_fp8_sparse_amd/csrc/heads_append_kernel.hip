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
// blocks.  A row takes D/8 lanes of 8 values, the rows of the block pass by in
// D/32 rounds that stay in registers between the maximum and the codes.
#include "kvpub.h"
#include "rotation.h"
#include "sequences.h"

namespace kvpub {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kThreads = 256;

template <class T>
struct alignas(16) Row8 {
    T v[8];
};

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

__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float inverse) {
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(x[4 * h] * inverse), clamp448(x[4 * h + 1] * inverse), 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(x[4 * h + 2] * inverse), clamp448(x[4 * h + 3] * inverse), w, true);
    }
    return c;
}

__device__ __forceinline__ u32x2 recode8(u32x2 old, float factor) {
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)old[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)old[h], true);
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * factor, a[1] * factor, 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(b[0] * factor, b[1] * factor, w, true);
    }
    return c;
}

template <class T, uint32_t D>
__global__ __launch_bounds__(kThreads) void heads_append_kernel(const HeadsAppendParams p, const Places places) {
    constexpr uint32_t kLanes = D / 8, kRows = kThreads / kLanes, kRounds = 64 / kRows;
    __shared__ float top[2][kThreads / 64];
    __shared__ int had[2];
    const uint32_t G = p.heads.groups, tid = threadIdx.x;
    const uint32_t place = p.first + blockIdx.x / G, g = blockIdx.x % G;
    const SeqOf s = find_sequence(p.seqs, place, places);
    if (!s.found || s.m == 0 || (p.head->status & kStatusPoisoned)) return;
    // positions [begin, end) are stored; base may be negative
    const int64_t base = (int64_t)s.kv - s.n;
    const int64_t begin = base < 0 ? 0 : base, end = base + s.m;
    const int64_t block = begin / 64 + s.place, low = block * 64;
    if (end <= begin || low >= end) return;
    const uint32_t r0 = begin > low ? (uint32_t)(begin - low) : 0u, r1 = end < low + 64 ? (uint32_t)(end - low) : 64u;
    const int32_t page = p.seqs.pages[(int64_t)s.b * p.seqs.pages_stride + block];
    if ((uint32_t)page >= p.heads.num_pages) {
        if (g == 0 && tid == 0) atomicAdd(p.invalid_count, 1ull);
        return;
    }
    const uint64_t at = (uint64_t)page * p.heads.page_stride, codes = at + (uint64_t)g * 128 * D, scales = at + (uint64_t)G * 128 * D + 2 * g;
    // the scale that older rows of the block have, read by one thread that later writes it
    if (tid == 0) {
        const uint8_t* o = p.base[0] + scales;
#pragma unroll
        for (int j = 0; j < 2; ++j) had[j] = r0 ? (o[j] < 1 ? 1 : (o[j] > 245 ? 245 : o[j])) : 0;
    }
    const uint32_t lane = tid % kLanes, row = tid / kLanes;
    float k[kRounds][8], v[kRounds][8], mk = 0.f, mv = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < kRounds; ++i) {
        const uint32_t r = i * kRows + row;
        if (r >= r0 && r < r1) {
            const int64_t pos = low + r, t = s.q0 + (pos - base);
            const T* kr = (const T*)p.k + t * p.k_token + (int64_t)g * p.k_head;
            const Row8<T> kx = *(const Row8<T>*)(kr + lane * 8);
            const Row8<T> vx = *(const Row8<T>*)((const T*)p.v + t * p.v_token + (int64_t)g * p.v_head + lane * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) k[i][e] = (float)kx.v[e], v[i][e] = (float)vx.v[e];
            if (p.rotation.dim) rotate8(k[i], kr, lane * 8, p.positions ? p.positions[t] : (int32_t)pos, p.rotation);
            mk = amax8(k[i], mk);
            mv = amax8(v[i], mv);
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        mk = fmaxf(mk, __shfl_xor(mk, d));
        mv = fmaxf(mv, __shfl_xor(mv, d));
    }
    if ((tid & 63u) == 0) top[0][tid >> 6] = mk, top[1][tid >> 6] = mv;
    __syncthreads();
    int byte[2];
    float inverse[2], factor[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int b = byte_of(fmaxf(fmaxf(top[j][0], top[j][1]), fmaxf(top[j][2], top[j][3])));
        byte[j] = b > had[j] ? b : had[j];
        inverse[j] = __uint_as_float((uint32_t)(254 - byte[j]) << 23);             // 2^(127 - byte)
        // what older codes are multiplied by; below 2^-100 all of them vanish alike
        factor[j] = __uint_as_float((uint32_t)(127 - (byte[j] - had[j] < 100 ? byte[j] - had[j] : 100)) << 23);
    }
    const bool again_k = r0 && byte[0] > had[0], again_v = r0 && byte[1] > had[1];
#pragma unroll
    for (uint32_t i = 0; i < kRounds; ++i) {
        const uint32_t r = i * kRows + row;
        const uint64_t ck = codes + (uint64_t)r * D + lane * 8, cv = ck + 64 * D;
        u32x2 wk, wv;
        bool put_k = true, put_v = true;
        if (r < r0) {
            put_k = again_k, put_v = again_v;
            if (put_k) wk = recode8(*(const u32x2*)(p.base[0] + ck), factor[0]);
            if (put_v) wv = recode8(*(const u32x2*)(p.base[0] + cv), factor[1]);
        } else if (r < r1) {
            wk = codes8(k[i], inverse[0]);
            wv = codes8(v[i], inverse[1]);
        } else {
            continue;
        }
        for (uint32_t x = 0; x < p.replicas; ++x) {
            if (put_k) *(u32x2*)(p.base[x] + ck) = wk;
            if (put_v) *(u32x2*)(p.base[x] + cv) = wv;
        }
    }
    if (tid == 0)
        for (uint32_t x = 0; x < p.replicas; ++x) *(uint16_t*)(p.base[x] + scales) = (uint16_t)(byte[0] | (byte[1] << 8));
}

}  // namespace

hipError_t launch_heads_append(const HeadsAppendParams& p, hipStream_t stream) {
    (void)hipGetLastError();
    uint64_t total;
    // n tokens lie in at most floor((n + 62) / 64) + 1 blocks
    const Places w = places(1, 6, 2, ((uint64_t)p.seqs.max_q + 62) / 64 + 1, p.seqs.num_seqs, p.seqs.num_tokens, &total);
    const uint32_t G = p.heads.groups;
    const uint64_t most = ((1u << 24) - 1) / G;                       // a launch holds fewer than 2^32 threads
    for (uint64_t first = 0; first < total; first += most) {
        HeadsAppendParams q = p;
        q.first = (uint32_t)first;
        const uint32_t blocks = (uint32_t)std::min(most, total - first) * G;
        const bool half = p.type == KVPUB_FP16;
        if (p.heads.dim == 64) {
            if (half) heads_append_kernel<_Float16, 64><<<blocks, kThreads, 0, stream>>>(q, w);
            else heads_append_kernel<__bf16, 64><<<blocks, kThreads, 0, stream>>>(q, w);
        } else if (p.heads.dim == 128) {
            if (half) heads_append_kernel<_Float16, 128><<<blocks, kThreads, 0, stream>>>(q, w);
            else heads_append_kernel<__bf16, 128><<<blocks, kThreads, 0, stream>>>(q, w);
        } else {
            if (half) heads_append_kernel<_Float16, 256><<<blocks, kThreads, 0, stream>>>(q, w);
            else heads_append_kernel<__bf16, 256><<<blocks, kThreads, 0, stream>>>(q, w);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kvpub
