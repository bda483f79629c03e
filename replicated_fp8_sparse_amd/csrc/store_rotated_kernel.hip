// The latent cache's store with the position rotation on the way: kvpub_store's
// bytes of rows whose RoPE and Indexer-K parts are rotated first (rotation.h).
//
// Mathematics.  Rotated values stay in binary32 until they are stored: RoPE values
// are rounded to bf16 once, Indexer-K values meet their scale and codes unrounded.
// A tile of 128: scale = RN32(amax / 448), code = e4m3fn(RN32(x / scale)).  For bf16
// values and scales from 2^-64 on the quotient is x y and one remainder step with y =
// RN32(1 / scale), which has the code of the division (the store's, checked there over all
// values); what is rotated, and smaller scales, divide.
//
// Mapping.  As the store's: a group of 4 tokens, a row of 16 lanes x 8 values is a
// tile.  Piece k < 4 is token k's latent, piece 4 the four Indexer-K rows, piece 5 the
// four RoPE rows (lanes 0..31).  Large batches: a wave takes a group's six pieces;
// small ones: a wave a piece, as what counts there is one wave's chain.  By groups the
// rows are put together in LDS first: stored as they lie in the lanes (8 bytes, 4, 16) 32768 tokens
// into 4 replicas took 52 us.  A fence on another lane may poison the context at any time: the status is read
// once for all pieces of a token, so its two rows are stored whole or left as they were.
//
// Bound.  Few tokens: a launch, three dependent reads and one wave's tile, 4.0-4.3 us up to
// 256.  Many: what lies between the reads and the writes: 8192 tokens into 4 replicas,
// 37 MB, 10.9-11.3 us (a large copy's rate would leave 7.3; kvpub_store, same rows, 7.8), 32768 30 us (29).  The
// divisions are 0.4 of that: 0.1 the Indexer-K tile's, 0.3 the latent tiles' scales and reciprocals.
#include "rotation.h"

namespace kvpub {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kPieces = 6;
constexpr int64_t kSmallTokens = 2048;                  // 2048 tokens, 2 replicas: 5.3 us by pieces, 6.0 by groups; 4096: 7.2 and 6.7
constexpr int64_t kStreamBytes = int64_t(32) << 20;                 // more than the L2s hold

__device__ __forceinline__ float row_max16(float v) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));    // quad_perm 1,0,3,2
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));    // quad_perm 2,3,0,1
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));   // row_half_mirror
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));  // row_mirror
}

// Codes of the lane's 8 values of a tile, and the tile's scale.  Fast: bf16 values.
template <bool Fast>
__device__ __forceinline__ u32x2 quantize(const float (&x)[8], float& scale) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    scale = row_max16(m) / 448.0f;
    float q[8];
    if (Fast && __all(scale >= 0x1p-64f && scale < INFINITY)) {
        const float y = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i] * y;
            q[i] = fmaf(-fmaf(a, scale, -x[i]), y, a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = scale == 0.f ? 0.f : x[i] / scale;
    }
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
    }
    return c;
}

// One of four values by a lane's index.
template <class A>
__device__ __forceinline__ A pick(const A (&v)[4], uint32_t i) {
    const A v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];      // values: a choice between elements would be one of addresses
    const A a = i & 1u ? v1 : v0, b = i & 1u ? v3 : v2;
    return i & 2u ? b : a;
}

template <bool Stream>
__device__ __forceinline__ void put16(uint8_t* to, u32x4 v) {
    if (Stream) __builtin_nontemporal_store(v, (u32x4*)to);
    else *(u32x4*)to = v;
}

// A lane's part of a row that turns.
struct Turning {
    RowUnit u;
    Row4<__bf16> a, b;
    Turns4 turns;
    int32_t position;
    __device__ __forceinline__ void load(const uint16_t* row, uint32_t unit, const RotationParams& r, int32_t pos) {
        u = row_unit(unit, r.dim, r.start, r.halves);
        a = *(const Row4<__bf16>*)(row + u.at0);
        b = *(const Row4<__bf16>*)(row + u.at1);
        turns.load(r.turns, unit, u.turned);
        position = pos;
    }
    __device__ __forceinline__ void turn(float (&x)[8], const RotationParams& r) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)a.v[i], x[4 + i] = (float)b.v[i];
        if (u.turned) {
            Angles4 angles;
            angles.set(position, turns, r.magnitude, r.magnitude);
            angles.turn(x, r.halves);
        }
    }
};

// Stream: the rows' whole pieces are stored past the L2s.
template <bool Split, bool Stream>
__global__ __launch_bounds__(Split ? kPieces * 64 : 256) void store_rotated_kernel(const StoreRotatedParams p) {
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __shared__ __attribute__((aligned(16))) uint8_t image[Split ? 1 : 4][Split ? 16 : 2624 + 512];
    __shared__ CtxHead decided;
    const uint32_t T = (uint32_t)p.s.num_tokens, t0 = (Split ? blockIdx.x : blockIdx.x * 4 + wave) * 4;
    if (t0 >= T) return;
    const uint32_t last = T - 1;
    auto token = [&](uint32_t k) { return t0 + k < last ? t0 + k : last; };
    auto mine = [&](uint32_t piece) { return !Split || wave == piece; };
    // token of the lane's Indexer-K piece and of its RoPE piece
    const uint32_t in = lane & 15u, row = lane >> 4, rr = (lane >> 3) & 3u;
    int64_t slot[4];
    u32x4 lat[4];
    Turning ix, rp;
    CtxHead head;
    if (!Split || threadIdx.x == 0) head = *p.s.head;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        slot[k] = p.s.slots[token(k)];
        if (mine(k)) lat[k] = __builtin_nontemporal_load((const u32x4*)(p.s.latent + (uint64_t)token(k) * p.s.latent_stride + lane * 8));
    }
    if (mine(4)) ix.load(p.s.indexer + (uint64_t)token(row) * p.s.indexer_stride, in, p.indexer, p.positions[token(row)]);
    if (mine(5)) rp.load(p.s.rope + (uint64_t)token(rr) * p.s.rope_stride, lane & 7u, p.rope, p.positions[token(rr)]);
    if constexpr (Split) {
        if (threadIdx.x == 0) decided = head;
        __syncthreads();
        head = decided;
    }
    if (head.status & kStatusPoisoned) return;               // a fence timed out: fail closed
    // a token's Main-KV row, its Indexer-K page and the place in it
    uint64_t main_at[4], page_at[4];
    uint32_t off[4], ok = 0, bad = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        if (t0 + k > last) slot[k] = -1;
        const uint64_t page = (uint64_t)slot[k] >> 6;
        off[k] = (uint32_t)slot[k] & 63u;
        main_at[k] = page * p.s.main_page_stride + off[k] * 656u;
        page_at[k] = page * p.s.idx_page_stride;
        const bool is = (uint64_t)slot[k] < (uint64_t)head.capacity;
        ok |= is ? 1u << k : 0u;
        bad += !is && slot[k] != -1;
    }
    if (bad && lane == 0 && mine(0)) atomicAdd(p.s.invalid_count, (unsigned long long)bad);

    u32x2 code[4];
    float scale[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
        if (mine(k)) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(lat[k][i] << 16), x[2 * i + 1] = __uint_as_float(lat[k][i] & 0xFFFF0000u);
            code[k] = quantize<true>(x, scale[k]);
        }
    u32x2 icode;
    float iscale;
    Row4<__bf16> r0, r1;
    if (mine(4)) {
        float x[8];
        ix.turn(x, p.indexer);
        icode = quantize<false>(x, iscale);
    }
    if (mine(5)) {
        float x[8];
        rp.turn(x, p.rope);
#pragma unroll
        for (int i = 0; i < 4; ++i) r0.v[i] = (__bf16)x[i], r1.v[i] = (__bf16)x[4 + i];
    }
    if constexpr (Split) {
        const uint64_t ti = pick(page_at, row), tr = pick(main_at, rr);
        const uint32_t oi = pick(off, row);
        for (uint32_t r = 0; r < p.replicas; ++r) {
            uint8_t* main = p.s.main_base[r];
            uint8_t* idx = p.s.idx_base[r];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
                if (mine(k) && ((ok >> k) & 1u)) {
                    *(u32x2*)(main + main_at[k] + lane * 8) = code[k];
                    if (in == 0) *(float*)(main + main_at[k] + 512 + row * 4) = scale[k];
                }
            if (mine(5) && ((ok >> rr) & 1u) && lane < 32) {
                *(Row4<__bf16>*)(main + tr + 528 + rp.u.at0 * 2) = r0;
                *(Row4<__bf16>*)(main + tr + 528 + rp.u.at1 * 2) = r1;
            }
            if (mine(4) && ((ok >> row) & 1u)) {
                uint8_t* c = idx + ti + oi * 128;
                *(uint32_t*)(c + ix.u.at0) = icode.x;
                *(uint32_t*)(c + ix.u.at1) = icode.y;
                if (in == 0) *(float*)(idx + ti + 8192 + oi * 4) = iscale;
            }
        }
    } else {
        // the rows put together in LDS, by the wave alone, and stored in pieces of 16 bytes: 41 a Main-KV row,
        // 8 an Indexer-K row
        uint8_t* img = image[wave];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            *(u32x2*)(img + k * 656 + lane * 8) = code[k];
            if (in == 0) *(float*)(img + k * 656 + 512 + row * 4) = scale[k];
        }
        if (lane < 32) {
            *(Row4<__bf16>*)(img + rr * 656 + 528 + rp.u.at0 * 2) = r0;
            *(Row4<__bf16>*)(img + rr * 656 + 528 + rp.u.at1 * 2) = r1;
        }
        *(uint32_t*)(img + 2624 + row * 128 + ix.u.at0) = icode.x;
        *(uint32_t*)(img + 2624 + row * 128 + ix.u.at1) = icode.y;
        __builtin_amdgcn_wave_barrier();
        u32x4 piece[3];
        uint64_t to[3];
        bool put[3];
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j) {
            const uint32_t i = lane + 64 * j, k = i / 41;
            put[j] = i < 164 && ((ok >> (k & 3u)) & 1u);
            to[j] = pick(main_at, k & 3u) + (i - k * 41) * 16;
            piece[j] = *(const u32x4*)(img + (i < 164 ? i : 0) * 16);
        }
        const uint32_t ki = (lane >> 3) & 3u;
        const u32x4 ipiece = *(const u32x4*)(img + 2624 + (lane & 31u) * 16);
        const uint64_t ito = pick(page_at, ki) + pick(off, ki) * 128 + (lane & 7u) * 16;
        const uint64_t sto = pick(page_at, row) + 8192 + pick(off, row) * 4;
        const bool iput = lane < 32 && ((ok >> ki) & 1u), sput = in == 0 && ((ok >> row) & 1u);
        for (uint32_t r = 0; r < p.replicas; ++r) {
            uint8_t* main = p.s.main_base[r];
            uint8_t* idx = p.s.idx_base[r];
#pragma unroll
            for (uint32_t j = 0; j < 3; ++j)
                if (put[j]) put16<Stream>(main + to[j], piece[j]);
            if (iput) put16<Stream>(idx + ito, ipiece);
            if (sput) *(float*)(idx + sto) = iscale;
        }
    }
}

}  // namespace

hipError_t launch_store_rotated(const StoreRotatedParams& p, hipStream_t stream) {
    (void)hipGetLastError();
    for (int64_t t = 0; t < p.s.num_tokens; t += kMaxTokensPerLaunch) {
        StoreRotatedParams q = p;
        q.s.num_tokens = p.s.num_tokens - t < kMaxTokensPerLaunch ? p.s.num_tokens - t : kMaxTokensPerLaunch;
        q.s.latent = p.s.latent + t * p.s.latent_stride;
        q.s.rope = p.s.rope + t * p.s.rope_stride;
        q.s.indexer = p.s.indexer + t * p.s.indexer_stride;
        q.s.slots = p.s.slots + t;
        q.positions = p.positions + t;
        const uint32_t groups = (uint32_t)((q.s.num_tokens + 3) / 4);
        if (q.s.num_tokens <= kSmallTokens) store_rotated_kernel<true, false><<<groups, kPieces * 64, 0, stream>>>(q);
        else if (q.s.num_tokens * 788 * q.replicas <= kStreamBytes) store_rotated_kernel<false, false><<<(groups + 3) / 4, 256, 0, stream>>>(q);
        else store_rotated_kernel<false, true><<<(groups + 3) / 4, 256, 0, stream>>>(q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kvpub
