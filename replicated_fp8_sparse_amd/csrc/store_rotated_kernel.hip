// The latent cache's store with the position rotation on the way: kvpub_store's
// bytes of rows whose RoPE and Indexer-K parts are rotated first (rotation.h).
//
// Mathematics.  Rotated values stay in binary32 until they are stored: RoPE values
// are rounded to bf16 once, Indexer-K values meet their scale and codes unrounded.
// A tile of 128: scale = RN32(amax / 448), code = e4m3fn(RN32(x / scale)), the
// divisions IEEE, so that what is not rotated has the store's bytes.
//
// Mapping.  As the store's: a wave owns 4 tokens, a row of 16 lanes x 8 values is a
// tile; round k < 4 is token k's latent, round 4 the four Indexer-K rows; lanes
// 0..31 carry the RoPE rows.
#include "rotation.h"

namespace kvpub {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;

__device__ __forceinline__ float row_max16(float v) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));    // quad_perm 1,0,3,2
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));    // quad_perm 2,3,0,1
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));   // row_half_mirror
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));  // row_mirror
}

__device__ __forceinline__ void unpack8(u32x4 d, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(d[i] << 16);
        x[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
}

// Codes of the lane's 8 values of a tile, and the tile's scale.
__device__ __forceinline__ u32x2 quantize(const float (&x)[8], float& scale) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    scale = row_max16(m) / 448.0f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = scale == 0.f ? 0.f : x[i] / scale;
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
    }
    return c;
}

__global__ __launch_bounds__(kWaves * 64) void store_rotated_kernel(const StoreRotatedParams p) {
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t T = (uint32_t)p.s.num_tokens, t0 = (blockIdx.x * kWaves + wave) * 4;
    if (t0 >= T) return;
    const uint32_t last = T - 1;
    const CtxHead head = *p.s.head;
    if (head.status & kStatusPoisoned) return;               // a fence timed out: fail closed
    const uint32_t in = lane & 15u, row = lane >> 4;
    // token of the lane's Indexer-K piece and of its RoPE piece
    const uint32_t ti = t0 + row < last ? t0 + row : last;
    const uint32_t rr = (lane >> 3) & 3u, tr = t0 + rr < last ? t0 + rr : last;
    int64_t slot[4];
    u32x4 lat[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t t = t0 + k < last ? t0 + k : last;
        slot[k] = t0 + k <= last ? p.s.slots[t] : -1;
        lat[k] = __builtin_nontemporal_load((const u32x4*)(p.s.latent + (uint64_t)t * p.s.latent_stride + lane * 8));
    }
    const uint16_t* irow = p.s.indexer + (uint64_t)ti * p.s.indexer_stride;
    const uint16_t* rrow = p.s.rope + (uint64_t)tr * p.s.rope_stride;
    // what the lane takes of the rows that turn: 4 pairs (rotation.h)
    const RowUnit ui = row_unit(in, p.indexer.dim, p.indexer.start, p.indexer.halves), ur = row_unit(lane & 7u, p.rope.dim, p.rope.start, p.rope.halves);
    const Row4<__bf16> i0 = *(const Row4<__bf16>*)(irow + ui.at0), i1 = *(const Row4<__bf16>*)(irow + ui.at1);
    const Row4<__bf16> p0 = *(const Row4<__bf16>*)(rrow + ur.at0), p1 = *(const Row4<__bf16>*)(rrow + ur.at1);
    Turns4 ti4, tr4;
    ti4.load(p.indexer.turns, in, ui.turned);
    tr4.load(p.rope.turns, lane & 7u, ur.turned);
    const int32_t pos_i = p.positions[ti], pos_r = p.positions[tr];
    uint32_t bad = 0;
    bool ok[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        ok[k] = (uint64_t)slot[k] < (uint64_t)head.capacity;
        bad += !ok[k] && slot[k] != -1;
    }
    if (bad && lane == 0) atomicAdd(p.s.invalid_count, (unsigned long long)bad);

    u32x2 code[5];
    float scale[5];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x[8];
        unpack8(lat[k], x);
        code[k] = quantize(x, scale[k]);
    }
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)i0.v[i], x[4 + i] = (float)i1.v[i], y[i] = (float)p0.v[i], y[4 + i] = (float)p1.v[i];
    Angles4 angles;
    if (ui.turned) {
        angles.set(pos_i, ti4, p.indexer.magnitude, p.indexer.magnitude);
        angles.turn(x, p.indexer.halves);
    }
    code[4] = quantize(x, scale[4]);
    if (ur.turned) {
        angles.set(pos_r, tr4, p.rope.magnitude, p.rope.magnitude);
        angles.turn(y, p.rope.halves);
    }
    Row4<__bf16> r0, r1;
#pragma unroll
    for (int i = 0; i < 4; ++i) r0.v[i] = (__bf16)y[i], r1.v[i] = (__bf16)y[4 + i];

    uint64_t main_at[4], idx_at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t page = (uint64_t)slot[k] >> 6, off = (uint64_t)slot[k] & 63u;
        main_at[k] = page * p.s.main_page_stride + off * 656u;
        idx_at[k] = page * p.s.idx_page_stride + off * 128u;
    }
    auto pick = [](uint64_t a, uint64_t b, uint64_t c, uint64_t d, uint32_t i) { return i & 2u ? (i & 1u ? d : c) : (i & 1u ? b : a); };
    const uint64_t ri = pick(main_at[0], main_at[1], main_at[2], main_at[3], rr);
    const uint64_t ii = pick(idx_at[0], idx_at[1], idx_at[2], idx_at[3], row);
    const uint64_t si = pick(slot[0] & 63, slot[1] & 63, slot[2] & 63, slot[3] & 63, row);
    const bool ok_r = lane < 32 && (rr & 2u ? (rr & 1u ? ok[3] : ok[2]) : (rr & 1u ? ok[1] : ok[0]));
    const bool ok_i = row & 2u ? (row & 1u ? ok[3] : ok[2]) : (row & 1u ? ok[1] : ok[0]);
    for (uint32_t r = 0; r < p.replicas; ++r) {
        uint8_t* main = p.s.main_base[r];
        uint8_t* idx = p.s.idx_base[r];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (ok[k]) {
                *(u32x2*)(main + main_at[k] + lane * 8) = code[k];
                if (in == 0) *(float*)(main + main_at[k] + 512 + row * 4) = scale[k];
            }
        if (ok_r) {
            *(Row4<__bf16>*)(main + ri + 528 + ur.at0 * 2) = r0;
            *(Row4<__bf16>*)(main + ri + 528 + ur.at1 * 2) = r1;
        }
        if (ok_i) {
            *(uint32_t*)(idx + ii + ui.at0) = code[4].x;
            *(uint32_t*)(idx + ii + ui.at1) = code[4].y;
            if (in == 0) *(float*)(idx + ii + 8192 + si * 4 - si * 128) = scale[4];
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
        store_rotated_kernel<<<(uint32_t)((q.s.num_tokens + 4 * kWaves - 1) / (4 * kWaves)), kWaves * 64, 0, stream>>>(q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kvpub
