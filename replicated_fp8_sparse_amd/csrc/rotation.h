// Rotary positions in device code: the angle of a pair, its sine and cosine, and
// 8 values of a row rotated.
//
// An angle is position * turns modulo 2^64 in units of 2^-64 turns, where turns is
// the pair's frequency: one 64-bit product, exact, so a position of a million is
// as good as the first (in binary32 the angle itself would be off by 0.03).  Its
// high 32 bits, rounded, are the nearest quarter turn and a signed rest of at most
// an eighth; sine and cosine of the rest are Taylor's polynomials in Horner's form,
// up to x^9 and x^10: what is cut off stays below 2^-29.
#pragma once

#include "kvpub_internal.h"

namespace kvpub {

struct Turn {
    float c;     // cosine
    float s;     // sine
};

__device__ __forceinline__ Turn turn_of(int32_t position, uint64_t turns) {
    const uint64_t a = (uint64_t)(int64_t)position * turns;
    const uint32_t u = (uint32_t)((a + (1ull << 31)) >> 32);
    const uint32_t quarter = (u + (1u << 29)) >> 30;
    const int32_t rest = (int32_t)(u - (quarter << 30));              // -2^29 .. 2^29 - 1
    const float x = (float)rest * 1.46291807926715968e-09f;           // 2 pi / 2^32
    const float z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    // quarters 1 and 3 exchange the two; the cosine is negative in quarters 1 and 2, the sine in 2 and 3
    const float cc = quarter & 1u ? s : c, ss = quarter & 1u ? c : s;
    Turn t;
    t.c = __uint_as_float(__float_as_uint(cc) ^ (((quarter + 1u) & 2u) << 30));
    t.s = __uint_as_float(__float_as_uint(ss) ^ ((quarter & 2u) << 30));
    return t;
}

// Pair (u, v) turned: the first and the second value.  c and s hold the magnitude.
__device__ __forceinline__ float turned_first(float u, float v, float c, float s) { return fmaf(u, c, -(v * s)); }
__device__ __forceinline__ float turned_second(float u, float v, float c, float s) { return fmaf(u, s, v * c); }

// x, the values e0 .. e0+7 of `row` (e0 a multiple of 8), rotated where the
// rotation covers them.  Halves: a value's partner lies half the rotated part away
// and is read from the row again.
template <class T>
__device__ __forceinline__ void rotate8(float (&x)[8], const T* row, uint32_t e0, int32_t position, const RotationParams& r) {
#pragma unroll
    for (uint32_t g = 0; g < 2; ++g) {
        const uint32_t rel = e0 + 4 * g - r.start;
        if (rel >= r.dim) continue;                       // also where e0 + 4 g < start
        if (r.halves) {
            const uint32_t half = r.dim / 2;
            const bool second = rel >= half;
            const uint32_t pair = second ? rel - half : rel;
            const T* other = row + r.start + (second ? pair : pair + half);
            T w[4];
            __builtin_memcpy(w, __builtin_assume_aligned(other, 4 * sizeof(T)), sizeof w);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const Turn t = turn_of(position, r.turns[pair + i]);
                const float c = t.c * r.magnitude, s = t.s * r.magnitude, o = (float)w[i], m = x[4 * g + i];
                x[4 * g + i] = second ? turned_second(o, m, c, s) : turned_first(m, o, c, s);
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                const Turn t = turn_of(position, r.turns[rel / 2 + i]);
                const float c = t.c * r.magnitude, s = t.s * r.magnitude, u = x[4 * g + 2 * i], v = x[4 * g + 2 * i + 1];
                x[4 * g + 2 * i] = turned_first(u, v, c, s);
                x[4 * g + 2 * i + 1] = turned_second(u, v, c, s);
            }
        }
    }
}

}  // namespace kvpub
