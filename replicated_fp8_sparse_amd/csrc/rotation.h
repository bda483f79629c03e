// Rotary positions in device code: the angle of a pair, its sine and cosine, and
// 8 values of a row rotated.
//
// An angle is position * turns modulo 2^64 in units of 2^-64 turns, where turns is
// the pair's frequency: one 64-bit product, exact, so a position of a million is
// as good as the first (in binary32 the angle itself would be off by 0.03).  Its
// high 32 bits, rounded, are the nearest quarter turn and a signed rest of at most an eighth;
// sine and cosine of the rest are Taylor's polynomials in Horner's form, up to x^9 and
// x^10: what is cut off stays below 2^-29.  With the roundings of x and of the last step the two are off by up to
// 1.7 * 2^-24, over 2^22 angles by 2.9e-8 in the mean square where the nearest numbers are by 2.1e-8; a rotated value, which
// fuses its second product, by as much as from the nearest ones without that.  (The vector unit's own sine and cosine take
// turns at a third of the instructions, but are off by up to 3.1 * 2^-24, measured over 2^28
// angles: several times as many values rounded to the wrong neighbour, for 20 % of a long
// append's time and less elsewhere.)
#pragma once

#include "kvpub_internal.h"

namespace kvpub {

struct Turn {
    float c;     // cosine
    float s;     // sine
};

__device__ __forceinline__ Turn turn_of(int32_t position, uint64_t turns) {
    // the product's high word, rounded by the bit below it: two 32-bit products, and the sign's part of the low one
    const uint32_t lo = (uint32_t)turns, hi = (uint32_t)(turns >> 32);
    const uint32_t u = (uint32_t)(((uint64_t)(uint32_t)position * lo + 0x80000000u) >> 32) + (uint32_t)position * hi - (position < 0 ? lo : 0u);
    // the nearest quarter is the two high bits of u + an eighth; the low 30 bits of u, as a signed number, are the rest
    const uint32_t w = u + (1u << 29);
    const float x = (float)(int32_t)(u << 2) * 3.65729519816789921e-10f;       // 2 pi / 2^34
    const float z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    // quarters 1 and 3 exchange the two; the cosine is negative in quarters 1 and 2, the sine in 2 and 3
    const bool odd = (w & (1u << 30)) != 0;
    Turn t;
    t.c = __uint_as_float(__float_as_uint(odd ? s : c) ^ ((w + (1u << 30)) & (1u << 31)));
    t.s = __uint_as_float(__float_as_uint(odd ? c : s) ^ (w & (1u << 31)));
    return t;
}

// Pair (u, v) turned: the first and the second value.  c and s hold the magnitude.
__device__ __forceinline__ float turned_first(float u, float v, float c, float s) { return fmaf(u, c, -(v * s)); }
__device__ __forceinline__ float turned_second(float u, float v, float c, float s) { return fmaf(u, s, v * c); }

// Eight values of a row that one lane takes: two groups of 4, which are 4 pairs
// where the rotation covers them.  Units below dim/8 are its pairs in order (neighbours:
// 8 values in a row; halves: 4 of each half), the others what lies around them.
struct RowUnit {
    uint32_t at0, at1;       // first values of the groups
    bool turned;
};
__device__ __forceinline__ RowUnit row_unit(uint32_t unit, uint32_t dim, uint32_t start, bool halves) {
    RowUnit u;
    u.turned = unit < dim / 8;
    if (!u.turned) {
        u.at0 = (unit - dim / 8) * 8;
        if (u.at0 >= start) u.at0 += dim;
        u.at1 = u.at0 + 4;
    } else {
        u.at0 = start + unit * (halves ? 4 : 8);
        u.at1 = u.at0 + (halves ? dim / 2 : 4);
    }
    return u;
}

// The frequencies of a unit's pairs, the sines and cosines at a position, and the pairs turned.
struct Turns4 {
    uint64_t f[4];
    __device__ __forceinline__ void load(const uint64_t* turns, uint32_t unit, bool turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = turned ? turns[unit * 4 + i] : 0;
    }
};
struct Angles4 {
    float c[4], s[4];
    __device__ __forceinline__ void set(int32_t position, const Turns4& t, float magnitude, float sign) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Turn w = turn_of(position, t.f[i]);
            c[i] = w.c * magnitude;
            s[i] = w.s * sign;
        }
    }
    // x: the unit's first group, then the second
    __device__ __forceinline__ void turn(float (&x)[8], bool halves) const {
        float y[8];
        if (halves) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = turned_first(x[i], x[4 + i], c[i], s[i]);
                y[4 + i] = turned_second(x[i], x[4 + i], c[i], s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = turned_first(x[2 * i], x[2 * i + 1], c[i], s[i]);
                y[2 * i + 1] = turned_second(x[2 * i], x[2 * i + 1], c[i], s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i];
    }
};

// Four values of a row.
template <class T>
struct alignas(4 * sizeof(T)) Row4 {
    T v[4];
};

}  // namespace kvpub
