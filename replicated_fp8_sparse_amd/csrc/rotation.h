// Rotary positions in device code: the angle of a pair, its sine and cosine, and
// 8 values of a row rotated.
//
// An angle is position * turns modulo 2^64 in units of 2^-64 turns, where turns is
// the pair's frequency: one 64-bit product, exact, so a position of a million is
// as good as the first (in binary32 the angle itself would be off by 0.03).  Its
// high 32 bits, as a signed part of a turn, go to the vector unit's sine and cosine, which
// take turns: both within 3.2 * 2^-24 of the exact values (measured over 2^28 angles), a
// third of the instructions of a reduction and two polynomials.
#pragma once

#include "kvpub_internal.h"

namespace kvpub {

struct Turn {
    float c;     // cosine
    float s;     // sine
};

__device__ __forceinline__ Turn turn_of(int32_t position, uint64_t turns) {
    // the product's high word: two 32-bit products, and the sign's part of the low one
    const uint32_t lo = (uint32_t)turns, hi = (uint32_t)(turns >> 32);
    const uint32_t u = __umulhi((uint32_t)position, lo) + (uint32_t)position * hi - (position < 0 ? lo : 0u);
    const float x = (float)(int32_t)u * 0x1p-32f;
    return Turn{__builtin_amdgcn_cosf(x), __builtin_amdgcn_sinf(x)};
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
