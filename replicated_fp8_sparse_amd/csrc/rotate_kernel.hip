// Rows of heads rotated by their tokens' positions (rotation.h has the angles).
//
// Mathematics.  y1 = m (x1 cos a - x2 sin a), y2 = m (x1 sin a + x2 cos a) for each
// pair; the transpose takes -a.  The magnitude m goes into the sine and cosine.
//
// Mapping.  A thread takes 8 values of a row: 4 pairs, neighbours (one 16-byte load
// of 16-bit values) or 4 of each half (two of 8 bytes), the same in several heads of
// its token, so that a pair's angle is computed once for them.
#include <algorithm>

#include "kvpub.h"
#include "rotation.h"

namespace kvpub {
namespace {

constexpr uint32_t kThreads = 256;

template <class T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// Units before dim/8 rotate 4 pairs, the others copy 8 values around the rotated ones.
// H: heads a thread takes at once.
template <class T, bool Halves, int H>
__global__ __launch_bounds__(kThreads) void rotate_kernel(const RotateParams p) {
    const uint32_t rows = kThreads / p.units;                 // heads that a block takes at once
    const uint32_t row = threadIdx.x / p.units, unit = threadIdx.x - row * p.units;
    const uint32_t turned = p.rotation.dim / 8;
    const uint32_t head0 = blockIdx.x * rows * H + row;
    if (row >= rows || head0 >= p.heads) return;
    const bool copies = unit >= turned;
    // the unit's two groups of 4 values
    uint32_t at0, at1;
    if (copies) {
        at0 = (unit - turned) * 8;
        if (at0 >= p.rotation.start) at0 += p.rotation.dim;
        at1 = at0 + 4;
    } else if (Halves) {
        at0 = p.rotation.start + unit * 4;
        at1 = at0 + p.rotation.dim / 2;
    } else {
        at0 = p.rotation.start + unit * 8;
        at1 = at0 + 4;
    }
    uint64_t turns[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) turns[i] = copies ? 0 : p.rotation.turns[unit * 4 + i];
    for (uint32_t t = blockIdx.y; t < p.num_tokens; t += gridDim.y) {
        const T* x = (const T*)p.x + (int64_t)t * p.x_token;
        T* y = (T*)p.y + (int64_t)t * p.y_token;
        Vec<T, 4> a[H], b[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const uint32_t head = head0 + h * rows < p.heads ? head0 + h * rows : head0;
            const T* r = x + (int64_t)head * p.x_head;
            a[h] = *(const Vec<T, 4>*)(r + at0);
            b[h] = *(const Vec<T, 4>*)(r + at1);
        }
        float c[4], s[4];
        const int32_t pos = p.positions[t];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Turn w = turn_of(pos, turns[i]);
            c[i] = w.c * p.rotation.magnitude;
            s[i] = w.s * p.sign;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (head0 + h * rows >= p.heads) break;
            if (!copies) {
                float u[8], v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = (float)a[h].v[i], u[4 + i] = (float)b[h].v[i];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = Halves ? i : 2 * i, k = Halves ? i + 4 : 2 * i + 1;
                    v[j] = turned_first(u[j], u[k], c[i], s[i]);
                    v[k] = turned_second(u[j], u[k], c[i], s[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) a[h].v[i] = (T)v[i], b[h].v[i] = (T)v[4 + i];
            }
            T* r = y + (int64_t)(head0 + h * rows) * p.y_head;
            *(Vec<T, 4>*)(r + at0) = a[h];
            *(Vec<T, 4>*)(r + at1) = b[h];
        }
    }
}

template <class T, int H>
void launch(const RotateParams& p, hipStream_t stream) {
    const uint32_t rows = kThreads / p.units;
    const uint32_t across = (p.heads + rows * H - 1) / (rows * H);
    const uint32_t most = std::min(65535u, (1u << 23) / across);       // a launch holds fewer than 2^32 threads
    const dim3 grid(across, std::min(p.num_tokens, most));
    if (p.rotation.halves) rotate_kernel<T, true, H><<<grid, kThreads, 0, stream>>>(p);
    else rotate_kernel<T, false, H><<<grid, kThreads, 0, stream>>>(p);
}

template <class T>
void launch(const RotateParams& p, hipStream_t stream) {
    // several heads a thread once that still leaves every compute unit two blocks
    const uint64_t rows = kThreads / p.units;
    if (p.heads >= 4 * rows && (uint64_t)p.num_tokens * (p.heads / (4 * rows)) >= 512) launch<T, 4>(p, stream);
    else launch<T, 1>(p, stream);
}

}  // namespace

hipError_t launch_rotate(const RotateParams& p, hipStream_t stream) {
    (void)hipGetLastError();
    if (p.type == KVPUB_BF16) launch<__bf16>(p, stream);
    else if (p.type == KVPUB_FP16) launch<_Float16>(p, stream);
    else launch<float>(p, stream);
    return hipGetLastError();
}

}  // namespace kvpub
