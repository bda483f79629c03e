// Rows of heads rotated by their tokens' positions (rotation.h has the angles).
//
// Mathematics.  y1 = m (x1 cos a - x2 sin a), y2 = m (x1 sin a + x2 cos a) for each
// pair; the transpose takes -a.  The magnitude m goes into the sine and cosine.
//
// Mapping.  A thread takes 8 values of a row: 4 pairs, neighbours (one 16-byte load
// of 16-bit values) or 4 of each half (two of 8 bytes), the same in several heads of
// its token, so that a pair's angle is computed once for them.
//
// Bound.  Memory: 8192 tokens of 128 heads, 64 of 192 values rotated, bf16 55.7 us, 3000 of 32
// heads of 128, 48 rotated, binary32 20.0: a large copy's 5.16 TB/s would leave 52 and 19.  One token: a
// launch and two dependent reads, 2.9 us.
#include <algorithm>

#include "kvpub.h"
#include "rotation.h"

namespace kvpub {
namespace {

constexpr uint32_t kThreads = 256;

// H: heads a thread takes at once.
template <class T, bool Halves, int H>
__global__ __launch_bounds__(kThreads) void rotate_kernel(const RotateParams p) {
    const uint32_t rows = p.across;
    const uint32_t row = threadIdx.x / p.units, unit = threadIdx.x - row * p.units, token = row / rows;
    const uint32_t head0 = blockIdx.x * rows * H + row - token * rows;
    if (token >= p.tokens || head0 >= p.heads) return;
    const RowUnit u = row_unit(unit, p.rotation.dim, p.rotation.start, Halves);
    Turns4 turns;
    turns.load(p.rotation.turns, unit, u.turned);
    for (uint32_t t = blockIdx.y * p.tokens + token; t < p.num_tokens; t += gridDim.y * p.tokens) {
        const T* x = (const T*)p.x + (int64_t)t * p.x_token;
        T* y = (T*)p.y + (int64_t)t * p.y_token;
        Row4<T> a[H], b[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const uint32_t head = head0 + h * rows < p.heads ? head0 + h * rows : head0;
            const T* r = x + (int64_t)head * p.x_head;
            a[h] = *(const Row4<T>*)(r + u.at0);
            b[h] = *(const Row4<T>*)(r + u.at1);
        }
        Angles4 angles;
        angles.set(p.positions[t], turns, p.rotation.magnitude, p.sign);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (head0 + h * rows >= p.heads) break;
            if (u.turned) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = (float)a[h].v[i], w[4 + i] = (float)b[h].v[i];
                angles.turn(w, Halves);
                // a sum is rounded to binary32 before its type: joined with the conversion in some places and not in others,
                // one value would have different bits in different heads
                if constexpr (__is_same(T, _Float16)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) asm("" : "+v"(w[i]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) a[h].v[i] = (T)w[i], b[h].v[i] = (T)w[4 + i];
            }
            T* r = y + (int64_t)(head0 + h * rows) * p.y_head;
            *(Row4<T>*)(r + u.at0) = a[h];
            *(Row4<T>*)(r + u.at1) = b[h];
        }
    }
}

template <class T, int H>
void launch(const RotateParams& p, hipStream_t stream) {
    const uint32_t across = (p.heads + p.across * H - 1) / (p.across * H);
    const uint32_t most = std::min(65535u, (1u << 23) / across);       // a launch holds fewer than 2^32 threads
    const dim3 grid(across, std::min((p.num_tokens + p.tokens - 1) / p.tokens, most));
    if (p.rotation.halves) rotate_kernel<T, true, H><<<grid, kThreads, 0, stream>>>(p);
    else rotate_kernel<T, false, H><<<grid, kThreads, 0, stream>>>(p);
}

template <class T>
void launch(RotateParams p, hipStream_t stream) {
    const uint32_t rows = kThreads / p.units;
    // four heads a thread, which share its angles, once that still leaves every compute unit two blocks
    // (4096 tokens of 32 heads of 128, bf16: 13.2 us for 16.8; in 32 bits the bytes bound it: 28.5 for 27.4)
    constexpr bool kMayFour = sizeof(T) == 2;
    const bool four = kMayFour && p.heads >= 4 && (uint64_t)p.num_tokens * ((p.heads + 3) / 4) >= 512 * rows;
    p.across = std::min(four ? (p.heads + 3) / 4 : p.heads, rows);
    p.tokens = rows / p.across;
    if constexpr (kMayFour)
        if (four) return launch<T, 4>(p, stream);
    launch<T, 1>(p, stream);
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
