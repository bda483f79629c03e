// Attention over the replicated cache of key and value heads (e4m3 codes, a
// power-of-two scale for each block of 64 positions and head).
//
// Mathematics.  With codes c and d of a block's keys and values and its scales a, b,
//   score = (scale * a) (q . c),   out = sum_p w_p (b d_p) / sum_p w_p.
// A code is exact in bf16 and fp16, and so is a value's code times its scale in
// bf16: nothing of the cache is rounded again.  Weights are rounded to bf16 for the
// second product (their low parts follow as a second operand for fp16 outputs,
// whose own step is finer).  One pass: a row's running maximum moves only when a
// score exceeds it by more than 2^8, so most tiles neither rescale nor shuffle.
//
// Mapping.  Rows are (token, query head) pairs that share a key-value head: a unit
// is 16 RT of them and one key-value head.  Scores come out transposed: positions
// down, rows across, so that a lane holds 8 positions of one row, and its weights
// are an operand of the second product as they are if the values' positions come in the
// same order.  Values are read by position, 16 lanes a row, and brought to columns by
// byte permutes within a lane: no LDS before the end.  The 4 waves of a block take
// every 4th tile of 32 positions, each from memory straight to registers one
// tile ahead, and join their parts through LDS; long sequences are cut into chunks
// for several blocks, which join_kernel joins in order.
#include <algorithm>
#include <cfloat>

#include "kvpub.h"
#include "sequences.h"

namespace kvpub {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kThreads = 256, kWaves = 4;
constexpr uint32_t kTile = 32;                    // positions of a wave's step
constexpr float kLazy = 8.0f;                     // rescale when a maximum grows past 2^8
constexpr float kLn2 = 0.693147180559945309f;

template <class E> struct Operand;
template <> struct Operand<__bf16> {
    typedef bf16x8 x8;
    static __device__ __forceinline__ x8 widen(int c0, int c1) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, true);
        return x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
    static __device__ __forceinline__ f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Operand<_Float16> {
    typedef f16x8 x8;
    static __device__ __forceinline__ x8 widen(int c0, int c1) {
        const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, 1.0f, true);
        const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, 1.0f, true);
        return x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
    static __device__ __forceinline__ f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// A unit of work and what its rows see.
struct Unit {
    SeqOf s;
    int64_t base;            // position of the sequence's first token
    uint32_t row0;           // the unit's first row
    uint32_t rows;           // rows of the sequence
    uint32_t reach;          // positions that any row of the unit may see
    uint32_t chunks;         // cuts that hold some of them, at least 1
};

__device__ __forceinline__ Unit unit_of(const HeadsAttendParams& p, const Places& w, uint32_t place, uint32_t R) {
    Unit u;
    u.s = find_sequence(p.seqs, place, w);
    u.rows = u.s.m * p.group;
    u.row0 = u.s.place * R;
    if (!u.s.found || u.row0 >= u.rows) {
        u.rows = 0;
        return u;
    }
    u.base = (int64_t)u.s.kv - u.s.n;
    const uint32_t last = (u.row0 + R < u.rows ? u.row0 + R : u.rows) - 1;
    const int64_t lim = u.base + last / p.group + 1;
    u.reach = p.tree ? u.s.kv : (lim > 0 ? (uint32_t)lim : 0u);
    u.chunks = u.reach ? (u.reach + p.chunk - 1) / p.chunk : 1u;
    return u;
}

// 64 bits of a tree row from node j on (j below 0: the positions before the tree, seen by all).
__device__ __forceinline__ uint64_t tree_bits(const uint64_t* row, uint32_t words, int64_t j) {
    if (j < 0) {
        if (j <= -64) return ~0ull;
        return (row[0] << (-j)) | ((1ull << (-j)) - 1);
    }
    const uint64_t i = (uint64_t)j >> 6;
    const uint32_t s = (uint32_t)j & 63u;
    const uint64_t a = i < words ? row[i] : 0ull;
    if (s == 0) return a;
    const uint64_t b = i + 1 < words ? row[i + 1] : 0ull;
    return (a >> s) | (b << (64 - s));
}

// Some token of the sequence sees one of the 64 positions from pos on (the whole wave asks).
__device__ __forceinline__ bool any_sees(const HeadsAttendParams& p, const Unit& u, uint32_t pos) {
    if ((int64_t)pos < u.base || !p.tree) return true;
    const uint32_t left = u.s.kv - pos;
    const uint64_t real = left >= 64 ? ~0ull : (1ull << left) - 1;
    bool sees = false;
    for (uint32_t i = threadIdx.x & 63u; i < u.s.m; i += 64)
        sees |= (tree_bits(p.tree + (uint64_t)(u.s.q0 + i) * p.tree_words, p.tree_words, (int64_t)pos - u.base) & real) != 0;
    return __any(sees);
}

// The codes of a tile of 32 positions in one wave's registers.
template <int D>
struct Tile {
    i32x4 k[2][D / 64];              // position 16 u + l%16, values 64 c + 16 (l/16) ..
    uint32_t v[8][D / 64];           // position j of this lane group, values (D/16) (l%16) ..
    uint32_t scales;                 // bytes of the keys and of the values

    __device__ __forceinline__ void load(const uint8_t* page, uint32_t head, uint32_t groups, uint32_t half, uint32_t l16, uint32_t g4) {
        const uint8_t* kp = page + (uint64_t)head * 128 * D + half * (kTile * D);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) k[u][c] = *(const i32x4*)(kp + (u * 16 + l16) * D + c * 64 + g4 * 16);
        const uint8_t* vp = kp + 64 * D;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint8_t* a = vp + ((j >> 2) * 16 + g4 * 4 + (j & 3)) * D + l16 * (D / 16);
            if constexpr (D == 64) v[j][0] = *(const uint32_t*)a;
            else if constexpr (D == 128) {
                const u32x2 w = *(const u32x2*)a;
                v[j][0] = w.x, v[j][1] = w.y;
            } else {
                const u32x4 w = *(const u32x4*)a;
                v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
            }
        }
        const uint32_t at = 2 * head;
        scales = *(const uint32_t*)(page + (uint64_t)groups * 128 * D + (at & ~3u)) >> ((at & 2u) * 8);
    }
    static __device__ __forceinline__ float power(uint32_t byte) {
        const uint32_t b = byte < 1 ? 1u : (byte > 245 ? 245u : byte);
        return __uint_as_float(b << 23);
    }
    __device__ __forceinline__ float key_scale() const { return power(scales & 255u); }
    __device__ __forceinline__ float value_scale() const { return power((scales >> 8) & 255u); }
};

template <class E, int D, int RT>
__global__ __launch_bounds__(kThreads, D * RT <= 128 ? 3 : (D * RT <= 256 ? 2 : 1)) void heads_attend_kernel(const HeadsAttendParams p, const Places places) {
    typedef Operand<E> Op;
    constexpr uint32_t R = 16 * RT;
    constexpr int NB = D / 16;
    __shared__ float obuf[kWaves][16][D + 4];
    __shared__ float ml[kWaves][16][2];
    const uint32_t G = p.heads.groups, tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t l16 = lane & 15u, g4 = lane >> 4;
    const uint32_t g = blockIdx.x % G, rest = blockIdx.x / G, cut = rest % p.chunks, place = rest / p.chunks;
    const Unit u = unit_of(p, places, p.first + place, R);
    if (u.rows == 0 || cut >= u.chunks) return;

    // queries, and what each row sees: positions below lim (tree: of those before the tree, then its bits)
    typename Op::x8 q[RT][D / 32];
    uint32_t lim[RT];
    const uint64_t* tree[RT];
    uint32_t least = 0xFFFFFFFFu;          // positions that all rows see
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const uint32_t row = u.row0 + r * 16 + l16;
        const bool is = row < u.rows;
        const uint32_t i = is ? row / p.group : 0u, h = g * p.group + (is ? row - i * p.group : 0u);
        const E* src = (const E*)p.q + (int64_t)(u.s.q0 + i) * p.q_token + (int64_t)h * p.q_head + g4 * 16;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            if (is) q[r][c] = *(const typename Op::x8*)(src + (c >> 1) * 64 + (c & 1) * 8);
            else q[r][c] = typename Op::x8{};
        }
        const int64_t top = u.base + (p.tree ? 0 : (int64_t)i + 1);
        lim[r] = is ? (top > 0 ? (uint32_t)top : 0u) : 0xFFFFFFFFu;
        tree[r] = p.tree && is ? p.tree + (uint64_t)(u.s.q0 + i) * p.tree_words : nullptr;
        least = lim[r] < least ? lim[r] : least;
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
        const uint32_t o = __shfl_xor(least, d);
        least = o < least ? o : least;
    }
    least = __builtin_amdgcn_readfirstlane(least);
    least = least < u.s.kv ? least : u.s.kv;

    f32x4 o[RT][NB];
    float m[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        m[r] = -FLT_MAX, l[r] = 0.f;
#pragma unroll
        for (int n = 0; n < NB; ++n) o[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t* table = p.seqs.pages + (int64_t)u.s.b * p.seqs.pages_stride;
    const uint32_t end = u.reach < (cut + 1) * p.chunk ? u.reach : (cut + 1) * p.chunk;
    const uint32_t last = (end + kTile - 1) / kTile;
    const bool counts = g == 0 && u.row0 + R >= u.rows;
    auto page_of = [&](uint32_t t) { return t < last ? __builtin_amdgcn_readfirstlane(table[t >> 1]) : 0; };
    auto at = [&](int32_t page) { return p.base + ((uint32_t)page < p.heads.num_pages ? (uint64_t)(uint32_t)page * p.heads.page_stride : 0ull); };

    uint32_t t = cut * (p.chunk / kTile) + wave;
    int32_t page = page_of(t), page1 = page_of(t + kWaves);
    Tile<D> cur;
    if (t < last) cur.load(at(page), g, G, t & 1u, l16, g4);
    while (t < last) {
        Tile<D> next = cur;
        if (t + kWaves < last) next.load(at(page1), g, G, t & 1u, l16, g4);
        const int32_t page2 = page_of(t + 2 * kWaves);
        const uint32_t pos0 = t * kTile;
        if ((uint32_t)page >= p.heads.num_pages) {
            // hidden; counted by the rows that see most of the sequence, at a page's first half
            if (counts && !(t & 1u) && any_sees(p, u, pos0) && lane == 0) atomicAdd(p.invalid_count, 1ull);
        } else {
            float x[RT][8];
            {
                f32x4 s[RT][2];
#pragma unroll
                for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const typename Op::x8 a = Op::widen(cur.k[j][c][2 * h], cur.k[j][c][2 * h + 1]);
#pragma unroll
                            for (int r = 0; r < RT; ++r) s[r][j] = Op::mfma(a, q[r][2 * c + h], s[r][j]);
                        }
                const float ks = p.scale_log2 * cur.key_scale();
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[r][j] = s[r][j >> 2][j & 3] * ks;
            }
            if (pos0 + kTile > least) {
                // some row does not see the whole tile.  Bit j: this lane's position j
                uint32_t nan = 0, seen[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint32_t bits = 0xFFFFFFFFu;
                    if (tree[r]) bits = (uint32_t)tree_bits(tree[r], p.tree_words, (int64_t)pos0 - u.base);
                    seen[r] = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t at = (j >> 2) * 16 + g4 * 4 + (j & 3), pos = pos0 + at;
                        const bool sees = pos < u.s.kv && (p.tree ? ((bits >> at) & 1u) != 0 : pos < lim[r]);
                        seen[r] |= sees ? 1u << j : 0u;
                        x[r][j] = sees ? x[r][j] : -INFINITY;
                    }
                }
                // values that do not exist become zeros, and so do rows that hold a NaN code,
                // with a NaN score for who sees them: a weight of 0 does not hide a NaN
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool is = pos0 + (j >> 2) * 16 + g4 * 4 + (j & 3) < u.s.kv;
#pragma unroll
                    for (int w = 0; w < D / 64; ++w) {
                        cur.v[j][w] = is ? cur.v[j][w] : 0u;
                        nan |= (((cur.v[j][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) ? 1u << j : 0u;
                    }
                }
                if (__any(nan)) {
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) nan |= __shfl_xor(nan, d);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if ((nan >> j) & 1u) {
#pragma unroll
                            for (int w = 0; w < D / 64; ++w) cur.v[j][w] = 0;
#pragma unroll
                            for (int r = 0; r < RT; ++r) x[r][j] = (seen[r] >> j) & 1u ? NAN : x[r][j];
                        }
                }
            }
            bool grows = false;
            float high[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                high[r] = fmaxf(fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3])), fmaxf(fmaxf(x[r][4], x[r][5]), fmaxf(x[r][6], x[r][7])));
                grows |= high[r] > m[r] + kLazy;
            }
            if (__any(grows)) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    high[r] = fmaxf(high[r], __shfl_xor(high[r], 16));
                    high[r] = fmaxf(high[r], __shfl_xor(high[r], 32));
                    const float to = high[r] > m[r] + kLazy ? high[r] : m[r], f = exp2f(m[r] - to);
                    m[r] = to;
                    l[r] *= f;
#pragma unroll
                    for (int n = 0; n < NB; ++n) o[r][n] *= f;
                }
            }
            bf16x8 w[RT], low[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float e = __builtin_amdgcn_exp2f(x[r][j] - m[r]);
                    sum += e;
                    w[r][j] = (__bf16)e;
                    if constexpr (sizeof(E) == 2 && !__is_same(E, __bf16)) low[r][j] = (__bf16)(e - (float)w[r][j]);
                }
                l[r] += sum;
            }
            const float vs = cur.value_scale();
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                bf16x8 a[4];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const int lo = (int)__builtin_amdgcn_perm(cur.v[j + 1][c], cur.v[j][c], 0x05010400u);
                    const int hi = (int)__builtin_amdgcn_perm(cur.v[j + 1][c], cur.v[j][c], 0x07030602u);
                    const bf16x2 b0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, vs, false), b1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, vs, true);
                    const bf16x2 b2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, vs, false), b3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, vs, true);
                    a[0][j] = b0.x, a[0][j + 1] = b0.y, a[1][j] = b1.x, a[1][j + 1] = b1.y;
                    a[2][j] = b2.x, a[2][j + 1] = b2.y, a[3][j] = b3.x, a[3][j + 1] = b3.y;
                }
#pragma unroll
                for (int d = 0; d < 4; ++d)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        o[r][4 * c + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[d], w[r], o[r][4 * c + d], 0, 0, 0);
                        if constexpr (!__is_same(E, __bf16))
                            o[r][4 * c + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[d], low[r], o[r][4 * c + d], 0, 0, 0);
                    }
            }
        }
        cur = next;
        page = page1;
        page1 = page2;
        t += kWaves;
    }

    // the waves' parts, 16 rows at a time
    const uint32_t row = tid >> 4, seg = (tid & 15u) * NB;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (u.row0 + r * 16 >= u.rows) break;
        l[r] += __shfl_xor(l[r], 16);
        l[r] += __shfl_xor(l[r], 32);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n) obuf[wave][l16][(g4 * 4 + i) * NB + n] = o[r][n][i];
        if (g4 == 0) ml[wave][l16][0] = m[r], ml[wave][l16][1] = l[r];
        __syncthreads();
        const uint32_t mine = u.row0 + r * 16 + row;
        if (mine < u.rows) {
            float top = ml[0][row][0], sum = 0.f, acc[NB];
#pragma unroll
            for (uint32_t w = 1; w < kWaves; ++w) top = fmaxf(top, ml[w][row][0]);
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[n] = 0.f;
#pragma unroll
            for (uint32_t w = 0; w < kWaves; ++w) {
                const float f = exp2f(ml[w][row][0] - top);
                sum = fmaf(ml[w][row][1], f, sum);
#pragma unroll
                for (int n = 0; n < NB; ++n) acc[n] = fmaf(obuf[w][row][seg + n], f, acc[n]);
            }
            if (u.chunks > 1) {
                const uint64_t slot = (((uint64_t)place * G + g) * p.chunks + cut) * R + r * 16 + row;
#pragma unroll
                for (int n = 0; n < NB; ++n) p.part[slot * D + seg + n] = acc[n];
                if (seg == 0) p.part_ml[slot * 2] = top, p.part_ml[slot * 2 + 1] = sum;
            } else {
                const uint32_t i = mine / p.group, h = g * p.group + mine - i * p.group;
                E* dst = (E*)p.out + (int64_t)(u.s.q0 + i) * p.out_token + (int64_t)h * p.out_head + seg;
                const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int n = 0; n < NB; ++n) dst[n] = (E)(acc[n] * f);
                if (seg == 0 && p.lse) p.lse[(int64_t)(u.s.q0 + i) * p.lse_token + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            }
        }
        __syncthreads();
    }
}

// The parts of units that several blocks cut, joined in their order.
template <class E, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(const HeadsAttendParams p, const Places places, uint32_t R) {
    constexpr int NB = D / 16;
    const uint32_t G = p.heads.groups, g = blockIdx.x % G, place = blockIdx.x / G;
    const Unit u = unit_of(p, places, p.first + place, R);
    if (u.rows == 0 || u.chunks <= 1) return;
    const uint32_t seg = (threadIdx.x & 15u) * NB;
    for (uint32_t r = threadIdx.x >> 4; r < R && u.row0 + r < u.rows; r += 16) {
        const uint64_t slot = ((uint64_t)place * G + g) * p.chunks * R + r;
        float top = -FLT_MAX, sum = 0.f, acc[NB];
        for (uint32_t c = 0; c < u.chunks; ++c) top = fmaxf(top, p.part_ml[(slot + (uint64_t)c * R) * 2]);
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[n] = 0.f;
        for (uint32_t c = 0; c < u.chunks; ++c) {
            const uint64_t s = slot + (uint64_t)c * R;
            const float f = exp2f(p.part_ml[s * 2] - top);
            sum = fmaf(p.part_ml[s * 2 + 1], f, sum);
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[n] = fmaf(p.part[s * D + seg + n], f, acc[n]);
        }
        const uint32_t mine = u.row0 + r, i = mine / p.group, h = g * p.group + mine - i * p.group;
        E* dst = (E*)p.out + (int64_t)(u.s.q0 + i) * p.out_token + (int64_t)h * p.out_head + seg;
        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int n = 0; n < NB; ++n) dst[n] = (E)(acc[n] * f);
        if (seg == 0 && p.lse) p.lse[(int64_t)(u.s.q0 + i) * p.lse_token + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// Blocks that a launch is cut for, by the rows of a unit: what the card holds at once, twice.
uint64_t wanted_blocks(uint32_t rows) { return 32768 / rows; }

Places unit_places(uint32_t rows, uint32_t group, uint64_t num_seqs, uint64_t num_tokens, uint64_t max_q, uint64_t* total) {
    uint32_t shift = 0;
    while ((1u << shift) < rows) ++shift;
    return places(group, shift, 1, (max_q * group + rows - 1) / rows, num_seqs, num_tokens, total);
}

template <class E, int D, int RT>
hipError_t launch(HeadsAttendParams p, const Places& w, hipStream_t stream) {
    const uint32_t G = p.heads.groups, total = p.units;
    const uint32_t most = std::max<uint32_t>(1, ((1u << 24) - 1) / (G * p.chunks));     // a launch holds fewer than 2^32 threads
    for (uint64_t first = 0; first < total; first += most) {
        p.first = (uint32_t)first;
        p.units = (uint32_t)std::min<uint64_t>(most, total - first);
        heads_attend_kernel<E, D, RT><<<p.units * G * p.chunks, kThreads, 0, stream>>>(p, w);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (p.chunks > 1) {
            join_kernel<E, D><<<p.units * G, kThreads, 0, stream>>>(p, w, 16 * RT);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

template <class E, int D>
hipError_t launch(const HeadsAttendParams& p, const Places& w, uint32_t rows, hipStream_t stream) {
    if (rows == 16) return launch<E, D, 1>(p, w, stream);
    if (rows == 32 || D == 256) return launch<E, D, 2>(p, w, stream);
    if constexpr (D < 256) return launch<E, D, 4>(p, w, stream);
    return hipErrorInvalidValue;
}

}  // namespace

HeadsAttendPlan plan_heads_attend(const HeadsParams& h, uint32_t group, uint64_t num_seqs, uint64_t num_tokens, uint64_t max_q,
                                  uint64_t max_kv) {
    HeadsAttendPlan a;
    const uint64_t rows = max_q * group;
    a.rows = rows <= 16 ? 16 : (rows <= 32 || h.dim == 256 ? 32 : 64);
    (void)unit_places(a.rows, group, num_seqs, num_tokens, max_q, &a.units);
    const uint64_t most = std::max<uint64_t>(1, (max_kv + 127) / 128), blocks = a.units * h.groups;
    const uint64_t cuts = std::max<uint64_t>(1, std::min(most, wanted_blocks(a.rows) / std::max<uint64_t>(1, blocks)));
    a.chunk = (uint32_t)std::max<uint64_t>(128, ((max_kv + cuts - 1) / cuts + 127) / 128 * 128);
    a.chunks = (uint32_t)std::max<uint64_t>(1, (max_kv + a.chunk - 1) / a.chunk);
    // parts of as many rows as the wanted blocks hold, or as the bounds allow: either grows with every bound
    const uint64_t parts = std::min(wanted_blocks(a.rows) * a.rows, (num_tokens * group + num_seqs * a.rows) * h.groups * most);
    a.bytes = parts * (h.dim + 2) * 4;
    return a;
}

hipError_t launch_heads_attend(const HeadsAttendParams& p, void* workspace, hipStream_t stream) {
    (void)hipGetLastError();
    HeadsAttendParams a = p;
    const HeadsAttendPlan plan = plan_heads_attend(p.heads, p.group, p.seqs.num_seqs, p.seqs.num_tokens, p.seqs.max_q, p.seqs.max_kv);
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    uint64_t total;
    const Places w = unit_places(plan.rows, p.group, p.seqs.num_seqs, p.seqs.num_tokens, p.seqs.max_q, &total);
    a.units = (uint32_t)total;
    a.part = static_cast<float*>(workspace);
    a.part_ml = a.part + plan.bytes / 4 / (p.heads.dim + 2) * p.heads.dim;
    const bool half = p.type == KVPUB_FP16;
    if (p.heads.dim == 64) return half ? launch<_Float16, 64>(a, w, plan.rows, stream) : launch<__bf16, 64>(a, w, plan.rows, stream);
    if (p.heads.dim == 128) return half ? launch<_Float16, 128>(a, w, plan.rows, stream) : launch<__bf16, 128>(a, w, plan.rows, stream);
    return half ? launch<_Float16, 256>(a, w, plan.rows, stream) : launch<__bf16, 256>(a, w, plan.rows, stream);
}

}  // namespace kvpub
