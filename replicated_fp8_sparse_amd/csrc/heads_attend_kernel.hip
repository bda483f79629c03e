// Attention over the replicated cache of key and value heads (e4m3 codes, a
// power-of-two scale for each block of 64 positions and head).
//
// Mathematics.  With codes c and d of a block's keys and values and its scales a, b,
//   score = (scale * a) (q . c),   out = sum_p w_p (b d_p) / sum_p w_p.
// A code is exact in bf16 and fp16, and so is a value's code times its scale in
// bf16 (but for multiples of 2^-135 below 2^-126, which the two least scales have): nothing of the cache is rounded again.  Weights are rounded to bf16 for the
// second product: that leaves bf16 outputs off by 0.0021 of their norm where their own
// rounding alone leaves 0.0017, and a second operand for the low parts costs 38 % in long
// prompts.  Units of 16 rows, which memory bounds, take that operand (2 % of a large
// decode), and so do fp16 outputs, whose own step is finer.  One pass: a row's running maximum moves only when a
// score exceeds it by more than 2^8, so most tiles neither rescale nor shuffle.
//
// Mapping.  Rows are (token, query head) pairs that share a key-value head: a unit
// is 16, 32 or 64 of them and one key-value head.  Scores come out transposed: positions
// down, rows across, so that a lane holds 8 positions of one row, and its weights
// are an operand of the second product as they are if the values' positions come in the
// same order.  Values are read by position, 16 lanes a row, and brought to columns by
// byte permutes within a lane: no LDS before the end (but for the queries of 32 rows of 128
// values and more, and of 64 rows).  The 4 waves of a block take every 4th tile of 32 positions, each from
// memory straight to registers: keys as soon as the last tile's scores are computed, values as
// soon as its products are, so both are on their way behind the other half of the work.
// Page numbers, lengths and scales come through the scalar cache, whose waits leave those
// loads alone.  The waves join their parts through LDS; long sequences are cut into
// chunks for several blocks, which join_kernel joins in order.
//
// Bound.  16 rows: memory.  64 sequences of up to 8192 positions over 8 heads of 128: 107 us for
// 545 MB, a large copy's 5.1 TB/s, and 5 for the join.  64 rows: a tile takes 270 vector
// instructions (80 of them the widening, 128 the weights) and 64 matrix instructions, which exclude each
// other more than they overlap: beside a wave that issues 16 x 16 x 32 products
// back to back the other waves of its SIMD issue nothing for 14 of 16 cycles (32 x 32 x 16:
// 21 of 32), so 2100 cycles of work a tile, of which two waves a SIMD reach some 2270: by the counters matrix instructions
// take 45 % of the SIMDs' cycles and the other vector instructions 47 %.  Prompts of 2 x 4096 tokens behind as
// much context, 16 heads over 4: 230-256 us from card to card, 72-80 % of a large bf16 product's rate.
// (Built and measured when it took 254-260: 32 x 32 x 16 products throughout, 247; the same with the next
// tile's scores between this one's weights, one wave a SIMD, 300; 32 rows a unit, 300-315.)  Short
// prompts: a block's start (lengths, pages, queries, the first tile: 5 us) and the join of 64 rows (3).
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

constexpr uint32_t kWaves = 4, kThreads = kWaves * 64;
// How a call is cut (plan_heads_attend), by its bounds alone.  Blocks are units times key-value heads.
//
// Up to kWhole positions a sequence stays whole; beyond, the blocks of units of 16 and 32 rows are cut into as many parts as
// the most of three rules asks for, at most kMostChunks: with few blocks for a block a compute unit (kFill), in cuts of
// kLeastChunk positions; for two a compute unit, in cuts of 2 kChunk; and for kWanted blocks of 16 rows, or kWantedWide of
// 32, in cuts of at least kChunk and of kChunkRows for each row, as each row of a cut writes a part.  Units of 64
// rows, 512 blocks and more, are not cut.  Measured, us (8 query heads a key-value head and 128 values where nothing
// else is said):
//   kWhole 768, one token, whole / cut: over 640 positions, 2 heads 7.5 / 8.4, 768 8.2 / 8.4, 769 9.1 / 8.5, 1024 9.7 / 8.5;
//   heads of 64 values over 768 6.9 / 7.8, 1024 8.0 / 7.8, of 256 640 9.9 / 9.8, 768 11.0 / 9.9; 16 sequences, 32 over 8,
//   768 10.3 / 12.0, 1024 12.3 / 13.3, 1300 15.2 / 15.1
//   kLeastChunk 256 / 512 / 1024, one token over 8192, 2 heads: 9.9 / 10.8 / 12.9, over 1000 8.7 / 10.0 / -; for the few
//   blocks alone: 8 x 4096, 32 over 8 heads, 512 blocks 15.9 / 15.0, 16 x 8192 of 256 values 46.1 / 43.5
//   kMostChunks 64 / 128, one token over 65536: 17.1 / 14.9
constexpr uint32_t kLeastChunk = 256, kChunk = 512, kWhole = 768, kMostChunks = 128;
//   16 / 32 / 64 positions a row: 8 tokens of each of 16 sequences of 8192 (32 rows) 66 / 66 / 61
constexpr uint32_t kChunkRows = 64;
//   cut for up to 2048 / 4096 / 8192 blocks of 16 rows: one token of 64 sequences of up to 8192 121.6 / 121.0 / 126.3;
//   for 768 / 1024 of 32 rows: 16 trees of 24 63 / 52
constexpr uint32_t kWanted = 4096, kWantedWide = 1024;
//   with kFill 1 / 256 / 512: trees of 2 x 26 tokens, 16 heads over 1 of 256, 6215 positions 27 / 19 / 19, 1 x 5, 32 over 2,
//   5772 20.8 / 12.9 / 12.9, prompts of 6 x 534 behind 409 positions 14.9 / 14.8 / 18.6; without the cuts for twice as
//   many: trees of 23 x 28 tokens, 2 heads of 64, over 8926 20.6 / 17.9
constexpr uint32_t kFill = 256;
//   units of 64 rows from kFull blocks on, as many as the card holds at once, twice as many for 64 values, of which it
//   holds three blocks of 32 rows a compute unit; else of 32.  4 chunks of n tokens, 32 heads over 8, the last of
//   kv positions, 32 / 64 rows: n = 192 (384 blocks of 64), kv = 2048 48 / 45, 8192 141 / 123; n = 240 (480) 55 / 45,
//   179 / 153; n = 256 (512) 53 / 45, 182 / 142; n = 272 (544) 64 / 58, 221 / 192.  Below 512 the others lose:
//   4 x 676 over 1243, 20 over 4 (about 420) 30 / 33, 16 trees of 24 52 / 76.  2 x 1547 over 4701, 15 over 3 (726) 142 / 115, in
//   fp16 166 / 150; prompts of 1 x 2048, 24 over 4 of 64 (768) 30 / 34.  512 blocks of 64 rows in two cuts: the n = 256 above
//   over 5000 110, whole 91, over 8192 160, whole 142; ragged, over up to 5000 93 / 82, 16384 225 / 220
constexpr uint32_t kFull = 512;
// what is cut writes at most kPartRows rows of parts, whatever its units' rows: the workspace's size goes by it
constexpr uint32_t kPartRows = kWanted * 16;
static_assert(kWantedWide * 32 <= kPartRows && 2 * kFill * 32 <= kPartRows, "units of 32 rows, each cut of which writes as many");
constexpr uint32_t kTile = 32;                    // positions of a wave's step
constexpr float kLazy = 8.0f;                     // rescale when a maximum grows past 2^8
constexpr float kLn2 = 0.693147180559945309f;


// Waves that a SIMD should hold: what the registers of the accumulators leave room for
// (16 rows of 128 values: 3; at 4 they spill, 133 us for 121 in the large decode).
constexpr int waves_a_simd(int D, int RT) { return RT * D <= 64 ? 4 : (RT * D <= 128 ? 3 : (RT * D <= 512 ? 2 : 1)); }

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

__device__ __forceinline__ uint32_t token_of(const HeadsAttendParams& p, uint32_t row) {
    return (uint32_t)(((uint64_t)row * p.group_magic) >> p.group_shift);
}

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
    const int64_t lim = u.base + token_of(p, last) + 1;
    u.reach = p.tree ? u.s.kv : (lim > 0 ? (uint32_t)lim : 0u);
    u.chunks = u.reach ? (u.reach + p.chunk - 1) / p.chunk : 1u;
    return u;
}

// A row's output from its joined parts: N pieces of 4 values a lane, 64 values apart, the first at `seg`.
template <class E, int N>
__device__ __forceinline__ void put_row(const HeadsAttendParams& p, const Unit& u, uint32_t g, uint32_t row, uint32_t seg, const f32x4 (&acc)[N],
                                        float top, float sum) {
    const uint32_t i = token_of(p, row), h = g * p.group + row - i * p.group;
    E* dst = (E*)p.out + (int64_t)(u.s.q0 + i) * p.out_token + (int64_t)h * p.out_head + seg;
    const float f = sum == 0.f ? 0.f : 1.f / sum;           // no position seen: 0
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const f32x4 x = acc[n] * f;
        E y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = (E)x[k];
        __builtin_memcpy(__builtin_assume_aligned(dst + n * 64, 8), y, sizeof y);
    }
    if (seg == 0 && p.lse) p.lse[(int64_t)(u.s.q0 + i) * p.lse_token + h] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
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

// Bits of the positions pos .. pos + 31 that lie below lim.
__device__ __forceinline__ uint32_t first_bits(uint32_t lim, uint32_t pos) {
    const uint32_t left = lim > pos ? lim - pos : 0u;
    return left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1;
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

__device__ __forceinline__ float power(uint32_t byte) {
    const uint32_t b = byte < 1 ? 1u : (byte > 245 ? 245u : byte);
    return __uint_as_float(b << 23);
}

// A descriptor of `bytes` bytes from p on, both uniform: loads beyond them give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t bytes_at(const uint8_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00027000);
}

// The lane's number, got anew where it is asked for.
__device__ __forceinline__ uint32_t lane_anew() {
    uint32_t l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

template <int D> __device__ __forceinline__ uint32_t key_at(uint32_t l16, uint32_t g4) { return l16 * D + g4 * 16; }
template <int D> __device__ __forceinline__ uint32_t value_at(uint32_t l16, uint32_t g4) { return g4 * 4 * D + l16 * (D / 16); }

// The codes of a tile of 32 positions in one wave's registers.
template <int D>
struct Tile {
    i32x4 k[2][D / 64];              // position 16 u + l%16, values 64 c + 16 (l/16) ..
    uint32_t v[8][D / 64];           // position j of this lane group, values (D/16) (l%16) ..
    uint32_t scales;                 // word that holds this head's bytes, for the keys and for the values: shifted only where
                                     // they are used, as a shift here would wait for the load

    // Through a descriptor of the tile's bytes, whose offsets are 32-bit; one of none (`any` false) gives zeros without a
    // look at memory.  A branch about the loads would leave the compiler no number of loads on the way to count down
    // to: it would wait for all of them (2 x 1024 tokens over 2048 of 256 values 60.5 us, so 57.0).
    // Of 256 values the offsets are computed again each time: beside 32 rows they would be spilled, and a spilled one's
    // wait is for all loads on the way, too.
    __device__ __forceinline__ void load_keys(const uint8_t* page, uint32_t head, uint32_t groups, uint32_t half, uint32_t lane_at, bool any) {
        if (D == 256) {
            const uint32_t lane = lane_anew();
            lane_at = key_at<D>(lane & 15u, lane >> 4);
        } else asm volatile("" : "+v"(lane_at));             // sums with it stay with the instructions
        const __amdgpu_buffer_rsrc_t from = bytes_at(page + head * (128 * D) + half * (kTile * D), any ? kTile * D : 0u);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                k[u][c] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(from, lane_at + c * 64, u * 16 * D, 0));
        scales = *(kptr<uint32_t>)(page + groups * (128 * D) + (2 * head & ~3u));
    }
    __device__ __forceinline__ void load_values(const uint8_t* page, uint32_t head, uint32_t half, uint32_t lane_at, bool any) {
        if (D == 256) {
            const uint32_t lane = lane_anew();
            lane_at = value_at<D>(lane & 15u, lane >> 4);
        } else asm volatile("" : "+v"(lane_at));             // sums with it stay with the instructions
        const __amdgpu_buffer_rsrc_t from = bytes_at(page + head * (128 * D) + 64 * D + half * (kTile * D), any ? kTile * D : 0u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t at = lane_at + (j & 3) * D, base = (j >> 2) * 16 * D;
            if constexpr (D == 64) v[j][0] = __builtin_amdgcn_raw_buffer_load_b32(from, at, base, 0);
            else if constexpr (D == 128) {
                const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(from, at, base, 0));
                v[j][0] = w.x, v[j][1] = w.y;
            } else {
                const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at, base, 0));
                v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
            }
        }
    }
};

template <class E>
__device__ __forceinline__ typename Operand<E>::x8 load_query(const E* src, uint32_t signs) {
    const u32x4 w = *(const u32x4*)src ^ signs;
    return __builtin_bit_cast(typename Operand<E>::x8, w);
}

// Shared: the queries' operands stay in LDS.  64 rows of 128 values would lose the second wave a
// SIMD to their registers; 32 rows of 128 take 52.7 us for 54.3 (16 trees of 24), 64 of 64 57.1
// for 58.0 (prompts of 2 x 2048); 16 rows of 256 47.1 for 45.2, and keep them.
template <class E, int D, int RT>
__global__ __launch_bounds__(kThreads, waves_a_simd(D, RT)) void heads_attend_kernel(const HeadsAttendParams p, const Places places) {
    typedef Operand<E> Op;
    constexpr uint32_t R = 16 * RT;
    constexpr int NB = D / 16, NQ = D / 32, W = kWaves;
    constexpr bool Shared = RT > 1 && RT * D >= 256;
    constexpr bool Low = RT == 1 || !__is_same(E, __bf16);         // the weights' low parts as a second operand: see above
    // two of them where blocks leave the room: a wave may write the next rows before all have read these
    constexpr int kJoins = RT > 1 && D < 256 ? 2 : 1;
    struct Join {
        float o[W][16][D + 4];
        float ml[W][16][2];
    };
    union Lds {
        Join join[kJoins];
        typename Op::x8 q[Shared ? RT * NQ : 1][64];
        __device__ Lds() {}
    };
    __shared__ Lds lds;
    const uint32_t G = p.heads.groups, tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t l16 = lane & 15u, g4 = lane >> 4;
    // the longest first: a causal sequence's last rows
    const uint32_t turn = blockIdx.x / G, g = blockIdx.x - turn * G, place = p.units - 1 - turn, cut = blockIdx.y;
    const Unit u = unit_of(p, places, p.first + place, R);
    if (u.rows == 0 || cut >= u.chunks) return;

    const int32_t* table = p.seqs.pages + (int64_t)u.s.b * p.seqs.pages_stride;
    const uint32_t end = u.reach < (cut + 1) * p.chunk ? u.reach : (cut + 1) * p.chunk;
    const uint32_t last = (end + kTile - 1) / kTile;
    const bool counts = g == 0 && u.row0 + R >= u.rows;
    auto page_of = [&](uint32_t t) { return t < last ? uniform_load(table, t >> 1) : 0; };
    auto at = [&](int32_t page) { return p.base + ((uint32_t)page < p.heads.num_pages ? (uint64_t)(uint32_t)page * p.heads.page_stride : 0ull); };
    uint32_t t = cut * (p.chunk / kTile) + wave;
    int32_t page = page_of(t), page1 = page_of(t + W);
    const uint32_t keys = key_at<D>(l16, g4), values = value_at<D>(l16, g4);
    Tile<D> tile;
    tile.load_keys(at(page), g, G, t & 1u, keys, t < last);

    // queries, and what each row sees: positions below lim (tree: of those before the tree, then its bits); rows of none
    // take the sequence's first
    const uint32_t signs = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const auto query = [&](uint32_t r, uint32_t c) {
        const uint32_t row = u.row0 + r * 16 + l16, i = row < u.rows ? token_of(p, row) : 0u, h = g * p.group + (row < u.rows ? row - i * p.group : 0u);
        const E* src = (const E*)p.q + (int64_t)(u.s.q0 + i) * p.q_token + (int64_t)h * p.q_head + g4 * 16;
        return load_query<E>(src + (c >> 1) * 64 + (c & 1u) * 8, signs);
    };
    constexpr uint32_t kMine = RT * NQ / W;
    typename Op::x8 q[Shared ? 1 : RT][NQ], mine[Shared ? kMine : 1];
    if constexpr (Shared) {
#pragma unroll
        for (uint32_t i = 0; i < kMine; ++i) mine[i] = query((wave + i * W) / NQ, (wave + i * W) % NQ);
    } else {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < NQ; ++c) q[r][c] = query(r, c);
    }
    tile.load_values(at(page), g, t & 1u, values, t < last);
    uint32_t lim[RT];
    uint32_t tree[RT];                     // first word of the row's bits
    uint32_t least = 0xFFFFFFFFu;          // positions that all rows see
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const uint32_t row = u.row0 + r * 16 + l16;
        const bool is = row < u.rows;
        const uint32_t i = is ? token_of(p, row) : 0u;
        const int64_t top = u.base + (p.tree ? 0 : (int64_t)i + 1);
        lim[r] = is ? (top > 0 ? (uint32_t)top : 0u) : 0xFFFFFFFFu;
        tree[r] = (u.s.q0 + i) * p.tree_words;
        least = lim[r] < least ? lim[r] : least;
    }
    if constexpr (Shared) {
#pragma unroll
        for (uint32_t i = 0; i < kMine; ++i) lds.q[wave + i * W][lane] = mine[i];
        __syncthreads();
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

    // as a function of its own, inlined: the compiler then keeps its scalars in registers (1-2 % of every call)
    const auto step = [&]() __attribute__((always_inline)) {
        const uint32_t pos0 = t * kTile, next = t + W;
        const bool bad = (uint32_t)page >= p.heads.num_pages;
        // a bad page is hidden; counted by the rows that see most of the sequence, at a page's first half
        if (bad && counts && !(t & 1u) && any_sees(p, u, pos0) && lane == 0) atomicAdd(p.invalid_count, 1ull);

        f32x4 s[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        typename Op::x8 b[RT];
        if constexpr (Shared) {
#pragma unroll
            for (int r = 0; r < RT; ++r) b[r] = lds.q[r * NQ][lane];
        }
#pragma unroll
        for (int c = 0; c < NQ; ++c) {
            // queries from LDS are read a step ahead
            typename Op::x8 a[2], ahead[RT];
            if constexpr (Shared) {
#pragma unroll
                for (int r = 0; r < RT; ++r) ahead[r] = lds.q[r * NQ + (c + 1 < NQ ? c + 1 : c)][lane];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) a[j] = Op::widen(tile.k[j][c >> 1][2 * (c & 1)], tile.k[j][c >> 1][2 * (c & 1) + 1]);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (Shared) s[r][j] = Op::mfma(a[j], b[r], s[r][j]);
                    else s[r][j] = Op::mfma(a[j], q[r][c], s[r][j]);
                }
            if constexpr (Shared) {
#pragma unroll
                for (int r = 0; r < RT; ++r) b[r] = ahead[r];
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the scale of a score in powers of 2 is kept above 0 and below infinity, so that a hidden score stays -infinity
        const uint32_t scales = tile.scales >> ((2 * g & 2u) * 8);
        const float ks = fminf(fmaxf(fabsf(p.scale_log2) * power(scales & 255u), FLT_MIN), FLT_MAX), vs = power((scales >> 8) & 255u);
        const int32_t page2 = page_of(next + W);
        tile.load_keys(at(page1), g, G, next & 1u, keys, next < last);

        if (pos0 + kTile > least || bad) {
            // some row does not see the whole tile.  Bits of its 32 positions; those of this lane are
            // j and 16 + j, j < 4, of the bits from 4 (l/16) on
            const uint32_t real = bad ? 0u : first_bits(u.s.kv, pos0), mine = real >> (g4 * 4);
            uint32_t sees[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t bits = p.tree ? (uint32_t)tree_bits(p.tree + tree[r], p.tree_words, (int64_t)pos0 - u.base) : first_bits(lim[r], pos0);
                sees[r] = (bits & real) >> (g4 * 4);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[r][j >> 2][j & 3] = (sees[r] >> ((j >> 2) * 16 + (j & 3))) & 1u ? s[r][j >> 2][j & 3] : -INFINITY;
            }
            // values that do not exist become zeros, and so do rows that hold a NaN code,
            // with a NaN score for who sees them: a weight of 0 does not hide a NaN
            uint32_t nan = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t bit = 1u << ((j >> 2) * 16 + (j & 3));
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    tile.v[j][w] = mine & bit ? tile.v[j][w] : 0u;
                    nan |= (((tile.v[j][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) ? bit : 0u;
                }
            }
            if (__any(nan)) {
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) nan |= __shfl_xor(nan, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t bit = 1u << ((j >> 2) * 16 + (j & 3));
#pragma unroll
                    for (int w = 0; w < D / 64; ++w) tile.v[j][w] = nan & bit ? 0u : tile.v[j][w];
#pragma unroll
                    for (int r = 0; r < RT; ++r) s[r][j >> 2][j & 3] = nan & sees[r] & bit ? NAN : s[r][j >> 2][j & 3];
                }
            }
        }
        bool grows = false;
        float high[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float a = fmaxf(fmaxf(s[r][0][0], s[r][0][1]), s[r][0][2]), b = fmaxf(fmaxf(s[r][0][3], s[r][1][0]), s[r][1][1]);
            high[r] = fmaxf(fmaxf(fmaxf(s[r][1][2], s[r][1][3]), a), b) * ks;
            grows |= high[r] > m[r] + kLazy;
        }
        if (__any(grows)) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                high[r] = fmaxf(high[r], __shfl_xor(high[r], 16));
                high[r] = fmaxf(high[r], __shfl_xor(high[r], 32));
                const float to = high[r] > m[r] + kLazy ? high[r] : m[r], f = __builtin_amdgcn_exp2f(m[r] - to);
                m[r] = to;
                l[r] *= f;
#pragma unroll
                for (int n = 0; n < NB; ++n) o[r][n] *= f;
            }
        }
        bf16x8 w[RT], low[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = __builtin_amdgcn_exp2f(fmaf(s[r][j >> 2][j & 3], ks, -m[r]));
                w[r][j] = (__bf16)e[j];
                if constexpr (Low) low[r][j] = (__bf16)(e[j] - (float)w[r][j]);
            }
            l[r] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            bf16x8 a[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const int lo = (int)__builtin_amdgcn_perm(tile.v[j + 1][c], tile.v[j][c], 0x05010400u);
                const int hi = (int)__builtin_amdgcn_perm(tile.v[j + 1][c], tile.v[j][c], 0x07030602u);
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
                    if constexpr (Low)
                        o[r][4 * c + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[d], low[r], o[r][4 * c + d], 0, 0, 0);
                }
        }
        tile.load_values(at(page1), g, next & 1u, values, next < last);
        page = page1;
        page1 = page2;
        t = next;
    };
    // the queries are waited for here: left to the loop, the wait would be in every step and for all loads on the way
    if constexpr (!Shared) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < NQ; ++c) asm volatile("" : "+v"(q[r][c]));
    }
    while (t < last) step();

    // the waves' parts, 16 rows at a time: 16 lanes a row, which read 64 values side by side
    const uint32_t row = tid >> 4, seg = (tid & 15u) * 4;
    if constexpr (Shared) __syncthreads();          // their queries' last reads
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (u.row0 + r * 16 >= u.rows) break;
        Join& join = lds.join[r % kJoins];
        l[r] += __shfl_xor(l[r], 16);
        l[r] += __shfl_xor(l[r], 32);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n) join.o[wave][l16][(g4 * 4 + i) * NB + n] = o[r][n][i];
        if (g4 == 0) join.ml[wave][l16][0] = m[r], join.ml[wave][l16][1] = l[r];
        __syncthreads();
        const uint32_t mine = u.row0 + r * 16 + row;
        if (mine < u.rows) {
            float top = join.ml[0][row][0], sum = 0.f;
            f32x4 acc[D / 64];
#pragma unroll
            for (uint32_t w = 1; w < W; ++w) top = fmaxf(top, join.ml[w][row][0]);
#pragma unroll
            for (int n = 0; n < D / 64; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t w = 0; w < W; ++w) {
                const float f = __builtin_amdgcn_exp2f(join.ml[w][row][0] - top);
                sum = fmaf(join.ml[w][row][1], f, sum);
#pragma unroll
                for (int n = 0; n < D / 64; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[n][k] = fmaf(join.o[w][row][seg + n * 64 + k], f, acc[n][k]);
            }
            if (RT < 4 && u.chunks > 1) {                     // units of 64 rows are not cut
                const uint64_t slot = (((uint64_t)place * G + g) * p.chunks + cut) * R + r * 16 + row;
#pragma unroll
                for (int n = 0; n < D / 64; ++n) *(f32x4*)(p.part + slot * D + seg + n * 64) = acc[n];
                if (seg == 0) p.part_ml[slot * 2] = top, p.part_ml[slot * 2 + 1] = sum;
            } else {
                put_row<E>(p, u, g, mine, seg, acc, top, sum);
            }
        }
        if constexpr (kJoins == 1) __syncthreads();
    }
}

// The parts of units that several blocks cut, joined in their order: D/4 lanes a row, which share out the cuts'
// maxima and sums; 2^shift such groups of lanes a row, each with its run of the cuts, 16 on the way at a time.
// One token over 65536, 128 cuts: 15.8 us with the cuts shared out, 26.3 with one group a row.  Up to 16 cuts
// one group takes them (Split false), and its loops are the whole block's, 0.2 us less.
template <class E, int D, bool Split>
__global__ __launch_bounds__(256) void join_kernel(const HeadsAttendParams p, const Places places, uint32_t R, uint32_t shift_) {
    constexpr uint32_t kLanes = D / 4, kGroups = 256 / kLanes, kEach = kMostChunks / kLanes, kBatch = 16;
    __shared__ float factors[kGroups][kMostChunks];
    __shared__ f32x4 sums[Split ? 256 : 1];
    const uint32_t shift = Split ? shift_ : 0u;
    const uint32_t G = p.heads.groups, place = blockIdx.x / G, g = blockIdx.x - place * G;
    const Unit u = unit_of(p, places, p.first + place, R);
    if (u.rows == 0 || u.chunks <= 1) return;
    const uint32_t lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, part = group & ((1u << shift) - 1);
    const uint32_t rows = u.rows - u.row0 < R ? u.rows - u.row0 : R;
    const uint32_t r = blockIdx.y * (kGroups >> shift) + (group >> shift);
    float top = -FLT_MAX, sum = 0.f;
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    if (r < rows) {
        const uint64_t slot = ((uint64_t)place * G + g) * p.chunks * R + r;
        float m[kEach], l[kEach];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            const uint32_t c = i * kLanes + lane;
            m[i] = -FLT_MAX, l[i] = 0.f;
            if (c < u.chunks) {
                const float2 ml = *(const float2*)(p.part_ml + (slot + (uint64_t)c * R) * 2);
                m[i] = ml.x, l[i] = ml.y;
            }
        }
        const uint32_t each = (u.chunks + (1u << shift) - 1) >> shift, first = Split ? part * each : 0u;
        const uint32_t end = Split && first + each < u.chunks ? first + each : u.chunks;
        for (uint32_t c0 = first; c0 < end; c0 += kBatch) {
            f32x4 x[kBatch];
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i)
                if (c0 + i < end) x[i] = *(const f32x4*)(p.part + (slot + (uint64_t)(c0 + i) * R) * D + lane * 4);
            if (c0 == first) {
#pragma unroll
                for (uint32_t i = 0; i < kEach; ++i) top = fmaxf(top, m[i]);
#pragma unroll
                for (uint32_t d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll
                for (uint32_t i = 0; i < kEach; ++i) {
                    const float f = __builtin_amdgcn_exp2f(m[i] - top);
                    sum = fmaf(l[i], f, sum);
                    factors[group][i * kLanes + lane] = f;
                }
#pragma unroll
                for (uint32_t d = 1; d < kLanes; d <<= 1) sum += __shfl_xor(sum, d);
                __builtin_amdgcn_wave_barrier();             // a group lies in one wave
            }
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i)
                if (c0 + i < end) acc[0] += x[i] * factors[group][c0 + i];
        }
    }
    if constexpr (Split) {
        sums[threadIdx.x] = acc[0];
        __syncthreads();
        if (part != 0) return;
        for (uint32_t i = 1; i < 1u << shift; ++i) acc[0] += sums[threadIdx.x + i * kLanes];
    }
    if (r < rows) put_row<E>(p, u, g, u.row0 + r, lane * 4, acc, top, sum);
}

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
        heads_attend_kernel<E, D, RT><<<dim3(p.units * G, p.chunks), kThreads, 0, stream>>>(p, w);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (p.chunks > 1) {
            constexpr uint32_t groups = 1024 / D;
            uint32_t shift = 0;
            while (p.chunks > 16u << shift && 2u << shift <= groups) ++shift;
            const dim3 grid(p.units * G, std::max<uint32_t>(1, 16 * RT / (groups >> shift)));
            if (shift) join_kernel<E, D, true><<<grid, 256, 0, stream>>>(p, w, 16 * RT, shift);
            else join_kernel<E, D, false><<<grid, 256, 0, stream>>>(p, w, 16 * RT, shift);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

template <class E, int D>
hipError_t launch(const HeadsAttendParams& p, const Places& w, const HeadsAttendPlan& plan, hipStream_t stream) {
    if (plan.rows == 16) return launch<E, D, 1>(p, w, stream);
    if (plan.rows == 32) return launch<E, D, 2>(p, w, stream);
    if constexpr (D < 256) return launch<E, D, 4>(p, w, stream);
    return hipErrorInvalidValue;
}

}  // namespace

HeadsAttendPlan plan_heads_attend(const HeadsParams& h, uint32_t group, uint64_t num_seqs, uint64_t num_tokens, uint64_t max_q,
                                  uint64_t max_kv) {
    HeadsAttendPlan a;
    const uint64_t rows = max_q * group;
    a.rows = rows <= 16 ? 16 : (rows <= 32 || h.dim == 256 ? 32 : 64);
    if (a.rows == 64) {
        (void)unit_places(64, group, num_seqs, num_tokens, max_q, &a.units);
        if (a.units * h.groups < (h.dim == 64 ? 2 * kFull : kFull)) a.rows = 32;
    }
    (void)unit_places(a.rows, group, num_seqs, num_tokens, max_q, &a.units);
    const uint64_t blocks = std::max<uint64_t>(1, a.units * h.groups);
    const auto cuts = [&](uint64_t most, uint64_t wanted) { return std::min(std::min<uint64_t>(most, kMostChunks), wanted / blocks); };
    const uint64_t by_rows = std::max<uint64_t>(kChunk, std::min<uint64_t>(rows, a.rows) * kChunkRows);
    uint64_t n = 1;
    if (max_kv > kWhole && a.rows < 64) {
        n = std::max(n, cuts((max_kv + by_rows - 1) / by_rows, a.rows == 16 ? kWanted : kWantedWide));
        n = std::max(n, cuts((max_kv + kLeastChunk - 1) / kLeastChunk, kFill));
        n = std::max(n, cuts(max_kv / (2 * kChunk), 2 * kFill));
    }
    a.chunk = (uint32_t)std::max<uint64_t>(kLeastChunk, ((max_kv + n - 1) / n + 127) / 128 * 128);
    a.chunks = (uint32_t)std::max<uint64_t>(1, (max_kv + a.chunk - 1) / a.chunk);
    // parts of as many rows as the bounds allow, which grows with each of them; the rows of a unit that none has count too
    const uint64_t parts = std::min<uint64_t>(kPartRows, (num_tokens * group + num_seqs * 64) * h.groups * std::min<uint64_t>(kMostChunks, (max_kv + kLeastChunk - 1) / kLeastChunk + 1));
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
    // ceil(2^(31 + s) / group), 2^s >= group: exact for rows below 2^31
    uint32_t shift = 0;
    while ((1u << shift) < p.group) ++shift;
    a.group_shift = 31 + shift;
    a.group_magic = (uint32_t)(((1ull << a.group_shift) + p.group - 1) / p.group);
    a.part = static_cast<float*>(workspace);
    a.part_ml = a.part + plan.bytes / 4 / (p.heads.dim + 2) * p.heads.dim;
    const bool half = p.type == KVPUB_FP16;
    if (p.heads.dim == 64) return half ? launch<_Float16, 64>(a, w, plan, stream) : launch<__bf16, 64>(a, w, plan, stream);
    if (p.heads.dim == 128) return half ? launch<_Float16, 128>(a, w, plan, stream) : launch<__bf16, 128>(a, w, plan, stream);
    return half ? launch<_Float16, 256>(a, w, plan, stream) : launch<__bf16, 256>(a, w, plan, stream);
}

}  // namespace kvpub
