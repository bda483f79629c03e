// Latent attention over the published cache for gfx950: the reader that the
// store writes for.  vLLM PR #52863 "[Kernel][PCP] Publish replicated KV updates
// through PyTorch symmetric memory", Summary and Design: attention reads the
// local replica in the layout the store writes; a row is key and value of all heads.
//
// Mathematics.  With codes k_j (tile j of 128) and tile scales a_j of a row,
//   score = scale * (sum_j a_j (q_j . k_j) + q_r . r),   out_j = sum_p (w_p a_pj) k_pj / sum_p w_p,
// so the codes enter the matrix instructions as they are and each tile's scale
// multiplies an accumulator (scores) or the weight (values): no row is rounded
// to bf16.  A code is exact in bf16, and so is its product with a bf16 query in
// the accumulator.  (The scaled e4m3 instruction would take the codes as they
// are and each query as the sum of two e4m3 numbers at the same rate; its sums
// were found off by 2^-16 of the largest product, too much for lse.)  The
// weights are rounded to bf16 for the second product: a second operand for their
// low part would double its matrix instructions, and outputs are off by 0.0022 of
// their norm where their own rounding alone leaves 0.0017.
//
// Mapping.  A block of 8 waves takes a unit (sequence, M rows = (token, head)
// pairs) over a run of 64-row tiles (a page), a tile being one copy of 41984
// contiguous bytes straight into LDS, two tiles ahead of its use.  Scores come
// out transposed (keys down, query rows across): a lane holds 4 keys of one query
// row, row maxima and sums need two shuffles, and the weights are already laid
// out as an operand of the second product if its key order follows;
// ds_read_b64_tr_b8 picks the values' columns in that order.  The page's own row
// stride (656 bytes: 164 banks, 36 modulo 64) is read as it is: 16-byte reads of
// 16 rows take 8.0 cycles (two rows share banks), a column read 2.3 with half of
// the rows rotated by 8 (4.1 without).  One pass: running maximum and sum, the
// accumulator rescaled only when the maximum grew by more than 2^8.
// M = 16 and 32: attend_kernel, the row's 512 values split between waves; M = 64:
// attend_wide_kernel.  plan_attend() says which and what either costs.
//
// Bound.  The matrix units need 2200 cycles for a tile of 64 rows, its widening to
// bf16 (4 instructions for 8 codes) and softmax about 2000 on the vector unit, LDS
// 2500; with one barrier a tile and two waves a SIMD they overlap by half: 6300
// cycles a tile.  64 sequences of up to 8192 positions, 128 heads: 160-180 us in all
// (61 at the rate of a large bf16 matrix product, 430 TFLOP/s reached).
//
// Work split.  All units' tiles form one line that the blocks cut into equal
// runs, whatever the lengths of the sequences; a unit cut between blocks leaves
// partial results that combine_kernel joins in block order.  The block that has a
// cut unit's first tiles names it, so the join visits those units and no others:
// what it costs goes by the blocks, not by the call's bounds.
#include "kvpub_internal.h"

#include <type_traits>

namespace kvpub {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
template <class T> using lptr = __attribute__((address_space(3))) T*;

constexpr int kRow = 656;
constexpr int kTileBytes = 64 * kRow;            // 41984 = 41 copies of 1024 bytes
constexpr int kRing = 3;
constexpr int kWaves = 8;                        // two a SIMD: 256 registers each
constexpr int kThreads = kWaves * 64;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLazy = 8.0f;                    // rescale when a maximum grows past 2^8
constexpr uint32_t kMostBlocks = 256;            // of a launch: one a CU
constexpr uint64_t kCutBytes = kMostBlocks * (sizeof(uint32_t) + sizeof(AttendCut));

// LDS: the tile ring (after the last tile it holds the join of key halves), the
// waves' exchange of partial scores, the tiles' scales by tile of 128, slot
// lists 3 tiles deep.  160 KB in all.
constexpr int kSlotRing = 3;
constexpr int kExchange = 32768;
struct Shared {
    alignas(16) uint8_t ring[kRing * kTileBytes];
    alignas(16) uint8_t exchange[kExchange];
    alignas(16) float scales[kRing][4][64];
    alignas(16) int64_t slots[kSlotRing][64];
};
static_assert(sizeof(Shared) <= 163840, "160 KB of LDS");

// Tile t's place in the ring; opaque, so that addresses stay a base and immediate
// offsets instead of one induction variable each.
__device__ __forceinline__ uint32_t ring_of(uint32_t t) {
    uint32_t r = __builtin_amdgcn_readfirstlane(t % kRing);
    asm("" : "+s"(r));
    return r;
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(lptr<const uint8_t>)(const uint8_t*)p;
}

// 64 lanes x 16 bytes from each lane's address to 1024 consecutive LDS bytes.
// Written as asm because the compiler otherwise waits for every outstanding copy
// before any LDS read; wait_own() below counts them instead.
// (m0 is a reserved register, which the compiler warns of: it holds no value of its own
// there, but may set it once for several uses.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const uint8_t* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void copy4_to_lds(const uint8_t* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's own copies of all but the newest tile have landed.  A tile is 41
// copies of rows, wave, wave + 8, ..., and one of each tile's scales by waves
// 1..4: 6 copies for waves 0..4 and 5 for the others.
__device__ __forceinline__ void wait_own(uint32_t wave, bool newer) {
    if (!newer) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else if (wave <= 4) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(5)" ::: "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// One 16-row group of queries as operands, T tiles of 128 and P of the two RoPE
// halves: lane (l%16, l/16) = (row, 16 of each 64 values: the first 8 go with one
// matrix instruction, the others with the next), and 8 of each 32 RoPE values.
template <int T, int P>
struct QFrag {
    bf16x8 lat[4 * T];
    bf16x8 rope[P];
    __device__ __forceinline__ void load(const uint16_t* latent, const uint16_t* rp, uint32_t g) {
#pragma unroll
        for (int c = 0; c < 4 * T; ++c) lat[c] = *(const bf16x8*)(latent + (c >> 1) * 64 + g * 16 + (c & 1) * 8);
#pragma unroll
        for (int c = 0; c < P; ++c) rope[c] = *(const bf16x8*)(rp + c * 32 + g * 8);
    }
    // The loads have landed: without this the compiler waits for them where they
    // are used, in the loop, and with them for every tile in flight.
    __device__ __forceinline__ void landed() {
#pragma unroll
        for (int c = 0; c < 4 * T; ++c) asm volatile("" : "+v"(lat[c]));
#pragma unroll
        for (int c = 0; c < P; ++c) asm volatile("" : "+v"(rope[c]));
    }
};

// 8 codes as bf16 (exact).
__device__ __forceinline__ bf16x8 widen(int c0, int c1) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, true);
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The 32 keys of a step in the order of the matrix units: row m of half u is key
// u * 16 + (m ^ 8 u).  The 8 keys that a lane group's column read takes (4 of each
// half) and its neighbour group's then fall on distinct LDS banks, as rows 16 apart
// do not.
__device__ __forceinline__ uint32_t key_of(uint32_t u, uint32_t g) { return u * 16 + 4 * (u ? g ^ 2 : g); }   // of lane group g: + 0..3

// Value i of this lane's quad: scales are read one a lane and spread by the
// multiply itself, a quarter of the LDS time of reading 4 a lane.
template <int I>
__device__ __forceinline__ float quad(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), I | (I << 2) | (I << 4) | (I << 6), 15, 15, true));
}
__device__ __forceinline__ f32x4 quads(float v) { return f32x4{quad<0>(v), quad<1>(v), quad<2>(v), quad<3>(v)}; }

// Scores times `scale` of 32 keys x 16 query rows over T tiles of 128 (and the
// RoPE halves of q, if `ropes`): x[u][r], keys key_of(u, l/16) + i of query row
// l%16.  rows: the keys' LDS rows from the first tile's codes on; rope: its RoPE
// values; scales: the first key's in [tile][64].  The codes of the next two matrix
// steps are read while the last two are in the matrix units.
template <int R16, int T, int P>
__device__ __forceinline__ void scores32(f32x4 (*x)[R16], const uint8_t* rows, const uint8_t* rope, const float* scales,
                                         const QFrag<T, P>* q, float scale, bool ropes, uint32_t l16, uint32_t g) {
    const uint32_t at[2] = {l16 * kRow + g * 16, (16 + (l16 ^ 8)) * kRow + g * 16};
    const float* sc[2] = {scales + key_of(0, g) + (l16 & 3), scales + key_of(1, g) + (l16 & 3)};
    i32x4 raw[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) raw[u] = *(const i32x4*)(rows + at[u]);
    if (ropes) {
        bf16x8 k[2][P];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < P; ++h) k[u][h] = *(const bf16x8*)(rope + at[u] + h * 64);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < R16; ++r) {
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < P; ++h) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u][h], q[r].rope[h], c, 0, 0, 0);
                x[u][r] = c * scale;
            }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < R16; ++r) x[u][r] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int j = 0; j < T; ++j) {
        f32x4 c[2][R16];
        float a[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) a[u] = sc[u][j * 64];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 next[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) next[u] = j * 2 + h + 1 < 2 * T ? *(const i32x4*)(rows + at[u] + (j * 2 + h + 1) * 64) : raw[u];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bf16x8 w = widen(raw[u][k * 2], raw[u][k * 2 + 1]);
#pragma unroll
                    for (int r = 0; r < R16; ++r) {
                        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
                        c[u][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, q[r].lat[j * 4 + h * 2 + k], h + k ? c[u][r] : z, 0, 0, 0);
                    }
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) raw[u] = next[u];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 s = quads(a[u] * scale);
#pragma unroll
            for (int r = 0; r < R16; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][r][i] = fmaf(s[i], c[u][r][i], x[u][r][i]);
        }
    }
}

// ---- the line of work ---------------------------------------------------------

// What one sequence (or one token's slot list) asks for.
struct Seq {
    uint32_t q0;         // first token
    uint32_t n;          // tokens
    uint32_t kv;         // positions
    uint32_t units;      // row groups of M
    uint32_t tiles;      // 64-row tiles of each, at least 1
};

// Arrays that no kernel of the call writes, read through the scalar cache where
// the index is uniform: their waits then do not drain the tiles in flight.
template <class T> using kptr = const __attribute__((address_space(4))) T*;
__device__ __forceinline__ int32_t uniform_load(const int32_t* p, uint32_t i) { return ((kptr<int32_t>)p)[i]; }

__device__ __forceinline__ Seq shape(const AttendParams& p, int32_t kv, int64_t q0, int64_t q1, uint32_t M, bool empty) {
    Seq s;
    q0 = q0 < 0 ? 0 : q0;
    q1 = q1 > (int64_t)p.num_tokens ? (int64_t)p.num_tokens : q1;
    s.q0 = (uint32_t)q0;
    s.n = q1 > q0 ? (uint32_t)(q1 - q0) : 0u;
    s.kv = kv < 0 || empty ? 0u : ((uint32_t)kv > p.max_kv ? p.max_kv : (uint32_t)kv);
    const uint32_t m = s.n > p.max_q ? p.max_q : s.n;     // tokens beyond max_q_len are not computed
    s.units = (m * p.heads + M - 1) / M;
    s.tiles = s.kv ? (s.kv + 63) / 64 : 1u;
    return s;
}

// Sequence b; Uniform: the same for the whole wave.
template <bool Slots, bool Uniform>
__device__ __forceinline__ Seq sequence(const AttendParams& p, uint32_t b, uint32_t M, bool empty) {
    if (Slots) {
        Seq s;
        s.q0 = b;
        s.n = 1;
        s.kv = empty ? 0u : p.num_slots;
        s.units = (p.heads + M - 1) / M;
        s.tiles = s.kv ? (s.kv + 63) / 64 : 1u;
        return s;
    }
    if (Uniform) {
        const int32_t kv = uniform_load(p.kv_len, b);
        if (!p.q_start) return shape(p, kv, b, (int64_t)b + 1, M, empty);
        return shape(p, kv, uniform_load(p.q_start, b), uniform_load(p.q_start, b + 1), M, empty);
    }
    const int32_t kv = p.kv_len[b];
    if (!p.q_start) return shape(p, kv, b, (int64_t)b + 1, M, empty);
    return shape(p, kv, p.q_start[b], p.q_start[b + 1], M, empty);
}

__device__ __forceinline__ uint32_t scan64(uint32_t x, uint32_t lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= (uint32_t)d) x += y;
    }
    return x;
}

// Tiles a block takes: an equal share.
__device__ __forceinline__ uint32_t share(uint32_t total, uint32_t blocks) {
    const uint32_t c = (total + blocks - 1) / blocks;
    return c < 1 ? 1 : c;
}

struct Place {
    uint32_t b, off;         // the sequence, and the tile within its work
    uint32_t each, total;
};

// Where this block's run begins, from prefix sums of the sequences' work: by each
// wave alone up to 64 sequences, else by the whole block.
__device__ __forceinline__ Place place(const AttendParams& p, uint32_t M, bool empty, uint8_t* scratch) {
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    Place r;
    if (p.num_seqs <= 64) {
        uint32_t w = 0;
        if (lane < p.num_seqs) {
            const Seq s = sequence<false, false>(p, lane, M, empty);
            w = s.units * s.tiles;
        }
        const uint32_t x = p.num_seqs == 1 ? w : scan64(w, lane), first = x - w;
        r.total = __builtin_amdgcn_readlane(x, p.num_seqs - 1);
        r.each = share(r.total, gridDim.x);
        const uint32_t at = r.each * blockIdx.x;
        const uint64_t here = __ballot(w && at >= first && at < x);
        r.b = here ? (uint32_t)__builtin_ctzll(here) : 0u;
        r.off = at - __builtin_amdgcn_readlane(first, r.b);
    } else {
        uint32_t* scan = (uint32_t*)scratch;
        uint32_t carry = 0, at = 0;
        for (int pass = 0; pass < 2; ++pass) {       // the total, then the place
            carry = 0;
            for (uint32_t b0 = 0; b0 < p.num_seqs; b0 += kThreads) {
                const uint32_t b = b0 + tid;
                uint32_t w = 0;
                if (b < p.num_seqs) {
                    const Seq s = sequence<false, false>(p, b, M, empty);
                    w = s.units * s.tiles;
                }
                const uint32_t x = scan64(w, lane);
                __syncthreads();
                if (lane == 63) scan[wave] = x;
                __syncthreads();
                uint32_t before = carry;
                for (uint32_t v = 0; v < kWaves; ++v) {
                    if (v < wave) before += scan[v];
                    carry += scan[v];
                }
                const uint32_t first = before + x - w;
                if (pass == 1 && w && at >= first && at < first + w) {
                    scan[kWaves] = b;
                    scan[kWaves + 1] = at - first;
                }
            }
            if (pass == 0) at = share(carry, gridDim.x) * blockIdx.x;
        }
        __syncthreads();
        r.total = __builtin_amdgcn_readfirstlane(carry);
        r.each = share(r.total, gridDim.x);
        r.b = __builtin_amdgcn_readfirstlane(scan[kWaves]);
        r.off = __builtin_amdgcn_readfirstlane(scan[kWaves + 1]);
        __syncthreads();
    }
    return r;
}

// One run of tiles of one unit.
struct Segment {
    Seq s;
    uint32_t b, unit;
    uint32_t t0, t1;         // tiles
    uint32_t slot;           // of partial results
    bool whole;              // all of the unit's tiles
};

// The block's run of the line, segment by segment.
template <bool Slots>
struct Line {
    const AttendParams& p;
    uint32_t M;
    bool empty;
    uint32_t begin, end, pos, b, off;

    __device__ __forceinline__ Line(const AttendParams& p_, uint32_t M_, bool empty_, uint8_t* scratch) : p(p_), M(M_), empty(empty_) {
        Place at;
        if (Slots) {
            const Seq s = sequence<true, true>(p, 0, M, empty);
            const uint32_t w = s.units * s.tiles;
            at.total = p.num_seqs * w;
            at.each = share(at.total, gridDim.x);
            at.b = at.each * blockIdx.x / w;
            at.off = at.each * blockIdx.x - at.b * w;
        } else {
            at = place(p, M, empty, scratch);
        }
        b = __builtin_amdgcn_readfirstlane(at.b);      // the same for the block: kept in scalar registers
        off = __builtin_amdgcn_readfirstlane(at.off);
        const uint32_t each = __builtin_amdgcn_readfirstlane(at.each), total = __builtin_amdgcn_readfirstlane(at.total);
        pos = begin = each * blockIdx.x;
        end = begin + each < total ? begin + each : total;
    }
    __device__ __forceinline__ bool next(Segment& g) {
        while (pos < end) {
            g.s = sequence<Slots, true>(p, b, M, empty);
            if (off >= g.s.units * g.s.tiles) { ++b; off = 0; continue; }     // pos < end <= total: a later sequence has work
            g.b = b;
            g.unit = off / g.s.tiles;
            g.t0 = off - g.unit * g.s.tiles;
            g.t1 = g.s.tiles - g.t0 < end - pos ? g.s.tiles : g.t0 + (end - pos);
            g.whole = g.t0 == 0 && g.t1 == g.s.tiles;
            g.slot = 2u * blockIdx.x + (pos == begin ? 0u : 1u);
            pos += g.t1 - g.t0;
            off += g.t1 - g.t0;
            return true;
        }
        return false;
    }
    // Names for combine_kernel the unit that this block began and others end, if
    // there is one: it can only be the last segment's.
    __device__ __forceinline__ void leave_none() const {
        if (begin >= end && threadIdx.x == 0) p.cut_last[blockIdx.x] = 0;
    }
    __device__ __forceinline__ void leave(const Segment& g, uint32_t rows) const {
        if (pos < end || threadIdx.x != 0) return;
        const uint32_t rest = g.s.tiles - g.t1, each = end - begin;     // a run that is cut is a whole share
        p.cut_last[blockIdx.x] = g.t0 == 0 && rest ? blockIdx.x + (rest + each - 1) / each : 0u;
        p.cuts[blockIdx.x] = AttendCut{g.slot, g.s.q0, g.unit * M, rows};
    }
};

// Runs that keep to one sequence, for up to 64 sequences: the shortest length with
// which they are no more than the blocks.  A block that would take the end of one
// sequence and the start of another pays a start twice, and all wait for it.  (64 lanes:
// 64 sequences of 4096 positions, 128 heads, 65 us; 65 of them, on one line, 80.)
struct Runs {
    const AttendParams& p;
    uint32_t b, t0, t1;
    bool left;

    __device__ __forceinline__ Runs(const AttendParams& p_, uint32_t M, bool empty) : p(p_) {
        const uint32_t lane = threadIdx.x & 63u;
        uint32_t w = 0;
        if (lane < p.num_seqs) {
            const Seq s = sequence<false, false>(p, lane, M, empty);
            w = s.units * s.tiles;
        }
        const uint32_t total = __builtin_amdgcn_readlane(scan64(w, lane), 63);
        uint32_t each = (total + gridDim.x - 1) / gridDim.x, x = 0;
        each = each < 1 ? 1 : each;
        while (true) {
            x = scan64((w + each - 1) / each, lane);
            // ends: with `each` as long as the longest sequence they are 64 at most, and with a
            // grid of fewer blocks than 256 there is a block for every tile
            if ((uint32_t)__builtin_amdgcn_readlane(x, 63) <= gridDim.x) break;
            each += 1 + each / 16;
        }
        const uint32_t first = x - (w + each - 1) / each, at = blockIdx.x;
        const uint64_t here = __ballot(at >= first && at < x);
        left = here != 0;
        b = here ? (uint32_t)__builtin_ctzll(here) : 0u;
        t0 = (at - __builtin_amdgcn_readlane(first, b)) * each;
        const uint32_t tiles = __builtin_amdgcn_readlane(w, b);
        t1 = tiles - t0 < each ? tiles : t0 + each;
    }
    __device__ __forceinline__ bool next(Segment& g) {
        if (!left) return false;
        left = false;
        g.s = sequence<false, true>(p, b, p.max_q * p.heads, p.head->capacity <= 0);
        g.b = b;
        g.unit = 0;
        g.t0 = t0;
        g.t1 = t1;
        return true;
    }
};

// ---- tiles -----------------------------------------------------------------------

// Where a unit's tiles come from, and which keys of a tile exist.
template <bool Slots>
struct Source {
    const AttendParams& p;
    const int32_t* table;      // this sequence's pages
    const int64_t* list;       // this token's slots
    uint32_t kv;
    int64_t capacity;
    uint8_t* ring;
    float (*scales)[4][64];
    int64_t (*slots)[64];
    uint32_t wave, lane;

    __device__ __forceinline__ int64_t page(uint32_t t) const {   // -1: no such page
        const int64_t g = uniform_load(table, t);
        return g >= 0 && g < capacity / 64 ? g : -1;
    }
    // Slots of tile t (clamped to the list: always in bounds); by wave 5.
    __device__ __forceinline__ void fetch_slots(uint32_t t) const {
        if (wave != 5) return;
        const uint32_t last = 2u * kv - 1u;
        uint32_t i = t * 128u + lane;
        const uint32_t at = lds_offset(&slots[t % kSlotRing][0]);
        copy4_to_lds((const uint8_t*)list + 4ull * (i < last ? i : last), at);
        i += 64;
        copy4_to_lds((const uint8_t*)list + 4ull * (i < last ? i : last), at + 256);
    }
    __device__ __forceinline__ bool good(int64_t s) const { return (uint64_t)s < (uint64_t)capacity; }
    __device__ __forceinline__ uint64_t row_of(int64_t s) const {
        const uint64_t v = good(s) ? (uint64_t)s : 0u;
        return (v >> 6) * p.main_page_stride + (v & 63u) * (uint64_t)kRow;
    }
    // Pages of the first three tiles (or their slots), and the first two tiles on their way.
    __device__ __forceinline__ void start(uint32_t t0, uint32_t t_end, int64_t* pg) const {
        pg[0] = pg[1] = pg[2] = -1;
        if (t0 >= t_end) return;
        if (Slots) {
            for (uint32_t t = t0; t < t0 + 3 && t < t_end; ++t) fetch_slots(t);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            barrier();
        } else {
            pg[0] = page(t0);
            if (t0 + 1 < t_end) pg[1] = page(t0 + 1);
            if (t0 + 2 < t_end) pg[2] = page(t0 + 2);
        }
        fetch(t0, pg[0]);
        if (t0 + 1 < t_end) fetch(t0 + 1, pg[1]);
    }
    // Tile t + 2 on its way, and the slots of the one behind it.
    __device__ __forceinline__ void ahead(uint32_t t, uint32_t t_end, const int64_t* pg) const {
        if (t + 2 >= t_end) return;
        if (Slots && t + 3 < t_end) fetch_slots(t + 3);
        fetch(t + 2, pg[2]);
    }
    __device__ __forceinline__ void turn(uint32_t t, uint32_t t_end, int64_t* pg) const {    // t: the new first tile
        pg[0] = pg[1];
        pg[1] = pg[2];
        if (!Slots) pg[2] = t + 2 < t_end ? page(t + 2) : -1;
    }
    // This wave's share of tile t: chunks wave, wave + 8, ..., and a tile's scales.
    __device__ __forceinline__ void fetch(uint32_t t, int64_t pg) const {
        const uint32_t buf = lds_offset(ring) + ring_of(t) * kTileBytes;
        const uint32_t at = lds_offset(&scales[ring_of(t)][0][0]) + (wave - 1) * 256u;
        if (Slots) {
            const int64_t* my = &slots[t % kSlotRing][0];
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                const uint32_t c = wave + kWaves * i;
                if (i == 5 && wave != 0) break;
                const uint32_t x = c * 64u + lane, r = x / 41u, o = (x - r * 41u) * 16u;
                copy16_to_lds(p.main_base + row_of(my[r]) + o, buf + c * 1024u);
            }
            if (wave >= 1 && wave <= 4) copy4_to_lds(p.main_base + row_of(my[lane]) + 508u + wave * 4u, at);
        } else {
            const uint8_t* page = p.main_base + (uint64_t)(pg < 0 ? 0 : pg) * p.main_page_stride;
            const uint8_t* base = page + wave * 1024u + lane * 16u;
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                if (i == 5 && wave != 0) break;
                copy16_to_lds(base + i * (kWaves * 1024), buf + wave * 1024u + i * (kWaves * 1024));
            }
            if (wave >= 1 && wave <= 4) copy4_to_lds(page + lane * kRow + 508u + wave * 4u, at);
        }
    }
};

// A tile that some query row does not see whole: rows that exist for none
// (bit clear in `live`) become zeros, and so do the codes of rows that hold a NaN
// code or an infinite or NaN scale, with a NaN among their RoPE values for whoever
// sees them; the others are not touched by it.  All threads; ends in a barrier.
__device__ __forceinline__ void clean_tile(uint8_t* tile, float* scales, uint64_t live) {
    const uint32_t key = threadIdx.x >> 3, j = threadIdx.x & 7u;     // 64 codes a thread
    uint8_t* row = tile + key * kRow;
    const bool gone = !((live >> key) & 1u);
    bool nan = false;
    if (!gone) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const i32x4 v = *(const i32x4*)(row + j * 64 + c * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= ((((uint32_t)v[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
        }
        if (j < 4) nan |= (__float_as_uint(scales[j * 64 + key]) & 0x7F800000u) == 0x7F800000u;
    }
    const uint64_t who = __ballot(nan);
    const bool bad = ((who >> ((threadIdx.x & 63u) & ~7u)) & 255u) != 0;
    if (gone || bad) {
        const i32x4 z = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) *(i32x4*)(row + j * 64 + c * 16) = z;
        if (j < 4) scales[j * 64 + key] = 0.f;
    }
    if (bad && j == 0) *(uint16_t*)(row + 528) = 0x7FC0;
    barrier();
}

// What one query row sees: positions below `lim`, and drafted nodes by their bits.
struct Sees {
    uint32_t lim;              // positions below lim are seen
    const uint64_t* tree;      // bits of the drafted positions from `base` on, or null
    int64_t base;
    uint32_t words;
    __device__ __forceinline__ uint64_t word(int64_t i) const { return i < (int64_t)words ? tree[i] : 0ull; }
    // Bit k: position pos + k is seen (as far as it exists).
    __device__ __forceinline__ uint64_t bits(uint32_t pos) const {
        const uint32_t left = lim > pos ? lim - pos : 0u;
        uint64_t m = left >= 64 ? ~0ull : (1ull << left) - 1;
        if (tree) {
            const int64_t j = (int64_t)pos - base;       // node of bit 0
            if (j >= 0) {
                const uint32_t s = (uint32_t)j & 63u;
                m |= word(j >> 6) >> s;
                m |= s ? word((j >> 6) + 1) << (64u - s) : 0ull;
            } else if (j > -64) {
                m |= word(0) << (uint32_t)-j;
            }
        }
        return m;
    }
};

// Sees of token i (of n) of a sequence of kv positions.
template <bool Slots>
__device__ __forceinline__ Sees sees(const AttendParams& p, const Seq& s, uint32_t i) {
    Sees v;
    v.tree = nullptr;
    v.base = (int64_t)s.kv - s.n;
    v.words = p.tree_words;
    int64_t lim = Slots ? (int64_t)s.kv : v.base + i + 1;
    if (!Slots && p.tree) {
        lim = v.base;
        v.tree = p.tree + (uint64_t)(s.q0 + i) * p.tree_words;
    }
    v.lim = lim < 0 ? 0u : (uint32_t)lim;
    return v;
}

// What a unit's rows see of its tiles.
struct View {
    uint32_t clear;            // positions below are seen by every row
    uint32_t t_end;            // none of the segment's tiles from here on is seen by any row
};

template <bool Slots>
__device__ __forceinline__ View view_of(const AttendParams& p, const Segment& g, uint32_t M, uint32_t rows, uint32_t row0) {
    View v;
    v.clear = sees<Slots>(p, g.s, row0 / p.heads).lim;
    v.t_end = g.s.kv ? g.t1 : g.t0;
    if (!Slots && !p.tree) {
        const uint32_t last = (row0 + M < rows ? row0 + M : rows) - 1;
        const uint32_t tl = (sees<Slots>(p, g.s, last / p.heads).lim + 63) / 64;
        v.t_end = v.t_end < tl ? v.t_end : tl;
    }
    return v;
}

// Counts the bad pages among tiles t0 .. t_end - 1 of which some token of the sequence
// that is computed sees a position.  By one wave, where inspect() met any: behind the
// loop over the tiles (in it, its scalars cost the loop 3 %).
__device__ __forceinline__ void count_bad_pages(const AttendParams& p, const Seq& s, const int32_t* table, int64_t capacity,
                                                uint32_t t0, uint32_t t_end) {
    const uint32_t lane = threadIdx.x & 63u, m = s.n > p.max_q ? p.max_q : s.n;
    uint32_t n = 0;
    for (uint32_t from = t0; from < t_end; from += 64) {
        const int64_t page = from + lane < t_end ? table[from + lane] : 0;
        uint64_t bad = __ballot(page < 0 || page >= capacity / 64);
        while (bad) {
            const uint32_t t = from + (uint32_t)__builtin_ctzll(bad), left = s.kv - t * 64u;
            const uint64_t live = left < 64 ? (1ull << left) - 1 : ~0ull;
            bad &= bad - 1;
            bool seen = false;
            for (uint32_t i = 0; i < m && !seen; i += 64)
                seen = __ballot(i + lane < m && (sees<false>(p, s, i + lane).bits(t * 64u) & live) != 0) != 0;
            n += seen;
        }
    }
    if (n && lane == 0) atomicAdd(p.invalid_count, (unsigned long long)n);
}

// The rows of tile t that exist (bits of live) and whether some row of the unit may
// not see it whole; such a tile is cleaned.  Bad slots are counted by the unit that has
// the token's last rows; `bad` is raised for a bad page.
template <bool Slots, class Src>
__device__ __forceinline__ void inspect(const AttendParams& p, const Src& src, const Segment& g, const View& view, uint32_t t,
                                        int64_t page, uint8_t* tile, float* scales, uint64_t& live, bool& masked, bool& bad) {
    const uint32_t left = g.s.kv - t * 64u;
    if (Slots) {
        const int64_t v = src.slots[t % kSlotRing][src.lane];
        const bool in = src.lane < left;
        live = __ballot(in && src.good(v));
        const uint64_t wrong = __ballot(in && v != -1 && !src.good(v));
        if (wrong && g.unit + 1 == g.s.units && threadIdx.x == 0) atomicAdd(p.invalid_count, (unsigned long long)__popcll(wrong));
        masked = live != ~0ull;
    } else {
        live = left < 64 ? (1ull << left) - 1 : ~0ull;
        masked = t * 64u + 64u > view.clear;
        if (page < 0) {                              // page 0 was copied in its place
            bad = true;
            live = 0;
            masked = true;
        }
    }
    if (masked) clean_tile(tile, scales, live);
}

// ---- attention ---------------------------------------------------------------------

// Row `at` of the unit, values col .. col + 16 * NB - 1: the result, or the segment's part of it.
template <int M, int NB>
__device__ __forceinline__ void write_row(const AttendParams& p, const Segment& s, uint32_t at, uint32_t col, const f32x4* o,
                                          float mx, float sum, uint32_t g) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = sum == 0.f ? -INFINITY : (mx == -INFINITY ? 0.f : mx) + log2f(sum);
    if (s.whole) {
        const uint32_t row = s.unit * M + at, i = row / p.heads, h = row - i * p.heads;
        const uint64_t t = (uint64_t)s.s.q0 + i;
        uint16_t* out = p.out + t * p.out_token + h * p.out_head + col;
#pragma unroll
        for (int d = 0; d < NB; ++d) {
            const f32x4 v = o[d] * inv;
            *(bf16x4*)(out + d * 16 + g * 4) = __builtin_convertvector(v, bf16x4);
        }
        if (p.lse && g == 0 && col == 0) p.lse[t * p.lse_token + h] = lse2 * kLn2;
    } else {
        const uint64_t x = (uint64_t)s.slot * M + at;
        float* out = p.part + x * 512 + col;
#pragma unroll
        for (int d = 0; d < NB; ++d) *(f32x4*)(out + d * 16 + g * 4) = o[d] * inv;
        if (g == 0 && col == 0) p.part_lse[x] = lse2;
    }
}

// 16 * RW rows.  RW waves split the rows, 2 a tile's keys, TW = 4 / RW the row's 512
// values: a wave forms its tiles' part of the scores, adds up the others' through LDS,
// and takes its tiles' columns of the output.  The widening (4 instructions for 8
// codes) is what the vector unit spends most of its time on.  Splitting the values
// keeps a wave's share of the queries small: a first tile is under way 2 us earlier
// than with whole rows (one sequence of 700 positions, 16 heads: 14 us, of which 4
// join; whole rows 5 us more).
template <int RW, bool Slots>
__global__ __launch_bounds__(kThreads) void attend_kernel(const AttendParams p) {
    constexpr int M = 16 * RW;
    constexpr int TW = 4 / RW;
    constexpr int T = 4 / TW;                       // tiles of 128 of a wave
    constexpr int NB = 8 * T;                       // 16-column blocks of a wave
    constexpr int kOthers = RW * 2;                 // waves between two that share rows and keys
    static_assert(RW * 2 * TW == kWaves, "every wave has its part");
    static_assert(2 * kWaves * 2048 <= kExchange, "partial scores of two tiles");
    static_assert(kWaves / 2 * (NB * 1024 + 512) <= kRing * kTileBytes, "join of key halves");
    __shared__ Shared sh;
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rw = wave % RW, kw = (wave / RW) % 2, tw = wave / kOthers;
    const uint32_t k0 = kw * 32u;                   // its keys of a tile
    const bool ropes = tw < 2;                      // RoPE half tw
    const int64_t capacity = p.head->capacity;
    Line<Slots> line(p, M, capacity <= 0, sh.exchange);
    line.leave_none();
    Segment seg;
    while (line.next(seg)) {
        const Seq& s = seg.s;
        const uint32_t b = seg.b, unit = seg.unit, t0 = seg.t0;

        // this wave's query rows
        const uint32_t m = s.n > p.max_q ? p.max_q : s.n;
        const uint32_t rows = m * p.heads, row0 = unit * M, mine = row0 + rw * 16u + l16;
        QFrag<T, 1> q[1];
        uint32_t token;
        {
            // rows behind the last one repeat it and are not written
            const uint32_t row = mine < rows ? mine : rows - 1;
            token = row / p.heads;
            const uint32_t h = row - token * p.heads;
            const uint64_t t = (uint64_t)s.q0 + token;
            q[0].load(p.q_latent + t * p.q_latent_token + h * p.q_latent_head + tw * T * 128,
                      p.q_rope + t * p.q_rope_token + h * p.q_rope_head + (tw & 1) * 32, g);
        }
        const View view = view_of<Slots>(p, seg, M, rows, row0);
        const uint32_t t_end = view.t_end;

        __builtin_amdgcn_sched_barrier(0);
        f32x4 o[NB];
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int d = 0; d < NB; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

        const Source<Slots> src{p, Slots ? nullptr : p.pages + (uint64_t)b * p.pages_stride,
                                Slots ? p.slots + (uint64_t)b * p.slots_stride : nullptr, s.kv, capacity, sh.ring, sh.scales, sh.slots, wave, lane};
        int64_t pg[3];                                   // pages of tiles t, t + 1, t + 2
        src.start(t0, t_end, pg);
        q[0].landed();
        __builtin_amdgcn_sched_barrier(0);
        // this wave's part of a tile's scores
        auto part_of = [&](uint32_t t, f32x4 (*x)[1]) {
            const uint8_t* rows32 = sh.ring + ring_of(t) * kTileBytes + k0 * kRow;
            scores32<1, T, 1>(x, rows32 + tw * T * 128, rows32 + 528 + (tw & 1) * 64,
                              &sh.scales[ring_of(t)][tw * T][k0], q, p.scale_log2, ropes, l16, g);
        };
        f32x4* const part = (f32x4*)sh.exchange + lane;  // [step & 1][wave][half u][lane]
        auto give = [&](uint32_t step, f32x4 (*x)[1]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) part[(((step & 1u) * kWaves + wave) * 2 + u) * 64] = x[u][0];
        };
        // add up the parts of the waves that share rows and keys, in one order
        auto gather = [&](uint32_t step, f32x4 (*x)[1]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const f32x4* from = part + (((step & 1u) * kWaves + wave) * 2 + u) * 64;
                if (TW == 2) {
                    x[u][0] += from[(int)((wave ^ kOthers) - wave) * 2 * 64];
                } else {
                    from -= tw * kOthers * 2 * 64;
                    f32x4 total = from[0];
#pragma unroll
                    for (int k = 1; k < TW; ++k) total += from[k * kOthers * 2 * 64];
                    x[u][0] = total;
                }
            }
        };

        // The next tile's scores are formed beside this one's weights and values, so
        // their waits overlap; one barrier a tile publishes the parts, the next tile
        // and that the last one is done with.
        f32x4 x[2][1];
        uint64_t live = ~0ull;
        bool masked = false, bad = false;
        auto look = [&](uint32_t t, int64_t page) {
            inspect<Slots>(p, src, seg, view, t, page, sh.ring + ring_of(t) * kTileBytes, &sh.scales[ring_of(t)][0][0], live, masked, bad);
        };
        if (t0 < t_end) {
            wait_own(wave, t0 + 1 < t_end);
            barrier();
            look(t0, pg[0]);
            part_of(t0, x);
            give(0, x);
        }
        uint32_t t = t0;
        for (uint32_t step = 0; t < t_end; ++step) {     // counted apart from t: 10 registers less
            const bool more = t + 1 < t_end;
            if (more) wait_own(wave, false);
            barrier();
            src.ahead(t, t_end, pg);
            gather(step, x);
            if (masked) {
                uint64_t on = live;
                if (!Slots) on &= sees<Slots>(p, s, token).bits(t * 64u);
                on >>= k0;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][0][i] = (on >> (key_of(u, g) + i)) & 1u ? x[u][0][i] : -INFINITY;
            }
            if (more) look(t + 1, pg[1]);
            float top = fmaxf(fmaxf(fmaxf(x[0][0][0], x[0][0][1]), fmaxf(x[0][0][2], x[0][0][3])),
                              fmaxf(fmaxf(x[1][0][0], x[1][0][1]), fmaxf(x[1][0][2], x[1][0][3])));
            if (__any(top > mx + kLazy || (mx == -INFINITY && top > mx))) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float next = fmaxf(mx, top);
                const float keep = mx == -INFINITY ? 0.f : exp2f(mx - next);
                mx = next;
                sum *= keep;
#pragma unroll
                for (int d = 0; d < NB; ++d) o[d] *= keep;
            }
            // the next tile's scores (behind the last tile: this one's again, not used)
            f32x4 xn[2][1];
            part_of(more ? t + 1 : t, xn);
            // weights
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[u][0][i] = __builtin_amdgcn_exp2f(x[u][0][i] - ref);
                    sum += x[u][0][i];
                }
            // values: 8 keys of this lane group (4 of each half) x 16 columns
            const uint32_t vk = key_of(l16 >> 3, g) + ((l16 >> 1) & 3u);
            const uint8_t* vrow = sh.ring + ring_of(t) * kTileBytes + (k0 + vk) * kRow + (l16 & 1u) * 8u + tw * NB * 16;
            const float* scale[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) scale[u] = &sh.scales[ring_of(t)][tw * T][k0 + key_of(u, g) + (l16 & 3)];
#pragma unroll
            for (int j = 0; j < T; ++j) {
                bf16x8 w;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const f32x4 a = quads(scale[u][j * 64]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[u * 4 + i] = (__bf16)(a[i] * x[u][0][i]);
                }
#pragma unroll
                for (int d = j * 8; d < j * 8 + 8; ++d) {
                    const i32x2 c = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lptr<i32x2>)(vrow + d * 16));
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(c.x, c.y), w, o[d], 0, 0, 0);
                }
            }
            if (!more) break;
            give(step + 1, xn);
#pragma unroll
            for (int u = 0; u < 2; ++u) x[u][0] = xn[u][0];
            ++t;
            src.turn(t, t_end, pg);
        }
        barrier();    // the ring is free

        // join the key halves, then write
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        f32x4* ex = (f32x4*)sh.ring + (uint32_t)(tw * RW + rw) * (NB * 64) + lane;
        float* stat = (float*)(sh.ring + kWaves / 2 * NB * 1024) + (uint32_t)(tw * RW + rw) * 128 + lane;
        if (kw == 1) {
#pragma unroll
            for (int d = 0; d < NB; ++d) ex[d * 64] = o[d];
            stat[0] = mx;
            stat[64] = sum;
        }
        barrier();
        if (kw == 0) {
            const float m2 = stat[0], s2 = stat[64];
            const float next = fmaxf(mx, m2);
            const float k1 = mx == -INFINITY ? 0.f : exp2f(mx - next), k2 = m2 == -INFINITY ? 0.f : exp2f(m2 - next);
            // a NaN sum with no maximum (every weight of a half a NaN) has to stay one
            sum = (mx == -INFINITY ? sum : sum * k1) + (m2 == -INFINITY ? s2 : s2 * k2);
            mx = next;
#pragma unroll
            for (int d = 0; d < NB; ++d) {
                if (d % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                const f32x4 other = ex[d * 64];
                o[d] = o[d] * (mx == -INFINITY ? 1.f : k1) + other * (mx == -INFINITY ? 1.f : k2);
            }
            if (mine < rows) write_row<M, NB>(p, seg, rw * 16u + l16, tw * NB * 16, o, mx, sum, g);
        }
        line.leave(seg, rows);
        if (!Slots && bad && wave == 0 && seg.unit + 1 == s.units) count_bad_pages(p, s, src.table, capacity, t0, t_end);
        barrier();    // before the ring takes the next unit's tiles
    }
}

// Many rows (units of 64).  A wave forms the scores of 16 rows and 32 keys of a
// tile, gives their weights to LDS, and takes 32 rows' weights for one tile of 128
// values: no score is formed twice, and a value's code is widened once for 32 rows.
// The next tile's scores are formed beside this tile's values; one barrier a tile.
// Against 4 waves of twice the rows (200 us), tiles widened once into LDS (217 us) and
// two barriers a tile (214 us) at 64 sequences of up to 8192 positions and 128 heads:
// 170 us; 16 drafted trees of 64 tokens, 32 heads, 8192 positions: 237-340 us (490-700
// TFLOP/s).  512 lists of 2048 slots, 128 heads: 521 us (units of 32 rows 738).
// The maximum the weights refer to is held by all waves alike: a row that outgrows
// it raises a flag, and all waves then agree on new ones before the weights are used.
struct WideShared {
    alignas(16) uint8_t ring[kRing * kTileBytes];
    alignas(16) f32x4 weights[2][4][2][2][64];       // [tile & 1][16 rows][32 keys][half u][lane]
    alignas(16) float scales[kRing][4][64];
    alignas(16) int64_t slots[kSlotRing][64];
    uint32_t flag[2];                                // [tile & 1]: a row outgrew its maximum
};
static_assert(sizeof(WideShared) <= 163840, "160 KB of LDS");

template <bool Slots>
__global__ __launch_bounds__(kThreads) void attend_wide_kernel(const AttendParams p) {
    constexpr int M = 64;
    using RowStats = float (*)[2][16];                   // [16 rows][32 keys][row]
    __shared__ WideShared sh;
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rw = wave & 3u, kh = wave >> 2;       // scores: rows 16 rw, keys 32 kh
    const uint32_t rp = wave & 1u, j = wave >> 1;        // values: rows 32 rp, tile j
    const int64_t capacity = p.head->capacity;
    Line<Slots> line(p, M, capacity <= 0, (uint8_t*)sh.weights);
    line.leave_none();
    Segment seg;
    if (threadIdx.x < 2) sh.flag[threadIdx.x] = 0;       // seen by all after the first barrier of a segment
    while (line.next(seg)) {
        const Seq& s = seg.s;
        const uint32_t t0 = seg.t0;
        const uint32_t m = s.n > p.max_q ? p.max_q : s.n, rows = m * p.heads, row0 = seg.unit * M;
        QFrag<4, 2> q[1];
        uint32_t token;
        {
            // rows behind the last one repeat it and are not written
            const uint32_t at = row0 + rw * 16u + l16, row = at < rows ? at : rows - 1;
            token = row / p.heads;
            const uint32_t h = row - token * p.heads;
            const uint64_t t = (uint64_t)s.q0 + token;
            q[0].load(p.q_latent + t * p.q_latent_token + h * p.q_latent_head, p.q_rope + t * p.q_rope_token + h * p.q_rope_head, g);
        }
        const View view = view_of<Slots>(p, seg, M, rows, row0);
        const uint32_t t_end = view.t_end;
        const Source<Slots> src{p, Slots ? nullptr : p.pages + (uint64_t)seg.b * p.pages_stride,
                                Slots ? p.slots + (uint64_t)seg.b * p.slots_stride : nullptr, s.kv, capacity, sh.ring, sh.scales,
                                sh.slots, wave, lane};
        int64_t pg[3];
        src.start(t0, t_end, pg);
        q[0].landed();

        f32x4 o[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int d = 0; d < 8; ++d) o[r][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float mx = -INFINITY, mo[2] = {-INFINITY, -INFINITY};     // of the score rows and of the value rows
        float sum = 0.f, fresh_sum = 0.f;
        f32x4 x[2][1];                                   // scores of the tile whose weights are given
        uint64_t live = ~0ull;
        bool masked = false, bad = false;

        auto look = [&](uint32_t t, int64_t page) {
            inspect<Slots>(p, src, seg, view, t, page, sh.ring + ring_of(t) * kTileBytes, &sh.scales[ring_of(t)][0][0], live, masked, bad);
        };
        auto scores = [&](uint32_t t, f32x4 (*to)[1]) {
            const uint8_t* rows32 = sh.ring + ring_of(t) * kTileBytes + kh * 32 * kRow;
            scores32<1, 4, 2>(to, rows32, rows32 + 528, &sh.scales[ring_of(t)][0][kh * 32], q, p.scale_log2, true, l16, g);
        };
        auto top_of = [&]() {
            return fmaxf(fmaxf(fmaxf(x[0][0][0], x[0][0][1]), fmaxf(x[0][0][2], x[0][0][3])),
                         fmaxf(fmaxf(x[1][0][0], x[1][0][1]), fmaxf(x[1][0][2], x[1][0][3])));
        };
        auto publish = [&](uint32_t t) {
            const float ref = mx == -INFINITY ? 0.f : mx;
            fresh_sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                f32x4 e;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(x[u][0][i] - ref);
                    fresh_sum += e[i];
                }
                sh.weights[t & 1u][rw][kh][u][lane] = e;
            }
        };
        // masks tile t's scores and gives their weights; raises its flag if a row outgrew its maximum
        auto offer = [&](uint32_t t) {
            if (masked) {
                uint64_t on = live;
                if (!Slots) on &= sees<Slots>(p, s, token).bits(t * 64u);
                on >>= kh * 32;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][0][i] = (on >> (key_of(u, g) + i)) & 1u ? x[u][0][i] : -INFINITY;
            }
            const float top = top_of();
            if (__any(top > mx + kLazy || (mx == -INFINITY && top > mx)) && lane == 0) sh.flag[t & 1u] = 1;
            publish(t);
        };

        if (t0 < t_end) {
            wait_own(wave, t0 + 1 < t_end);
            barrier();
            look(t0, pg[0]);
            scores(t0, x);
            offer(t0);
        }
        for (uint32_t t = t0; t < t_end; ++t) {
            const bool more = t + 1 < t_end;
            if (more) wait_own(wave, false);
            barrier();
            src.ahead(t, t_end, pg);
            if (__builtin_amdgcn_readfirstlane(sh.flag[t & 1u])) {
                RowStats tops = (RowStats)sh.weights[(t + 1) & 1u];      // free until the next tile's weights
                // new maxima, from both key halves; the weights again
                float top = top_of();
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                if (g == 0) tops[rw][kh][l16] = top;
                barrier();
                if (threadIdx.x == 0) sh.flag[t & 1u] = 0;
                const float next = fmaxf(mx, fmaxf(tops[rw][0][l16], tops[rw][1][l16]));
                sum *= mx == -INFINITY ? 0.f : exp2f(mx - next);
                mx = next;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float to = fmaxf(mo[r], fmaxf(tops[rp * 2 + r][0][l16], tops[rp * 2 + r][1][l16]));
                    const float keep = mo[r] == -INFINITY ? 0.f : exp2f(mo[r] - to);
                    mo[r] = to;
#pragma unroll
                    for (int d = 0; d < 8; ++d) o[r][d] *= keep;
                }
                publish(t);
                barrier();
            }
            sum += fresh_sum;
            if (more) look(t + 1, pg[1]);
            // this tile's values; the next one's scores (behind the last tile: this one's again, not used)
            scores(more ? t + 1 : t, x);
            // Read in this order, each code four steps ahead of its use: left to itself
            // the compiler waits for every read right behind it.
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t vk = key_of(l16 >> 3, g) + ((l16 >> 1) & 3u);
            const uint8_t* vrow = sh.ring + ring_of(t) * kTileBytes + vk * kRow + (l16 & 1u) * 8u + j * 128;
            auto column = [&](int n) {                   // 32 keys of half n / 8 by 16 columns n % 8
                return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lptr<i32x2>)(vrow + (n >> 3) * (32 * kRow) + (n & 7) * 16));
            };
            f32x4 e[2][2];
            float a[2];
            auto read_weights = [&](int half) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    a[u] = sh.scales[ring_of(t)][j][half * 32 + key_of(u, g) + (l16 & 3)];
#pragma unroll
                    for (int r = 0; r < 2; ++r) e[u][r] = sh.weights[t & 1u][rp * 2 + r][half][u][lane];
                }
            };
            bf16x8 w[2];
            auto scale_weights = [&]() {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const f32x4 s4 = quads(a[u]);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[r][u * 4 + i] = (__bf16)(s4[i] * e[u][r][i]);
                }
            };
            i32x2 c[4];
            read_weights(0);
#pragma unroll
            for (int n = 0; n < 4; ++n) c[n] = column(n);
            __builtin_amdgcn_sched_barrier(0);
            scale_weights();
            bf16x8 v = widen(c[0].x, c[0].y);
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                bf16x8 next = v;
                if (n + 4 < 16) c[n & 3] = column(n + 4);
                if (n == 3) read_weights(1);
                __builtin_amdgcn_sched_barrier(0);
                if (n < 15) next = widen(c[(n + 1) & 3].x, c[(n + 1) & 3].y);
#pragma unroll
                for (int r = 0; r < 2; ++r) o[r][n & 7] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[r], o[r][n & 7], 0, 0, 0);
                if (n == 7) scale_weights();
                v = next;
                __builtin_amdgcn_sched_barrier(0);
            }
            if (!more) break;
            src.turn(t + 1, t_end, pg);
            offer(t + 1);
        }
        // the rows' sums, from both key halves
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        barrier();
        RowStats sums = (RowStats)sh.weights[0];
        if (g == 0) sums[rw][kh][l16] = sum;
        barrier();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t at = (rp * 2 + r) * 16u + l16;
            const float total = sums[rp * 2 + r][0][l16] + sums[rp * 2 + r][1][l16];
            if (row0 + at < rows) write_row<M, 8>(p, seg, at, j * 128, o[r], mo[r], total, g);
        }
        line.leave(seg, rows);
        if (!Slots && bad && wave == 0 && seg.unit + 1 == s.units) count_bad_pages(p, s, src.table, capacity, t0, t_end);
        barrier();    // before the ring and the sums serve the next unit
    }
}

// Joins the partial results of the units that were cut between blocks: a group of
// 128 threads takes one (token, head) row, 4 columns a thread, and adds the blocks'
// parts in order, four on their way together (one at a time: 2.5 us more for 6
// parts).  Each wave counts the cut units for itself, by ballots over the blocks'
// notes: a grid with blocks for units that are not there costs 4 us more (slots 16 x
// 2048).  4 us for 256 rows of 4 parts, a chain of three reads from memory; 12 us for
// 8192 rows of 1 to 3 parts.
__global__ __launch_bounds__(256) void combine_kernel(const AttendParams p, uint32_t M, uint32_t blocks) {
    const uint32_t lane = threadIdx.x & 63u, col = (threadIdx.x & 127u) * 4u;
    uint32_t last[4];
    uint64_t mask[4];
    uint32_t cut = 0;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) last[j] = j * 64u + lane < blocks ? p.cut_last[j * 64u + lane] : 0u;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        mask[j] = __ballot(last[j] != 0);
        cut += (uint32_t)__popcll(mask[j]);
    }
    for (uint32_t x = blockIdx.x * 2u + (threadIdx.x >> 7); x < cut * M; x += gridDim.x * 2u) {
        // the unit that block w0 began and block w1 ends, by its place among the cut ones
        uint32_t k = __builtin_amdgcn_readfirstlane(x >> __builtin_ctz(M)), w0 = 0, w1 = 0;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t n = (uint32_t)__popcll(mask[j]);
            if (w1 == 0 && k < n) {
                const bool it = ((mask[j] >> lane) & 1u) && (uint32_t)__popcll(mask[j] & ((1ull << lane) - 1)) == k;
                const uint32_t at = (uint32_t)__builtin_ctzll(__ballot(it));
                w0 = j * 64u + at;
                w1 = __builtin_amdgcn_readlane(last[j], at);
            }
            k -= n;
        }
        const kptr<AttendCut> unit = (kptr<AttendCut>)(p.cuts + w0);
        const uint32_t in = x & (M - 1), row = unit->row0 + in, slot = unit->slot, q0 = unit->q0;
        if (row >= unit->rows) continue;
        // four parts at a time, their sums and rows on the way together; behind the
        // last part it again, with no weight
        float top = -INFINITY, total = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t w = w0; w <= w1; w += 4) {
            float lse[4];
            f32x4 v[4];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const uint32_t c = w + k < w1 ? w + k : w1;
                const uint64_t at = (uint64_t)(c == w0 ? slot : 2 * c) * M + in;
                lse[k] = p.part_lse[at];
                v[k] = *(const f32x4*)(p.part + at * 512 + col);
            }
            float next = top;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                lse[k] = w + k <= w1 ? lse[k] : -INFINITY;
                next = fmaxf(next, lse[k]);
            }
            const float keep = top == -INFINITY ? 1.f : exp2f(top - next);      // nothing with a weight yet, or a NaN
            total *= keep;
            o *= keep;
            top = next;
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const float e = exp2f(lse[k] - ref);
                total += e;
                o += v[k] * e;
            }
        }
        const float ref = top == -INFINITY ? 0.f : top;
        const uint32_t i = row / p.heads, h = row - i * p.heads;
        const uint64_t t = (uint64_t)q0 + i;
        o = o * (total == 0.f ? 0.f : 1.f / total);
        *(bf16x4*)(p.out + t * p.out_token + h * p.out_head + col) = __builtin_convertvector(o, bf16x4);
        if (p.lse && col == 0) p.lse[t * p.lse_token + h] = total == 0.f ? -INFINITY : (ref + log2f(total)) * kLn2;
    }
}

// ---- accumulated weights ------------------------------------------------------------

// A block takes a run of a sequence's tiles (with many sequences its run of the line,
// a unit being all rows of a sequence), up to kWeightTiles of them at a time, and passes over the
// sequence's query rows, 128 at a time: 4 waves of 32 rows for either half of a
// tile's keys, the operands in registers.  A position belongs to one block: its sum over rows
// runs within a wave (DPP over the 16 rows of a lane group), pass by pass and wave
// by wave, always in that order.  A wave has 32 rows, so that a widened operand (4
// vector instructions) serves two matrix instructions: with 16 rows 87 us, with 32
// 69 us for 16 sequences of up to 16384 positions and 128 heads; one line instead of
// equal runs of each sequence's bound 53 us, runs that keep to one sequence 39-48 us
// (92 MB: 18 us at a copy's rate; 28 us with the scores left out).  Bound by the vector
// unit: 6000 cycles a tile of 128 rows, of which the matrix units need 2300.
constexpr uint32_t kWeightTiles = 16;

struct WeightShared {
    alignas(16) uint8_t ring[kRing * kTileBytes];
    alignas(16) float scales[kRing][4][64];
    float sums[4][kWeightTiles * 64];                // [rows][position]
};

// Sum over the 16 lanes of a row: every lane gets it.
template <int R>
__device__ __forceinline__ float rotate_add(float v) {      // row_ror:R
    return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + R, 15, 15, true));
}
__device__ __forceinline__ float sum16(float v) { return rotate_add<1>(rotate_add<2>(rotate_add<4>(rotate_add<8>(v)))); }

__device__ __forceinline__ void add_weights(const AttendParams& p, uint32_t b, uint32_t pos, float v) {
    const uint64_t at = (uint64_t)b * p.weights_stride + pos;
    p.weights_out[at] = (p.weights_in ? p.weights_in[at] : 0.f) + v;
}

template <bool Few>
__global__ __launch_bounds__(kThreads) void weights_kernel(const AttendParams p) {
    __shared__ WeightShared sh;
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rw = wave & 3u, kh = wave >> 2;       // rows 32 rw of a pass, keys 32 kh of a tile
    const uint32_t M = p.max_q * p.heads;                // one unit a sequence
    const int64_t capacity = p.head->capacity;

    // positions that no tile of the line holds, 1024 at a time: nothing is added
    const uint32_t spans = (p.max_kv + 1023) / 1024;
    for (uint64_t i = blockIdx.x; i < (uint64_t)spans * p.num_seqs; i += gridDim.x) {
        const uint32_t b = (uint32_t)(i / spans), from = (uint32_t)(i - (uint64_t)b * spans) * 1024u;
        uint32_t held = 0;
        if (p.num_tokens) {
            const Seq s = sequence<false, true>(p, b, M, capacity <= 0);
            held = s.units * s.tiles * 64u;
        }
        const uint32_t end = from + 1024u < p.max_kv ? from + 1024u : p.max_kv;
        for (uint32_t pos = (from < held ? held : from) + threadIdx.x; pos < end; pos += kThreads) add_weights(p, b, pos, 0.f);
    }
    if (!p.num_tokens) return;

    std::conditional_t<Few, Runs, Line<false>> line = [&] {
        if constexpr (Few) return Runs(p, M, capacity <= 0);
        else return Line<false>(p, M, capacity <= 0, (uint8_t*)sh.sums);
    }();
    Segment seg;
    uint32_t t1 = 0;
    bool left = line.next(seg);
    while (left) {
        const Seq& s = seg.s;
        const uint32_t t0 = seg.t0;
        t1 = seg.t1 < t0 + kWeightTiles ? seg.t1 : t0 + kWeightTiles;
        const uint32_t end = s.kv ? t1 : t0;                 // a sequence without positions has one empty tile
        const uint32_t m = s.n > p.max_q ? p.max_q : s.n, rows = m * p.heads;
        for (uint32_t i = threadIdx.x; i < 4 * kWeightTiles * 64; i += kThreads) (&sh.sums[0][0])[i] = 0.f;
        const int64_t base = (int64_t)s.kv - s.n;
        View view;                                           // every token sees the positions below `clear`
        view.clear = base < 0 ? 0u : (uint32_t)(p.tree ? base : base + 1);
        view.t_end = end;
        bool bad = false;
        const Source<false> src{p, p.pages + (uint64_t)seg.b * p.pages_stride, nullptr, s.kv, capacity, sh.ring, sh.scales, nullptr, wave, lane};

        for (uint32_t row0 = 0; row0 < rows && t0 < end; row0 += 128) {
            QFrag<4, 2> q[2];
            uint32_t token[2];
            float lse2[2];
            bool adds[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t at = row0 + rw * 32u + r * 16u + l16, row = at < rows ? at : rows - 1;
                token[r] = row / p.heads;
                const uint32_t h = row - token[r] * p.heads;
                const uint64_t t = (uint64_t)s.q0 + token[r];
                q[r].load(p.q_latent + t * p.q_latent_token + h * p.q_latent_head, p.q_rope + t * p.q_rope_token + h * p.q_rope_head, g);
                // a row of -inf saw nothing; rows behind the last one add nothing
                const float lse = p.lse[t * p.lse_token + h];
                adds[r] = at < rows && lse != -INFINITY;
                lse2[r] = lse * 1.44269504088896341f;
            }
            barrier();                                       // the ring is free
            int64_t pg[3];
            src.start(t0, end, pg);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                q[r].landed();
                asm volatile("" : "+v"(lse2[r]));
            }
            for (uint32_t t = t0; t < end; ++t) {
                wait_own(wave, t + 1 < end);
                barrier();
                src.ahead(t, end, pg);
                uint8_t* tile = sh.ring + ring_of(t) * kTileBytes;
                float* scales = &sh.scales[ring_of(t)][0][0];
                uint64_t live;
                bool masked;
                inspect<false>(p, src, seg, view, t, pg[0], tile, scales, live, masked, bad);
                src.turn(t + 1, end, pg);
                f32x4 x[2][2];
                const uint8_t* rows32 = tile + kh * 32 * kRow;
                scores32<2, 4, 2>(x, rows32, rows32 + 528, scales + kh * 32, q, p.scale_log2, true, l16, g);
                if (masked) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint64_t on = (live & sees<false>(p, s, token[r]).bits(t * 64u)) >> (kh * 32);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[u][r][i] = (on >> (key_of(u, g) + i)) & 1u ? x[u][r][i] : -INFINITY;
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float keep = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float w = 0.f;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float e = __builtin_amdgcn_exp2f(x[u][r][i] - lse2[r]);
                            w += adds[r] ? e : 0.f;
                        }
                        const float total = sum16(w);
                        keep = (int)l16 == i ? total : keep;
                    }
                    if (l16 < 4) sh.sums[rw][(t - t0) * 64 + kh * 32 + key_of(u, g) + l16] += keep;
                }
            }
        }
        __syncthreads();
        if (bad && wave == 0) count_bad_pages(p, s, src.table, capacity, t0, end);
        for (uint32_t k = threadIdx.x; k < (t1 - t0) * 64u; k += kThreads) {
            const uint32_t pos = t0 * 64u + k;
            if (pos >= p.max_kv) break;
            add_weights(p, seg.b, pos, (sh.sums[0][k] + sh.sums[1][k]) + (sh.sums[2][k] + sh.sums[3][k]));
        }
        __syncthreads();
        if (t1 < seg.t1) seg.t0 = t1;
        else left = line.next(seg);
    }
}

}  // namespace

AttendPlan plan_attend(uint64_t rows, uint64_t num_seqs, uint64_t num_tokens, uint64_t heads, uint64_t max_kv) {
    AttendPlan a;
    const uint64_t tiles = max_kv ? (max_kv + 63) / 64 : 1;
    uint64_t units = 0;
    const auto runs_of = [&](uint32_t M) {
        units = num_seqs * ((rows + M - 1) / M);
        const uint64_t by_tokens = num_tokens * heads / M + num_seqs;       // ragged: no more units than that
        units = units < by_tokens ? units : by_tokens;
        return units * tiles + 1;
    };
    // Rows of a unit.  64 (attend_wide_kernel) from ten tiles a block on: its tile of 64
    // rows takes 3.1 us, two of 32 rows 4.2 us, but it starts 8 us later (16 sequences
    // of 128 heads, 4096 positions: 56.4 us against 54.9; 8192: 81.3 against 88.6; lists of
    // 2048 slots for 40 tokens: 80 against 76; 64 tokens: 83 against 88; 128: 123 against 167).
    // 16 where that holds all rows, or where a line of longer units would leave CUs idle
    // (4 tokens of 64 heads, 256 slots: 15.4 us against 23 with units of 64 rows).  A run
    // may be one tile: 12.4 us then, against 14.7 with two at least.
    uint64_t runs = runs_of(64);
    a.rows = 64;
    if (rows <= 32 || units * tiles < 10 * 256) {
        runs = runs_of(16);
        a.rows = 16;
        if (rows > 16 && runs > 512) {
            runs = runs_of(32);
            a.rows = 32;
        }
    }
    a.fits = units * tiles < (1ull << 31);
    // one block a CU; never more than the line has runs
    a.blocks = (uint32_t)(runs >= kMostBlocks ? kMostBlocks : runs);
    // two rows a block of the join; no more units are cut than blocks end inside one
    const uint64_t cut_rows = (units < a.blocks ? units : a.blocks) * a.rows;
    a.joins = (uint32_t)(cut_rows / 2 < 4096 ? cut_rows / 2 : 4096);
    a.lse_bytes = (uint64_t)a.blocks * 2 * a.rows * 4;
    a.bytes = kCutBytes + a.lse_bytes + (uint64_t)a.blocks * 2 * a.rows * 512 * 4;
    return a;
}

hipError_t launch_attend(const AttendParams& given, void* workspace, hipStream_t stream) {
    AttendParams p = given;
    const AttendPlan a = plan_attend((uint64_t)p.max_q * p.heads, p.num_seqs, p.num_tokens, p.heads,
                                     p.by_slots ? p.num_slots : p.max_kv);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.cut_last = reinterpret_cast<uint32_t*>(ws);
    p.cuts = reinterpret_cast<AttendCut*>(ws + kMostBlocks * sizeof(uint32_t));
    p.part_lse = reinterpret_cast<float*>(ws + kCutBytes);
    p.part = reinterpret_cast<float*>(ws + kCutBytes + a.lse_bytes);
    (void)hipGetLastError();
    const dim3 grid(a.blocks), block(kThreads);
    if (a.rows == 16) {
        if (p.by_slots) attend_kernel<1, true><<<grid, block, 0, stream>>>(p);
        else attend_kernel<1, false><<<grid, block, 0, stream>>>(p);
    } else if (a.rows == 32) {
        if (p.by_slots) attend_kernel<2, true><<<grid, block, 0, stream>>>(p);
        else attend_kernel<2, false><<<grid, block, 0, stream>>>(p);
    } else {
        if (p.by_slots) attend_wide_kernel<true><<<grid, block, 0, stream>>>(p);
        else attend_wide_kernel<false><<<grid, block, 0, stream>>>(p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    combine_kernel<<<dim3(a.joins), dim3(256), 0, stream>>>(p, a.rows, a.blocks);
    return hipGetLastError();
}

hipError_t launch_attend_weights(const AttendParams& given, hipStream_t stream) {
    AttendParams p = given;
    const uint64_t tiles = (uint64_t)((p.max_kv + 63) / 64) * p.num_seqs;
    (void)hipGetLastError();
    const dim3 grid((uint32_t)(tiles < 256 ? tiles : 256));
    if (p.num_seqs <= 64) weights_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else weights_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace kvpub
