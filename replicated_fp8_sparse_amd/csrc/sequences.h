// The sequences of a call on the cache of heads (kvpub_pages), in device code.
#pragma once

#include <algorithm>

#include "kvpub_internal.h"

namespace kvpub {

struct SeqOf {
    uint32_t b;          // the sequence
    uint32_t q0;         // its first token
    uint32_t n;          // its tokens
    uint32_t m;          // of these, the first max_q that the call takes
    uint32_t kv;         // its positions, the new ones included
    uint32_t place;      // of the looked-for place among its own
    bool found;
};

// Places for `pieces` a token: num / 2^shift of them, and `more` a sequence.
struct Places {
    uint32_t num, shift, more;
    __device__ __forceinline__ uint64_t key(uint32_t q0, uint32_t b) const {
        return (((uint64_t)q0 * num) >> shift) + (uint64_t)b * more;
    }
};

// Call-wide places for pieces of the sequences (blocks of 64 positions, units of
// query rows) without a list of them: sequence b's begin at key(b) = floor(q_start[b] *
// num / 2^shift) + b * more, which leaves at least floor(n num / 2^shift) + more for its n
// tokens.  Every lane of the wave gets the same answer: 64 candidates a step, 3 steps for 65536.
// q_start is taken as within the call's tokens; what is not ascending gives
// places that are found wrong, never outside the arrays.
__device__ __forceinline__ uint32_t within_tokens(const SeqParams& p, int32_t q) {
    return q < 0 ? 0u : ((uint32_t)q > p.num_tokens ? p.num_tokens : (uint32_t)q);
}

// A uniform load through the scalar cache, of what no kernel of the call writes: its
// wait does not drain the vector loads in flight.
template <class T> using kptr = const __attribute__((address_space(4))) T*;
__device__ __forceinline__ int32_t uniform_load(const int32_t* p, uint64_t i) { return ((kptr<int32_t>)p)[i]; }

__device__ __forceinline__ SeqOf find_sequence(const SeqParams& p, uint32_t place, const Places& w) {
    uint32_t lo = 0;
    bool found = true;
    if (w.num == 0) {                       // as many places for each sequence
        lo = place / w.more;
        found = lo < p.num_seqs;
        lo = found ? lo : 0;
    } else {
        const uint32_t lane = threadIdx.x & 63u;
        uint32_t size = p.num_seqs;
        while (size > 1) {
            const uint32_t step = (size + 63) / 64, at = lo + lane * step;
            const bool is = lane * step < size;
            const uint64_t key = is ? w.key(within_tokens(p, p.q_start[at]), at) : ~0ull;
            const uint64_t below = __ballot(is && key <= place);
            if (!below) { found = false; break; }
            const uint32_t k = 63u - (uint32_t)__builtin_clzll(below);
            const uint32_t end = lo + size;
            lo += k * step;
            size = step < end - lo ? step : end - lo;
        }
    }
    SeqOf s;
    s.b = __builtin_amdgcn_readfirstlane(lo);
    const int32_t len = uniform_load(p.kv_len, s.b);
    uint32_t end = s.b + 1;
    s.q0 = s.b;
    if (p.q_start) {
        const int32_t q0 = uniform_load(p.q_start, s.b), q1 = uniform_load(p.q_start, s.b + 1);
        s.q0 = within_tokens(p, q0);
        end = within_tokens(p, q1);
    }
    s.n = end > s.q0 ? end - s.q0 : 0u;
    s.m = s.n < p.max_q ? s.n : p.max_q;
    s.kv = len < 0 ? 0u : ((uint32_t)len < p.max_kv ? (uint32_t)len : p.max_kv);
    const uint64_t key = w.key(s.q0, s.b);
    s.found = found && place >= key;
    s.place = (uint32_t)(place - key);
    return s;
}

// By tokens, or as many for each sequence as its bound asks for (`most`), whichever
// pads less; *total: how many in all.
inline Places places(uint32_t num, uint32_t shift, uint32_t more, uint64_t most, uint64_t num_seqs, uint64_t num_tokens, uint64_t* total) {
    const uint64_t by_tokens = ((num_tokens * num) >> shift) + num_seqs * more;
    *total = std::min(by_tokens, num_seqs * most);
    return num_seqs * most <= by_tokens ? Places{0, 0, (uint32_t)most} : Places{num, shift, more};
}

}  // namespace kvpub
