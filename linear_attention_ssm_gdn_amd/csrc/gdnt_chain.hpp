// gdnt_chain.hpp -- how a state travels from tile to tile inside one launch:
// the published single-pass scan with decoupled look-back (Merrill and Garland,
// 2016), for runs h -> a h + u.
//
// Tiles are handed out by a ticket in the order of the recurrence, so a tile
// only ever waits for tiles that already run: every wait ends.  A tile first
// publishes its run (h -> a h + u), then looks back over up to four tiles
// for the nearest one whose end state is known, applies the runs in between
// in order, and publishes its own end state.  The order makes the bits the
// same whichever tile the state was found at.  A value and its ready mark
// share one 64-bit word, stored and loaded with device-scope atomics, so no
// fence is needed; the words start from zero.
#pragma once

#include "gdnt_device.hpp"

namespace gdnt {

// A run that contains a first row (in the direction of the recurrence) is
// marked by a negative `a`: nothing before it matters.  The mark comes from the
// row map alone, never from the sign of what was computed: a NaN gate's sign
// says nothing, and a tile's channels have to agree (end_known).
__device__ __forceinline__ float marked(float a, bool first) {
    const float m = fmaxf(a, kTiny);  // a decay, so a >= 0; a NaN becomes kTiny, and is in u as well
    return first ? -m : m;
}
__device__ __forceinline__ float walk(float a, float u, float h) { return a < 0.0f ? u : fmaf(a, h, u); }
// first `p`, then `q`, into q.  |a| stays a normal number, so an Inf passes
// through a run whose decays underflow as Inf, not as NaN; a finite state is
// changed by less than 1e-38 of it.
__device__ __forceinline__ void join(float pa, float pu, float& qa, float& qu) {
    if (qa >= 0.0f) {
        qu = fmaf(qa, pu, qu);
        qa = copysignf(fmaxf(fabsf(pa) * qa, kTiny), pa);
    }
}

struct Chain {
    uint64_t* state;  // {1, end state}
    int64_t run;      // as many words further: {a with its sign bit set, u}, a > 0
};
constexpr int kLookBack = 4;
constexpr int kSpins = 1 << 21;  // some seconds, far beyond any tile's run

__device__ __forceinline__ uint64_t chain_load(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void chain_store(uint64_t* p, uint32_t hi, float lo) {
    __hip_atomic_store(p, ((uint64_t)hi << 32) | (uint64_t)__float_as_uint(lo), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// One wave, NCH channels a lane from word `at` on; `step` words to the tile
// before, of which n_pred exist.  The state before the tile, into h.  Every
// poll asks for all words at once: a trip to memory costs as much as a walk
// (forward and backward over 32768 x 4096 in bf16: 910 us one tile at a time,
// 838 four at once; six cost registers, 278 against 260 us forward).
template <int NCH>
__device__ __forceinline__ void look_back(const Chain& C, int64_t at, int64_t step, int64_t n_pred, float (&h)[NCH],
                                          int32_t* err) {
    const uint64_t* p = C.state + at + (threadIdx.x & 63) * NCH;
    for (int spin = 0; spin < kSpins; ++spin) {
        uint64_t s[kLookBack][NCH], g[kLookBack][NCH];
#pragma unroll
        for (int q = 0; q < kLookBack; ++q)
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                s[q][i] = q < n_pred ? chain_load(p + (q + 1) * step + i) : 0;
                g[q][i] = q < n_pred && q < kLookBack - 1 ? chain_load(p + C.run + (q + 1) * step + i) : 0;
            }
        // the nearest known state with every run behind it known, in all channels
        int found = -1;
        bool runs = true;
#pragma unroll
        for (int q = 0; q < kLookBack; ++q) {
            bool ready = true, run = true;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                ready = ready && (s[q][i] >> 32) != 0;
                run = run && (g[q][i] >> 32) != 0;
            }
            if (found < 0 && runs && __all(ready)) found = q;
            runs = runs && __all(run);
        }
        if (found >= 0) {
#pragma unroll
            for (int q = kLookBack - 1; q >= 0; --q)
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    if (q == found) h[i] = __uint_as_float((uint32_t)s[q][i]);
                    else if (q < found)
                        h[i] = fmaf(__uint_as_float((uint32_t)(g[q][i] >> 32) & 0x7fffffffu), h[i],
                                    __uint_as_float((uint32_t)g[q][i]));
                }
            return;
        }
        __builtin_amdgcn_s_sleep(2);
    }
    // not a number from here on: whoever does not look at err sees it in the results
    raise(err, GDNT_DEVERR_TIMEOUT);
#pragma unroll
    for (int i = 0; i < NCH; ++i) h[i] = __uint_as_float(0x7fc00000u);
}

// A tile with a first row in it, or that continues nothing, knows its end from
// its run alone (the same in every channel).
template <int NCH> __device__ __forceinline__ bool end_known(const float (&a)[NCH], bool cont) {
    return a[0] < 0.0f || !cont;
}
// One wave tells the tile after it, if one continues, its run or known end.
template <int NCH>
__device__ __forceinline__ void tell_run(const Chain& C, int64_t at, bool cont, bool next, const float (&a)[NCH],
                                         const float (&u)[NCH]) {
    uint64_t* mine = C.state + at + (threadIdx.x & 63) * NCH;
    if (!next) return;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        if (end_known(a, cont)) chain_store(mine + i, 1u, u[i]);
        else chain_store(mine + C.run + i, __float_as_uint(a[i]) | 0x80000000u, u[i]);
    }
}
// The same wave, later: the state before the tile into h (0 where nothing
// continues into it), and the tile's end to the tile after it.
template <int NCH>
__device__ __forceinline__ void hand_on(const Chain& C, int64_t at, int64_t step, int64_t n_pred, bool cont, bool next,
                                        const float (&a)[NCH], const float (&u)[NCH], float (&h)[NCH], int32_t* err) {
    uint64_t* mine = C.state + at + (threadIdx.x & 63) * NCH;
#pragma unroll
    for (int i = 0; i < NCH; ++i) h[i] = 0.0f;
    if (cont) look_back<NCH>(C, at, step, n_pred, h, err);
    if (next && !end_known(a, cont)) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) chain_store(mine + i, 1u, fmaf(a[i], h[i], u[i]));
    }
}

}  // namespace gdnt
