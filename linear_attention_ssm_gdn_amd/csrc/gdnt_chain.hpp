// gdnt_chain.hpp -- how a state travels from tile to tile inside one launch.
//
// Tiles are handed out by a ticket in the order of the recurrence, so a tile
// only ever waits for tiles that already run: every wait ends.  A tile first
// publishes its run (h -> a h + u), then looks back over up to eight tiles
// for the nearest one whose end state is known, applies the runs in between
// in order, and publishes its own end state.  The order makes the bits the
// same whichever tile the state was found at.  A value and its ready mark
// share one 64-bit word, stored and loaded with device-scope atomics, so no
// fence is needed; the words start from zero.
#pragma once

#include "gdnt_device.hpp"

namespace gdnt {

// A run that contains a first row (in the direction of the recurrence) is
// marked by a negative `a`: nothing before it matters.
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
constexpr int kLookBack = 8;
constexpr int kSpins = 1 << 21;  // some seconds, far beyond any tile's run

__device__ __forceinline__ uint64_t chain_load(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void chain_store(uint64_t* p, uint32_t hi, float lo) {
    __hip_atomic_store(p, ((uint64_t)hi << 32) | (uint64_t)__float_as_uint(lo), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// One wave, NCH channels a lane from word `at` on; `step` words to the tile
// before, of which n_pred exist.  The state before the tile, into h.
template <int NCH>
__device__ __forceinline__ void look_back(const Chain& C, int64_t at, int64_t step, int64_t n_pred, float (&h)[NCH],
                                          int32_t* err) {
    const int lane = threadIdx.x & 63, j = (lane & 7) + 1;
    // first the column's first channel alone, for all eight tiles
    int found = -1;
    for (int spin = 0; spin < kSpins; ++spin) {
        uint64_t v = 0;
        if (lane < 2 * kLookBack && j <= n_pred) v = chain_load(C.state + (lane & 8 ? C.run : 0) + at + j * step);
        const uint64_t ready = __ballot((v >> 32) != 0);
        const uint32_t states = (uint32_t)ready & 0xffu, runs = (uint32_t)(ready >> 8) & 0xffu;
        if (states) {
            const int k = __builtin_ctz(states);
            if (!(~runs & ((1u << k) - 1u))) {
                found = k;
                break;
            }
        }
        __builtin_amdgcn_s_sleep(2);
    }
    if (found >= 0) {
        for (int spin = 0; spin < kSpins; ++spin) {
            uint64_t s[NCH], g[kLookBack - 1][NCH];
            const int64_t mine = at + lane * NCH;
            bool ok = true;
#pragma unroll
            for (int i = 0; i < NCH; ++i) s[i] = chain_load(C.state + mine + (found + 1) * step + i);
#pragma unroll
            for (int q = 0; q < kLookBack - 1; ++q)
                if (q < found) {
#pragma unroll
                    for (int i = 0; i < NCH; ++i) g[q][i] = chain_load(C.state + C.run + mine + (q + 1) * step + i);
                }
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                ok = ok && (s[i] >> 32) != 0;
                h[i] = __uint_as_float((uint32_t)s[i]);
            }
#pragma unroll
            for (int q = kLookBack - 2; q >= 0; --q)
                if (q < found) {
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        ok = ok && (g[q][i] >> 32) != 0;
                        h[i] = fmaf(__uint_as_float((uint32_t)(g[q][i] >> 32) & 0x7fffffffu), h[i],
                                    __uint_as_float((uint32_t)g[q][i]));
                    }
                }
            if (__all(ok)) return;
            __builtin_amdgcn_s_sleep(1);
        }
    }
    raise(err, GDNT_DEVERR_TIMEOUT);
#pragma unroll
    for (int i = 0; i < NCH; ++i) h[i] = 0.0f;
}

// One wave: from the tile's run (a, u) the state before it, into h (0 where
// nothing continues into it); the tile after it, where one continues, is told.
template <int NCH>
__device__ __forceinline__ void hand_on(const Chain& C, int64_t at, int64_t step, int64_t n_pred, bool cont, bool next,
                                        const float (&a)[NCH], const float (&u)[NCH], float (&h)[NCH], int32_t* err) {
    const int64_t mine = at + (threadIdx.x & 63) * NCH;
    // a tile with a first row in it, or that continues nothing, knows its end
    const bool known = a[0] < 0.0f || !cont;  // the same in every channel
    if (next) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (known) chain_store(C.state + mine + i, 1u, u[i]);
            else chain_store(C.state + C.run + mine + i, __float_as_uint(a[i]) | 0x80000000u, u[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) h[i] = 0.0f;
    if (cont) look_back<NCH>(C, at, step, n_pred, h, err);
    if (next && !known) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) chain_store(C.state + mine + i, 1u, fmaf(a[i], h[i], u[i]));
    }
}

}  // namespace gdnt
