// gdnt_scan_bwd.hip -- the backward pass of the vector-state gated linear
// recurrence.  With alpha = e^{g} and mu_t = alpha_t lambda_t,
//   lambda_t = dh_t + mu_{t+1},
// a recurrence of the same kind from the last row to the first; h_{t-1} is
// made again from the state kept every 256 rows.
//
// A tile is therefore 256 packed rows by 64 channels, one workgroup of eight
// waves: half a wave holds 16 consecutive rows, a lane two channels of each.
// A lane turns its rows into two runs (h -> a h + u), one in each direction;
// the runs of a tile are joined between the halves and through LDS, mu comes
// from the tile behind (gdnt_chain.hpp), and each lane walks its rows again
// from registers: first forward for the states, then back for the gradients.
// What a gradient needs of the gates is kept from the first walk: 256
// registers cost less than the transcendentals again (with 128, and so two
// workgroups on a compute unit, it does not fit without spilling).  One
// workgroup on a compute unit has nothing to compute while it loads, so it
// stays there, draws tile after tile, and loads the next tile's rows into LDS
// (128 KB in bf16) while it computes.
//
// 32768 x 4096 in bf16 takes 460 us for 1.88 GB (4.1 TB/s, 81% of a large
// copy's rate) at 72 vector instructions an element (58% of the issue slots);
// from the checkpoint 470 us for 1.50 GB, 82 instructions (64%).  What is left
// is neither: a tile's eight waves meet three times, and wait for mu from the
// tile behind (10 to 20 of some 50 thousand cycles).  fp32 rows take all 256
// registers and nine more, which are spilled (40 bytes a lane); 13212 x 2050
// take 228 us.
#include "gdnt_chain.hpp"
#include "gdnt_rows.hpp"

namespace gdnt {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
static_assert(kWaves * 2 * FR == kTileRows && 32 * 2 == kTileCols, "tile shape");
static_assert(kThreads == kScanThreads, "launch size");

// The largest scale whose 127-fold is finite: that of a block around the
// largest fp32 number is one step above it.
constexpr float kTopScale = 0x1.020406p+121f;

// The lane's 16 rows by two channels of one tensor of the checkpoint.
// A value is taken by half: byte * (sc / 2) - 64 sc, the byte unsigned (offset
// by 128), in one fused operation.  64 sc is exact and finite for every scale,
// while 128 sc is not for a block that holds the largest numbers, and halving
// and doubling change no digit, so what is rounded is q * scale / 2.
struct Ckpt2 {
    uint32_t w[FR / 2];
    float sc, off;
    // eight whole rows of the block, as this lane stored them; sc is set to the scale
    __device__ __forceinline__ void set(uint4 lo, uint4 hi, int lane) {
        const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        sc = 0.5f * (sc > kTopScale ? kTopScale : sc);  // a NaN stays
        off = -128.0f * sc;
#pragma unroll
        for (int r = 0; r < FR / 2; ++r) w[r] = swap_halves(v[r], lane) ^ 0x80808080u;
    }
    __device__ __forceinline__ float half(int r, int i) const {
        const uint32_t b = (w[r & 7] >> ((r >> 3) * 16 + i * 8)) & 0xffu;
        return fmaf((float)b, sc, off);
    }
};

// Makes the compiler take a register's value for a new one: what was computed
// from it before is computed again instead of being kept in more registers.
__device__ __forceinline__ void again(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void again(uint32_t& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void again(float2& v) { again(v.x); again(v.y); }
// The same for a uniform value, and for a lane's number: keeps what a tile
// makes of them from being held in registers from tile to tile.
__device__ __forceinline__ uint32_t fresh_scalar(uint32_t v) {
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ int fresh_lane(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// One 16-byte (or 4-byte) load a lane from sbase + voff straight into LDS at
// lds + 16 (4) * lane.  Written as an instruction the compiler does not see as
// an LDS write: it would put a wait for all of them before every later LDS
// read.  The kernel waits itself (stage_wait); the load has no result register.
__device__ __forceinline__ void stage16(const void* sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void stage4(const void* sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
// Every load of this wave has arrived, in LDS too.
__device__ __forceinline__ void stage_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// The LDS reads of what the stage held are done.
__device__ __forceinline__ void stage_free() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <typename P> __device__ __forceinline__ P* scalar_ptr(P* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<P*>((uintptr_t)((hi << 32) | lo));
}

// A wave's place in LDS for its next rows: 4 KB for each bf16 tensor, line r
// of 256 bytes being row r of the first half and row r of the second; of a
// checkpoint 2 KB for each tensor, two lots of 16 bytes a lane, and the scales.
// In front of them, of the tile's 64 channels: dt_bias, A_log and the kept state.
constexpr int kStageHead = 3 * 256, kStageRows = 4096, kStageCkpt = 2048 + 256;
constexpr int stage_bytes(bool ckpt) { return kStageHead + (ckpt ? kStageRows + 3 * kStageCkpt : 4 * kStageRows); }

// The kernel's arguments read again where they are used once in a while: kept
// in registers all the time they would push others out.
__device__ __forceinline__ const __attribute__((address_space(4))) ScanArgs* rare_args() {
    auto p = (const __attribute__((address_space(4))) ScanArgs*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// PIPE: x, a, b (or the checkpoint) and dh of the next tile load into LDS
// while this one is computed.  For bf16 rows on 16 bytes and channels a
// multiple of 8: forward and backward over 16692 rows take 401 us with 4096
// channels, 571 with 4094, which go without (fp32 rows would not fit in LDS).
template <typename T, bool PAIR, bool CKPT, bool PIPE>
__global__ __launch_bounds__(kThreads, 2) void k_scan_backward(const ScanArgs A, int n_cols, int64_t n_tiles) {
    using Rows = WaveRows<T, PAIR, !PIPE>;
    __shared__ float2 s_a[kWaves][32], s_u[kWaves][32], s_ra[kWaves][32], s_ru[kWaves][32], s_h[32];
    __shared__ float2 s_s1[kWaves][32], s_s2[kWaves][32];
    __shared__ uint32_t s_ticket;
    __shared__ __attribute__((aligned(16))) char s_stage[PIPE ? kWaves * stage_bytes(CKPT) : 16];
    const int lane0 = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t Cp = (int64_t)n_cols * kTileCols;
    const uint32_t total = (uint32_t)(n_tiles * n_cols);
    char* const stage = s_stage + (PIPE ? wave * stage_bytes(CKPT) : 0);
    const uint32_t stage_lds = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)stage);

    auto tile_of = [&](uint32_t ticket) -> int64_t {
        return ticket < total ? n_tiles - 1 - ticket / (uint32_t)n_cols : 0;
    };
    // The row map of the wave's 32 rows, a lane each; in lanes 32 to 34 that of
    // the tile's last row, of the row before the tile, of its first row.
    auto map_of = [&](int64_t tile) {
        const int lane = fresh_lane(lane0);
        const int32_t* map = A.map + tile * kTileRows;
        int at = wave * 2 * FR + lane;
        if (lane == 32) at = kTileRows - 1;
        if (lane == 33) at = -1;
        if (lane == 34) at = 0;
        return lane < 35 && (at >= 0 || tile > 0) ? map[at] : -1;
    };
    auto whole_of = [&](int32_t m) { return (uint32_t)__ballot(m >= 0) == 0xffffffffu; };
    // A tile's head and rows on their way into the stage; m: its row map.
    auto fetch = [&](uint32_t ticket, int64_t tile, int32_t m) {
        if constexpr (PIPE) {
            const int lane = fresh_lane(lane0), half = lane >> 5, hl = lane & 31;
            const int64_t cb = (int64_t)(ticket % (uint32_t)n_cols) * kTileCols;
            const int64_t r0 = tile * kTileRows + wave * 2 * FR;
            stage_free();
            const uint32_t c1 = (cb + lane < A.C ? lane : 0) * 4;  // lanes beyond the last channel: the column's first
            stage4(scalar_ptr(A.dt_bias + cb), c1, stage_lds);
            stage4(scalar_ptr(A.a_log + cb), c1, stage_lds + 256);
            stage4(scalar_ptr(A.states + tile * A.C + cb), c1, stage_lds + 512);  // not used where nothing was kept
            if (!whole_of(m)) return;  // such a wave loads its rows itself
            const uint32_t c8 = cb + (lane & 7) * 8 < A.C ? (lane & 7) * 8 : 0;
            const uint32_t stage_rows = stage_lds + kStageHead;
            auto rows = [&](const void* base, int64_t stride, int slot) {
                const T* p = scalar_ptr(static_cast<const T*>(base) + r0 * stride + cb);
                const uint32_t row = fresh_scalar((uint32_t)stride * (uint32_t)sizeof(T));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    stage16(p, ((lane >> 3 & 1) * FR + 4 * q + (lane >> 4)) * row + c8 * (uint32_t)sizeof(T),
                            stage_rows + slot + q * 1024);
            };
            if constexpr (CKPT) {
                const int64_t n4 = Cp / 4;
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const int64_t at = ((r0 / FR) * 3 + t) * n4 + cb / 4;  // of the first half; the second 3 n4 blocks on
                    const char* p = scalar_ptr(reinterpret_cast<const char*>(A.q) + at * 64);
                    const float* s = scalar_ptr(A.q_scale + at);
                    const uint32_t block = (uint32_t)half * 3u * (uint32_t)n4 + (hl >> 1);
                    const uint32_t slot = stage_rows + kStageRows + t * kStageCkpt;
                    stage16(p, block * 64 + (hl & 1) * 32, slot);
                    stage16(p, block * 64 + (hl & 1) * 32 + 16, slot + 1024);
                    stage4(s, block * 4, slot + 2048);
                }
            } else {
                rows(A.a, A.ab_stride, 1 * kStageRows);
                rows(A.b, A.ab_stride, 2 * kStageRows);
                rows(A.x, A.x_stride, 3 * kStageRows);
            }
            rows(A.dh, A.dh_stride, 0);
        }
    };

    // Tickets are drawn two ahead: by the time a tile's rows are asked for,
    // its place and row map have long arrived.
    if (threadIdx.x == 0) s_ticket = atomicAdd(A.ticket, 1u);
    __syncthreads();
    const uint32_t ticket0 = __builtin_amdgcn_readfirstlane(s_ticket);
    __syncthreads();
    uint32_t ticket = ticket0, ticket1 = total;
    if constexpr (PIPE) {
        if (threadIdx.x == 0) s_ticket = atomicAdd(A.ticket, 1u);
        __syncthreads();
        ticket1 = __builtin_amdgcn_readfirstlane(s_ticket);
        __syncthreads();
    }
    if (ticket >= total) return;
    int64_t tile = tile_of(ticket), tile1 = tile_of(ticket1);
    int32_t m_next = map_of(tile);
    fetch(ticket, tile, m_next);
    while (ticket < total) {
        const int lane = fresh_lane(lane0), half = lane >> 5, hl = lane & 31;
        const int col = (int)(ticket % (uint32_t)n_cols);
        const int64_t r0 = tile * kTileRows + wave * 2 * FR, cb = (int64_t)col * kTileCols, c0 = cb + hl * 2;
        const int64_t left = (int64_t)A.C - c0;
        const int nc = left >= 2 ? 2 : left > 0 ? (int)left : 0;
        const int32_t m32 = m_next;
        if constexpr (PIPE) stage_wait();
        // on their way through the first walk: the next row map and a ticket
        uint32_t drawn = total;
        const int32_t m_last = __builtin_amdgcn_readlane(m32, 32), m_prev = __builtin_amdgcn_readlane(m32, 33),
                      m_first = __builtin_amdgcn_readlane(m32, 34);
        const bool behind = m_last >= 0 && !(m_last & 2), ahead = m_prev >= 0 && !(m_prev & 2);
        const bool cont = m_first >= 0 && !(m_first & 1);
        if constexpr (PIPE) {
            m_next = map_of(tile1);
            if (threadIdx.x == 0) drawn = atomicAdd(A.ticket, 1u);
        }

        // the wave's 32 rows as bits, and this half's 16
        const uint32_t in = (uint32_t)__ballot(m32 >= 0), firsts = (uint32_t)__ballot(m32 >= 0 && (m32 & 1)),
                       lasts = (uint32_t)__ballot(m32 >= 0 && (m32 & 2));
        const uint32_t my_in = in >> (half * FR), my_firsts = firsts >> (half * FR), my_lasts = lasts >> (half * FR);
        const uint32_t any_first = firsts | firsts >> FR, any_last = lasts | lasts >> FR;
        auto seq_of = [&](int r) { return __shfl(m32, half * FR + r) >> 2; };  // all lanes together

        auto rows = [&](const void* base, int64_t stride) {
            return Rows(base, stride, A.n_rows, r0, A.C, cb, half * FR * stride + hl * 2);
        };
        const bool whole = in == 0xffffffffu;
        const Rows D = rows(A.dh, A.dh_stride);
        Raw2<T> rd[FR], rx[FR], ra[FR], rb[FR];
        Ckpt2 qx, qa, qb;
        if (PIPE && whole) {
            const char* stage_rows = stage + kStageHead;
            auto get = [&](int slot, Raw2<T> (&v)[FR]) {
#pragma unroll
                for (int r = 0; r < FR; ++r)
                    v[r].v = *reinterpret_cast<const decltype(v[r].v)*>(stage_rows + slot + r * 256 + lane * 4);
            };
            if constexpr (CKPT) {
                auto getq = [&](int t, Ckpt2& q) {
                    const char* p = stage_rows + kStageRows + t * kStageCkpt;
                    const uint4 lo = *reinterpret_cast<const uint4*>(p + lane * 16);
                    const uint4 hi = *reinterpret_cast<const uint4*>(p + 1024 + lane * 16);
                    q.sc = *reinterpret_cast<const float*>(p + 2048 + lane * 4);
                    q.set(lo, hi, lane);
                };
                getq(1, qa);
                getq(2, qb);
                getq(0, qx);
            } else {
                get(1 * kStageRows, ra);
                get(2 * kStageRows, rb);
                get(3 * kStageRows, rx);
            }
            get(0, rd);
        } else {
            if constexpr (CKPT) {
                const int64_t n4 = Cp / 4, blk = r0 / FR + half, c4 = cb / 4 + (hl >> 1);
                auto getq = [&](int t, Ckpt2& q) {
                    const int64_t at = (blk * 3 + t) * n4 + c4;
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    q.sc = 0.0f;
                    if (r0 + half * FR < A.n_rows) {
                        const uint4* p = reinterpret_cast<const uint4*>(A.q + at * 64 + (hl & 1) * 32);
                        lo = p[0];
                        hi = p[1];
                        q.sc = A.q_scale[at];
                    }
                    q.set(lo, hi, lane);
                };
                getq(1, qa);
                getq(2, qb);
                getq(0, qx);
            }
            const Rows X = rows(A.x, A.x_stride), Ag = rows(A.a, A.ab_stride), Bg = rows(A.b, A.ab_stride);
            auto row = [&](int r) {
                if constexpr (!CKPT) {
                    ra[r] = Ag.load(r);
                    rb[r] = Bg.load(r);
                    rx[r] = X.load(r);
                }
                rd[r] = D.load(r);
            };
            if (whole && nc > 0) {  // no branch between the rows: all loads go out at once
#pragma unroll
                for (int r = 0; r < FR; ++r) row(r);
            } else {
#pragma unroll
                for (int r = 0; r < FR; ++r) {
                    rd[r] = zero2<T>();
                    if constexpr (!CKPT) { rx[r] = zero2<T>(); ra[r] = zero2<T>(); rb[r] = zero2<T>(); }
                    if ((my_in >> r & 1u) && nc > 0) row(r);
                }
            }
            if (!PIPE && (A.C & 1) && col == n_cols - 1) {
                D.last_alone(rd, my_in, nc);
                if constexpr (!CKPT) {
                    Ag.last_alone(ra, my_in, nc);
                    Bg.last_alone(rb, my_in, nc);
                    X.last_alone(rx, my_in, nc);
                }
            }
        }
        float dtb[2], kk[2], h[2];  // h: the kept state
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float dt, al;
            if constexpr (PIPE) {
                const float* head = reinterpret_cast<const float*>(stage) + hl * 2 + i;
                dt = head[0];
                al = head[64];
                h[i] = head[128];
            } else {
                dt = i < nc ? A.dt_bias[c0 + i] : 0.0f;
                al = i < nc ? A.a_log[c0 + i] : 0.0f;
                h[i] = 0.0f;
            }
            dtb[i] = i < nc ? dt : 0.0f;
            kk[i] = i < nc ? -expf(al) * kLog2e : 0.0f;
            h[i] = cont && i < nc ? h[i] : 0.0f;
        }
        // x, or half of it beside twice beta: the product is beta x either way
        auto get_x = [&](int r, int i) { return CKPT ? qx.half(r, i) : rx[r].get(i); };

        // the state a sequence starts from (seq -1: none)
        auto initial = [&](int seq, float (&h0)[2]) {
            const auto* R = rare_args();
            const bool init = seq >= 0 && (R->has_init ? R->has_init[seq] != 0 : true);
            const int64_t at = init ? (int64_t)R->page_idx[seq] * R->st_in_stride + c0 : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) h0[i] = init && i < nc ? load_state(R->st_in, at + i, R->state_dtype) : 0.0f;
        };

        auto final_gradient = [&](int seq, int i) {
            const auto* R = rare_args();
            return R->d_state && i < nc ? R->d_state[(int64_t)seq * R->C + c0 + i] : 0.0f;
        };

        // first walk: y = g log2(e), sigmoid(z), beta (twice it from the checkpoint), and the rows' run.  Rows of
        // no sequence run along on zeros (see the forward pass).
        float y[FR][2], sg[FR][2], be[FR][2];
        // The run from the last row to the first, mu -> fa mu + fu, is gathered on the
        // same walk: row r adds its dh through the decays of the rows up to it.
        float ea[2] = {1.0f, 1.0f}, eu[2] = {}, fa[2] = {1.0f, 1.0f}, fu[2] = {};
        bool ended = false;  // a last row is passed: mu from behind does not reach up
        const SoftplusC spc = softplus_consts();
#pragma unroll
        for (int r = 0; r < FR; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t;
                const float z = CKPT ? fmaf(2.0f, qa.half(r, i), dtb[i]) : ra[r].get(i) + dtb[i];
                y[r][i] = kk[i] * softplus_t(spc, z, t);
                const float s = rcp(1.0f + t);
                sg[r][i] = z >= 0.0f ? s : t * s;
                if constexpr (CKPT) be[r][i] = rcp(fmaf(0.5f, exp2_hw(qb.half(r, i) * (-2.0f * kLog2e)), 0.5f));
                else be[r][i] = sigmoid_hw(rb[r].get(i));
                const float al = exp2_hw(y[r][i]), u = be[r][i] * get_x(r, i);
                eu[i] = fmaf(al, eu[i], u);
                ea[i] *= al;
                fa[i] *= al;
                const float f = fmaf(fa[i], rd[r].get(i), fu[i]);
                fu[i] = lasts && ended ? fu[i] : f;
            }
            if (any_last >> r & 1u) {
                const int seq = seq_of(r);
                if ((my_lasts >> r & 1u) && !ended) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) fu[i] = fmaf(fa[i], final_gradient(seq, i), fu[i]);
                    ended = true;
                }
            }
            if (any_first >> r & 1u) {
                float h0[2];
                initial(seq_of(r), h0);
                if (my_firsts >> r & 1u) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) eu[i] = fmaf(exp2_hw(y[r][i]), h0[i], be[r][i] * get_x(r, i));
                }
            }
        }
        float xa[2], xu[2], ya[2], yu[2];  // the run of the wave's other half
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ea[i] = marked(ea[i], (my_firsts & 0xffffu) != 0);
            fa[i] = marked(fa[i], ended);
            xa[i] = __shfl_xor(ea[i], 32);
            xu[i] = __shfl_xor(eu[i], 32);
            ya[i] = __shfl_xor(fa[i], 32);
            yu[i] = __shfl_xor(fu[i], 32);
            if (half) join(xa[i], xu[i], ea[i], eu[i]);
            else join(ya[i], yu[i], fa[i], fu[i]);
        }
        if (half) {
            s_a[wave][hl] = make_float2(ea[0], ea[1]);
            s_u[wave][hl] = make_float2(eu[0], eu[1]);
        } else {
            s_ra[wave][hl] = make_float2(fa[0], fa[1]);
            s_ru[wave][hl] = make_float2(fu[0], fu[1]);
        }
        if (PIPE && threadIdx.x == 0) s_ticket = drawn;
        __syncthreads();
        if constexpr (!PIPE) {
#pragma unroll
            for (int i = 0; i < 2; ++i) h[i] = cont && i < nc ? rare_args()->states[tile * A.C + c0 + i] : 0.0f;
        }
        const uint32_t ticket2 = PIPE ? __builtin_amdgcn_readfirstlane(s_ticket) : total;
        if (wave == 0) {  // one channel a lane
            const auto* R = rare_args();
            const Chain chain{R->chain, n_tiles * Cp};
            float ta[1], tu[1], m1[1];
            const float* pa = reinterpret_cast<const float*>(s_ra) + lane;
            const float* pu = reinterpret_cast<const float*>(s_ru) + lane;
            ta[0] = pa[(kWaves - 1) * kTileCols];
            tu[0] = pu[(kWaves - 1) * kTileCols];
#pragma unroll
            for (int v = kWaves - 2; v >= 0; --v) {
                float ja = pa[v * kTileCols], ju = pu[v * kTileCols];
                join(ta[0], tu[0], ja, ju);
                ta[0] = ja; tu[0] = ju;
            }
            tell_run<1>(chain, tile * Cp + cb, behind, ahead, ta, tu);
            hand_on<1>(chain, tile * Cp + cb, Cp, n_tiles - 1 - tile, behind, ahead, ta, tu, m1, R->err);
            reinterpret_cast<float*>(s_h)[lane] = m1[0];
        } else if (ticket1 < total) {
            fetch(ticket1, tile1, m_next);
        }
        __syncthreads();
        if (wave == 0 && ticket1 < total) fetch(ticket1, tile1, m_next);  // not before the state is handed on
        float mu[2] = {s_h[hl].x, s_h[hl].y};
        for (int v = kWaves - 1; v > wave; --v) {
            const float2 va = s_ra[v][hl], vu = s_ru[v][hl];
            mu[0] = walk(va.x, vu.x, mu[0]);
            mu[1] = walk(va.y, vu.y, mu[1]);
        }
        if (!half) {
            mu[0] = walk(ya[0], yu[0], mu[0]);
            mu[1] = walk(ya[1], yu[1], mu[1]);
        }
        for (int v = 0; v < wave; ++v) {
            const float2 va = s_a[v][hl], vu = s_u[v][hl];
            h[0] = walk(va.x, vu.x, h[0]);
            h[1] = walk(va.y, vu.y, h[1]);
        }
        if (half) {
            h[0] = walk(xa[0], xu[0], h[0]);
            h[1] = walk(xa[1], xu[1], h[1]);
        }
        // second walk: the state before each row
#pragma unroll
        for (int r = 0; r < FR; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) { again(y[r][i]); again(be[r][i]); }
            again(rd[r].v);
            if constexpr (!CKPT) again(rx[r].v);
            else again(qx.w[r & 7]);
        }
        float hp[FR][2];
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            if (any_first >> r & 1u) {
                float h0[2];
                initial(seq_of(r), h0);
                if (my_firsts >> r & 1u) { h[0] = h0[0]; h[1] = h0[1]; }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                hp[r][i] = h[i];
                h[i] = fmaf(exp2_hw(y[r][i]), h[i], be[r][i] * get_x(r, i));
            }
        }
#pragma unroll
        for (int r = 0; r < FR; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) { again(y[r][i]); again(be[r][i]); }
            if constexpr (!CKPT) again(rx[r].v);
            else again(qx.w[r & 7]);
        }
        // third walk: the gradients, from the last row to the first
        const Rows DX = rows(A.dx, A.dx_stride), DA = rows(A.da, A.dab_stride), DB = rows(A.db, A.dab_stride);
        const float kg[2] = {kk[0] / kLog2e, kk[1] / kLog2e};
        float s1[2] = {}, s2[2] = {};  // sums of dg y and of dg sigmoid(z)
#pragma unroll
        for (int r = FR - 1; r >= 0; --r) {
            float lam[2], dx[2], da[2], db[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) lam[i] = rd[r].get(i) + mu[i];
            if (any_last >> r & 1u) {
                const int seq = seq_of(r);
                if (my_lasts >> r & 1u) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        lam[i] = rd[r].get(i) + final_gradient(seq, i);
                    }
                }
            }
            const bool mine = whole || (my_in >> r & 1u);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mu[i] = exp2_hw(y[r][i]) * lam[i];
                const float dg = mine ? mu[i] * hp[r][i] : 0.0f;
                const float ds = dg * sg[r][i];
                const float beta = CKPT ? 0.5f * be[r][i] : be[r][i];
                dx[i] = beta * lam[i];
                // in this order nothing overflows on the way: beta lambda (1 - beta) is smaller than lambda
                db[i] = dx[i] * ((CKPT ? 2.0f : 1.0f) - be[r][i]) * get_x(r, i);
                da[i] = ds * kg[i];
                s1[i] = fmaf(dg, y[r][i], s1[i]);
                s2[i] += ds;
            }
            if (mine && nc > 0) {
                DX.store(r, nc, dx[0], dx[1]);
                DA.store(r, nc, da[0], da[1]);
                DB.store(r, nc, db[0], db[1]);
            }
            if (any_first >> r & 1u) {
                const auto* R = rare_args();
                const int seq = seq_of(r);
                if ((my_firsts >> r & 1u) && R->d_state0) {
                    const bool init = R->has_init ? R->has_init[seq] != 0 : true;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i < nc) R->d_state0[(int64_t)seq * R->C + c0 + i] = init ? mu[i] : 0.0f;
                }
            }
        }
        // sums over the tile's rows: halves, then waves; g = y ln 2
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s1[i] *= 0.6931471805599453f;
            s2[i] *= kg[i];
            s1[i] += __shfl_xor(s1[i], 32);
            s2[i] += __shfl_xor(s2[i], 32);
        }
        if (!half) {
            s_s1[wave][hl] = make_float2(s1[0], s1[1]);
            s_s2[wave][hl] = make_float2(s2[0], s2[1]);
        }
        __syncthreads();
        if (wave < 2) {
            const float* p = reinterpret_cast<const float*>(wave ? s_s2 : s_s1) + lane;
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) v += p[q * kTileCols];
            rare_args()->part[(tile * 2 + wave) * Cp + cb + lane] = v;
        }
        ticket = ticket1;
        tile = tile1;
        ticket1 = ticket2;
        tile1 = tile_of(ticket2);
    }
}

// ------------------------------------------------------------------- launches

// With the stage, one workgroup for each of MI355X's 256 compute units: they draw tiles.
constexpr int64_t kGroups = 256;

template <typename T, bool PAIR, bool CKPT> static hipError_t backward_t(const ScanArgs& a, hipStream_t s) {
    const int nc = (int)(padded_channels(a.C) / kTileCols);
    const int64_t nt = n_tiles(a.n_rows), grid = nt * nc;
    if (grid > 0) {
        if (sizeof(T) == 2 && PAIR && a.vec8)
            hipLaunchKernelGGL((k_scan_backward<T, PAIR, CKPT, sizeof(T) == 2 && PAIR>),
                               dim3((unsigned)(grid < kGroups ? grid : kGroups)), dim3(kThreads), 0, s, a, nc, nt);
        else
            hipLaunchKernelGGL((k_scan_backward<T, PAIR, CKPT, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, a,
                               nc, nt);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_sum_tiles(a.part, nt, a.C, 2, a.d_a_log, a.d_dt_bias, s);
}

template <typename T> static hipError_t backward_d(const ScanArgs& a, hipStream_t s) {
    if (a.q) return a.C > 1 ? backward_t<T, true, true>(a, s) : backward_t<T, false, true>(a, s);
    return a.C > 1 ? backward_t<T, true, false>(a, s) : backward_t<T, false, false>(a, s);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    MapArgs m = scan_map_args(a);
    m.pass_src = a.d_state; m.pass_dst = a.d_state0; m.pass_width = a.C;
    const hipError_t e = launch_map(m, s);
    if (e != hipSuccess) return e;
    return a.act_dtype == GDN_BF16 ? backward_d<bf16_t>(a, s) : backward_d<float>(a, s);
}

}  // namespace gdnt
