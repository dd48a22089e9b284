// gdnt_scan.hip -- the vector-state gated linear recurrence
//   h_t = e^{g_t} h_{t-1} + beta_t x_t  per channel, forward.
//
// A tile is 128 packed rows by 128 channels, one workgroup of eight waves: a
// wave holds 16 consecutive rows, a lane two channels of each, so everything
// about a row (its sequence, its address) is uniform over the wave and costs
// no vector instruction, and a row's piece is 256 consecutive bytes in bf16
// (a copy in such pieces runs at 5.4 TB/s here, in 128-byte pieces at 4.7).
// A wave turns its rows into a run (h -> a h + u) per channel, the runs of a
// tile are joined through LDS, the state comes from the tile before
// (gdnt_chain.hpp), and each wave walks its rows again from registers: x, a
// and b are read once.  Sequence boundaries may fall anywhere.
//
// Bound by memory: 32768 x 4096 in bf16 takes 250 us for 1.07 GB (4.3 TB/s,
// 85% of what a large copy reaches), at 33 vector instructions an element
// (52% of the issue slots) and with two workgroups on a compute unit, one
// loading while the other walks; 301 us and 1.50 GB (5.0 TB/s) with the 8-bit
// checkpoint, 64% of the slots.  fp32 fits in the same 128 registers
// (two spilled with the checkpoint): 16692 x 4096 take 216 us, 266 with one
// workgroup on a compute unit.  30011 x 1001 in fp32 takes 130 us (3.7 TB/s): its 8
// columns leave the chain of 235 tiles in sight.
#include "gdnt_chain.hpp"
#include "gdnt_rows.hpp"

namespace gdnt {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
static_assert(kThreads == kScanThreads, "launch size");
constexpr int kFwdRows = FR * kWaves;        // 128
constexpr int kFwdCols = 128;
static_assert(kTileRows % kFwdRows == 0, "tile shape");

// The wave's 16 rows of one tensor by this lane's two channels in 8 bits.
template <typename T>
__device__ __forceinline__ void put_ckpt(const Raw2<T> (&v)[FR], int8_t* q, float* scale, int lane, bool mine) {
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < FR; ++r) top = v[r].top(top);
    top = Raw2<T>::top_bits(top);
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false);
    top = top > other ? top : other;
    const float m = __uint_as_float(top);
    const bool finite = top < 0x7f800000u, live = m >= 7.888609052210118e-31f && finite;  // 2^-100
    const float up = live ? 127.0f / m : 0.0f;
    const float sc = !finite ? __uint_as_float(0x7fc00000u) : live ? m / 127.0f : 0.0f;
    uint32_t w[FR / 2];
#pragma unroll
    for (int r = 0; r < FR / 2; ++r) {
        // v * up + 1.5 * 2^23 rounds once to an integer, which then is the low byte
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            e[k] = __float_as_uint(fmaf(v[r + (k >> 1) * (FR / 2)].get(k & 1), up, 12582912.0f));
        // row r in the low half, row r + 8 in the high half
        const uint32_t lo = __builtin_amdgcn_perm(e[1], e[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(e[3], e[2], 0x04000c0cu);
        w[r] = swap_halves(lo | hi, lane);
    }
    if (mine) {
        uint4* out = reinterpret_cast<uint4*>(q + (lane >> 1) * 64 + (lane & 1) * 32);
        out[0] = make_uint4(w[0], w[1], w[2], w[3]);
        out[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (!(lane & 1)) scale[lane >> 1] = sc;
    }
}

template <typename T, bool PAIR, bool CKPT>
__global__ __launch_bounds__(kThreads, 4) void k_scan_forward(const ScanArgs A, int n_cols,
                                                                                    int64_t n_tiles) {
    __shared__ float2 s_a[kWaves][64], s_u[kWaves][64], s_h[64];
    __shared__ uint32_t s_ticket;
    if (threadIdx.x == 0) s_ticket = atomicAdd(A.ticket, 1u);
    __syncthreads();
    const uint32_t ticket = __builtin_amdgcn_readfirstlane(s_ticket);
    const int64_t tile = ticket / (uint32_t)n_cols;
    const int col = (int)(ticket % (uint32_t)n_cols);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t r0 = tile * kFwdRows + wave * FR, c0 = (int64_t)col * kFwdCols + lane * 2;
    const int64_t left = (int64_t)A.C - c0;
    const int nc = left >= 2 ? 2 : left > 0 ? (int)left : 0;
    // rows of a sequence, and its first and last ones among them, as bits
    const int32_t m16 = lane < FR ? A.map[r0 + lane] : -1;
    const uint32_t in = (uint32_t)__ballot(m16 >= 0), firsts = (uint32_t)__ballot(m16 >= 0 && (m16 & 1)),
                   lasts = (uint32_t)__ballot(m16 >= 0 && (m16 & 2));
    auto seq_of = [&](int r) { return __builtin_amdgcn_readlane(m16, r) >> 2; };

    const int64_t cb = (int64_t)col * kFwdCols;
    const WaveRows<T, PAIR> X(A.x, A.x_stride, A.n_rows, r0, A.C, cb, lane * 2),
        Ag(A.a, A.ab_stride, A.n_rows, r0, A.C, cb, lane * 2), Bg(A.b, A.ab_stride, A.n_rows, r0, A.C, cb, lane * 2),
        H(A.h, A.h_stride, A.n_rows, r0, A.C, cb, lane * 2);
    Raw2<T> rx[FR], ra[FR], rb[FR];
    if (in == 0xffffu && nc > 0) {
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            ra[r] = Ag.load(r);
            rx[r] = X.load(r);
            rb[r] = Bg.load(r);
        }
    } else {
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            rx[r] = zero2<T>(); ra[r] = zero2<T>(); rb[r] = zero2<T>();
            if ((in >> r & 1u) && nc > 0) {
                ra[r] = Ag.load(r);
                rx[r] = X.load(r);
                rb[r] = Bg.load(r);
            }
        }
    }
    if ((A.C & 1) && col == n_cols - 1) {
        X.last_alone(rx, in, nc);
        Ag.last_alone(ra, in, nc);
        Bg.last_alone(rb, in, nc);
    }
    float dt[2], kk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        dt[i] = i < nc ? A.dt_bias[c0 + i] : 0.0f;
        kk[i] = i < nc ? -expf(A.a_log[c0 + i]) * kLog2e : 0.0f;
    }
    if constexpr (CKPT) {
        const int64_t n4 = padded_channels(A.C) / 4, c4 = (int64_t)col * (kFwdCols / 4);
        if (r0 < A.n_rows) {
            const bool mine = c4 + (lane >> 1) < n4;
            const int64_t at = (r0 / FR) * 3 * n4 + c4;
            put_ckpt<T>(rx, A.q + at * 64, A.q_scale + at, lane, mine);
            put_ckpt<T>(ra, A.q + (at + n4) * 64, A.q_scale + at + n4, lane, mine);
            put_ckpt<T>(rb, A.q + (at + 2 * n4) * 64, A.q_scale + at + 2 * n4, lane, mine);
        }
    }

    float al[FR][2], u[FR][2];
    float ea[2] = {1.0f, 1.0f}, eu[2] = {0.0f, 0.0f};
    // Rows of no sequence run along on zeros: what they make of the state goes
    // nowhere, a first row follows them.
    const SoftplusC spc = softplus_consts();
#pragma unroll
    for (int r = 0; r < FR; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t;
            al[r][i] = exp2_hw(kk[i] * softplus_t(spc, ra[r].get(i) + dt[i], t));
            u[r][i] = sigmoid_hw(rb[r].get(i)) * rx[r].get(i);
            eu[i] = fmaf(al[r][i], eu[i], u[r][i]);
            ea[i] *= al[r][i];
        }
        if (firsts >> r & 1u) {  // the state page joins a first row, nothing before it does
            const int seq = seq_of(r);
            const bool init = A.has_init ? A.has_init[seq] != 0 : true;
            const int64_t at = (int64_t)A.page_idx[seq] * A.st_in_stride + c0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (init && i < nc) u[r][i] = fmaf(al[r][i], load_state(A.st_in, at + i, A.state_dtype), u[r][i]);
                eu[i] = u[r][i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) ea[i] = marked(ea[i], firsts != 0);
    s_a[wave][lane] = make_float2(ea[0], ea[1]);
    s_u[wave][lane] = make_float2(eu[0], eu[1]);
    __syncthreads();
    if (wave == 0) {
        float ta[2] = {ea[0], ea[1]}, tu[2] = {eu[0], eu[1]};
#pragma unroll
        for (int v = 1; v < kWaves; ++v) {
            float2 qa = s_a[v][lane], qu = s_u[v][lane];
            join(ta[0], tu[0], qa.x, qu.x);
            join(ta[1], tu[1], qa.y, qu.y);
            ta[0] = qa.x; ta[1] = qa.y; tu[0] = qu.x; tu[1] = qu.y;
        }
        const int32_t m_next = tile + 1 < n_tiles ? A.map[(tile + 1) * kFwdRows] : -1;
        const bool cont = (in & ~firsts) & 1u;
        const int64_t Cw = (int64_t)n_cols * kFwdCols;
        const Chain chain{A.chain, n_tiles * Cw};
        const int64_t at = tile * Cw + (int64_t)col * kFwdCols;
        const bool next = m_next >= 0 && !(m_next & 1);
        float h[2];
        tell_run<2>(chain, at, cont, next, ta, tu);
        hand_on<2>(chain, at, -Cw, tile, cont, next, ta, tu, h, A.err);
        s_h[lane] = make_float2(h[0], h[1]);
        if (A.states && cont && r0 % kTileRows == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i < nc) A.states[r0 / kTileRows * A.C + c0 + i] = h[i];
        }
    }
    __syncthreads();
    float h[2] = {s_h[lane].x, s_h[lane].y};
    for (int v = 0; v < wave; ++v) {
        const float2 va = s_a[v][lane], vu = s_u[v][lane];
        h[0] = walk(va.x, vu.x, h[0]);
        h[1] = walk(va.y, vu.y, h[1]);
    }
#pragma unroll
    for (int r = 0; r < FR; ++r) {
        h[0] = fmaf(al[r][0], h[0], u[r][0]);
        h[1] = fmaf(al[r][1], h[1], u[r][1]);
        if (firsts >> r & 1u) { h[0] = u[r][0]; h[1] = u[r][1]; }
        if (in >> r & 1u) H.store(r, nc, h[0], h[1]);
        if (lasts >> r & 1u) {
            const int64_t at = (int64_t)A.page_idx[seq_of(r)] * A.st_out_stride + c0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i < nc) store_state(A.st_out, at + i, A.state_dtype, h[i]);
        }
    }
}

// A few rows a sequence (decode and short verify-like steps): one thread
// walks four channels of one sequence, one launch, no row map.  64 sequences
// of one row by 4096 channels take 4.2 us, a launch's own time: 4 MB are 0.8
// us of memory.
template <typename T, bool VEC>
__global__ __launch_bounds__(kRowsThreads) void k_scan_rows(const ScanArgs A, int n_x) {
    const int seq = (int)(blockIdx.x / n_x);
    const int64_t c0 = ((int64_t)(blockIdx.x % n_x) * kRowsThreads + threadIdx.x) * 4;
    const bool tell = blockIdx.x % n_x == 0 && threadIdx.x == 0;
    const int page = A.page_idx[seq], r0 = A.cu[seq], r1 = A.cu[seq + 1];
    // all bounds up to this sequence's, as the row map does
    bool bad = false;
    for (int s = threadIdx.x; s <= seq; s += kRowsThreads) bad |= !bounds_ok(A.n_rows, A.cu[s], A.cu[s + 1]);
    bad = __syncthreads_or(bad) != 0;
    if (page < 0) return;
    if (page >= A.page_limit) {
        if (tell) raise(A.err, GDN_DEVERR_PAGE);
        return;
    }
    if ((bad && !valid_slow(A.cu, A.n_rows, seq)) || r1 - r0 > A.max_len) {
        if (tell) raise(A.err, GDN_DEVERR_BATCH);
        return;
    }
    if (r0 == r1 || c0 >= A.C) return;
    const int nc = A.C - c0 >= 4 ? 4 : (int)(A.C - c0);
    const bool init = A.has_init ? A.has_init[seq] != 0 : true;
    float h[4] = {};
    const int64_t at_in = (int64_t)page * A.st_in_stride + c0, at_out = (int64_t)page * A.st_out_stride + c0;
    if (init) {
        if (A.state_dtype == GDN_BF16) {
            const Raw4<bf16_t> v = load4<bf16_t, VEC>(static_cast<const bf16_t*>(A.st_in) + at_in, nc);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = v.get(i);
        } else {
            const Raw4<float> v = load4<float, VEC>(static_cast<const float*>(A.st_in) + at_in, nc);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = v.get(i);
        }
    }
    const SoftplusC spc = softplus_consts();
    const ChanP P = load_params(A.a_log, A.dt_bias, c0, nc);
    for (int64_t r = r0; r < r1; ++r) {
        const Raw4<T> x = load4<T, VEC>(static_cast<const T*>(A.x) + r * A.x_stride + c0, nc);
        const Raw4<T> a = load4<T, VEC>(static_cast<const T*>(A.a) + r * A.ab_stride + c0, nc);
        const Raw4<T> b = load4<T, VEC>(static_cast<const T*>(A.b) + r * A.ab_stride + c0, nc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t;
            const float sp = softplus_t(spc, a.get(i) + P.dt[i], t);
            h[i] = fmaf(exp2_hw(P.k[i] * sp), h[i], sigmoid_hw(b.get(i)) * x.get(i));
        }
        store4<VEC>(static_cast<T*>(A.h) + r * A.h_stride + c0, h, nc);
    }
    if (A.state_dtype == GDN_BF16) store4<VEC>(static_cast<bf16_t*>(A.st_out) + at_out, h, nc);
    else store4<VEC>(static_cast<float*>(A.st_out) + at_out, h, nc);
}

// ------------------------------------------------------------------- launches

size_t scan_chain_bytes(int64_t n_rows, int32_t C) {
    // the forward tiles are the smaller ones: two words a channel and tile
    const int64_t cols = (C + kFwdCols - 1) / kFwdCols;
    return (size_t)((n_rows + kFwdRows - 1) / kFwdRows) * (size_t)(cols * kFwdCols) * 2 * sizeof(uint64_t);
}

MapArgs scan_map_args(const ScanArgs& a) {
    MapArgs m{};
    m.cu = a.cu; m.page_idx = a.page_idx; m.n_seqs = a.n_seqs;
    m.n_rows = a.n_rows; m.n_map = n_tiles(a.n_rows) * kTileRows;
    m.page_limit = a.page_limit; m.max_len = a.max_len; m.map = a.map; m.err = a.err;
    // the ticket (256 bytes) and the chain words behind it start from zero
    m.zero = a.ticket; m.n_zero = (int64_t)((256 + scan_chain_bytes(a.n_rows, a.C)) / sizeof(uint32_t));
    return m;
}

template <typename T, bool VEC> static hipError_t rows_t(const ScanArgs& a, hipStream_t s) {
    const int64_t n_x = scan_rows_groups(1, a.C), grid = scan_rows_groups(a.n_seqs, a.C);
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((k_scan_rows<T, VEC>), dim3((unsigned)grid), dim3(kRowsThreads), 0, s, a, (int)n_x);
    return hipGetLastError();
}

hipError_t launch_scan_rows(const ScanArgs& a, hipStream_t s) {
    if (a.act_dtype == GDN_BF16) return a.vec ? rows_t<bf16_t, true>(a, s) : rows_t<bf16_t, false>(a, s);
    return a.vec ? rows_t<float, true>(a, s) : rows_t<float, false>(a, s);
}

template <typename T, bool PAIR> static hipError_t forward_t(const ScanArgs& a, hipStream_t s) {
    const int nc = (int)((a.C + kFwdCols - 1) / kFwdCols);
    const int64_t nt = (a.n_rows + kFwdRows - 1) / kFwdRows, grid = nt * nc;
    if (grid == 0) return hipSuccess;
    if (a.q)
        hipLaunchKernelGGL((k_scan_forward<T, PAIR, true>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, nc, nt);
    else
        hipLaunchKernelGGL((k_scan_forward<T, PAIR, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, nc, nt);
    return hipGetLastError();
}

hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s) {
    const hipError_t e = launch_map(scan_map_args(a), s);
    if (e != hipSuccess) return e;
    if (a.act_dtype == GDN_BF16) return a.C > 1 ? forward_t<bf16_t, true>(a, s) : forward_t<bf16_t, false>(a, s);
    return a.C > 1 ? forward_t<float, true>(a, s) : forward_t<float, false>(a, s);
}

}  // namespace gdnt
