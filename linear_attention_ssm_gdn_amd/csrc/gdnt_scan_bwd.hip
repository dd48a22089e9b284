// gdnt_scan_bwd.hip -- the backward pass of the vector-state gated linear
// recurrence.
//
// A tile is 256 packed rows by 64 channels, one workgroup of 512 threads: 16
// lanes side by side hold four channels each, 32 row groups hold eight
// consecutive rows each.  A thread turns its rows into two runs, one in each
// direction; the runs of a tile are joined by lane shuffles and through LDS,
// and with the states before and behind its rows each thread walks them
// again from registers.
#include "gdnt_chain.hpp"

namespace gdnt {

constexpr int R = 8;                         // rows of a thread
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
static_assert(kThreads / 16 * R == kTileRows && 16 * 4 == kTileCols, "tile shape");

template <typename T> struct Rows {
    int32_t m[R];   // row map
    int nc;         // channels of this thread that exist, 0..4
    int64_t c0, r0;
};

template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const ScanArgs& A, int64_t tile, int col, int cl, int rg) {
    Rows<T> w;
    w.r0 = tile * kTileRows + rg * R;
    w.c0 = (int64_t)col * kTileCols + cl * 4;
    const int64_t left = (int64_t)A.C - w.c0;
    w.nc = left >= 4 ? 4 : left > 0 ? (int)left : 0;
    const int4* mp = reinterpret_cast<const int4*>(A.map + w.r0);
    const int4 m0 = mp[0], m1 = mp[1];
    w.m[0] = m0.x; w.m[1] = m0.y; w.m[2] = m0.z; w.m[3] = m0.w;
    w.m[4] = m1.x; w.m[5] = m1.y; w.m[6] = m1.z; w.m[7] = m1.w;
    return w;
}

// The backward pass.  With mu_t = alpha_t lambda_t the reverse recurrence is
// lambda_t = dh_t + mu_{t+1}, mu_t = alpha_t lambda_t: the same kind of run,
// from the last row to the first, and new at a last row.
// h_{t-1} comes from the kept state before the tile and the same runs as in
// the forward pass; only the reverse recurrence goes from tile to tile.
template <typename T, bool VEC, bool CKPT>
__global__ __launch_bounds__(kThreads) void k_scan_backward(const ScanArgs A, int n_cols, int64_t n_tiles) {
    __shared__ float4 s_a[kWaves][16], s_u[kWaves][16], s_ra[kWaves][16], s_ru[kWaves][16], s_h[16];
    __shared__ uint32_t s_ticket;
    if (threadIdx.x == 0) s_ticket = atomicAdd(A.ticket, 1u);
    __syncthreads();
    const int64_t tile = n_tiles - 1 - s_ticket / (uint32_t)n_cols;
    const int col = (int)(s_ticket % (uint32_t)n_cols);
    const int lane = threadIdx.x & 63, cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t Cp = (int64_t)n_cols * kTileCols;
    const Rows<T> w = rows_of<T>(A, tile, col, cl, rg);

    float x[R][4], a[R][4], b[R][4];
    Raw4<T> rd[R];
    const T* pd = static_cast<const T*>(A.dh) + w.r0 * A.dh_stride + w.c0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rd[r] = zero4<T>();
        if (w.m[r] >= 0 && w.nc > 0) rd[r] = load4<T, VEC>(pd + r * A.dh_stride, w.nc);
    }
    if constexpr (CKPT) {
        const int64_t n4 = Cp / 4, blk = w.r0 / GDNT_CKPT_ROWS, c4 = w.c0 / 4;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            const int64_t at = (blk * 3 + t) * n4 + c4;
            uint32_t q[R];
            if (w.r0 < A.n_rows) {
                const uint4* p = reinterpret_cast<const uint4*>(A.q + at * 64 + (rg & 1) * 32);
                const uint4 q0 = p[0], q1 = p[1];
                q[0] = q0.x; q[1] = q0.y; q[2] = q0.z; q[3] = q0.w;
                q[4] = q1.x; q[5] = q1.y; q[6] = q1.z; q[7] = q1.w;
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) q[r] = 0;
            }
            const float sc = w.r0 < A.n_rows ? A.q_scale[at] : 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    (t == 0 ? x : t == 1 ? a : b)[r][i] = (float)(int8_t)(q[r] >> (8 * i)) * sc;
        }
    } else {
        const T* px = static_cast<const T*>(A.x) + w.r0 * A.x_stride + w.c0;
        const T* pa = static_cast<const T*>(A.a) + w.r0 * A.ab_stride + w.c0;
        const T* pb = static_cast<const T*>(A.b) + w.r0 * A.ab_stride + w.c0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Raw4<T> rx = zero4<T>(), ra = zero4<T>(), rb = zero4<T>();
            if (w.m[r] >= 0 && w.nc > 0) {
                rx = load4<T, VEC>(px + r * A.x_stride, w.nc);
                ra = load4<T, VEC>(pa + r * A.ab_stride, w.nc);
                rb = load4<T, VEC>(pb + r * A.ab_stride, w.nc);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) { x[r][i] = rx.get(i); a[r][i] = ra.get(i); b[r][i] = rb.get(i); }
        }
    }
    const SoftplusC spc = softplus_consts();
    const ChanP P = load_params(A.a_log, A.dt_bias, w.c0, w.nc);

    // forward run (ea, eu) and reverse run (fa, fu) of the rows; h0[r] is kept in u
    float al[R][4], u[R][4];
    float ea[4] = {1.0f, 1.0f, 1.0f, 1.0f}, eu[4] = {}, fa[4] = {1.0f, 1.0f, 1.0f, 1.0f}, fu[4] = {};
    float h0[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = w.m[r] >= 0, first = in && (w.m[r] & 1);
        int64_t at = 0;
        bool init = false;
        if (first) {
            const int seq = w.m[r] >> 2;
            init = A.has_init ? A.has_init[seq] != 0 : true;
            at = (int64_t)A.page_idx[seq] * A.st_in_stride + w.c0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t;
            const float sp = softplus_t(spc, a[r][i] + P.dt[i], t);
            al[r][i] = in ? exp2_hw(P.k[i] * sp) : 1.0f;
            u[r][i] = in ? sigmoid_hw(b[r][i]) * x[r][i] : 0.0f;
            h0[r][i] = 0.0f;
            if (first) {
                if (init && i < w.nc) h0[r][i] = load_state(A.st_in, at + i, A.state_dtype);
                eu[i] = fmaf(al[r][i], h0[r][i], u[r][i]);
                ea[i] = -1.0f;
            } else {
                eu[i] = fmaf(al[r][i], eu[i], u[r][i]);
                ea[i] *= al[r][i];
            }
        }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        const bool in = w.m[r] >= 0, last = in && (w.m[r] & 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lam = rd[r].get(i);
            if (last) {
                if (A.d_state && i < w.nc) lam += A.d_state[(int64_t)(w.m[r] >> 2) * A.C + w.c0 + i];
                fa[i] = -1.0f;
            } else {
                lam += fu[i];
            }
            fu[i] = in ? al[r][i] * lam : fu[i];
            fa[i] = fa[i] * al[r][i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ea[i] = copysignf(fmaxf(fabsf(ea[i]), kTiny), ea[i]);
        fa[i] = copysignf(fmaxf(fabsf(fa[i]), kTiny), fa[i]);
    }
#pragma unroll
    for (int d = 16; d <= 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float qa = __shfl_up(ea[i], d), qu = __shfl_up(eu[i], d);
            const float sa = __shfl_down(fa[i], d), su = __shfl_down(fu[i], d);
            if (lane >= d) join(qa, qu, ea[i], eu[i]);
            if (lane + d < 64) join(sa, su, fa[i], fu[i]);
        }
    }
    if (lane >= 48) {
        s_a[wave][cl] = make_float4(ea[0], ea[1], ea[2], ea[3]);
        s_u[wave][cl] = make_float4(eu[0], eu[1], eu[2], eu[3]);
    }
    if (lane < 16) {
        s_ra[wave][cl] = make_float4(fa[0], fa[1], fa[2], fa[3]);
        s_ru[wave][cl] = make_float4(fu[0], fu[1], fu[2], fu[3]);
    }
    float xa[4], xu[4], ya[4], yu[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        xa[i] = __shfl_up(ea[i], 16);
        xu[i] = __shfl_up(eu[i], 16);
        ya[i] = __shfl_down(fa[i], 16);
        yu[i] = __shfl_down(fu[i], 16);
        if (lane < 16) { xa[i] = 1.0f; xu[i] = 0.0f; }
        if (lane >= 48) { ya[i] = 1.0f; yu[i] = 0.0f; }
    }
    __syncthreads();
    const int32_t m_first = A.map[tile * kTileRows];
    if (threadIdx.x < 64) {
        const int32_t m_last = A.map[tile * kTileRows + kTileRows - 1];
        const int32_t m_prev = tile > 0 ? A.map[tile * kTileRows - 1] : -1;
        const float* pa = reinterpret_cast<const float*>(s_ra) + threadIdx.x;
        const float* pu = reinterpret_cast<const float*>(s_ru) + threadIdx.x;
        float ta = pa[(kWaves - 1) * kTileCols], tu = pu[(kWaves - 1) * kTileCols];
#pragma unroll
        for (int v = kWaves - 2; v >= 0; --v) {
            float qa = pa[v * kTileCols], qu = pu[v * kTileCols];
            join(ta, tu, qa, qu);
            ta = qa; tu = qu;
        }
        const Chain chain{A.chain, A.chain + n_tiles * Cp};
        const float a1[1] = {ta}, u1[1] = {tu};
        float h1[1];
        hand_on<1>(chain, tile * Cp + (int64_t)col * kTileCols, Cp, n_tiles - 1 - tile, m_last >= 0 && !(m_last & 2),
                   m_prev >= 0 && !(m_prev & 2), a1, u1, h1, A.err);
        reinterpret_cast<float*>(s_h)[threadIdx.x] = h1[0];
    }
    __syncthreads();
    float h[4] = {}, mu[4] = {s_h[cl].x, s_h[cl].y, s_h[cl].z, s_h[cl].w};
    if (m_first >= 0 && !(m_first & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < w.nc) h[i] = A.states[tile * A.C + w.c0 + i];
    }
    for (int v = 0; v < wave; ++v) {
        const float4 va = s_a[v][cl], vu = s_u[v][cl];
        h[0] = walk(va.x, vu.x, h[0]); h[1] = walk(va.y, vu.y, h[1]);
        h[2] = walk(va.z, vu.z, h[2]); h[3] = walk(va.w, vu.w, h[3]);
    }
    for (int v = kWaves - 1; v > wave; --v) {
        const float4 va = s_ra[v][cl], vu = s_ru[v][cl];
        mu[0] = walk(va.x, vu.x, mu[0]); mu[1] = walk(va.y, vu.y, mu[1]);
        mu[2] = walk(va.z, vu.z, mu[2]); mu[3] = walk(va.w, vu.w, mu[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = walk(xa[i], xu[i], h[i]);
        mu[i] = walk(ya[i], yu[i], mu[i]);
    }
    // h before each row, in h0
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool first = w.m[r] >= 0 && (w.m[r] & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h0[r][i] = first ? h0[r][i] : h[i];
            h[i] = fmaf(al[r][i], h0[r][i], u[r][i]);
        }
    }
    float s1[4] = {}, s2[4] = {};  // sums of dg softplus(z) and of dg sigmoid(z)
    T* pdx = static_cast<T*>(A.dx) + w.r0 * A.dx_stride + w.c0;
    T* pda = static_cast<T*>(A.da) + w.r0 * A.dab_stride + w.c0;
    T* pdb = static_cast<T*>(A.db) + w.r0 * A.dab_stride + w.c0;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        const bool in = w.m[r] >= 0, last = in && (w.m[r] & 2);
        float dx[4], da[4], db[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lam = rd[r].get(i);
            if (last) {
                if (A.d_state && i < w.nc) lam += A.d_state[(int64_t)(w.m[r] >> 2) * A.C + w.c0 + i];
            } else {
                lam += mu[i];
            }
            float t;
            const float z = a[r][i] + P.dt[i];
            const float sp = softplus_t(spc, z, t);
            const float sg = (z >= 0.0f ? 1.0f : t) * rcp(1.0f + t);
            const float be = sigmoid_hw(b[r][i]);
            mu[i] = in ? al[r][i] * lam : mu[i];
            const float dg = in ? mu[i] * h0[r][i] : 0.0f;
            dx[i] = be * lam;
            db[i] = dx[i] * x[r][i] * (1.0f - be);
            const float ds = dg * sg;
            da[i] = ds * (P.k[i] / kLog2e);
            s1[i] = fmaf(dg, sp, s1[i]);
            s2[i] += ds;
        }
        if (in && w.nc > 0) {
            store4<VEC>(pdx + r * A.dx_stride, dx, w.nc);
            store4<VEC>(pda + r * A.dab_stride, da, w.nc);
            store4<VEC>(pdb + r * A.dab_stride, db, w.nc);
            if ((w.m[r] & 1) && A.d_state0) {
                const int seq = w.m[r] >> 2;
                const bool init = A.has_init ? A.has_init[seq] != 0 : true;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < w.nc) A.d_state0[(int64_t)seq * A.C + w.c0 + i] = init ? mu[i] : 0.0f;
            }
        }
    }
    // sums over the tile's rows: lanes, then waves
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float k = P.k[i] / kLog2e;
        s1[i] *= k; s2[i] *= k;
        s1[i] += __shfl_xor(s1[i], 16); s2[i] += __shfl_xor(s2[i], 16);
        s1[i] += __shfl_xor(s1[i], 32); s2[i] += __shfl_xor(s2[i], 32);
    }
    __syncthreads();
    if (lane < 16) {
        s_a[wave][cl] = make_float4(s1[0], s1[1], s1[2], s1[3]);
        s_u[wave][cl] = make_float4(s2[0], s2[1], s2[2], s2[3]);
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const int ch = threadIdx.x & 63, which = threadIdx.x >> 6;
        const float* p = reinterpret_cast<const float*>(which ? s_u : s_a) + ch;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += p[k * kTileCols];
        A.part[(tile * 2 + which) * Cp + (int64_t)col * kTileCols + ch] = v;
    }
}

// ------------------------------------------------------------------- launches

template <typename T, bool VEC, bool CKPT> static hipError_t backward_t(const ScanArgs& a, hipStream_t s) {
    const int nc = (int)(padded_channels(a.C) / kTileCols);
    const int64_t nt = n_tiles(a.n_rows), grid = nt * nc;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (grid > 0)
        hipLaunchKernelGGL((k_scan_backward<T, VEC, CKPT>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, nc, nt);
    return launch_sum_tiles(a.part, nt, a.C, 2, a.d_a_log, a.d_dt_bias, s);
}

template <typename T> static hipError_t backward_d(const ScanArgs& a, hipStream_t s) {
    if (a.q) return a.vec ? backward_t<T, true, true>(a, s) : backward_t<T, false, true>(a, s);
    return a.vec ? backward_t<T, true, false>(a, s) : backward_t<T, false, false>(a, s);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    MapArgs m = scan_map_args(a);
    m.pass_src = a.d_state; m.pass_dst = a.d_state0; m.pass_width = a.C;
    const hipError_t e = launch_map(m, s);
    if (e != hipSuccess) return e;
    return a.act_dtype == GDN_BF16 ? backward_d<bf16_t>(a, s) : backward_d<float>(a, s);
}

}  // namespace gdnt
