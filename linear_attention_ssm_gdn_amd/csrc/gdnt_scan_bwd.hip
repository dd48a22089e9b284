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
// registers and one workgroup on a compute unit cost less than the
// transcendentals again.
#include "gdnt_chain.hpp"
#include "gdnt_rows.hpp"

namespace gdnt {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
static_assert(kWaves * 2 * FR == kTileRows && 32 * 2 == kTileCols, "tile shape");

// The lane's 16 rows by two channels of one tensor of the checkpoint.
struct Ckpt2 {
    uint32_t w[FR / 2];
    float sc, off;  // value = byte * sc + off, the byte unsigned (offset by 128)
    __device__ __forceinline__ float get(int r, int i) const {
        const uint32_t b = (w[r & 7] >> ((r >> 3) * 16 + i * 8)) & 0xffu;
        return fmaf((float)b, sc, off);  // 128 * sc is exact: one rounding, that of q * sc
    }
};

// Makes the compiler take a register's value for a new one: what was computed
// from it before is computed again instead of being kept in more registers.
__device__ __forceinline__ void again(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void again(uint32_t& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void again(float2& v) { again(v.x); again(v.y); }

template <typename T, bool VEC, bool CKPT>
__global__ __launch_bounds__(kThreads, 2) void k_scan_backward(const ScanArgs A, int n_cols, int64_t n_tiles) {
    __shared__ float2 s_a[kWaves][32], s_u[kWaves][32], s_ra[kWaves][32], s_ru[kWaves][32], s_h[32];
    __shared__ uint32_t s_ticket;
    if (threadIdx.x == 0) s_ticket = atomicAdd(A.ticket, 1u);
    __syncthreads();
    const uint32_t ticket = __builtin_amdgcn_readfirstlane(s_ticket);
    const int64_t tile = n_tiles - 1 - ticket / (uint32_t)n_cols;
    const int col = (int)(ticket % (uint32_t)n_cols);
    const int lane = threadIdx.x & 63, half = lane >> 5, hl = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t Cp = (int64_t)n_cols * kTileCols;
    const int64_t r0 = tile * kTileRows + wave * 2 * FR, cb = (int64_t)col * kTileCols, c0 = cb + hl * 2;
    const int64_t left = (int64_t)A.C - c0;
    const int nc = left >= 2 ? 2 : left > 0 ? (int)left : 0;

    // the wave's 32 rows as bits, and this half's 16
    const int32_t m32 = lane < 2 * FR ? A.map[r0 + lane] : -1;
    const uint32_t in = (uint32_t)__ballot(m32 >= 0), firsts = (uint32_t)__ballot(m32 >= 0 && (m32 & 1)),
                   lasts = (uint32_t)__ballot(m32 >= 0 && (m32 & 2));
    const uint32_t my_in = in >> (half * FR), my_firsts = firsts >> (half * FR), my_lasts = lasts >> (half * FR);
    const uint32_t any_first = firsts | firsts >> FR, any_last = lasts | lasts >> FR;
    auto seq_of = [&](int r) { return __shfl(m32, half * FR + r) >> 2; };  // all lanes together

    auto rows = [&](const void* base, int64_t stride) {
        return WaveRows<T, VEC>(base, stride, A.n_rows, r0, A.C, cb, half * FR * stride + hl * 2);
    };
    const bool whole = in == 0xffffffffu;
    const WaveRows<T, VEC> D = rows(A.dh, A.dh_stride);
    Raw2<T> rd[FR], rx[FR], ra[FR], rb[FR];
    Ckpt2 qx, qa, qb;
    if constexpr (CKPT) {
        const int64_t n4 = Cp / 4, blk = r0 / FR + half, c4 = cb / 4 + (hl >> 1);
        auto get = [&](int t, Ckpt2& q) {
            const int64_t at = (blk * 3 + t) * n4 + c4;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            q.sc = 0.0f;
            if (r0 + half * FR < A.n_rows) {
                const uint4* p = reinterpret_cast<const uint4*>(A.q + at * 64 + (hl & 1) * 32);
                lo = p[0];
                hi = p[1];
                q.sc = A.q_scale[at];
            }
            q.off = -128.0f * q.sc;
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int r = 0; r < FR / 2; ++r) q.w[r] = swap_halves(w[r], lane) ^ 0x80808080u;
        };
        get(1, qa);
        get(2, qb);
        get(0, qx);
    } else {
        const WaveRows<T, VEC> X = rows(A.x, A.x_stride), Ag = rows(A.a, A.ab_stride), Bg = rows(A.b, A.ab_stride);
        if (whole && nc > 0) {
#pragma unroll
            for (int r = 0; r < FR; ++r) {
                ra[r] = Ag.load(r, nc);
                rb[r] = Bg.load(r, nc);
                rx[r] = X.load(r, nc);
            }
        } else {
#pragma unroll
            for (int r = 0; r < FR; ++r) {
                rx[r] = zero2<T>(); ra[r] = zero2<T>(); rb[r] = zero2<T>();
                if ((my_in >> r & 1u) && nc > 0) {
                    ra[r] = Ag.load(r, nc);
                    rb[r] = Bg.load(r, nc);
                    rx[r] = X.load(r, nc);
                }
            }
        }
    }
    if (whole && nc > 0) {
#pragma unroll
        for (int r = 0; r < FR; ++r) rd[r] = D.load(r, nc);
    } else {
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            rd[r] = zero2<T>();
            if ((my_in >> r & 1u) && nc > 0) rd[r] = D.load(r, nc);
        }
    }
    if (VEC && (A.C & 1) && col == n_cols - 1) {
        fix_last(rd, nc);
        if constexpr (!CKPT) {
            fix_last(rx, nc);
            fix_last(ra, nc);
            fix_last(rb, nc);
        }
    }
    float dt[2], kk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        dt[i] = i < nc ? A.dt_bias[c0 + i] : 0.0f;
        kk[i] = i < nc ? -expf(A.a_log[c0 + i]) * kLog2e : 0.0f;
    }
    auto get_x = [&](int r, int i) { return CKPT ? qx.get(r, i) : rx[r].get(i); };

    // the state a sequence starts from (seq -1: none)
    auto initial = [&](int seq, float (&h0)[2]) {
        const bool init = seq >= 0 && (A.has_init ? A.has_init[seq] != 0 : true);
        const int64_t at = init ? (int64_t)A.page_idx[seq] * A.st_in_stride + c0 : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) h0[i] = init && i < nc ? load_state(A.st_in, at + i, A.state_dtype) : 0.0f;
    };

    // first walk: y = g log2(e), sigmoid(z), beta, and the rows' run.  Rows of
    // no sequence run along on zeros (see the forward pass).
    float y[FR][2], sg[FR][2], be[FR][2];
    float ea[2] = {1.0f, 1.0f}, eu[2] = {};
    const SoftplusC spc = softplus_consts();
#pragma unroll
    for (int r = 0; r < FR; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t;
            const float z = (CKPT ? qa.get(r, i) : ra[r].get(i)) + dt[i];
            y[r][i] = kk[i] * softplus_t(spc, z, t);
            const float s = rcp(1.0f + t);
            sg[r][i] = z >= 0.0f ? s : t * s;
            be[r][i] = sigmoid_hw(CKPT ? qb.get(r, i) : rb[r].get(i));
            const float al = exp2_hw(y[r][i]), u = be[r][i] * get_x(r, i);
            eu[i] = fmaf(al, eu[i], u);
            ea[i] *= al;
        }
        if (any_first >> r & 1u) {
            float h0[2];
            initial(seq_of(r), h0);
            if (my_firsts >> r & 1u) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    eu[i] = fmaf(exp2_hw(y[r][i]), h0[i], be[r][i] * get_x(r, i));
                    ea[i] = -1.0f;
                }
            }
        }
    }
    // the run from the last row to the first: mu -> fa mu + fu
    float fa[2] = {fabsf(ea[0]), fabsf(ea[1])}, fu[2] = {};
    if (firsts | lasts) { fa[0] = fa[1] = 1.0f; }
#pragma unroll
    for (int r = FR - 1; r >= 0; --r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float al = exp2_hw(y[r][i]);
            fu[i] = al * (rd[r].get(i) + fu[i]);
            if (firsts | lasts) fa[i] *= al;
        }
        if (any_last >> r & 1u) {
            const int seq = seq_of(r);
            if (my_lasts >> r & 1u) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float lam = rd[r].get(i);
                    if (A.d_state && i < nc) lam += A.d_state[(int64_t)seq * A.C + c0 + i];
                    fu[i] = exp2_hw(y[r][i]) * lam;
                    fa[i] = -1.0f;
                }
            }
        }
    }
    float xa[2], xu[2], ya[2], yu[2];  // the run of the wave's other half
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ea[i] = copysignf(fmaxf(fabsf(ea[i]), kTiny), ea[i]);
        fa[i] = copysignf(fmaxf(fabsf(fa[i]), kTiny), fa[i]);
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
    __syncthreads();
    const int32_t m_first = A.map[tile * kTileRows];
    if (wave == 0) {  // one channel a lane
        const int32_t m_last = A.map[tile * kTileRows + kTileRows - 1];
        const int32_t m_prev = tile > 0 ? A.map[tile * kTileRows - 1] : -1;
        const float* pa = reinterpret_cast<const float*>(s_ra) + lane;
        const float* pu = reinterpret_cast<const float*>(s_ru) + lane;
        float ta = pa[(kWaves - 1) * kTileCols], tu = pu[(kWaves - 1) * kTileCols];
#pragma unroll
        for (int v = kWaves - 2; v >= 0; --v) {
            float ja = pa[v * kTileCols], ju = pu[v * kTileCols];
            join(ta, tu, ja, ju);
            ta = ja; tu = ju;
        }
        const Chain chain{A.chain, n_tiles * Cp};
        const float a1[1] = {ta}, u1[1] = {tu};
        float h1[1];
        hand_on<1>(chain, tile * Cp + cb, Cp, n_tiles - 1 - tile, m_last >= 0 && !(m_last & 2),
                   m_prev >= 0 && !(m_prev & 2), a1, u1, h1, A.err);
        reinterpret_cast<float*>(s_h)[lane] = h1[0];
    }
    __syncthreads();
    float h[2] = {}, mu[2] = {s_h[hl].x, s_h[hl].y};
    if (m_first >= 0 && !(m_first & 1)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < nc) h[i] = A.states[tile * A.C + c0 + i];
    }
    for (int v = 0; v < wave; ++v) {
        const float2 va = s_a[v][hl], vu = s_u[v][hl];
        h[0] = walk(va.x, vu.x, h[0]);
        h[1] = walk(va.y, vu.y, h[1]);
    }
    for (int v = kWaves - 1; v > wave; --v) {
        const float2 va = s_ra[v][hl], vu = s_ru[v][hl];
        mu[0] = walk(va.x, vu.x, mu[0]);
        mu[1] = walk(va.y, vu.y, mu[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (half) h[i] = walk(xa[i], xu[i], h[i]);
        else mu[i] = walk(ya[i], yu[i], mu[i]);
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
    const WaveRows<T, VEC> DX = rows(A.dx, A.dx_stride), DA = rows(A.da, A.dab_stride), DB = rows(A.db, A.dab_stride);
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
                    lam[i] = rd[r].get(i);
                    if (A.d_state && i < nc) lam[i] += A.d_state[(int64_t)seq * A.C + c0 + i];
                }
            }
        }
        const bool mine = whole || (my_in >> r & 1u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mu[i] = exp2_hw(y[r][i]) * lam[i];
            const float dg = mine ? mu[i] * hp[r][i] : 0.0f;
            const float ds = dg * sg[r][i];
            dx[i] = be[r][i] * lam[i];
            db[i] = dx[i] * get_x(r, i) * (1.0f - be[r][i]);
            da[i] = ds * kg[i];
            s1[i] = fmaf(dg, y[r][i], s1[i]);
            s2[i] += ds;
        }
        if (mine && nc > 0) {
            DX.store(r, nc, dx[0], dx[1]);
            DA.store(r, nc, da[0], da[1]);
            DB.store(r, nc, db[0], db[1]);
        }
        if ((any_first >> r & 1u) && A.d_state0) {
            const int seq = seq_of(r);
            if (my_firsts >> r & 1u) {
                const bool init = A.has_init ? A.has_init[seq] != 0 : true;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (i < nc) A.d_state0[(int64_t)seq * A.C + c0 + i] = init ? mu[i] : 0.0f;
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
    __syncthreads();
    if (!half) {
        s_a[wave][hl] = make_float2(s1[0], s1[1]);
        s_u[wave][hl] = make_float2(s2[0], s2[1]);
    }
    __syncthreads();
    if (wave < 2) {
        const float* p = reinterpret_cast<const float*>(wave ? s_u : s_a) + lane;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += p[k * kTileCols];
        A.part[(tile * 2 + wave) * Cp + cb + lane] = v;
    }
}

// ------------------------------------------------------------------- launches

template <typename T, bool VEC, bool CKPT> static hipError_t backward_t(const ScanArgs& a, hipStream_t s) {
    const int nc = (int)(padded_channels(a.C) / kTileCols);
    const int64_t nt = n_tiles(a.n_rows), grid = nt * nc;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    // VEC addresses a wave's 32 rows by 32-bit byte offsets
    if (VEC && ((CKPT ? 0 : a.x_stride | a.ab_stride) | a.dh_stride | a.dx_stride | a.dab_stride) >> 24)
        return backward_t<T, false, CKPT>(a, s);
    if (grid > 0)
        hipLaunchKernelGGL((k_scan_backward<T, VEC, CKPT>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, nc, nt);
    return launch_sum_tiles(a.part, nt, a.C, 2, a.d_a_log, a.d_dt_bias, s);
}

template <typename T> static hipError_t backward_d(const ScanArgs& a, hipStream_t s) {
    if (a.q) return a.vec2 ? backward_t<T, true, true>(a, s) : backward_t<T, false, true>(a, s);
    return a.vec2 ? backward_t<T, true, false>(a, s) : backward_t<T, false, false>(a, s);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    MapArgs m = scan_map_args(a);
    m.pass_src = a.d_state; m.pass_dst = a.d_state0; m.pass_width = a.C;
    const hipError_t e = launch_map(m, s);
    if (e != hipSuccess) return e;
    return a.act_dtype == GDN_BF16 ? backward_d<bf16_t>(a, s) : backward_d<float>(a, s);
}

}  // namespace gdnt
