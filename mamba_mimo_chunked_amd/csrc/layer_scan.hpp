// Selective scan with a decay for each (channel, state): parameters and device code of the forward
// pass, the chunk aggregates and the carry between chunks, which the backward pass shares.
//
//   h[t] = exp(dt[t] a) h[t-1] + dt[t] u[t] b[t],  y[t] = <c[t], h[t]> + d u[t],  out = y silu(z)
//
// The decay depends on token, channel and state, so there is no matrix form: a token costs a channel
// N exponentials (a quarter of the rate of a multiply-add) and four multiplies or multiply-adds each.
// A lane owns one channel with NS states in registers (no exchange between lanes: <c, h> is a sum
// inside the lane), a block 64 channels with N split over KS waves; b and c of a tile of TT tokens
// lie in LDS and are read as broadcasts. Loads of the next tile are in flight during a tile.
//
// Where channels alone do not fill the GPU the time axis is cut into chunks: k_aggregate walks every
// chunk but a sequence's last from zero (its last state, and the sum of dt, which gives the chunk's
// decay exp(a sum dt)), k_carry chains the states that enter the chunks, and k_scan_fwd walks the
// chunks from them.
#pragma once
#include "layer.hpp"

namespace mimo {
namespace layer {

struct ScanParams {
    Seqs q;
    int D, G, N, Dg, tpg;           // channels, groups, states, channels and channel tiles of a group
    int softplus, zero_tail, chunked, has_z;
    Rows u, dt, b, c, z, dout;
    const float *a, *d, *bias;
    const float *init, *dstate;
    void* out;
    float* state;
    float *agg, *gagg, *sdt;        // [slots][N][D] twice, [slots][D]
    // backward
    void *du, *ddt, *db, *dc, *dz;
    float *da, *dd, *dbias, *dinit;
    float *pbc, *pdd;               // [tpg][tokens][G][2][N], [slots][2][D]
    long slots, tokens;
};

constexpr int TT = 16;   // tokens of a tile

// first row of the flat token axis of a place
__device__ __forceinline__ long flat_row(const Seqs& q, const Place& pl) { return q.cu ? (long)pl.row0 : (long)pl.i * q.S; }

// the channel tile of blockIdx.y: CPB channels of one group
struct Tile {
    int g, c0, left;   // group, first channel, channels left in the group from there
};
template <int CPB> __device__ __forceinline__ Tile tile_of(const ScanParams& p, int y) {
    Tile t;
    t.g = y / p.tpg;
    const int in = (y - t.g * p.tpg) * CPB;
    t.c0 = t.g * p.Dg + in;
    t.left = p.Dg - in;
    return t;
}

// FWD: the outputs. AGG: a chunk's last state from zero. AGG2: also the adjoint that leaves it to the
// left, sum_t exp(a sum_{s <= t} dt) c[t] dy[t], from the same exponentials.
enum { FWD, AGG, AGG2 };

template <int DT, int NS, int KS, int MODE> __global__ __launch_bounds__(64 * KS) void k_walk(ScanParams p) {
    typedef raw_t<DT> raw;
    constexpr int NP = NS * KS, TPW = (TT + KS - 1) / KS, NB = (TT * NP) / (64 * KS);
    constexpr bool C = MODE != AGG, OUT = MODE == FWD;
    __shared__ float s_dt[TT][64], s_du[TT][64], s_dy[MODE == AGG2 ? TT : 1][64];
    __shared__ __attribute__((aligned(16))) float s_b[TT][NP], s_c[C ? TT : 1][NP];
    __shared__ float s_y[OUT ? KS : 1][OUT ? TT : 1][64];
    const Place pl = place(p.q, blockIdx.x);
    if (!pl.ok) return;
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    if (MODE == AGG && (pl.i == p.q.n || t1 == pl.len)) return;
    if (MODE == AGG2 && pl.i == p.q.n) return;
    const int lane = threadIdx.x & 63, w = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile tile = tile_of<64>(p, blockIdx.y);
    const bool act = lane < tile.left;
    const int d = tile.c0 + (act ? lane : 0);
    const long D = p.D;
    raw* out = static_cast<raw*>(p.out) + flat_row(p.q, pl) * D + d;
    if (OUT && pl.i == p.q.n) {
        if (p.zero_tail && act)
            for (int t = t0 + w; t < t1; t += KS) out[t * D] = to_raw<DT>(0.f);
        return;
    }
    const raw *u = at<DT>(p.u, pl) + d, *dt = at<DT>(p.dt, pl) + d;
    const raw *z = p.has_z ? at<DT>(p.z, pl) + d : nullptr, *dout = MODE == AGG2 ? at<DT>(p.dout, pl) + d : nullptr;
    const raw *b = at<DT>(p.b, pl) + tile.g * p.N, *c = C ? at<DT>(p.c, pl) + tile.g * p.N : nullptr;
    const float bias = p.bias ? p.bias[d] : 0.f, skip = OUT && p.d ? p.d[d] : 0.f;

    float a[NS], h[NS], gr[MODE == AGG2 ? NS : 1], pr[MODE == AGG2 ? NS : 1];
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int n = w * NS + k;
        a[k] = n < p.N ? p.a[(long)d * p.N + n] * LOG2E : 0.f;
        h[k] = 0.f;
        if (MODE == AGG2) gr[k] = 0.f, pr[k] = 1.f;
        if (OUT && n < p.N) {
            if (p.chunked) h[k] = p.agg[((long)blockIdx.x * p.N + n) * D + d];
            else if (p.init) h[k] = p.init[((long)pl.i * D + d) * p.N + n];
        }
    }

    raw r_dt[TPW], r_u[TPW], r_z[TPW], r_g[TPW], r_b[NB], r_c[NB];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            const long row = min(t + w * TPW + k, t1 - 1);
            if (w * TPW + k < TT) {
                r_dt[k] = dt[row * p.dt.ts];
                r_u[k] = u[row * p.u.ts];
                if (C && z) r_z[k] = z[row * p.z.ts];
                if (MODE == AGG2) r_g[k] = dout[row * p.dout.ts];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = threadIdx.x + k * 64 * KS, n = e % NP;
            const long row = min(t + e / NP, t1 - 1);
            r_b[k] = n < p.N ? b[row * p.b.ts + n] : raw(0);
            if (C) r_c[k] = n < p.N ? c[row * p.c.ts + n] : raw(0);
        }
    };
    if (t0 < t1) fetch(t0);
    for (int tt = t0; tt < t1; tt += TT) {
        float fu[TPW], fz[TPW];
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            const int t = w * TPW + k;
            if (t < TT) {
                const float x = to_f<DT>(r_dt[k]) + bias, v = p.softplus ? softplus(x) : x;
                fu[k] = to_f<DT>(r_u[k]);
                s_dt[t][lane] = v;
                s_du[t][lane] = v * fu[k];
                if (OUT) fz[k] = z ? to_f<DT>(r_z[k]) : 0.f;
                if (MODE == AGG2) {
                    float dy = to_f<DT>(r_g[k]);
                    if (z) {
                        const float x = to_f<DT>(r_z[k]);
                        dy *= x * sigmoid(x);
                    }
                    s_dy[t][lane] = dy;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = threadIdx.x + k * 64 * KS;
            s_b[e / NP][e % NP] = to_f<DT>(r_b[k]);
            if (C) s_c[e / NP][e % NP] = to_f<DT>(r_c[k]);
        }
        __syncthreads();
        if (tt + TT < t1) fetch(tt + TT);
        const int cnt = min(TT, t1 - tt);
#pragma unroll 2
        for (int t = 0; t < cnt; ++t) {
            const float v = s_dt[t][lane], vu = s_du[t][lane];
            const float g = MODE == AGG2 ? s_dy[t][lane] : 0.f;
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            if (MODE != FWD) total += v;
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const float e = exp2_hw(v * a[k]);
                h[k] = __builtin_fmaf(e, h[k], vu * s_b[t][w * NS + k]);
                if (OUT) y[k & 3] = __builtin_fmaf(h[k], s_c[t][w * NS + k], y[k & 3]);
                if (MODE == AGG2) {
                    pr[k] *= e;
                    gr[k] = __builtin_fmaf(pr[k], g * s_c[t][w * NS + k], gr[k]);
                }
            }
            if (OUT) s_y[w][t][lane] = (y[0] + y[1]) + (y[2] + y[3]);
        }
        __syncthreads();
        if (OUT && act) {
#pragma unroll
            for (int k = 0; k < TPW; ++k) {
                const int t = w * TPW + k;
                if (t < cnt) {
                    float y = skip * fu[k];
#pragma unroll
                    for (int v = 0; v < KS; ++v) y += s_y[v][t][lane];
                    if (z) y *= fz[k] * sigmoid(fz[k]);
                    out[(tt + t) * D] = to_raw<DT>(y);
                }
            }
        }
    }
    if (!act) return;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int n = w * NS + k;
        if (n >= p.N) continue;
        if (OUT) {
            if (p.state && t1 == pl.len) p.state[((long)pl.i * D + d) * p.N + n] = h[k];
        } else {
            p.agg[((long)blockIdx.x * p.N + n) * D + d] = h[k];
            if (MODE == AGG2) p.gagg[((long)blockIdx.x * p.N + n) * D + d] = gr[k];
        }
    }
    if (!OUT && w == 0) p.sdt[(long)blockIdx.x * D + d] = total;
}

// The states that enter the chunks of sequence blockIdx.z, in place of the aggregates: a thread for each
// (channel, state blockIdx.y), AHEAD chunks of loads in flight. With ADJ, odd blockIdx.y run the adjoints
// from the last chunk to the first, from dstate, and leave the gradient of the initial state.
constexpr int AHEAD = 8;
template <bool ADJ> __global__ __launch_bounds__(256) void k_carry(ScanParams p) {
    const int d = blockIdx.x * 256 + threadIdx.x, i = blockIdx.z;
    const int n = ADJ ? blockIdx.y >> 1 : blockIdx.y;
    const bool rev = ADJ && (blockIdx.y & 1);
    if (d >= p.D) return;
    const long D = p.D, N = p.N, step = N * D;
    const int slot0 = p.q.cu ? p.q.base(i) : i * p.q.nc;
    const int len = p.q.cu ? max((i < p.q.n ? p.q.start(i + 1) : p.q.S) - p.q.start(i), 0) : p.q.S;
    const int nc = max((len + p.q.CH - 1) / p.q.CH, 1);
    const float a = p.a[d * N + n] * LOG2E;
    const long own = ((long)i * D + d) * N + n;
    const float* from = rev ? p.dstate : p.init;
    float h = from ? from[own] : 0.f;
    float* agg = (rev ? p.gagg : p.agg) + (long)slot0 * step + n * D + d;
    const float* sdt = p.sdt + (long)slot0 * D + d;
    // FWD has no aggregate of the last chunk, and needs none
    for (int j0 = 0; j0 < nc; j0 += AHEAD) {
        float x[AHEAD], s[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int j = min(j0 + k, nc - 1), at = rev ? nc - 1 - j : j;
            const bool have = ADJ ? len > 0 : j < nc - 1;
            x[k] = have ? agg[at * step] : 0.f;
            s[k] = have ? sdt[(long)at * D] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int j = j0 + k;
            if (j < nc) {
                agg[(rev ? nc - 1 - j : j) * step] = h;
                h = __builtin_fmaf(exp2_hw(a * s[k]), h, x[k]);
            }
        }
    }
    if (rev && p.dinit) p.dinit[own] = h;
}

// ---------------------------------------------------------------- host side
// (states of a lane, waves) of the walk: the smallest that hold N
template <int DT, int MODE> mimo_status launch_walk(const ScanParams& p, hipStream_t st) {
    const dim3 grid((unsigned)p.slots, (unsigned)(p.G * p.tpg));
    if (p.N <= 4) return launch(&k_walk<DT, 4, 1, MODE>, grid, 64, 0, st, p);
    if (p.N <= 8) return launch(&k_walk<DT, 8, 1, MODE>, grid, 64, 0, st, p);
    if (p.N <= 16) return launch(&k_walk<DT, 16, 1, MODE>, grid, 64, 0, st, p);
    if (p.N <= 32) return launch(&k_walk<DT, 16, 2, MODE>, grid, 128, 0, st, p);
    if (p.N <= 64) return launch(&k_walk<DT, 16, 4, MODE>, grid, 256, 0, st, p);
    return launch(&k_walk<DT, 16, 8, MODE>, grid, 512, 0, st, p);
}
inline int waves_for(int64_t N) { return N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8; }

inline mimo_status check_scan(int64_t n, int64_t S, int64_t D, int64_t G, int64_t N, int dtype) {
    const mimo_status s = check_sequences(n, S, D, dtype);
    if (s != MIMO_OK) return s;
    if (G < 1 || N < 1) return bad("G and N must be positive");
    if (D % G) return bad("the channels must be divisible by the groups");
    if (N > MAMBA_SCAN_MAX_STATE) return unsupported("more than 128 states");
    if (G > 1024) return unsupported("more than 1024 groups");
    if (n * S > (int64_t)1 << 40) return unsupported("too many tokens");
    return MIMO_OK;
}


}  // namespace layer
}  // namespace mimo
