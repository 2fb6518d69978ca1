// Selective scan, backward pass.
//
// With dy = dout silu(z) and the adjoint g[t] = c[t] dy[t] + exp(dt[t+1] a) g[t+1]:
//   dc = sum_d dy h          db = sum_d g dt u        s = <g, b>        X = g exp(dt a) h[t-1]
//   du = dt s + d dy         d(dt) = u s + <X, a>     da = sum X dt     dz = dout y silu'(z)
// k_walk<AGG2> cuts the time axis into chunks (one walk for the states and the adjoints that
// leave each chunk), k_carry chains both, k_scan_bwd makes the gradients of each chunk, k_sums adds
// up the partial sums in order (no atomics: equal inputs give equal bits).
//
// k_scan_bwd. A wave holds 64 / Q channels; the Q lanes of a channel hold NS states each, so <c, h>,
// <g, b> and <X, a> are sums over Q neighbouring lanes, and the sums over channels (db, dc) are folds
// of NS values over the 64 / Q others: each fold halves the values a lane keeps, two operations a
// pair. A chunk is taken in units of 16 tokens from the last to the first, a unit in sub-tiles of ST
// tokens likewise: forward with the states and decays of its ST tokens in registers (2 * NS * ST of
// them: 128, or 64 for Q = 2, whose staging takes the rest), then backward through them. The state in
// front of a unit comes from the walk, which leaves it (from zero, at the chunk's start) with the sum of
// dt to there: h = uh + exp(a udt) h(chunk). So an exponential is computed twice (walk, sub-tile) and no
// state but every sixteenth goes to memory. 4 x 4096 tokens, D = 1024, N = 16, bf16: 330 us, of them the
// walk 86, this kernel 250 (its vector units busy 77 % of the time: 97 vector instructions a token and
// 64 states), sums 12 (times under a profiler); walking the chunk a third time for its states, with 64-bit row addresses, took
// 415 us. Vector instructions bind; two waves a SIMD fill 256 registers each (with 168 and three waves:
// 436 us) and more: what lives across a sub-tile (the states of the chunk and the unit, the next unit's, da) stays in scratch
// memory in part, 4 registers at N = 9 to 16, 28 to 30 to N = 32, 19 to 24 to N = 64, 31 to 33 to N = 128, none to N = 8.
// 2 x 2048 tokens, D = 1024, bf16: N = 8 79 us, 32 (fp32) 208, 64 335; 2 x 1024, N = 128 396.
// Lanes work on nothing where N is less than the shape's states (8, 16, 32, 64, 128: at N = 1 seven eighths of them) and where
// the channels of a group do not fill its tile (128 channels to N = 8, 64 to 32, 32 to 64, 16 to 128).
#include "layer_scan.hpp"

namespace mimo {
namespace layer {
namespace {

// channels of a block, LDS floats: staging of dt, dt u, dy, three sums; b, c, and zeros in their place for lanes without a
// channel (zero times an infinite b or c would be NaN in the folds); fold results of four waves; the states in front of
// a unit's later sub-tiles
template <int NS, int Q> struct Shape {
    static constexpr int ST = NS == 4 && Q == 4 ? 16 : 8, NP = NS * Q, CPW = 64 / Q, CPB = 4 * CPW;
    static constexpr int ROWS = ST * CPB, BC = ST * NP, FOLD = 4 * 2 * BC;
    static constexpr int SUBS = UNIT / ST, CKPT = SUBS > 1 ? (SUBS - 1) * 256 * NS : 0;
    static constexpr size_t lds = sizeof(float) * (6 * ROWS + 4 * BC + FOLD + CKPT);
};

// the NS values of the lanes that hold other channels of the same states, summed: NS / 4 (CPW = 4),
// else one value is left to a lane: state `own` of the lane's NS (and the next ones)
template <int NS, int Q> __device__ __forceinline__ void fold_channels(float (&v)[NS], bool bit3) {
    constexpr int CPW = 64 / Q;
#pragma unroll
    for (int k = 0; k < NS / 2; ++k) v[k] = fold32(v[k], v[k + NS / 2]);
#pragma unroll
    for (int k = 0; k < NS / 4; ++k) v[k] = fold16(v[k], v[k + NS / 4]);
    if constexpr (CPW >= 8) {
        if constexpr (NS == 8) v[0] = fold8(v[0], v[1], bit3);
        else v[0] = add_dpp<DPP_ROR8>(v[0]);
    }
    if constexpr (CPW >= 16) v[0] = NS == 8 ? add_xor4(v[0]) : add_dpp<DPP_ROR4>(v[0]);
    if constexpr (CPW >= 32) v[0] = add_dpp<DPP_XOR2>(v[0]);
}

//
// The places of a channel's states behind the last one read zeros for b and c, but an infinite input times zero is NaN, and
// so would the sums over the states be. PAD = 1, whole lanes of them: left out of the three sums; 2, some of a lane: its h
// and g are set to zero there in each step, and a is so small that no finite step makes more than 2^34 of its decay, an
// infinite one zero ([2 x 2048, 1024] bf16, N = 24: 192 us, 190 without; N = 13: 110 and 108; [2 x 2048, 512], N = 100: 398 and 384).
template <int DT, int NS, int Q, int PAD> __global__ __launch_bounds__(256, 2) void k_scan_bwd(ScanParams p) {
    typedef raw_t<DT> raw;
    typedef Shape<NS, Q> H;
    constexpr int ST = H::ST, NP = H::NP, CPB = H::CPB, SUBS = H::SUBS, NT = (ST * CPB + 255) / 256, NB = (H::BC + 255) / 256;
    constexpr int LEFT = H::CPW == 4 ? NS / 4 : 1;    // values a lane keeps of a fold
    constexpr int SD = 256 / CPB;                     // tokens staged at a time
    static_assert(CPB <= 256 && 256 % CPB == 0 && H::FOLD >= 512 && UNIT % ST == 0, "staging");
    extern __shared__ __attribute__((aligned(16))) float lds[];
    float *s_dt = lds, *s_du = s_dt + H::ROWS, *s_dy = s_du + H::ROWS;   // [ST][CPB]
    float* s_sum = s_dy + H::ROWS;                                       // y, s, <X, a>: [3][ST][CPB]
    float *s_b = s_sum + 3 * H::ROWS, *s_c = s_b + H::BC;                // [ST][NP]
    float* s_fold = s_c + 3 * H::BC;                                     // behind 2 * BC zeros; [4][2][ST][NP]
    float* s_ck = s_fold + H::FOLD;                                      // [SUBS - 1][NS/4][256][4]
    const Place pl = place(p.q, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane % Q, cb = w * H::CPW + lane / Q;
    const Tile tile = tile_of<CPB>(p, blockIdx.y);
    const long D = p.D, N = p.N, G = p.G;
    if (!pl.ok || pl.i == p.q.n) {  // no tokens of a sequence: nothing for the parameters' gradients
        for (int e = tid; e < min(CPB, tile.left) * p.N; e += 256) p.agg[(blockIdx.x * D + tile.c0) * N + e] = 0.f;
        for (int e = tid; e < CPB * 2; e += 256)
            if (e % CPB < tile.left) p.pdd[((long)blockIdx.x * 2 + e / CPB) * D + tile.c0 + e % CPB] = 0.f;
        if (!pl.ok) return;
    }
    const long flat = flat_row(p.q, pl);
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    const int in_group = blockIdx.y - tile.g * p.tpg;
    // partial db, dc of this channel tile: [token][group][2][N]
    float* pbc = p.pbc + (((long)in_group * p.tokens + flat) * G + tile.g) * 2 * N;
    // Staging: a thread takes channel sc of the tile and tokens st + k * SD (the same for a whole wave where
    // the tile has 64 channels: the row's address is scalar then)
    const int sc = tid % CPB, st = CPB >= 64 ? __builtin_amdgcn_readfirstlane(tid / CPB) : tid / CPB;
    const bool sact = sc < tile.left;
    const unsigned off = sact ? sc : 0;
    const int sd = tile.c0 + off;
    raw *du = static_cast<raw*>(p.du) + flat * D + tile.c0, *ddt = static_cast<raw*>(p.ddt) + flat * D + tile.c0;
    raw* dz = p.has_z ? static_cast<raw*>(p.dz) + flat * D + tile.c0 : nullptr;
    if (pl.i == p.q.n) {            // behind the last sequence
        const raw zero = to_raw<DT>(0.f);
        for (int t = t0 + st; t < t1; t += SD)
            if (sact) {
                (du + t * D)[off] = zero;
                (ddt + t * D)[off] = zero;
                if (dz) (dz + t * D)[off] = zero;
            }
        for (int e = tid; e < (t1 - t0) * 2 * p.N; e += 256) pbc[(long)(t0 + e / (2 * p.N)) * G * 2 * N + e % (2 * p.N)] = 0.f;
        return;
    }
    const raw *gu = at<DT>(p.u, pl) + tile.c0, *gdt = at<DT>(p.dt, pl) + tile.c0, *gdo = at<DT>(p.dout, pl) + tile.c0;
    const raw* gz = p.has_z ? at<DT>(p.z, pl) + tile.c0 : nullptr;
    const float bias = p.bias ? p.bias[sd] : 0.f, skip = p.d ? p.d[sd] : 0.f;
    // element tid (and tid + 256, ...) of the rows of b and c
    const int bn = tid % NP, br = tid / NP;
    constexpr int BR = 256 / NP;
    const bool bon = bn < p.N && br < ST;
    const raw *gb = at<DT>(p.b, pl) + (long)br * p.b.ts + tile.g * p.N + bn, *gc = at<DT>(p.c, pl) + (long)br * p.c.ts + tile.g * p.N + bn;

    const bool act = cb < tile.left;
    const int bq = act ? q * NS : 2 * H::BC + q * NS;
    if (tile.left < CPB)
        for (int e = tid; e < 2 * H::BC; e += 256) s_c[H::BC + e] = 0.f;
    const int d = tile.c0 + (act ? cb : 0);
    float a[NS], hc[NS], h[NS], g[NS], da[NS] = {};   // hc: the chunk's first state
    const long dn = d * N;
    const float* h0 = p.chunked ? p.agg + blockIdx.x * D * N : p.init ? p.init + pl.i * D * N : nullptr;
    const float* g0 = p.chunked ? p.gagg + blockIdx.x * D * N : p.dstate ? p.dstate + pl.i * D * N : nullptr;
    load_states(p.a + dn, q * NS, p.N, p.vec, 0.f, a);
    if (h0) load_states(h0 + dn, q * NS, p.N, p.vec, 0.f, hc);
    if (g0) load_states(g0 + dn, q * NS, p.N, p.vec, 0.f, g);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        a[k] = act ? decay_base(a[k]) : 0.f;
        hc[k] = h0 && act ? hc[k] : 0.f;
        g[k] = g0 && act ? g[k] : 0.f;
    }
    bool on[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        on[k] = PAD != 2 || q * NS + k < p.N;
        if (!on[k]) a[k] = -1e-37f;
    }
    const bool lane_on = PAD != 1 || q * NS < p.N;
    const int nunit = (t1 - t0 + UNIT - 1) / UNIT;

    raw r_dt[NT], r_u[NT], r_z[NT], r_g[NT], r_b[NB], r_c[NB];
    auto fetch = [&](int tt, bool all) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            if (NT * SD > ST && st + k * SD >= ST) continue;
            const long row = min(tt + st + k * SD, t1 - 1);
            r_dt[k] = (gdt + row * p.dt.ts)[off];
            r_u[k] = (gu + row * p.u.ts)[off];
            if (all) {
                r_g[k] = (gdo + row * p.dout.ts)[off];
                if (gz) r_z[k] = (gz + row * p.z.ts)[off];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const bool on = bon && tt + br + k * BR < t1;
            r_b[k] = raw(0);
            if (on) r_b[k] = gb[(tt + k * BR) * p.b.ts];
            if (all) {
                r_c[k] = raw(0);
                if (on) r_c[k] = gc[(tt + k * BR) * p.c.ts];
            }
        }
    };
    float f_u[NT], f_z[NT], f_g[NT], f_x[NT], f_dt[NT], f_dy[NT], f_gate[NT];
    // A tile's values to LDS. Tokens past the chunk and lanes past the group take no step (dt = 0): they pass the
    // state and the adjoint on and add nothing.
    auto stage = [&](int tt, bool all) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            f_x[k] = to_f<DT>(r_dt[k]) + bias;
            f_u[k] = to_f<DT>(r_u[k]);
            f_dt[k] = f_x[k];
        }
        if (p.softplus) {
#pragma unroll
            for (int k = 0; k < NT; ++k) f_dt[k] = softplus(f_x[k]);
        }
        if (all) {
#pragma unroll
            for (int k = 0; k < NT; ++k) f_dy[k] = f_g[k] = to_f<DT>(r_g[k]);
            if (gz) {
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    f_z[k] = to_f<DT>(r_z[k]);
                    f_gate[k] = sigmoid(f_z[k]);
                    f_dy[k] *= f_z[k] * f_gate[k];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const int t = st + k * SD;
            if (NT * SD > ST && t >= ST) continue;
            if (!sact || tt + t >= t1) f_dt[k] = f_u[k] = f_dy[k] = 0.f;
            s_dt[t * CPB + sc] = f_dt[k];
            s_du[t * CPB + sc] = f_dt[k] * f_u[k];
            if (all) s_dy[t * CPB + sc] = f_dy[k];
        }
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (br + k * BR < ST) {
                s_b[(br + k * BR) * NP + bn] = to_f<DT>(r_b[k]);
                if (all) s_c[(br + k * BR) * NP + bn] = to_f<DT>(r_c[k]);
            }
    };
    float uh[NS], ut = 0.f;
    const long unit0 = first_unit(p, pl) - 1;
    auto fetch_unit = [&](int k) {
        const long at = unit0 + k;
        load_states(p.uh + at * D * N + dn, q * NS, p.N, p.vec, 0.f, uh);
        ut = p.udt[at * D + d];
    };
    // the state a lane's first kept value of a fold belongs to; which of the three sums lane q of a channel writes
    const int own = q * NS + ((lane >> 5) & 1) * (NS / 2) + ((lane >> 4) & 1) * (NS / 4) + (NS == 8 && H::CPW >= 8 ? (lane >> 3) & 1 : 0);
    float* fold_at = s_fold + w * 2 * H::BC + own;
    float* sum_at = s_sum + min(q, 2) * H::ROWS + cb;

    float acc_d = 0.f, acc_bias = 0.f;
    if (nunit > 1) fetch_unit(nunit - 1);
    // A unit's sub-tiles but the last are walked for the states behind them (SUBS > 1), then all taken from the last
    // to the first. What a stage writes is not read behind the barrier at the end of the computation, and what that
    // computation left is read before the next stage's barrier, so two barriers a sub-tile suffice.
    if (nunit > 0) fetch(t0 + (nunit - 1) * UNIT, SUBS == 1);
    for (int unit = nunit - 1; unit >= 0; --unit) {
        const int tu = t0 + unit * UNIT;
        float hu[NS];
#pragma unroll
        for (int k = 0; k < NS; ++k) hu[k] = unit > 0 && act ? __builtin_fmaf(exp2_hw(a[k] * ut), hc[k], uh[k]) : hc[k];
        if (unit > 1) fetch_unit(unit - 1);
        if constexpr (SUBS > 1) {
#pragma unroll
            for (int k = 0; k < NS; ++k) h[k] = hu[k];
#pragma unroll 1
            for (int s = 0; s + 1 < SUBS; ++s) {
                stage(tu + s * ST, false);
                __syncthreads();
                fetch(tu + (s + 1) * ST, s + 2 == SUBS);
#pragma unroll
                for (int t = 0; t < ST; ++t) {
                    const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb];
#pragma unroll
                    for (int k = 0; k < NS; ++k) {
                        h[k] = __builtin_fmaf(exp2_hw(v * a[k]), h[k], vu * s_b[t * NP + bq + k]);
                        if (PAD == 2) h[k] = on[k] ? h[k] : 0.f;
                    }
                }
#pragma unroll
                for (int k = 0; k < NS; k += 4)
                    *reinterpret_cast<float4*>(s_ck + ((s * (NS / 4) + k / 4) * 256 + tid) * 4) = make_float4(h[k], h[k + 1], h[k + 2], h[k + 3]);
                __syncthreads();
            }
        }
#pragma unroll 1
        for (int s = SUBS - 1; s >= 0; --s) {
            const int tt = tu + s * ST;
            stage(tt, true);
            __syncthreads();
            if (s > 0) fetch(tt - ST, true);
            else if (unit > 0) fetch(tu - UNIT, SUBS == 1);
            // waves that compute go first: the other block's staging and stores fill the gaps (353 -> 347 us)
            __builtin_amdgcn_s_setprio(1);
            float hp[ST][NS], e[ST][NS];   // the state in front of each token, its decay
#pragma unroll
            for (int k = 0; k < NS; ++k) h[k] = hu[k];
            if (s > 0) {
#pragma unroll
                for (int k = 0; k < NS; k += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(s_ck + (((s - 1) * (NS / 4) + k / 4) * 256 + tid) * 4);
                    h[k] = x.x, h[k + 1] = x.y, h[k + 2] = x.z, h[k + 3] = x.w;
                }
            }
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb];
#pragma unroll
                for (int k = 0; k < NS; ++k) {
                    hp[t][k] = h[k];
                    e[t][k] = exp2_hw(v * a[k]);
                    h[k] = __builtin_fmaf(e[t][k], h[k], vu * s_b[t * NP + bq + k]);
                    if (PAD == 2) h[k] = on[k] ? h[k] : 0.f;
                }
            }
#pragma unroll
            for (int t = ST - 1; t >= 0; --t) {
                const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb], dy = s_dy[t * CPB + cb];
                float y = 0.f, sgb = 0.f, sxa = 0.f, vb[NS], vc[NS];
#pragma unroll
                for (int k = 0; k < NS; ++k) {
                    const float b = s_b[t * NP + bq + k], c = s_c[t * NP + bq + k];
                    const float ht = t == ST - 1 ? h[k] : hp[t + 1 < ST ? t + 1 : 0][k];
                    g[k] = __builtin_fmaf(c, dy, g[k]);
                    if (PAD == 2) g[k] = on[k] ? g[k] : 0.f;
                    y = __builtin_fmaf(c, ht, y);
                    sgb = __builtin_fmaf(g[k], b, sgb);
                    vc[k] = dy * ht;
                    vb[k] = g[k] * vu;
                    g[k] *= e[t][k];
                    const float x = g[k] * hp[t][k];
                    sxa = __builtin_fmaf(x, a[k], sxa);
                    da[k] = __builtin_fmaf(x, v, da[k]);
                }
                if (PAD == 1) {
                    y = lane_on ? y : 0.f;
                    sgb = lane_on ? sgb : 0.f;
                    sxa = lane_on ? sxa : 0.f;
                }
                y = sum_lanes<Q>(y);
                sgb = sum_lanes<Q>(sgb);
                sxa = sum_lanes<Q>(sxa);
                if constexpr (Q >= 4) sum_at[t * CPB] = q == 0 ? y : q == 1 ? sgb : sxa;
                else {
                    sum_at[t * CPB] = q == 0 ? y : sgb;
                    if (q == 0) s_sum[2 * H::ROWS + t * CPB + cb] = sxa;
                }
                fold_channels<NS, Q>(vb, lane & 8);
                fold_channels<NS, Q>(vc, lane & 8);
#pragma unroll
                for (int k = 0; k < LEFT; ++k) {
                    fold_at[t * NP + k] = vb[k];
                    fold_at[(ST + t) * NP + k] = vc[k];
                }
            }
            __syncthreads();
            __builtin_amdgcn_s_setprio(0);
            if (sact) {
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    const int t = st + k * SD;
                    if (t >= ST || tt + t >= t1) continue;
                    const float* s = s_sum + t * CPB + sc;
                    const float y = s[0], sgb = s[H::ROWS], sxa = s[2 * H::ROWS] * LN2;
                    float x = __builtin_fmaf(f_u[k], sgb, sxa);
                    if (p.softplus) x *= sigmoid(f_x[k]);
                    const long row = (tt + t) * D;
                    (du + row)[off] = to_raw<DT>(__builtin_fmaf(f_dt[k], sgb, skip * f_dy[k]));
                    (ddt + row)[off] = to_raw<DT>(x);
                    if (dz) (dz + row)[off] = to_raw<DT>(f_g[k] * __builtin_fmaf(skip, f_u[k], y) * silu_slope(f_z[k], f_gate[k]));
                    acc_d = __builtin_fmaf(f_dy[k], f_u[k], acc_d);
                    acc_bias += x;
                }
            }
#pragma unroll
            for (int k = 0; k < (2 * H::BC + 255) / 256; ++k) {   // [m][token][state] of the four waves
                const int i = tid + k * 256, n = i % NP, row = i / NP, m = row / ST, t = row % ST;
                if (i < 2 * H::BC && n < p.N && tt + t < t1) {
                    const float* f = s_fold + i;
                    pbc[(tt + t) * G * 2 * N + m * N + n] = (f[0] + f[2 * H::BC]) + (f[4 * H::BC] + f[6 * H::BC]);
                }
            }
        }
    }

    // this chunk's share of da, dd, d(dt_bias); the gradient of the initial state where nothing was cut
    if (act) {
        store_states(p.agg + blockIdx.x * D * N + dn, q * NS, p.N, p.vec, da);
        if (!p.chunked && p.dinit) store_states(p.dinit + pl.i * D * N + dn, q * NS, p.N, p.vec, g);
    }
    __syncthreads();
    s_fold[tid] = acc_d;
    s_fold[256 + tid] = acc_bias;
    __syncthreads();
    if (tid < CPB && sact) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < SD; ++k) {
            x += s_fold[tid + k * CPB];
            y += s_fold[256 + tid + k * CPB];
        }
        p.pdd[((long)blockIdx.x * 2 + 0) * D + sd] = x;
        p.pdd[((long)blockIdx.x * 2 + 1) * D + sd] = y;
    }
}

__host__ __device__ inline int blocks_of(long n, int per) { return (int)((n + per - 1) / per); }

// blocks [0, na): da over the slots; [na, na + nd): dd and d(dt_bias); the rest, up to SUM_BLOCKS: db and dc over the
// channel tiles of a group, an element a thread and, where there are more, others behind
constexpr long SUM_BLOCKS = 1 << 22;
template <int DT> __global__ __launch_bounds__(256) void k_sums(ScanParams p) {
    const long D = p.D, N = p.N;
    const int na = blocks_of(N * D, SUM_COLS), nd = blocks_of(2 * D, SUM_COLS);
    int blk = blockIdx.x;
    if (blk < na) {
        column_sums(p.agg, N * D, p.slots, (long)blk * SUM_COLS, N * D, [&](long col, float s) { p.da[col] = s; });
        return;
    }
    blk -= na;
    if (blk < nd) {
        column_sums(p.pdd, 2 * D, p.slots, (long)blk * SUM_COLS, 2 * D, [&](long col, float s) {
            if (col < D) {
                if (p.dd) p.dd[col] = s;
            } else if (p.dbias) p.dbias[col - D] = s;
        });
        return;
    }
    blk -= nd;
    const long per = p.tokens * p.G * 2 * N;
    for (long e = (long)blk * 256 + threadIdx.x; e < per; e += SUM_BLOCKS * 256) {
        float s = 0.f;
        for (int k = 0; k < p.tpg; ++k) s += p.pbc[k * per + e];
        const long n = e % N, m = e / N % 2, row = e / (2 * N);   // row: token and group
        static_cast<raw_t<DT>*>(m ? p.dc : p.db)[row * N + n] = to_raw<DT>(s);
    }
}

// ---------------------------------------------------------------- host side
struct BwdPlan {
    Seqs q;
    int tpg;
    long slots, tokens;
    bool chunked;
    bool walked;                    // chunks of more than a unit, or more than one chunk
    int units, seq_units;           // as in ScanParams
    size_t off_gagg, off_sdt, off_pdd, off_uh, off_udt, off_pbc, bytes;
};

// f<NS, Q>() for the smallest pair that holds N states
template <class F> auto with_shape(int64_t N, F f) {
    if (N <= 8) return f.template operator()<4, 2>();
    if (N <= 16) return f.template operator()<4, 4>();
    if (N <= 32) return f.template operator()<8, 4>();
    if (N <= 64) return f.template operator()<8, 8>();
    return f.template operator()<8, 16>();
}
struct Sizes {
    int cpb;
};
struct GetSizes {
    template <int NS, int Q> Sizes operator()() { return Sizes{Shape<NS, Q>::CPB}; }
};

// Chunks of 128 tokens, halved while fewer than 1024 blocks would walk, down to 16: longer ones leave fewer
// aggregates and partial sums, but too few blocks to even out the GPU's load (4 x 4096 x 1024: 367 us at 128, 390 at
// 64, 429 at 256).
constexpr int LONGEST = 128;
mimo_status plan_bwd(const mamba_scan_bwd_args* a, BwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_scan(a->n, a->S, a->D, a->G, a->N, a->dtype);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    const Sizes z = with_shape(a->N, GetSizes{});
    pl->tpg = (int)((a->D / a->G + z.cpb - 1) / z.cpb);
    pl->tokens = packed ? a->S : a->n * a->S;
    int CH = LONGEST;
    while (CH > UNIT && pl->tokens / CH * a->G * pl->tpg < 1024) CH /= 2;
    if (a->S <= LONGEST && a->S <= 2 * CH) CH = LONGEST;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    pl->chunked = a->S > CH;
    pl->walked = a->S > UNIT;
    const long per = pl->tokens * a->G * 2 * a->N;
    const int threads = walk_threads(a->N) > 256 ? walk_threads(a->N) : 256;   // the sums' blocks are at most 2^24
    if (pl->slots > 0x7fffffffL || !grid_fits(pl->slots, threads) || a->G * pl->tpg > 65535) return unsupported("too many tokens or channels");
    pl->units = CH / UNIT - 1;
    pl->seq_units = (int)((a->S + UNIT - 1) / UNIT) - pl->q.nc;
    const size_t agg = up256((size_t)pl->slots * a->N * a->D * sizeof(float));
    pl->off_gagg = agg;
    pl->off_sdt = pl->off_gagg + (pl->chunked ? agg : 0);
    pl->off_pdd = pl->off_sdt + (pl->chunked ? up256((size_t)pl->slots * a->D * sizeof(float)) : 0);
    pl->off_uh = pl->off_pdd + up256((size_t)pl->slots * 2 * a->D * sizeof(float));
    const size_t units = !pl->walked || pl->units == 0 ? 0 : (size_t)(packed ? a->S * pl->units / CH + a->n : a->n * pl->seq_units) * a->D;
    pl->off_udt = pl->off_uh + up256(units * a->N * sizeof(float));
    pl->off_pbc = pl->off_udt + up256(units * sizeof(float));
    pl->bytes = pl->off_pbc + up256((size_t)pl->tpg * per * sizeof(float));
    return MIMO_OK;
}

template <int DT> struct Run {
    const ScanParams& p;
    hipStream_t st;
    template <int NS, int Q> mimo_status operator()() {
        mimo_status s;
        if (p.uh) {
            ScanParams w = p;      // the walk's channel tiles are 64 wide
            w.tpg = (p.Dg + 63) / 64;
            if ((s = launch_walk<DT, AGG2>(w, st)) != MIMO_OK) return s;
        }
        if (p.chunked) {
            if ((s = launch_carry<true>(p, st)) != MIMO_OK) return s;
        }
        const auto grad = p.N == NS * Q ? &k_scan_bwd<DT, NS, Q, 0> : p.N % NS == 0 ? &k_scan_bwd<DT, NS, Q, 1> : &k_scan_bwd<DT, NS, Q, 2>;
        s = launch(grad, dim3((unsigned)p.slots, p.G * p.tpg), 256, Shape<NS, Q>::lds, st, p);
        if (s != MIMO_OK) return s;
        const long per = p.tokens * p.G * 2 * p.N;
        const long rest = (per + 255) / 256 < SUM_BLOCKS ? (per + 255) / 256 : SUM_BLOCKS;
        const long blocks = (long)blocks_of((long)p.N * p.D, SUM_COLS) + blocks_of(2L * p.D, SUM_COLS) + rest;
        return launch(&k_sums<DT>, dim3((unsigned)blocks), 256, 0, st, p);
    }
};

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_scan_bwd_workspace_size(const mamba_scan_bwd_args* a, size_t* bytes) {
    BwdPlan pl;
    const mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = pl.bytes;
    return MIMO_OK;
}

mimo_status mamba_scan_bwd(const mamba_scan_bwd_args* a, void* stream) {
    BwdPlan pl;
    mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (!a->dout.data || !a->u.data || !a->dt.data || !a->a || !a->b.data || !a->c.data)
        return bad("dout, u, dt, a, b and c must not be NULL");
    if (!a->du || !a->ddt || !a->da || !a->db || !a->dc) return bad("du, ddt, da, db and dc must not be NULL");
    if ((a->z.data == nullptr) != (a->dz == nullptr)) return bad("dz must be given exactly when z is given");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, pl.bytes)) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    ScanParams p{};
    p.q = pl.q;
    p.D = (int)a->D, p.G = (int)a->G, p.N = (int)a->N, p.Dg = p.D / p.G, p.tpg = pl.tpg;
    p.softplus = a->dt_softplus, p.chunked = pl.chunked, p.has_z = a->z.data != nullptr;
    p.u = rows_of(a->u, packed), p.dt = rows_of(a->dt, packed), p.b = rows_of(a->b, packed), p.c = rows_of(a->c, packed);
    p.z = rows_of(a->z, packed), p.dout = rows_of(a->dout, packed);
    p.a = a->a, p.d = a->d, p.bias = a->dt_bias, p.init = a->initial_state, p.dstate = a->dstate;
    p.du = a->du, p.ddt = a->ddt, p.db = a->db, p.dc = a->dc, p.dz = a->dz;
    p.da = a->da, p.dd = a->dd, p.dbias = a->ddt_bias, p.dinit = a->dinitial_state;
    char* ws = static_cast<char*>(a->workspace);
    p.agg = reinterpret_cast<float*>(ws);
    p.gagg = reinterpret_cast<float*>(ws + pl.off_gagg);
    p.sdt = reinterpret_cast<float*>(ws + pl.off_sdt);
    p.pdd = reinterpret_cast<float*>(ws + pl.off_pdd);
    p.pbc = reinterpret_cast<float*>(ws + pl.off_pbc);
    p.uh = pl.walked ? reinterpret_cast<float*>(ws + pl.off_uh) : nullptr;
    p.udt = reinterpret_cast<float*>(ws + pl.off_udt);
    p.units = pl.units, p.seq_units = pl.seq_units;
    p.slots = pl.slots, p.tokens = pl.tokens;
    p.vec = p.N % 4 == 0;
    for (const void* x : {(const void*)p.a, (const void*)p.init, (const void*)p.dstate, (const void*)p.dinit}) p.vec = p.vec && aligned(x, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == BF16) return with_shape(a->N, Run<BF16>{p, st});
    if (a->dtype == F16) return with_shape(a->N, Run<F16>{p, st});
    return with_shape(a->N, Run<F32>{p, st});
}

}  // extern "C"
