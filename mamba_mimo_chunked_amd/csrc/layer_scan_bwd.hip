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
// pair. A block walks its chunk forward in sub-tiles of ST tokens and keeps the state in front of each in
// LDS, then takes the sub-tiles from the last to the first: forward once more with the states and
// decays of its ST tokens in registers (2 * NS * ST = 128), then backward through them. So each
// exponential is computed three times in all (aggregate, walk, sub-tile), and no state but the chunks'
// goes to memory.
#include "layer_scan.hpp"

namespace mimo {
namespace layer {
namespace {

// channels of a block, LDS floats: staging of dt, dt u, dy, three sums; b, c; fold results of four
// waves; checkpoints
template <int NS, int Q> struct Shape {
    static constexpr int ST = 64 / NS, NP = NS * Q, CPW = 64 / Q, CPB = 4 * CPW;
    static constexpr int ROWS = ST * CPB, BC = ST * NP, FOLD = 4 * 2 * BC;
    // tokens of the longest chunk: two blocks fit the 160 KB of a CU
    static constexpr int CK = NS == 4 ? (Q == 2 ? 64 : 128) : Q == 16 ? 32 : 48;
    static constexpr int CKPT = CK / ST * 256 * NS;
    static constexpr size_t lds = sizeof(float) * (6 * ROWS + 2 * BC + FOLD + CKPT);
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

template <int DT, int NS, int Q> __global__ __launch_bounds__(256, 2) void k_scan_bwd(ScanParams p) {
    typedef raw_t<DT> raw;
    typedef Shape<NS, Q> H;
    constexpr int ST = H::ST, NP = H::NP, CPB = H::CPB, NT = (ST * CPB + 255) / 256, NB = (H::BC + 255) / 256;
    constexpr int LEFT = H::CPW == 4 ? NS / 4 : 1;    // values a lane keeps of a fold
    static_assert(CPB <= 256 && 256 % CPB == 0 && H::FOLD >= 512, "staging");
    extern __shared__ __attribute__((aligned(16))) float lds[];
    float *s_dt = lds, *s_du = s_dt + H::ROWS, *s_dy = s_du + H::ROWS;          // [ST][CPB]
    float *s_y = s_dy + H::ROWS, *s_gb = s_y + H::ROWS, *s_xa = s_gb + H::ROWS; // [ST][CPB]
    float *s_b = s_xa + H::ROWS, *s_c = s_b + H::BC;                            // [ST][NP]
    float *s_fold = s_c + H::BC;                                                // [4][2][ST][NP]
    float *s_ck = s_fold + H::FOLD;                                             // [sub-tile][NS/4][256][4]
    const Place pl = place(p.q, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, q = lane % Q, cb = w * H::CPW + lane / Q;
    const Tile tile = tile_of<CPB>(p, blockIdx.y);
    const long D = p.D, N = p.N, G = p.G;
    if (!pl.ok || pl.i == p.q.n) {  // no tokens of a sequence: nothing for the parameters' gradients
        for (int e = tid; e < CPB * p.N; e += 256)
            if (e % CPB < tile.left) p.agg[((long)blockIdx.x * N + e / CPB) * D + tile.c0 + e % CPB] = 0.f;
        for (int e = tid; e < CPB * 2; e += 256)
            if (e % CPB < tile.left) p.pdd[((long)blockIdx.x * 2 + e / CPB) * D + tile.c0 + e % CPB] = 0.f;
        if (!pl.ok) return;
    }
    const long flat = flat_row(p.q, pl);
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    const int in_group = blockIdx.y - tile.g * p.tpg;
    // partial db, dc of this channel tile: [token][group][2][N]
    float* pbc = p.pbc + (((long)in_group * p.tokens + flat) * G + tile.g) * 2 * N;
    // staging: thread -> channel sc of the tile, tokens st + k * (256 / CPB)
    const int sc = tid % CPB, st = tid / CPB;
    constexpr int SD = 256 / CPB;
    const bool sact = sc < tile.left;
    const int sd = tile.c0 + (sact ? sc : 0);
    raw *du = static_cast<raw*>(p.du) + flat * D + sd, *ddt = static_cast<raw*>(p.ddt) + flat * D + sd;
    raw* dz = p.has_z ? static_cast<raw*>(p.dz) + flat * D + sd : nullptr;
    if (pl.i == p.q.n) {            // behind the last sequence
        const raw zero = to_raw<DT>(0.f);
        for (int t = t0 + st; t < t1; t += SD)
            if (sact) {
                du[t * D] = zero;
                ddt[t * D] = zero;
                if (dz) dz[t * D] = zero;
            }
        for (int e = tid; e < (t1 - t0) * 2 * p.N; e += 256) pbc[(long)(t0 + e / (2 * p.N)) * G * 2 * N + e % (2 * p.N)] = 0.f;
        return;
    }
    const raw *gu = at<DT>(p.u, pl) + sd, *gdt = at<DT>(p.dt, pl) + sd, *gdo = at<DT>(p.dout, pl) + sd;
    const raw *gz = p.has_z ? at<DT>(p.z, pl) + sd : nullptr;
    const raw *gb = at<DT>(p.b, pl) + tile.g * p.N, *gc = at<DT>(p.c, pl) + tile.g * p.N;
    const float bias = p.bias ? p.bias[sd] : 0.f, skip = p.d ? p.d[sd] : 0.f;

    const bool act = cb < tile.left;
    const int d = tile.c0 + (act ? cb : 0);
    float a[NS], h[NS], g[NS], da[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int n = q * NS + k;
        const bool on = act && n < p.N;
        a[k] = on ? p.a[d * N + n] * LOG2E : 0.f;
        const long own = ((long)pl.i * D + d) * N + n, cut = ((long)blockIdx.x * N + n) * D + d;
        h[k] = !on ? 0.f : p.chunked ? p.agg[cut] : p.init ? p.init[own] : 0.f;
        g[k] = !on ? 0.f : p.chunked ? p.gagg[cut] : p.dstate ? p.dstate[own] : 0.f;
        da[k] = 0.f;
    }
    const int nsub = (t1 - t0 + ST - 1) / ST;

    raw r_dt[NT], r_u[NT], r_z[NT], r_g[NT], r_b[NB], r_c[NB];
    auto fetch = [&](int tt, bool all) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const long row = min(tt + st + k * SD, t1 - 1);
            if (NT * SD > ST && st + k * SD >= ST) continue;
            r_dt[k] = gdt[row * p.dt.ts];
            r_u[k] = gu[row * p.u.ts];
            if (all) {
                r_g[k] = gdo[row * p.dout.ts];
                if (gz) r_z[k] = gz[row * p.z.ts];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = tid + k * 256, n = e % NP;
            const long row = min(tt + e / NP, t1 - 1);
            const bool on = e < H::BC && n < p.N;
            r_b[k] = on ? gb[row * p.b.ts + n] : raw(0);
            if (all) r_c[k] = on ? gc[row * p.c.ts + n] : raw(0);
        }
    };
    float f_u[NT], f_z[NT], f_g[NT], f_x[NT], f_dt[NT], f_dy[NT];
    // a tile's values to LDS; tokens past the chunk and lanes past the group take no step (dt = 0)
    auto stage = [&](int tt, bool all) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const int t = st + k * SD;
            if (NT * SD > ST && t >= ST) continue;
            const bool on = sact && tt + t < t1;
            f_x[k] = to_f<DT>(r_dt[k]) + bias;
            f_u[k] = to_f<DT>(r_u[k]);
            f_dt[k] = on ? (p.softplus ? softplus(f_x[k]) : f_x[k]) : 0.f;
            s_dt[t * CPB + sc] = f_dt[k];
            s_du[t * CPB + sc] = on ? f_dt[k] * f_u[k] : 0.f;
            if (all) {
                f_g[k] = to_f<DT>(r_g[k]);
                f_z[k] = gz ? to_f<DT>(r_z[k]) : 0.f;
                f_dy[k] = on ? (gz ? f_g[k] * f_z[k] * sigmoid(f_z[k]) : f_g[k]) : 0.f;
                s_dy[t * CPB + sc] = f_dy[k];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = tid + k * 256;
            if (e < H::BC) {
                const bool on = tt + e / NP < t1;
                s_b[e] = on ? to_f<DT>(r_b[k]) : 0.f;
                if (all) s_c[e] = on ? to_f<DT>(r_c[k]) : 0.f;
            }
        }
    };
    auto checkpoint = [&](int s) {
#pragma unroll
        for (int k = 0; k < NS; k += 4)
            *reinterpret_cast<float4*>(s_ck + ((s * (NS / 4) + k / 4) * 256 + tid) * 4) = make_float4(h[k], h[k + 1], h[k + 2], h[k + 3]);
    };

    // forward: the state in front of every sub-tile
    if (nsub > 1) fetch(t0, false);
    for (int s = 0; s < nsub; ++s) {
        checkpoint(s);
        if (s + 1 == nsub) break;
        const int tt = t0 + s * ST;
        stage(tt, false);
        __syncthreads();
        if (s + 2 < nsub) fetch(tt + ST, false);
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb];
#pragma unroll
            for (int k = 0; k < NS; ++k) h[k] = __builtin_fmaf(exp2_hw(v * a[k]), h[k], vu * s_b[t * NP + q * NS + k]);
        }
        __syncthreads();
    }

    // backward
    float acc_d = 0.f, acc_bias = 0.f;
    if (nsub > 0) fetch(t0 + (nsub - 1) * ST, true);
    for (int s = nsub - 1; s >= 0; --s) {
        const int tt = t0 + s * ST;
        stage(tt, true);
        __syncthreads();
        if (s > 0) fetch(tt - ST, true);
        float hp[ST][NS], e[ST][NS];   // the state in front of each token, its decay
#pragma unroll
        for (int k = 0; k < NS; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(s_ck + ((s * (NS / 4) + k / 4) * 256 + tid) * 4);
            h[k] = x.x, h[k + 1] = x.y, h[k + 2] = x.z, h[k + 3] = x.w;
        }
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb];
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                hp[t][k] = h[k];
                e[t][k] = exp2_hw(v * a[k]);
                h[k] = __builtin_fmaf(e[t][k], h[k], vu * s_b[t * NP + q * NS + k]);
            }
        }
#pragma unroll
        for (int t = ST - 1; t >= 0; --t) {
            const float v = s_dt[t * CPB + cb], vu = s_du[t * CPB + cb], dy = s_dy[t * CPB + cb];
            float y = 0.f, sgb = 0.f, sxa = 0.f, vb[NS], vc[NS];
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const float b = s_b[t * NP + q * NS + k], c = s_c[t * NP + q * NS + k];
                const float ht = t == ST - 1 ? h[k] : hp[t + 1 < ST ? t + 1 : 0][k];
                g[k] = __builtin_fmaf(c, dy, g[k]);
                y = __builtin_fmaf(c, ht, y);
                sgb = __builtin_fmaf(g[k], b, sgb);
                vc[k] = dy * ht;
                vb[k] = g[k] * vu;
                g[k] *= e[t][k];
                const float x = g[k] * hp[t][k];
                sxa = __builtin_fmaf(x, a[k], sxa);
                da[k] = __builtin_fmaf(x, v, da[k]);
            }
            y = sum_lanes<Q>(y);
            sgb = sum_lanes<Q>(sgb);
            sxa = sum_lanes<Q>(sxa);
            if (q == 0) {
                s_y[t * CPB + cb] = y;
                s_gb[t * CPB + cb] = sgb;
                s_xa[t * CPB + cb] = sxa;
            }
            fold_channels<NS, Q>(vb, lane & 8);
            fold_channels<NS, Q>(vc, lane & 8);
            // the state a lane's first kept value belongs to
            const int own = q * NS + ((lane >> 5) & 1) * (NS / 2) + ((lane >> 4) & 1) * (NS / 4) +
                            (NS == 8 && H::CPW >= 8 ? (lane >> 3) & 1 : 0);
#pragma unroll
            for (int k = 0; k < LEFT; ++k) {
                s_fold[((w * 2 + 0) * ST + t) * NP + own + k] = vb[k];
                s_fold[((w * 2 + 1) * ST + t) * NP + own + k] = vc[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const int t = st + k * SD;
            if (sact && t < ST && tt + t < t1) {
                const float y = s_y[t * CPB + sc], sgb = s_gb[t * CPB + sc], sxa = s_xa[t * CPB + sc] * LN2;
                float x = __builtin_fmaf(f_u[k], sgb, sxa);
                if (p.softplus) x *= sigmoid(f_x[k]);
                const long row = (long)(tt + t) * D;
                du[row] = to_raw<DT>(__builtin_fmaf(f_dt[k], sgb, skip * f_dy[k]));
                ddt[row] = to_raw<DT>(x);
                if (dz) dz[row] = to_raw<DT>(f_g[k] * __builtin_fmaf(skip, f_u[k], y) * silu_slope(f_z[k], sigmoid(f_z[k])));
                acc_d = __builtin_fmaf(f_dy[k], f_u[k], acc_d);
                acc_bias += x;
            }
        }
        for (int i = tid; i < 2 * H::BC; i += 256) {
            const int n = i % NP, m = (i / NP) & 1, t = i / (2 * NP);
            if (n < p.N && tt + t < t1) {
                const float* f = s_fold + (m * ST + t) * NP + n;
                pbc[(long)(tt + t) * G * 2 * N + m * N + n] = (f[0] + f[2 * H::BC]) + (f[4 * H::BC] + f[6 * H::BC]);
            }
        }
        __syncthreads();
    }

    // this chunk's share of da, dd, d(dt_bias); the gradient of the initial state where nothing was cut
    if (act) {
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            const int n = q * NS + k;
            if (n < p.N) {
                p.agg[((long)blockIdx.x * N + n) * D + d] = da[k];
                if (!p.chunked && p.dinit) p.dinit[((long)pl.i * D + d) * N + n] = g[k];
            }
        }
    }
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

// blocks [0, na): da over the slots; [na, na + nd): dd and d(dt_bias); the rest: db and dc over the
// channel tiles of a group
template <int DT> __global__ __launch_bounds__(256) void k_sums(ScanParams p) {
    const long D = p.D, N = p.N;
    const int na = blocks_of(N * D, SUM_COLS), nd = blocks_of(2 * D, SUM_COLS);
    int blk = blockIdx.x;
    if (blk < na) {
        column_sums(p.agg, N * D, p.slots, (long)blk * SUM_COLS, N * D, [&](long col, float s) { p.da[(col % D) * N + col / D] = s; });
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
    const long per = p.tokens * p.G * 2 * N, e = (long)blk * 256 + threadIdx.x;
    if (e >= per) return;
    float s = 0.f;
    for (int k = 0; k < p.tpg; ++k) s += p.pbc[k * per + e];
    const long n = e % N, m = e / N % 2, row = e / (2 * N);   // row: token and group
    static_cast<raw_t<DT>*>(m ? p.dc : p.db)[row * N + n] = to_raw<DT>(s);
}

// ---------------------------------------------------------------- host side
struct BwdPlan {
    Seqs q;
    int tpg;
    long slots, tokens;
    bool chunked;
    size_t off_gagg, off_sdt, off_pdd, off_pbc, bytes;
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
    int cpb, st, ck;
};
struct GetSizes {
    template <int NS, int Q> Sizes operator()() { return Sizes{Shape<NS, Q>::CPB, Shape<NS, Q>::ST, Shape<NS, Q>::CK}; }
};

// The longest chunks the checkpoints allow (fewer aggregates and partial sums), halved while fewer than
// 1024 blocks would walk, down to 16 tokens.
mimo_status plan_bwd(const mamba_scan_bwd_args* a, BwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_scan(a->n, a->S, a->D, a->G, a->N, a->dtype);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    const Sizes z = with_shape(a->N, GetSizes{});
    pl->tpg = (int)((a->D / a->G + z.cpb - 1) / z.cpb);
    pl->tokens = packed ? a->S : a->n * a->S;
    int CH = z.ck;
    while (CH > 16 && pl->tokens / CH * a->G * pl->tpg < 1024) CH = (CH / 2 + z.st - 1) / z.st * z.st;
    if (a->S <= z.ck && a->S <= 2 * CH) CH = z.ck;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    pl->chunked = a->S > CH;
    const long per = pl->tokens * a->G * 2 * a->N;
    if (pl->slots > 0x7fffffffL || per / 256 > 0x70000000L || a->G * pl->tpg > 65535) return unsupported("too many tokens or channels");
    const size_t agg = up256((size_t)pl->slots * a->N * a->D * sizeof(float));
    pl->off_gagg = agg;
    pl->off_sdt = pl->off_gagg + (pl->chunked ? agg : 0);
    pl->off_pdd = pl->off_sdt + up256((size_t)pl->slots * a->D * sizeof(float));
    pl->off_pbc = pl->off_pdd + up256((size_t)pl->slots * 2 * a->D * sizeof(float));
    pl->bytes = pl->off_pbc + up256((size_t)pl->tpg * per * sizeof(float));
    return MIMO_OK;
}

template <int DT> struct Run {
    const ScanParams& p;
    hipStream_t st;
    template <int NS, int Q> mimo_status operator()() {
        mimo_status s;
        if (p.chunked) {
            ScanParams w = p;      // the walk's channel tiles are 64 wide
            w.tpg = (p.Dg + 63) / 64;
            if ((s = launch_walk<DT, AGG2>(w, st)) != MIMO_OK) return s;
            if ((s = launch(&k_carry<true>, dim3((p.D + 255) / 256, 2 * p.N, p.q.n), 256, 0, st, p)) != MIMO_OK) return s;
        }
        s = launch(&k_scan_bwd<DT, NS, Q>, dim3((unsigned)p.slots, p.G * p.tpg), 256, Shape<NS, Q>::lds, st, p);
        if (s != MIMO_OK) return s;
        const long per = p.tokens * p.G * 2 * p.N;
        const long blocks = (long)blocks_of((long)p.N * p.D, SUM_COLS) + blocks_of(2L * p.D, SUM_COLS) + (per + 255) / 256;
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
    p.slots = pl.slots, p.tokens = pl.tokens;
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == BF16) return with_shape(a->N, Run<BF16>{p, st});
    if (a->dtype == F16) return with_shape(a->N, Run<F16>{p, st});
    return with_shape(a->N, Run<F32>{p, st});
}

}  // extern "C"
