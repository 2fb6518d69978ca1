// Gated linear recurrence, backward pass (formulas, gates, carry: layer_recur.hpp). Nothing is kept from the forward pass.
// A block takes one chunk of WAVES * TT tokens; k_recur_agg leaves each chunk's joined step, forward and for the adjoint, the
// carry turns them into the state and the adjoint that enter, and k_recur_bwd walks its tokens forward for the states and
// back for the adjoints and the gradients. Parameters' gradients leave one partial row a chunk, added up in order.
#include <initializer_list>

#include "layer_recur.hpp"

namespace mimo {
namespace layer {
namespace {

constexpr int WAVES = 8, TT = 8, CHUNK = WAVES * TT;

// a wave's tokens: inputs as they lie in memory, steps, and the gradient that meets the state
template <int DT, int VC> struct Tokens {
    RowsOf<DT, VC, TT> x, r, i, z, g;
    float a[TT][VC], b[TT][VC], dh[TT][VC];

    __device__ __forceinline__ void fetch(const RecurParams& p, const Place& pl, int tw, int last, unsigned d) {
        x.fetch(at<DT>(p.x, pl), p.x.ts, tw, last, d);
        r.fetch(at<DT>(p.r, pl), p.r.ts, tw, last, d);
        i.fetch(at<DT>(p.i, pl), p.i.ts, tw, last, d);
        g.fetch(at<DT>(p.dout, pl), p.dout.ts, tw, last, d);
        if (p.has_z) z.fetch(at<DT>(p.z, pl), p.z.ts, tw, last, d);
    }
    __device__ __forceinline__ void steps(const RecurParams& p, const Gates<VC>& gates, int tw, int t1) {
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            float fx[VC], fr[VC], fi[VC], fz[VC];
            unpack<DT, VC>(x.t[k], fx);
            unpack<DT, VC>(r.t[k], fr);
            unpack<DT, VC>(i.t[k], fi);
            unpack<DT, VC>(g.t[k], dh[k]);
            if (p.has_z) unpack<DT, VC>(z.t[k], fz);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                float e2;
                keep_and_enter(gates.speed[v] * sigmoid(fr[v] + gates.rb[v]), a[k][v], e2);
                b[k][v] = root(e2) * (sigmoid(fi[v] + gates.ib[v]) * fx[v]);
                if (p.has_z) dh[k][v] *= fz[v] * sigmoid(fz[v]);
            }
        }
        if (tw + TT > t1) {         // tokens behind the chunk change nothing
#pragma unroll
            for (int k = 0; k < TT; ++k)
                if (tw + k >= t1) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) a[k][v] = 1.f, b[k][v] = dh[k][v] = 0.f;
                }
        }
    }
    // the joined step: last state from zero, product of a, adjoint that leaves to the left from zero
    __device__ __forceinline__ void fold(float (&h)[VC], float (&q)[VC], float (&c)[VC]) const {
#pragma unroll
        for (int v = 0; v < VC; ++v) h[v] = c[v] = 0.f, q[v] = 1.f;
#pragma unroll
        for (int k = 0; k < TT; ++k)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                h[v] = __builtin_fmaf(a[k][v], h[v], b[k][v]);
                q[v] *= a[k][v];
                c[v] = a[TT - 1 - k][v] * (dh[TT - 1 - k][v] + c[v]);
            }
    }
};

template <int VC> struct Join {
    float h[WAVES][64 * VC], q[WAVES][64 * VC], c[WAVES][64 * VC];
    __device__ __forceinline__ void put(int w, int lane, const float (&fh)[VC], const float (&fq)[VC], const float (&fc)[VC]) {
#pragma unroll
        for (int v = 0; v < VC; ++v) h[w][lane * VC + v] = fh[v], q[w][lane * VC + v] = fq[v], c[w][lane * VC + v] = fc[v];
    }
};

template <int DT, int VC> __global__ __launch_bounds__(64 * WAVES) void k_recur_agg(RecurParams p) {
    __shared__ Join<VC> s;
    const unsigned slot = blockIdx.x / p.tiles, tile = blockIdx.x - slot * p.tiles;
    const Place pl = place(p.q, slot);
    if (!pl.ok || pl.i == p.q.n) return;
    const int t0 = pl.j * CHUNK, t1 = min(t0 + CHUNK, pl.len);
    if (t0 >= t1) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tw = t0 + w * TT;
    const unsigned vec = tile * 64 + lane;
    const bool act = vec < (unsigned)p.nvec;
    const unsigned d = act ? vec * VC : 0;
    Tokens<DT, VC> k;
    k.fetch(p, pl, tw, t1 - 1, d);
    const Gates<VC> gates(p, d);
    k.steps(p, gates, tw, t1);
    float h[VC], q[VC], c[VC];
    k.fold(h, q, c);
    s.put(w, lane, h, q, c);
    __syncthreads();
    if (w != 0 || !act) return;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        float hh = 0.f, qq = 1.f, cc = 0.f;
#pragma unroll
        for (int o = 0; o < WAVES; ++o) {
            hh = __builtin_fmaf(s.q[o][lane * VC + v], hh, s.h[o][lane * VC + v]);
            qq *= s.q[o][lane * VC + v];
            cc = __builtin_fmaf(s.q[WAVES - 1 - o][lane * VC + v], cc, s.c[WAVES - 1 - o][lane * VC + v]);
        }
        const long at = (long)slot * p.D + d + v;
        p.agg_h[at] = hh, p.agg_p[at] = qq, p.agg_g[at] = cc;
    }
}

template <int DT, int VC> __global__ __launch_bounds__(64 * WAVES) void k_recur_bwd(RecurParams p) {
    typedef raw_t<DT> raw;
    __shared__ Join<VC> s;
    const unsigned slot = blockIdx.x / p.tiles, tile = blockIdx.x - slot * p.tiles;
    const Place pl = place(p.q, slot);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned vec = tile * 64 + lane;
    const bool act = vec < (unsigned)p.nvec;
    const unsigned d = act ? vec * VC : 0;
    const long D = p.D;
    const int t0 = pl.j * CHUNK, t1 = pl.ok ? min(t0 + CHUNK, pl.len) : t0, tw = t0 + w * TT;
    const long flat = recur_row(p.q, pl) * D + d;
    raw *dx = static_cast<raw*>(p.dx) + flat, *dr = static_cast<raw*>(p.dr) + flat, *di = static_cast<raw*>(p.di) + flat;
    raw* dz = p.has_z ? static_cast<raw*>(p.dz) + flat : nullptr;
    float* part = p.part + (long)slot * 3 * D + d;
    const bool tail = pl.i == p.q.n;
    if (t0 >= t1 || tail) {         // no tokens, or those behind the last sequence
        const float zero[VC] = {};
        if (tail && act)
            for (int t = t0 + w; t < t1; t += WAVES) {
                store<DT, VC>(dx + t * D, zero);
                store<DT, VC>(dr + t * D, zero);
                store<DT, VC>(di + t * D, zero);
                if (dz) store<DT, VC>(dz + t * D, zero);
            }
        if (w == 0 && act) {
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                part[v] = part[D + v] = part[2 * D + v] = 0.f;
                if (!p.chunked && p.dinit && pl.ok && !tail) p.dinit[pl.i * D + d + v] = p.dstate ? p.dstate[pl.i * D + d + v] : 0.f;
            }
        }
        return;
    }
    Tokens<DT, VC> k;
    k.fetch(p, pl, tw, t1 - 1, d);
    const Gates<VC> gates(p, d);
    float h[VC], c[VC];
    const float* from = p.chunked ? p.agg_h + slot * D : p.init ? p.init + pl.i * D : nullptr;
    const float* late = p.chunked ? p.agg_g + slot * D : p.dstate ? p.dstate + pl.i * D : nullptr;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        h[v] = from ? from[d + v] : 0.f;
        c[v] = late ? late[d + v] : 0.f;
    }
    k.steps(p, gates, tw, t1);
    {
        float fh[VC], fq[VC], fc[VC];
        k.fold(fh, fq, fc);
        s.put(w, lane, fh, fq, fc);
    }
    __syncthreads();
    // the state that enters this wave's tokens, and the adjoint
    for (int o = 0; o < w; ++o)
#pragma unroll
        for (int v = 0; v < VC; ++v) h[v] = __builtin_fmaf(s.q[o][lane * VC + v], h[v], s.h[o][lane * VC + v]);
    for (int o = WAVES - 1; o > w; --o)
#pragma unroll
        for (int v = 0; v < VC; ++v) c[v] = __builtin_fmaf(s.q[o][lane * VC + v], c[v], s.c[o][lane * VC + v]);
    float sum[3][VC] = {};
    // b becomes the state in front of a token
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float b = k.b[t][v];
            k.b[t][v] = h[v];
            h[v] = __builtin_fmaf(k.a[t][v], h[v], b);
        }
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
        float fx[VC], fr[VC], fi[VC], fz[VC], fg[VC], ox[VC], orr[VC], oi[VC], oz[VC];
        unpack<DT, VC>(k.x.t[t], fx);
        unpack<DT, VC>(k.r.t[t], fr);
        unpack<DT, VC>(k.i.t[t], fi);
        unpack<DT, VC>(k.g.t[t], fg);
        if (dz) unpack<DT, VC>(k.z.t[t], fz);
        const bool real = tw + t < t1;
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float sr = sigmoid(fr[v] + gates.rb[v]), si = sigmoid(fi[v] + gates.ib[v]), l2 = gates.speed[v] * sr;
            float a, e2;
            keep_and_enter(l2, a, e2);
            const float inv = e2 > 0.f ? __builtin_amdgcn_rsqf(e2) : e2 - e2, e = root(e2);     // 0 where nothing enters; NaN stays
            const float g = k.dh[t][v] + c[v], hp = k.b[t][v], u = si * fx[v], l = l2 * LN2;
            const float W = a * g * (l * hp - (l * inv) * (a * u));
            const float du = g * e;
            c[v] = k.a[t][v] * g;
            ox[v] = du * si;
            oi[v] = du * u * (1.f - si);
            orr[v] = (1.f - sr) * W;
            if (dz) {
                const float now = __builtin_fmaf(a, hp, e * u), sg = sigmoid(fz[v]);
                oz[v] = fg[v] * now * silu_slope(fz[v], sg);
            }
            if (real) {
                sum[0][v] += W;
                sum[1][v] += orr[v];
                sum[2][v] += oi[v];
            }
        }
        if (real && act) {
            const long at = (tw + t) * D;
            store<DT, VC>(dx + at, ox);
            store<DT, VC>(dr + at, orr);
            store<DT, VC>(di + at, oi);
            if (dz) store<DT, VC>(dz + at, oz);
        }
    }
    if (!p.chunked && p.dinit && w == 0 && act) {
#pragma unroll
        for (int v = 0; v < VC; ++v) p.dinit[pl.i * D + d + v] = c[v];
    }
    __syncthreads();
    s.put(w, lane, sum[0], sum[1], sum[2]);
    __syncthreads();
    if (w == 0 && act) {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            float x = 0.f, y = 0.f, zz = 0.f;
#pragma unroll
            for (int o = 0; o < WAVES; ++o) x += s.h[o][lane * VC + v], y += s.q[o][lane * VC + v], zz += s.c[o][lane * VC + v];
            part[v] = x, part[D + v] = y, part[2 * D + v] = zz;
        }
    }
}

__global__ __launch_bounds__(256) void k_recur_sums(RecurParams p) {
    const long D = p.D;
    column_sums(p.part, 3 * D, p.slots, (long)blockIdx.x * SUM_COLS, 3 * D, [&](long col, float s) {
        if (col >= 2 * D) {
            if (p.dib) p.dib[col - 2 * D] = s;
        } else if (col >= D) {
            if (p.drb) p.drb[col - D] = s;
        } else {
            // sigmoid / softplus, one where both vanish
            const float x = p.decay[col], sp = softplus(x);
            p.ddecay[col] = sp > 0.f ? s * (sigmoid(x) / sp) : s;
        }
    });
}

struct BwdPlan {
    Seqs q;
    int VC;
    unsigned tiles;
    long slots;
    bool chunked;
    size_t agg, part, bytes;
};

mimo_status plan_bwd(const mamba_recur_bwd_args* a, BwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_recur(a->n, a->S, a->D, a->dtype, a->rate);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->VC = channels_of(a->D, a->dtype, packed, {&a->dout, &a->x, &a->r, &a->i, &a->z}, {a->dx, a->dr, a->di, a->dz});
    pl->tiles = (unsigned)((a->D + 64 * pl->VC - 1) / (64 * pl->VC));
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, CHUNK, (int)((a->S + CHUNK - 1) / CHUNK)};
    pl->slots = slots_of(pl->q);
    if (!grid_fits(pl->slots * pl->tiles, 64 * WAVES)) return unsupported("the call needs more than 2^32 threads");
    pl->chunked = a->S > CHUNK;
    pl->agg = up256((size_t)pl->slots * a->D * sizeof(float));
    pl->part = up256((size_t)pl->slots * 3 * a->D * sizeof(float));
    pl->bytes = pl->part + (pl->chunked ? 3 * pl->agg : 0);
    return MIMO_OK;
}

template <int DT, int VC> mimo_status run_bwd(const RecurParams& p, hipStream_t st) {
    const dim3 grid((unsigned)(p.slots * p.tiles));
    if (p.chunked) {
        mimo_status s = launch(&k_recur_agg<DT, VC>, grid, 64 * WAVES, 0, st, p);
        if (s != MIMO_OK) return s;
        s = launch_recur_carry<true>(p, st);
        if (s != MIMO_OK) return s;
    }
    const mimo_status s = launch(&k_recur_bwd<DT, VC>, grid, 64 * WAVES, 0, st, p);
    if (s != MIMO_OK) return s;
    return launch(&k_recur_sums, dim3((unsigned)((3L * p.D + SUM_COLS - 1) / SUM_COLS)), 256, 0, st, p);
}

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_recur_bwd_workspace_size(const mamba_recur_bwd_args* a, size_t* bytes) {
    BwdPlan pl;
    const mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = pl.bytes;
    return MIMO_OK;
}

mimo_status mamba_recur_bwd(const mamba_recur_bwd_args* a, void* stream) {
    BwdPlan pl;
    mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (!a->dout.data || !a->x.data || !a->r.data || !a->i.data || !a->decay || !a->dx || !a->dr || !a->di || !a->ddecay)
        return bad("dout, x, r, i, decay, dx, dr, di and ddecay must not be NULL");
    if ((a->z.data == nullptr) != (a->dz == nullptr)) return bad("dz must be given exactly when z is given");
    if ((a->r_bias == nullptr) != (a->dr_bias == nullptr)) return bad("dr_bias must be given exactly when r_bias is given");
    if ((a->i_bias == nullptr) != (a->di_bias == nullptr)) return bad("di_bias must be given exactly when i_bias is given");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, pl.bytes)) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    char* ws = static_cast<char*>(a->workspace);
    RecurParams p{};
    p.q = pl.q, p.D = (int)a->D, p.nvec = p.D / pl.VC, p.tiles = pl.tiles, p.slots = pl.slots;
    p.has_z = a->z.data != nullptr, p.chunked = pl.chunked, p.rate = a->rate;
    p.dout = rows_of(a->dout, packed), p.x = rows_of(a->x, packed), p.r = rows_of(a->r, packed), p.i = rows_of(a->i, packed);
    p.z = rows_of(a->z, packed);
    p.decay = a->decay, p.rb = a->r_bias, p.ib = a->i_bias, p.init = a->initial_state, p.dstate = a->dstate;
    p.dx = a->dx, p.dr = a->dr, p.di = a->di, p.dz = a->dz;
    p.ddecay = a->ddecay, p.drb = a->dr_bias, p.dib = a->di_bias, p.dinit = a->dinitial_state;
    p.part = reinterpret_cast<float*>(ws);
    p.agg_h = reinterpret_cast<float*>(ws + pl.part), p.agg_p = reinterpret_cast<float*>(ws + pl.part + pl.agg);
    p.agg_g = reinterpret_cast<float*>(ws + pl.part + 2 * pl.agg);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == BF16) return pl.VC == 2 ? run_bwd<BF16, 2>(p, st) : run_bwd<BF16, 1>(p, st);
    if (a->dtype == F16) return pl.VC == 2 ? run_bwd<F16, 2>(p, st) : run_bwd<F16, 1>(p, st);
    return pl.VC == 2 ? run_bwd<F32, 2>(p, st) : run_bwd<F32, 1>(p, st);
}

}  // extern "C"
