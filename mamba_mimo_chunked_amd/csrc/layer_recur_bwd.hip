// Gated linear recurrence, backward pass (formulas, gates, rows: layer_recur.hpp). Nothing is kept from the forward pass.
// A block takes one chunk of WAVES * TT tokens; k_recur_agg leaves each chunk's joined step, forward and for the adjoint, the
// carry turns them into the state and the adjoint that enter, and k_recur_bwd walks its tokens forward for the states and
// back for the adjoints and the gradients. Parameters' gradients leave one partial row a chunk, added up in order.
#include "layer_recur.hpp"

namespace mimo {
namespace layer {
namespace {

constexpr int TT = 8;               // tokens of a wave
// Just below the root of fp32's smallest normal number: below 2^-126 the hardware's root counts 1 - a^2 as zero, while l, half of it, may still be
// there. l / e, in truth e / 2, is taken with at least this e, so it is off by 1e-19 at most.
constexpr float LEAST_ROOT = 1e-19f;

// Two halves are split where they are used: else the compiler holds them in a register each and lacks twelve ([4 x 4096, 2048] fp16: 200 us, 277 without).
template <int DT, int VC> __device__ __forceinline__ void unpack_late(Pack<DT, VC> x, float (&y)[VC]) {
    if constexpr (DT == F16 && VC == 2) renew<DT, VC>(x);
    unpack<DT, VC>(x, y);
}
// A wave's tokens: the rows that are needed to the end, the gates, and b, later the state in front of a token. What is cheap to have
// again (a: one 2^x) is not kept, so that four waves a SIMD fit.
template <int DT, int VC, bool GATE, int AUX> struct Tokens {
    RowsOf<DT, VC, TT, AUX> x, r, i, g, z;
    float l2[TT][VC], si[TT][VC], e[TT][VC], b[TT][VC];     // l2: l in powers of two

    __device__ __forceinline__ void fetch(const RecurParams& p, const Place& pl, int tw, int t1, unsigned lane) {
        x.place(p.x, pl, p.D, tw, t1), r.place(p.r, pl, p.D, tw, t1), i.place(p.i, pl, p.D, tw, t1), g.place(p.dout, pl, p.D, tw, t1);
        if constexpr (GATE) z.place(p.z, pl, p.D, tw, t1);
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            x.fetch(k, lane), r.fetch(k, lane), i.fetch(k, lane), g.fetch(k, lane);
            if constexpr (GATE) z.fetch(k, lane);
        }
    }
    // dout silu(z)
    __device__ __forceinline__ void meets(int k, float (&dh)[VC]) const {
        float fz[VC];
        unpack_late<DT, VC>(g.t[k], dh);
        if constexpr (GATE) {
            unpack_late<DT, VC>(z.t[k], fz);
#pragma unroll
            for (int v = 0; v < VC; ++v) dh[v] *= fz[v] * sigmoid(fz[v]);
        }
    }
    // From here on values are taken for new: what follows from them is computed again, not kept in registers for its second use.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            renew(x.t[k]), renew(g.t[k]);
            if constexpr (GATE) renew(z.t[k]);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                asm("" : "+v"(l2[k][v]));
                asm("" : "+v"(si[k][v]));
            }
        }
    }
    // Gates of the tokens, and their joined step: last state from zero, product of a, adjoint that leaves to the left from zero.
    __device__ __forceinline__ void join(const Gates<VC>& gates, int left, float (&h)[VC], float (&q)[VC], float (&c)[VC]) {
#pragma unroll
        for (int v = 0; v < VC; ++v) h[v] = c[v] = 0.f, q[v] = 1.f;
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            float fr[VC], fi[VC], fx[VC], dh[VC], a[VC];
            unpack_late<DT, VC>(x.t[k], fx);
            unpack_late<DT, VC>(r.t[k], fr);
            unpack_late<DT, VC>(i.t[k], fi);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                float e2;
                l2[k][v] = speed_of(gates, v, k, left) * gates.open(fr[v], gates.rb[v]);
                si[k][v] = gates.open(fi[v], gates.ib[v]);
                keep_and_enter(l2[k][v], a[v], e2);
                e[k][v] = root(e2);
                b[k][v] = e[k][v] * (si[k][v] * fx[v]);
            }
            meets(k, dh);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                h[v] = __builtin_fmaf(a[v], h[v], b[k][v]);
                q[v] *= a[v];
                c[v] = __builtin_fmaf(q[v], dh[v], c[v]);
            }
        }
    }
};

template <int VC, int WAVES> struct Join {
    float h[WAVES][64 * VC], q[WAVES][64 * VC], c[WAVES][64 * VC];
    __device__ __forceinline__ void put(int w, int lane, const float (&fh)[VC], const float (&fq)[VC], const float (&fc)[VC]) {
#pragma unroll
        for (int v = 0; v < VC; ++v) h[w][lane * VC + v] = fh[v], q[w][lane * VC + v] = fq[v], c[w][lane * VC + v] = fc[v];
    }
};

// One channel a lane, 52 registers: 32 waves a CU hide its loads ([4 x 4096, 2048] bf16 72 us, 4.7 TB/s, vector units 65 % busy). Its loads stay in the
// last-level cache for k_recur_bwd.
template <int DT, bool GATE, int WAVES> __global__ __launch_bounds__(64 * WAVES) void k_recur_agg(RecurParams p) {
    constexpr int CHUNK = WAVES * TT;
    __shared__ Join<1, WAVES> s;
    const unsigned tiles = (p.D + 63) / 64, slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    const Place pl = place_by_wave(p.q, slot);
    if (!pl.ok || pl.i == p.q.n) return;
    const int t0 = pl.j * CHUNK, t1 = min(t0 + CHUNK, pl.len);
    if (t0 >= t1) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tw = t0 + w * TT;
    const bool act = tile * 64 + lane < (unsigned)p.D;
    const unsigned d = act ? tile * 64 + lane : 0;
    Tokens<DT, 1, GATE, 0> k;
    float h[1] = {0.f}, q[1] = {1.f}, c[1] = {0.f};
    if (tw < t1) {                  // a short sequence leaves waves without tokens
        k.fetch(p, pl, tw, t1, d * sizeof(raw_t<DT>));
        k.join(Gates<1>(p, d), t1 - tw, h, q, c);
    }
    s.put(w, lane, h, q, c);
    __syncthreads();
    if (w != 0 || !act) return;
    float hh = 0.f, qq = 1.f, cc = 0.f;
#pragma unroll
    for (int o = 0; o < WAVES; ++o) {
        hh = __builtin_fmaf(s.q[o][lane], hh, s.h[o][lane]);
        qq *= s.q[o][lane];
        cc = __builtin_fmaf(s.q[WAVES - 1 - o][lane], cc, s.c[WAVES - 1 - o][lane]);
    }
    const long at = (long)slot * p.D + d;
    p.agg_h[at] = hh, p.agg_p[at] = qq, p.agg_g[at] = cc;
}

// The states that enter the chunks of sequence blockIdx.z, in place of the aggregates. Wave w of a block takes SPAN chunks of
// every SPAN * waves: it folds them from zero, the waves' folds are chained in LDS, and it walks them again from what enters
// them, so that all loads of up to 128 chunks are in flight together. blockIdx.y = 1 runs the adjoints from the last chunk to the
// first, from dstate, and leaves the gradient of the initial state. Latency: 64 chunks of 4 sequences, D = 2048, 5 us.
constexpr int RSPAN = 8, RSPAN_WAVES = 16;
__global__ __launch_bounds__(64 * RSPAN_WAVES) void k_recur_carry(RecurParams p) {
    __shared__ float s_h[RSPAN_WAVES][64], s_p[RSPAN_WAVES][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int i = blockIdx.z;
    const unsigned d0 = blockIdx.x * 64 + lane;
    const bool rev = blockIdx.y, act = d0 < (unsigned)p.D;
    const unsigned d = act ? d0 : 0;
    const long D = p.D;
    const int slot0 = p.q.cu ? p.q.base(i) : i * p.q.nc;
    const int len = p.q.cu ? max((i < p.q.n ? p.q.start(i + 1) : p.q.S) - p.q.start(i), 0) : p.q.S;
    const int nc = max((len + p.q.CH - 1) / p.q.CH, 1);
    const int have = len > 0 ? nc : 0;      // chunks with an aggregate
    const float* from = rev ? p.dstate : p.init;
    float h = from ? from[(long)i * D + d] : 0.f;
    float* agg = (rev ? p.agg_g : p.agg_h) + (long)slot0 * D + d;
    const float* prod = p.agg_p + (long)slot0 * D + d;
    for (int j0 = 0; j0 < nc; j0 += RSPAN * waves) {
        float x[RSPAN], e[RSPAN], fold = 0.f, all = 1.f;
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            const int j = j0 + w * RSPAN + k, at = rev ? nc - 1 - j : j;
            x[k] = j < have ? agg[(long)at * D] : 0.f;
            e[k] = j < have ? prod[(long)at * D] : 1.f;
        }
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            fold = __builtin_fmaf(e[k], fold, x[k]);
            all *= e[k];
        }
        s_h[w][lane] = fold;
        s_p[w][lane] = all;
        __syncthreads();
        float g = h;
        for (int o = 0; o < waves; ++o) {
            if (o == w) g = h;
            h = __builtin_fmaf(s_p[o][lane], h, s_h[o][lane]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            const int j = j0 + w * RSPAN + k;
            if (j < nc && act) agg[(long)(rev ? nc - 1 - j : j) * D] = g;
            g = __builtin_fmaf(e[k], g, x[k]);
        }
    }
    if (rev && p.dinit && w == 0 && act) p.dinit[(long)i * D + d] = h;
}

// AUX: the policy of its accesses, the last ones to the inputs. The chunks come from the last to the first: the inputs that the
// aggregates read last are still in the last-level cache. [4 x 4096, 2048] bf16: 128 to 132 us for 604 MB, vector units 67 % busy; two channels a lane
// where 4 bytes allow it ([16384, 1000] 147 us, with one 175).
template <int DT, int VC, bool GATE, int AUX, int WAVES> __global__ __launch_bounds__(64 * WAVES, 4) void k_recur_bwd(RecurParams p) {
    typedef raw_t<DT> raw;
    constexpr int CHUNK = WAVES * TT;
    __shared__ Join<VC, WAVES> s;
    const unsigned index = blockIdx.x / p.tiles, tile = blockIdx.x - index * p.tiles, slot = (unsigned)p.slots - 1 - index;
    const Place pl = place_by_wave(p.q, slot);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned vec = tile * 64 + lane;
    const bool act = vec < (unsigned)p.nvec;
    const unsigned d = act ? vec * VC : 0, db = d * sizeof(raw);
    const long D = p.D;
    const int t0 = pl.j * CHUNK, t1 = pl.ok ? min(t0 + CHUNK, pl.len) : t0, tw = t0 + w * TT, left = t1 - tw;
    float* part = p.part + (long)slot * 3 * D + d;
    const bool tail = pl.i == p.q.n;
    const long flat = (recur_row(p.q, pl) + tw) * D;
    const auto dx = buffer_of(static_cast<raw*>(p.dx) + flat), dr = buffer_of(static_cast<raw*>(p.dr) + flat), di = buffer_of(static_cast<raw*>(p.di) + flat),
               dz = buffer_of(static_cast<raw*>(GATE ? p.dz : p.dx) + flat);
    const unsigned step = (unsigned)D * sizeof(raw);
    if (t0 >= t1 || tail) {         // no tokens, or those behind the last sequence
        const float zero[VC] = {};
        if (tail && act)
            for (int k = 0; k < min(left, TT); ++k) {
                store_at<DT, VC>(dx, db, k * step, zero);
                store_at<DT, VC>(dr, db, k * step, zero);
                store_at<DT, VC>(di, db, k * step, zero);
                if constexpr (GATE) store_at<DT, VC>(dz, db, k * step, zero);
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
    Tokens<DT, VC, GATE, AUX> k;
    if (left > 0) k.fetch(p, pl, tw, t1, db);
    const Gates<VC> gates(p, d);
    float h[VC], c[VC];
    const float* from = p.chunked ? p.agg_h + slot * D : p.init ? p.init + pl.i * D : nullptr;
    const float* late = p.chunked ? p.agg_g + slot * D : p.dstate ? p.dstate + pl.i * D : nullptr;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        h[v] = from ? from[d + v] : 0.f;
        c[v] = late ? late[d + v] : 0.f;
    }
    {
        float fh[VC], fq[VC], fc[VC];
#pragma unroll
        for (int v = 0; v < VC; ++v) fh[v] = fc[v] = 0.f, fq[v] = 1.f;
        if (left > 0) k.join(gates, left, fh, fq, fc);
        s.put(w, lane, fh, fq, fc);
    }
    __syncthreads();
    k.forget();
    // the state that enters this wave's tokens, and the adjoint
    for (int o = 0; o < w; ++o)
#pragma unroll
        for (int v = 0; v < VC; ++v) h[v] = __builtin_fmaf(s.q[o][lane * VC + v], h[v], s.h[o][lane * VC + v]);
    for (int o = WAVES - 1; o > w; --o)
#pragma unroll
        for (int v = 0; v < VC; ++v) c[v] = __builtin_fmaf(s.q[o][lane * VC + v], c[v], s.c[o][lane * VC + v]);
    float sum[3][VC] = {};
    if (left > 0) {
        // b becomes the state in front of a token
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float b = k.b[t][v];
                k.b[t][v] = h[v];
                h[v] = __builtin_fmaf(exp2_hw(k.l2[t][v]), h[v], b);
            }
        k.forget();
        float shut[VC];                 // -ln(2) / speed: what takes l2 to -ln(2) sigmoid(r)
#pragma unroll
        for (int v = 0; v < VC; ++v) shut[v] = gates.speed[v] < 0.f ? -LN2 / gates.speed[v] : 0.f;
        unsigned at = TT * step;
#pragma unroll
        for (int t = TT - 1; t >= 0; --t) {
            float fx[VC], fz[VC], fg[VC], g[VC], ox[VC], orr[VC], oi[VC], oz[VC], W[VC];
            unpack_late<DT, VC>(k.x.t[t], fx);
            unpack_late<DT, VC>(k.g.t[t], fg);
            if constexpr (GATE) unpack_late<DT, VC>(k.z.t[t], fz);
            k.meets(t, g);
            at -= step;
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float l2 = k.l2[t][v], si = k.si[t][v], e = k.e[t][v], hp = k.b[t][v], a = exp2_hw(l2);
                // l / e, which vanishes with e
                const float part = l2 * __builtin_amdgcn_rcpf(__builtin_fmaxf(e, LEAST_ROOT));
                g[v] += c[v];
                const float ga = a * g[v], u = si * fx[v], du = g[v] * e, dgate = du * u;
                // l times a log2(e), before it meets a state: where a token keeps nothing that is zero, and l h may be beyond fp32's range
                W[v] = __builtin_fmaf(ga * l2, hp, -(ga * part) * (a * u));
                c[v] = ga;
                ox[v] = du * si;
                oi[v] = __builtin_fmaf(-dgate, si, dgate);
                orr[v] = W[v] * __builtin_fmaf(l2, shut[v], LN2);           // 1 - sigmoid(r), times ln(2)
                if constexpr (GATE) {
                    const float sz = sigmoid(fz[v]), out = __builtin_fmaf(-fz[v], sz, fz[v]);
                    oz[v] = fg[v] * (t + 1 < TT ? k.b[t + 1 < TT ? t + 1 : 0][v] : h[v]) * __builtin_fmaf(sz, out, sz);
                }
            }
            if (t < left) {
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    sum[0][v] += W[v];
                    sum[1][v] += orr[v];
                    sum[2][v] += oi[v];
                }
                if (act) {
                    store_at<DT, VC, AUX>(dx, db, at, ox);
                    store_at<DT, VC, AUX>(dr, db, at, orr);
                    store_at<DT, VC, AUX>(di, db, at, oi);
                    if constexpr (GATE) store_at<DT, VC, AUX>(dz, db, at, oz);
                }
            }
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
            p.ddecay[col] = LN2 * (sp > 0.f ? s * (sigmoid(x) / sp) : s);
        }
    });
}

// Waves for the chunks of a sequence, of a packed one for twice the average: longer ones take more rounds.
mimo_status launch_recur_carry(const RecurParams& p, hipStream_t st) {
    long chunks = p.q.nc;
    if (p.q.cu && 2 * p.slots / p.q.n < chunks) chunks = 2 * p.slots / p.q.n;
    const int waves = (int)(chunks <= RSPAN ? 1 : chunks < RSPAN * RSPAN_WAVES ? (chunks + RSPAN - 1) / RSPAN : RSPAN_WAVES);
    return launch(&k_recur_carry, dim3((unsigned)((p.D + 63) / 64), 2, p.q.n), 64 * waves, 0, st, p);
}
struct BwdPlan {
    Seqs q;
    int VC, waves;
    unsigned tiles;
    long slots;
    bool chunked;
    size_t agg, part, bytes;
};

mimo_status plan_bwd(const mamba_recur_bwd_args* a, BwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_recur(a->n, a->S, a->D, a->dtype, a->rate);
    if (s != MIMO_OK || (s = check_strides(a->S, {&a->dout, &a->x, &a->r, &a->i, &a->z})) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->VC = channels_of(a->D, a->dtype, packed, {&a->dout, &a->x, &a->r, &a->i, &a->z}, {a->dx, a->dr, a->di, a->dz});
    pl->tiles = (unsigned)((a->D + 64 * pl->VC - 1) / (64 * pl->VC));
    pl->waves = waves_of(packed, a->n, a->S, TT);
    const int CH = pl->waves * TT;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    if (!grid_fits(pl->slots * ((a->D + 63) / 64), 64 * pl->waves)) return unsupported("the call needs more than 2^32 threads");
    pl->chunked = a->S > CH;
    pl->agg = up256((size_t)pl->slots * a->D * sizeof(float));
    pl->part = up256((size_t)pl->slots * 3 * a->D * sizeof(float));
    pl->bytes = pl->part + (pl->chunked ? 3 * pl->agg : 0);
    return MIMO_OK;
}

template <int DT, int VC, bool GATE, int WAVES> mimo_status run_bwd(const RecurParams& p, hipStream_t st) {
    if (p.chunked) {
        mimo_status s = launch(&k_recur_agg<DT, GATE, WAVES>, dim3((unsigned)(p.slots * ((p.D + 63) / 64))), 64 * WAVES, 0, st, p);
        if (s != MIMO_OK) return s;
        s = launch_recur_carry(p, st);
        if (s != MIMO_OK) return s;
    }
    const dim3 grid((unsigned)(p.slots * p.tiles));
    const mimo_status s = passes_by<DT>(p.q, p.D, GATE ? 9 : 7) ? launch(&k_recur_bwd<DT, VC, GATE, NT, WAVES>, grid, 64 * WAVES, 0, st, p)
                                                                : launch(&k_recur_bwd<DT, VC, GATE, 0, WAVES>, grid, 64 * WAVES, 0, st, p);
    if (s != MIMO_OK) return s;
    return launch(&k_recur_sums, dim3((unsigned)((3L * p.D + SUM_COLS - 1) / SUM_COLS)), 256, 0, st, p);
}
template <int DT, int VC, bool GATE> mimo_status run_waves(const BwdPlan& pl, const RecurParams& p, hipStream_t st) {
    return pl.waves == 8 ? run_bwd<DT, VC, GATE, 8>(p, st) : pl.waves == 4 ? run_bwd<DT, VC, GATE, 4>(p, st) : run_bwd<DT, VC, GATE, 2>(p, st);
}
template <int DT> mimo_status run_type(const BwdPlan& pl, const RecurParams& p, hipStream_t st) {
    if constexpr (DT != F32) {
        if (pl.VC == 2) return p.has_z ? run_waves<DT, 2, true>(pl, p, st) : run_waves<DT, 2, false>(pl, p, st);
    }
    return p.has_z ? run_waves<DT, 1, true>(pl, p, st) : run_waves<DT, 1, false>(pl, p, st);
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
    if (a->dtype == BF16) return run_type<BF16>(pl, p, st);
    return a->dtype == F16 ? run_type<F16>(pl, p, st) : run_type<F32>(pl, p, st);
}

}  // extern "C"
