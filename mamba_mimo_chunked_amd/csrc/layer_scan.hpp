// Selective scan with a decay for each (channel, state): parameters and device code of the forward
// pass, the chunk aggregates and the carry between chunks, which the backward pass shares.
//
//   h[t] = exp(dt[t] a) h[t-1] + dt[t] u[t] b[t],  y[t] = <c[t], h[t]> + d u[t],  out = y silu(z)
//
// The decay depends on token, channel and state, so there is no matrix form: a token costs a channel
// N exponentials (half the rate of a multiply-add on this GPU) and four multiplies or multiply-adds
// each, which bind, not memory: 6 issue slots a state forward, against 0.5 bytes at N = 16. A lane owns
// one channel with NS states in registers, a block 64 channels with N split over KS waves; the waves share
// the steps of a tile of tokens and add up <c, h> in LDS, where b and c of the tile lie too and are read as
// broadcasts. Loads of the next tile are in flight during a tile; rows are addressed by scalars; tokens
// behind the chunk take a step of zero, so that nothing in a tile branches.
//
// Where channels alone do not fill the GPU the time axis is cut into chunks: k_walk<AGG> walks every
// chunk but a sequence's last from zero (its last state, and the sum of dt, which gives the chunk's
// decay exp(a sum dt)), k_carry chains the states that enter the chunks, and k_walk<FWD> walks the
// chunks from them. Measured, [8192, 1024] bf16, N = 16: 67 us for the three; [8 x 2048, 2048]: 224 us.
#pragma once
#include <type_traits>

#include "layer.hpp"

namespace mimo {
namespace layer {

struct ScanParams {
    Seqs q;
    int D, G, N, Dg, tpg;           // channels, groups, states, channels and channel tiles of a group
    int softplus, zero_tail, chunked, has_z, vec;   // vec: rows of N floats in 16-byte accesses
    Rows u, dt, b, c, z, dout;
    const float *a, *d, *bias;
    const float *init, *dstate;
    void* out;
    float* state;
    float *agg, *gagg, *sdt;        // [slots][D][N] twice, [slots][D]
    // backward
    void *du, *ddt, *db, *dc, *dz;
    float *da, *dd, *dbias, *dinit;
    float *pbc, *pdd;               // [tpg][tokens][G][2][N], [slots][2][D]
    float *uh, *udt;                // units of a chunk behind its first: state from zero and sum of dt in front, [..][D][N], [..][D]
    int units, seq_units;           // of those: a full chunk's, a dense sequence's
    long slots, tokens;
};

// first row of the flat token axis of a place
__device__ __forceinline__ long flat_row(const Seqs& q, const Place& pl) { return q.cu ? (long)pl.row0 : (long)pl.i * q.S; }

// Where a chunk's units behind its first lie (backward): in the order of the tokens, CH / UNIT - 1 = p.units a full chunk.
// Packed, sequence i starts at floor(start(i) * units / CH) + i: as many units as its length needs lie in front of where the
// next one starts, and the room goes by the tokens, not by the chunks that the sequences start.
__device__ __forceinline__ long first_unit(const ScanParams& p, const Place& pl) {
    const long in = (long)pl.j * p.units;
    if (p.q.cu == nullptr) return (long)pl.i * p.seq_units + in;
    const int whole = pl.row0 / p.q.CH;
    return whole * p.units + (pl.row0 - whole * p.q.CH) * p.units / p.q.CH + pl.i + in;
}

// a channel tile: CPB channels of one group
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

// K floats of a row of N, from state n0 on, `none` past the row
template <int K> __device__ __forceinline__ void load_states(const float* row, int n0, int N, bool vec, float none, float (&x)[K]) {
#pragma unroll
    for (int k = 0; k < K; k += 4) {
        if (vec && n0 + k < N) {
            const float4 v = *reinterpret_cast<const float4*>(row + n0 + k);
            x[k] = v.x, x[k + 1] = v.y, x[k + 2] = v.z, x[k + 3] = v.w;
        } else {
#pragma unroll
            for (int i = k; i < k + 4; ++i) x[i] = !vec && n0 + i < N ? row[n0 + i] : none;
        }
    }
}
template <int K> __device__ __forceinline__ void store_states(float* row, int n0, int N, bool vec, const float (&x)[K]) {
#pragma unroll
    for (int k = 0; k < K; k += 4) {
        if (vec) {
            if (n0 + k < N) *reinterpret_cast<float4*>(row + n0 + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
        } else {
#pragma unroll
            for (int i = k; i < k + 4; ++i)
                if (n0 + i < N) row[n0 + i] = x[i];
        }
    }
}
// the decay's base: exp(dt a) = exp2(dt * decay_base(a)); finite, so that a step of zero is no decay for a = -inf too
// (NaN stays)
__device__ __forceinline__ float decay_base(float a) {
    const float x = a * LOG2E;
    return x < -3e38f ? -3e38f : x;
}

// FWD: the outputs. AGG: a chunk's last state from zero. AGG2: also the adjoint that leaves it to the
// left, sum_t exp(a sum_{s <= t} dt) c[t] dy[t], from the same exponentials.
enum { FWD, AGG, AGG2 };
// Waves a SIMD that the registers have to allow: five where the states are split over many waves, whose registers hold that
// many without scratch memory ([8192, 1024], N = 16: 70.5 us without the bound, 69 with; [16 x 1024, 4096], N = 64: 741 and 734);
// six spill in the backward walk (N = 8: 91 us instead of 80). Four in the outputs' walk by two waves, which five left with 2 to
// 9 registers in scratch memory ([2048, 512], N = 8: 23.1 us, 24.1 with five; [4096, 512], N = 7: 25.4 and 27.2). Six for four
// states by eight waves, of which LDS lets three blocks in (N = 24: 103 us, 113 with the 82 registers that five allow). 16 waves
// a block are four a SIMD.
constexpr int walk_waves(int NS, int KS, int MODE) {
    return KS == 1 ? 2 : KS == 16 || (KS == 2 && MODE == FWD) ? 4 : NS == 4 && KS == 8 && MODE == FWD ? 6 : 5;
}

constexpr int UNIT = 16;   // tokens of a unit (backward)

// Tokens of a tile: what a lane keeps in registers, or the waves of a block share in LDS: 16, or 8 where one wave holds
// all states and in the backward walk of few waves ([4 x 4096, 1024], N = 16, backward: 327 us with 8, 332 with 16; forward
// [8 x 2048, 2048]: 224 us with 16, 231 with 8, 260 with 32).
constexpr int tile_tokens(int KS, int MODE) { return KS == 1 || (KS <= 4 && MODE == AGG2) ? 8 : 16; }

// f(n) with n = `states` as a constant: 0 (or less) to NS (or more)
template <int NS, class F> __device__ __forceinline__ void with_states(int states, F f) {
    if constexpr (NS > 0) {
        if (states >= NS) f(std::integral_constant<int, NS>{});
        else with_states<NS - 1>(states, f);
    } else f(std::integral_constant<int, 0>{});
}

// PAD: the waves hold more than N states. A place behind the last one reads zeros for b and c, but an infinite input times
// zero is NaN, and so would <c, h> be: the outputs' walk leaves those places out, by a loop for each number of states
// that a wave may hold ([8192, 1024] bf16, N = 7: 54 us, 63 with a condition in each step; [8192, 512], N = 100: 207 and 248;
// with the places in the sum 55 and 223).
template <int DT, int NS, int KS, int MODE, bool PAD> __global__ __launch_bounds__(64 * KS, walk_waves(NS, KS, MODE)) void k_walk(ScanParams p) {
    typedef raw_t<DT> raw;
    constexpr int TT = tile_tokens(KS, MODE), NP = NS * KS, TPW = TT / KS, NB = (TT * NP + 64 * KS - 1) / (64 * KS);
    constexpr bool C = MODE != AGG, OUT = MODE == FWD, ONE = KS == 1;
    __shared__ float s_dt[ONE ? 1 : TT][64], s_du[ONE ? 1 : TT][64], s_dy[!ONE && MODE == AGG2 ? TT : 1][64];
    __shared__ __attribute__((aligned(16))) float s_b[TT][NP], s_c[C ? TT : 1][NP];
    __shared__ float s_y[OUT && !ONE ? KS : 1][OUT && !ONE ? TT : 1][64];
    const Place pl = place(p.q, blockIdx.x);
    if (!pl.ok) return;
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    if (MODE == AGG && (pl.i == p.q.n || t1 == pl.len)) return;
    if (MODE == AGG2 && pl.i == p.q.n) return;
    const int lane = threadIdx.x & 63, w = ONE ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile tile = tile_of<64>(p, blockIdx.y);
    const bool act = lane < tile.left;
    const unsigned off = act ? lane : 0;    // rows are addressed as a scalar base and this offset
    const int d = tile.c0 + off;
    const long D = p.D;
    raw* out = static_cast<raw*>(p.out) + flat_row(p.q, pl) * D + tile.c0;
    if (OUT && pl.i == p.q.n) {
        if (p.zero_tail && act)
            for (int t = t0 + w; t < t1; t += KS) (out + t * D)[off] = to_raw<DT>(0.f);
        return;
    }
    const raw *u = at<DT>(p.u, pl) + tile.c0, *dt = at<DT>(p.dt, pl) + tile.c0;
    const raw *z = p.has_z ? at<DT>(p.z, pl) + tile.c0 : nullptr, *dout = MODE == AGG2 ? at<DT>(p.dout, pl) + tile.c0 : nullptr;
    const raw *b = at<DT>(p.b, pl) + tile.g * p.N, *c = C ? at<DT>(p.c, pl) + tile.g * p.N : nullptr;
    const float bias = p.bias ? p.bias[d] : 0.f, skip = OUT && p.d ? p.d[d] : 0.f;

    float a[NS], h[NS], gr[MODE == AGG2 ? NS : 1], pr[MODE == AGG2 ? NS : 1];
    float total = 0.f;
    load_states(p.a + d * (long)p.N, w * NS, p.N, p.vec, 0.f, a);
    const float* from = !OUT ? nullptr : p.chunked ? p.agg + blockIdx.x * D * p.N : p.init ? p.init + pl.i * D * p.N : nullptr;
    if (from) load_states(from + d * (long)p.N, w * NS, p.N, p.vec, 0.f, h);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        a[k] = decay_base(a[k]);
        if (!from) h[k] = 0.f;
        if (MODE == AGG2) gr[k] = 0.f, pr[k] = 1.f;
    }

    raw r_dt[TPW], r_u[TPW], r_z[TPW], r_g[TPW], r_b[NB], r_c[NB];
    // this thread's elements of b and c: rows e / NP + t0, from tile to tile TT rows on
    const int e0 = threadIdx.x, bn = e0 % NP, br = e0 / NP;
    constexpr int BR = 64 * KS / NP;            // rows between a thread's elements
    const bool bon = bn < p.N && (64 * KS <= TT * NP || e0 < TT * NP);
    const raw *pb = b + (long)(t0 + br) * p.b.ts + bn, *pc = C ? c + (long)(t0 + br) * p.c.ts + bn : nullptr;
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            const long row = min(t + w * TPW + k, t1 - 1);
            r_dt[k] = (dt + row * p.dt.ts)[off];
            r_u[k] = (u + row * p.u.ts)[off];
            if (C && z) r_z[k] = (z + row * p.z.ts)[off];
            if (MODE == AGG2) r_g[k] = (dout + row * p.dout.ts)[off];
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const bool on = bon && t + br + k * BR < t1;
            r_b[k] = raw(0);
            if (on) r_b[k] = pb[(long)k * BR * p.b.ts];
            if (C) {
                r_c[k] = raw(0);
                if (on) r_c[k] = pc[(long)k * BR * p.c.ts];
            }
        }
        pb += (long)TT * p.b.ts;
        if (C) pc += (long)TT * p.c.ts;
    };
    // one token of step v: the wave's first `real` states, and <c, h> (or, with dy = g, the adjoint). A step of zero changes
    // nothing: so pass the tokens of a tile behind the chunk.
    auto token = [&](auto real, int t, float v, float vu, float g) {
        float y[2] = {0.f, 0.f};
        if (MODE != FWD) total += v;
#pragma unroll
        for (int k = 0; k < real; ++k) {
            const float e = exp2_hw(v * a[k]);
            h[k] = __builtin_fmaf(e, h[k], vu * s_b[t][w * NS + k]);
            if (OUT) y[k & 1] = __builtin_fmaf(h[k], s_c[t][w * NS + k], y[k & 1]);
            if (MODE == AGG2) {
                pr[k] *= e;
                gr[k] = __builtin_fmaf(pr[k], g * s_c[t][w * NS + k], gr[k]);
            }
        }
        return y[0] + y[1];
    };
    const long unit0 = MODE == AGG2 ? first_unit(p, pl) - 1 : 0;
    if (t0 < t1) fetch(t0);
    for (int tt = t0; tt < t1; tt += TT) {
        float f_v[TPW], f_u[TPW], f_z[TPW], f_g[TPW];   // step, input, gate, dy of this wave's tokens
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            f_v[k] = to_f<DT>(r_dt[k]) + bias;
            f_u[k] = to_f<DT>(r_u[k]);
            f_z[k] = 1.f;
        }
        if (p.softplus) {
#pragma unroll
            for (int k = 0; k < TPW; ++k) f_v[k] = softplus(f_v[k]);
        }
        if (C && z) {
#pragma unroll
            for (int k = 0; k < TPW; ++k) {
                const float x = to_f<DT>(r_z[k]);
                f_z[k] = x * sigmoid(x);
            }
        }
        if (tt + TT > t1) {
#pragma unroll
            for (int k = 0; k < TPW; ++k)
                if (tt + w * TPW + k >= t1) {
                    f_v[k] = f_u[k] = f_z[k] = 0.f;
                    if (MODE == AGG2) r_g[k] = raw(0);
                }
        }
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            f_g[k] = MODE == AGG2 ? to_f<DT>(r_g[k]) * f_z[k] : 0.f;
            if (!ONE) {
                s_dt[w * TPW + k][lane] = f_v[k];
                s_du[w * TPW + k][lane] = f_v[k] * f_u[k];
                if (MODE == AGG2) s_dy[w * TPW + k][lane] = f_g[k];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            if (64 * KS > TT * NP && e0 >= TT * NP) continue;
            s_b[br + k * BR][bn] = to_f<DT>(r_b[k]);
            if (C) s_c[br + k * BR][bn] = to_f<DT>(r_c[k]);
        }
        __syncthreads();
        if (tt + TT < t1) fetch(tt + TT);
        if constexpr (MODE == AGG2) {   // the backward pass starts again from every unit
            const int k = (tt - t0) / UNIT;
            if (k > 0 && (tt - t0) % UNIT == 0 && act) {
                const long at = unit0 + k;
                store_states(p.uh + (at * D + d) * p.N, w * NS, p.N, p.vec, h);
                if (w == 0) p.udt[at * D + d] = total;
            }
        }
        auto tokens = [&](auto real) {
            if constexpr (ONE) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const float y = token(real, t, f_v[t], f_v[t] * f_u[t], f_g[t]);
                    if (OUT && act && tt + t < t1) (out + (tt + t) * D)[off] = to_raw<DT>(__builtin_fmaf(skip, f_u[t], y) * f_z[t]);
                }
            } else {
                // the reads of a whole tile ahead of their use (packed prompts [4100, 2048], N = 64: 221 us with four tokens,
                // 207 with 16; backward 327 with four, 329)
#pragma unroll (MODE == AGG2 ? 4 : TT)
                for (int t = 0; t < TT; ++t) {
                    const float y = token(real, t, s_dt[t][lane], s_du[t][lane], MODE == AGG2 ? s_dy[t][lane] : 0.f);
                    if (OUT) s_y[w][t][lane] = y;
                }
            }
        };
        if constexpr (PAD) with_states<NS>(p.N - w * NS, tokens);
        else tokens(std::integral_constant<int, NS>{});
        __syncthreads();
        if (OUT && !ONE && act) {
#pragma unroll
            for (int k = 0; k < TPW; ++k) {
                const int t = w * TPW + k;
                if (tt + t < t1) {
                    float y = skip * f_u[k];
#pragma unroll
                    for (int v = 0; v < KS; ++v) y += s_y[v][t][lane];
                    (out + (tt + t) * D)[off] = to_raw<DT>(y * f_z[k]);
                }
            }
        }
    }
    if (!act || (MODE == AGG2 && !p.chunked)) return;
    float* to = !OUT ? p.agg + blockIdx.x * D * p.N : p.state && t1 == pl.len ? p.state + pl.i * D * p.N : nullptr;
    if (to) store_states(to + d * (long)p.N, w * NS, p.N, p.vec, h);
    if constexpr (MODE == AGG2) store_states(p.gagg + (blockIdx.x * D + d) * p.N, w * NS, p.N, p.vec, gr);
    if (!OUT && w == 0) p.sdt[blockIdx.x * D + d] = total;
}

// The states that enter the chunks of sequence blockIdx.z, in place of the aggregates, for 64 times V of the
// D * N states.
// Wave w of a block takes SPAN chunks of every SPAN * waves: it folds them from zero, the waves'
// folds are chained in LDS, and it walks them again from what enters them, so that all loads of up to 128 chunks
// are in flight together. With ADJ, blockIdx.y = 1 runs the adjoints from the last chunk to the first, from dstate,
// and leave the gradient of the initial state.
constexpr int SPAN = 8, SPAN_WAVES = 16;
template <bool ADJ, int V> __global__ __launch_bounds__(64 * SPAN_WAVES) void k_carry(ScanParams p) {
    typedef float vec __attribute__((ext_vector_type(V)));
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    vec *s_h = reinterpret_cast<vec*>(lds), *s_p = s_h + waves * 64;   // [waves][64] each
    const int i = blockIdx.z;
    const unsigned step = (unsigned)p.D * p.N, s = min((blockIdx.x * 64 + lane) * V, step - V), d = s / (unsigned)p.N;
    const bool rev = ADJ && blockIdx.y, act = (blockIdx.x * 64 + lane) * V < step;
    const long D = p.D;
    const int slot0 = p.q.cu ? p.q.base(i) : i * p.q.nc;
    const int len = p.q.cu ? max((i < p.q.n ? p.q.start(i + 1) : p.q.S) - p.q.start(i), 0) : p.q.S;
    const int nc = max((len + p.q.CH - 1) / p.q.CH, 1);
    const int have = ADJ ? (len > 0 ? nc : 0) : nc - 1;    // chunks with an aggregate: FWD needs none of the last
    auto get = [](const float* x) { return *reinterpret_cast<const vec*>(x); };
    vec a = get(p.a + s);
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = decay_base(a[v]);
    const long own = (long)i * step + s;
    const float* from = rev ? p.dstate : p.init;
    vec h = from ? get(from + own) : vec(0.f);
    float* agg = (rev ? p.gagg : p.agg) + (long)slot0 * step + s;
    const float* sdt = p.sdt + (long)slot0 * D + d;
    for (int j0 = 0; j0 < nc; j0 += SPAN * waves) {
        vec x[SPAN], e[SPAN], fold = vec(0.f), prod = vec(1.f);
        float dt[SPAN];
#pragma unroll
        for (int k = 0; k < SPAN; ++k) {
            const int j = j0 + w * SPAN + k, at = rev ? nc - 1 - j : j;
            x[k] = j < have ? get(agg + (long)at * step) : vec(0.f);
            dt[k] = j < have ? sdt[(long)at * D] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < SPAN; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e[k][v] = exp2_hw(a[v] * dt[k]);
                fold[v] = __builtin_fmaf(e[k][v], fold[v], x[k][v]);
                prod[v] *= e[k][v];
            }
        vec g = h;
        if (waves > 1) {
            s_h[w * 64 + lane] = fold;
            s_p[w * 64 + lane] = prod;
            __syncthreads();
            for (int o = 0; o < waves; ++o) {
                if (o == w) g = h;
                const vec f = s_h[o * 64 + lane], q = s_p[o * 64 + lane];
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(q[v], h[v], f[v]);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(prod[v], h[v], fold[v]);
        }
#pragma unroll
        for (int k = 0; k < SPAN; ++k) {
            const int j = j0 + w * SPAN + k;
            if (j < nc && act) *reinterpret_cast<vec*>(agg + (long)(rev ? nc - 1 - j : j) * step) = g;
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] = __builtin_fmaf(e[k][v], g[v], x[k][v]);
        }
    }
    if (rev && p.dinit && w == 0 && act) *reinterpret_cast<vec*>(p.dinit + own) = h;
}

// ---------------------------------------------------------------- host side
// 64 channels by sixteen states: the unit in which the work of a walk is counted
inline int waves_for(int64_t N) { return N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8; }

// States of a lane by waves of a block. Few states a lane leave the registers for five waves a SIMD and more: [8192,
// 1024], N = 16 forward 78 us with 16 states a lane, 69 with four (8 x 2048 x 2048: 245 and 224; N = 32: 146 and 109).
// What it costs, <c, h> joined in LDS over more waves, weighs more from N = 64 on, where eight are as fast as 16 or
// faster ([16 x 1024, 4096] 783 us with 16 by 4, 741 with 8 by 8; [1024, 1024] 48 and 43; four, packed prompts: 270, 207 with
// eight). For N <= 8 one wave needs no joining, so those are split only where the blocks do not fill the GPU, up to ten a CU, and
// in the backward walk, which joins nothing (N = 8, split and not: [2048, 512] 24.7 us and 26.6, [8192, 512], 2048 blocks, 35.0 and
// 37.0, [8192, 1024], as many, 52.5 and 54.4, [2 x 4096, 768], 2064 blocks, 47.6 and 53.7; [8192, 2048], 4096 blocks, 90.7 and 86.6;
// N = 6, [2 x 8192, 1024], as many, 87.0 and 80.4; fp32 [4096, 1024], 2048 blocks, 37.5 and 36.7).
constexpr long FEW = 2560;
inline int walk_threads(int64_t N) { return N <= 4 ? 64 : N <= 8 ? 128 : N <= 16 ? 256 : N <= 64 ? 512 : 1024; }   // at most
inline int walk_places(int64_t N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }
template <int DT, int MODE, bool PAD> mimo_status launch_shape(const ScanParams& p, hipStream_t st) {
    const dim3 grid((unsigned)p.slots, (unsigned)(p.G * p.tpg));
    if (p.N <= 4) return launch(&k_walk<DT, 4, 1, MODE, PAD>, grid, 64, 0, st, p);
    if (p.N <= 8) {
        if constexpr (MODE != AGG2) {
            if (p.slots * p.G * p.tpg > FEW) return launch(&k_walk<DT, 8, 1, MODE, PAD>, grid, 64, 0, st, p);
        }
        return launch(&k_walk<DT, 4, 2, MODE, PAD>, grid, 128, 0, st, p);
    }
    if (p.N <= 16) return launch(&k_walk<DT, 4, 4, MODE, PAD>, grid, 256, 0, st, p);
    if (p.N <= 32) return launch(&k_walk<DT, 4, 8, MODE, PAD>, grid, 512, 0, st, p);
    if (p.N <= 64) return launch(&k_walk<DT, 8, 8, MODE, PAD>, grid, 512, 0, st, p);
    return launch(&k_walk<DT, 8, 16, MODE, PAD>, grid, 1024, 0, st, p);
}
template <int DT, int MODE> mimo_status launch_walk(const ScanParams& p, hipStream_t st) {
    return p.N < walk_places(p.N) && MODE == FWD ? launch_shape<DT, MODE, MODE == FWD>(p, st) : launch_shape<DT, MODE, false>(p, st);
}
// Four states a thread where that still makes a block for each CU (7 x 2048 x 64 states: 13 us, 23 with one), else one
// ([1024, 16]: 6.3 us, 7.8 with four). Waves for the chunks of a sequence, of a packed one for twice the average: longer
// ones take more rounds, but blocks for the longest that could be leave most waves idle.
template <bool ADJ> mimo_status launch_carry(const ScanParams& p, hipStream_t st) {
    long chunks = p.q.nc;
    if (p.q.cu && 2 * p.slots / p.q.n < chunks) chunks = 2 * p.slots / p.q.n;
    const long states = (long)p.D * p.N;
    const int waves = (int)(chunks <= SPAN ? 1 : chunks < SPAN * SPAN_WAVES ? (chunks + SPAN - 1) / SPAN : SPAN_WAVES), dirs = ADJ ? 2 : 1;
    const size_t lds = waves > 1 ? sizeof(float) * 2 * 64 * waves : 0;
    if (p.vec && (states + 255) / 256 * dirs * p.q.n >= 256)
        return launch(&k_carry<ADJ, 4>, dim3((unsigned)((states + 255) / 256), dirs, p.q.n), 64 * waves, 4 * lds, st, p);
    return launch(&k_carry<ADJ, 1>, dim3((unsigned)((states + 63) / 64), dirs, p.q.n), 64 * waves, lds, st, p);
}
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
