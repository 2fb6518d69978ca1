// Gated linear recurrence, forward pass and step of one token (formulas, gates, carry: layer_recur.hpp).
#include <initializer_list>

#include "layer_recur.hpp"

namespace mimo {
namespace layer {
namespace {

constexpr int WAVES = 8;            // of a block
constexpr int tile_tokens(int DT) { return DT == F32 ? 8 : 16; }    // of a wave

// A block takes one chunk of 64 VC channels, WAVES * TT tokens a round, and the next round's rows are asked for during a
// round. AGG: the chunk's last state from zero and its product of a; else the outputs.
template <int DT, int VC, bool AGG> __global__ __launch_bounds__(64 * WAVES) void k_recur(RecurParams p) {
    typedef raw_t<DT> raw;
    constexpr int TT = tile_tokens(DT), ROUND = WAVES * TT;
    __shared__ float s_h[2][WAVES][64 * VC], s_p[2][WAVES][64 * VC];
    const unsigned slot = blockIdx.x / p.tiles, tile = blockIdx.x - slot * p.tiles;
    const Place pl = place(p.q, slot);
    if (!pl.ok) return;
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    if (AGG && (pl.i == p.q.n || t1 == pl.len)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned vec = tile * 64 + lane;
    const bool act = vec < (unsigned)p.nvec;
    const unsigned d = act ? vec * VC : 0;
    const long D = p.D;
    raw* out = static_cast<raw*>(p.out) + recur_row(p.q, pl) * D;
    if (!AGG && pl.i == p.q.n) {    // behind the last sequence
        const float zero[VC] = {};
        if (p.zero_tail && act)
            for (int t = t0 + w; t < t1; t += WAVES) store<DT, VC>(out + t * D + d, zero);
        return;
    }
    const raw *x = at<DT>(p.x, pl), *r = at<DT>(p.r, pl), *in = at<DT>(p.i, pl);
    const raw* z = !AGG && p.has_z ? at<DT>(p.z, pl) : nullptr;
    const Gates<VC> gates(p, d);
    float h[VC], all[VC];
    const float* from = AGG ? nullptr : p.chunked ? p.agg_h + slot * D : p.init ? p.init + pl.i * D : nullptr;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        h[v] = from ? from[d + v] : 0.f;
        all[v] = 1.f;
    }
    RowsOf<DT, VC, TT> rx, rr, ri, rz;
    auto fetch = [&](int t) {
        t += w * TT;
        rx.fetch(x, p.x.ts, t, t1 - 1, d);
        rr.fetch(r, p.r.ts, t, t1 - 1, d);
        ri.fetch(in, p.i.ts, t, t1 - 1, d);
    };
    if (t0 < t1) {
        fetch(t0);
        if (z) rz.fetch(z, p.z.ts, t0 + w * TT, t1 - 1, d);
    }
    int buf = 0;
    for (int tt = t0; tt < t1; tt += ROUND, buf ^= 1) {
        const int tw = tt + w * TT;
        float a[TT][VC], b[TT][VC], fold[VC], prod[VC];
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            float fx[VC], fr[VC], fi[VC];
            unpack<DT, VC>(rx.t[k], fx);
            unpack<DT, VC>(rr.t[k], fr);
            unpack<DT, VC>(ri.t[k], fi);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                float e2;
                keep_and_enter(gates.speed[v] * sigmoid(fr[v] + gates.rb[v]), a[k][v], e2);
                b[k][v] = root(e2) * (sigmoid(fi[v] + gates.ib[v]) * fx[v]);
            }
        }
        if (tw + TT > t1) {         // tokens behind the chunk change nothing
#pragma unroll
            for (int k = 0; k < TT; ++k)
                if (tw + k >= t1) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) a[k][v] = 1.f, b[k][v] = 0.f;
                }
        }
        if (tt + ROUND < t1) fetch(tt + ROUND);
#pragma unroll
        for (int v = 0; v < VC; ++v) fold[v] = 0.f, prod[v] = 1.f;
#pragma unroll
        for (int k = 0; k < TT; ++k)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                fold[v] = __builtin_fmaf(a[k][v], fold[v], b[k][v]);
                prod[v] *= a[k][v];
            }
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            s_h[buf][w][lane * VC + v] = fold[v];
            s_p[buf][w][lane * VC + v] = prod[v];
        }
        __syncthreads();            // one a round: the next one writes the other half
        float enter[VC] = {};
#pragma unroll
        for (int o = 0; o < WAVES; ++o)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                if (o == w) enter[v] = h[v];
                const float q = s_p[buf][o][lane * VC + v];
                h[v] = __builtin_fmaf(q, h[v], s_h[buf][o][lane * VC + v]);
                if (AGG) all[v] *= q;
            }
        if constexpr (!AGG) {
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                float y[VC], fz[VC];
                if (z) unpack<DT, VC>(rz.t[k], fz);
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    enter[v] = __builtin_fmaf(a[k][v], enter[v], b[k][v]);
                    y[v] = z ? enter[v] * (fz[v] * sigmoid(fz[v])) : enter[v];
                }
                if (act && tw + k < t1) store<DT, VC>(out + (tw + k) * D + d, y);
            }
            if (z && tt + ROUND < t1) rz.fetch(z, p.z.ts, tw + ROUND, t1 - 1, d);
        }
    }
    if (!act || w != 0) return;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        if (AGG) p.agg_h[slot * D + d + v] = h[v], p.agg_p[slot * D + d + v] = all[v];
        else if (p.state && t1 == pl.len) p.state[pl.i * D + d + v] = h[v];
    }
}

struct StepParams {
    RecurParams p;                  // rows by their batch stride
    int n, slots;
    long slot_stride;
    float* state;
    const int* idx;
};

// One token of row blockIdx.y, a thread a lane's channels. Everything it reads is asked for before the index is looked at: the
// chain from a row's index to its store is what a wave waits for.
template <int DT, int VC> __global__ __launch_bounds__(256) void k_recur_step(StepParams s) {
    typedef raw_t<DT> raw;
    const RecurParams& p = s.p;
    int row = blockIdx.y;
    const unsigned vec = blockIdx.x * 256 + threadIdx.x;
    const bool act = vec < (unsigned)p.nvec;
    const unsigned d = act ? vec * VC : 0;
    const int slot = s.idx ? s.idx[row] : row;
    raw* out = static_cast<raw*>(p.out);
    if (slot < 0 || slot >= s.slots) {
        const float zero[VC] = {};
        if (act) store<DT, VC>(out + (long)row * p.D + d, zero);
        return;
    }
    float* state = s.state + slot * s.slot_stride + d;
    float h[VC];
#pragma unroll
    for (int v = 0; v < VC; ++v) h[v] = state[v];
    Pack<DT, VC> rx, rr, ri, rz;
    auto inputs = [&](int row) {
        rx = load<DT, VC>(static_cast<const raw*>(p.x.p) + row * p.x.bs + d);
        rr = load<DT, VC>(static_cast<const raw*>(p.r.p) + row * p.r.bs + d);
        ri = load<DT, VC>(static_cast<const raw*>(p.i.p) + row * p.i.bs + d);
        if (p.has_z) rz = load<DT, VC>(static_cast<const raw*>(p.z.p) + row * p.z.bs + d);
    };
    inputs(row);
    const Gates<VC> gates(p, d);
    if (s.idx && !first_of(s.idx, row, slot)) return;
    for (;;) {
        float fx[VC], fr[VC], fi[VC], fz[VC], y[VC];
        unpack<DT, VC>(rx, fx);
        unpack<DT, VC>(rr, fr);
        unpack<DT, VC>(ri, fi);
        if (p.has_z) unpack<DT, VC>(rz, fz);
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            float a, e2;
            keep_and_enter(gates.speed[v] * sigmoid(fr[v] + gates.rb[v]), a, e2);
            h[v] = __builtin_fmaf(a, h[v], root(e2) * (sigmoid(fi[v] + gates.ib[v]) * fx[v]));
            y[v] = p.has_z ? h[v] * (fz[v] * sigmoid(fz[v])) : h[v];
        }
        if (act) store<DT, VC>(out + (long)row * p.D + d, y);
        row = s.idx ? next_of(s.idx, row, s.n, slot) : s.n;
        if (row >= s.n) break;
        inputs(row);
    }
    if (act) {
#pragma unroll
        for (int v = 0; v < VC; ++v) state[v] = h[v];
    }
}

struct FwdPlan {
    Seqs q;
    int VC;
    unsigned tiles;
    long slots;
    bool chunked;
    size_t part, bytes;             // of one aggregate, in all
};

mimo_status plan_fwd(const mamba_recur_fwd_args* a, FwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_recur(a->n, a->S, a->D, a->dtype, a->rate);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->VC = channels_of(a->D, a->dtype, packed, {&a->x, &a->r, &a->i, &a->z}, {a->out});
    pl->tiles = (unsigned)((a->D + 64 * pl->VC - 1) / (64 * pl->VC));
    const int64_t round = WAVES * tile_tokens(a->dtype), T = packed ? a->S : a->n * a->S;
    int64_t CH = (T * pl->tiles / 512 + round - 1) / round * round;
    CH = CH < round ? round : CH > 4096 ? 4096 : CH;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, (int)CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    if (!grid_fits(pl->slots * pl->tiles, 64 * WAVES)) return unsupported("the call needs more than 2^32 threads");
    pl->chunked = a->S > CH;
    pl->part = up256((size_t)pl->slots * a->D * sizeof(float));
    pl->bytes = pl->chunked ? 2 * pl->part : 0;
    return MIMO_OK;
}

template <int DT, int VC> mimo_status run_fwd(const RecurParams& p, hipStream_t st) {
    const dim3 grid((unsigned)(p.slots * p.tiles));
    if (p.chunked) {
        mimo_status s = launch(&k_recur<DT, VC, true>, grid, 64 * WAVES, 0, st, p);
        if (s != MIMO_OK) return s;
        s = launch_recur_carry<false>(p, st);
        if (s != MIMO_OK) return s;
    }
    return launch(&k_recur<DT, VC, false>, grid, 64 * WAVES, 0, st, p);
}

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_recur_fwd_workspace_size(const mamba_recur_fwd_args* a, size_t* bytes) {
    FwdPlan pl;
    const mimo_status s = plan_fwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = pl.bytes;
    return MIMO_OK;
}

mimo_status mamba_recur_fwd(const mamba_recur_fwd_args* a, void* stream) {
    FwdPlan pl;
    mimo_status s = plan_fwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (!a->x.data || !a->r.data || !a->i.data || !a->decay || !a->out) return bad("x, r, i, decay and out must not be NULL");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, pl.bytes)) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    RecurParams p{};
    p.q = pl.q, p.D = (int)a->D, p.nvec = p.D / pl.VC, p.tiles = pl.tiles, p.slots = pl.slots;
    p.has_z = a->z.data != nullptr, p.zero_tail = a->zero_tail, p.chunked = pl.chunked, p.rate = a->rate;
    p.x = rows_of(a->x, packed), p.r = rows_of(a->r, packed), p.i = rows_of(a->i, packed), p.z = rows_of(a->z, packed);
    p.decay = a->decay, p.rb = a->r_bias, p.ib = a->i_bias, p.init = a->initial_state;
    p.out = a->out, p.state = a->state;
    p.agg_h = static_cast<float*>(a->workspace);
    p.agg_p = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + pl.part);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == BF16) return pl.VC == 2 ? run_fwd<BF16, 2>(p, st) : run_fwd<BF16, 1>(p, st);
    if (a->dtype == F16) return pl.VC == 2 ? run_fwd<F16, 2>(p, st) : run_fwd<F16, 1>(p, st);
    return pl.VC == 2 ? run_fwd<F32, 2>(p, st) : run_fwd<F32, 1>(p, st);
}

mimo_status mamba_recur_step(const mamba_recur_step_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_recur(a->n, 1, a->D, a->dtype, a->rate);
    if (s != MIMO_OK) return s;
    if (!a->x.data || !a->r.data || !a->i.data || !a->decay || !a->state || !a->out) return bad("x, r, i, decay, state and out must not be NULL");
    if (a->slots < 1 || a->slots > (int64_t)1 << 30) return bad("slots must be in [1, 2^30]");
    if (!a->indices && a->slots < a->n) return bad("without indices the state needs a slot for each row");
    StepParams q{};
    RecurParams& p = q.p;
    const int VC = channels_of(a->D, a->dtype, false, {&a->x, &a->r, &a->i, &a->z}, {a->out});
    p.D = (int)a->D, p.nvec = p.D / VC, p.has_z = a->z.data != nullptr, p.rate = a->rate;
    p.x = rows_of(a->x, false), p.r = rows_of(a->r, false), p.i = rows_of(a->i, false), p.z = rows_of(a->z, false);
    p.decay = a->decay, p.rb = a->r_bias, p.ib = a->i_bias, p.out = a->out;
    q.n = (int)a->n, q.slots = (int)a->slots, q.slot_stride = a->slot_stride, q.state = a->state, q.idx = a->indices;
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)((p.nvec + 255) / 256), q.n);
    auto go = [&](auto f) { return launch(f, grid, 256, 0, st, q); };
    if (a->dtype == BF16) return VC == 2 ? go(&k_recur_step<BF16, 2>) : go(&k_recur_step<BF16, 1>);
    if (a->dtype == F16) return VC == 2 ? go(&k_recur_step<F16, 2>) : go(&k_recur_step<F16, 1>);
    return VC == 2 ? go(&k_recur_step<F32, 2>) : go(&k_recur_step<F32, 1>);
}

}  // extern "C"
