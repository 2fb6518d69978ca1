// Gated linear recurrence, forward pass and step of one token (formulas, gates, rows: layer_recur.hpp).
#include "layer_recur.hpp"

namespace mimo {
namespace layer {
namespace {

constexpr int TT = 16;              // tokens of a wave
constexpr int EACH = 4;             // chunks of a wave's share of a group
constexpr int POLLS = 1 << 18;      // a wait's limit: some tenths of a second
constexpr int LINE = 64;            // counters lie this far apart: neighbours would wait for each other
typedef unsigned long long word;

__device__ __forceinline__ word look(const word* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void tell(word* p, float lo, unsigned hi) {
    __hip_atomic_store(p, (word)hi << 32 | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool there(word w) { return (unsigned)(w >> 32) != ~0u; }
__device__ __forceinline__ float low(word w) { return __uint_as_float((unsigned)w); }
__device__ __forceinline__ float high(word w) { return __uint_as_float((unsigned)(w >> 32)); }

// Before a call of several chunks: no step is told yet, no chunk taken.
__global__ __launch_bounds__(256) void k_recur_clear(RecurParams p) {
    const long step = (long)gridDim.x * 256, at = (long)blockIdx.x * 256 + threadIdx.x;
    for (long k = at; k < p.words; k += step) p.told[k] = ~word(0);
    for (long k = at; k <= p.tiles * LINE; k += step) p.taken[k] = 0;
}

// The outputs, in one pass over the inputs. A block takes one chunk of WAVES * TT tokens by 64 channels, all of it in registers:
// it joins its tokens' steps, tells the joined step (last state from zero, product of a; one word of 64 bits a channel) to the
// chunks behind it, joins those of the chunks in front, and walks its tokens from there. The chunks of a sequence are joined in
// groups of WAVES * EACH: a chunk looks at those of its group, and at the state that the last chunk of the group in front tells. The order in
// which steps are joined is fixed, so equal inputs give equal bits. (Scans in one pass whose blocks look back: D. Merrill and M. Garland, "Single-pass
// parallel prefix scan with decoupled look-back", 2016.)
// Every wait ends: a block takes the next chunk of its tile from a counter, so that whatever it waits for belongs to a block that runs
// already, and a chunk's step is told before its block waits, a group's state after waiting for lower chunks alone. cu_seqlens that
// decrease may leave a word that nobody tells: POLLS ends the first such wait, its mark behind the counters all others, and outputs
// are NaN (the host hears nothing of it: the call has returned). A word holds value and mark, so no fence is needed.
// [8192, 2048] bf16: 42 us, 4.0 TB/s, vector units 46 % busy; in two passes over the inputs 82. What is left is that a block loads, joins,
// waits and walks one after the other, with three blocks of 79 registers on a CU.
// AUX: the policy of its accesses: past the last-level cache where the call is larger than it (bf16, D = 2048: [8 x 2048] 75 us, 79 through it,
// [1 x 8192], which is smaller, 43 and 46, but what reads the outputs next finds them there).
template <int DT, bool GATE, int AUX, int WAVES> __global__ __launch_bounds__(64 * WAVES, 6) void k_recur(RecurParams p) {
    typedef raw_t<DT> raw;
    constexpr int CH = WAVES * TT, GROUP = WAVES * EACH;
    __shared__ float s_h[WAVES][64], s_p[WAVES][64], s_gh[WAVES][64], s_gp[WAVES][64];
    __shared__ unsigned s_slot;
    const unsigned tile = blockIdx.x % p.tiles;
    unsigned slot = blockIdx.x / p.tiles;
    if (p.chunked) {
        if (threadIdx.x == 0) s_slot = __hip_atomic_fetch_add(p.taken + tile * LINE, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        slot = __builtin_amdgcn_readfirstlane(s_slot);
    }
    const Place pl = place_by_wave(p.q, slot);
    if (!pl.ok) return;
    const int t0 = pl.j * CH, t1 = min(t0 + CH, pl.len);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tw = t0 + w * TT, left = t1 - tw;
    const bool act = tile * 64 + lane < (unsigned)p.D;
    const unsigned d = act ? tile * 64 + lane : (unsigned)p.D - 1, db = d * sizeof(raw);     // of the same tile: its words are told
    const long D = p.D;
    const auto out = buffer_of(static_cast<raw*>(p.out) + (recur_row(p.q, pl) + tw) * D);
    const unsigned step = (unsigned)D * sizeof(raw);
    if (pl.i == p.q.n) {            // behind the last sequence
        const float zero[1] = {};
        if (p.zero_tail && act)
            for (int k = 0; k < min(left, TT); ++k) store_at<DT, 1>(out, db, k * step, zero);
        return;
    }
    const int group = pl.j / GROUP;
    float h = group == 0 && p.init ? p.init[pl.i * D + d] : 0.f;
    if (t0 < t1) {
        RowsOf<DT, 1, TT, AUX> rx, rr, ri, rz;
        float a[TT], b[TT], fold = 0.f, prod = 1.f;
        if (left > 0) {             // a short sequence leaves waves without tokens
            rx.place(p.x, pl, p.D, tw, t1), rr.place(p.r, pl, p.D, tw, t1), ri.place(p.i, pl, p.D, tw, t1);
            if constexpr (GATE) rz.place(p.z, pl, p.D, tw, t1);
#pragma unroll
            for (int k = 0; k < TT; ++k) rx.fetch(k, db), rr.fetch(k, db), ri.fetch(k, db);
            const Gates<1> gates(p, d);
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                float e2;
                keep_and_enter(speed_of(gates, 0, k, left) * gates.open(to_f<DT>(rr.t[k].v[0]), gates.rb[0]), a[k], e2);
                b[k] = root(e2) * (gates.open(to_f<DT>(ri.t[k].v[0]), gates.ib[0]) * to_f<DT>(rx.t[k].v[0]));
            }
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                fold = __builtin_fmaf(a[k], fold, b[k]);
                prod *= a[k];
            }
        }
        s_h[w][lane] = fold;
        s_p[w][lane] = prod;
        __syncthreads();
        const bool last = t1 == pl.len, closes = !last && pl.j % GROUP == GROUP - 1;
        word* const ends = p.told + p.slots * D;
        if (w == 0 && !last && !closes) {
            float hh = 0.f, pp = 1.f;
#pragma unroll
            for (int o = 0; o < WAVES; ++o) {
                hh = __builtin_fmaf(s_p[o][lane], hh, s_h[o][lane]);
                pp *= s_p[o][lane];
            }
            // a NaN that came in must not look like a word that is not there yet
            if (act) tell(p.told + slot * D + d, hh, pp == pp ? __float_as_uint(pp) : 0x7fc00000u);
        }
        if constexpr (GATE) {       // late, in the registers that x, r and i have left ([8 x 2048, 2048] bf16 75 us, asked for with them 78)
            if (left > 0) {
#pragma unroll
                for (int k = 0; k < TT; ++k) rz.fetch(k, db);
            }
        }
        if (pl.j > 0) {
            // this wave's share of the group's chunks in front, and in wave 0 the state that enters the group
            const int first = group * GROUP + w * EACH, before = pl.j - first;      // how many of them: up to EACH
            const word* from = p.told + ((long)slot - before) * D + d;
            const word* base = ends + (long)((slot - pl.j + group * GROUP - 1) / GROUP) * D + d;
            const bool wants = group > 0 && w == 0;
            word told[EACH], enters;
            for (int poll = 0;; ++poll) {
                bool all = true;
#pragma unroll
                for (int e = 0; e < EACH; ++e)
                    if (e < before) told[e] = look(from + e * D);
                if (wants) enters = look(base);
#pragma unroll
                for (int e = 0; e < EACH; ++e)
                    if (e < before) all = all && there(told[e]);
                if (wants) all = all && there(enters);
                if (__all(all) || __hip_atomic_load(p.taken + p.tiles * LINE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) break;
                if (poll == POLLS) __hip_atomic_store(p.taken + p.tiles * LINE, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __builtin_amdgcn_s_sleep(4);
            }
            if (wants) h = there(enters) ? low(enters) : __builtin_nanf("");
            float gh = w == 0 ? h : 0.f, gp = 1.f;
#pragma unroll
            for (int e = 0; e < EACH; ++e)
                if (e < before) {
                    gh = __builtin_fmaf(high(told[e]), gh, low(told[e]));
                    gp *= high(told[e]);
                }
            s_gh[w][lane] = gh;
            s_gp[w][lane] = gp;
            __syncthreads();
            h = s_gh[0][lane];      // from the state that enters the group
#pragma unroll
            for (int o = 1; o < WAVES; ++o) h = __builtin_fmaf(s_gp[o][lane], h, s_gh[o][lane]);
        }
        float enter = 0.f;
#pragma unroll
        for (int o = 0; o < WAVES; ++o) {
            if (o == w) enter = h;
            h = __builtin_fmaf(s_p[o][lane], h, s_h[o][lane]);
        }
        if (closes && w == 0 && act) tell(ends + (long)(slot / GROUP) * D + d, h, 0u);
        unsigned row = 0;
        if (act && left > 0) {
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                enter = __builtin_fmaf(a[k], enter, b[k]);
                float y[1] = {enter};
                if constexpr (GATE) {
                    const float z = to_f<DT>(rz.t[k].v[0]);
                    y[0] *= z * sigmoid(z);
                }
                if (k < left) store_at<DT, 1, AUX>(out, db, row, y);
                row += step;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (act && w == 0 && p.state && t1 == pl.len) p.state[pl.i * D + d] = h;
}

struct StepParams {
    RecurParams p;                  // rows by their batch stride
    int n, slots;
    long slot_stride;
    float* state;
    const int* idx;
};

// One token of row blockIdx.y, a thread a lane's channels. Everything it reads is asked for before the index is looked at: the
// chain from a row's index to its store is what a wave waits for. One row of 1024 channels 3.0 us, 128 of 2048 from a pool 4.4.
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
            keep_and_enter(gates.speed[v] * gates.open(fr[v], gates.rb[v]), a, e2);
            h[v] = __builtin_fmaf(a, h[v], root(e2) * (gates.open(fi[v], gates.ib[v]) * fx[v]));
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
    unsigned tiles;
    int waves;
    long slots;
    bool chunked;
    long words;
    size_t told, bytes;             // of the words, in all
};

mimo_status plan_fwd(const mamba_recur_fwd_args* a, FwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_recur(a->n, a->S, a->D, a->dtype, a->rate);
    if (s != MIMO_OK || (s = check_strides(a->S, {&a->x, &a->r, &a->i, &a->z})) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->tiles = (unsigned)((a->D + 63) / 64);
    pl->waves = waves_of(packed, a->n, a->S, TT);
    const int CH = pl->waves * TT, GROUP = pl->waves * EACH;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    if (!grid_fits(pl->slots * pl->tiles, 64 * pl->waves)) return unsupported("the call needs more than 2^32 threads");
    pl->chunked = a->S > CH;
    // a word of every chunk and of every group's end
    pl->words = pl->chunked ? (pl->slots + pl->slots / GROUP + 1) * (long)a->D : 0;
    pl->told = up256((size_t)pl->words * sizeof(word));
    pl->bytes = pl->chunked ? pl->told + up256((pl->tiles * LINE + 1) * sizeof(unsigned)) : 0;
    return MIMO_OK;
}

template <int DT, bool GATE, int WAVES> mimo_status run_fwd(const RecurParams& p, hipStream_t st) {
    if (p.chunked) {
        const long blocks = (p.words + 1023) / 1024;
        const mimo_status s = launch(&k_recur_clear, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), 256, 0, st, p);
        if (s != MIMO_OK) return s;
    }
    const dim3 grid((unsigned)(p.slots * p.tiles));
    return passes_by<DT>(p.q, p.D, GATE ? 5 : 4) ? launch(&k_recur<DT, GATE, NT, WAVES>, grid, 64 * WAVES, 0, st, p)
                                                 : launch(&k_recur<DT, GATE, 0, WAVES>, grid, 64 * WAVES, 0, st, p);
}

template <int DT, bool GATE> mimo_status run_waves(const FwdPlan& pl, const RecurParams& p, hipStream_t st) {
    return pl.waves == 8 ? run_fwd<DT, GATE, 8>(p, st) : pl.waves == 4 ? run_fwd<DT, GATE, 4>(p, st) : run_fwd<DT, GATE, 2>(p, st);
}
template <int DT> mimo_status run_type(const FwdPlan& pl, const RecurParams& p, hipStream_t st) {
    return p.has_z ? run_waves<DT, true>(pl, p, st) : run_waves<DT, false>(pl, p, st);
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
    p.q = pl.q, p.D = (int)a->D, p.tiles = pl.tiles, p.slots = pl.slots;
    p.has_z = a->z.data != nullptr, p.zero_tail = a->zero_tail, p.chunked = pl.chunked, p.rate = a->rate;
    p.x = rows_of(a->x, packed), p.r = rows_of(a->r, packed), p.i = rows_of(a->i, packed), p.z = rows_of(a->z, packed);
    p.decay = a->decay, p.rb = a->r_bias, p.ib = a->i_bias, p.init = a->initial_state;
    p.out = a->out, p.state = a->state;
    p.words = pl.words, p.told = static_cast<unsigned long long*>(a->workspace);
    p.taken = reinterpret_cast<unsigned*>(static_cast<char*>(a->workspace) + pl.told);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == BF16) return run_type<BF16>(pl, p, st);
    return a->dtype == F16 ? run_type<F16>(pl, p, st) : run_type<F32>(pl, p, st);
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
    return go(&k_recur_step<F32, 1>);
}

}  // extern "C"
