// Selective scan, forward pass and step of one token (device code of the walk: layer_scan.hpp).
#include "layer_scan.hpp"

namespace mimo {
namespace layer {
namespace {

struct StepParams {
    int n, D, G, N, Dg, slots, softplus;
    long slot_stride;
    Rows u, dt, b, c, z;            // bs: row stride
    const float *a, *d, *bias;
    float* state;
    const int* idx;
    void* out;
};

// One token of row blockIdx.y. LPC lanes share a channel, each with four consecutive states: a wave
// reads and writes whole lines of the state [D, N], which is nearly all the traffic (8 bytes a state
// against some twenty operations), and <c, h> is a sum over LPC lanes. A thread takes STEP_CH channels,
// and everything it reads is asked for before the first use: the chain from a row's index to its store is
// what a wave waits for. VEC: four states (and four of b, of c) in one
// access. 128 rows, D = 2048, N = 64 from a pool: 28.6 us, 4.8 TB/s (40 with the inputs asked for behind the index
// check; two channels 30.2, one 31.3, four 37.8 at that point).
constexpr int STEP_CH = 2;
template <int DT, int LPC, bool VEC> __global__ __launch_bounds__(256) void k_step(StepParams p) {
    typedef raw_t<DT> raw;
    constexpr int U = STEP_CH, CPB = 256 / LPC;
    const int q = threadIdx.x % LPC, n0 = q * 4;
    int row = blockIdx.y;
    const long D = p.D;
    const int slot = p.idx ? p.idx[row] : row;
    int d[U];
    bool act[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        d[j] = (blockIdx.x * U + j) * CPB + threadIdx.x / LPC;
        act[j] = d[j] < p.D;
        d[j] = act[j] ? d[j] : p.D - 1;
    }
    raw* out = static_cast<raw*>(p.out);
    if (slot < 0 || slot >= p.slots) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (act[j] && q == 0) out[row * D + d[j]] = to_raw<DT>(0.f);
        return;
    }
    float* state = p.state + slot * p.slot_stride;
    float h[U][4], a[U][4], bias[U], skip[U];
    raw r_u[U], r_dt[U], r_z[U], r_b[U][4], r_c[U][4];
    auto four = [&](const raw* x, raw (&r)[4]) {
        if (VEC) {
            Pack<DT, 4> v{};
            if (n0 < p.N) v = load<DT, 4>(x);
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = v.v[k];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = n0 + k < p.N ? x[k] : raw(0);
        }
    };
    auto inputs = [&](int row) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int at = d[j] / p.Dg * p.N + n0;
            r_u[j] = static_cast<const raw*>(p.u.p)[row * p.u.bs + d[j]];
            r_dt[j] = static_cast<const raw*>(p.dt.p)[row * p.dt.bs + d[j]];
            if (p.z.p) r_z[j] = static_cast<const raw*>(p.z.p)[row * p.z.bs + d[j]];
            four(static_cast<const raw*>(p.b.p) + row * p.b.bs + at, r_b[j]);
            four(static_cast<const raw*>(p.c.p) + row * p.c.bs + at, r_c[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < U; ++j) {
        load_states(state + (long)d[j] * p.N, n0, p.N, VEC, 0.f, h[j]);
        load_states(p.a + (long)d[j] * p.N, n0, p.N, VEC, 0.f, a[j]);
        bias[j] = p.bias ? p.bias[d[j]] : 0.f;
        skip[j] = p.d ? p.d[d[j]] : 0.f;
    }
    inputs(row);
    if (p.idx && !first_of(p.idx, row, slot)) return;
    for (;;) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float u = to_f<DT>(r_u[j]), x = to_f<DT>(r_dt[j]) + bias[j], dt = p.softplus ? softplus(x) : x, du = dt * u;
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[j][k] = __builtin_fmaf(exp2_hw(dt * decay_base(a[j][k])), h[j][k], du * to_f<DT>(r_b[j][k]));
                // places behind the last state take no part: an infinite input times their zero b is NaN
                if (n0 + (VEC ? 0 : k) < p.N) y = __builtin_fmaf(h[j][k], to_f<DT>(r_c[j][k]), y);
            }
            y = sum_lanes<LPC < 16 ? LPC : 16>(y);
            if (LPC == 32) y += __shfl_xor(y, 16);
            y = __builtin_fmaf(skip[j], u, y);
            if (p.z.p) {
                const float z = to_f<DT>(r_z[j]);
                y *= z * sigmoid(z);
            }
            if (act[j] && q == 0) out[row * D + d[j]] = to_raw<DT>(y);
        }
        row = p.idx ? next_of(p.idx, row, p.n, slot) : p.n;
        if (row >= p.n) break;
        inputs(row);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
        if (act[j]) store_states(state + (long)d[j] * p.N, n0, p.N, VEC, h[j]);
}

template <int DT, bool VEC> mimo_status launch_step(const StepParams& p, hipStream_t st) {
    auto grid = [&](int lpc) { return dim3((unsigned)(((long)p.D * lpc + 256 * STEP_CH - 1) / (256 * STEP_CH)), p.n); };
    if (p.N <= 4) return launch(&k_step<DT, 1, VEC>, grid(1), 256, 0, st, p);
    if (p.N <= 8) return launch(&k_step<DT, 2, VEC>, grid(2), 256, 0, st, p);
    if (p.N <= 16) return launch(&k_step<DT, 4, VEC>, grid(4), 256, 0, st, p);
    if (p.N <= 32) return launch(&k_step<DT, 8, VEC>, grid(8), 256, 0, st, p);
    if (p.N <= 64) return launch(&k_step<DT, 16, VEC>, grid(16), 256, 0, st, p);
    return launch(&k_step<DT, 32, VEC>, grid(32), 256, 0, st, p);
}

struct FwdPlan {
    Seqs q;
    int tpg;
    long slots;
    bool chunked;
    size_t off_sdt, bytes;
};

// Chunks are cut until about 6144 units of work (waves_for) walk, but, as a chunk costs its loads and its aggregate, not
// below 64 tokens while 2048 walk, nor below 32 at all ([8192, 1024], N = 16: 67 us at 64 tokens, 70 at 48, 74 at 96;
// [8192, 1024], N = 32: 107 us, 116 with half as many units; packed prompts [4100, 2048], N = 64: 206 us, 216 with half,
// 214 with a third more). A dense batch of 512 units is not cut, as the second walk (the aggregates) nearly doubles the work: bf16
// [4 x 4096, 8192], N = 16, 677 us, 862 cut; [4 x 4096, 4096], N = 32, 583 and 731; [16 x 1024, 4096], N = 64, 744 and 1700. But
// that counts units, and a tile is one block whatever N is: with few sequences of a wide state, or a narrow one, the blocks
// leave CUs idle, and cut it would be faster ([8192, 4096], N = 128, 64 blocks: 2961 us, 1401 cut; [2 x 8192, 4096], N = 64: 1829
// and 1310; [8 x 2048, 1024], N = 64: 460 and 361; [8 x 2048, 4096], N = 8: 504 and 313, N = 4: 516 and 242).
mimo_status plan_fwd(const mamba_scan_fwd_args* a, FwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_scan(a->n, a->S, a->D, a->G, a->N, a->dtype);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->tpg = (int)((a->D / a->G + 63) / 64);
    const int64_t waves = a->G * pl->tpg * waves_for(a->N), T = packed ? a->S : a->n * a->S;
    auto tokens_for = [&](int64_t count) { return (T * waves / count + 15) / 16 * 16; };
    int64_t CH = tokens_for(6144);
    if (CH < 64) CH = tokens_for(2048) < 64 ? tokens_for(2048) : 64;
    CH = CH < 32 ? 32 : CH > 4096 ? 4096 : CH;
    if (a->S <= 64 || (!packed && a->n * waves >= 512)) CH = (a->S + 15) / 16 * 16;
    pl->q = Seqs{a->cu_seqlens, (int)a->n, (int)a->S, (int)CH, (int)((a->S + CH - 1) / CH)};
    pl->slots = slots_of(pl->q);
    if (pl->slots > 0x7fffffffL) return unsupported("too many tokens");
    pl->chunked = a->S > CH;
    pl->off_sdt = up256((size_t)pl->slots * a->N * a->D * sizeof(float));
    pl->bytes = pl->chunked ? pl->off_sdt + up256((size_t)pl->slots * a->D * sizeof(float)) : 0;
    return MIMO_OK;
}

template <int DT> mimo_status run_fwd(const ScanParams& p, hipStream_t st) {
    if (p.chunked) {
        mimo_status s = launch_walk<DT, AGG>(p, st);
        if (s != MIMO_OK) return s;
        s = launch_carry<false>(p, st);
        if (s != MIMO_OK) return s;
    }
    return launch_walk<DT, FWD>(p, st);
}

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_scan_fwd_workspace_size(const mamba_scan_fwd_args* a, size_t* bytes) {
    FwdPlan pl;
    const mimo_status s = plan_fwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = pl.bytes;
    return MIMO_OK;
}

mimo_status mamba_scan_fwd(const mamba_scan_fwd_args* a, void* stream) {
    FwdPlan pl;
    mimo_status s = plan_fwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (!a->u.data || !a->dt.data || !a->a || !a->b.data || !a->c.data || !a->out) return bad("u, dt, a, b, c and out must not be NULL");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, pl.bytes)) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    ScanParams p{};
    p.q = pl.q;
    p.D = (int)a->D, p.G = (int)a->G, p.N = (int)a->N, p.Dg = p.D / p.G, p.tpg = pl.tpg;
    p.softplus = a->dt_softplus, p.zero_tail = a->zero_tail, p.chunked = pl.chunked, p.has_z = a->z.data != nullptr;
    p.u = rows_of(a->u, packed), p.dt = rows_of(a->dt, packed), p.b = rows_of(a->b, packed), p.c = rows_of(a->c, packed);
    p.z = rows_of(a->z, packed);
    p.a = a->a, p.d = a->d, p.bias = a->dt_bias, p.init = a->initial_state;
    p.out = a->out, p.state = a->state;
    p.agg = static_cast<float*>(a->workspace);
    p.sdt = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + pl.off_sdt);
    p.slots = pl.slots;
    p.vec = p.N % 4 == 0 && aligned(p.a, 0, 0, 16, 1) && aligned(p.init, 0, 0, 16, 1) && aligned(p.state, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == BF16 ? run_fwd<BF16>(p, st) : a->dtype == F16 ? run_fwd<F16>(p, st) : run_fwd<F32>(p, st);
}

mimo_status mamba_scan_step(const mamba_scan_step_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_scan(a->n, 1, a->D, a->G, a->N, a->dtype);
    if (s != MIMO_OK) return s;
    if (!a->u.data || !a->dt.data || !a->a || !a->b.data || !a->c.data || !a->state || !a->out)
        return bad("u, dt, a, b, c, state and out must not be NULL");
    if (a->slots < 1 || a->slots > (int64_t)1 << 30) return bad("slots must be in [1, 2^30]");
    if (!a->indices && a->slots < a->n) return bad("without indices the state needs a slot for each row");
    StepParams p{};
    p.n = (int)a->n, p.D = (int)a->D, p.G = (int)a->G, p.N = (int)a->N, p.Dg = p.D / p.G, p.slots = (int)a->slots;
    p.softplus = a->dt_softplus, p.slot_stride = a->slot_stride;
    p.u = rows_of(a->u, false), p.dt = rows_of(a->dt, false), p.b = rows_of(a->b, false), p.c = rows_of(a->c, false);
    p.z = rows_of(a->z, false);
    p.a = a->a, p.d = a->d, p.bias = a->dt_bias;
    p.state = a->state, p.idx = a->indices, p.out = a->out;
    if ((s = require_gfx950()) != MIMO_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int esz = a->dtype == F32 ? 4 : 2;
    const bool vec = p.N % 4 == 0 && aligned(p.state, p.slot_stride, 0, 16, 4) && aligned(p.a, 0, 0, 16, 1) &&
                     aligned(p.b.p, p.b.bs, 0, 4 * esz, esz) && aligned(p.c.p, p.c.bs, 0, 4 * esz, esz);
    if (a->dtype == BF16) return vec ? launch_step<BF16, true>(p, st) : launch_step<BF16, false>(p, st);
    if (a->dtype == F16) return vec ? launch_step<F16, true>(p, st) : launch_step<F16, false>(p, st);
    return vec ? launch_step<F32, true>(p, st) : launch_step<F32, false>(p, st);
}

}  // extern "C"
