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
// against some twenty operations), and <c, h> is a sum over LPC lanes. VEC: 16-byte accesses.
template <int DT, int LPC, bool VEC> __global__ __launch_bounds__(256) void k_step(StepParams p) {
    typedef raw_t<DT> raw;
    const int q = threadIdx.x % LPC, d0 = blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
    const bool act = d0 < p.D;
    const int d = act ? d0 : p.D - 1;
    int row = blockIdx.y;
    const long D = p.D;
    raw* out = static_cast<raw*>(p.out) + d;
    const int slot = p.idx ? p.idx[row] : row;
    if (slot < 0 || slot >= p.slots) {
        if (act && q == 0) out[row * D] = to_raw<DT>(0.f);
        return;
    }
    const int n0 = q * 4, g = d / p.Dg;
    float* state = p.state + slot * p.slot_stride + (long)d * p.N + n0;
    const float* pa = p.a + (long)d * p.N + n0;
    float h[4] = {}, a[4] = {};
    if (VEC) {
        if (n0 < p.N) {
            const float4 x = *reinterpret_cast<const float4*>(state), y = *reinterpret_cast<const float4*>(pa);
            h[0] = x.x, h[1] = x.y, h[2] = x.z, h[3] = x.w;
            a[0] = y.x, a[1] = y.y, a[2] = y.z, a[3] = y.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < p.N) h[k] = state[k], a[k] = pa[k];
    }
    const float bias = p.bias ? p.bias[d] : 0.f, skip = p.d ? p.d[d] : 0.f;
    if (p.idx && !first_of(p.idx, row, slot)) return;
    for (;;) {
        const float u = to_f<DT>(static_cast<const raw*>(p.u.p)[row * p.u.bs + d]);
        const float x = to_f<DT>(static_cast<const raw*>(p.dt.p)[row * p.dt.bs + d]) + bias;
        const raw* b = static_cast<const raw*>(p.b.p) + row * p.b.bs + g * p.N + n0;
        const raw* c = static_cast<const raw*>(p.c.p) + row * p.c.bs + g * p.N + n0;
        const float dt = p.softplus ? softplus(x) : x, du = dt * u;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < p.N) {
                h[k] = __builtin_fmaf(exp2_hw(dt * (a[k] * LOG2E)), h[k], du * to_f<DT>(b[k]));
                y = __builtin_fmaf(h[k], to_f<DT>(c[k]), y);
            }
        y = sum_lanes<LPC < 16 ? LPC : 16>(y);
        if (LPC == 32) y += __shfl_xor(y, 16);
        y = __builtin_fmaf(skip, u, y);
        if (p.z.p) {
            const float z = to_f<DT>(static_cast<const raw*>(p.z.p)[row * p.z.bs + d]);
            y *= z * sigmoid(z);
        }
        if (act && q == 0) out[row * D] = to_raw<DT>(y);
        row = p.idx ? next_of(p.idx, row, p.n, slot) : p.n;
        if (row >= p.n) break;
    }
    if (!act) return;
    if (VEC) {
        if (n0 < p.N) *reinterpret_cast<float4*>(state) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < p.N) state[k] = h[k];
    }
}

template <int DT, bool VEC> mimo_status launch_step(const StepParams& p, hipStream_t st) {
    auto grid = [&](int lpc) { return dim3((unsigned)(((long)p.D * lpc + 255) / 256), p.n); };
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

// One wave per SIMD keeps the vector units busy (NS independent recurrences), two hide the loads: chunks
// are cut until about 2048 waves walk, but not below 32 tokens. A second walk (the aggregates) nearly
// doubles the work, so half the GPU's waves (512) without chunks are as good as chunks.
mimo_status plan_fwd(const mamba_scan_fwd_args* a, FwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_scan(a->n, a->S, a->D, a->G, a->N, a->dtype);
    if (s != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    pl->tpg = (int)((a->D / a->G + 63) / 64);
    const int64_t waves = a->G * pl->tpg * waves_for(a->N), T = packed ? a->S : a->n * a->S;
    int64_t CH = (T * waves / 3072 + 15) / 16 * 16;
    if (CH < 64) CH = (T * waves / 2048 + 15) / 16 * 16 < 64 ? (T * waves / 2048 + 15) / 16 * 16 : 64;
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
        s = launch_carry<false>(p, p.q.nc, st);
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
    const bool vec = p.N % 4 == 0 && aligned(p.state, p.slot_stride, 0, 16, 4) && aligned(p.a, 0, 0, 16, 1);
    if (a->dtype == BF16) return vec ? launch_step<BF16, true>(p, st) : launch_step<BF16, false>(p, st);
    if (a->dtype == F16) return vec ? launch_step<F16, true>(p, st) : launch_step<F16, false>(p, st);
    return vec ? launch_step<F32, true>(p, st) : launch_step<F32, false>(p, st);
}

}  // extern "C"
