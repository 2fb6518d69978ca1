// Addition to the residual stream and root-mean-square norm of the sum, backward (formulas: layer_add_norm.hpp). A block
// takes every nth row, keeps its share of dw in registers over them and leaves one partial row, added up in order by
// k_add_norm_sums, and asks for its next row before it works on one. Memory binds: [4100, 4096] bf16 with dropout 37 us for 168 MB, the sums
// of 256 rows 4.
#include "layer_add_norm.hpp"

namespace mimo {
namespace layer {
namespace {

struct AddNormBwdParams {
    long rows, gs, ss, ds;          // row strides of dout, sum, dsum
    int D, nblk;
    unsigned drop;
    float factor, eps, inv;
    const void *dout, *sum, *dsum;
    const long* seed;
    const float* w;
    void *dx, *dres;
    float *part, *dw;               // part: [nblk][D]
};

typedef float f4v __attribute__((ext_vector_type(4)));
// Eight floats of a thread for each of its accesses: in registers, or, where it has two (1024 threads, 128 registers each), in LDS of its own
// ([1024, 16384] bf16 42 us; with registers in scratch memory, and half as many blocks, 87).
template <int IT> struct Held {
    float v[IT][NV];
    __device__ __forceinline__ void put(f4v*, int k, const float (&x)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[k][i] = x[i];
    }
    __device__ __forceinline__ void get(const f4v*, int k, float (&x)[NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = v[k][i];
    }
};
template <> struct Held<2> {
    __device__ __forceinline__ void put(f4v* s, int k, const float (&x)[NV]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) s[(2 * k + j) * 1024 + threadIdx.x] = f4v{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
    }
    __device__ __forceinline__ void get(const f4v* s, int k, float (&x)[NV]) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f4v q = s[(2 * k + j) * 1024 + threadIdx.x];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * j + i] = q[i];
        }
    }
};

template <int DT, int ST, bool WIDE, int TPR, int IT> __global__ __launch_bounds__(most_threads(TPR)) void k_add_norm_bwd(AddNormBwdParams p) {
    constexpr int RPB = TPR ? 256 / (TPR ? TPR : 1) : 1;
    // fp32 [8192, 2047] 52 us, 65 without; bf16 [1024, 16384] 42 and 46; but bf16 [4100, 4096] with dropout 46 and 40
    constexpr bool LATE = !WIDE || IT == 2;
    __shared__ float s[2][16];
    __shared__ float s_dw[RPB > 1 ? RPB * TPR * NV : 1];
    __shared__ f4v s_w[IT == 2 ? 4096 : 1], s_sum[IT == 2 ? 4096 : 1];
    const int t = lane_of_row<TPR>(), lanes = lanes_of_row<TPR>(), sub = TPR ? threadIdx.x / (TPR ? TPR : 1) : 0;
    Held<IT> w, dw;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        Eight<F32, WIDE> rw;
        float x[NV];
        const float zero[NV] = {};
        rw.fetch(p.w, (t + k * lanes) * NV, p.D);
        rw.read((t + k * lanes) * NV, p.D, x);
        w.put(s_w, k, x);
        dw.put(s_sum, k, zero);
    }
    Eight<ST, WIDE> rv[IT], rs[IT];
    Eight<DT, WIDE> rg[IT];
    auto fetch = [&](long row) {
        row = row < p.rows ? row : p.rows - 1;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = (t + k * lanes) * NV;
            rv[k].fetch(static_cast<const raw_t<ST>*>(p.sum) + row * p.ss, c, p.D);
            rg[k].fetch(static_cast<const raw_t<DT>*>(p.dout) + row * p.gs, c, p.D);
        }
    };
    // dsum, which a row needs last: asked for with the others, or, for the registers' sake, when the row before is done
    auto fetch_dsum = [&](long row) {
        row = row < p.rows ? row : p.rows - 1;
        if (p.dsum) {
#pragma unroll
            for (int k = 0; k < IT; ++k) rs[k].fetch(static_cast<const raw_t<ST>*>(p.dsum) + row * p.ds, (t + k * lanes) * NV, p.D);
        }
    };
    const long step = (long)gridDim.x * RPB;
    fetch((long)blockIdx.x * RPB + sub);
    fetch_dsum((long)blockIdx.x * RPB + sub);
    for (long row0 = (long)blockIdx.x * RPB; row0 < p.rows; row0 += step) {
        const bool act = row0 + sub < p.rows;
        const long row = act ? row0 + sub : p.rows - 1;
        unsigned keep[IT];
        if (p.drop) {
#pragma unroll
            for (int k = 0; k < IT; ++k) keep[k] = kept8(p.seed, t + k * lanes, (unsigned)row, p.drop);
        }
        float v[IT][NV], g[IT][NV], d[IT][NV] = {}, q = 0.f, m = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            rv[k].read((t + k * lanes) * NV, p.D, v[k]);
            rg[k].read((t + k * lanes) * NV, p.D, g[k]);
            if (!LATE && p.dsum) rs[k].read((t + k * lanes) * NV, p.D, d[k]);
#pragma unroll
            for (int i = 0; i < NV; ++i) q = __builtin_fmaf(v[k][i], v[k][i], q);
        }
        if (row0 + step < p.rows) {
            fetch(row0 + step + sub);
            if (!LATE) fetch_dsum(row0 + step + sub);
        }
        q = sum_row<TPR>(q, s[0]) * p.inv;
        const float r = 1.f / __builtin_sqrtf(q + p.eps);
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            float ww[NV], sum[NV];
            w.get(s_w, k, ww);
            dw.get(s_sum, k, sum);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[k][i] *= r;
                if (act) sum[i] = __builtin_fmaf(g[k][i], v[k][i], sum[i]);
                g[k][i] *= ww[i];
                m = __builtin_fmaf(g[k][i], v[k][i], m);
            }
            dw.put(s_sum, k, sum);
        }
        m = sum_row<TPR>(m, s[1]) * p.inv;
        if (!act) continue;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = (t + k * lanes) * NV;
            float dv[NV];
            if (LATE && p.dsum) rs[k].read(c, p.D, d[k]);
#pragma unroll
            for (int i = 0; i < NV; ++i) dv[i] = __builtin_fmaf(r, __builtin_fmaf(-v[k][i], m, g[k][i]), d[k][i]);
            if (p.dres) put8<ST, WIDE>(static_cast<raw_t<ST>*>(p.dres) + row * p.D, c, p.D, dv);
            if (p.drop) {
#pragma unroll
                for (int i = 0; i < NV; ++i) dv[i] = keep[k] >> i & 1 ? dv[i] * p.factor : 0.f;
            }
            put8<DT, WIDE>(static_cast<raw_t<DT>*>(p.dx) + row * p.D, c, p.D, dv);
        }
        if (LATE && row0 + step < p.rows) fetch_dsum(row0 + step + sub);
    }
    float* part = p.part + (long)blockIdx.x * p.D;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = (t + k * lanes) * NV;
        float sum[NV];
        dw.get(s_sum, k, sum);
        if constexpr (RPB > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s_dw[threadIdx.x * NV + i] = sum[i];
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    for (int y = 1; y < RPB; ++y) sum[i] += s_dw[(y * TPR + t) * NV + i];
            }
        }
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c + i < p.D) part[c + i] = sum[i];
        }
    }
}

__global__ __launch_bounds__(256) void k_add_norm_sums(AddNormBwdParams p) {
    column_sums(p.part, p.D, p.nblk, (long)blockIdx.x * SUM_COLS, p.D, [&](long col, float s) { p.dw[col] = s; });
}

// blocks: as many a CU as have 512 threads, none without a row of its own
int64_t blocks_of(const mamba_add_norm_bwd_args* a) {
    const RowShape shape = shape_of(a->D);
    const int64_t want = 256 * ((511 + shape.threads) / shape.threads), have = (a->rows + shape.rows - 1) / shape.rows;
    return have < want ? have : want;
}

struct Run {
    AddNormBwdParams p;
    hipStream_t st;
    template <int DT, int ST, bool WIDE> mimo_status operator()() {
        return with_row(p.D, Row<DT, ST, WIDE>{p, st});
    }
    template <int DT, int ST, bool WIDE> struct Row {
        AddNormBwdParams p;
        hipStream_t st;
        template <int TPR, int IT> mimo_status operator()() {
            const mimo_status s = launch(&k_add_norm_bwd<DT, ST, WIDE, TPR, IT>, dim3(p.nblk), shape_of(p.D).threads, 0, st, p);
            if (s != MIMO_OK) return s;
            return launch(&k_add_norm_sums, dim3((unsigned)((p.D + SUM_COLS - 1) / SUM_COLS)), 256, 0, st, p);
        }
    };
};

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_add_norm_bwd_workspace_size(const mamba_add_norm_bwd_args* a, size_t* bytes) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_add_norm(a->rows, a->D, a->dtype, a->eps, a->drop, a->seed);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = up256((size_t)blocks_of(a) * a->D * sizeof(float));
    return MIMO_OK;
}

mimo_status mamba_add_norm_bwd(const mamba_add_norm_bwd_args* a, void* stream) {
    size_t need = 0;
    mimo_status s = mamba_add_norm_bwd_workspace_size(a, &need);
    if (s != MIMO_OK) return s;
    if (!a->dout || !a->sum || !a->weight || !a->dx || !a->dweight) return bad("dout, sum, weight, dx and dweight must not be NULL");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != MIMO_OK) return s;
    const bool stream_f32 = a->wide || a->dtype == F32;
    AddNormBwdParams p{};
    p.rows = a->rows, p.D = (int)a->D, p.gs = a->dout_stride, p.ss = a->sum_stride, p.ds = a->dsum_stride;
    p.drop = (unsigned)a->drop, p.factor = drop_factor(a->drop), p.eps = a->eps, p.inv = 1.f / (float)p.D;
    p.dout = a->dout, p.sum = a->sum, p.dsum = a->dsum, p.seed = reinterpret_cast<const long*>(a->seed), p.w = a->weight;
    p.dx = a->dx, p.dres = a->dresidual, p.part = static_cast<float*>(a->workspace), p.dw = a->dweight;
    p.nblk = (int)blocks_of(a);
    const int esz = a->dtype == F32 ? 4 : 2, ssz = stream_f32 ? 4 : 2;
    const bool even = p.D % NV == 0 && aligned(a->dout, a->dout_stride, 0, 16, esz) && aligned(a->sum, a->sum_stride, 0, 16, ssz) &&
                      aligned(a->dsum, a->dsum ? a->dsum_stride : 0, 0, 16, ssz) && aligned(a->weight, 0, 0, 16, 1) && aligned(a->dx, 0, 0, 16, 1) &&
                      aligned(a->dresidual, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return with_types(a->dtype, stream_f32, even, Run{p, static_cast<hipStream_t>(stream)});
}

}  // extern "C"
