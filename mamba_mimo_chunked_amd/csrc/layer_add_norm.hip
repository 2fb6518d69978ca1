// Addition to the residual stream and root-mean-square norm of the sum, forward (what it shares with the backward
// pass: layer_add_norm.hpp). A row's values stay in registers between the sum of squares and the output, so each input
// is read once and each output written once: memory binds ([8192, 2048] bf16 with a stream in fp32, to e4m3 with scales: 33 us, 5.5 TB/s),
// for single rows the launch.
//
// 8 bits: the largest |v w| of a block of columns joins the same exchange between waves as the sum of squares, and
// times r it is the largest |y|, as rounding keeps the order. Largest values are compared as bit patterns, in which a
// NaN lies above every number and stays.
#include "layer_add_norm.hpp"

namespace mimo {
namespace layer {
namespace {

struct AddNormParams {
    long rows, xs, rs;              // row strides of x, residual
    int D, kind, block, blocks;     // block: columns of a scale (0: the row), blocks: of a row
    unsigned drop;
    float factor, eps, inv;         // inv: 1 / D
    const void *x, *res;
    const long* seed;
    const float* w;
    void *sum, *out;
    float* scale;
};

typedef unsigned pair __attribute__((ext_vector_type(2)));
constexpr float LEAST = 0x1p-100f;  // a scale is made from at least this

__device__ __forceinline__ unsigned larger(unsigned a, unsigned b) { return a > b ? a : b; }
template <int CTRL> __device__ __forceinline__ unsigned max_dpp(unsigned x) {
    return larger(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}
// the largest over `lanes` = 4, 8, 16, 32 or 64 neighbouring lanes, in all of them
__device__ __forceinline__ unsigned max_lanes(unsigned x, int lanes) {
    x = max_dpp<DPP_XOR1>(x);
    x = max_dpp<DPP_XOR2>(x);
    if (lanes >= 8) x = max_dpp<DPP_HALF_MIRROR>(x);
    if (lanes >= 16) x = max_dpp<DPP_ROR8>(x);
    if (lanes >= 32) x = larger(x, __shfl_xor(x, 16));
    if (lanes >= 64) x = larger(x, __shfl_xor(x, 32));
    return x;
}

template <bool WIDE> __device__ __forceinline__ void put_bytes(unsigned char* p, int c, int D, const unsigned (&q)[2]) {
    if (WIDE ? c < D : c + NV <= D) {
        if constexpr (WIDE) *reinterpret_cast<pair*>(p + c) = pair{q[0], q[1]};
        else *reinterpret_cast<typename Loose<pair, 1>::type*>(p + c) = pair{q[0], q[1]};
    } else if (!WIDE) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (c + k < D) p[c + k] = (unsigned char)(q[k / 4] >> (8 * (k % 4)));
    }
}

template <int DT, int ST, bool WIDE, int TPR, int IT> __global__ __launch_bounds__(most_threads(TPR)) void k_add_norm(AddNormParams p) {
    constexpr int RPB = TPR ? 256 / (TPR ? TPR : 1) : 1;
    const int lanes = lanes_of_row<TPR>();
    __shared__ float s_sum[16];
    __shared__ unsigned s_max[16];
    const long item = ((long)blockIdx.y * gridDim.x + blockIdx.x) * RPB + (TPR ? threadIdx.x / (TPR ? TPR : 1) : 0);
    const bool act = item < p.rows;
    const long row = act ? item : p.rows - 1;
    const int t = lane_of_row<TPR>();
    const raw_t<DT>* x = static_cast<const raw_t<DT>*>(p.x) + row * p.xs;
    Eight<DT, WIDE> rx[IT];
    Eight<ST, WIDE> rr[IT];
    Eight<F32, WIDE> rw[IT];
#pragma unroll
    for (int k = 0; k < IT; ++k) rx[k].fetch(x, (t + k * lanes) * NV, p.D);
    if (p.res) {
#pragma unroll
        for (int k = 0; k < IT; ++k) rr[k].fetch(static_cast<const raw_t<ST>*>(p.res) + row * p.rs, (t + k * lanes) * NV, p.D);
    }
#pragma unroll
    for (int k = 0; k < IT; ++k) rw[k].fetch(p.w, (t + k * lanes) * NV, p.D);
    float v[IT][NV];
#pragma unroll
    for (int k = 0; k < IT; ++k) rx[k].read((t + k * lanes) * NV, p.D, v[k]);
    if (p.drop) {
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const unsigned keep = kept8(p.seed, t + k * lanes, (unsigned)row, p.drop);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[k][i] = keep >> i & 1 ? v[k][i] * p.factor : 0.f;
        }
    }
    if (p.res) {
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            float r[NV];
            rr[k].read((t + k * lanes) * NV, p.D, r);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[k][i] += r[i];
        }
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) q = __builtin_fmaf(v[k][i], v[k][i], q);
    if (p.sum && act) {
#pragma unroll
        for (int k = 0; k < IT; ++k) put8<ST, WIDE>(static_cast<raw_t<ST>*>(p.sum) + row * p.D, (t + k * lanes) * NV, p.D, v[k]);
    }
    unsigned top[IT] = {};
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        float w[NV];
        rw[k].read((t + k * lanes) * NV, p.D, w);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[k][i] *= w[i];
            top[k] = larger(top[k], __float_as_uint(v[k][i]) & 0x7fffffffu);
        }
    }
    if (p.kind != MAMBA_OUT_SAME) {
        if (p.block) {
#pragma unroll
            for (int k = 0; k < IT; ++k) top[k] = max_lanes(top[k], min(p.block / NV, TPR && TPR < 64 ? TPR : 64));
        } else {
#pragma unroll
            for (int k = 1; k < IT; ++k) top[0] = larger(top[0], top[k]);
            top[0] = max_lanes(top[0], TPR && TPR < 64 ? TPR : 64);
            if ((TPR == 0 || TPR > 64) && (threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = top[0];
        }
    }
    q = sum_row<TPR>(q, s_sum) * p.inv;     // its barrier also serves s_max
    const float r = 1.f / __builtin_sqrtf(q + p.eps);
    if (!act) return;
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[k][i] *= r;
    if (p.kind == MAMBA_OUT_SAME) {
#pragma unroll
        for (int k = 0; k < IT; ++k) put8<DT, WIDE>(static_cast<raw_t<DT>*>(p.out) + row * p.D, (t + k * lanes) * NV, p.D, v[k]);
        return;
    }
    if (p.block == 0) {
        if constexpr (TPR == 128) top[0] = larger(s_max[threadIdx.x >> 7 << 1], s_max[(threadIdx.x >> 7 << 1) + 1]);
        if constexpr (TPR == 0) top[0] = max_lanes((threadIdx.x & 15) < blockDim.x >> 6 ? s_max[threadIdx.x & 15] : 0u, 16);
#pragma unroll
        for (int k = 1; k < IT; ++k) top[k] = top[0];
    }
    const float most = p.kind == MAMBA_OUT_E4M3 ? 448.f : 127.f;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = (t + k * lanes) * NV;
        float m = __uint_as_float(top[k]) * r;
        const bool fine = m < __builtin_inff();     // false for NaN too
        m = m < LEAST ? LEAST : m;
        const float up = fine ? most / m : __builtin_nanf("");
        unsigned o[2] = {0, 0};
        if (p.kind == MAMBA_OUT_E4M3) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int word = __builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * h] * up, v[k][4 * h + 1] * up, 0, false);
                o[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * h + 2] * up, v[k][4 * h + 3] * up, word, true);
            }
        } else if (fine) {
#pragma unroll
            for (int i = 0; i < NV; ++i) o[i / 4] |= ((unsigned)(int)__builtin_rintf(v[k][i] * up) & 0xffu) << (8 * (i % 4));
        }
        put_bytes<WIDE>(static_cast<unsigned char*>(p.out) + row * p.D, c, p.D, o);
        const float scale = fine ? m * (1.f / most) : __builtin_nanf("");
        if (p.block == 0) {
            if (t == 0 && k == 0) p.scale[row] = scale;
        } else if (c < p.D && c % p.block == 0) p.scale[row * p.blocks + c / p.block] = scale;
    }
}

struct Run {
    AddNormParams p;
    hipStream_t st;
    template <int DT, int ST, bool WIDE> mimo_status operator()() {
        return with_row(p.D, Row<DT, ST, WIDE>{p, st});
    }
    template <int DT, int ST, bool WIDE> struct Row {
        AddNormParams p;
        hipStream_t st;
        template <int TPR, int IT> mimo_status operator()() {
            const RowShape shape = shape_of(p.D);
            // in more than one row of blocks where they are too many for one
            const long blocks = (p.rows + shape.rows - 1) / shape.rows, most = 0xffffffffL / shape.threads, along = blocks < most ? blocks : most;
            return launch(&k_add_norm<DT, ST, WIDE, TPR, IT>, dim3((unsigned)along, (unsigned)((blocks + along - 1) / along)), shape.threads,
                          0, st, p);
        }
    };
};

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_add_norm_fwd(const mamba_add_norm_fwd_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_add_norm(a->rows, a->D, a->dtype, a->eps, a->drop, a->seed);
    if (s != MIMO_OK) return s;
    if (!a->x || !a->weight || !a->out) return bad("x, weight and out must not be NULL");
    if (a->out_kind < MAMBA_OUT_SAME || a->out_kind > MAMBA_OUT_INT8) return set_error(MIMO_ERR_TYPE, "out_kind must be a MAMBA_OUT_* code");
    if (a->block != 0 && a->block != 32 && a->block != 64 && a->block != 128 && a->block != 256)
        return bad("block must be 0, 32, 64, 128 or 256");
    if (a->out_kind == MAMBA_OUT_SAME && a->block) return bad("a block of scales needs an output of 8 bits");
    if (a->out_kind != MAMBA_OUT_SAME && !a->scale) return bad("an output of 8 bits needs a scale");
    const bool stream_f32 = a->wide || a->dtype == F32;
    if (!a->sum && (a->residual || a->drop || (stream_f32 && a->dtype != F32))) return bad("sum must not be NULL where it is not x");
    AddNormParams p{};
    p.rows = a->rows, p.D = (int)a->D, p.xs = a->x_stride, p.rs = a->residual_stride;
    p.kind = a->out_kind, p.block = a->block, p.blocks = a->block ? (p.D + a->block - 1) / a->block : 1;
    p.drop = (unsigned)a->drop, p.factor = drop_factor(a->drop), p.eps = a->eps, p.inv = 1.f / (float)p.D;
    p.x = a->x, p.res = a->residual, p.seed = reinterpret_cast<const long*>(a->seed), p.w = a->weight;
    p.sum = a->sum, p.out = a->out, p.scale = a->scale;
    const int esz = a->dtype == F32 ? 4 : 2, ssz = stream_f32 ? 4 : 2;
    const bool even = p.D % NV == 0 && aligned(a->x, a->x_stride, 0, 16, esz) && aligned(a->residual, a->residual ? a->residual_stride : 0, 0, 16, ssz) &&
                      aligned(a->weight, 0, 0, 16, 1) && aligned(a->sum, 0, 0, 16, 1) && aligned(a->out, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return with_types(a->dtype, stream_f32, even, Run{p, static_cast<hipStream_t>(stream)});
}

}  // extern "C"
