// Gated group norm over the channels of a row, forward and backward.
//
//   v = x silu(z) (gate before) or x;  m = mean(v) or 0;  r = 1 / sqrt(mean((v - m)^2) + eps)
//   hat = (v - m) r;  p = hat w + b;   out = p silu(z) (gate after), silu(p), or p
//   backward: dp from dout;  dw = sum dp hat;  db = sum dp;  q = dp w;
//             dv = r (q - [mean(q)] - hat mean(q hat)), then through the gate
//
// TPR threads share a group of a row and keep it in registers (IT accesses of VEC elements each), so
// every input is read once: memory binds. Sums run over lanes; groups that need a whole block join the
// waves' sums in LDS. The variance is taken from the centred values, not from a difference of sums.
// The backward pass gives each block one group and every nth row, keeps the sums for dw and db in
// registers over the rows, and leaves one partial row a block, added up in order by k_norm_sums.
#include "layer.hpp"

namespace mimo {
namespace layer {
namespace {

struct NormParams {
    long rows, xs, zs, gs;          // row strides of x, z, dout
    int D, G, W;                    // channels, groups, channels of a group
    int center, after, silu, has_z;
    float eps;
    const void *x, *z, *dout;
    const float *w, *b;
    void *out, *dz;                 // out: also dx
    float *part, *dw, *db;          // part: [blocks][2][D]
    int nblk;
};

// the sum over the TPR threads of a group, in all of them; `s`: LDS of four floats, safe to use again after
// the next call on another one
template <int TPR> __device__ __forceinline__ float sum_group(float x, float* s) {
    if constexpr (TPR <= 64) return sum_wave<TPR>(x);
    else {
        x = sum_wave<64>(x);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        return (s[0] + s[1]) + (s[2] + s[3]);
    }
}

template <int DT, int VEC, int TPR, int IT> struct Group {
    typedef raw_t<DT> raw;
    float x[IT][VEC], z[IT][VEC], hat[IT][VEC];
    float r;
    __device__ __forceinline__ static int col(int k) { return (threadIdx.x % TPR + k * TPR) * VEC; }
    // element col(k) of row data at p, zeros past the group
    __device__ __forceinline__ static void read(const raw* p, int W, float (&x)[IT][VEC]) {
        Pack<DT, VEC> t[IT];
#pragma unroll
        for (int k = 0; k < IT; ++k)
            if (col(k) < W) t[k] = load<DT, VEC>(p + col(k));
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            if (col(k) < W) unpack<DT, VEC>(t[k], x[k]);
            else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[k][v] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void normalise(const NormParams& p, float (*s)[4]) {
        const float inv = 1.f / (float)p.W;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                hat[k][v] = x[k][v];
                if (p.has_z && !p.after) hat[k][v] *= z[k][v] * sigmoid(z[k][v]);
                m += hat[k][v];
            }
        if (p.center) {
            m = sum_group<TPR>(m, s[0]) * inv;
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) hat[k][v] = col(k) < p.W ? hat[k][v] - m : 0.f;
        }
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) q = __builtin_fmaf(hat[k][v], hat[k][v], q);
        q = sum_group<TPR>(q, s[1]) * inv;
        r = 1.f / __builtin_sqrtf(q + p.eps);
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) hat[k][v] *= r;
    }
};

template <int DT, int VEC, int TPR, int IT> __global__ __launch_bounds__(256) void k_norm_fwd(NormParams p) {
    typedef raw_t<DT> raw;
    typedef Group<DT, VEC, TPR, IT> Grp;
    __shared__ float s[2][4];
    const long item = (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR, items = p.rows * p.G;
    const bool act = item < items;
    const long row = act ? item / p.G : 0;
    const int c0 = act ? (int)(item - row * p.G) * p.W : 0;
    Grp g;
    Grp::read(static_cast<const raw*>(p.x) + row * p.xs + c0, p.W, g.x);
    if (p.has_z) Grp::read(static_cast<const raw*>(p.z) + row * p.zs + c0, p.W, g.z);
    g.normalise(p, s);
    if (!act) return;
    raw* out = static_cast<raw*>(p.out) + row * p.D + c0;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = Grp::col(k);
        if (c >= p.W) continue;
        float y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float t = g.hat[k][v] * p.w[c0 + c + v];
            if (p.b) t += p.b[c0 + c + v];
            if (p.has_z && p.after) t *= g.z[k][v] * sigmoid(g.z[k][v]);
            else if (p.silu) t *= sigmoid(t);
            y[v] = t;
        }
        store<DT, VEC>(out + c, y);
    }
}

template <int DT, int VEC, int TPR, int IT> __global__ __launch_bounds__(256) void k_norm_bwd(NormParams p) {
    typedef raw_t<DT> raw;
    typedef Group<DT, VEC, TPR, IT> Grp;
    constexpr int RPB = 256 / TPR;
    __shared__ float s[4][4];
    __shared__ float s_sum[RPB > 1 ? 256 * VEC : 1];
    const int sub = threadIdx.x / TPR, c0 = blockIdx.y * p.W;
    const float inv = 1.f / (float)p.W;
    float w[IT][VEC], b[IT][VEC], dw[IT][VEC] = {}, db[IT][VEC] = {};
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int c = Grp::col(k) + v;
            w[k][v] = c < p.W ? p.w[c0 + c] : 0.f;
            b[k][v] = c < p.W && p.b ? p.b[c0 + c] : 0.f;
        }
    for (long row0 = (long)blockIdx.x * RPB; row0 < p.rows; row0 += (long)gridDim.x * RPB) {
        const bool act = row0 + sub < p.rows;
        const long row = act ? row0 + sub : p.rows - 1;
        Grp g;
        float dy[IT][VEC];
        Grp::read(static_cast<const raw*>(p.x) + row * p.xs + c0, p.W, g.x);
        if (p.has_z) Grp::read(static_cast<const raw*>(p.z) + row * p.zs + c0, p.W, g.z);
        Grp::read(static_cast<const raw*>(p.dout) + row * p.gs + c0, p.W, dy);
        g.normalise(p, s);
        float dz[IT][VEC], m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hat = g.hat[k][v], t = __builtin_fmaf(hat, w[k][v], b[k][v]);
                if (p.has_z && p.after) {
                    const float z = g.z[k][v], gate = sigmoid(z);
                    dz[k][v] = dy[k][v] * t * silu_slope(z, gate);
                    dy[k][v] *= z * gate;
                } else if (p.silu) dy[k][v] *= silu_slope(t, sigmoid(t));
                if (act) {
                    dw[k][v] = __builtin_fmaf(dy[k][v], hat, dw[k][v]);
                    db[k][v] += dy[k][v];
                }
                dy[k][v] *= w[k][v];
                m1 += dy[k][v];
                m2 = __builtin_fmaf(dy[k][v], hat, m2);
            }
        m1 = p.center ? sum_group<TPR>(m1, s[2]) * inv : 0.f;
        m2 = sum_group<TPR>(m2, s[3]) * inv;
        raw* dx = static_cast<raw*>(p.out) + row * p.D + c0;
        raw* pz = p.has_z ? static_cast<raw*>(p.dz) + row * p.D + c0 : nullptr;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = Grp::col(k);
            if (!act || c >= p.W) continue;
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o[v] = g.r * (dy[k][v] - m1 - g.hat[k][v] * m2);
                if (p.has_z && !p.after) {
                    const float z = g.z[k][v], gate = sigmoid(z);
                    dz[k][v] = o[v] * g.x[k][v] * silu_slope(z, gate);
                    o[v] *= z * gate;
                }
            }
            store<DT, VEC>(dx + c, o);
            if (pz) store<DT, VEC>(pz + c, dz[k]);
        }
    }
    float* part = p.part + (long)blockIdx.x * 2 * p.D + c0;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            if constexpr (RPB > 1) {
                __syncthreads();
#pragma unroll
                for (int v = 0; v < VEC; ++v) s_sum[threadIdx.x * VEC + v] = m ? db[k][v] : dw[k][v];
                __syncthreads();
            }
            if (sub == 0 && Grp::col(k) < p.W) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float t = m ? db[k][v] : dw[k][v];
                    if constexpr (RPB > 1) {
#pragma unroll
                        for (int y = 1; y < RPB; ++y) t += s_sum[(y * TPR + threadIdx.x) * VEC + v];
                    }
                    part[m * (long)p.D + Grp::col(k) + v] = t;
                }
            }
        }
}

__global__ __launch_bounds__(256) void k_norm_sums(NormParams p) {
    const long D = p.D;
    column_sums(p.part, 2 * D, p.nblk, (long)blockIdx.x * 64, 2 * D, [&](long col, float s) {
        if (col < D) p.dw[col] = s;
        else if (p.db) p.db[col - D] = s;
    });
}

// ---------------------------------------------------------------- host side
// Threads of a group: the fewest lanes that take it in one access each, up to a wave; a wave takes four
// accesses a thread (its sums need no LDS), wider groups a block.
template <int DT, int VEC, class F> mimo_status with_shape(int W, F f) {
    const int nv = (W + VEC - 1) / VEC;
    if (nv <= 8) return f.template operator()<DT, VEC, 8, 1>();
    if (nv <= 16) return f.template operator()<DT, VEC, 16, 1>();
    if (nv <= 32) return f.template operator()<DT, VEC, 32, 1>();
    if (nv <= 64) return f.template operator()<DT, VEC, 64, 1>();
    if (nv <= 128) return f.template operator()<DT, VEC, 64, 2>();
    if (nv <= 256) return f.template operator()<DT, VEC, 64, 4>();
    if (nv <= 512) return f.template operator()<DT, VEC, 256, 2>();
    if (VEC == 8 || nv <= 1024) return f.template operator()<DT, VEC, 256, 4>();
    if constexpr (VEC <= 4) {
        if (VEC == 4 || nv <= 2048) return f.template operator()<DT, VEC, 256, 8>();
        if constexpr (VEC == 1) return f.template operator()<DT, VEC, 256, 32>();
    }
    return unsupported("group too wide");
}
template <class F> mimo_status dispatch(int dtype, bool even, int W, F f) {
    if (dtype == BF16) return even ? with_shape<BF16, 8>(W, f) : with_shape<BF16, 1>(W, f);
    if (dtype == F16) return even ? with_shape<F16, 8>(W, f) : with_shape<F16, 1>(W, f);
    return even ? with_shape<F32, 4>(W, f) : with_shape<F32, 1>(W, f);
}

mimo_status check_norm(int64_t rows, int64_t D, int64_t G, int dtype, float eps, const void* z, int after, int silu) {
    if (rows < 1 || D < 1 || G < 1) return bad("rows, channels and groups must be positive");
    if (dtype < BF16 || dtype > F32) return set_error(MIMO_ERR_TYPE, "dtype must be a MIMO_DTYPE_* code");
    if (D % G) return bad("the channels must be divisible by the groups");
    if (!(eps >= 0.f)) return bad("eps must not be negative");
    if (silu && z) return bad("silu and a gate z exclude each other");
    if (D / G > MAMBA_NORM_MAX_WIDTH) return unsupported("more than 8192 channels in a group");
    if (G > 65535 || D > (int64_t)1 << 20) return unsupported("more than 65535 groups or 2^20 channels");
    if (rows > (int64_t)1 << 36) return unsupported("too many rows");
    return MIMO_OK;
}

struct FwdRun {
    NormParams p;
    hipStream_t st;
    template <int DT, int VEC, int TPR, int IT> mimo_status operator()() {
        const long per = 256 / TPR, blocks = (p.rows * p.G + per - 1) / per;
        if (blocks > 0x7fffffffL) return unsupported("too many rows");
        return launch(&k_norm_fwd<DT, VEC, TPR, IT>, dim3((unsigned)blocks), 256, 0, st, p);
    }
};
struct BwdRun {
    NormParams p;
    hipStream_t st;
    template <int DT, int VEC, int TPR, int IT> mimo_status operator()() {
        const mimo_status s = launch(&k_norm_bwd<DT, VEC, TPR, IT>, dim3(p.nblk, p.G), 256, 0, st, p);
        if (s != MIMO_OK) return s;
        return launch(&k_norm_sums, dim3((unsigned)((2L * p.D + 63) / 64)), 256, 0, st, p);
    }
};

// blocks of a group: about 1024 blocks in all, none without a row of its own
int64_t bwd_blocks(const mamba_norm_bwd_args* a) {
    const int64_t want = 1024 / a->G < 1 ? 1 : 1024 / a->G;
    return a->rows < want ? a->rows : want;
}

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_norm_fwd(const mamba_norm_fwd_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_norm(a->rows, a->D, a->G, a->dtype, a->eps, a->z, a->gate_after, a->silu);
    if (s != MIMO_OK) return s;
    if (!a->x || !a->weight || !a->out) return bad("x, weight and out must not be NULL");
    NormParams p{};
    p.rows = a->rows, p.D = (int)a->D, p.G = (int)a->G, p.W = p.D / p.G;
    p.xs = a->x_stride, p.zs = a->z_stride;
    p.center = a->center, p.after = a->gate_after, p.silu = a->silu, p.has_z = a->z != nullptr, p.eps = a->eps;
    p.x = a->x, p.z = a->z, p.w = a->weight, p.b = a->bias, p.out = a->out;
    const int esz = a->dtype == F32 ? 4 : 2;
    const bool even = p.W % (16 / esz) == 0 && aligned(a->x, a->x_stride, 0, 16, esz) && aligned(a->z, a->z ? a->z_stride : 0, 0, 16, esz) &&
                      aligned(a->out, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, even, p.W, FwdRun{p, static_cast<hipStream_t>(stream)});
}

mimo_status mamba_norm_bwd_workspace_size(const mamba_norm_bwd_args* a, size_t* bytes) {
    if (a == nullptr) return bad("args must not be NULL");
    const mimo_status s = check_norm(a->rows, a->D, a->G, a->dtype, a->eps, a->z, a->gate_after, a->silu);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = up256((size_t)bwd_blocks(a) * 2 * a->D * sizeof(float));
    return MIMO_OK;
}

mimo_status mamba_norm_bwd(const mamba_norm_bwd_args* a, void* stream) {
    size_t need = 0;
    mimo_status s = mamba_norm_bwd_workspace_size(a, &need);
    if (s != MIMO_OK) return s;
    if (!a->dout || !a->x || !a->weight || !a->dx || !a->dweight) return bad("dout, x, weight, dx and dweight must not be NULL");
    if ((a->z == nullptr) != (a->dz == nullptr)) return bad("dz must be given exactly when z is given");
    if ((a->bias == nullptr) != (a->dbias == nullptr)) return bad("dbias must be given exactly when bias is given");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != MIMO_OK) return s;
    NormParams p{};
    p.rows = a->rows, p.D = (int)a->D, p.G = (int)a->G, p.W = p.D / p.G;
    p.xs = a->x_stride, p.zs = a->z_stride, p.gs = a->dout_stride;
    p.center = a->center, p.after = a->gate_after, p.silu = a->silu, p.has_z = a->z != nullptr, p.eps = a->eps;
    p.x = a->x, p.z = a->z, p.dout = a->dout, p.w = a->weight, p.b = a->bias;
    p.out = a->dx, p.dz = a->dz, p.part = static_cast<float*>(a->workspace), p.dw = a->dweight, p.db = a->dbias;
    p.nblk = (int)bwd_blocks(a);
    const int esz = a->dtype == F32 ? 4 : 2;
    bool even = p.W % (16 / esz) == 0 && aligned(a->x, a->x_stride, 0, 16, esz) && aligned(a->dout, a->dout_stride, 0, 16, esz) &&
                aligned(a->z, a->z ? a->z_stride : 0, 0, 16, esz);
    even = even && aligned(a->dx, 0, 0, 16, 1) && aligned(a->dz, 0, 0, 16, 1);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, even, p.W, BwdRun{p, static_cast<hipStream_t>(stream)});
}

}  // extern "C"
