// Gated group norm over the channels of a row, forward and backward.
//
//   v = x silu(z) (gate before) or x;  m = mean(v) or 0;  r = 1 / sqrt(mean((v - m)^2) + eps)
//   hat = (v - m) r;  p = hat w + b;   out = p silu(z) (gate after), silu(p), or p
//   backward: dp from dout;  dw = sum dp hat;  db = sum dp;  q = dp w;
//             dv = r (q - [mean(q)] - hat mean(q hat)), then through the gate
//
// TPR threads share a group of a row and keep it in registers (IT accesses of VEC elements each, up to
// 16 bytes), so every input is read once: memory binds ([8192, 2048] bf16 with z: in 8 groups forward 18.3 us, 5.5 TB/s, backward
// 36.4 us, 4.6 TB/s, in one group backward 42.7 us). Parameters are loaded before the sums, and nothing in an element's loop
// branches: with one load a parameter and branches inside, the forward pass took 39 us. Sums run over
// lanes; groups that need more than a wave join the waves' sums in LDS. The variance is taken from the
// centred values, not from a difference of sums.
// The backward pass gives each block one group and every nth row, keeps the sums for dw and db in
// registers over the rows, and leaves one partial row a block, added up in order by k_norm_sums.
#include "layer.hpp"

namespace mimo {
namespace layer {
namespace {

// what becomes of the normalised p, or of x: nothing, x silu(z), p silu(z), silu(p)
enum { PLAIN, BEFORE, AFTER, SILU };

struct NormParams {
    long rows, xs, zs, gs;          // row strides of x, z, dout
    int D, G, W;                    // channels, groups, channels of a group
    int center, mode;
    float eps, inv;                 // inv: 1 / W
    const void *x, *z, *dout;
    const float *w, *b;
    void *out, *dz;                 // out: also dx
    float *part, *dw, *db;          // part: [blocks][2][D]
    int nblk;
};

constexpr int threads_of(int TPR) { return TPR < 256 ? 256 : TPR; }

// the sum over the TPR threads of a group, in all of them; `s`: LDS of a float a wave, safe to use again after
// the next call on another one
template <int TPR> __device__ __forceinline__ float sum_group(float x, float* s) {
    if constexpr (TPR <= 64) return sum_wave<TPR>(x);
    else {
        x = sum_wave<64>(x);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        const int first = threadIdx.x / TPR * (TPR / 64);
        x = 0.f;
#pragma unroll
        for (int k = 0; k < TPR / 64; ++k) x += s[first + k];
        return x;
    }
}

template <int DT, int VEC, int TPR, int IT> struct Group {
    typedef raw_t<DT> raw;
    float x[IT][VEC], z[IT][VEC], hat[IT][VEC];
    float r;
    __device__ __forceinline__ static int col(int k) { return (threadIdx.x % TPR + k * TPR) * VEC; }
    // elements col(k) of row data at p; zeros past the group once unpacked
    struct Raw {
        Pack<DT, VEC> t[IT];
    };
    __device__ __forceinline__ static Raw fetch(const raw* p, int W) {
        Raw r;
#pragma unroll
        for (int k = 0; k < IT; ++k)
            if (col(k) < W) r.t[k] = load<DT, VEC>(p + col(k));
        return r;
    }
    __device__ __forceinline__ static void read(const Raw& r, int W, float (&x)[IT][VEC]) {
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            if (col(k) < W) unpack<DT, VEC>(r.t[k], x[k]);
            else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[k][v] = 0.f;
            }
        }
    }
    // the same of an fp32 parameter (NULL: zeros)
    __device__ __forceinline__ static void param(const float* p, int W, float (&x)[IT][VEC]) {
        constexpr int V = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; v += V) {
                Pack<F32, V> t;
                if (p != nullptr && col(k) < W) t = load<F32, V>(p + col(k) + v);
                else {
#pragma unroll
                    for (int i = 0; i < V; ++i) t.v[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) x[k][v + i] = t.v[i];
            }
    }
    __device__ __forceinline__ void normalise(const NormParams& p, float (*s)[16]) {
        const float inv = p.inv;
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) hat[k][v] = x[k][v];
        if (p.mode == BEFORE) {
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) hat[k][v] *= z[k][v] * sigmoid(z[k][v]);
        }
        if (p.center) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) m += hat[k][v];
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

template <int DT, int VEC, int TPR, int IT> __global__ __launch_bounds__(threads_of(TPR)) void k_norm_fwd(NormParams p) {
    typedef raw_t<DT> raw;
    typedef Group<DT, VEC, TPR, IT> Grp;
    __shared__ float s[2][16];
    const unsigned item = (blockIdx.y * gridDim.x + blockIdx.x) * (threads_of(TPR) / TPR) + threadIdx.x / TPR;
    const bool act = item < (unsigned)p.rows * (unsigned)p.G;
    const unsigned in = act ? item / (unsigned)p.G : 0;
    const long row = in;
    const int c0 = act ? (int)(item - in * (unsigned)p.G) * p.W : 0;
    Grp g;
    const auto rx = Grp::fetch(static_cast<const raw*>(p.x) + row * p.xs + c0, p.W);
    typename Grp::Raw rz;
    if (p.z) rz = Grp::fetch(static_cast<const raw*>(p.z) + row * p.zs + c0, p.W);
    float w[IT][VEC], b[IT][VEC];
    Grp::param(p.w + c0, p.W, w);
    Grp::param(p.b ? p.b + c0 : nullptr, p.W, b);
    Grp::read(rx, p.W, g.x);
    if (p.z) Grp::read(rz, p.W, g.z);
    g.normalise(p, s);
    if (!act) return;
    raw* out = static_cast<raw*>(p.out) + row * p.D + c0;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = Grp::col(k);
        if (c >= p.W) continue;
        float y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = __builtin_fmaf(g.hat[k][v], w[k][v], b[k][v]);
        if (p.mode == AFTER) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) y[v] *= g.z[k][v] * sigmoid(g.z[k][v]);
        } else if (p.mode == SILU) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) y[v] *= sigmoid(y[v]);
        }
        store<DT, VEC>(out + c, y);
    }
}

template <int DT, int VEC, int TPR, int IT> __global__ __launch_bounds__(threads_of(TPR)) void k_norm_bwd(NormParams p) {
    typedef raw_t<DT> raw;
    typedef Group<DT, VEC, TPR, IT> Grp;
    constexpr int RPB = threads_of(TPR) / TPR;
    __shared__ float s[4][16];
    __shared__ float s_sum[RPB > 1 ? 256 * VEC : 1];
    const int sub = threadIdx.x / TPR, c0 = blockIdx.y * p.W;
    const float inv = p.inv;
    float w[IT][VEC], b[IT][VEC], dw[IT][VEC] = {}, db[IT][VEC] = {};
    Grp::param(p.w + c0, p.W, w);
    Grp::param(p.b ? p.b + c0 : nullptr, p.W, b);
    // the next row's loads are in flight during a row, with 16-bit types: [8192, 2048] bf16, one group, 42.7 us instead of 43.4,
    // [4100, 4096] fp16 46.8 instead of 48.0, but [4100, 2048] fp32 39.3 instead of 36.7
    constexpr bool AHEAD = DT != F32;
    typename Grp::Raw rx, rz, rd;
    auto fetch = [&](long row) {
        row = row < p.rows ? row : p.rows - 1;
        rx = Grp::fetch(static_cast<const raw*>(p.x) + row * p.xs + c0, p.W);
        if (p.z) rz = Grp::fetch(static_cast<const raw*>(p.z) + row * p.zs + c0, p.W);
        rd = Grp::fetch(static_cast<const raw*>(p.dout) + row * p.gs + c0, p.W);
    };
    const long step = (long)gridDim.x * RPB;
    if (AHEAD) fetch((long)blockIdx.x * RPB + sub);
    for (long row0 = (long)blockIdx.x * RPB; row0 < p.rows; row0 += step) {
        const bool act = row0 + sub < p.rows;
        const long row = act ? row0 + sub : p.rows - 1;
        Grp g;
        float dy[IT][VEC];
        if (!AHEAD) fetch(row);
        Grp::read(rx, p.W, g.x);
        if (p.z) Grp::read(rz, p.W, g.z);
        Grp::read(rd, p.W, dy);
        if (AHEAD && row0 + step < p.rows) fetch(row0 + step + sub);
        g.normalise(p, s);
        float dz[IT][VEC], m1 = 0.f, m2 = 0.f;
        if (p.mode == AFTER) {
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float z = g.z[k][v], gate = sigmoid(z);
                    dz[k][v] = dy[k][v] * __builtin_fmaf(g.hat[k][v], w[k][v], b[k][v]) * silu_slope(z, gate);
                    dy[k][v] *= z * gate;
                }
        } else if (p.mode == SILU) {
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float t = __builtin_fmaf(g.hat[k][v], w[k][v], b[k][v]);
                    dy[k][v] *= silu_slope(t, sigmoid(t));
                }
        }
        if (!act) {
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) dy[k][v] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hat = g.hat[k][v];
                dw[k][v] = __builtin_fmaf(dy[k][v], hat, dw[k][v]);
                db[k][v] += dy[k][v];
                dy[k][v] *= w[k][v];
                m1 += dy[k][v];
                m2 = __builtin_fmaf(dy[k][v], hat, m2);
            }
        m1 = p.center ? sum_group<TPR>(m1, s[2]) * inv : 0.f;
        m2 = sum_group<TPR>(m2, s[3]) * inv;
        raw* dx = static_cast<raw*>(p.out) + row * p.D + c0;
        raw* pz = p.z ? static_cast<raw*>(p.dz) + row * p.D + c0 : nullptr;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = Grp::col(k);
            if (!act || c >= p.W) continue;
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] = g.r * (dy[k][v] - m1 - g.hat[k][v] * m2);
            if (p.mode == BEFORE) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
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
    column_sums(p.part, 2 * D, p.nblk, (long)blockIdx.x * SUM_COLS, 2 * D, [&](long col, float s) {
        if (col < D) p.dw[col] = s;
        else if (p.db) p.db[col - D] = s;
    });
}

// ---------------------------------------------------------------- host side
// Threads of a group: one access each where 1024 threads allow it (a group's values cost a thread about
// a hundred registers an access in the backward pass), in whole waves beyond 32. 1024 threads leave a thread 128 registers: the
// backward pass in 16-bit types keeps 8 of its values in scratch memory with one access (fp16, groups over 4096 wide), 19 to
// 23 with eight of one element each (groups over 2048 wide that are odd or not aligned).
template <int DT, int VEC, class F> mimo_status with_shape(int W, F f) {
    const int nv = (W + VEC - 1) / VEC;
    if (nv <= 8) return f.template operator()<DT, VEC, 8, 1>();
    if (nv <= 16) return f.template operator()<DT, VEC, 16, 1>();
    if (nv <= 32) return f.template operator()<DT, VEC, 32, 1>();
    if (nv <= 64) return f.template operator()<DT, VEC, 64, 1>();
    if (nv <= 128) return f.template operator()<DT, VEC, 128, 1>();
    if (nv <= 256) return f.template operator()<DT, VEC, 256, 1>();
    if (nv <= 512) return f.template operator()<DT, VEC, 512, 1>();
    if (VEC == 8 || nv <= 1024) return f.template operator()<DT, VEC, 1024, 1>();
    if constexpr (VEC <= 4) {
        if (VEC == 4 || nv <= 2048) return f.template operator()<DT, VEC, 1024, 2>();
        if constexpr (VEC == 1) return f.template operator()<DT, VEC, 1024, 8>();
    }
    return unsupported("group too wide");
}
int lanes_of(int W, int VEC) {
    const int nv = (W + VEC - 1) / VEC;
    int t = 8;
    while (t < nv && t < 1024) t *= 2;
    return t;
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
    if (rows > (int64_t)1 << 31) return unsupported("more than 2^31 rows");
    if (G > 65535 || D > (int64_t)1 << 20) return unsupported("more than 65535 groups or 2^20 channels");
    if (rows * G > (int64_t)1 << 31) return unsupported("more than 2^31 groups of rows");
    return MIMO_OK;
}

struct FwdRun {
    NormParams p;
    hipStream_t st;
    template <int DT, int VEC, int TPR, int IT> mimo_status operator()() {
        // in more than one row of blocks where they are too many for one; rows * G + a row of blocks is below 2^32
        const long per = threads_of(TPR) / TPR, blocks = (p.rows * p.G + per - 1) / per, most = 0xffffffffL / threads_of(TPR);
        const long along = blocks < most ? blocks : most;
        return launch(&k_norm_fwd<DT, VEC, TPR, IT>, dim3((unsigned)along, (unsigned)((blocks + along - 1) / along)), threads_of(TPR), 0, st, p);
    }
};
struct BwdRun {
    NormParams p;
    hipStream_t st;
    template <int DT, int VEC, int TPR, int IT> mimo_status operator()() {
        const mimo_status s = launch(&k_norm_bwd<DT, VEC, TPR, IT>, dim3(p.nblk, p.G), threads_of(TPR), 0, st, p);
        if (s != MIMO_OK) return s;
        return launch(&k_norm_sums, dim3((unsigned)((2L * p.D + SUM_COLS - 1) / SUM_COLS)), 256, 0, st, p);
    }
};

bool even_of(const mamba_norm_bwd_args* a) {
    const int esz = a->dtype == F32 ? 4 : 2;
    bool even = a->D / a->G % (16 / esz) == 0 && aligned(a->x, a->x_stride, 0, 16, esz) && aligned(a->dout, a->dout_stride, 0, 16, esz) &&
                aligned(a->z, a->z ? a->z_stride : 0, 0, 16, esz);
    for (const void* x : {(const void*)a->dx, (const void*)a->dz, (const void*)a->weight, (const void*)a->bias}) even = even && aligned(x, 0, 0, 16, 1);
    return even;
}

// blocks of a group: 1024 threads a CU in all, none without a row of its own
int64_t bwd_blocks(const mamba_norm_bwd_args* a) {
    const int lanes = lanes_of((int)(a->D / a->G), !even_of(a) ? 1 : a->dtype == F32 ? 4 : 8), threads = threads_of(lanes);
    int64_t want = 256 * 1024 / threads / a->G;
    want = want < 1 ? 1 : want;
    const int64_t have = (a->rows + threads / lanes - 1) / (threads / lanes);
    return have < want ? have : want;
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
    p.center = a->center, p.mode = a->z ? (a->gate_after ? AFTER : BEFORE) : a->silu ? SILU : PLAIN;
    p.eps = a->eps, p.inv = 1.f / (float)p.W;
    p.x = a->x, p.z = a->z, p.w = a->weight, p.b = a->bias, p.out = a->out;
    const int esz = a->dtype == F32 ? 4 : 2;
    const bool even = p.W % (16 / esz) == 0 && aligned(a->x, a->x_stride, 0, 16, esz) && aligned(a->z, a->z ? a->z_stride : 0, 0, 16, esz) &&
                      aligned(a->out, 0, 0, 16, 1) && aligned(a->weight, 0, 0, 16, 1) && aligned(a->bias, 0, 0, 16, 1);
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
    p.center = a->center, p.mode = a->z ? (a->gate_after ? AFTER : BEFORE) : a->silu ? SILU : PLAIN;
    p.eps = a->eps, p.inv = 1.f / (float)p.W;
    p.x = a->x, p.z = a->z, p.dout = a->dout, p.w = a->weight, p.b = a->bias;
    p.out = a->dx, p.dz = a->dz, p.part = static_cast<float*>(a->workspace), p.dw = a->dweight, p.db = a->dbias;
    p.nblk = (int)bwd_blocks(a);
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, even_of(a), p.W, BwdRun{p, static_cast<hipStream_t>(stream)});
}

}  // extern "C"
