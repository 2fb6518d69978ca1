// Short causal convolution over channels-last sequences: forward, backward, one token.
//
//   pre[t] = bias + sum_k w[k] e[t + k],  out = silu(pre) or pre,  e = (W - 1 rows of state, x)
//   dpre = dout * silu'(pre);  dx[t] = sum_k w[k] dpre[t + W-1 - k];  dw[k] = sum_t dpre[t] e[t + k]
//
// A thread owns two neighbouring channels over one chunk of CH tokens and slides the window through
// registers, so a token of x is read once and W - 1 rows more at each chunk's start. Memory binds.
// Two channels a thread and many threads beat wider accesses, whose windows cost the registers that
// keep waves, and so loads, in flight: [8192, 2048] bf16 forward 18.5 us with eight channels, 17.1 with
// four, 16.1 with two; [4, 4100, 2048] bf16 backward 156, 60 and 57 us. With scalar rows and the blocks' order
// below, 15.4 us (4.4 TB/s; 14.3 of them the kernel) and 50 us (4.0); 8 x 8192 x 2048 forward 104 us (5.2 TB/s, as a copy).
#include "layer.hpp"

namespace mimo {
namespace layer {
namespace {

constexpr int UNROLL = 8;   // rows of loads in flight in a thread (forward)
constexpr int UNROLL_B = 4; // backward (twice that for one channel): two streams, the windows of both in registers

struct ConvParams {
    Seqs q;
    int D, nvec, silu, zero_tail;
    long slots;
    unsigned tiles;                 // blocks along the channels
    Rows x, dout;
    const float *w, *bias;
    const void *init, *dstate;
    void *out, *state, *dinit;      // out: also dx
    float* part;                    // backward: [groups][W + 1][D]
    float *dw, *db;
    int groups;
};

template <int VEC, int W> struct Filter {
    float w[W][VEC], bias[VEC];
    __device__ __forceinline__ Filter(const float* pw, const float* pb, int d) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            bias[v] = pb ? pb[d + v] : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][v] = pw[(long)(d + v) * W + k];
        }
    }
};

// row t of x, or of the state in front of it where t < 0
template <int DT, int VEC, int W>
__device__ __forceinline__ void row_before(const raw_t<DT>* x, long ts, const raw_t<DT>* init, long D, int t, unsigned d, float (&e)[VEC]) {
    if (t >= 0) unpack<DT, VEC>(load<DT, VEC>(x + t * ts + d), e);
    else if (init != nullptr) unpack<DT, VEC>(load<DT, VEC>(init + (t + W - 1) * D + d), e);
    else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = 0.f;
    }
}

// A wave takes one chunk (slot) and 64 channel vectors, so places, row addresses and conditions on tokens are
// scalar. Blocks of one chunk follow each other, so that the blocks in flight read whole rows: with the chunks
// following each other, 8 x 8192 x 2048 bf16 forward took 141 us instead of 107.
template <int DT, int VEC, int W> __global__ __launch_bounds__(256) void k_conv_fwd(ConvParams p) {
    typedef raw_t<DT> raw;
    const unsigned slot = blockIdx.x / p.tiles, tile = blockIdx.x - slot * p.tiles;
    const Place pl = place(p.q, slot);
    if (!pl.ok) return;
    const int vec = tile * blockDim.x + threadIdx.x;
    if (vec >= p.nvec) return;
    const unsigned d = vec * VEC;
    const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
    const long D = p.D;
    raw* out = static_cast<raw*>(p.out) + (p.q.cu ? (long)pl.row0 : (long)pl.i * p.q.S) * D;
    if (pl.i == p.q.n) {            // behind the last sequence
        const float zero[VEC] = {};
        if (p.zero_tail)
            for (int t = t0; t < t1; ++t) store<DT, VEC>(out + t * D + d, zero);
        return;
    }
    const raw* x = at<DT>(p.x, pl);
    const long ts = p.x.ts;
    const raw* init = p.init ? static_cast<const raw*>(p.init) + (long)pl.i * (W - 1) * D : nullptr;
    const Filter<VEC, W> f(p.w, p.bias, d);
    float e[W - 1 + UNROLL][VEC];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row_before<DT, VEC, W>(x, ts, init, D, t0 - (W - 1) + k, d, e[k]);
    for (int t = t0; t < t1; t += UNROLL) {
        Pack<DT, VEC> r[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) r[u] = load<DT, VEC>(x + (long)min(t + u, t1 - 1) * ts + d);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) unpack<DT, VEC>(r[u], e[W - 1 + u]);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            float y[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float s = f.bias[v];
#pragma unroll
                for (int k = 0; k < W; ++k) s = __builtin_fmaf(f.w[k][v], e[u + k][v], s);
                y[v] = p.silu ? s * sigmoid(s) : s;
            }
            if (t + u < t1) store<DT, VEC>(out + (t + u) * D + d, y);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) e[k][v] = e[UNROLL + k][v];
    }
    if (p.state != nullptr && t1 == pl.len) {
        raw* state = static_cast<raw*>(p.state) + (long)pl.i * (W - 1) * D + d;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float s[VEC];
            row_before<DT, VEC, W>(x, ts, init, D, pl.len - (W - 1) + k, d, s);
            store<DT, VEC>(state + k * D, s);
        }
    }
}

// Backward. A wave walks s over its chunk and W - 1 tokens more: dpre[s] from the window of x, then
// dx[s - (W-1)] from the window of dpre. In a sequence's first chunk the rows in front of token 0 are those of
// the state. The sums for dw and db stay in registers, are joined over the block's slots in LDS and leave one
// partial row for each block, which k_conv_sums adds up in order (no atomics). A block takes WS neighbouring slots of 64 channel vectors.
constexpr int WS = 4;
template <int DT, int VEC, int W> __global__ __launch_bounds__(64 * WS) void k_conv_bwd(ConvParams p) {
    typedef raw_t<DT> raw;
    constexpr int U = UNROLL_B * (3 - VEC);
    constexpr int TC = 64;
    __shared__ float s_sum[WS][TC * VEC];
    const int tx = threadIdx.x % TC, ty = __builtin_amdgcn_readfirstlane(threadIdx.x / TC);
    const unsigned group = blockIdx.x / p.tiles, tile = blockIdx.x - group * p.tiles;
    const int vec = tile * TC + tx;
    const unsigned d = vec * VEC;
    const long slot = (long)group * WS + ty, D = p.D;
    float acc[W + 1][VEC] = {};
    Place pl = {};
    if (slot < p.slots) pl = place(p.q, (int)slot);
    if (pl.ok && vec < p.nvec) {
        const int t0 = pl.j * p.q.CH, t1 = min(t0 + p.q.CH, pl.len);
        raw* dx = static_cast<raw*>(p.out) + (p.q.cu ? (long)pl.row0 : (long)pl.i * p.q.S) * D;
        if (pl.i == p.q.n) {
            const float zero[VEC] = {};
            for (int t = t0; t < t1; ++t) store<DT, VEC>(dx + t * D + d, zero);
        } else {
            const raw *x = at<DT>(p.x, pl), *dout = at<DT>(p.dout, pl);
            const long xs = p.x.ts, gs = p.dout.ts, sd = (long)pl.i * (W - 1) * D;
            const raw* init = p.init ? static_cast<const raw*>(p.init) + sd : nullptr;
            const raw* dstate = p.dstate ? static_cast<const raw*>(p.dstate) + sd : nullptr;
            raw* dinit = p.dinit ? static_cast<raw*>(p.dinit) + sd : nullptr;
            const Filter<VEC, W> f(p.w, p.bias, d);
            float e[W - 1 + U][VEC], g[W - 1 + U][VEC];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                row_before<DT, VEC, W>(x, xs, init, D, t0 - (W - 1) + k, d, e[k]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) g[k][v] = 0.f;
            }
            const int s1 = t1 + W - 1;   // dx up to t1 - 1
            for (int s = t0; s < s1; s += U) {
                Pack<DT, VEC> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long t = max(min(s + u, pl.len - 1), 0);
                    if (pl.len > 0) {
                        rx[u] = load<DT, VEC>(x + t * xs + d);
                        rg[u] = load<DT, VEC>(dout + t * gs + d);
                    } else {
                        rx[u] = Pack<DT, VEC>{};
                        rg[u] = Pack<DT, VEC>{};
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    unpack<DT, VEC>(rx[u], e[W - 1 + u]);
                    unpack<DT, VEC>(rg[u], g[W - 1 + u]);
                    if (s + u >= pl.len) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) g[W - 1 + u][v] = 0.f;
                    } else if (p.silu) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            float pre = f.bias[v];
#pragma unroll
                            for (int k = 0; k < W; ++k) pre = __builtin_fmaf(f.w[k][v], e[u + k][v], pre);
                            g[W - 1 + u][v] *= silu_slope(pre, sigmoid(pre));
                        }
                    }
                    if (s + u < t1) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            const float dp = g[W - 1 + u][v];
#pragma unroll
                            for (int k = 0; k < W; ++k) acc[k][v] = __builtin_fmaf(dp, e[u + k][v], acc[k][v]);
                            acc[W][v] += dp;
                        }
                    }
                    const int t = s + u - (W - 1);
                    if (s + u < s1 && (t >= t0 || pl.j == 0)) {
                        float r[VEC];
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            r[v] = 0.f;
#pragma unroll
                            for (int k = 0; k < W; ++k) r[v] = __builtin_fmaf(f.w[k][v], g[u + W - 1 - k][v], r[v]);
                        }
                        const int k = t - (pl.len - (W - 1));   // this row's place in the last state
                        if (dstate != nullptr && k >= 0) {
                            float a[VEC];
                            unpack<DT, VEC>(load<DT, VEC>(dstate + k * D + d), a);
#pragma unroll
                            for (int v = 0; v < VEC; ++v) r[v] += a[v];
                        }
                        if (t >= 0) store<DT, VEC>(dx + t * D + d, r);
                        else if (dinit != nullptr) store<DT, VEC>(dinit + (t + W - 1) * D + d, r);
                    }
                }
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        e[k][v] = e[U + k][v];
                        g[k][v] = g[U + k][v];
                    }
            }
        }
    }
    float* part = p.part + (long)group * (W + 1) * D;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) s_sum[ty][tx * VEC + v] = acc[k][v];
        __syncthreads();
        if (threadIdx.x < TC * VEC) {
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < WS; ++y) s += s_sum[y][threadIdx.x];
            const long col = (long)tile * TC * VEC + threadIdx.x;
            if (col < D) part[k * D + col] = s;
        }
        __syncthreads();
    }
}

template <int W> __global__ __launch_bounds__(256) void k_conv_sums(ConvParams p) {
    const long D = p.D;
    column_sums(p.part, (W + 1) * D, p.groups, (long)blockIdx.x * SUM_COLS, (W + 1) * D, [&](long col, float s) {
        const int k = (int)(col / D);
        const long d = col - k * D;
        if (k < W) p.dw[d * W + k] = s;
        else if (p.db != nullptr) p.db[d] = s;
    });
}

struct StepParams {
    int n, D, slots, silu;
    long slot_stride, x_stride;
    const void* x;
    void *state, *out;
    const float *w, *bias;
    const int* idx;
};

// One token: a thread takes VEC channels of a row (blockIdx.y), reads its state row and x, writes
// both back shifted. Rows of one slot are taken by the first of them, in order.
template <int DT, int VEC, int W> __global__ __launch_bounds__(256) void k_conv_step(StepParams p) {
    typedef raw_t<DT> raw;
    int row = blockIdx.y;
    const int vec = blockIdx.x * 256 + threadIdx.x, d = vec * VEC;
    const bool act = d < p.D;
    const long D = p.D;
    const int slot = p.idx ? p.idx[row] : row;
    raw* out = static_cast<raw*>(p.out) + d;
    if (slot < 0 || slot >= p.slots) {
        const float zero[VEC] = {};
        if (act) store<DT, VEC>(out + row * D, zero);
        return;
    }
    raw* state = static_cast<raw*>(p.state) + slot * p.slot_stride + d;
    float e[W][VEC] = {};
    const Filter<VEC, W> f(p.w, p.bias, act ? d : 0);
    if (act) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) unpack<DT, VEC>(load<DT, VEC>(state + k * D), e[k]);
    }
    if (p.idx && !first_of(p.idx, row, slot)) return;
    for (;;) {
        if (act) {
            unpack<DT, VEC>(load<DT, VEC>(static_cast<const raw*>(p.x) + row * p.x_stride + d), e[W - 1]);
            float y[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float s = f.bias[v];
#pragma unroll
                for (int k = 0; k < W; ++k) s = __builtin_fmaf(f.w[k][v], e[k][v], s);
                y[v] = p.silu ? s * sigmoid(s) : s;
            }
            store<DT, VEC>(out + row * D, y);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) e[k][v] = e[k + 1][v];
        row = p.idx ? next_of(p.idx, row, p.n, slot) : p.n;
        if (row >= p.n) break;
    }
    if (act) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store<DT, VEC>(state + k * D, e[k]);
    }
}

// ---------------------------------------------------------------- host side
// Tokens of a chunk, 16 at least: longer chunks read fewer rows twice, and the backward pass leaves fewer partial
// sums; shorter ones keep more threads, and so loads, in flight. Forward 2048 threads a CU and up to 32 tokens
// ([8192, 2048] bf16, the same inputs: 14.5 us, 15.9 with 1024 threads; 8 x 8192 x 2048: 104 us at 32 tokens, 115 at 128); backward
// 1024 threads a CU, whose registers allow no more, and up to 128 tokens ([4, 4100, 2048] bf16: 52 us before chunks were
// equal, 55 with 2048;
// 8 x 8192 x 2048: 243 us at 64 tokens, 208 at 128, before the scalar rows).
int chunk_tokens(int64_t n, int64_t S, bool packed, int64_t nvec, bool backward) {
    const int64_t T = packed ? S : n * S, c = T * nvec / (256 * (backward ? 1024 : 2048)) / 8 * 8, most = backward ? 128 : 32;
    return (int)(c < 16 ? 16 : c > most ? most : c);
}

Seqs make_seqs(int64_t n, int64_t S, const int32_t* cu, int CH) {
    return Seqs{cu, (int)n, (int)S, CH, (int)((S + CH - 1) / CH)};
}

mimo_status check_filter(int32_t W, const float* w) {
    if (W < MAMBA_CONV_MIN_TAPS || W > MAMBA_CONV_MAX_TAPS) return unsupported("the filter must have 2 to 8 taps");
    if (w == nullptr) return bad("weight must not be NULL");
    return MIMO_OK;
}

// channels of a thread: two where every row starts at a multiple of both, else one
int vec_of(int64_t D, bool even) { return even && D % 2 == 0 ? 2 : 1; }

template <int DT, int W, class F> mimo_status with_vec(int vec, F f) {
    return vec == 2 ? f.template operator()<DT, 2, W>() : f.template operator()<DT, 1, W>();
}
template <int DT, class F> mimo_status with_taps(int W, int vec, F f) {
    switch (W) {
        case 2: return with_vec<DT, 2>(vec, f);
        case 3: return with_vec<DT, 3>(vec, f);
        case 4: return with_vec<DT, 4>(vec, f);
        case 5: return with_vec<DT, 5>(vec, f);
        case 6: return with_vec<DT, 6>(vec, f);
        case 7: return with_vec<DT, 7>(vec, f);
        default: return with_vec<DT, 8>(vec, f);
    }
}
template <class F> mimo_status dispatch(int dtype, int W, int vec, F f) {
    if (dtype == BF16) return with_taps<BF16>(W, vec, f);
    if (dtype == F16) return with_taps<F16>(W, vec, f);
    return with_taps<F32>(W, vec, f);
}

struct FwdRun {
    ConvParams p;
    hipStream_t st;
    template <int DT, int VEC, int W> mimo_status operator()() {
        const int block = p.nvec >= 256 ? 256 : (p.nvec + 63) / 64 * 64;
        p.tiles = (p.nvec + block - 1) / block;
        if (p.slots * p.tiles > 0x7fffffffL) return unsupported("too many tokens");
        return launch(&k_conv_fwd<DT, VEC, W>, dim3((unsigned)(p.slots * p.tiles)), block, 0, st, p);
    }
};
struct BwdRun {
    ConvParams p;
    hipStream_t st;
    template <int DT, int VEC, int W> mimo_status operator()() {
        p.tiles = (p.nvec + 63) / 64;
        if ((long)p.groups * p.tiles > 0x7fffffffL) return unsupported("too many tokens");
        mimo_status s = launch(&k_conv_bwd<DT, VEC, W>, dim3(p.groups * p.tiles), 64 * WS, 0, st, p);
        if (s != MIMO_OK) return s;
        return launch(&k_conv_sums<W>, dim3((unsigned)(((W + 1) * (long)p.D + SUM_COLS - 1) / SUM_COLS)), 256, 0, st, p);
    }
};
struct StepRun {
    StepParams p;
    hipStream_t st;
    template <int DT, int VEC, int W> mimo_status operator()() {
        const int nvec = p.D / VEC;
        return launch(&k_conv_step<DT, VEC, W>, dim3((nvec + 255) / 256, p.n), 256, 0, st, p);
    }
};

struct BwdPlan {
    int vec, CH, groups;
    size_t bytes;
};
mimo_status plan_bwd(const mamba_conv_bwd_args* a, BwdPlan* pl) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_sequences(a->n, a->S, a->D, a->dtype);
    if (s != MIMO_OK) return s;
    if (a->W < MAMBA_CONV_MIN_TAPS || a->W > MAMBA_CONV_MAX_TAPS) return unsupported("the filter must have 2 to 8 taps");
    const int esz = a->dtype == F32 ? 4 : 2;
    bool even = aligned(a->x.data, a->x.batch_stride, a->x.token_stride, 2 * esz, esz) &&
                aligned(a->dout.data, a->dout.batch_stride, a->dout.token_stride, 2 * esz, esz);
    for (const void* x : {a->initial_state, a->dstate, (const void*)a->dx, (const void*)a->dinitial_state}) even = even && aligned(x, 0, 0, 2 * esz, 1);
    pl->vec = vec_of(a->D, even);
    const bool packed = a->cu_seqlens != nullptr;
    pl->CH = chunk_tokens(a->n, a->S, packed, a->D / pl->vec, true);
    if (packed) {   // a wave walks W - 1 tokens past its chunk: whole unrolled steps ([5003, 517] fp32, W = 3: 14.7 us, 16.7 with 16 tokens)
        const int U = UNROLL_B * (3 - pl->vec), over = (int)a->W - 1;
        pl->CH = (pl->CH + over + U / 2) / U * U - over;
    } else if (a->S > pl->CH) {   // equal chunks (4100 tokens: 48.5 us with 32 chunks of 129 tokens, 52.5 with 33, the last of 4)
        const int64_t count = (a->S + pl->CH / 2) / pl->CH;
        pl->CH = (int)((a->S + count - 1) / count);
    }
    const Seqs q = make_seqs(a->n, a->S, a->cu_seqlens, pl->CH);
    const long groups = (slots_of(q) + WS - 1) / WS;
    if (slots_of(q) > (long)1 << 30) return unsupported("too many tokens");
    pl->groups = (int)groups;
    pl->bytes = up256((size_t)groups * (a->W + 1) * a->D * sizeof(float));
    return MIMO_OK;
}

}  // namespace
}  // namespace layer
}  // namespace mimo

using namespace mimo;
using namespace mimo::layer;

extern "C" {

mimo_status mamba_conv_fwd(const mamba_conv_fwd_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_sequences(a->n, a->S, a->D, a->dtype);
    if (s != MIMO_OK || (s = check_filter(a->W, a->weight)) != MIMO_OK) return s;
    if (!a->x.data || !a->out) return bad("x and out must not be NULL");
    const int esz = a->dtype == F32 ? 4 : 2;
    bool even = aligned(a->x.data, a->x.batch_stride, a->x.token_stride, 2 * esz, esz);
    for (const void* x : {a->initial_state, (const void*)a->out, (const void*)a->state}) even = even && aligned(x, 0, 0, 2 * esz, 1);
    const int vec = vec_of(a->D, even);
    const bool packed = a->cu_seqlens != nullptr;
    ConvParams p{};
    p.D = (int)a->D;
    p.nvec = p.D / vec;
    p.q = make_seqs(a->n, a->S, a->cu_seqlens, chunk_tokens(a->n, a->S, packed, p.nvec, false));
    p.slots = slots_of(p.q);
    if (p.slots > (long)1 << 30) return unsupported("too many tokens");
    p.silu = a->silu;
    p.zero_tail = a->zero_tail;
    p.x = rows_of(a->x, packed);
    p.w = a->weight;
    p.bias = a->bias;
    p.init = a->initial_state;
    p.out = a->out;
    p.state = a->state;
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, a->W, vec, FwdRun{p, static_cast<hipStream_t>(stream)});
}

mimo_status mamba_conv_bwd_workspace_size(const mamba_conv_bwd_args* a, size_t* bytes) {
    BwdPlan pl;
    const mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK) return s;
    if (bytes == nullptr) return bad("bytes must not be NULL");
    *bytes = pl.bytes;
    return MIMO_OK;
}

mimo_status mamba_conv_bwd(const mamba_conv_bwd_args* a, void* stream) {
    BwdPlan pl;
    mimo_status s = plan_bwd(a, &pl);
    if (s != MIMO_OK || (s = check_filter(a->W, a->weight)) != MIMO_OK) return s;
    if (!a->x.data || !a->dout.data || !a->dx || !a->dweight) return bad("dout, x, dx and dweight must not be NULL");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, pl.bytes)) != MIMO_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    ConvParams p{};
    p.D = (int)a->D;
    p.nvec = p.D / pl.vec;
    p.q = make_seqs(a->n, a->S, a->cu_seqlens, pl.CH);
    p.slots = slots_of(p.q);
    p.groups = pl.groups;
    p.silu = a->silu;
    p.x = rows_of(a->x, packed);
    p.dout = rows_of(a->dout, packed);
    p.w = a->weight;
    p.bias = a->bias;
    p.init = a->initial_state;
    p.dstate = a->dstate;
    p.out = a->dx;
    p.dinit = a->dinitial_state;
    p.part = static_cast<float*>(a->workspace);
    p.dw = a->dweight;
    p.db = a->dbias;
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, a->W, pl.vec, BwdRun{p, static_cast<hipStream_t>(stream)});
}

mimo_status mamba_conv_step(const mamba_conv_step_args* a, void* stream) {
    if (a == nullptr) return bad("args must not be NULL");
    mimo_status s = check_sequences(a->n, 1, a->D, a->dtype);
    if (s != MIMO_OK || (s = check_filter(a->W, a->weight)) != MIMO_OK) return s;
    if (!a->x || !a->out || !a->state) return bad("x, state and out must not be NULL");
    if (a->slots < 1 || a->slots > (int64_t)1 << 30) return bad("slots must be in [1, 2^30]");
    if (!a->indices && a->slots < a->n) return bad("without indices the state needs a slot for each row");
    const int esz = a->dtype == F32 ? 4 : 2;
    const bool even = aligned(a->x, a->x_stride, 0, 2 * esz, esz) && aligned(a->state, a->slot_stride, 0, 2 * esz, esz) && aligned(a->out, 0, 0, 2 * esz, 1);
    const StepParams p{(int)a->n, (int)a->D, (int)a->slots, a->silu, (long)a->slot_stride, (long)a->x_stride, a->x, a->state, a->out,
                       a->weight, a->bias, a->indices};
    if ((s = require_gfx950()) != MIMO_OK) return s;
    return dispatch(a->dtype, a->W, vec_of(a->D, even), StepRun{p, static_cast<hipStream_t>(stream)});
}

}  // extern "C"
